"""Rotation, append and attention of new tokens together, as a server runs them: prompts in
pieces, single tokens, drafted trees; from the host's block tables, and captured with the
device's."""
import math

import numpy as np
import pytest
import torch

import test_chunk as C
import test_rope as P
from paged_kv_cache_273_gb300 import pkv

DEV = "cuda"
i32 = C.i32


def _state(kv, hq, H, D, bs, nb, B, maxb, dtype):
    pool = pkv.kv_block_pool_init(nb, bs, H, D, C.KV[kv])
    kc, vc, ks, vs = pool.alloc_cache()
    return dict(pool=pool, kc=kc, vc=vc, ks=ks, vs=vs, hq=hq, H=H, D=D, bs=bs, nb=nb, kv=kv, dtype=dtype,
                tables=np.zeros((B, maxb), np.int32))


def _rows(s, T, seed):
    """q, K and V of T tokens, side by side in one buffer, as one product writes them."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, s["hq"] + 2 * s["H"], s["D"], generator=g) * 1.5).to(C.DT[s["dtype"]]).to(DEV)
    return x[:, :s["hq"]], x[:, s["hq"]:s["hq"] + s["H"]], x[:, s["hq"] + s["H"]:]


def _values(s):
    """The caches as they are, for the float64 attention."""
    for n in "kv":
        x = s[n + "c"].double().cpu()
        s[n] = x * s[n + "s"].double().cpu()[:, :, None, None] if s["kv"] == "f8" else x
    s["bt"] = torch.from_numpy(s["tables"].copy())
    return s


PLANS = {"f16": dict(rot=64, layout="half", scaling="plain"), "bf16": dict(rot=64, layout="interleaved", scaling="wavelength"),
         "f8": dict(rot=128, layout="half", scaling="parts")}


@pytest.mark.gpu
@pytest.mark.parametrize("kv,dtype", [("f16", "f16"), ("bf16", "bf16"), ("f8", "bf16"), ("f8", "f16")])
def test_gpu_prompts_tokens_and_drafts(kv, dtype):
    hq, H, D, bs, B = 8, 2, 128, 16, 3
    s = _state(kv, hq, H, D, bs, 120, B, 32, dtype)
    c = PLANS[kv]
    plan = pkv.rope_plan(c["rot"], layout=c["layout"], scaling=c["scaling"], **P.SCALINGS[c["scaling"]])
    lens = np.zeros(B, np.int32)
    ws = pkv.alloc_chunk_workspace(s["pool"], B, hq, 260)
    raw = [[] for _ in range(B)]
    scale = 1.0 / math.sqrt(D)
    for step, new in enumerate([[40, 0, 260], [1, 200, 7], [1, 1, 1], [5, 64, 2], [3, 1, 0]]):
        tree = C._tree(new, "drafts", step) if step == 3 else None
        slots = pkv.kv_reserve_slots(s["pool"], lens, s["tables"], new)
        T = sum(new)
        q, k, v = _rows(s, T, step)
        # drafted tokens stand where they would on their path: any position will do here
        pos = np.concatenate([np.arange(L, L + n) for L, n in zip(lens, new)])
        q_out = torch.empty(T, hq, D, dtype=q.dtype, device=DEV)
        pkv.kv_rope_append(s["pool"], plan, q, k, v, i32(pos), i32(slots), q_out, s["kc"], s["vc"], s["ks"], s["vs"])
        lens = lens + np.array(new, np.int32)
        start = np.concatenate([[0], np.cumsum(new)]).astype(int)
        for b in range(B):
            raw[b].append(k[start[b]:start[b + 1]].double().cpu().numpy())
        s.update(lens=[int(x) for x in lens], new=list(new), start=start.tolist(), T=T, tree=tree, q=q_out.cpu())
        out = C.run(s, scale, ws=ws, max_q=260, tables=i32(s["tables"]))
        C.check(_values(s), out, scale=scale)
        y, tol = P.turn(q.double().cpu().numpy(), pos, c["rot"], c["layout"], c["scaling"])
        P.close(q_out, y, tol, dtype)
        if kv != "f8":                                 # the cache holds every token's rotated K
            for b in range(B):
                ids = s["tables"][b, :-(-int(lens[b]) // bs)]
                got = s["kc"][torch.from_numpy(ids.astype(np.int64)).to(DEV)].transpose(1, 2).reshape(-1, H, D)[:int(lens[b])]
                y, tol = P.turn(np.concatenate(raw[b]), np.arange(lens[b]), c["rot"], c["layout"], c["scaling"])
                P.close(got, y, tol, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "f8"])
def test_gpu_captured_step(kv):
    """Device reservation, rotation with append, and attention in one captured graph, replayed with
    other token counts (a padded batch among them); two graphs on one workspace."""
    hq, H, D, bs, B, maxb, cap = 4, 2, 64, 16, 4, 16, 96
    s = _state(kv, hq, H, D, bs, 64, B, maxb, "bf16")
    pool = s["pool"]
    plan = pkv.rope_plan(D)
    free_ids = i32(list(range(64)))
    state = i32([64, 0])
    lens, new, start = i32([0] * B), i32([0] * B), i32([0] * (B + 1))
    tables, slots, pos = i32([[0] * maxb] * B), i32([-1] * cap), i32([0] * cap)
    x = torch.zeros(cap, hq + 2 * H, D, dtype=torch.bfloat16, device=DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + H], x[:, hq + H:]
    ws = pkv.alloc_chunk_workspace(pool, B, hq, cap)
    scale = 0.125

    def step(out, q_out):
        pkv.kv_device_reserve(pool, free_ids, state, lens, tables, slots, num_new=new, q_start=start)
        pkv.kv_rope_append(pool, plan, q, k, v, pos, slots, q_out, s["kc"], s["vc"], s["ks"], s["vs"])
        pkv.paged_chunk_attention(pool, q_out, s["kc"], s["vc"], tables, start, lens, scale, out, ws, cap, s["ks"], s["vs"])

    torch.cuda.synchronize()
    graphs, outs, turned = [], [], []
    for _ in range(2):
        outs.append(torch.zeros(cap, hq, D, dtype=torch.bfloat16, device=DEV))
        turned.append(torch.zeros_like(outs[-1]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(outs[-1], turned[-1])
        graphs.append(g)
    now = [0] * B
    for t, n in enumerate([[40, 1, 0, 50], [1, 1, 1, 1], [0, 30, 60, 6], [0, 0, 0, 0], [2, 1, 3, 1]]):
        T = sum(n)
        a, b, c = _rows(s, T, 50 + t)
        x.zero_()
        x[:T] = torch.cat([a, b, c], 1)
        new.copy_(i32(n))
        pos.zero_()
        pos[:T] = i32(np.concatenate([np.arange(L, L + m) for L, m in zip(now, n)]))
        now = [L + m for L, m in zip(now, n)]
        out, q_out = outs[t % 2], turned[t % 2]
        out.fill_(7.0)
        graphs[t % 2].replay()
        torch.cuda.synchronize()
        assert pkv.pkv_check_error(pool) == pkv.PKV_OK and lens.tolist() == now
        assert start.tolist() == [0] + np.cumsum(n).tolist()
        s["tables"] = tables.cpu().numpy()
        s.update(lens=list(now), new=list(n), start=start.tolist(), T=cap, tree=None, q=q_out.cpu())
        C.check(_values(s), out, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "f8"])
def test_gpu_blocks_beyond_4_gib(kv):
    """Rows more than 2^32 bytes into the caches, and blocks that lie before them."""
    hq, H, D, bs, dtype = 8, 8, 128, 64, "bf16"
    nb = 2 ** 32 // (H * bs * D * (1 if kv == "f8" else 2)) + 40
    s = _state(kv, hq, H, D, bs, nb, 2, 4, dtype)
    plan = pkv.rope_plan(D)
    s["tables"][0] = [nb - 1, 3, nb - 17, nb - 2]
    s["tables"][1] = [nb - 5, nb - 30, 0, nb - 3]
    lens = new = [230, 140]
    slots = pkv.kv_slot_mapping(s["tables"], bs, [0, 0], new)
    T = sum(new)
    q, k, v = _rows(s, T, 1)
    pos = np.concatenate([np.arange(n) for n in new])
    q_out = torch.empty(T, hq, D, dtype=q.dtype, device=DEV)
    pkv.kv_rope_append(s["pool"], plan, q, k, v, i32(pos), i32(slots), q_out, s["kc"], s["vc"], s["ks"], s["vs"])
    s.update(lens=lens, new=new, start=[0, 230, 370], T=T, tree=None, q=q_out.cpu())
    out = C.run(s, 0.1, tables=i32(s["tables"]))
    # (the blocks in use only: they stand in the order of the tables)
    ids = torch.from_numpy(s["tables"].reshape(-1).astype(np.int64)).to(DEV)
    r = dict(s, bt=torch.arange(8).reshape(2, 4))
    for n in "kv":
        y = s[n + "c"][ids].double().cpu()
        r[n] = y * s[n + "s"][ids].double().cpu()[:, :, None, None] if kv == "f8" else y
    C.check(r, out, scale=0.1)
    if kv != "f8":
        turned = pkv.kv_rope_rotate(plan, k, i32(pos))
        assert torch.equal(s["kc"][ids[:4]].transpose(1, 2).reshape(-1, H, D)[:230], turned[:230])
