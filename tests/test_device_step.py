"""The device-resident decode step as a serving loop runs it: release, reserve,
append, bounds and attention, one captured graph, sequences of different
lengths ending and being replaced; against host loops."""
import numpy as np
import pytest
import torch

import block_reference as R
from paged_kv_cache_273_gb300 import pkv
from test_f8_cache import DEV, DT, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["f8", "bf16"])
def test_captured_serving_loop(kv):
    B, H, G, D, bs, maxb, budget, cap = 6, 2, 4, 128, 16, 12, 4, 64
    nb = B * maxb
    code = {"f8": pkv.PKV_F8, "bf16": pkv.PKV_BF16}[kv]
    pool = pkv.kv_block_pool_init(nb, bs, H, D, code)
    kc, vc, ks, vs = pool.alloc_cache(DEV)
    bounds, exps = pkv.alloc_bounds(pool, DEV)
    ids = pkv.kv_block_alloc(pool, nb)
    free_ids, state = pkv.alloc_device_free_list(ids, DEV)
    free = ids.tolist()
    i32 = dict(dtype=torch.int32, device=DEV)
    lens, tables = torch.zeros(B, **i32), torch.zeros(B, maxb, **i32)
    done, new, slots = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros(cap, **i32)
    k_new, v_new = (torch.zeros(cap, H, D, dtype=DT["bf16"], device=DEV) for _ in range(2))
    q = torch.zeros(B, H * G, D, dtype=DT["bf16"], device=DEV)
    dense, sparse = (torch.zeros(B, H * G, D, device=DEV) for _ in range(2))
    sel = torch.zeros(B, H, budget, **i32)
    ws = pkv.alloc_workspace(pool, B, H * G)
    wss = pkv.alloc_sparse_workspace(pool, B, H * G, maxb * bs, budget)
    scale = 0.08
    torch.cuda.synchronize()

    def step():
        pkv.kv_device_release(pool, free_ids, state, lens, done, tables)
        pkv.kv_device_reserve(pool, free_ids, state, lens, tables, slots, num_new=new)
        pkv.kv_append(pool, k_new, v_new, slots, kc, vc, ks, vs)
        pkv.kv_bounds_append(pool, k_new, slots, bounds, exps)
        pkv.paged_decode_attention(pool, q, kc, vc, tables, lens, scale, dense, ws, maxb * bs, ks,
                                   vs)
        pkv.paged_decode_attention_sparse(pool, q, kc, vc, bounds, exps, tables, lens, scale,
                                          sparse, sel, wss, maxb * bs, ks, vs)

    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        step()
    # host state
    rng = np.random.default_rng(5)
    hl, ht = np.zeros(B, np.int64), np.zeros((B, maxb), np.int32)
    hk, hv = (np.zeros((nb, H, bs, D), np.uint8 if kv == "f8" else np.float64) for _ in range(2))
    hks, hvs = np.zeros((nb, H)), np.zeros((nb, H))
    hb, he = np.zeros((nb, H, 2, D), np.int8), np.zeros((nb, H), np.int32)
    for it in range(14):
        d = (rng.random(B) < 0.2).astype(np.int32)
        n = np.where(rng.random(B) < 0.3, rng.integers(0, 11, B), 1)
        hold = np.where(d != 0, 0, hl)
        n = np.minimum(n, maxb * bs - hold)
        if it == 0:
            n[:] = [20, 1, 0, 16, 9, 15]
        kn, vn = _rows(100 + it, (cap, H, D), "bf16"), _rows(200 + it, (cap, H, D), "bf16", 2.0)
        qq = _rows(300 + it, (B, H * G, D), "bf16", 1.5)
        for dst, src in ((k_new, kn), (v_new, vn), (q, qq), (done, torch.from_numpy(d)),
                         (new, torch.from_numpy(n.astype(np.int32)))):
            dst.copy_(src)
        g.replay()
        for b in np.nonzero(d)[0]:
            free += ht[b, :-(-hl[b] // bs)].tolist()
            hl[b] = 0
        want = R.reserve(free, hl, n, ht, bs)
        assert slots.cpu().tolist() == want + [-1] * (cap - len(want))
        assert lens.cpu().tolist() == hl.tolist() and np.array_equal(tables.cpu().numpy(), ht)
        k64, v64 = kn.double().cpu().numpy()[:len(want)], vn.double().cpu().numpy()[:len(want)]
        R.append_bounds(k64, want, bs, hb, he)
        if kv == "f8":
            R.append_f8(k64, want, bs, hk, hks)
            R.append_f8(v64, want, bs, hv, hvs)
            rk = R.E4M3[hk] * np.maximum(hks, 2.0 ** -96)[:, :, None, None]
            rv = R.E4M3[hv] * np.maximum(hvs, 2.0 ** -96)[:, :, None, None]
        else:
            for t, s in enumerate(want):
                hk[s // bs, :, s % bs], hv[s // bs, :, s % bs] = k64[t], v64[t]
            rk, rv = hk, hv
        assert np.array_equal(exps.cpu().numpy(), he) and np.array_equal(bounds.cpu().numpy(), hb)
        q64 = qq.double().cpu().numpy()
        for b in range(B):
            nblk = -(-hl[b] // bs)
            blocks = ht[b, :nblk]
            for h in range(H):
                gq = q64[b, h * G:(h + 1) * G]
                for out, at in ((dense, np.arange(nblk)),
                                (sparse, R.choose(gq, blocks, hb, he, h, budget)
                                 if nblk else np.arange(0))):
                    m = max(0, len(at) * bs - (nblk * bs - hl[b]))
                    o, tol = R.attend(gq, rk[blocks[at], h].reshape(-1, D)[:m],
                                      rv[blocks[at], h].reshape(-1, D)[:m],
                                      float(np.float32(scale)),
                                      R.BF16_PARTS if kv == "bf16" else 2.0 ** -22)
                    got = out[b, h * G:(h + 1) * G].double().cpu().numpy()
                    assert np.abs(got - o).max() <= tol, (it, b, h)
        assert pkv.pkv_check_error(pool) == pkv.PKV_OK
