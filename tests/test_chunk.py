"""paged_chunk_attention against float64 attention over rows gathered through the
block tables."""
import ctypes
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_273_gb300 import pkv

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
KV = {"f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16, "f8": pkv.PKV_F8}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


# --------------------------------------------------------------------------- CPU
def _call(pools, a, pool="bf16", q=..., dt=pkv.PKV_BF16, hq=4, T=3, kc=..., vc=..., ks=None, vs=None, bt=..., mb=2, qs=..., sl=..., B=1, mq=3,
          window=0, vis=None, scale=0.125, out=..., ws=..., wsb=1 << 30):
    v = [a if x is ... else x for x in (q, kc, vc, bt, qs, sl, out, ws)]
    q, kc, vc, bt, qs, sl, out, ws = v
    return pkv.load().paged_chunk_attention(None if pool is None else pools[pool].handle, q, dt, hq, T, kc, vc, ks, vs, bt, mb, qs, sl, B, mq, window,
                                            vis, scale, out, ws, wsb, None)


def test_refusals():
    buf = (ctypes.c_uint8 * 4096)()
    a = (ctypes.addressof(buf) + 15) // 16 * 16
    inv, uns = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED
    pools = {k: pkv.kv_block_pool_init(8, 16, 2, 64, t) for k, t in
             dict(KV, f32=pkv.PKV_F32, i8=pkv.PKV_I8).items()}
    pools["i4"] = pkv.kv_block_pool_init(8, 16, 2, 128, pkv.PKV_I4)

    def call(**kw):
        return _call(pools, a, **kw)
    assert call(pool=None) == inv and call(hq=3) == inv and call(hq=0) == inv
    assert call(hq=6) == uns and call(hq=32) == uns                     # 3 and 16 heads a KV head
    for pool, dt in (("f32", pkv.PKV_F32), ("i8", pkv.PKV_F16), ("i4", pkv.PKV_F16)):
        assert call(pool=pool, dt=dt) == uns
    assert call(dt=pkv.PKV_F16) == inv and call(pool="f16") == inv
    assert call(pool="f8", dt=pkv.PKV_F32, ks=a, vs=a) == inv
    assert call(pool="f8") == inv and call(pool="f8", ks=a) == inv and call(pool="f8", ks=a, vs=a + 2) == inv
    for bad in (0.0, -0.1, float("inf"), float("nan")):
        assert call(scale=bad) == inv
    assert call(window=-1) == inv and call(window=4, vis=a) == inv and call(vis=a + 4) == inv
    for kw in (dict(B=-1), dict(T=-1), dict(mb=-1), dict(mq=-1)):
        assert call(**kw) == inv
    assert call(B=65536) == uns and call(hq=2 * 65536) == uns
    for name in ("q", "kc", "vc", "bt", "qs", "sl", "out", "ws"):
        assert call(**{name: None}) == inv, name
        assert call(**{name: a + 2}) == inv, name
    for kw in (dict(B=0), dict(T=0), dict(mq=0)):
        assert call(q=None, **kw) == pkv.PKV_OK
    if not torch.cuda.is_available():
        assert call() == pkv.PKV_ERR_CUDA


def test_workspace_bytes():
    p = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_BF16)
    small, large = pkv.paged_chunk_workspace_bytes(p, 4, 8, 32), pkv.paged_chunk_workspace_bytes(p, 4, 8, 33)
    assert 0 < small < large == pkv.paged_chunk_workspace_bytes(p, 9, 8, 100000)
    for args in ((-1, 8, 4), (4, 7, 4), (4, 0, 4), (4, 8, -1)):
        assert pkv.paged_chunk_workspace_bytes(p, *args) == 0


# --------------------------------------------------------------------------- reference
def make(lens, new, hq, H, D, bs, dtype, kv, seed=0, tree=None, spread=0, poison=True, gap=3):
    """A paged cache of sequences of lens[b] rows, the last new[b] of them with queries; rows that no
    sequence holds are NaN (16 bits) or NaN codes (8 bits)."""
    g = torch.Generator().manual_seed(seed)
    B, T = len(lens), sum(new) + gap
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    ids = torch.randperm(nb, generator=g).tolist()
    bt = torch.full((B, max(1, max(need)) + 1), 2 ** 30, dtype=torch.int32)      # entries that nothing may look at
    at = 0
    for b in range(B):
        bt[b, :need[b]] = torch.tensor(ids[at:at + need[b]], dtype=torch.int32)
        at += need[b]
    s = dict(lens=list(lens), new=list(new), hq=hq, H=H, D=D, bs=bs, dtype=dtype, kv=kv, tree=tree, T=T, nb=nb, bt=bt)
    s["pool"] = pkv.kv_block_pool_init(nb, bs, H, D, KV[kv])
    for n in ("k", "v"):
        x = torch.randn(nb, H, bs, D, generator=g)
        x = torch.where(torch.rand(x.shape, generator=g) < 0.01, x * 8, x)
        used = torch.zeros(nb, bs, dtype=torch.bool)
        for b in range(B):
            for j in range(need[b]):
                used[bt[b, j], :min(bs, lens[b] - j * bs)] = True
        if kv == "f8":
            e = torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448.0))
            if spread:
                e = e + torch.randint(-spread, spread + 1, e.shape, generator=g)
            scale = torch.exp2(e).float()
            code = (x / torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3), keepdim=True) / 448.0)))).to(torch.float8_e4m3fn)
            s[n] = code.double() * scale.double()[:, :, None, None]
            code = code.view(torch.uint8).clone()
            if poison:
                code[~used[:, None, :].expand(nb, H, bs)] = 0x7f
            s[n + "c"], s[n + "s"] = code.view(torch.float8_e4m3fn).to(DEV), scale.to(DEV)
        else:
            x = x.to(DT[dtype])
            s[n] = x.double()
            c = x.clone()
            if poison:
                c[~used[:, None, :].expand(nb, H, bs)] = float("nan")
            s[n + "c"], s[n + "s"] = c.to(DEV), None
    s["q"] = (torch.randn(T, hq, D, generator=g) * 1.5).to(DT[dtype])
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s["start"] = start
    return s


def reference(s, scale, window=0):
    """Float64 outputs and the bound of each, [T, Hq, D] (rows without a token: NaN).

    The bound of an element, with w the weights (sum 1) and A = sum w |v|: a score is a sum of
    D / 16 MMA accumulations in fp32, each off by at most 2^-22 of the sum of magnitudes a = max
    scale sum_d |q_d k_d| (an MMA may truncate), plus its roundings to the log2 domain: e =
    (D / 16 + 4) 2^-22 a, and 2^-22 for the exponential.  Numerator and denominator each carry
    that and their own accumulations, n / 16 + 15 roundings of 2^-22.  A weight enters the product
    rounded to u: half a step of q's type, and over e4m3 of fp16 (what the codes are multiplied
    as); as fp16, times 2^7 below the running maximum's 2^8, a weight (times its block's scale)
    is off by 2^-32 of the largest at least.  The quotient is rounded once more, to the output's type, half a step."""
    H, D, G = s["H"], s["D"], s["hq"] // s["H"]
    out = torch.full((s["T"], s["hq"], D), math.nan, dtype=torch.float64)
    lim = torch.zeros_like(out)
    u_out = HALF_STEP[s["dtype"]]
    u_p = u_out if s["kv"] != "f8" else HALF_STEP["f16"]
    for b, (L, n) in enumerate(zip(s["lens"], s["new"])):
        if n == 0:
            continue
        ids = s["bt"][b, :-(-L // s["bs"])].long()
        key, pos = torch.arange(L), torch.arange(L - n, L)[:, None]
        sees = key <= pos
        if window:
            sees &= key > pos - window
        if s["tree"] is not None:
            own = torch.tensor([[(w >> j) & 1 for j in range(n)] for w in s["tree"][s["start"][b]:s["start"][b + 1]]], dtype=torch.bool)
            sees = torch.cat([torch.ones(n, L - n, dtype=torch.bool), own.reshape(n, n)], dim=1)
        r = slice(s["start"][b], s["start"][b + 1])
        for h in range(H):
            k, v = (s[x][ids, h].reshape(-1, D)[:L] for x in "kv")
            q = s["q"][r, h * G:(h + 1) * G].double()                    # [n, G, D]
            sc = torch.einsum("igd,jd->igj", q, k) * scale
            sc = sc.masked_fill(~sees[:, None, :], -math.inf)
            some = sees.any(dim=1)[:, None, None]
            w = torch.where(some, torch.softmax(torch.where(some, sc, 0.0), dim=2), 0.0)
            a = scale * float((q.abs().reshape(-1, D) @ k.abs().T).max())
            y, A = w @ v, w @ v.abs()
            e = 2.0 ** -22 * ((D / 16 + 4) * a + 1 + L / 16 + 15)
            err = A * (u_p + 2 * e) * (1 + 2.0 ** -6) + L * 2.0 ** -32 * float(v.abs().max())
            out[r, h * G:(h + 1) * G] = y
            lim[r, h * G:(h + 1) * G] = err + u_out * (y.abs() + err) + (2.0 ** -25 if s["dtype"] == "f16" else 0.0)
    return out, lim


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def run(s, scale, window=0, out=None, ws=None, max_q=None, stream=None, tables=None):
    pool, T = s["pool"], s["T"]
    max_q = max(s["new"] + [1]) if max_q is None else max_q
    out = torch.full((T, s["hq"], s["D"]), 7.0, dtype=DT[s["dtype"]], device=DEV) if out is None else out
    ws = pkv.alloc_chunk_workspace(pool, len(s["lens"]), s["hq"], max_q) if ws is None else ws
    vis = None
    if s["tree"] is not None:
        words = [w - (1 << 64) if w >> 63 else w for w in s["tree"]] + [0] * (T - len(s["tree"]))
        vis = torch.tensor(words, dtype=torch.int64).to(DEV)
    pkv.paged_chunk_attention(pool, s["q"].to(DEV), s["kc"], s["vc"], s["bt"].to(DEV) if tables is None else tables, i32(s["start"]), i32(s["lens"]),
                              scale, out, ws, max_q, s["ks"], s["vs"], window=window, visible=vis, stream=stream)
    return out


def check(s, out, window=0, scale=None):
    scale = 1.0 / math.sqrt(s["D"]) if scale is None else scale
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK
    y, lim = reference(s, scale, window)
    n = s["start"][-1]
    assert bool((out[n:] == 7).all())                                     # rows behind the last sequence
    err = (out[:n].double().cpu() - y[:n]).abs()
    bad = ~(err <= lim[:n])
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((err / lim[:n]).nan_to_num(99.0).max()))


# --------------------------------------------------------------------------- GPU
CASES = [  # lens, new, hq, H, D, bs, dtype, kv
    ([5], [1], 1, 1, 64, 16, "f16", "f16"),
    ([130], [3], 4, 1, 128, 16, "bf16", "bf16"),
    ([1], [1], 8, 1, 128, 8, "bf16", "f8"),
    ([200, 64, 1], [8, 64, 1], 8, 2, 64, 8, "f16", "f8"),
    ([700], [700], 4, 4, 64, 4, "f16", "f16"),
    ([300, 0, 513, 128], [300, 0, 1, 127], 12, 3, 128, 32, "bf16", "bf16"),
    ([257, 1000], [129, 33], 16, 2, 128, 16, "f16", "f8"),
    ([257, 1000], [129, 33], 16, 2, 128, 256, "bf16", "f8"),
    ([2000], [5], 8, 1, 128, 64, "bf16", "bf16"),
    ([9000], [2], 2, 2, 64, 16, "f16", "f16"),
    ([6000, 17], [300, 17], 8, 1, 64, 16, "bf16", "f8"),
    ([40, 41, 42, 43] * 20, [1, 2, 3, 4] * 20, 2, 1, 128, 16, "f16", "f16"),
    ([385] * 6, [385, 384, 257, 256, 128, 1], 2, 1, 128, 128, "bf16", "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_gpu_causal(case):
    s = make(*case)
    check(s, run(s, 1.0 / math.sqrt(s["D"])))


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 7, 128, 300])
@pytest.mark.parametrize("case", [CASES[3], CASES[5], CASES[7], CASES[9], CASES[10], CASES[12]], ids=[3, 5, 7, 9, 10, 12])
def test_gpu_window(case, window):
    s = make(*case)
    # blocks before every token's window are not looked at: freed ones' ids are gone
    t = s["bt"].clone()
    for b, (L, n) in enumerate(zip(s["lens"], s["new"])):
        if n:
            t[b, :max(0, L - n - window + 1) // s["bs"]] = -5
    check(s, run(s, 1.0 / math.sqrt(s["D"]), window, tables=t.to(DEV)), window)


def _tree(new, kind, seed=0):
    rng = np.random.default_rng(seed)
    words = []
    for n in new:
        mine = []
        for i in range(n):
            if kind == "chain":
                w = (1 << (i + 1)) - 1
            elif kind == "drafts":
                p = int(rng.integers(-1, i)) if i else -1
                w = (mine[p] if p >= 0 else 0) | 1 << i
            elif kind == "none":
                w = 0
            else:                                     # any, later tokens among them
                w = int(rng.integers(0, 2 ** 62)) << 2 | int(rng.integers(0, 4))
            mine.append(w)
        words += mine
    return words


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["chain", "drafts", "none", "any"])
@pytest.mark.parametrize("case", [
    ([200, 64, 1], [8, 64, 1], 8, 2, 64, 8, "f16", "f8"),
    ([64, 130, 7, 1000], [64, 3, 7, 40], 4, 1, 128, 16, "bf16", "bf16"),
    ([64, 190, 128], [64, 63, 2], 8, 1, 128, 16, "bf16", "f8"),
    ([300, 3], [33, 3], 8, 8, 64, 32, "f16", "f16"),
], ids=range(4))
def test_gpu_tree(case, kind):
    lens, new = case[0], case[1]
    s = make(*case, tree=_tree(new, kind))
    out = run(s, 1.0 / math.sqrt(s["D"]))
    check(s, out)
    if kind == "none":                                # tokens of a sequence without cached rows see nothing
        assert bool((out[:s["start"][-1]][torch.tensor([n == L for L, n in zip(lens, new) for _ in range(n)])] == 0).all())
    if kind == "chain":                               # what causal attention gives, bit for bit
        t = dict(s, tree=None)
        assert torch.equal(run(t, 1.0 / math.sqrt(s["D"])), out)


@pytest.mark.gpu
def test_gpu_against_the_other_entry_points():
    """Whole prompts: paged_prefill_attention's result to both bounds; a single token:
    paged_decode_attention's."""
    s = make([300, 77], [300, 77], 8, 2, 128, 16, "bf16", "bf16", poison=False)
    out = run(s, 0.09)
    full = torch.zeros(s["T"], 8, 128, device=DEV)
    pkv.paged_prefill_attention(s["pool"], s["q"].to(DEV), s["kc"], s["vc"], s["bt"].to(DEV), i32(s["start"]), i32(s["lens"]), 0.09, full, 300)
    y, lim = reference(s, 0.09)
    n = s["start"][-1]
    # prefill's own bound: 2^-16 of the weights, and the rest of the chunk's
    assert bool(((out[:n].double() - full[:n].double()).abs().cpu() <= 2 * lim[:n]).all())
    d = make([300, 77], [1, 1], 8, 2, 128, 16, "bf16", "bf16", poison=False, gap=0)
    one = run(d, 0.09)
    dec = torch.zeros(2, 8, 128, device=DEV)
    ws = pkv.alloc_workspace(d["pool"], 2, 8)
    pkv.paged_decode_attention(d["pool"], d["q"].to(DEV), d["kc"], d["vc"], d["bt"].to(DEV), i32(d["lens"]), 0.09, dec, ws, 300)
    y, lim = reference(d, 0.09)
    assert bool(((one.double() - dec.double()).abs().cpu() <= 2 * lim).all())


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [3, 30])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gpu_f8_scales_far_apart(dtype, spread):
    """Blocks whose scales differ by up to 2^(2 spread)."""
    s = make([500, 1200], [20, 3], 8, 2, 128, 16, dtype, "f8", seed=5, spread=spread)
    # keys of one size: the scores' bound is their own magnitude's
    s["k"], one = s["k"] / s["ks"].double().cpu()[:, :, None, None] * 2.0 ** -7, torch.full_like(s["ks"], 2.0 ** -7)
    s["ks"] = one
    scale = 1.0 / math.sqrt(128)
    out = run(s, scale)
    if dtype == "f16" and spread > 10:                # values beyond fp16's largest number are inf in the output
        y, _ = reference(s, scale)
        n = s["start"][-1]
        fine = y[:n].abs() < 60000
        assert bool(torch.isfinite(out[:n].cpu())[fine].all())
        return
    check(s, out, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "f8"])
def test_gpu_bad_indices(kv):
    s = make([100, 200, 150], [10, 20, 5], 8, 2, 64, 16, "bf16", kv, gap=0)
    good = run(s, 0.1)
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK
    for what in ("long", "short", "many", "id", "negative"):
        t = dict(s, bt=s["bt"].clone(), lens=list(s["lens"]), start=list(s["start"]))
        max_q = 20
        if what == "long":
            t["lens"][1] = t["bt"].shape[1] * 16 + 1
        elif what == "short":
            t["lens"][1] = 19
        elif what == "many":
            max_q = 19
        elif what == "id":
            t["bt"][1, 3] = s["nb"]
        else:
            t["bt"][1, 0] = -1
        out = run(t, 0.1, max_q=max_q)
        assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_ERR_BAD_INDEX, what
        assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK
        same = [b for b in (0, 2)]
        for b in same:
            r = slice(s["start"][b], s["start"][b + 1])
            if what not in ("id", "negative"):         # (another cut of the work rounds otherwise)
                assert torch.allclose(out[r].float(), good[r].float(), rtol=0.02, atol=0.02), what
            else:
                assert torch.equal(out[r], good[r]), what
        if what not in ("id", "negative"):
            assert bool((out[s["start"][1]:s["start"][2]] == 7).all()), what


@pytest.mark.gpu
def test_gpu_streams_graph_and_workspaces():
    """A side stream, a captured and replayed call, a larger workspace: the same bits; a call after
    another of another shape on the same workspace too."""
    a = make([3000, 100], [20, 9], 8, 2, 128, 16, "bf16", "bf16", gap=0)
    b = make([700] * 3, [200, 30, 64], 8, 1, 64, 16, "f16", "f8", gap=0)
    sa, sb = 1.0 / math.sqrt(128), 0.125
    wa, wb = run(a, sa), run(b, sb)
    size = max(pkv.paged_chunk_workspace_bytes(a["pool"], 2, 8, 20), pkv.paged_chunk_workspace_bytes(b["pool"], 3, 8, 200)) + 4096
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        assert torch.equal(run(a, sa, ws=ws), wa) and torch.equal(run(b, sb, ws=ws), wb)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty_like(wa)
    with torch.cuda.stream(stream):
        run(a, sa, ws=ws, out=out)
    stream.synchronize()
    assert torch.equal(out, wa)
    q, bt, st, ln = a["q"].to(DEV), a["bt"].to(DEV), i32(a["start"]), i32(a["lens"])
    q2, bt2, st2, ln2 = b["q"].to(DEV), b["bt"].to(DEV), i32(b["start"]), i32(b["lens"])
    oa, ob = torch.zeros_like(wa), torch.zeros_like(wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_chunk_attention(a["pool"], q, a["kc"], a["vc"], bt, st, ln, sa, oa, ws, 20)
        pkv.paged_chunk_attention(b["pool"], q2, b["kc"], b["vc"], bt2, st2, ln2, sb, ob, ws, 200, b["ks"], b["vs"])
    for _ in range(2):
        oa.zero_(), ob.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)
    # other lengths in the same graph: what a serving loop replays
    ln.copy_(i32([2500, 60]))
    graph.replay()
    torch.cuda.synchronize()
    check(dict(a, lens=[2500, 60], T=a["T"]), oa, scale=sa)


@pytest.mark.gpu
def test_gpu_nothing_to_do():
    s = make([10, 20], [0, 0], 4, 2, 64, 16, "f16", "f16")
    out = run(s, 0.125)
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK and bool((out == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    ([33, 1, 700] * 340, [1, 1, 2] * 340, 1, 1, 64, 16, "f16", "f16"),       # more sequences than threads
    ([33, 1, 700] * 340, [1, 0, 2] * 340, 4, 1, 128, 16, "bf16", "f8"),
    ([70000], [1], 4, 1, 64, 64, "bf16", "bf16"),                            # one item in more than 32 shares
    ([90001, 5], [3, 5], 8, 1, 128, 16, "f16", "f8"),
    ([40000, 300], [200, 300], 2, 1, 64, 32, "f16", "f16"),
], ids=["many", "many_f8", "long", "long_f8", "long_256"])
def test_gpu_many_and_long(case):
    s = make(*case)
    check(s, run(s, 1.0 / math.sqrt(s["D"])))
    check(s, run(s, 1.0 / math.sqrt(s["D"]), 100), 100)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "f8"])
def test_gpu_keys_not_finite_where_masked(kv):
    """K rows of NaN and infinity change no output of a token that does not see them."""
    s = make([300, 90], [40, 90], 4, 2, 64, 16, "bf16", kv, gap=0)
    want = run(s, 0.125)
    g = s["bt"].long()
    new = 290                                          # the first sequence's position from which K is spoilt
    if kv == "f8":
        c = s["kc"].view(torch.uint8)
        for p in range(new, 300):
            c[g[0, p // 16], :, p % 16] = 0x7f if p % 2 else 0xff
    else:
        for p in range(new, 300):
            s["kc"][g[0, p // 16], :, p % 16] = [math.nan, math.inf, -math.inf][p % 3]
    got = run(s, 0.125)
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK
    keep = torch.tensor(list(range(30)) + list(range(40, 130)), device=DEV)
    assert torch.equal(got[keep], want[keep])
    # in a tree: token 0's row is seen by nobody but itself
    t = make([200], [6], 4, 2, 64, 16, "bf16", kv, gap=0, tree=[1, 2, 6, 14, 30, 62])
    want = run(t, 0.125)
    b, off = int(t["bt"][0, 194 // 16]), 194 % 16
    t["kc"].view(torch.uint8)[b, :, off] = 0x7f         # (0x7f7f is no NaN of bf16, but 3.4e38)
    assert torch.equal(run(t, 0.125)[1:], want[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["f16", "f8"])
def test_gpu_shared_blocks_and_a_sequence_twice(kv):
    """Two sequences on the same blocks, and one as long as another's prefix."""
    s = make([200, 200, 200], [20, 20, 9], 8, 2, 128, 16, "f16", kv, gap=0)
    s["bt"][1], s["bt"][2] = s["bt"][0], s["bt"][0]
    s["lens"][2] = 50
    check(s, run(s, 0.1), scale=0.1)
    s["q"][20:40] = s["q"][:20]
    out = run(s, 0.1)
    n = s["start"]
    assert bool(((out[:20].double() - out[20:40].double()).abs() <= 2 * reference(s, 0.1)[1][:20].to(DEV)).all())


@pytest.mark.gpu
def test_gpu_two_calls_at_once():
    """Two streams, a workspace each: the bits of the calls one after the other."""
    a = make([20000, 100], [20, 9], 8, 2, 128, 16, "bf16", "bf16", gap=0)
    b = make([9000] * 3, [200, 30, 64], 8, 1, 64, 16, "f16", "f8", gap=0)
    wa, wb = run(a, 0.09), run(b, 0.125)
    args = []
    for s, n in ((a, 20), (b, 200)):
        args.append((s["q"].to(DEV), s["bt"].to(DEV), i32(s["start"]), i32(s["lens"]), pkv.alloc_chunk_workspace(s["pool"], len(s["lens"]), 8, n)))
    oa, ob = torch.zeros_like(wa), torch.zeros_like(wb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        q, bt, st, ln, ws = args[0]
        pkv.paged_chunk_attention(a["pool"], q, a["kc"], a["vc"], bt, st, ln, 0.09, oa, ws, 20, stream=sa)
        q, bt, st, ln, ws = args[1]
        pkv.paged_chunk_attention(b["pool"], q, b["kc"], b["vc"], bt, st, ln, 0.125, ob, ws, 200, b["ks"], b["vs"], stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)


@pytest.mark.gpu
def test_gpu_a_larger_limit_of_new_tokens():
    """max_q_len above every sequence's own count, and far above."""
    s = make([200, 64, 1000], [8, 3, 1], 8, 2, 64, 16, "bf16", "bf16")
    for max_q in (8, 9, 17, 1000, 2 ** 31 - 1):
        check(s, run(s, 0.125, max_q=max_q), scale=0.125)


def test_tensors_elsewhere_are_refused():
    s = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_BF16)
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.paged_chunk_attention(s, x, None, None, None, None, None, 0.1, x, None, 3)


@pytest.mark.gpu
def test_gpu_binding_refusals():
    s = make([20], [3], 4, 2, 64, 16, "bf16", "bf16", gap=0)
    pool, q, bt, st, ln = s["pool"], s["q"].to(DEV), s["bt"].to(DEV), i32(s["start"]), i32(s["lens"])
    out, ws = torch.zeros_like(q), pkv.alloc_chunk_workspace(s["pool"], 1, 4, 3)

    def call(q=q, kc=s["kc"], vc=s["vc"], bt=bt, st=st, ln=ln, out=out, ws=ws, **kw):
        pkv.paged_chunk_attention(pool, q, kc, vc, bt, st, ln, 0.1, out, ws, 3, **kw)
    call()
    one = torch.zeros(1, dtype=torch.uint8, device=DEV)
    for kw in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)), dict(kc=s["kc"].half()), dict(vc=s["vc"][:1]),
               dict(kc=s["kc"].cpu()), dict(bt=bt.long()), dict(bt=bt[:0]), dict(bt=bt[:, ::2]), dict(st=st[:1]), dict(st=st.cpu()), dict(ln=ln.float()),
               dict(out=out.float()), dict(out=out[:2]), dict(out=out.cpu()), dict(ws=ws.cpu()), dict(ws=one.expand(ws.numel())),
               dict(visible=torch.zeros(2, dtype=torch.int64, device=DEV)), dict(visible=torch.zeros(3, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(pkv.PkvError):
        call(ws=ws[:ws.numel() - 16])
    torch.cuda.synchronize()
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK
