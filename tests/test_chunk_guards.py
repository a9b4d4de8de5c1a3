"""Guard regions around every device buffer of kv_rope_rotate, kv_rope_append and
paged_chunk_attention: what they may not write keeps its bytes, their inputs too."""
import math

import pytest
import torch

import test_chunk as C
import test_rope as P
from paged_kv_cache_273_gb300 import pkv

DEV = "cuda"
GUARD = 8192                                           # bytes on either side of a buffer
i32 = P.i32


class Arena:
    """Buffers that each lie between two guard regions."""

    def __init__(self):
        self.whole, self.inputs = [], []

    def put(self, x, written=False):
        """x (a device tensor or None) in a guarded buffer of its own; not `written`: an input, that
        keeps its bytes."""
        if x is None:
            return None
        n = x.numel() * x.element_size()
        buf = torch.full((2 * GUARD + (n + 255) // 256 * 256,), 0xa5, dtype=torch.uint8, device=DEV)
        y = buf[GUARD:GUARD + n].view(x.dtype).view(x.shape)
        y.copy_(x)
        self.whole.append((buf, n))
        if not written:
            self.inputs.append((buf, buf.clone()))
        return y

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.whole:
            assert bool((buf[:GUARD] == 0xa5).all()) and bool((buf[GUARD + n:] == 0xa5).all())
        for buf, before in self.inputs:
            assert torch.equal(buf, before)


CHUNKS = [  # lens, new, hq, H, D, bs, dtype, kv, window, tree
    ([5], [1], 1, 1, 64, 16, "f16", "f16", 0, None),
    ([130, 0, 64], [3, 0, 5], 4, 1, 128, 16, "bf16", "bf16", 0, "drafts"),
    ([700, 40], [700, 1], 4, 4, 64, 4, "f16", "f16", 100, None),
    ([300, 513, 128], [300, 1, 127], 12, 3, 128, 256, "bf16", "bf16", 0, None),
    ([257, 1000], [129, 33], 16, 2, 128, 16, "f16", "f8", 0, None),
    ([200, 64, 1], [8, 64, 1], 8, 2, 64, 8, "bf16", "f8", 0, "any"),
    ([6000, 17], [300, 17], 8, 1, 64, 64, "bf16", "f8", 500, None),
    ([70000], [1], 4, 1, 64, 64, "bf16", "bf16", 0, None),        # states of one item from every CTA
    ([40000, 300], [200, 300], 2, 1, 64, 32, "f16", "f8", 0, None),
    ([33, 1, 700] * 100, [1, 1, 2] * 100, 1, 1, 128, 16, "f16", "f16", 0, None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CHUNKS, ids=range(len(CHUNKS)))
def test_gpu_chunk_guards(case):
    lens, new, hq, H, D, bs, dtype, kv, window, tree = case
    s = C.make(lens, new, hq, H, D, bs, dtype, kv, tree=C._tree(new, tree) if tree else None)
    a = Arena()
    pool, max_q = s["pool"], max(new)
    for n in ("kc", "vc", "ks", "vs"):
        s[n] = a.put(s[n])
    q, bt, start, ln = (a.put(x.to(DEV)) for x in (s["q"], s["bt"], i32(s["start"]), i32(s["lens"])))
    vis = None
    if tree:
        words = [w - (1 << 64) if w >> 63 else w for w in s["tree"]] + [0] * (s["T"] - len(s["tree"]))
        vis = a.put(torch.tensor(words, dtype=torch.int64).to(DEV))
    out = a.put(torch.full((s["T"], hq, D), 7.0, dtype=C.DT[dtype], device=DEV), True)
    size = pkv.paged_chunk_workspace_bytes(pool, len(lens), hq, max_q)
    ws = a.put(torch.full((size,), 255, dtype=torch.uint8, device=DEV), True)
    pkv.paged_chunk_attention(pool, q, s["kc"], s["vc"], bt, start, ln, 1.0 / math.sqrt(D), out, ws, max_q, s["ks"], s["vs"], window=window,
                              visible=vis)
    a.check()
    C.check(s, out, window)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "f8"])
def test_gpu_chunk_guards_bad_indices(kv):
    """Lengths and block ids out of range: nothing behind any buffer is written, no input."""
    s = C.make([100, 200, 150], [10, 20, 5], 8, 2, 64, 16, "bf16", kv)
    for what in ("long", "short", "many", "id", "negative"):
        bt, lens, max_q = s["bt"].clone(), list(s["lens"]), 20
        if what == "long":
            lens[1] = 2 ** 31 - 1
        elif what == "short":
            lens[1] = -5
        elif what == "many":
            max_q = 19
        elif what == "id":
            bt[1, 3] = 2 ** 31 - 1
        else:
            bt[1, 0] = -2 ** 31
        a = Arena()
        kc, vc, ks, vs = (a.put(s[n]) for n in ("kc", "vc", "ks", "vs"))
        q, t, start, ln = (a.put(x.to(DEV)) for x in (s["q"], bt, i32(s["start"]), i32(lens)))
        out = a.put(torch.full((s["T"], 8, 64), 7.0, dtype=torch.bfloat16, device=DEV), True)
        ws = a.put(pkv.alloc_chunk_workspace(s["pool"], 3, 8, max_q), True)
        pkv.paged_chunk_attention(s["pool"], q, kc, vc, t, start, ln, 0.125, out, ws, max_q, ks, vs)
        a.check()
        assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_ERR_BAD_INDEX, what
        assert bool((out[35:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [False, True])
@pytest.mark.parametrize("case", P.APPENDS, ids=range(len(P.APPENDS)))
def test_gpu_append_guards(case, pad):
    """Rows, scales and q_out between guards; pad: padding and slots out of range among the tokens.
    Rows of the caches that no slot names keep their bytes (an 8-bit block's may be brought to
    a new scale: those of blocks that the call does not touch)."""
    s = P._append_state(case)
    kv, bs = case[10], case[5]
    slots = list(s["slots"])
    if pad:
        slots = [-1 if i % 7 == 3 else 2 ** 31 - 1 if i % 11 == 5 else x for i, x in enumerate(slots)]
        if kv == "f8":                                 # (a block gets at most one run a call: whole ones go)
            slots = [x if i == 0 or s["slots"][i] // bs == s["slots"][0] // bs else -1 if i % 2 else 2 ** 31 - 1 for i, x in enumerate(s["slots"])]
    a = Arena()
    hq, H = case[2], case[3]
    qkv = a.put(s["q"]._base if s["q"]._base is not None else torch.cat([s["q"], s["k"], s["v"]], 1))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + H], qkv[:, hq + H:]
    before = {}
    for n in ("kc", "vc", "ks", "vs", "q_out"):
        before[n] = None if s[n] is None else s[n].clone()
        s[n] = a.put(s[n], True)
    pos, sl = a.put(i32(s["pos"])), a.put(i32(slots))
    pkv.kv_rope_append(s["pool"], s["plan"], q if hq else None, k, v, pos, sl, s["q_out"] if hq else None, s["kc"], s["vc"], s["ks"], s["vs"])
    a.check()
    good = [x for x in slots if 0 <= x < s["pool"].num_blocks * bs]
    want = pkv.PKV_OK if all(x < 0 or x < s["pool"].num_blocks * bs for x in slots) else pkv.PKV_ERR_BAD_INDEX
    assert pkv.pkv_check_error(s["pool"]) == want
    keep = torch.ones(s["pool"].num_blocks, bs, dtype=torch.bool, device=DEV)
    for x in good:
        keep[x // bs] &= False if kv == "f8" else True
        keep[x // bs, x % bs] = False
    for n in ("kc", "vc"):
        got, was = (c.view(torch.uint8).transpose(1, 2)[keep] for c in (s[n], before[n]))
        assert torch.equal(got, was), n
    for n in ("ks", "vs"):
        if s[n] is not None:
            assert torch.equal(s[n][keep.all(1)], before[n][keep.all(1)]), n
    left = torch.tensor([not 0 <= x < s["pool"].num_blocks * bs for x in slots], device=DEV)
    assert torch.equal(s["q_out"][left], before["q_out"][left])


@pytest.mark.gpu
@pytest.mark.parametrize("case", P.CASES, ids=lambda c: "-".join(map(str, c)))
def test_gpu_rotate_guards(case):
    T, H, D, rot, layout, scaling, dtype = case
    plan = pkv.rope_plan(rot, layout=layout, scaling=scaling, **P.SCALINGS[scaling])
    a = Arena()
    words = plan.freqs
    plan.freqs = a.put(words)
    plan.struct.freqs = plan.freqs.data_ptr()
    x, _ = P.rows(T, H, D, dtype, 1)
    wide = a.put(torch.full((T, H + 2, D), 7.0, dtype=x.dtype, device=DEV), True)
    y = a.put(x.contiguous())
    pkv.kv_rope_rotate(plan, y, a.put(i32([17 * t for t in range(T)])), wide[:, :H])
    a.check()
    assert bool((wide[:, H:] == 7).all())
    again = pkv.kv_rope_rotate(plan, y, i32([17 * t for t in range(T)]))
    assert torch.equal(again, wide[:, :H])
