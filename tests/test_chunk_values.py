"""paged_chunk_attention over values that are not finite, and results at the ends of fp16's range."""
import math

import pytest
import torch

import test_chunk as C
from paged_kv_cache_273_gb300 import pkv

DEV = "cuda"
BEFORE, BEHIND = 254, 382          # include/pkv.h: how far a row of V that is not finite reaches


def _spoil(s, b, rows):
    """The caches with these rows of sequence b's V not finite."""
    vc = s["vc"].clone()
    for i, r in enumerate(rows):
        blk, off = int(s["bt"][b, r // s["bs"]]), r % s["bs"]
        if s["kv"] == "f8":
            vc.view(torch.uint8)[blk, :, off] = 0x7f
        else:
            vc[blk, :, off] = [math.nan, math.inf, -math.inf][i % 3]
    return dict(s, vc=vc)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 1, 200])
@pytest.mark.parametrize("hq,bs,kv", [(1, 16, "bf16"), (1, 256, "f16"), (4, 16, "bf16"), (1, 16, "f8"), (2, 256, "f8")])
def test_gpu_values_not_finite_reach_no_further(hq, bs, kv, window):
    """A spoilt row of V at every place of a tile and of an item of 256 rows: tokens outside of its
    reach keep their bits, tokens that see it are not finite, other sequences keep theirs."""
    dtype = "f16" if kv == "f16" else "bf16"
    # new tokens from position 513 on: items' first tokens are the second of a tile
    L, n = 1600, 1087
    s = C.make([300, L], [140, n], hq, 1, 64, bs, dtype, kv, gap=0)
    scale = 0.125
    want = C.run(s, scale, window)
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK and bool(torch.isfinite(want).all())
    p = torch.arange(L - n, L, device=DEV)
    for r in [0, 130, 400, 512, 513, 514, 639, 640, 641, 766, 767, 768, 769, 895, 896, 1023, 1024, 1025, 1280, 1599]:
        got = C.run(_spoil(s, 1, [r]), scale, window)
        assert torch.equal(got[:140], want[:140]), r
        mine, was = got[140:], want[140:]
        first = p - window + 1 if window else torch.zeros_like(p)
        out_of_reach = (r - p > BEFORE) | (first - r > BEHIND)
        assert torch.equal(mine[out_of_reach], was[out_of_reach]), r
        sees = (r <= p) & (r >= first)
        assert not bool(torch.isfinite(mine[sees]).any()), r
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "f8"])
def test_gpu_values_not_finite_in_a_tree(kv):
    """A drafted token's spoilt V reaches its own sequence alone; a cached row's every token, which
    all see it."""
    new = [64, 40]
    s = C.make([200, 90], new, 4, 2, 64, 16, "bf16", kv, gap=0, tree=C._tree(new, "drafts"))
    want = C.run(s, 0.125)
    for r in (136, 199, 135, 0):
        got = C.run(_spoil(s, 0, [r]), 0.125)
        assert torch.equal(got[64:], want[64:]), r
        sees = [r < 136 or bool((w >> (r - 136)) & 1) for w in s["tree"][:64]]
        assert not bool(torch.isfinite(got[:64][torch.tensor(sees, device=DEV)]).any()), r
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK


def _far_apart(dtype, shift):
    """Blocks whose V scales differ by up to 2^60, all times 2^shift; keys of one size."""
    s = C.make([500, 1200], [20, 3], 8, 2, 128, 16, dtype, "f8", seed=5, spread=30)
    s["k"], one = s["k"] / s["ks"].double().cpu()[:, :, None, None] * 2.0 ** -7, torch.full_like(s["ks"], 2.0 ** -7)
    s["ks"] = one
    s["v"], s["vs"] = s["v"] * 2.0 ** shift, s["vs"] * 2.0 ** shift
    return s


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shift", [("f16", 0), ("f16", -12), ("f16", -24), ("f16", -34), ("bf16", 0), ("bf16", 80), ("bf16", -50)])
def test_gpu_f8_scales_far_apart_to_the_bound(dtype, shift):
    """Every output to its bound; in fp16 those beyond its largest number are infinite, and those
    within their bound of it either."""
    s = _far_apart(dtype, shift)
    scale = 1.0 / math.sqrt(128)
    out = C.run(s, scale)
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK
    y, lim = C.reference(s, scale)
    n = s["start"][-1]
    y, lim, got = y[:n], lim[:n], out[:n].double().cpu()
    # half a step above the largest number is where rounding goes to infinity
    border = 65520.0 if dtype == "f16" else float("inf")
    small, large = y.abs() + lim < border, y.abs() - lim > border
    if dtype == "f16" and shift <= -24:
        assert bool(small.all())                       # (nothing is left out where all are in range)
    err = (got - y).abs()
    assert bool((err[small] <= lim[small]).all()), float((err[small] / lim[small]).max())
    assert torch.equal(got[large], torch.where(y > 0, math.inf, -math.inf).double()[large])
    assert bool((out[n:] == 7).all())
