"""Decode attention over 8-bit float caches and over chosen blocks where a few rows or blocks
outweigh the rest: rows of large scores and no value, blocks of far larger scales, scores and
sums at the ends of fp32's range; against float64, each element held to its own weighted sum of
magnitudes."""
import math

import numpy as np
import pytest
import torch

import block_reference as R
from test_f8_cache import DEV, Cache, _attend, _batch, _rows
from test_sparse import Sparse, _tables
from paged_kv_cache_273_gb300 import pkv

pytestmark = pytest.mark.gpu


def attend(q, k, v, scale, floor=2.0 ** -40, parts=2.0 ** -22):
    """softmax(scale q k^T) v in float64 and each element's error bound.

    As in block_reference.attend a weight is off, relatively, by e = (D / 16 + 4) 2^-22 a +
    2^-22 + `parts`, a the largest sum of magnitudes of a score, and the sums over n rows by
    (n / 16 + 14) 2^-22: numerator and denominator both, so the element by twice that of
    sum_t w_t |v_t| / sum_t w_t.  Besides, weights of at most 2^15 for the largest row of a
    sequence lie on fp16's grid of 2^-24, which leaves 2^-25: `floor` = 2^-40 of the largest
    weight for each row, and through it floor * sum_t |v_t| / sum_t w_t (w = 1 for the largest)."""
    s = scale * (q @ k.T)
    w = np.exp(s - s.max(1, keepdims=True))
    a = np.abs(scale) * (np.abs(q) @ np.abs(k).T)
    a = a[np.isfinite(s) & (w > 0)].max() if (w > 0).any() else 0.0
    D, n = k.shape[1], k.shape[0]
    rel = 2.0 * (2.0 ** -22 * ((D / 16 + 4) * a + n / 16 + 15) + parts)
    tot = w.sum(1, keepdims=True)
    return (w @ v) / tot, (rel * (w @ np.abs(v)) + floor * np.abs(v).sum(0)) / tot


def hold(got, q, k, v, scale, **kw):
    want, tol = attend(q, k, v, float(np.float32(scale)), **kw)
    err = np.abs(got - want)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), got.flat[0],
                                want.flat[0])


def floor_of(bs):
    """Two blocks of 8 rows in a tile may share a reference that is up to 2^4 above the one's."""
    return 2.0 ** -36 if bs == 8 else 2.0 ** -40


def check(c, q, tables, lens, scale, out, seqs=None, **kw):
    got, qh, G = out.double().cpu().numpy(), q.double().cpu().numpy(), q.shape[1] // c.H
    for b in range(len(lens)) if seqs is None else seqs:
        n = lens[b]
        ids = tables[b, :-(-n // c.bs)]
        for h in range(c.H):
            hold(got[b, h * G:(h + 1) * G], qh[b, h * G:(h + 1) * G], c.rows(ids, h, n, "k"),
                 c.rows(ids, h, n, "v"), scale, **kw)
    assert pkv.pkv_check_error(c.pool) == pkv.PKV_OK


# ---------------------------------------------------------------- rows of large score, no value
@pytest.mark.parametrize("nats", [12.0, 17.5, 22.0])
@pytest.mark.parametrize("D,G,bs,dt", [(128, 4, 16, "bf16"), (64, 1, 16, "f16"),
                                       (64, 8, 8, "f16"), (128, 8, 64, "bf16")])
def test_sinks_without_value(nats, D, G, bs, dt):
    H, scale = 2, 0.125
    c = Cache(80, H, bs, D, seed=1)
    g = np.random.default_rng(2)
    k = g.normal(size=(80, H, bs, D)) * 0.05
    v = g.normal(size=(80, H, bs, D))
    k[..., 0] = 0.0
    k[:, :, 3, 0] = nats / scale / 4.0                    # q is 4 there
    v[:, :, 3] = 0.0
    for x, hc, hs in ((k, c.hk, c.hks), (v, c.hv, c.hvs)):
        e = np.vectorize(lambda a: R.exponent(a, 448.0))(np.abs(x).max((2, 3)))
        hc[:], hs[:] = R.e4m3_encode(x * np.exp2(-e)[:, :, None, None]), np.exp2(e)
    c.upload()
    lens = [60 * bs, 3, 33 * bs + 7, 4]
    tables = _batch(c, lens, 3, extra=0)
    q = _rows(4, (len(lens), H * G, D), dt)
    q[..., 0] = 4.0
    out = _attend(c, q, tables, lens, scale)
    check(c, q, tables, lens, scale, out, floor=floor_of(bs))


@pytest.mark.parametrize("kv", ["f16", "bf16", "f8"])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 2), (128, 8)])
def test_sparse_sinks_without_value(kv, D, G):
    H, bs, nats, scale, budget = 2, 16, 17.5, 0.125, 30
    s = Sparse(kv, 60, H, bs, D, seed=3)
    if kv == "f8":
        kc, vc = s.c.hk, s.c.hv
        kc[:, :, 3] = R.e4m3_encode(np.eye(1, D)[0] * 256.0)
        s.c.hks[:] = nats / scale / 4.0 / 256.0
        s.c.hks[:] = np.exp2(np.round(np.log2(s.c.hks)))
        kc[:, :, :3, 0], kc[:, :, 4:, 0], vc[:, :, 3] = 0, 0, 0
        s.c.upload()
        s.hk = R.E4M3[kc] * s.c.hks[:, :, None, None]
        s.hv = R.E4M3[vc] * s.c.hvs[:, :, None, None]
    else:
        s.k[..., 0] = 0.0
        s.k[:, :, 3] = 0.0
        s.k[:, :, 3, 0] = nats / scale / 4.0
        s.v[:, :, 3] = 0.0
        s.hk, s.hv = s.k.double().cpu().numpy(), s.v.double().cpu().numpy()
    lens = [50 * bs, 33 * bs + 7, 4]
    tables = _tables(60, lens, bs, 3)
    q = _rows(4, (len(lens), H * G, D), "bf16" if kv == "bf16" else "f16") * 0.1
    q[..., 0] = 4.0
    out, sel, _ = s.call(q, tables, lens, budget, scale)
    got, qh, sh = out.double().cpu().numpy(), q.double().cpu().numpy(), sel.cpu().numpy()
    for b, n in enumerate(lens):
        nb = -(-n // bs)
        for h in range(H):
            at = sh[b, h][sh[b, h] >= 0]
            m = len(at) * bs - (nb * bs - n)
            hold(got[b, h * G:(h + 1) * G], qh[b, h * G:(h + 1) * G],
                 s.hk[tables[b, at], h].reshape(-1, D)[:m],
                 s.hv[tables[b, at], h].reshape(-1, D)[:m], scale,
                 # bf16: three parts of 8 bits, the third off by half a step of what the first
                 # two leave: 2^-27; its exponents are fp32's
                 **({"floor": 0.0, "parts": 2.0 ** -27} if kv == "bf16" else {}))


# ------------------------------------------------------------------ V scales that are far apart
@pytest.mark.parametrize("D,bs", [(128, 16), (64, 16), (64, 8), (128, 8), (64, 32)])
@pytest.mark.parametrize("far", [5, 20, 24, 60, 100])
def test_blocks_of_far_larger_scales_and_no_value(D, bs, far):
    # attended codes of 0 under a large scale: what made the scale large is behind the length, or
    # was rounded away when an even larger row came
    H, G = 2, 4
    c = Cache(64, H, bs, D, seed=far, exp=(-9, -6))
    c.hvs[::3] *= 2.0 ** far
    c.hv[::3] = 0
    c.upload()
    lens = [60 * bs, 2 * bs, 21 * bs + 5, bs, 7]
    tables = np.stack([np.random.default_rng(b).permutation(64) for b in range(5)]).astype(np.int32)
    q = _rows(5, (5, H * G, D), "f16")
    out = _attend(c, q, tables, lens, 0.09)
    check(c, q, tables, lens, 0.09, out, floor=floor_of(bs))


@pytest.mark.parametrize("D,bs", [(128, 8), (64, 8), (64, 16)])
def test_scales_of_every_distance(D, bs):
    H, G = 1, 2
    c = Cache(64, H, bs, D, seed=9, exp=(-9, -6))
    c.hvs[:] = np.exp2(np.random.default_rng(1).integers(-60, 60, c.hvs.shape))
    c.upload()
    lens = [bs * n for n in (1, 2, 3, 4, 7, 40)] + [5, bs + 3]
    tables = np.stack([np.random.default_rng(b).permutation(64) for b in range(len(lens))])
    q = _rows(5, (len(lens), H * G, D), "f16")
    out = _attend(c, q, tables.astype(np.int32), lens, 0.09)
    check(c, q, tables, lens, 0.09, out, floor=floor_of(bs))


# ---------------------------------------------------------------------- the ends of fp32's range
@pytest.mark.parametrize("lens", [[100, 16, 1], [2000, 40, 900]])
@pytest.mark.parametrize("kexp,amp,scale", [
    (100, 2.0 ** -98, 0.09), (115, 2.0 ** -100, 2.0 ** -11), (112, 2.0 ** -110, 0.09),
    (118, 2.0 ** -117, 0.09), (-60, 2.0 ** 60, 0.09), (-85, 2.0 ** 85, 0.09),
    (30, 2.0 ** 90, 2.0 ** -125)])
def test_key_scales_of_any_size(kexp, amp, scale, lens):
    # scores of ordinary size from keys and queries that are not
    c = Cache(130, 2, 16, 128, seed=4)
    c.hks[:] = np.exp2(np.random.default_rng(1).integers(kexp - 9, kexp - 6, c.hks.shape))
    c.upload()
    tables = _batch(c, lens, 5, extra=0)
    q = _rows(3, (3, 8, 128), "bf16", amp)
    out = _attend(c, q, tables, lens, scale)
    check(c, q, tables, lens, scale, out)


def test_zero_scores_of_the_largest_scales():
    # q . k is 0 where q's one channel meets codes of 0, whatever the scales are
    c = Cache(20, 1, 16, 64, seed=4)
    c.hk[..., 0] = 0
    c.hks[:] = 2.0 ** 119
    c.upload()
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 2.0 ** 120
    tables = _batch(c, [200, 17], 5, extra=0)
    out = _attend(c, q, tables, [200, 17], 0.125)
    check(c, q, tables, [200, 17], 0.125, out)


def test_scores_below_fp32s_range_weigh_nothing():
    # whole tiles at the front, then one in the middle, score -inf in fp32
    c = Cache(200, 1, 16, 64, seed=4, exp=(-9, -6))
    c.hk[:, :, :, 0] = R.e4m3_encode(np.zeros(1))[0]
    far = np.r_[0:12, 30:33]
    c.hk[far, :, :, 0] = R.e4m3_encode(np.array([-448.0]))[0]
    c.hk[far, :, :, 1:] = 0
    c.hks[far] = 2.0 ** 119
    c.upload()
    lens = [190 * 16, 13 * 16, 12 * 16 + 1]
    tables = np.stack([np.arange(200)] * 3).astype(np.int32)
    q = _rows(3, (3, 4, 64), "bf16")
    q[..., 0] = 64.0
    out = _attend(c, q, tables, lens, 1.0)
    got, qh = out.double().cpu().numpy(), q.double().cpu().numpy()
    for b, n in enumerate(lens):
        k, v = c.rows(tables[b, :-(-n // 16)], 0, n, "k"), c.rows(tables[b, :-(-n // 16)], 0, n, "v")
        at = ~np.isin(np.arange(n) // 16, far)
        hold(got[b], qh[b], k[at], v[at], 1.0)
    assert pkv.pkv_check_error(c.pool) == pkv.PKV_OK


@pytest.mark.parametrize("lens", [[30], [3000], [4800, 900, 17]])
def test_values_near_fp32s_largest(lens):
    # their mean is in range, their weighted sum is not
    c = Cache(300, 1, 16, 128, seed=4, exp=(-9, -6))
    c.hvs[:] = 2.0 ** 119
    c.hv[:] = np.where(c.hv & 128, c.hv, 126 - c.hv % 20)
    c.upload()
    tables = _batch(c, lens, 5, extra=0)
    q = _rows(3, (len(lens), 4, 128), "f16")
    out = _attend(c, q, tables, lens, 0.09)
    check(c, q, tables, lens, 0.09, out)
