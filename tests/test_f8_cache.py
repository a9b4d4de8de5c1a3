"""8-bit float caches (e4m3 codes, one power-of-two scale for each block and KV
head): append, attention and the calls around them, against float64 references."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_reference as R
from paged_kv_cache_273_gb300 import pkv

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- CPU
def test_reference_codes_are_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(R.E4M3))
    assert np.array_equal(t[~np.isnan(t)], R.E4M3[~np.isnan(t)])
    x = np.concatenate([np.linspace(-448, 448, 20001), np.random.default_rng(0).normal(size=5000) * 0.02,
                        np.array([2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 0.0])])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = R.e4m3_encode(x.astype(np.float32))
    assert np.array_equal(R.E4M3[got], R.E4M3[want])


def test_reference_exponents():
    assert R.exponent(448.0, 448.0) == 0 and R.exponent(448.1, 448.0) == 1
    assert R.exponent(224.0, 448.0) == -1 and R.exponent(0.0, 448.0) == -96
    assert R.exponent(2.0 ** -120, 448.0) == -96 and R.exponent(3e38, 448.0) == 120
    assert R.exponent(127.0, 127.0) == 0 and R.exponent(127.5, 127.0) == 1


def test_pool_and_sizes():
    p = pkv.kv_block_pool_init(10, 16, 8, 128, pkv.PKV_F8)
    assert pkv.kv_cache_bytes(p) == 10 * 8 * 16 * 128
    assert pkv.kv_scales_bytes(p) == 10 * 8 * 4
    k, v, ks, vs = p.alloc_cache(device="cpu")
    assert k.dtype == torch.float8_e4m3fn and k.shape == (10, 8, 16, 128)
    assert ks.dtype == torch.float32 and ks.shape == (10, 8)
    for args in [(16, 4, 8, 128, pkv.PKV_F8), (16, 16, 8, 96, pkv.PKV_F8)]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.kv_block_pool_init(*args)
        assert e.value.status == pkv.PKV_ERR_UNSUPPORTED


def test_refusals():
    lib = pkv.load()
    pool = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_F8)
    buf = (ctypes.c_uint8 * 4096)()
    a = (ctypes.addressof(buf) + 15) // 16 * 16
    inv, uns = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED

    def append(dt=pkv.PKV_F16, ks=a, vs=a, n=1):
        return lib.kv_append(pool.handle, a, a, dt, a, n, a, a, ks, vs, None)
    assert append(dt=pkv.PKV_I8) == uns and append(dt=pkv.PKV_F8) == uns
    assert append(ks=None) == inv and append(vs=None) == inv and append(ks=a + 4) == inv
    assert append(n=0) == pkv.PKV_OK

    def attend(qdt=pkv.PKV_F16, hq=4, ks=a, ws=1 << 30, batch=1, window=0):
        return lib.paged_decode_attention_window(pool.handle, a, qdt, hq, a, a, ks, a, a, 2, a,
                                                 batch, 32, window, 1.0, a, a, ws, None)
    assert attend(qdt=pkv.PKV_F32) == uns and attend(qdt=pkv.PKV_F8) == uns
    assert attend(hq=6) == uns and attend(hq=3) == inv and attend(ks=None) == inv
    assert attend(ws=8) == inv and attend(batch=4097) == uns and attend(window=-1) == inv
    assert attend(batch=0) == pkv.PKV_OK
    assert lib.paged_prefill_attention(pool.handle, a, 4, a, a, a, 2, a, a, 1, 1, 1.0, a,
                                       None) == uns
    assert lib.paged_decode_attention_cascade(pool.handle, a, pkv.PKV_F16, 4, a, a, a, 2, a, 1, 32,
                                              a, a, a, a, 1, 1, 16, 1.0, a, a, 1 << 30,
                                              None) == uns


def test_binding_refuses_other_scales():
    pool = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_F8)
    k, v, ks, vs = pool.alloc_cache(device="cpu")
    x, s = torch.zeros(1, 2, 64, dtype=torch.float16), torch.zeros(1, dtype=torch.int32)
    for bad in (None, ks.half(), torch.zeros(8, 2, 16), torch.zeros(8)):
        with pytest.raises(ValueError):
            pkv.kv_append(pool, x, x, s, k, v, bad, vs)
        with pytest.raises(ValueError):
            pkv.kv_append(pool, x, x, s, k, v, ks, bad)
        with pytest.raises(ValueError):
            pkv.paged_decode_attention(pool, torch.zeros(1, 4, 64, dtype=torch.float16), k, v,
                                       torch.zeros(1, 2, dtype=torch.int32), s, 1.0,
                                       torch.zeros(1, 4, 64), torch.zeros(64, dtype=torch.uint8),
                                       32, bad, vs)


# ------------------------------------------------------------------------ append, GPU
class Cache:
    """An F8 pool with random codes and scales in every block, and its host copy."""

    def __init__(self, nb, H, bs, D, seed=0, exp=(-6, 3)):
        g = np.random.default_rng(seed)
        self.nb, self.H, self.bs, self.D = nb, H, bs, D
        self.pool = pkv.kv_block_pool_init(nb, bs, H, D, pkv.PKV_F8)
        self.k, self.v, self.ks, self.vs = self.pool.alloc_cache(DEV)
        self.hk, self.hv = (self._codes(g, (nb, H, bs, D)) for _ in range(2))
        self.hks, self.hvs = (np.exp2(g.integers(*exp, (nb, H))).astype(np.float64)
                              for _ in range(2))
        self.upload()

    @staticmethod
    def _codes(g, shape):
        c = g.integers(0, 256, shape).astype(np.uint8)
        return np.where((c & 127) == 127, c & 128, c).astype(np.uint8)

    def upload(self):
        for d, h in ((self.k, self.hk), (self.v, self.hv)):
            d.view(torch.uint8).copy_(torch.from_numpy(h))
        self.ks.copy_(torch.from_numpy(self.hks))
        self.vs.copy_(torch.from_numpy(self.hvs))

    def append(self, k, v, slots):
        pkv.kv_append(self.pool, k, v, torch.tensor(slots, dtype=torch.int32, device=DEV), self.k,
                      self.v, self.ks, self.vs)
        ok = [s if s < self.nb * self.bs else -1 for s in slots]
        R.append_f8(k.double().cpu().numpy(), ok, self.bs, self.hk, self.hks)
        R.append_f8(v.double().cpu().numpy(), ok, self.bs, self.hv, self.hvs)

    def same(self):
        for d, h, ds, hs in ((self.k, self.hk, self.ks, self.hks),
                             (self.v, self.hv, self.vs, self.hvs)):
            assert np.array_equal(ds.double().cpu().numpy(), hs)
            got = d.view(torch.uint8).cpu().numpy()
            assert np.array_equal(R.E4M3[got], R.E4M3[h], equal_nan=True)

    def rows(self, ids, h, n, which):
        c, s = (self.hk, self.hks) if which == "k" else (self.hv, self.hvs)
        x = R.E4M3[c[ids, h]] * np.maximum(s[ids, h], 2.0 ** -96)[:, None, None]
        return x.reshape(-1, self.D)[:n]


def _rows(seed, shape, dt, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * amp
    return x.to(DT[dt]).to(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("D,H,bs,dt", [(128, 8, 16, "bf16"), (64, 3, 8, "f16"), (128, 1, 64, "f32"),
                                       (64, 12, 256, "bf16"), (128, 2, 32, "f16")])
def test_append_runs(D, H, bs, dt):
    c = Cache(12, H, bs, D, seed=bs)
    # a block begun, continued with larger and with smaller rows, gone back in, and a
    # neighbouring block; padding between runs
    h = bs // 2
    steps = [([3 * bs + i for i in range(h)], 1.0),
             ([3 * bs + h], 7.0), ([3 * bs + h + 1], 0.001), ([3 * bs + 1, 3 * bs + 2], 40.0),
             ([5 * bs + i for i in range(bs)] + [-1] + [7 * bs + bs - 1] + [0], 0.3),
             ([-1, 9 * bs + 1, -1, -1, 2 * bs + i] if (i := 0) == 0 else [], 1e-12)]
    for n, (slots, amp) in enumerate(steps):
        T = len(slots)
        c.append(_rows(n, (T, H, D), dt, amp if dt != "f16" else max(amp, 1e-4)),
                 _rows(n + 50, (T, H, D), dt, 3.0), slots)
        c.same()
    assert pkv.pkv_check_error(c.pool) == pkv.PKV_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_append_extremes(dt):
    # zeros, the smallest and the largest values, exactly representable limits
    c = Cache(4, 1, 8, 64, seed=3)
    big = 3.3e38 if dt == "f32" else 3.38e38
    for i, vals in enumerate([[0.0], [448.0, -448.0], [448.0 * 2 ** 10, 1e-3], [1e-40, 0.0],
                              [big, -big, 1.0], [2.0 ** -110, -2.0 ** -100], [464.0, 1.0]]):
        x = torch.zeros(2, 1, 64)
        x[0, 0, :len(vals)] = torch.tensor(vals)
        x = x.to(DT[dt]).to(DEV)
        c.append(x, -x, [8 * (i % 4), 8 * (i % 4) + 1])
        c.same()
        c.append(-x, x, [8 * (i % 4) + 2, 8 * (i % 4) + 3])
        c.same()


@pytest.mark.gpu
def test_append_bulk_prompts_with_padding():
    # enough rows for the many-tokens-a-warp form; ragged sequences, one continuing a block
    g = np.random.default_rng(7)
    H, bs, D = 8, 16, 128
    lens = [1000, 1, 15, 16, 17, 333, 2000]
    nblk = [-(-n // bs) for n in lens]
    ids = g.permutation(sum(nblk) + 5)
    c = Cache(sum(nblk) + 5, H, bs, D, seed=8)
    slots, at = [], 0
    for n, m in zip(lens, nblk):
        mine = ids[at:at + m]
        at += m
        first = 5 if n == 333 else 0
        slots += [int(mine[p // bs]) * bs + p % bs for p in range(first, n)] + [-1] * 3
    slots += [len(ids) * bs, -7]                          # out of range: recorded, skipped
    T = len(slots)
    c.append(_rows(1, (T, H, D), "bf16"), _rows(2, (T, H, D), "bf16", 5.0), slots)
    c.same()
    assert pkv.pkv_check_error(c.pool) == pkv.PKV_ERR_BAD_INDEX


@pytest.mark.gpu
def test_block_copy_takes_the_scales_along():
    c = Cache(9, 3, 8, 64, seed=11)
    src = torch.tensor([1, 4], dtype=torch.int32, device=DEV)
    dst = torch.tensor([7, 0], dtype=torch.int32, device=DEV)
    pkv.kv_block_copy(c.pool, src, dst, c.k, c.v, c.ks, c.vs)
    for a in (c.hk, c.hv, c.hks, c.hvs):
        a[[7, 0]] = a[[1, 4]]
    c.same()


# ------------------------------------------------------------------------ decode, GPU
def _batch(c, lens, seed, extra=2):
    """Random tables for `lens` over the cache's blocks (blocks may be shared)."""
    g = np.random.default_rng(seed)
    maxb = max(1, max(-(-n // c.bs) for n in lens)) + extra
    t = g.integers(0, c.nb, (len(lens), maxb)).astype(np.int32)
    return t


def _attend(c, q, tables, lens, scale, window=0, **kw):
    B, Hq, D = q.shape
    out = torch.full((B, Hq, D), 7.0, device=DEV)
    ws = kw.get("ws")
    ws = pkv.alloc_workspace(c.pool, B, Hq) if ws is None else ws
    pkv.paged_decode_attention_window(c.pool, q, c.k, c.v, torch.from_numpy(tables).to(DEV),
                                      torch.tensor(lens, dtype=torch.int32, device=DEV), scale,
                                      out, ws, max(lens) if len(lens) else 0, window, c.ks, c.vs)
    assert not ws[:B * c.H * 4].any().item()              # the counters are left zero
    return out


def _check(c, q, tables, lens, scale, out, window=0, seqs=None):
    got = out.double().cpu().numpy()
    qh = q.double().cpu().numpy()
    G = q.shape[1] // c.H
    for b in range(len(lens)) if seqs is None else seqs:
        n = lens[b]
        ids = tables[b, :-(-n // c.bs)]
        lo = max(0, n - window) if window else 0
        for h in range(c.H):
            want, tol = R.attend(qh[b, h * G:(h + 1) * G], c.rows(ids, h, n, "k")[lo:],
                                 c.rows(ids, h, n, "v")[lo:], float(np.float32(scale)))
            err = np.abs(got[b, h * G:(h + 1) * G] - want).max()
            assert err <= tol, (b, h, n, err, tol)
    assert pkv.pkv_check_error(c.pool) == pkv.PKV_OK


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [8, 16, 64])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_decode_shapes(D, G, bs, dt):
    H = 2
    c = Cache(60, H, bs, D, seed=D + G + bs, exp=(-9, -6))
    lens = [0, 1, 15, 16, 17, 31, 33, bs, bs + 1, 0, 255, 700, 2]
    tables = _batch(c, lens, bs)
    q = _rows(G, (len(lens), H * G, D), dt, 2.0)
    out = _attend(c, q, tables, lens, 1 / math.sqrt(D))
    _check(c, q, tables, lens, 1 / math.sqrt(D), out)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 5, 16, 100, 1000])
@pytest.mark.parametrize("bs", [8, 32])
def test_decode_window_looks_at_no_earlier_block(window, bs):
    c = Cache(50, 2, bs, 128, seed=5, exp=(-9, -6))
    lens = [1, 40, 333, 600, 0]
    tables = _batch(c, lens, 6)
    for b, n in enumerate(lens):                         # entries before the window: not ids
        tables[b, :max(0, n - window) // bs] = -1 if b % 2 else 10 ** 6
    q = _rows(1, (5, 8, 128), "bf16", 2.0)
    out = _attend(c, q, tables, lens, 0.1, window)
    safe = np.where((tables < 0) | (tables >= c.nb), 0, tables)
    _check(c, q, safe, lens, 0.1, out, window)


@pytest.mark.gpu
def test_decode_rows_outside_a_sequence_may_hold_anything():
    c = Cache(8, 1, 16, 64, seed=2, exp=(-9, -6))
    lens, tables = [5, 19], np.array([[1, 2], [3, 4]], np.int32)
    c.hk[1, :, 5:], c.hv[1, :, 5:] = 0x7F, 0xFF           # NaN codes behind the last row
    c.hk[4, :, 3:], c.hv[4, :, 3:] = 0xFF, 0x7F
    c.upload()
    q = _rows(3, (2, 4, 64), "f16")
    out = _attend(c, q, tables, lens, 0.125)
    _check(c, q, tables, lens, 0.125, out)


@pytest.mark.gpu
@pytest.mark.parametrize("top", [21, 61])
def test_decode_far_apart_scales(top):
    # blocks whose V differ by 2^60 and more, keys whose scores decide which counts; blocks never
    # written (scale 0) read as zeros
    c = Cache(12, 2, 16, 128, seed=4)
    c.hvs[:] = np.exp2(np.random.default_rng(1).integers(-40, top, c.hvs.shape))
    c.hks[:] = 2.0 ** -9
    c.hk[10], c.hv[10], c.hks[10], c.hvs[10] = 0, 0, 0.0, 0.0
    c.upload()
    lens = [16 * 7, 100, 16]
    tables = np.array([[0, 1, 2, 3, 4, 5, 6], [7, 8, 10, 9, 10, 11, 1], [10] * 7], np.int32)
    q = _rows(3, (3, 4, 128), "bf16")
    out = _attend(c, q, tables, lens, 0.09)
    _check(c, q, tables, lens, 0.09, out)


@pytest.mark.gpu
@pytest.mark.parametrize("amp", [1e-30, 1e-4, 300.0, 1e30])
def test_decode_bf16_queries_of_any_size(amp):
    c = Cache(12, 1, 16, 64, seed=4, exp=(-9, -6))
    lens, tables = [90, 3], np.array([[0, 1, 2, 3, 4, 5], [6, 0, 0, 0, 0, 0]], np.int32)
    q = _rows(3, (2, 2, 64), "bf16", amp)
    q[1, 1] = 0
    out = _attend(c, q, tables, lens, 1.0 / amp)
    _check(c, q, tables, lens, 1.0 / amp, out)


@pytest.mark.gpu
def test_decode_long_and_ragged():
    c = Cache(3000, 4, 16, 128, seed=12, exp=(-9, -6))
    g = np.random.default_rng(3)
    lens = [40000, 1, 0, 7000, 12345] + g.integers(0, 600, 40).tolist()
    tables = _batch(c, lens, 5, extra=0)
    q = _rows(1, (len(lens), 16, 128), "f16", 1.5)
    out = _attend(c, q, tables, lens, 0.088)
    _check(c, q, tables, lens, 0.088, out, seqs=[0, 1, 2, 3, 5, 17, 30, 44])
    again = _attend(c, q, tables, lens, 0.088)
    assert torch.equal(out, again)                        # no order that timing decides


@pytest.mark.gpu
def test_decode_largest_batch():
    c = Cache(300, 1, 8, 64, seed=12, exp=(-9, -6))
    lens = np.random.default_rng(3).integers(0, 20, 4096).tolist()
    tables = _batch(c, lens, 5, extra=0)
    q = _rows(1, (4096, 8, 64), "f16", 1.5)
    out = _attend(c, q, tables, lens, 0.125)
    _check(c, q, tables, lens, 0.125, out, seqs=range(0, 4096, 97))


@pytest.mark.gpu
@pytest.mark.parametrize("G", [1, 8])
def test_decode_of_empty_sequences_only(G):
    c = Cache(4, 2, 16, 128, seed=1)
    q = _rows(1, (7, 2 * G, 128), "bf16")
    out = _attend(c, q, np.zeros((7, 1), np.int32), [0] * 7, 0.1)
    assert not out.any().item()
    assert pkv.pkv_check_error(c.pool) == pkv.PKV_OK


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1], [5] * 9, [16] * 200, [300] * 152, [300] * 153, [2000] * 19,
                                  [2000] * 20 + [1900], [513] * 40 + [0], [97] * 3 + [4000]])
def test_decode_splits(lens):
    # whole pieces a CTA, shared ones, and the borders between the two
    c = Cache(500, 1, 16, 128, seed=7, exp=(-9, -6))
    tables = _batch(c, lens, 3)
    q = _rows(2, (len(lens), 4, 128), "bf16", 1.5)
    out = _attend(c, q, tables, lens, 0.09)
    _check(c, q, tables, lens, 0.09, out, seqs=range(0, len(lens), max(1, len(lens) // 7)))


@pytest.mark.gpu
def test_decode_bad_inputs_are_recorded():
    c = Cache(8, 2, 16, 64, seed=2, exp=(-9, -6))
    q = _rows(3, (4, 4, 64), "f16")
    tables = np.array([[1, 2], [3, 8], [5, 6], [7, -1]], np.int32)
    lens = torch.tensor([20, 20, 20, 10], dtype=torch.int32, device=DEV)
    ws = pkv.alloc_workspace(c.pool, 4, 4)
    out = torch.zeros(4, 4, 64, device=DEV)

    def call(lens, max_len=32):
        pkv.paged_decode_attention(c.pool, q, c.k, c.v, torch.from_numpy(tables).to(DEV), lens,
                                   0.125, out, ws, max_len, c.ks, c.vs)
        return pkv.pkv_check_error(c.pool)
    assert call(lens) == pkv.PKV_ERR_BAD_INDEX            # block 8 of sequence 1
    good = [0, 2, 3]
    full = out.clone()
    tables[1, 1] = 0
    assert call(lens) == pkv.PKV_OK
    assert torch.equal(full[good], out[good])
    bad = lens.clone()
    bad[2] = 33
    assert call(bad) == pkv.PKV_ERR_BAD_INDEX
    # (the rounding goes by how the whole batch's tiles are shared out: held to the bound)
    _check(c, q, tables, lens.tolist(), 0.125, out, seqs=[0, 3])
    bad[2] = -1
    assert call(bad) == pkv.PKV_ERR_BAD_INDEX
    assert call(lens, max_len=19) == pkv.PKV_ERR_BAD_INDEX


@pytest.mark.gpu
def test_step_and_noalloc_take_f8_pools():
    B, H, G, D, bs = 5, 2, 4, 128, 16
    c = Cache(40, H, bs, D, seed=21, exp=(-9, -6))
    g = np.random.default_rng(2)
    lens = np.array([33, 1, 16, 64, 20], np.int32)        # after the append
    tables = g.permutation(40)[:B * 4].reshape(B, 4).astype(np.int32)
    slots = [int(tables[b, (lens[b] - 1) // bs]) * bs + int(lens[b] - 1) % bs for b in range(B)]
    q, k, v = (_rows(i, (B, h, D), "bf16") for i, h in ((1, H * G), (2, H), (3, H)))
    tables_d = torch.from_numpy(tables).to(DEV)
    nkv, nq = B * H * D * 2, B * H * G * D * 2
    lay = pkv.StepLayout(0, nkv, 2 * nkv, 2 * nkv + nq, 2 * nkv + nq + 32)
    host = torch.zeros(2 * nkv + nq + 64, dtype=torch.uint8).pin_memory()
    for off, t in ((0, k), (nkv, v), (2 * nkv, q)):
        b = t.cpu().contiguous().view(torch.uint8).reshape(-1)
        host[off:off + b.numel()] = b
    host[lay.slot_mapping:lay.slot_mapping + 4 * B] = torch.tensor(slots, dtype=torch.int32).view(torch.uint8)
    host[lay.seq_lens:lay.seq_lens + 4 * B] = torch.from_numpy(lens).view(torch.uint8)
    dev_in = torch.zeros_like(host, device=DEV)
    out = torch.zeros(B, H * G, D, device=DEV)
    ws = pkv.alloc_workspace(c.pool, B, H * G)
    pkv.paged_decode_step(c.pool, host, dev_in, lay, torch.bfloat16, torch.bfloat16, H * G, c.k,
                          c.v, tables_d, B, 64, 0.09, out, None, ws, c.ks, c.vs)
    R.append_f8(k.double().cpu().numpy(), slots, bs, c.hk, c.hks)
    R.append_f8(v.double().cpu().numpy(), slots, bs, c.hv, c.hvs)
    c.same()
    _check(c, q, tables, lens.tolist(), 0.09, out)
    out2 = torch.zeros_like(out)
    pkv.paged_decode_attention_noalloc(c.pool, q, c.k, c.v, tables_d,
                                       torch.from_numpy(lens).to(DEV), 0.09, out2, 64, c.ks, c.vs)
    assert torch.equal(out, out2)


@pytest.mark.gpu
def test_one_workspace_for_calls_of_every_batch():
    # sized for the largest of them; each call's scratch must leave the others' counters alone
    c = Cache(300, 2, 16, 128, seed=41, exp=(-9, -6))
    ws = pkv.alloc_workspace(c.pool, 300, 16)
    g = np.random.default_rng(1)
    for B, top in ((1, 4000), (300, 200), (7, 3000), (1, 4800), (150, 700), (3, 4800), (300, 400)):
        lens = g.integers(0, top + 1, B).tolist()
        lens[0] = top
        tables = _batch(c, lens, B)
        q = _rows(B, (B, 16, 128), "bf16", 1.5)
        out = _attend(c, q, tables, lens, 0.09, ws=ws)
        assert not ws[:4 * 2 * 4096].any().item()
        _check(c, q, tables, lens, 0.09, out, seqs=range(0, B, max(1, B // 5)))


@pytest.mark.gpu
def test_caches_beyond_4_gib():
    # the last blocks of caches of 5 GB: append, bounds, attention, attention over chosen blocks
    NB, H, bs, D, G = 310000, 8, 16, 128, 4
    pool = pkv.kv_block_pool_init(NB, bs, H, D, pkv.PKV_F8)
    assert pkv.kv_cache_bytes(pool) > 2 ** 32
    k, v, ks, vs = pool.alloc_cache(DEV)
    bounds, exps = pkv.alloc_bounds(pool, DEV)
    ids = np.array([NB - 1, 5, NB - 3, NB - 2, NB - 7], np.int32)
    n = 75
    slots = [int(ids[p // bs]) * bs + p % bs for p in range(n)]
    kn, vn = _rows(1, (n, H, D), "bf16"), _rows(2, (n, H, D), "bf16", 2.0)
    sd = torch.tensor(slots, dtype=torch.int32, device=DEV)
    pkv.kv_append(pool, kn, vn, sd, k, v, ks, vs)
    pkv.kv_bounds_append(pool, kn, sd, bounds, exps)
    # the same in a pool of the five blocks alone
    small = Cache(5, H, bs, D)
    where = {int(b): i for i, b in enumerate(ids)}
    small.append(kn, vn, [where[s // bs] * bs + s % bs for s in slots])
    idl = torch.from_numpy(ids.astype(np.int64)).to(DEV)
    got = k.view(torch.uint8)[idl].cpu().numpy()
    off = n % bs                                          # the last block's unwritten rows differ
    assert np.array_equal(got[:4], small.hk[:4]) and np.array_equal(got[4, :, :off],
                                                                    small.hk[4, :, :off])
    assert np.array_equal(ks[idl].double().cpu().numpy(), small.hks)
    hb, he = np.zeros((5, H, 2, D), np.int8), np.zeros((5, H), np.int32)
    R.append_bounds(kn.double().cpu().numpy(), [where[s // bs] * bs + s % bs for s in slots], bs,
                    hb, he)
    assert np.array_equal(bounds[idl].cpu().numpy(), hb)
    assert np.array_equal(exps[idl].cpu().numpy(), he)
    q = _rows(3, (1, H * G, D), "bf16", 1.5)
    out = torch.zeros(1, H * G, D, device=DEV)
    td, ld = torch.from_numpy(ids[None]).to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    pkv.paged_decode_attention(pool, q, k, v, td, ld, 0.09, out, pkv.alloc_workspace(pool, 1, H * G),
                               n, ks, vs)
    _check(small, q, np.arange(5, dtype=np.int32)[None], [n], 0.09, out)
    sel = torch.zeros(1, H, 2, dtype=torch.int32, device=DEV)
    pkv.paged_decode_attention_sparse(pool, q, k, v, bounds, exps, td, ld, 0.09, out, sel,
                                      pkv.alloc_sparse_workspace(pool, 1, H * G, n, 2), n, ks, vs)
    qh, sh, oh = q.double().cpu().numpy(), sel.cpu().numpy(), out.double().cpu().numpy()
    for h in range(H):
        want = R.choose(qh[0, h * G:(h + 1) * G], np.arange(5), hb, he, h, 2)
        assert sh[0, h].tolist() == want.tolist()
        m = len(want) * bs - (5 * bs - n)
        o, tol = R.attend(qh[0, h * G:(h + 1) * G], small.rows(want, h, m, "k"),
                          small.rows(want, h, m, "v"), float(np.float32(0.09)))
        assert np.abs(oh[0, h * G:(h + 1) * G] - o).max() <= tol
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK


@pytest.mark.gpu
def test_graphs_that_share_a_workspace():
    # two captured calls on one workspace, replayed one after another, on a stream of their own
    c = Cache(400, 2, 16, 128, seed=31, exp=(-9, -6))
    lens = [3000, 17, 900]
    tables = _batch(c, lens, 1, extra=0)
    td, ld = torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = pkv.alloc_workspace(c.pool, 3, 16)
    qs = [_rows(i, (3, 16, 128), "bf16") for i in range(2)]
    outs = [torch.zeros(3, 16, 128, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for q, out in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pkv.paged_decode_attention(c.pool, q, c.k, c.v, td, ld, 0.09, out, ws, 3000, c.ks, c.vs)
        graphs.append(g)
    with torch.cuda.stream(side):
        for _ in range(5):
            for g in graphs:
                g.replay()
    side.synchronize()
    for q, out in zip(qs, outs):
        _check(c, q, tables, lens, 0.09, out)
