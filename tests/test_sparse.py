"""Key bounds and the attention over chosen blocks: bounds and choice exactly,
the attention against float64 over the rows that the choice gives."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_reference as R
from paged_kv_cache_273_gb300 import pkv
from test_f8_cache import Cache, DEV, DT, _rows

KV = {"f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16, "f8": pkv.PKV_F8}


# --------------------------------------------------------------------------- CPU
def test_refusals():
    lib = pkv.load()
    buf = (ctypes.c_uint8 * 4096)()
    a = (ctypes.addressof(buf) + 15) // 16 * 16
    inv, uns = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED
    pool = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_F16)

    def bounds(p=pool.handle, dt=pkv.PKV_F16, k=a, s=a, n=1, b=a, e=a):
        return lib.kv_bounds_append(p, k, dt, s, n, b, e, None)
    assert bounds(p=None) == inv and bounds(n=-1) == inv and bounds(dt=pkv.PKV_I8) == uns
    assert bounds(k=None) == inv and bounds(s=None) == inv and bounds(b=None) == inv
    assert bounds(e=None) == inv and bounds(k=a + 2) == inv and bounds(b=a + 8) == inv
    assert bounds(e=a + 2) == inv and bounds(n=0) == pkv.PKV_OK

    def sparse(p=pool, qdt=pkv.PKV_F16, hq=4, b=a, e=a, sel=a, n=2, ws=1 << 30, batch=1, ks=None,
               out=a, bt=a):
        return lib.paged_decode_attention_sparse(p.handle, a, qdt, hq, a, a, ks, ks, b, e, bt, 2,
                                                 a, batch, 32, n, 1.0, out, sel, a, ws, None)
    assert sparse(n=0) == inv and sparse(b=None) == inv and sparse(e=None) == inv
    assert sparse(sel=None) == inv and sparse(b=a + 4) == inv and sparse(sel=a + 1) == inv
    assert sparse(qdt=pkv.PKV_BF16) == inv and sparse(hq=6) == uns and sparse(hq=3) == inv
    assert sparse(ws=300) == inv and sparse(batch=4097) == uns and sparse(out=None) == inv
    assert sparse(bt=None) == inv and sparse(batch=0) == pkv.PKV_OK
    for kv in (pkv.PKV_F32, pkv.PKV_I8):
        p = pkv.kv_block_pool_init(8, 16, 2, 64, kv)
        assert sparse(p=p, ks=a) == uns
    p8 = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_F8)
    assert sparse(p=p8) == inv and sparse(p=p8, ks=a, qdt=pkv.PKV_F32) == uns
    for bad in [(1, 3, 10, 2), (-1, 4, 10, 2), (1, 4, -1, 2), (1, 4, 10, 0)]:
        assert pkv.paged_sparse_workspace_bytes(pool, *bad) == 0


def test_workspace_grows_with_what_it_holds():
    pool = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_F16)
    w = pkv.paged_sparse_workspace_bytes
    base = w(pool, 4, 8, 1000, 8)
    # counters of the largest batch, the chosen ids, the scores of 63 blocks
    assert base >= 4 * 2 * (4096 + 4 * 8 + 4 * 63)
    assert w(pool, 8, 8, 1000, 8) > base and w(pool, 4, 8, 100000, 8) > base
    assert w(pool, 4, 8, 1000, 64) > base


def test_binding_refuses_shapes():
    pool = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_F16)
    b, e = pkv.alloc_bounds(pool, device="cpu")
    k, s = torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    for args in [(k[:, :1], s, b, e), (k, s[:2], b, e), (k, s.long(), b, e), (k, s, b[:4], e),
                 (k, s, b.float(), e), (k, s, b, e.long()), (k.double(), s, b, e)]:
        with pytest.raises(ValueError):
            pkv.kv_bounds_append(pool, *args)


def test_reference_bounds_do_not_depend_on_the_split():
    g = np.random.default_rng(0)
    k = g.normal(size=(16, 2, 8)) * np.exp2(g.integers(-9, 9, (16, 1, 1)))
    whole, we = np.zeros((1, 2, 2, 8), np.int8), np.zeros((1, 2), np.int32)
    R.append_bounds(k, range(16), 16, whole, we)
    for cuts in ([1] * 16, [3, 5, 8], [15, 1]):
        b, e, at = np.full((1, 2, 2, 8), 9, np.int8), np.full((1, 2), 7, np.int32), 0
        for n in cuts:
            R.append_bounds(k[at:at + n], range(at, at + n), 16, b, e)
            at += n
        assert np.array_equal(b, whole) and np.array_equal(e, we)
    lo, hi = whole[0, :, 0] * 2.0 ** we[0, :, None], whole[0, :, 1] * 2.0 ** we[0, :, None]
    assert (lo <= k.min(0)).all() and (hi >= k.max(0)).all()


# ------------------------------------------------------------------------ bounds, GPU
class Bounds:
    def __init__(self, pool, seed=0):
        g = np.random.default_rng(seed)
        self.pool, self.bs = pool, pool.block_size
        self.b, self.e = pkv.alloc_bounds(pool, DEV)
        self.hb = g.integers(-127, 128, self.b.shape).astype(np.int8)
        self.he = g.integers(-9, 3, self.e.shape).astype(np.int32)
        self.b.copy_(torch.from_numpy(self.hb))
        self.e.copy_(torch.from_numpy(self.he))

    def append(self, k, slots):
        pkv.kv_bounds_append(self.pool, k, torch.tensor(slots, dtype=torch.int32, device=DEV),
                             self.b, self.e)
        cap = self.pool.num_blocks * self.bs
        R.append_bounds(k.double().cpu().numpy(), [s if s < cap else -1 for s in slots], self.bs,
                        self.hb, self.he)

    def same(self):
        assert np.array_equal(self.e.cpu().numpy(), self.he)
        assert np.array_equal(self.b.cpu().numpy(), self.hb)


@pytest.mark.gpu
@pytest.mark.parametrize("D,H,bs,dt", [(128, 8, 16, "bf16"), (64, 3, 4, "f16"), (128, 1, 64, "f32"),
                                       (64, 12, 256, "bf16")])
def test_bounds_runs(D, H, bs, dt):
    pool = pkv.kv_block_pool_init(10, bs, H, D, pkv.PKV_BF16)
    s = Bounds(pool, bs)
    h = bs // 2
    for n, (slots, amp) in enumerate([([3 * bs + i for i in range(h)], 1.0), ([3 * bs + h], 9.0),
                                      ([3 * bs + h + 1], 1e-3), ([3 * bs + 1], 50.0),
                                      ([5 * bs + i for i in range(bs)] + [-1, 7 * bs + bs - 1, 0],
                                       0.2), ([8 * bs], 0.0), ([8 * bs + 1], 3.0)]):
        s.append(_rows(n, (len(slots), H, D), dt, amp), slots)
        s.same()
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK


@pytest.mark.gpu
def test_bounds_bulk_and_bad_slots():
    H, bs, D = 8, 16, 128
    pool = pkv.kv_block_pool_init(400, bs, H, D, pkv.PKV_F16)
    s = Bounds(pool, 1)
    g = np.random.default_rng(4)
    ids = g.permutation(400)
    slots, at = [], 0
    for n in (1500, 3, 16, 33, 4000):
        m = -(-n // bs)
        slots += [int(ids[at + p // bs]) * bs + p % bs for p in range(7 if n == 33 else 0, n)]
        slots += [-1]
        at += m
    slots += [400 * bs + 5]
    s.append(_rows(1, (len(slots), H, D), "f16"), slots)
    s.same()
    assert pkv.pkv_check_error(pool) == pkv.PKV_ERR_BAD_INDEX


# -------------------------------------------------------------- choice and attention, GPU
class Sparse:
    """A pool with random contents, bounds of them, and their host copies."""

    def __init__(self, kv, nb, H, bs, D, seed=0, corr=0.8, exps=None):
        self.kv, self.H, self.bs, self.D, self.nb = kv, H, bs, D, nb
        g = torch.Generator().manual_seed(seed)
        x = torch.randn(nb, H, bs, D, generator=g) * 0.6 + torch.randn(nb, H, 1, D, generator=g) * corr
        v = torch.randn(nb, H, bs, D, generator=g)
        self.hb, self.he = np.zeros((nb, H, 2, D), np.int8), np.zeros((nb, H), np.int32)
        if kv == "f8":
            self.c = Cache(nb, H, bs, D, seed)
            self.pool = self.c.pool
            for src, hc, hs in ((x, self.c.hk, self.c.hks), (v, self.c.hv, self.c.hvs)):
                am = src.abs().amax(dim=(2, 3)).double().numpy()
                e = np.vectorize(lambda a: R.exponent(a, 448.0))(am)
                hc[:] = R.e4m3_encode(src.double().numpy() * np.exp2(-e)[:, :, None, None])
                hs[:] = np.exp2(e)
            self.c.upload()
            self.k, self.v, self.ks, self.vs = self.c.k, self.c.v, self.c.ks, self.c.vs
            self.hk = R.E4M3[self.c.hk] * self.c.hks[:, :, None, None]
            self.hv = R.E4M3[self.c.hv] * self.c.hvs[:, :, None, None]
        else:
            self.pool = pkv.kv_block_pool_init(nb, bs, H, D, KV[kv])
            self.k, self.v = x.to(DT[kv]).to(DEV), v.to(DT[kv]).to(DEV)
            self.ks = self.vs = None
            self.hk, self.hv = self.k.double().cpu().numpy(), self.v.double().cpu().numpy()
        xh = x.double().numpy()
        lo, hi = xh.min(2), xh.max(2)
        e = np.vectorize(lambda a: R.exponent(a, 127.0))(np.maximum(-lo, hi).max(2))
        if exps is not None:
            e = exps(e)
        self.he[:] = e
        f = np.exp2(-e.astype(np.float64))[:, :, None]
        self.hb[:, :, 0] = np.clip(np.floor(lo * f), -128, 127)
        self.hb[:, :, 1] = np.clip(np.ceil(hi * f), -128, 127)
        self.b, self.e = torch.from_numpy(self.hb).to(DEV), torch.from_numpy(self.he).to(DEV)

    def sync(self):
        self.b.copy_(torch.from_numpy(self.hb))
        self.e.copy_(torch.from_numpy(self.he))

    def call(self, q, tables, lens, budget, scale, ws=None, max_len=None):
        B, Hq, D = q.shape
        m = max(lens) if max_len is None else max_len
        ws = pkv.alloc_sparse_workspace(self.pool, B, Hq, m, budget) if ws is None else ws
        out = torch.full((B, Hq, D), 7.0, device=DEV)
        sel = torch.full((B, self.H, budget), 77, dtype=torch.int32, device=DEV)
        pkv.paged_decode_attention_sparse(self.pool, q, self.k, self.v, self.b, self.e,
                                          torch.from_numpy(tables).to(DEV),
                                          torch.tensor(lens, dtype=torch.int32, device=DEV), scale,
                                          out, sel, ws, m, self.ks, self.vs)
        return out, sel, ws

    def check(self, q, tables, lens, budget, scale, out, sel, seqs=None):
        got, s = out.double().cpu().numpy(), sel.cpu().numpy()
        qh = q.double().cpu().numpy()
        G = q.shape[1] // self.H
        for b in range(len(lens)) if seqs is None else seqs:
            n = -(-lens[b] // self.bs)
            ids = tables[b, :n]
            for h in range(self.H):
                qq = qh[b, h * G:(h + 1) * G]
                want = R.choose(qq, ids, self.hb, self.he, h, budget) if n else np.zeros(0, int)
                assert s[b, h, :len(want)].tolist() == want.tolist(), (b, h)
                assert (s[b, h, len(want):] == -1).all()
                m = max(0, len(want) * self.bs - (n * self.bs - lens[b]))
                k = self.hk[ids[want], h].reshape(-1, self.D)[:m]
                v = self.hv[ids[want], h].reshape(-1, self.D)[:m]
                o, tol = R.attend(qq, k, v, float(np.float32(scale)),
                                  R.BF16_PARTS if self.kv == "bf16" else 2.0 ** -22)
                err = np.abs(got[b, h * G:(h + 1) * G] - o).max()
                assert err <= tol, (b, h, err, tol)
        assert pkv.pkv_check_error(self.pool) == pkv.PKV_OK


def _tables(nb, lens, bs, seed):
    g = np.random.default_rng(seed)
    return g.integers(0, nb, (len(lens), max(1, -(-max(lens) // bs)))).astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,bs", [("f16", 4), ("bf16", 16), ("f8", 8), ("f8", 32), ("bf16", 64)])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 2), (64, 4), (128, 4), (128, 8), (64, 8)])
def test_sparse_shapes(kv, bs, D, G):
    H = 3
    s = Sparse(kv, 80, H, bs, D, seed=bs + G)
    lens = [0, 1, bs, bs + 1, 7 * bs, 7 * bs + 3, 40 * bs - 1, 63 * bs + 2, 5]
    tables = _tables(80, lens, bs, 1)
    q = _rows(G, (len(lens), H * G, D), "bf16" if kv == "bf16" else "f16", 1.5)
    for budget in (1, 2, 7, 8, 100):
        out, sel, _ = s.call(q, tables, lens, budget, 1 / math.sqrt(D))
        s.check(q, tables, lens, budget, 1 / math.sqrt(D), out, sel)


@pytest.mark.gpu
def test_sparse_over_several_ctas_and_key_counts():
    # block counts of every form of the choice: 4, 8 and 32 keys a thread, and more than that
    s = Sparse("f16", 600, 1, 4, 64, seed=3)
    lens = [4 * 2049, 4 * 2050 + 1, 4 * 4097 + 2, 4 * 16385, 4 * 16386, 4 * 30000 + 3, 4 * 513]
    tables = _tables(600, lens, 4, 2)
    q = _rows(1, (len(lens), 2, 64), "f16", 1.5)
    for budget in (33, 700):
        out, sel, ws = s.call(q, tables, lens, budget, 0.125)
        s.check(q, tables, lens, budget, 0.125, out, sel)
        assert not ws[:len(lens) * 4].any().item()
        out2, sel2, _ = s.call(q, tables, lens, budget, 0.125, ws=ws)   # the workspace as left
        assert torch.equal(out, out2) and torch.equal(sel, sel2)


@pytest.mark.gpu
def test_sparse_equal_scores_take_the_lowest_index():
    s = Sparse("bf16", 64, 2, 16, 128, seed=5)
    s.hb[:], s.he[:] = 3, -2                              # every block scores the same
    s.hb[10], s.he[11] = 5, 0
    s.sync()
    lens = [16 * 40, 16 * 64, 16 * 9 + 1]
    tables = np.stack([np.random.default_rng(i).permutation(64) for i in range(3)]).astype(np.int32)
    q = _rows(1, (3, 8, 128), "bf16").abs()
    for budget in (2, 5, 39):
        out, sel, _ = s.call(q, tables, lens, budget, 0.09)
        s.check(q, tables, lens, budget, 0.09, out, sel)
    q.zero_()                                             # all scores zero
    out, sel, _ = s.call(q, tables, lens, 5, 0.09)
    s.check(q, tables, lens, 5, 0.09, out, sel)


@pytest.mark.gpu
def test_sparse_exponents_far_apart():
    # scores over the whole fp32 range, negative ones among them
    g = np.random.default_rng(2)
    s = Sparse("bf16", 64, 2, 16, 64, seed=6, exps=lambda e: e + g.integers(-80, 80, e.shape))
    s.hb[:, :, 1] = np.where(g.random((64, 2, 1)) < 0.5, -1, s.hb[:, :, 1])
    s.sync()
    lens = [16 * 64, 500]
    tables = np.stack([g.permutation(64) for _ in range(2)]).astype(np.int32)
    q = _rows(1, (2, 4, 64), "bf16")
    out, sel, _ = s.call(q, tables, lens, 9, 0.125)
    s.check(q, tables, lens, 9, 0.125, out, sel)


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi", [(105, 121), (-96, -80)])
def test_sparse_exponents_at_the_ends(lo, hi):
    # whole-number sums up to 2^21 in units of up to 2^120: scores beyond fp32's largest number
    g = np.random.default_rng(4)
    s = Sparse("bf16", 64, 2, 16, 128, seed=7, exps=lambda e: g.integers(lo, hi, e.shape))
    s.hb[:] = np.sort(g.integers(-127, 128, s.hb.shape), 2)
    s.sync()
    lens = [16 * 64, 900]
    tables = np.stack([g.permutation(64) for _ in range(2)]).astype(np.int32)
    q = _rows(1, (2, 16, 128), "bf16")
    for budget in (2, 9, 40):
        out, sel, _ = s.call(q, tables, lens, budget, 0.09)
        s.check(q, tables, lens, budget, 0.09, out, sel)


@pytest.mark.gpu
def test_sparse_scores_crowded_in_a_few_digits():
    # a few blocks far off, so that the thousands of others share the first digits of the search
    # for the last one chosen; many of them equal
    s = Sparse("f16", 400, 2, 4, 64, seed=16)
    s.he[:] = -3
    s.hb[:] = np.random.default_rng(3).integers(-2, 3, (1, 2, 2, 64))
    s.hb[:, :, 1] = np.maximum(s.hb[:, :, 0], s.hb[:, :, 1])
    s.hb[:, :, 1, 0] = np.maximum(s.hb[:, :, 0, 0], np.arange(400)[:, None] % 50)
    s.he[7], s.he[8], s.he[9] = 40, -90, 90
    s.hb[9, :, 0], s.hb[9, :, 1] = -100, -99             # far below all others or far above
    s.sync()
    lens = [4 * 6000 + 1, 4 * 3000, 4 * 20000]
    tables = _tables(400, lens, 4, 7)
    q = _rows(1, (3, 8, 64), "f16")
    for budget in (2, 300, 1500):
        out, sel, _ = s.call(q, tables, lens, budget, 0.125)
        s.check(q, tables, lens, budget, 0.125, out, sel)


@pytest.mark.gpu
def test_sparse_with_room_for_all_is_the_dense_call():
    s = Sparse("f8", 100, 4, 16, 128, seed=8)
    lens = [1000, 3, 0, 16, 777]
    tables = _tables(100, lens, 16, 4)
    q = _rows(1, (5, 16, 128), "bf16", 1.5)
    out, sel, _ = s.call(q, tables, lens, 63, 0.09)
    s.check(q, tables, lens, 63, 0.09, out, sel)
    dense = torch.zeros_like(out)
    pkv.paged_decode_attention(s.pool, q, s.k, s.v, torch.from_numpy(tables).to(DEV),
                               torch.tensor(lens, dtype=torch.int32, device=DEV), 0.09, dense,
                               pkv.alloc_workspace(s.pool, 5, 16), 1000, s.ks, s.vs)
    assert torch.equal(out, dense)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["f16", "f8"])
def test_one_workspace_for_calls_of_every_shape(kv):
    s = Sparse(kv, 200, 2, 8, 64, seed=18)
    ws = pkv.alloc_sparse_workspace(s.pool, 90, 8, 8 * 700, 40)
    g = np.random.default_rng(2)
    for B, top, budget in ((1, 5600, 40), (90, 900, 5), (2, 5600, 3), (40, 2000, 40), (90, 5600, 17)):
        lens = g.integers(0, top + 1, B).tolist()
        lens[0] = top
        tables = _tables(200, lens, 8, B)
        q = _rows(B, (B, 8, 64), "f16", 1.5)
        out, sel, _ = s.call(q, tables, lens, budget, 0.125, ws=ws)
        assert not ws[:4 * 2 * 4096].any().item()
        s.check(q, tables, lens, budget, 0.125, out, sel, seqs=range(0, B, max(1, B // 6)))
        if kv == "f8":                                    # the dense call's counters are the same
            pkv.paged_decode_attention(s.pool, q, s.k, s.v, torch.from_numpy(tables).to(DEV),
                                       torch.tensor(lens, dtype=torch.int32, device=DEV), 0.125,
                                       torch.zeros_like(out), ws, top, s.ks, s.vs)


@pytest.mark.gpu
def test_sparse_infinite_keys():
    # scores of -inf for whole tiles, and for all of a sequence but its last rows, weigh nothing
    s = Sparse("f16", 40, 1, 16, 64, seed=19)
    s.k[:30] = 0
    s.k[:30, :, :, 0] = -math.inf
    s.hk = s.k.double().cpu().numpy()
    q = _rows(3, (2, 4, 64), "f16").abs() + 0.1           # q > 0: q . k = -inf there
    lens = [31 * 16 + 5, 35 * 16]
    tables = np.stack([np.arange(40), np.arange(40)]).astype(np.int32)
    out, sel, _ = s.call(q, tables, lens, 40, 0.125)
    for b, n in enumerate(lens):
        o, tol = R.attend(q[b].double().cpu().numpy(), s.hk[30:, 0].reshape(-1, 64)[:n - 480],
                          s.hv[30:, 0].reshape(-1, 64)[:n - 480], 0.125)
        assert np.abs(out[b].double().cpu().numpy() - o).max() <= tol


@pytest.mark.gpu
def test_sparse_bad_inputs_are_recorded():
    s = Sparse("f16", 32, 2, 16, 64, seed=9)
    lens = [300, 300, 40]
    tables = _tables(32, lens, 16, 5)
    q = _rows(1, (3, 4, 64), "f16")
    good, gsel, _ = s.call(q, tables, lens, 6, 0.125)
    assert pkv.pkv_check_error(s.pool) == pkv.PKV_OK
    bad = tables.copy()
    bad[1, 4], bad[1, 18] = 32, -5                        # one not the newest, the newest
    out, sel, _ = s.call(q, bad, lens, 6, 0.125)
    assert pkv.pkv_check_error(s.pool) == pkv.PKV_ERR_BAD_INDEX
    assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.equal(sel[[0, 2]], gsel[[0, 2]])
    out, sel, _ = s.call(q, tables, [300, 305, 40], 6, 0.125, max_len=300)
    assert pkv.pkv_check_error(s.pool) == pkv.PKV_ERR_BAD_INDEX
    assert not out[1].any().item() and (sel[1] == -1).all().item()
    # (how the tiles are shared out, and with it the rounding, goes by the whole batch's lengths:
    # held to the attention's bound rather than to the first call's bits)
    s.check(q, tables, lens, 6, 0.125, out, sel, seqs=[0, 2])
