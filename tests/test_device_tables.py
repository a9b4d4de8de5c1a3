"""kv_device_reserve / kv_device_release: block tables, slots and offsets built
on the device, against the host calls and a plain loop (whole numbers, so every
comparison is exact)."""
import ctypes

import numpy as np
import pytest
import torch

import block_reference as R
from paged_kv_cache_273_gb300 import pkv

DEV = "cuda"


def _host_buf(n=4096):
    buf = (ctypes.c_uint8 * n)()
    return buf, (ctypes.addressof(buf) + 15) // 16 * 16


# ------------------------------------------------------------------ refusals (no launch)
def _reserve_args(p, addr, **kw):
    a = dict(pool=p.handle, free_ids=addr, cap=4, free_in=addr, free_out=addr, lens=addr,
             new=None, batch=2, tables=addr, maxb=2, slots=addr, T=2, q=None, out=addr)
    a.update(kw)
    return [a[k] for k in ("pool", "free_ids", "cap", "free_in", "free_out", "lens", "new",
                           "batch", "tables", "maxb", "slots", "T", "q", "out")] + [None]


def _release_args(p, addr, **kw):
    a = dict(pool=p.handle, free_ids=addr, cap=4, free_in=addr, free_out=addr, lens=addr,
             done=addr, batch=2, tables=addr, maxb=2, out=addr)
    a.update(kw)
    return [a[k] for k in ("pool", "free_ids", "cap", "free_in", "free_out", "lens", "done",
                           "batch", "tables", "maxb", "out")] + [None]


def test_refusals():
    lib = pkv.load()
    pool = pkv.kv_block_pool_init(8, 16, 1, 64, pkv.PKV_F16)
    buf, addr = _host_buf()
    inv, uns = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED
    for kw, want in [(dict(pool=None), inv), (dict(batch=-1), inv), (dict(cap=-1), inv),
                     (dict(maxb=0), inv), (dict(batch=4097), uns), (dict(free_in=None), inv),
                     (dict(free_out=None), inv), (dict(lens=None), inv), (dict(out=None), inv),
                     (dict(tables=None), inv), (dict(free_ids=None), inv),
                     (dict(tables=addr + 2), inv), (dict(lens=addr + 1), inv),
                     (dict(batch=0), pkv.PKV_OK)]:
        assert lib.kv_device_reserve(*_reserve_args(pool, addr, **kw)) == want, kw
        assert lib.kv_device_release(*_release_args(pool, addr, **kw)) == want, kw
    for kw in (dict(T=-1), dict(slots=None), dict(slots=addr + 2), dict(new=addr + 2),
               dict(q=addr + 1)):
        assert lib.kv_device_reserve(*_reserve_args(pool, addr, **kw)) == inv, kw
    for kw in (dict(done=None), dict(done=addr + 2)):
        assert lib.kv_device_release(*_release_args(pool, addr, **kw)) == inv, kw


def test_binding_refuses_shapes_and_types():
    pool = pkv.kv_block_pool_init(8, 16, 1, 64, pkv.PKV_F16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = dict(free_ids=i(8), free_in=i(2), seq_lens=i(3), block_tables=i(3, 2),
                slot_mapping=i(3))
    for k, bad in [("free_in", i(1)), ("block_tables", i(2, 2)), ("block_tables", i(6)),
                   ("free_ids", i(8).long()), ("slot_mapping", i(3).float()),
                   ("num_new", i(2)), ("q_start", i(3)), ("seq_lens_out", i(2)),
                   ("free_out", i(3))]:
        with pytest.raises(ValueError):
            pkv.kv_device_reserve(pool, **{**good, k: bad})
    with pytest.raises(ValueError):
        pkv.kv_device_reserve(pool, **good)              # host tensors
    rel = dict(free_ids=i(8), free_in=i(2), seq_lens=i(3), done=i(3), block_tables=i(3, 2))
    for k, bad in [("done", i(2)), ("done", i(3).bool()), ("seq_lens_out", i(4))]:
        with pytest.raises(ValueError):
            pkv.kv_device_release(pool, **{**rel, k: bad})


def test_reference_loop_is_the_host_call():
    # the plain loop the GPU tests compare with gives what kv_reserve_slots gives
    rng = np.random.default_rng(0)
    for bs in (4, 16):
        B, maxb = 7, 9
        pool = pkv.kv_block_pool_init(B * maxb, bs, 1, 64, pkv.PKV_F16)
        free = list(range(B * maxb))[::-1]
        tables, ref = np.zeros((B, maxb), np.int32), np.zeros((B, maxb), np.int32)
        lens, rl = np.zeros(B, np.int32), np.zeros(B, np.int64)
        for _ in range(12):
            new = np.minimum(rng.integers(0, bs + 3, B), maxb * bs - lens).astype(np.int32)
            slots = pkv.kv_reserve_slots(pool, lens, tables, new)
            lens = lens + new
            assert slots.tolist() == R.reserve(free, rl, new, ref, bs)
            assert np.array_equal(tables, ref) and np.array_equal(lens, rl)


# ------------------------------------------------------------------------------- on the GPU
class Step:
    """Device state of a batch, and the same on the host."""

    def __init__(self, B, maxb, bs, nb, seed=0):
        self.rng = np.random.default_rng(seed)
        self.B, self.maxb, self.bs, self.nb = B, maxb, bs, nb
        self.pool = pkv.kv_block_pool_init(nb, bs, 1, 64, pkv.PKV_F16)
        ids = self.rng.permutation(nb).astype(np.int32)
        self.free = ids.tolist()
        self.free_ids, self.state = pkv.alloc_device_free_list(ids, DEV)
        self.lens = np.zeros(B, np.int64)
        self.tables = np.zeros((B, maxb), np.int32)
        self.dlens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.dtables = torch.zeros(B, maxb, dtype=torch.int32, device=DEV)

    def reserve(self, new, cap=None, null_new=False):
        T = int(np.sum(new))
        cap = T if cap is None else cap
        slots = torch.full((cap + 8,), 77, dtype=torch.int32, device=DEV)
        qs = torch.full((self.B + 1,), 77, dtype=torch.int32, device=DEV)
        pkv.kv_device_reserve(self.pool, self.free_ids, self.state, self.dlens, self.dtables,
                              slots[4:4 + cap],
                              num_new=None if null_new else
                              torch.as_tensor(new, dtype=torch.int32, device=DEV), q_start=qs)
        return slots, qs, cap

    def check_reserve(self, new, cap=None, null_new=False):
        slots, qs, cap = self.reserve(new, cap, null_new)
        want = R.reserve(self.free, self.lens, new, self.tables, self.bs)
        got = slots.cpu().numpy()
        assert got[4:4 + len(want)].tolist() == want
        assert (got[4 + len(want):4 + cap] == -1).all()
        assert (got[:4] == 77).all() and (got[4 + cap:] == 77).all()
        assert qs.cpu().tolist() == np.concatenate([[0], np.cumsum(new)]).tolist()
        self.same()

    def check_release(self, done):
        pkv.kv_device_release(self.pool, self.free_ids, self.state, self.dlens,
                              torch.as_tensor(done, dtype=torch.int32, device=DEV), self.dtables)
        for b in np.nonzero(done)[0]:
            self.free += self.tables[b, :-(-self.lens[b] // self.bs)].tolist()
            self.lens[b] = 0
        self.same()

    def same(self):
        assert self.dlens.cpu().tolist() == self.lens.tolist()
        assert np.array_equal(self.dtables.cpu().numpy(), self.tables)
        n = len(self.free)
        assert self.state.cpu().tolist() == [n, 0]
        assert self.free_ids.cpu().tolist()[:n] == self.free
        assert pkv.pkv_check_error(self.pool) == pkv.PKV_OK


@pytest.mark.gpu
@pytest.mark.parametrize("B,bs,maxb", [(1, 4, 3), (3, 16, 5), (33, 8, 7), (257, 16, 9),
                                       (1025, 32, 4), (4096, 16, 3)])
def test_steps_against_the_loop(B, bs, maxb):
    s = Step(B, maxb, bs, B * maxb, seed=B)
    for i in range(8):
        room = maxb * bs - s.lens
        new = np.minimum(s.rng.integers(0, 2 * bs, B), room)
        if i == 3:
            new[:] = 0                                   # nothing new at all
        if i == 4:
            new = np.minimum(1, room)
        s.check_reserve(new, cap=int(new.sum()) + (0 if i % 2 else 37))
        if i % 3 == 2:
            s.check_release((s.rng.random(B) < 0.4).astype(np.int32))
    s.check_release(np.ones(B, np.int32))
    assert len(s.free) == B * maxb and sorted(s.free) == list(range(B * maxb))


@pytest.mark.gpu
def test_long_prompts_over_many_ctas():
    s = Step(5, 8192, 16, 5 * 8192, seed=9)
    s.check_reserve(np.array([100000, 0, 1, 131072, 4097]))
    s.check_reserve(np.array([1, 1, 1, 0, 1]))
    s.check_release(np.array([1, 0, 0, 1, 0]))
    s.check_reserve(np.array([17, 1, 0, 70001, 16]), cap=300000)


@pytest.mark.gpu
def test_one_token_each_by_default_and_out_of_place():
    s = Step(6, 4, 4, 24)
    s.check_reserve(np.ones(6, np.int64), null_new=True)
    s.check_reserve(np.array([3, 4, 0, 1, 2, 5]))
    lens_out = torch.full((6,), -5, dtype=torch.int32, device=DEV)
    state_out = torch.tensor([99, 0], dtype=torch.int32, device=DEV)
    slots = torch.zeros(6, dtype=torch.int32, device=DEV)
    for _ in range(2):                                   # the inputs stay: the same answer twice
        pkv.kv_device_reserve(s.pool, s.free_ids, s.state, s.dlens, s.dtables, slots,
                              free_out=state_out, seq_lens_out=lens_out)
        free, lens, tables = list(s.free), s.lens.copy(), s.tables.copy()
        assert slots.cpu().tolist() == R.reserve(free, lens, np.ones(6, int), tables, s.bs)
        assert lens_out.cpu().tolist() == lens.tolist()
        assert state_out.cpu().tolist() == [len(free), 0]
        assert s.dlens.cpu().tolist() == s.lens.tolist()
        assert np.array_equal(s.dtables.cpu().numpy(), tables)


@pytest.mark.gpu
def test_too_few_blocks_changes_nothing():
    s = Step(4, 4, 16, 6)
    s.check_reserve(np.array([16, 17, 0, 5]))            # 4 of 6 blocks
    slots, qs, cap = s.reserve(np.array([1, 1, 16, 40]), cap=64)   # needs 1 + 0 + 1 + 2
    assert (slots.cpu().numpy()[4:4 + cap] == -1).all() and not qs.any().item()
    assert pkv.pkv_check_error(s.pool) == pkv.PKV_ERR_NO_BLOCKS
    s.same()
    s.check_reserve(np.array([1, 1, 16, 0]))             # what is left serves a smaller step


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["length", "negative length", "new", "tokens", "count",
                                  "negative count"])
def test_out_of_range_inputs_change_nothing(what):
    s = Step(3, 2, 16, 6)
    s.check_reserve(np.array([5, 20, 1]))
    lens, state, new, cap = s.dlens.clone(), s.state.clone(), [1, 1, 1], 8
    if what == "length":
        lens[1] = 33
    elif what == "negative length":
        lens[2] = -1
    elif what == "new":
        new = [1, 13, 1]                                 # 20 + 13 > 32
    elif what == "tokens":
        new, cap = [9, 0, 0], 8
    elif what == "count":
        state[0] = 7
    else:
        state[0] = -1
    out = lens.clone()
    st2 = state.clone()
    slots = torch.zeros(cap, dtype=torch.int32, device=DEV)
    pkv.kv_device_reserve(s.pool, s.free_ids, st2, out, s.dtables, slots,
                          num_new=torch.tensor(new, dtype=torch.int32, device=DEV))
    assert pkv.pkv_check_error(s.pool) == pkv.PKV_ERR_BAD_INDEX
    assert torch.equal(out, lens) and torch.equal(st2, state)
    assert (slots == -1).all().item()
    s.same()
    if what in ("length", "negative length", "count", "negative count"):
        done = torch.ones(3, dtype=torch.int32, device=DEV)
        pkv.kv_device_release(s.pool, s.free_ids, st2, out, done, s.dtables)
        assert pkv.pkv_check_error(s.pool) == pkv.PKV_ERR_BAD_INDEX
        assert torch.equal(out, lens) and torch.equal(st2, state)
        s.same()


@pytest.mark.gpu
def test_release_beyond_the_stack_is_refused():
    s = Step(2, 2, 4, 3)
    s.check_reserve(np.array([4, 4]))
    s.dlens[1] = 8                                       # claims a block more than was taken
    pkv.kv_device_release(s.pool, s.free_ids, s.state, s.dlens,
                          torch.ones(2, dtype=torch.int32, device=DEV), s.dtables)
    pkv.pkv_check_error(s.pool)
    assert s.state.cpu().tolist()[0] <= 3
    small, state = pkv.alloc_device_free_list([0], DEV)
    lens = torch.tensor([4, 4], dtype=torch.int32, device=DEV)
    pkv.kv_device_release(s.pool, small, state, lens, torch.ones(2, dtype=torch.int32, device=DEV),
                          s.dtables)
    assert pkv.pkv_check_error(s.pool) == pkv.PKV_ERR_BAD_INDEX
    assert state.cpu().tolist() == [1, 0] and lens.cpu().tolist() == [4, 4]


@pytest.mark.gpu
def test_ids_outside_the_pool_give_padding_slots():
    pool = pkv.kv_block_pool_init(4, 4, 1, 64, pkv.PKV_F16)
    free_ids, state = pkv.alloc_device_free_list([2, 9, 1], DEV)     # 9 is outside
    lens = torch.tensor([2, 0, 0], dtype=torch.int32, device=DEV)
    tables = torch.tensor([[7], [0], [0]], dtype=torch.int32, device=DEV)   # 7 is outside
    slots = torch.zeros(3, dtype=torch.int32, device=DEV)
    pkv.kv_device_reserve(pool, free_ids, state, lens, tables, slots)
    assert pkv.pkv_check_error(pool) == pkv.PKV_ERR_BAD_INDEX
    assert slots.cpu().tolist() == [-1, 4, -1]
    assert state.cpu().tolist() == [1, 0] and lens.cpu().tolist() == [3, 1, 1]


@pytest.mark.gpu
def test_captured_steps_replay():
    s = Step(9, 6, 4, 54)
    s.check_reserve(np.arange(9))
    new = torch.ones(9, dtype=torch.int32, device=DEV)
    slots = torch.zeros(16, dtype=torch.int32, device=DEV)
    done = torch.zeros(9, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pkv.kv_device_release(s.pool, s.free_ids, s.state, s.dlens, done, s.dtables)
        pkv.kv_device_reserve(s.pool, s.free_ids, s.state, s.dlens, s.dtables, slots, num_new=new)
    for i in range(12):
        n = s.rng.integers(0, 2, 9)
        d = (s.rng.random(9) < 0.2).astype(np.int32)
        new.copy_(torch.as_tensor(n, dtype=torch.int32))
        done.copy_(torch.as_tensor(d))
        g.replay()
        for b in np.nonzero(d)[0]:
            s.free += s.tables[b, :-(-s.lens[b] // s.bs)].tolist()
            s.lens[b] = 0
        want = R.reserve(s.free, s.lens, n, s.tables, s.bs)
        got = slots.cpu().tolist()
        assert got == want + [-1] * (16 - len(want)), i
        s.same()


@pytest.mark.gpu
@pytest.mark.parametrize("B,maxb", [(3, 5), (200, 300)])     # one CTA, several
def test_release_of_ids_outside_the_pool_is_refused(B, maxb):
    bs = 4
    s = Step(B, maxb, bs, B * maxb)
    s.check_reserve(s.rng.integers(1, (maxb - 1) * bs + 1, B))
    done = (s.rng.random(B) < 0.7).astype(np.int32)
    done[:2], done[2] = 1, 0
    s.check_reserve(np.array([3, 1] + [0] * (B - 2)))        # rows 0 and 1 hold a block
    good = s.dtables.clone()
    for row, at, bad in ((0, 0, -1), (1, -1, B * maxb), (0, 0, -2 ** 31), (B - 1, 0, 2 ** 31 - 1)):
        n = -(-int(s.lens[row]) // bs)
        s.dtables[row, at % n] = bad
        before = s.dlens.clone()
        free, state = s.free_ids.clone(), s.state.clone()
        pkv.kv_device_release(s.pool, s.free_ids, s.state, s.dlens,
                              torch.as_tensor(np.maximum(done, np.arange(B) == row),
                                              dtype=torch.int32, device=DEV), s.dtables)
        assert pkv.pkv_check_error(s.pool) == pkv.PKV_ERR_BAD_INDEX
        assert torch.equal(s.state, state) and torch.equal(s.dlens, before)
        top = int(state[0])
        assert torch.equal(s.free_ids[:top], free[:top])
        s.dtables.copy_(good)
    # an id that is not released is not looked at, nor one behind a row's blocks
    s.dtables[2, 0] = -1
    n = -(-int(s.lens[0]) // bs)
    if n < maxb:
        s.dtables[0, n] = -1
    s.tables = s.dtables.cpu().numpy()
    s.check_release(done)
