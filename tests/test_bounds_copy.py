"""Key bounds through copy-on-write: a copied block's bounds are copied too, and appends to it go
on from them."""
import ctypes

import numpy as np
import pytest
import torch

import block_reference as R
from paged_kv_cache_273_gb300 import pkv
from test_f8_cache import DEV, _rows
from test_sparse import Bounds


def test_refusals():
    lib = pkv.load()
    buf = (ctypes.c_uint8 * 4096)()
    a = (ctypes.addressof(buf) + 15) // 16 * 16
    pool = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_F16)

    def copy(p=pool.handle, s=a, d=a, n=1, b=a, e=a):
        return lib.kv_bounds_copy(p, s, d, n, b, e, None)
    for bad in (dict(p=None), dict(s=None), dict(d=None), dict(n=-1), dict(b=None), dict(e=None),
                dict(s=a + 2), dict(d=a + 1), dict(b=a + 8), dict(e=a + 2)):
        assert copy(**bad) == pkv.PKV_ERR_INVALID, bad
    assert copy(n=0) == pkv.PKV_OK
    b, e = pkv.alloc_bounds(pool, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    for args in [(i, i[:1], b, e), (i.long(), i, b, e), (i, i, b[:4], e), (i, i, b, e.long()),
                 (i, i, b.float(), e)]:
        with pytest.raises(ValueError):
            pkv.kv_bounds_copy(pool, *args)


@pytest.mark.gpu
@pytest.mark.parametrize("H,D,n", [(1, 64, 1), (8, 128, 40), (3, 64, 150)])
def test_copies_bounds_and_exponents(H, D, n):
    pool = pkv.kv_block_pool_init(400, 16, H, D, pkv.PKV_BF16)
    s = Bounds(pool, n)
    p = np.random.default_rng(n).permutation(400)[:2 * n].astype(np.int32)
    src, dst = p[:n].copy(), p[n:].copy()
    good = np.ones(n, bool)
    if n > 20:                                            # recorded, the pair skipped
        src[3], dst[11], src[17], dst[18] = -1, 400, 2 ** 31 - 1, -7
        good[[3, 11, 17, 18]] = False
    pkv.kv_bounds_copy(pool, torch.from_numpy(src).to(DEV), torch.from_numpy(dst).to(DEV), s.b, s.e)
    s.hb[dst[good]], s.he[dst[good]] = s.hb[src[good]], s.he[src[good]]
    s.same()
    assert pkv.pkv_check_error(pool) == (pkv.PKV_OK if n < 20 else pkv.PKV_ERR_BAD_INDEX)


@pytest.mark.gpu
def test_copy_on_write_keeps_the_bounds():
    # two sequences share a partly filled block; both append: one gets a copy in a block that
    # held much larger keys before.  Bounds as of sequences that share nothing
    H, bs, D, B = 2, 16, 128, 2
    pool = pkv.kv_block_pool_init(12, bs, H, D, pkv.PKV_BF16)
    s = Bounds(pool, 3)
    kc, vc, _, _ = pool.alloc_cache(DEV)
    ids = pkv.kv_block_alloc(pool, 2)
    n0 = bs + 5
    prompt = _rows(1, (n0, H, D), "bf16")
    slots = [int(ids[p // bs]) * bs + p % bs for p in range(n0)]
    st = torch.tensor(slots, dtype=torch.int32, device=DEV)
    pkv.kv_append(pool, prompt, prompt, st, kc, vc)
    s.append(prompt, slots)
    other = [i for i in range(12) if i not in ids]
    for t, h in ((s.b, s.hb), (s.e, s.he)):
        t[other] = 90
        h[other] = 90
    pkv.kv_block_share(pool, ids)
    tables = np.zeros((B, 3), np.int32)
    tables[:, :2] = ids
    slots, src, dst = pkv.kv_reserve_slots_cow(pool, np.full(B, n0, np.int32), tables)
    assert src.tolist() == [ids[1]] and len(dst) == 1 and dst[0] in other
    sd, dd = torch.from_numpy(src).to(DEV), torch.from_numpy(dst).to(DEV)
    pkv.kv_block_copy(pool, sd, dd, kc, vc)
    pkv.kv_bounds_copy(pool, sd, dd, s.b, s.e)
    new = _rows(2, (B, H, D), "bf16", 3.0)
    st = torch.from_numpy(slots).to(DEV)
    pkv.kv_append(pool, new, new, st, kc, vc)
    pkv.kv_bounds_append(pool, new, st, s.b, s.e)
    for b in range(B):
        alone, exps = np.zeros((2, H, 2, D), np.int8), np.zeros((2, H), np.int32)
        rows = torch.cat([prompt, new[b:b + 1]]).double().cpu().numpy()
        R.append_bounds(rows, range(n0 + 1), bs, alone, exps)
        blocks = torch.from_numpy(tables[b, :2].astype(np.int64)).to(DEV)
        assert np.array_equal(s.b[blocks].cpu().numpy(), alone), b
        assert np.array_equal(s.e[blocks].cpu().numpy(), exps), b
        held = kc[blocks].double().cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, H, D)[:n0 + 1]
        assert np.array_equal(held, rows)
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK
