"""The binding of kv_rope_rotate and kv_rope_append: rows as views give them, and arguments
that are missing."""
import pytest
import torch

import test_rope as P
from paged_kv_cache_273_gb300 import pkv

DEV = "cuda"
i32 = P.i32


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "f8"])
def test_gpu_append_of_q_needs_its_output(kv):
    pool = pkv.kv_block_pool_init(4, 16, 2, 64, P.POOL[kv])
    kc, vc, ks, vs = pool.alloc_cache()
    x = torch.zeros(3, 8, 64, dtype=torch.bfloat16, device=DEV)
    args = (x[:, 4:6], x[:, 6:], i32([0, 1, 2]), i32([0, 1, 2]))
    with pytest.raises(ValueError, match="q_out"):
        pkv.kv_rope_append(pool, pkv.rope_plan(64), x[:, :4], *args, None, kc, vc, ks, vs)
    pkv.kv_rope_append(pool, pkv.rope_plan(64), None, *args, None, kc, vc, ks, vs)
    torch.cuda.synchronize()
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK


def test_one_token_has_no_stride():
    """A view of one token says what the next would be apart by; nothing reads it."""
    D = 64
    for step in (0, 3, 4 * D, 6 * D + 1):
        x = torch.zeros(8 * D).as_strided((1, 4, D), (step, D, 1))
        assert pkv._head_rows("x", x, torch.float32, (1, 4, D), -1) == (x.data_ptr(), 4 * D)
    x = torch.zeros(20 * D).as_strided((2, 4, D), (6 * D, D, 1))
    assert pkv._head_rows("x", x, torch.float32, (2, 4, D), -1) == (x.data_ptr(), 6 * D)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["f16", "f8"])
def test_gpu_one_token_of_a_projection_of_odd_width(kv):
    """The last token of a projection whose rows are no multiple of 16 bytes apart, and one that is
    turned in place through a view of another width."""
    hq, H, D = 4, 2, 64
    width = (hq + 2 * H) * D + 4
    g = torch.Generator().manual_seed(3)
    whole = torch.randn(2 * width, generator=g).half().to(DEV)
    row = whole[width + 4:]                            # (16-byte aligned: width + 4 is a multiple of 8)
    x = row.as_strided((1, hq + 2 * H, D), (width, D, 1), row.storage_offset())
    plain = x.clone()
    plan = pkv.rope_plan(D)
    want = pkv.kv_rope_rotate(plan, plain[:, :hq + H].contiguous(), i32([977]))
    assert torch.equal(pkv.kv_rope_rotate(plan, x[:, :hq + H], i32([977])), want)
    pool = pkv.kv_block_pool_init(4, 16, H, D, P.POOL[kv])
    caches = []
    for y in (plain, x):
        c = pool.alloc_cache()
        for t in c[:2]:
            t.view(torch.uint8).zero_()
        out = torch.zeros(1, hq, D, dtype=torch.half, device=DEV)
        pkv.kv_rope_append(pool, plan, y[:, :hq], y[:, hq:hq + H], y[:, hq + H:], i32([977]), i32([16]), out, *c)
        assert torch.equal(out, want[:, :hq])
        caches.append(c)
    for a, b in zip(*caches):
        if a is not None:
            assert torch.equal(a[1].view(torch.uint8), b[1].view(torch.uint8))
    # in place, x and out views of other widths
    here = x[:, :hq + H]
    pkv.kv_rope_rotate(plan, here, i32([977]), here.as_strided(here.shape, (8 * D, D, 1), here.storage_offset()))
    assert torch.equal(here, want) and torch.equal(x[:, hq + H:], plain[:, hq + H:])
    torch.cuda.synchronize()
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK
