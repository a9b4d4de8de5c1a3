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
