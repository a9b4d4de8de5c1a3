"""Calls from host threads other than the first."""
import threading

import pytest
import torch

from paged_kv_cache_273_gb300 import pkv
from test_f8_cache import DEV

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


def _pool(kv, bs, nb=64, H=1, D=64):
    pool = pkv.kv_block_pool_init(nb, bs, H, D, kv)
    k, v, ks, vs = pool.alloc_cache(DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    for c in (k, v):
        c.copy_(torch.randn(c.shape, device=DEV, generator=g).to(c.dtype))
    for s in (ks, vs):
        if s is not None:
            s.fill_(0.5)
    return pool, k, v, ks, vs


def _in_a_thread(f):
    got = []

    def work():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001
            got.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    return got[0]


@pytest.mark.parametrize("kv", [pkv.PKV_F8, pkv.PKV_F16, pkv.PKV_BF16, pkv.PKV_I8])
def test_a_call_may_be_the_first_of_its_thread(kv):
    # nothing has given the thread a device context yet
    pool, k, v, ks, vs = _pool(kv, 16)
    q = torch.randn(3, 2, 64, device=DEV).half()
    q = q.to(pkv.TORCH_DTYPE[kv]) if kv in (pkv.PKV_F16, pkv.PKV_BF16) else q
    tables = torch.randint(0, 64, (3, 4), **I32)
    lens = torch.tensor([64, 9, 30], **I32)
    ws, outs = pkv.alloc_workspace(pool, 3, 2), [torch.zeros(3, 2, 64, device=DEV) for _ in "ab"]
    stream = torch.cuda.current_stream()

    def call(out):
        pkv.paged_decode_attention(pool, q, k, v, tables, lens, 0.1, out, ws, 64, ks, vs,
                                   stream=stream)
    torch.cuda.synchronize()
    assert _in_a_thread(lambda: call(outs[0])) is None
    call(outs[1])
    assert torch.equal(*outs)
    if kv in (pkv.PKV_F16, pkv.PKV_BF16):
        qs = torch.tensor([0, 1, 2, 3], **I32)
        outs = [torch.zeros(3, 2, 64, device=DEV) for _ in "ab"]

        def prompt(out):
            pkv.paged_prefill_attention(pool, q, k, v, tables, qs, lens, 0.1, out, 1,
                                        stream=stream)
        torch.cuda.synchronize()
        assert _in_a_thread(lambda: prompt(outs[0])) is None
        prompt(outs[1])
        assert torch.equal(*outs)
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK
