"""Calls from several host threads at once, each on its own stream and workspace, of sizes that
need different amounts of shared memory."""
import functools
import threading

import numpy as np
import pytest
import torch

from paged_kv_cache_273_gb300 import pkv
from test_f8_cache import DEV

pytestmark = pytest.mark.gpu
P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
I32 = dict(dtype=torch.int32, device=DEV)


def _together(calls, rounds=6000):
    """Every call in a thread of its own, `rounds` times and with little but the library between
    them; its first output is held to the last."""
    start, errors = threading.Barrier(len(calls)), []

    def work(call, out):
        try:
            stream = torch.cuda.Stream()
            torch.zeros(1, device=DEV)
            bare = call(stream.cuda_stream)
            assert bare() == pkv.PKV_OK
            stream.synchronize()
            first = out.clone()
            torch.cuda.synchronize()
            start.wait()
            for i in range(rounds):
                rc = bare()
                if rc != pkv.PKV_OK:
                    errors.append((i, rc))
                    break
                if i % 500 == 499:
                    stream.synchronize()
            stream.synchronize()
            assert torch.equal(first, out)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
            start.abort()
    threads = [threading.Thread(target=work, args=c) for c in calls]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


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


@pytest.mark.parametrize("kv", [pkv.PKV_F8, pkv.PKV_F16, pkv.PKV_BF16])
def test_decode_of_different_batches(kv):
    pool, k, v, ks, vs = _pool(kv, 16)
    qt = torch.float16 if kv == pkv.PKV_F8 else pkv.TORCH_DTYPE[kv]

    def case(B):
        g = torch.Generator(device=DEV).manual_seed(B)
        q = torch.randn(B, 2, 64, device=DEV, generator=g).to(qt)
        tables = torch.randint(0, 64, (B, 2), generator=g, **I32)
        lens = torch.randint(0, 33, (B,), generator=g, **I32)
        out, ws = torch.zeros(B, 2, 64, device=DEV), pkv.alloc_workspace(pool, B, 2)
        keep.append((q, tables, lens, out, ws))
        a = [pool.handle, q.data_ptr(), pkv.PKV_DTYPE[qt], 2, k.data_ptr(), v.data_ptr(), P(ks),
             P(vs), tables.data_ptr(), 2, lens.data_ptr(), B, 32, 0.1, out.data_ptr(),
             ws.data_ptr(), ws.numel()]
        return (lambda s: functools.partial(pkv.load().paged_decode_attention, *a, s)), out
    keep = []
    _together([case(1), case(4000), case(1500), case(60)])
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK


@pytest.mark.parametrize("kv", [pkv.PKV_F8, pkv.PKV_F16])
def test_sparse_of_different_lengths(kv):
    pool, k, v, ks, vs = _pool(kv, 8)
    bounds, exps = pkv.alloc_bounds(pool, DEV)
    bounds.copy_(torch.from_numpy(np.sort(np.random.default_rng(1).integers(
        -127, 128, bounds.shape).astype(np.int8), 2)))

    def case(n):
        g = torch.Generator(device=DEV).manual_seed(n)
        q = torch.randn(1, 2, 64, device=DEV, generator=g).half()
        tables = torch.randint(0, 64, (1, n), generator=g, **I32)
        lens = torch.full((1,), 8 * n, **I32)
        out, sel = torch.zeros(1, 2, 64, device=DEV), torch.zeros(1, 1, 20, **I32)
        ws = pkv.alloc_sparse_workspace(pool, 1, 2, 8 * n, 20)
        keep.append((q, tables, lens, out, sel, ws))
        a = [pool.handle, q.data_ptr(), pkv.PKV_F16, 2, k.data_ptr(), v.data_ptr(), P(ks), P(vs),
             bounds.data_ptr(), exps.data_ptr(), tables.data_ptr(), n, lens.data_ptr(), 1, 8 * n,
             20, 0.1, out.data_ptr(), sel.data_ptr(), ws.data_ptr(), ws.numel()]
        return (lambda s: functools.partial(pkv.load().paged_decode_attention_sparse, *a, s)), out
    keep = []
    _together([case(24000), case(6000), case(12000), case(100)])
    assert pkv.pkv_check_error(pool) == pkv.PKV_OK


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
