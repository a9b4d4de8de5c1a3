"""Forms of the block choice and of the weights that larger batches and every head count reach."""
import math

import numpy as np
import pytest
import torch

from test_f8_cache import DEV, DT, _rows
from test_sparse import Sparse, _tables
import block_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,bs,D,G", [("bf16", 16, 128, 4), ("f8", 8, 64, 8), ("f16", 4, 64, 2)])
def test_one_cta_a_head_scores_in_several_rounds(kv, bs, D, G):
    # 128 (sequence, KV head)s: one CTA of 16 warps each on a GPU of 128 to 192 SMs, which
    # scores 512 blocks a round and keeps the keys in shared memory
    B, H, nb = 16, 8, 300
    s = Sparse(kv, nb, H, bs, D, seed=2)
    g = np.random.default_rng(3)
    n = [513, 512, 511, 1024, 1025, 2100, 600, 1537, 2048, 700, 40, 1, 1600, 2099, 545, 0]
    lens = [max(0, x * bs - int(g.integers(0, bs))) for x in n]
    tables = _tables(nb, lens, bs, 4)
    q = _rows(5, (B, H * G, D), "bf16" if kv == "bf16" else "f16", 1.5)
    ws = None
    for budget in (600, 40, 2):                           # (one workspace, the largest first)
        out, sel, ws = s.call(q, tables, lens, budget, 1 / math.sqrt(D), ws)
        s.check(q, tables, lens, budget, 1 / math.sqrt(D), out, sel,
                seqs=range(0, B, 4 if budget > 40 else 1))


@pytest.mark.parametrize("kv", ["bf16", "f16", "f8"])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 1), (64, 2), (128, 2), (128, 4), (64, 4), (128, 8)])
def test_every_part_of_a_weight_counts(kv, D, G):
    """Two rows, scores x and 0, values 1 and 0: p / (p + 1) to 2^-20.

    One channel of q and k is not zero, so a score's product is exact; with x below 1.5 in the
    log2 domain its two roundings (the scale's, the product's) are 1.5 * 2^-23 in all, 2^-23 of
    the weight; the exponential is off by 2^-22, parts by 2^-22 (fp16) or 2^-27 (three of bf16),
    the MMA's sum of parts by 2^-22 (it may truncate), sum, reciprocal and product by 2^-24 each:
    below 2^-20.  Two bf16 parts leave 2^-18, one fp16 part 2^-12."""
    B, H, bs = 64, 2, 16
    s = Sparse(kv, B, H, bs, D, seed=1)
    g = np.random.default_rng(2)
    c = g.integers(32, 64, (B, H)) / 64.0                 # 0.5 .. 1: exact in every type
    hk, hv = np.zeros((B, H, bs, D)), np.zeros((B, H, bs, D))
    if kv == "f8":
        c = R.E4M3[R.e4m3_encode(c)]
    hk[:, :, 0, 3], hv[:, :, 0] = c, 1.0
    if kv == "f8":
        s.c.hk[:], s.c.hv[:], s.c.hks[:], s.c.hvs[:] = R.e4m3_encode(hk), R.e4m3_encode(hv), 1, 1
        s.c.upload()
    else:
        s.k.copy_(torch.from_numpy(hk))
        s.v.copy_(torch.from_numpy(hv))
    qt = "bf16" if kv == "bf16" else "f16"
    q = torch.zeros(B, H * G, D, dtype=DT[qt], device=DEV)
    qv = torch.from_numpy(g.integers(128, 256, (B, H * G)) / 256.0)   # 0.5 .. 1, 8 bits
    q[:, :, 3] = qv.to(DT[qt]).to(DEV)
    out, _, _ = s.call(q, np.arange(B, dtype=np.int32)[:, None], [2] * B, 1, 1.0)
    x = qv.numpy() * np.repeat(c, G, axis=1)
    want = 1.0 / (1.0 + np.exp(-x))
    err = np.abs(out.double().cpu().numpy() / want[:, :, None] - 1.0).max()
    assert err <= 2.0 ** -20, math.log2(err)
