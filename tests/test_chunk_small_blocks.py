"""paged_chunk_attention over blocks of 4 rows, which no tensor copy brings."""
import math
import os

import pytest

import test_chunk as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_map_of_4_row_blocks_is_looked_at():
    """Maps of K and V are encoded for blocks of 8 rows and more; every look at them is under that
    condition."""
    with open(os.path.join(ROOT, "paged_kv_cache_273_gb300", "csrc", "chunk.cu")) as f:
        src = f.read()
    assert "if (!f8 && pool->block_size >= 8 && (!encode_tile_map(" in src
    assert "if (!F8 && p.box_rows >= 8) {" in src and src.count("prefetch_map(&p.tm_k)") == src.count("prefetch_map(&p.tm_v)") == 1
    assert "const bool by_tma = inbox && R >= 8" in src and src.count("tma_load_5d(dst") == 1


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 3, 131])
@pytest.mark.parametrize("case", [
    ([1, 4, 5, 259], [1, 4, 2, 130], 4, 2, 128, 4, "bf16", "bf16"),
    ([3000], [3], 8, 1, 64, 4, "f16", "f16"),
    ([700, 300], [300, 300], 2, 1, 128, 4, "f16", "f16"),
], ids=range(3))
def test_gpu_blocks_of_4_rows(case, window):
    s = C.make(*case)
    C.check(s, C.run(s, 1.0 / math.sqrt(s["D"]), window), window)


@pytest.mark.gpu
def test_gpu_blocks_of_4_rows_in_a_tree():
    s = C.make([64, 130, 7], [64, 3, 7], 4, 1, 128, 4, "bf16", "bf16", tree=C._tree([64, 3, 7], "drafts"))
    C.check(s, C.run(s, 1.0 / math.sqrt(128)))
