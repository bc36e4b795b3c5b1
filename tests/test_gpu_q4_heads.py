"""Attention over the 4-bit cache with 5, 6 and 7 KV heads (one token phase, five to seven consumer warps, rows that end in
padding), and short chunks of long and large batches; cases and tolerance of the 4-bit attention tests."""

import pytest

from test_gpu_q4 import chunk_case, decode_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("hkv", [4, 5, 6, 7])
def test_decode(d, g, hkv):
    decode_case(d + g + hkv, [0, 1, 15, 16, 17, 33, 300, 64, 1200, 65], 16, hkv, g, d)
    decode_case(d + g + hkv, [700, 63, 128], 24, hkv, g, d, splits=3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,ql", [(1, 8), (2, 4), (4, 2), (8, 1)])
@pytest.mark.parametrize("hkv", [1, 2, 5, 6, 7])
def test_short_chunks(d, g, ql, hkv):
    chunk_case(g + ql, [4000, 0, 2100, 33, 5], [ql, 1, max(1, ql - 1), ql, 0], 16, hkv, g, d)
    chunk_case(g + ql, [900, 64, 700], [ql, ql, 1], 100, hkv, g, d, causal=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 8])
@pytest.mark.parametrize("hkv", [2, 5, 6, 7])
def test_chunks(d, g, hkv):
    chunk_case(d + g + hkv, [0, 130, 7, 0], [40, 150, 1, 65], 16, hkv, g, d)
