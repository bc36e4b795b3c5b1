"""Attention over quantized caches where scores, or what they are made of, are large or small.

The softmax weights enter the P V product as f16, which ends at 65504, so the reference that a
row's exponents start from, and the exponents themselves, must be taken so that no rounding of a
large score lets a weight pass it (or leaves all of them below its least number).

Large scores: q has two elements, of which the first makes two groups of keys, half the magnitude
apart, and the second spreads the upper group over some 12 units (log2 units, or steps of float32 where
those are larger), rising with the token, so that the running maximum moves by little again and again.
At such scores float32 cannot say how the group's keys compare, but their V rows are alike: the result
is that row, whatever their weights.  Every other query head has ordinary scores.  Tolerance: that of
the 4-bit attention tests, whose terms hold here as they stand (alike V rows leave nothing of
the scores' error).
"""

import numpy as np
import pytest
import torch

import pagedattention_kv_cache_gb300 as pkv
from pagedattention_kv_cache_gb300 import metadata as md
from oracle import attention as oa
from oracle import fp8 as of8
from oracle import q4 as oq

from _harness import as_np
from test_gpu_q4 import close

pytestmark = pytest.mark.gpu

T = 1.0 / 64
HKV, BS = 2, 16
LOG2E = 1.4426950408889634
CONTEXTS = [1, 2, 65, 3000]
POWERS = [18, 20, 23, 24, 25, 26, 27, 28, 29, 30, 34, 45, 60, 100, 120]


def _e4m3_levels():
    v = of8.e4m3_decode(np.arange(127, dtype=np.uint8))
    return np.sort(v[v >= 4])  # 4 ... 448


class Case:
    """Contexts of keys in an upper and a lower group, q of magnitude 2^power on even heads."""

    def __init__(self, cache, power, lens, rows, g, d):
        rng = np.random.default_rng(power * 10 + len(rows))
        self.cache, self.lens, self.rows, self.g, self.d, self.scale = cache, lens, rows, g, d, d ** -0.5
        fine = _e4m3_levels() * T * (7 if cache == "q4" else 1)
        blocks = [-(-n // BS) for n in lens]
        order, at, self.tables = rng.permutation(sum(blocks) + 1), 0, []
        k = np.zeros(((sum(blocks) + 1) * BS, HKV, d), dtype=np.float32)
        v = rng.standard_normal(k.shape).astype(np.float32)
        alike = rng.standard_normal((HKV, d)).astype(np.float32)
        for n, b in zip(lens, blocks):
            self.tables.append(order[at:at + b].tolist())
            at += b
            slot = np.array(self.tables[-1])[np.arange(n) // BS] * BS + np.arange(n) % BS
            upper = rng.random(n) < 0.5
            upper[0] = True
            k[slot, 0, 0] = np.where(upper, 7.0, 3.5)
            k[slot, 1, 0] = np.where(upper, -3.5, -7.0)
            k[slot, :, 16] = fine[np.sort(rng.integers(0, len(fine), n))][:, None]
            v[slot[upper]] = alike
        self.k, self.v = [torch.from_numpy(x).to(torch.bfloat16) for x in (k, v)]
        unit = self.scale * LOG2E
        step = max(1.0, 2.0 ** (np.floor(np.log2(unit * 7 * 2.0 ** power)) - 23))
        q = np.zeros((sum(rows), HKV * g, d), dtype=np.float32)
        q[:, ::2, 0] = 2.0 ** power
        q[:, ::2, 16] = 2.0 ** np.round(np.log2(12.5 * step / (unit * fine[-1])))
        q[:, 1::2, 0], q[:, 1::2, 16] = 8.0, 0.5
        self.q = torch.from_numpy(q).to(torch.bfloat16)
        nb = len(order)
        if cache == "q4":
            self.pools = [pkv.q4_cache(nb, BS, HKV, d) for _ in range(2)]
            pkv.kv_store_q4(self.k.cuda(), self.v.cuda(), *self.pools, torch.arange(nb * BS, dtype=torch.int32).cuda(), T, T)
            self.values = [oq.values(x.cpu().numpy(), HKV, d, T) for x in self.pools]
        else:
            codes = [of8.quantize(as_np(x), T).reshape(nb, BS, HKV, d) for x in (self.k, self.v)]
            self.pools = [torch.from_numpy(x).cuda() for x in codes]
            self.values = [of8.dequantize(x, T) for x in codes]
        self.table = md.table_matrix(self.tables)

    def check(self, got, attend, label):
        assert pkv.device_error() == 0
        k, v = self.values
        close(got, attend(k, v), attend(k, np.abs(v)), float(np.abs(v).max()) * 2.0 ** -32, max(self.lens), label)

    def decode(self, splits):
        lens = np.asarray(self.lens, dtype=np.int32)
        ints = torch.from_numpy(self.table).cuda(), torch.from_numpy(lens).cuda()
        if self.cache == "q4":
            got = pkv.paged_decode_attn_q4(self.q.cuda(), *self.pools, *ints, self.scale, T, T, HKV, num_splits=splits)
        else:
            got = pkv.paged_decode_attn_fp8(self.q.cuda(), *self.pools, *ints, self.scale, T, T, num_splits=splits)
        self.check(got, lambda k, v: oa.paged_decode_attention(as_np(self.q), k, v, self.table, lens, self.scale),
                   f"decode, {splits} splits")

    def chunk(self, **kw):
        cu_q, cu_k = [np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (self.rows, self.lens)]
        ints = [torch.from_numpy(x).cuda() for x in (self.table, cu_q, cu_k)]
        args = (self.q.cuda(), *self.pools, *ints, max(self.rows), max(self.lens), self.scale, T, T)
        if self.cache == "q4":
            got = pkv.paged_varlen_prefill_attn_q4(*args, HKV, **kw)
        else:
            got = pkv.paged_varlen_prefill_attn_fp8(*args, **kw)
        self.check(got, lambda k, v: oa.paged_prefill_attention(as_np(self.q), cu_q, cu_k, self.scale, k_cache=k, v_cache=v,
                                                                block_tables=self.table), f"chunk {self.rows} {kw}")


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("cache,g,d", [("q4", 2, 128), ("q4", 8, 64), ("e4m3", 2, 128), ("e4m3", 8, 128)])
def test_decode_of_large_scores(cache, g, d, power):
    case = Case(cache, power, CONTEXTS, [1] * len(CONTEXTS), g, d)
    for splits in (0, 1, 3):
        case.decode(splits)


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("cache,d", [("q4", 128), ("q4", 64), ("e4m3", 128)])
def test_drafted_tokens_of_large_scores(cache, d, power):
    Case(cache, power, CONTEXTS, [1, 2, 4, 4], 2, d).chunk()


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("cache,d", [("q4", 128), ("q4", 64), ("e4m3", 128), ("e4m3", 64)])
def test_chunks_of_large_scores(cache, d, power):
    case = Case(cache, power, CONTEXTS, [1, 2, 65, 70], 2, d)
    case.chunk()
    case.chunk(workspace=False)
