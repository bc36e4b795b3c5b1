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


def _pools(cache, k, v, t):
    """K, V rows [n, Hkv, D] in blocks in order, and the values that the pools hold."""
    n, hkv, d = k.shape
    slots = torch.arange(n, dtype=torch.int32).cuda()
    if cache == "q4":
        pools = [pkv.q4_cache(-(-n // BS), BS, hkv, d) for _ in range(2)]
        pkv.kv_store_q4(k.cuda(), v.cuda(), *pools, slots, t, t)
        return pools, [oq.values(x.cpu().numpy().reshape(-1, x.shape[2])[:n], hkv, d, t) for x in pools]
    pools = [torch.zeros(-(-n // BS), BS, hkv, d, dtype=torch.uint8).cuda() for _ in range(2)]
    pkv.kv_store_fp8(k.cuda(), v.cuda(), *pools, slots, t, t)
    return pools, [of8.e4m3_decode(x.cpu().numpy().reshape(-1, hkv, d)[:n]) * float(np.float32(t)) for x in pools]


def _calls(cache, q, pools, n, scale, t, hkv):
    """Decode (split and not), drafted tokens and a chunk over n keys in order; q [150, Hq, D], every row alike."""
    bt = torch.arange(pools[0].shape[0], dtype=torch.int32)[None].cuda()
    lens, cu_k = [torch.tensor(x, dtype=torch.int32).cuda() for x in ([n], [0, n])]
    decode, chunk = ((pkv.paged_decode_attn_q4, pkv.paged_varlen_prefill_attn_q4) if cache == "q4" else
                     (pkv.paged_decode_attn_fp8, pkv.paged_varlen_prefill_attn_fp8))
    heads = (hkv,) if cache == "q4" else ()
    if cache == "q4" or q.shape[2] == 128:
        for splits in (0, 1):
            yield "decode", decode(q[:1], *pools, bt, lens, scale, t, t, *heads, num_splits=splits)
    for new in (2, 150):
        cu_q = torch.tensor([0, new], dtype=torch.int32).cuda()
        yield f"chunk of {new}", chunk(q[:new], *pools, bt, cu_q, cu_k, new, n, scale, t, t, *heads, causal=False)


@pytest.mark.parametrize("cache,t,scale,q,level", [
    ("q4", 2.0 ** -64, 1.05 * 2.0 ** -80, 1.5 * 2.0 ** 127, 7 * 448.0),  # scale times the tensor scale is far below the
    ("e4m3", 2.0 ** -64, 1.05 * 2.0 ** -78, 1.5 * 2.0 ** 127, 448.0),    # normal numbers
    ("q4", 2.0 ** 64, 2.0 ** 67, 2.0 ** -132, 7 * 2.0 ** -6),            # and past the largest
    ("e4m3", 2.0 ** 64, 2.0 ** 70, 2.0 ** -132, 2.0 ** -6),
])
@pytest.mark.parametrize("d", [64, 128])
def test_softmax_scale_times_tensor_scale(cache, t, scale, q, level, d):
    """Ordinary scores from factors at their ends."""
    n, hkv = 600, 2
    gen = torch.Generator().manual_seed(3)
    sign = (torch.randint(0, 2, (n, hkv, d), generator=gen) * 2 - 1).float()
    sign[::7] = 1.0  # keys along q
    v = torch.randn(n, hkv, d, generator=gen)
    v[::7] += 2.0
    # keys of one magnitude, an E4M3 number (4 bits: 7 times one) times T, are stored exactly
    pools, (k, v) = _pools(cache, (sign * level * t).to(torch.bfloat16), (v * t).to(torch.bfloat16), t)
    s = np.einsum("d,nhd->hn", np.full(d, q), k) * scale
    assert 1 < np.abs(s).max() < 16  # what the case is to be
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    ref, weight = [np.einsum("hn,nhd->hd", p, x).repeat(2, 0)[None] / t for x in (v, np.abs(v))]
    rows = torch.full((150, 2 * hkv, d), q, dtype=torch.bfloat16).cuda()
    for label, got in _calls(cache, rows, pools, n, scale, t, hkv):
        close(got.float() / t, ref, weight, np.abs(v).max() / t * 2.0 ** -32, n, label)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("cache", ["q4", "e4m3"])
@pytest.mark.parametrize("power", [30, 64])
def test_zero_scores_of_a_large_q(cache, power):
    """q.K is 0 at every key: the mean of V, however large q and the tensor scale are."""
    n, hkv, d, t = 300, 2, 128, 2.0 ** power
    gen = torch.Generator().manual_seed(4)
    k = torch.randn(n, hkv, d, generator=gen)
    k[..., :16] = 0
    v = torch.randn(n, hkv, d, generator=gen)
    q = torch.zeros(150, 2 * hkv, d, dtype=torch.bfloat16)
    q[..., :16] = 2.0 ** 120
    pools, (_, value) = _pools(cache, *[(x * t).to(torch.bfloat16) for x in (k, v)], t)
    ref, weight = [x.mean(0).repeat(2, 0)[None] / t for x in (value, np.abs(value))]
    for label, got in _calls(cache, q.cuda(), pools, n, 0.1, t, hkv):
        close(got.float() / t, ref, weight, np.abs(value).max() / t * 2.0 ** -32, n, label)
    assert pkv.device_error() == 0
