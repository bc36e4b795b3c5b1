"""GPU parity of decode and chunk attention over the 4-bit cache.

Tolerance per element, against the float64 oracle on the values the cache stands for,
with A = sum_t p_t |v_t| (the oracle's attention over |V|):
    2^-8 |out|        the output's bf16 rounding (half a step)
  + 2^-10 A           weights enter the P V product as f16, 2^-11 each, in the sum and in its divisor
  + 2^-13 A           scores in float32: |s| < 64 off by 2^-21, and exp2's own error, far inside
  + 2^-32 T max|v|    f16 weights below 2^-14 are multiples of 2^-24, off by half of one.  The row's largest
                      is at least 2^7 (the reference they count from is 7 below the maximum, or less where the
                      maximum has grown since), so each of a row's T keys is off by 2^-25 / 2^7 of the largest
                      p_t <= 1.  Where the heavy keys' element is 0, nothing else is left of it.
Element by element; no mean is taken.
"""

import numpy as np
import pytest
import torch

import pagedattention_kv_cache_gb300 as pkv
from pagedattention_kv_cache_gb300 import _lib
from pagedattention_kv_cache_gb300 import metadata as md
from oracle import attention as oa
from oracle import q4 as oq

from _harness import as_np

pytestmark = pytest.mark.gpu

T_K, T_V = 1.0 / 64, 3.0 / 256


def close(got, ref, weight, unit, keys, label=""):
    g = got.detach().double().cpu().numpy()
    assert np.isfinite(g).all(), f"{label}: non-finite"
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2.0 ** -13) * weight + keys * unit + 1e-30
    worst = float((np.abs(g - ref) / bound).max()) if g.size else 0.0
    assert worst <= 1.0, f"{label}: {worst:.3f} of the bound"


def _rows(n, hkv, d, gen, t):
    """n random 4-bit rows, quantized from normal values."""
    x = torch.randn(n, hkv, d, generator=gen).cuda().to(torch.bfloat16)
    pool = torch.zeros(n, 1, oq.row_bytes(hkv, d), dtype=torch.uint8, device="cuda")
    pkv.kv_store_q4(x, x, pool, pool.clone(), torch.arange(n, dtype=torch.int32, device="cuda"), t, t)
    return pool[:, 0]


def _pools(seed, lens, bs, hkv, d, poison=True):
    """Tables and 4-bit K, V pools; every row outside the contexts has NaN scales and random codes."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // bs) for n in lens]
    blocks = sum(need) + 2
    order, at, tables = torch.randperm(blocks, generator=gen).tolist(), 0, []
    for n in need:
        tables.append(order[at:at + n])
        at += n
    pools = []
    for t in (T_K, T_V):
        rows = _rows(blocks * bs, hkv, d, gen, t)
        if poison:
            used = torch.zeros(blocks * bs, dtype=torch.bool)
            for table, n in zip(tables, lens):
                for j, b in enumerate(table):
                    used[b * bs:b * bs + max(0, min(bs, n - j * bs))] = True
            junk = torch.randint(0, 256, rows.shape, generator=gen, dtype=torch.uint8)
            junk[:, hkv * d // 2:] = 0x7F
            rows[~used.cuda()] = junk[~used].cuda()
        pools.append(rows.view(blocks, bs, -1))
    return gen, tables, pools[0], pools[1]


def _reference(attend, k_pool, v_pool, hkv, d):
    """attend(k, v) on the values, and on |v|, and 2^-32 max|v|; rows that no context holds become zeros."""
    k = np.nan_to_num(oq.values(k_pool.cpu().numpy(), hkv, d, T_K))
    v = np.nan_to_num(oq.values(v_pool.cpu().numpy(), hkv, d, T_V))
    return attend(k, v), attend(k, np.abs(v)), float(np.abs(v).max()) * 2.0 ** -32


def decode_case(seed, lens, bs, hkv, g, d, splits=0, q_scale=1.0, scale=None, workspace=None):
    gen, tables, kp, vp = _pools(seed, lens, bs, hkv, d)
    scale = d ** -0.5 if scale is None else scale
    q = (torch.randn(len(lens), hkv * g, d, generator=gen) * 3 * q_scale).to(torch.bfloat16)
    bt, cl = md.table_matrix(tables), np.asarray(lens, dtype=np.int32)
    out = pkv.paged_decode_attn_q4(q.cuda(), kp, vp, torch.from_numpy(bt).cuda(), torch.from_numpy(cl).cuda(), scale, T_K,
                                   T_V, hkv, num_splits=splits, workspace=workspace)
    assert pkv.device_error() == 0
    ref = _reference(lambda k, v: oa.paged_decode_attention(as_np(q), k, v, bt, cl, scale), kp, vp, hkv, d)
    close(out, *ref, max(lens), f"decode {lens[:4]} bs {bs} hkv {hkv} G {g} d {d} splits {splits}")
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("hkv", [1, 2, 3, 8])
def test_decode_heads(d, g, hkv):
    decode_case(d + g + hkv, [0, 1, 15, 16, 17, 33, 300, 64, 1200, 31], 16, hkv, g, d)


@pytest.mark.parametrize("bs", [1, 5, 8, 16, 24, 32, 100, 128, 256])
@pytest.mark.parametrize("splits", [0, 1, 3, 40])
def test_decode_blocks_and_splits(bs, splits):
    decode_case(bs, [517, 0, 1, 130, 2, 256], bs, 4, 2, 128, splits)
    decode_case(bs, [517, 0, 1, 130, 2, 256], bs, 3, 4, 64, splits)


def test_decode_batches():
    decode_case(1, [777], 16, 8, 2, 128)
    decode_case(2, [20000], 16, 8, 4, 128)
    decode_case(3, list(range(0, 700, 2)), 32, 2, 2, 64)
    decode_case(4, [0, 0, 0], 16, 2, 2, 64)


@pytest.mark.parametrize("q_scale", [1e-30, 1e-6, 3e4, 1e30])
def test_decode_q_of_any_magnitude(q_scale):
    # the scale takes the magnitude off again, so the scores are ordinary
    decode_case(5, [100, 40, 3], 16, 2, 4, 128, q_scale=q_scale, scale=0.08 / q_scale)


def test_decode_flat_tail_counts():
    # one dominant key and a long flat tail: weights of 2^-26 of the largest, whose mass is still 2^-9
    hkv, d, n, bs = 1, 128, 131072, 256
    kp = pkv.q4_cache(n // bs, bs, hkv, d)
    vp = pkv.q4_cache(n // bs, bs, hkv, d)
    k = torch.zeros(1, hkv, d, dtype=torch.bfloat16, device="cuda")
    k[..., 0] = 7.0
    v = torch.ones(n, hkv, d, dtype=torch.bfloat16, device="cuda") * 7
    v[0] = 0
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    pkv.kv_store_q4(torch.cat([k, torch.zeros(n - 1, hkv, d, dtype=torch.bfloat16, device="cuda")]), v, kp, vp, slots, 1.0, 1.0)
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    gap = 26 * np.log(2.0)
    out = pkv.paged_decode_attn_q4(q, kp, vp, slots[:n // bs].view(1, -1), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                   gap / 7, 1.0, 1.0, hkv)
    tail = (n - 1) * 2.0 ** -26
    # the tail's weights are f16 multiples of 2^-32 of the largest: exact here but for exp2; bf16 output
    want = 7 * tail / (1 + tail)
    assert abs(out.double().cpu().numpy() - want).max() <= want * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -13)


def test_decode_nan_shows_only_where_it_is_seen():
    lens, bs, hkv, d = [700, 90, 64], 16, 2, 128
    gen, tables, kp, vp = _pools(7, lens, bs, hkv, d)
    q = torch.randn(3, 4, d, generator=gen).to(torch.bfloat16).cuda()
    bt, cl = torch.from_numpy(md.table_matrix(tables)).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    args = (bt, cl, d ** -0.5, T_K, T_V, hkv)
    for splits in (0, 1, 4):
        clean = pkv.paged_decode_attn_q4(q, kp, vp, *args, num_splits=splits)
        bad = kp.clone()
        bad[tables[0][40], 3, hkv * d // 2 + 5] = 0x7F  # head 0 of sequence 0
        got = pkv.paged_decode_attn_q4(q, bad, vp, *args, num_splits=splits)
        assert torch.isnan(got[0, :2]).all() and torch.equal(got[0, 2:], clean[0, 2:]) and torch.equal(got[1:], clean[1:])
        # a whole context of NaN keys
        bad = kp.clone()
        bad[tables[1], :, hkv * d // 2:] = 0x7F
        got = pkv.paged_decode_attn_q4(q, bad, vp, *args, num_splits=splits)
        assert torch.isnan(got[1]).all() and torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    assert pkv.device_error() == 0


def test_decode_repeats_and_shares_its_workspace():
    lens = [3000, 17, 900, 0, 64]
    gen, tables, kp, vp = _pools(8, lens, 16, 4, 128)
    q = torch.randn(5, 8, 128, generator=gen).to(torch.bfloat16).cuda()
    bt, cl = torch.from_numpy(md.table_matrix(tables)).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ws = pkv.decode_workspace(64, 32, 128)
    first = pkv.paged_decode_attn_q4(q, kp, vp, bt, cl, 0.1, T_K, T_V, 4, workspace=ws)
    for seed in range(3):
        decode_case(20 + seed, [5000, 3], 16, 2, 4, 64, workspace=ws)
        assert torch.equal(first, pkv.paged_decode_attn_q4(q, kp, vp, bt, cl, 0.1, T_K, T_V, 4, workspace=ws))
    assert torch.equal(first, pkv.paged_decode_attn_q4(q, kp, vp, bt, cl, 0.1, T_K, T_V, 4))
    with pytest.raises(_lib.PagedKVError):
        pkv.paged_decode_attn_q4(q, kp, vp, bt, cl, 0.1, T_K, T_V, 4, workspace=ws[:256])


def chunk_case(seed, history, new, bs, hkv, g, d, causal=True, workspace=None, q_scale=1.0, scale=None):
    lens = [h + n for h, n in zip(history, new)]
    gen, tables, kp, vp = _pools(seed, lens, bs, hkv, d)
    total = sum(new)
    scale = d ** -0.5 if scale is None else scale
    q = (torch.randn(total, hkv * g, d, generator=gen) * 3 * q_scale).to(torch.bfloat16)
    bt = md.table_matrix(tables)
    cu_q = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    out = torch.full((total + 3, hkv * g, d), 5.0, dtype=torch.bfloat16, device="cuda")
    got = pkv.paged_varlen_prefill_attn_q4(q.cuda(), kp, vp, *[torch.from_numpy(x).cuda() for x in (bt, cu_q, cu_k)],
                                           max(new), max(lens), scale, T_K, T_V, hkv, causal=causal,
                                           workspace=workspace, out=out[:total])
    assert pkv.device_error() == 0
    assert (out[total:] == 5.0).all()  # rows behind the last sequence
    ref = _reference(lambda k, v: oa.paged_prefill_attention(as_np(q), cu_q, cu_k, scale, k_cache=k, v_cache=v,
                                                             block_tables=bt, causal=causal), kp, vp, hkv, d)
    close(got, *ref, max(lens), f"chunk {history[:4]} + {new[:4]} bs {bs} hkv {hkv} G {g} d {d}")
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_chunk_heads(d, g, hkv):
    chunk_case(d + g + hkv, [0, 130, 7, 0], [40, 150, 1, 65], 16, hkv, g, d)


@pytest.mark.parametrize("bs", [1, 4, 8, 12, 16, 24, 32, 64, 96, 100, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_blocks(bs, d):
    chunk_case(bs, [200, 0, 33], [70, 129, 128], bs, 2, 2, d)


@pytest.mark.parametrize("causal", [True, False])
def test_chunk_lengths(causal):
    chunk_case(1, [0], [1], 16, 2, 2, 128, causal)
    chunk_case(2, [0, 0, 5], [128, 256, 0], 16, 2, 2, 64, causal)
    chunk_case(3, [1000, 127, 128], [300, 1, 129], 32, 1, 8, 128, causal)


@pytest.mark.parametrize("workspace", [None, False])
def test_chunk_long_history_split_and_not(workspace):
    chunk_case(4, [5000], [300], 16, 2, 2, 128, workspace=workspace)
    chunk_case(5, [4096, 100], [200, 30], 24, 1, 4, 64, workspace=workspace)


@pytest.mark.parametrize("g,ql", [(1, 8), (1, 3), (2, 4), (4, 2), (8, 1), (2, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_short_chunks(g, ql, d):
    new = [ql, 1, max(1, ql - 1), ql, 0]
    chunk_case(g + ql, [4000, 0, 2100, 33, 5], new, 16, 8, g, d)
    chunk_case(g + ql, [4000, 0, 2100, 33, 5], new, 5, 3, g, d, causal=False)
    chunk_case(g + ql, [int(x) for x in np.random.default_rng(1).integers(0, 60, 70)], [ql] * 70, 16, 4, g, d)


@pytest.mark.parametrize("q_scale", [1e-30, 3e4, 1e30])
def test_chunk_q_of_any_magnitude(q_scale):
    chunk_case(6, [100, 40], [200, 3], 16, 2, 4, 128, q_scale=q_scale, scale=0.08 / q_scale)
    chunk_case(6, [3000, 40], [4, 3], 16, 2, 2, 128, q_scale=q_scale, scale=0.08 / q_scale)


def test_chunk_nan_shows_only_where_it_is_seen():
    for history, new in (([900, 300], [150, 90]), ([3000, 2000], [4, 4])):
        lens = [h + n for h, n in zip(history, new)]
        gen, tables, kp, vp = _pools(9, lens, 16, 2, 128)
        total = sum(new)
        q = torch.randn(total, 4, 128, generator=gen).to(torch.bfloat16).cuda()
        ints = [torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, new[0], total], [0, lens[0], sum(lens)])]
        args = (torch.from_numpy(md.table_matrix(tables)).cuda(), *ints, max(new), max(lens), 0.08, T_K, T_V, 2)
        for workspace in (None, False):
            clean = pkv.paged_varlen_prefill_attn_q4(q, kp, vp, *args, workspace=workspace)
            bad, at = kp.clone(), history[0] + 1  # a key that the first new token does not see
            bad[tables[0][at // 16], at % 16, 128 + 8 + 3] = 0x7F  # head 1
            got = pkv.paged_varlen_prefill_attn_q4(q, bad, vp, *args, workspace=workspace)
            rows = torch.arange(total, device="cuda")
            hit = ((rows >= 1) & (rows < new[0]))[:, None] & (torch.arange(4, device="cuda") >= 2)
            assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])
    assert pkv.device_error() == 0


@pytest.mark.parametrize("max_q", [6, 200])
def test_bad_lengths_and_blocks_raise_bits(max_q):
    gen, tables, kp, vp = _pools(10, [3000, 200], 16, 2, 128, poison=False)
    bt = torch.from_numpy(md.table_matrix(tables)).cuda()
    q = torch.randn(8, 4, 128, generator=gen).to(torch.bfloat16).cuda()

    def chunk(cu_q, cu_k, table=bt):
        out = torch.full_like(q, 9.0)
        pkv.paged_varlen_prefill_attn_q4(q, kp, vp, table, torch.tensor(cu_q, dtype=torch.int32).cuda(),
                                         torch.tensor(cu_k, dtype=torch.int32).cuda(), max_q, 3000, 0.1, T_K, T_V, 2, out=out)
        return out, pkv.device_error()

    pkv.device_error(reset=True)
    for cu_q, cu_k in (([0, 4, 9], [0, 100, 200]), ([0, 4, 8], [0, 3, 200]), ([-1, 4, 8], [0, 100, 200]),
                       ([0, 4, 8], [0, 100, 100000])):
        out, err = chunk(cu_q, cu_k)
        assert err == _lib.DERR_LEN_RANGE
        skipped = out[:4] if cu_k[1] == 3 or cu_q[0] < 0 else out[4:]
        assert (skipped == 9.0).all()
    wrong = bt.clone()
    wrong[0, 1], wrong[1, 2] = kp.shape[0], -1
    assert chunk([0, 4, 8], [0, 100, 200], wrong)[1] == _lib.DERR_BLOCK_RANGE
    cl = torch.tensor([100, 90], dtype=torch.int32).cuda()
    pkv.paged_decode_attn_q4(q[:2], kp, vp, wrong, cl, 0.1, T_K, T_V, 2)
    assert pkv.device_error() == _lib.DERR_BLOCK_RANGE
    cl[0] = -3
    out = pkv.paged_decode_attn_q4(q[:2], kp, vp, bt, cl, 0.1, T_K, T_V, 2)
    assert pkv.device_error() == _lib.DERR_LEN_RANGE and not out[0].any()
    cl[0] = bt.shape[1] * 16 + 1
    out = pkv.paged_decode_attn_q4(q[:2], kp, vp, bt, cl, 0.1, T_K, T_V, 2)
    assert pkv.device_error() == _lib.DERR_LEN_RANGE and not out[0].any()


@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-42, 3.0])
def test_decode_scales(scale):
    decode_case(31, [0, 1, 700, 64, 65], 16, 8, 2, 128, scale=scale)
    decode_case(32, [900, 3], 16, 2, 4, 64, scale=scale, splits=2)


@pytest.mark.parametrize("power", [-64, -50, 50, 64])
def test_tensor_scales_up_to_their_ends(power):
    """Values times 2^power, q's scale divided by it: the same scores, and outputs times 2^power, bit for bit."""
    hkv, d, bs, n, hq = 2, 128, 16, 3000, 8
    gen = torch.Generator().manual_seed(6)
    k, v = [torch.randn(n, hkv, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    q = torch.randn(n, hq, d, generator=gen).to(torch.bfloat16).cuda()
    slots = torch.arange(n, dtype=torch.int32).cuda()
    bt = torch.arange(-(-n // bs), dtype=torch.int32)[None].cuda()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    cu_k = torch.tensor([0, n], dtype=torch.int32).cuda()
    results = []
    for t in (1.0, 2.0 ** power):
        pools = [pkv.q4_cache(bt.shape[1], bs, hkv, d) for _ in range(2)]
        pkv.kv_store_q4((k.float() * t).to(torch.bfloat16), (v.float() * t).to(torch.bfloat16), *pools, slots, t, t)
        outs = [pkv.paged_decode_attn_q4(q[:1], *pools, bt, lens, 0.1 / t, t, t, hkv, num_splits=s) for s in (0, 1)]
        for new in (2, 200):
            cu_q = torch.tensor([0, new], dtype=torch.int32).cuda()
            outs += [pkv.paged_varlen_prefill_attn_q4(q[:new], *pools, bt, cu_q, cu_k, new, n, 0.1 / t, t, t, hkv, workspace=w)
                     for w in (None, False)]
        results.append([(o.float() / t) for o in outs])
    assert pkv.device_error() == 0
    for a, b in zip(*results):
        assert torch.equal(a, b) and torch.isfinite(a).all()


def test_rows_past_32_bits_of_bytes():
    """A pool of 4.5 GB: its last blocks give what the same rows give in a small pool, bit for bit."""
    hkv, d, bs, n, hq = 8, 128, 256, 1000, 16
    row = oq.row_bytes(hkv, d)
    blocks = (9 << 29) // (row * bs)
    gen = torch.Generator().manual_seed(5)
    k, v = [torch.randn(n, hkv, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    q = torch.randn(n, hq, d, generator=gen).to(torch.bfloat16).cuda()
    cu_q = torch.tensor([0, 300], dtype=torch.int32).cuda()
    cu_k = torch.tensor([0, n], dtype=torch.int32).cuda()
    lens = torch.tensor([n, n - 1], dtype=torch.int32).cuda()
    results = []
    for pool_blocks in (5, blocks):
        pools = [torch.zeros(pool_blocks, bs, row, dtype=torch.uint8, device="cuda") for _ in range(2)]
        order = pool_blocks - 1 - torch.tensor([2, 0, 3, 1])
        slots = (order[torch.arange(n) // bs] * bs + torch.arange(n) % bs).int().cuda()
        bt = order.int()[None].cuda()
        pkv.kv_store_q4(k, v, *pools, slots, T_K, T_V)
        results.append((*pkv.kv_load_q4(*pools, slots, T_K, T_V, hkv, d),
                        pkv.paged_decode_attn_q4(q[:2], *pools, bt.repeat(2, 1), lens, 0.1, T_K, T_V, hkv),
                        pkv.paged_varlen_prefill_attn_q4(q[:300], *pools, bt, cu_q, cu_k, 300, n, 0.1, T_K, T_V, hkv)))
        assert pkv.device_error() == 0
        del pools
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_refusals_of_the_binding():
    hkv, d = 2, 64
    kp, vp = pkv.q4_cache(4, 16, hkv, d), pkv.q4_cache(4, 16, hkv, d)
    q = torch.zeros(2, 4, d, dtype=torch.bfloat16, device="cuda")
    bt, cl = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")

    def decode(q=q, kp=kp, vp=vp, bt=bt, cl=cl, hkv=hkv, **kw):
        return pkv.paged_decode_attn_q4(q, kp, vp, bt, cl, 0.1, T_K, T_V, hkv, **kw)

    def chunk(q=q, kp=kp, vp=vp, bt=bt, cl=cu, hkv=hkv, **kw):
        return pkv.paged_varlen_prefill_attn_q4(q, kp, vp, bt, cl, cl, 1, 1, 0.1, T_K, T_V, hkv, **kw)

    for call in (decode, chunk):
        assert not call().any()
        for kw in (dict(q=q.cpu()), dict(q=q[0]), dict(q=q.transpose(0, 1)), dict(kp=kp[:2]), dict(vp=vp[..., :64]), dict(hkv=4),
                   dict(bt=bt[:1]), dict(bt=bt[0]), dict(out=q[:1]), dict(kp=kp.cpu())):
            with pytest.raises(ValueError):
                call(**kw)
        for kw in (dict(q=q.float()), dict(kp=kp.view(torch.int8)), dict(bt=bt.long()), dict(cl=cl.long()),
                   dict(out=torch.zeros(2, 4, d, device="cuda"))):
            with pytest.raises(TypeError):
                call(**kw)
    with pytest.raises(_lib.PagedKVError):
        decode(q=torch.zeros(2, 6, d, dtype=torch.bfloat16, device="cuda"))
    assert pkv.device_error() == 0


def test_a_serving_run():
    """Prompt, decode steps and drafted tokens with the rotating store, eager and captured, against the oracle."""
    hq, hkv, d, bs, base = 4, 2, 128, 16, 10000.0
    gen = torch.Generator().manual_seed(12)
    lens, blocks = [37, 130], 24
    tables = [list(range(0, 10)), list(range(10, 22))]
    bt = torch.from_numpy(md.table_matrix(tables)).cuda()
    table = md.rope_cos_sin(512, d, base)
    cs = torch.from_numpy(table).cuda()
    kp, vp = pkv.q4_cache(blocks, bs, hkv, d), pkv.q4_cache(blocks, bs, hkv, d)
    want_k, want_v = np.zeros((blocks, bs, kp.shape[2]), np.uint8), np.zeros((blocks, bs, kp.shape[2]), np.uint8)

    def places(starts, counts):
        pos = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, counts)]).astype(np.int32)
        slot = np.concatenate([[t[p // bs] * bs + p % bs for p in range(s, s + n)] for t, s, n in zip(tables, starts, counts)])
        return pos, slot.astype(np.int32)

    def step(starts, counts, call, graph):
        nonlocal want_k, want_v
        n = sum(counts)
        q, k, v = [torch.randn(n, h, d, generator=gen).to(torch.bfloat16) for h in (hq, hkv, hkv)]
        pos, slot = places(starts, counts)
        g = [x.cuda() for x in (q, k, v)] + [torch.from_numpy(x).cuda() for x in (pos, slot)]

        def run():
            turned = pkv.kv_rope_store_q4(g[0], g[1], g[2], g[3], cs, kp, vp, g[4], T_K, T_V)
            return call(turned)

        if graph:
            captured = torch.cuda.CUDAGraph()
            before = kp.clone(), vp.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                run()
            torch.cuda.current_stream().wait_stream(side)
            kp.copy_(before[0])
            vp.copy_(before[1])
            with torch.cuda.graph(captured):
                out = run()
            captured.replay()
        else:
            out = run()
        bf = lambda x: torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).float().numpy()  # noqa: E731
        want_k = oq.store(want_k, bf(oq.rotate(as_np(k), pos, table, False)), slot, T_K)
        want_v = oq.store(want_v, as_np(v), slot, T_V)
        assert np.array_equal(kp.cpu().numpy(), want_k) and np.array_equal(vp.cpu().numpy(), want_v)
        return out, bf(oq.rotate(as_np(q), pos, table, False))

    def chunk(starts, counts, graph):
        total = [s + n for s, n in zip(starts, counts)]
        cu_q, cu_k = [np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (counts, total)]
        gq, gk = torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda()
        out, q = step(starts, counts, lambda t: pkv.paged_varlen_prefill_attn_q4(
            t, kp, vp, bt, gq, gk, max(counts), max(total), 0.09, T_K, T_V, hkv), graph)
        ref = _reference(lambda k, v: oa.paged_prefill_attention(q, cu_q, cu_k, 0.09, k_cache=k, v_cache=v,
                                                                 block_tables=md.table_matrix(tables)), kp, vp, hkv, d)
        close(out, *ref, max(total), "run: chunk")

    chunk([0, 0], lens, False)
    for i, graph in enumerate((False, True, True)):
        now = [n + i + 1 for n in lens]
        cl = torch.tensor(now, dtype=torch.int32).cuda()
        out, q = step([n - 1 for n in now], [1, 1], lambda t: pkv.paged_decode_attn_q4(
            t, kp, vp, bt, cl, 0.09, T_K, T_V, hkv), graph)
        ref = _reference(lambda k, v: oa.paged_decode_attention(q, k, v, md.table_matrix(tables), np.array(now), 0.09), kp, vp,
                         hkv, d)
        close(out, *ref, max(now), "run: decode")
    chunk([n + 3 for n in lens], [4, 3], True)
    # the prefix moved to a bf16 cache: the plain decode over it agrees
    slots = torch.arange(blocks * bs, dtype=torch.int32, device="cuda")
    k16, v16 = [x.view(blocks, bs, hkv, d) for x in pkv.kv_load_q4(kp, vp, slots, T_K, T_V, hkv, d)]
    q = torch.randn(2, hq, d, generator=gen).to(torch.bfloat16).cuda()
    cl = torch.tensor([n + 6 for n in lens], dtype=torch.int32).cuda()
    a = pkv.paged_decode_attn_q4(q, kp, vp, bt, cl, 0.09, T_K, T_V, hkv).double()
    b = pkv.paged_decode_attn(q, k16, v16, bt, cl, 0.09).double()
    # V loses up to 2^-8 of itself in bf16 (T_V is no power of two), both outputs are bf16, weights are bf16 there
    assert (a - b).abs().max() <= 4 * 2.0 ** -8 * v16.abs().max()
    # copy-on-write of a 4-bit block
    pkv.copy_blocks([kp], [vp], torch.tensor([[0, 22]], dtype=torch.int32, device="cuda"))
    assert torch.equal(kp[22], kp[0]) and torch.equal(vp[22], vp[0]) and pkv.device_error() == 0
