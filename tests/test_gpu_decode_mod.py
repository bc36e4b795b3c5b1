"""GPU parity of paged_decode_attn_mod (softcap, distance bias, first visible key) against the float64 oracle."""

import numpy as np
import pytest
import torch

import pagedattention_kv_cache_gb300 as pkv
from pagedattention_kv_cache_gb300 import _lib
from pagedattention_kv_cache_gb300 import metadata as md
from pagedattention_kv_cache_gb300 import workloads as wl
from oracle import modified as omod

from _harness import as_np
from _modified import check, cuda, i32, slopes_of

pytestmark = pytest.mark.gpu


def _weights(dtype):
    """Type of the weights in the P V product: bf16 on the tensor-core kernel (bf16 caches), else fp32."""
    return dtype


def _case(seed, *, lens, block_size, hq, hkv, d=128, dtype=torch.bfloat16, q_scale=3.0):
    rng = np.random.default_rng(seed)
    blocks = sum(-(-n // block_size) for n in lens) + 5
    tables = wl._assign_blocks(rng, lens, block_size, blocks)
    gen = torch.Generator().manual_seed(seed)
    q = (torch.randn(len(lens), hq, d, generator=gen) * q_scale).to(dtype)
    kc, vc = [torch.randn(blocks, block_size, hkv, d, generator=gen).to(dtype) for _ in range(2)]
    return q, kc, vc, tables, i32(md.table_matrix(tables)), i32(lens)


def _hide(kc, vc, tables, lens, first, block_size, table):
    """NaN and infinities wherever no sequence sees a key; ids of blocks wholly outside are made invalid."""
    seen = torch.zeros(kc.shape[:2], dtype=torch.bool)
    table = table.clone()
    for b, (blocks, n) in enumerate(zip(tables, lens)):
        lo = max(0, int(first[b])) if first is not None else 0
        for t in range(min(lo, n), n):
            seen[blocks[t // block_size], t % block_size] = True
        table[b, : min(lo, n) // block_size] = 1 << 30
        if lo >= n:
            table[b] = -7
    kc[~seen], vc[~seen] = float("nan"), float("inf")
    return table


def _run(q, kc, vc, table, lens, scale, splits=0, **mods):
    out = pkv.paged_decode_attn_mod(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), scale, num_splits=splits,
                                    **{k: cuda(v) for k, v in mods.items()})
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    return out


def _compare(seed, lens, first, cap, alibi, *, splits=0, block_size=16, hq=8, hkv=2, d=128, dtype=torch.bfloat16,
             q_scale=3.0):
    q, kc, vc, tables, table, ln = _case(seed, lens=lens, block_size=block_size, hq=hq, hkv=hkv, d=d, dtype=dtype,
                                         q_scale=q_scale)
    first = None if first is None else i32(first)
    slopes = slopes_of(hq) if alibi else None
    ref, dev = omod.decode_attention(as_np(q), as_np(kc), as_np(vc), table.numpy(), lens, d ** -0.5, cap, slopes, first)
    table = _hide(kc, vc, tables, lens, first, block_size, table)
    out = _run(q, kc, vc, table, ln, d ** -0.5, splits, softcap=cap, alibi_slopes=slopes, first_keys=first)
    check(out, ref, dev, _weights(dtype), max(lens, default=0), f"cap {cap} alibi {alibi} first {first is not None}")
    return out


LENS = [0, 1, 2, 17, 64, 65, 300, 1111]
FIRST = [0, 0, 1, -5, 63, 66, 37, 1000]


@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("group,hkv", [(1, 8), (2, 3), (4, 2), (8, 1)])
@pytest.mark.parametrize("cap,alibi,first", [(50.0, False, False), (0.0, True, False), (0.0, False, True),
                                             (20.0, True, True)])
def test_bf16_every_group_and_modifier(splits, group, hkv, cap, alibi, first):
    _compare(group + splits, LENS, FIRST if first else None, cap, alibi, splits=splits, hq=group * hkv, hkv=hkv)


@pytest.mark.parametrize("block_size", [1, 5, 8, 16, 24, 48, 256])
def test_block_sizes(block_size):
    _compare(block_size, LENS, FIRST, 30.0, True, block_size=block_size)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.float32, 64), (torch.float32, 128)])
@pytest.mark.parametrize("group,hkv", [(1, 3), (2, 8), (4, 1), (8, 2)])
@pytest.mark.parametrize("splits", [0, 4])
@pytest.mark.parametrize("block_size", [24, 16])
def test_other_types_and_head_dims(dtype, d, group, hkv, splits, block_size):
    _compare(90 + group, LENS, FIRST, 30.0, True, splits=splits, hq=group * hkv, hkv=hkv, d=d, dtype=dtype,
             block_size=block_size)


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.bfloat16), (64, torch.float32)])
def test_many_short_sequences(d, dtype):
    # more sequences than threads of a block, most of them a token or two (or none) long
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 4, size=500).tolist()
    lens[77], lens[400] = 900, 333
    first = [int(x) for x in rng.integers(-1, 3, size=500)]
    _compare(22, lens, first, 30.0, True, d=d, dtype=dtype)


def test_no_modifier_is_the_plain_call():
    q, kc, vc, _, table, lens = _case(5, lens=LENS, block_size=16, hq=8, hkv=2)
    out = _run(q, kc, vc, table, lens, 0.1)
    plain = pkv.paged_decode_attn(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), 0.1)
    assert torch.equal(out, plain)


def test_window_of_every_offset_in_a_box():
    # the first visible key at each place of a 16-token box, and of a block that is not a multiple of one
    for block_size in (16, 24):
        _compare(7, [200] * 33, list(range(100, 133)), 0.0, False, block_size=block_size)


def test_scores_far_beyond_the_cap():
    # raw scores reach hundreds of times the cap, where tanh is 1 to the last bit
    q, kc, vc, _, table, lens = _case(8, lens=[40, 333], block_size=16, hq=4, hkv=2, q_scale=300.0)
    ref, dev = omod.decode_attention(as_np(q), as_np(kc), as_np(vc), table.numpy(), [40, 333], 128 ** -0.5, 5.0)
    check(_run(q, kc, vc, table, lens, 128 ** -0.5, softcap=5.0), ref, dev, torch.bfloat16, 333)


@pytest.mark.parametrize("cap", [1e-30, 1e-3, 1.0, 300.0, 1e4, 1e6, 1e30])
@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_caps_of_every_size(cap, dtype, d):
    _compare(21, LENS, None, cap, False, d=d, dtype=dtype)


def test_scores_that_overflow_are_capped():
    # every product of a key has that key's sign and is beyond float32: the score is +-infinity, the capped score
    # +-5.  (Products of both signs would sum to infinity - infinity, which float32 scores leave undefined.)
    q, kc, vc, _, table, lens = _case(8, lens=[40, 333], block_size=16, hq=4, hkv=2, q_scale=1e30)
    q, kc = q.abs().clamp_min(1e30), kc.abs().clamp_min(1.0) * torch.sign(kc[..., :1].float()).bfloat16() * 1e9
    ref, dev = omod.decode_attention(as_np(q), as_np(kc), as_np(vc), table.numpy(), [40, 333], 128 ** -0.5, 5.0)
    check(_run(q, kc, vc, table, lens, 128 ** -0.5, softcap=5.0), ref, dev, torch.bfloat16, 333)


def test_long_context_window_and_bias():
    lens = [20000, 33333, 9]
    _compare(9, lens, [19000, 33332, 0], 50.0, True, block_size=256, hq=16, hkv=8)
    _compare(10, lens, None, 0.0, True, block_size=16, hq=8, hkv=2)


def test_pool_past_32_bit_offsets():
    # element offsets beyond 2^31 and byte offsets beyond 2^32 in both pools
    bs, hkv, d, hq = 256, 8, 128, 16
    blocks = (1 << 31) // (bs * hkv * d) + 40
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(3)
    kc, vc = [torch.zeros(blocks, bs, hkv, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    ids = [blocks - 1, 3, blocks - 17, blocks - 2]
    for c in (kc, vc):
        c[ids] = torch.randn(4, bs, hkv, d, generator=gen, device=dev).bfloat16()
    q = torch.randn(1, hq, d, generator=gen, device=dev).bfloat16()
    table = i32([ids])
    out = pkv.paged_decode_attn_mod(q, kc, vc, table.cuda(), i32([1000]).cuda(), 0.1, softcap=20.0,
                                    first_keys=i32([130]).cuda())
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    small = [as_np(c[ids]) for c in (kc, vc)]
    ref, dv = omod.decode_attention(as_np(q), *small, np.arange(4)[None], [1000], 0.1, 20.0, None, [130])
    check(out, ref, dv, torch.bfloat16, 1000)


def test_bad_lengths_and_pages_raise_bits():
    q, kc, vc, _, table, lens = _case(11, lens=[20, 20, 20], block_size=16, hq=4, hkv=2)
    bad_table, bad_lens = table.clone(), lens.clone()
    bad_table[0, 0], bad_lens[1] = kc.shape[0], 33
    pkv.device_error(reset=True)
    out = pkv.paged_decode_attn_mod(q.cuda(), kc.cuda(), vc.cuda(), bad_table.cuda(), bad_lens.cuda(), 0.1,
                                    first_keys=i32([3, 3, 3]).cuda())
    assert pkv.device_error() == _lib.DERR_BLOCK_RANGE | _lib.DERR_LEN_RANGE
    assert torch.count_nonzero(out[1]) == 0
    ref, dev = omod.decode_attention(as_np(q), as_np(kc), as_np(vc), table.numpy(), [20, 20, 20], 0.1, 0.0, None, [3, 3, 3])
    check(out[2:], ref[2:], dev[2:], torch.bfloat16, 20)


def test_captured_without_a_workspace():
    q, kc, vc, _, table, lens = [cuda(x) for x in _case(14, lens=[3000, 650, 33, 0], block_size=16, hq=8, hkv=2)]
    call = lambda: pkv.paged_decode_attn_mod(q, kc, vc, table, lens, 0.1, softcap=20.0)  # noqa: E731
    ref = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and pkv.device_error() == 0


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.bfloat16), (64, torch.float32)])
@pytest.mark.parametrize("splits", [0, 1])
def test_nan_reaches_only_the_rows_that_see_it(d, dtype, splits):
    lens = [1500, 40, 1500, 1]
    q, kc, vc, tables, table, ln = _case(15, lens=lens, block_size=16, hq=4, hkv=2, d=d, dtype=dtype)
    first = i32([0, 0, 700, 0])
    ref, dev = omod.decode_attention(as_np(q), as_np(kc), as_np(vc), table.numpy(), lens, 0.1, 20.0, None, first)
    q[0, 3, 5] = float("nan")  # a head of the first sequence
    kc[tables[2][0], 3, 1, 0] = float("nan")  # a key before the third sequence's first
    kc[tables[2][80], 3, 0, 0] = float("nan")  # one after it, of KV head 0
    kc[tables[3][0], 0, 1, 0] = float("nan")  # the only key of the last, of KV head 1
    out = _run(q, kc, vc, table, ln, 0.1, splits, softcap=20.0, first_keys=first)
    want = torch.zeros(4, 4, dtype=torch.bool)
    want[0, 3], want[2, :2], want[3, 2:] = True, True, True
    bad = torch.isnan(out).all(-1)
    assert torch.equal(bad.cpu(), want)
    check(out[~bad], ref[~want.numpy()], dev[~want.numpy()], _weights(dtype), 1500)


def test_empty_batch():
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(0, 1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    assert pkv.paged_decode_attn_mod(q, kc, kc, table, lens, 0.1, softcap=5.0).shape == q.shape
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes = torch.zeros(4, 16, 2, 128, dtype=torch.uint8, device="cuda")
    assert pkv.paged_varlen_prefill_attn_mod(q, cu, cu, 0, 0, 0.1, k_cache=kc, v_cache=kc, block_tables=table).shape == q.shape
    assert pkv.paged_varlen_prefill_attn_fp8(q, codes, codes, table, cu, cu, 0, 0, 0.1, 1.0, 1.0).shape == q.shape
    assert pkv.device_error() == 0


def test_binding_refusals():
    q, kc, vc, _, table, lens = [cuda(x) for x in _case(12, lens=[20, 20], block_size=16, hq=4, hkv=2)]
    call = pkv.paged_decode_attn_mod
    with pytest.raises(ValueError, match="alibi_slopes must have shape"):
        call(q, kc, vc, table, lens, 0.1, alibi_slopes=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError, match="alibi_slopes must be"):
        call(q, kc, vc, table, lens, 0.1, alibi_slopes=torch.ones(4, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError, match="first_keys must have shape"):
        call(q, kc, vc, table, lens, 0.1, first_keys=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="first_keys must be"):
        call(q, kc, vc, table, lens, 0.1, first_keys=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        call(q, kc, vc, table, lens, 0.1, first_keys=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        call(q, kc, vc, table, lens, 0.1, alibi_slopes=torch.ones(8, device="cuda")[::2])
    with pytest.raises(ValueError, match="out must have shape"):
        call(q, kc, vc, table, lens, 0.1, out=torch.empty_like(q[:1]))
    for cap in (-1.0, float("nan"), float("inf")):
        with pytest.raises(_lib.PagedKVError):
            call(q, kc, vc, table, lens, 0.1, softcap=cap)
    assert pkv.device_error() == 0


def test_captured_step_with_new_windows_and_another_stream():
    # one captured call replayed with new lengths, windows and tables, beside eager calls on another
    # stream with a workspace of their own; results equal the eager ones bit for bit
    hq, hkv, bs = 8, 2, 16
    q, kc, vc, _, table, lens = [cuda(x) for x in _case(13, lens=[700, 650, 33, 0], block_size=bs, hq=hq, hkv=hkv)]
    slopes = slopes_of(hq).cuda()
    first, out = i32([0, 0, 0, 0]).cuda(), torch.empty_like(q)
    ws = pkv.decode_workspace(4, hq, 128)

    def step(stream=None, workspace=ws, out=out):
        return pkv.paged_decode_attn_mod(q, kc, vc, table, lens, 0.1, softcap=20.0, alibi_slopes=slopes, first_keys=first,
                                         workspace=workspace, out=out, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for new_first, new_lens in (([0, 0, 0, 0], [700, 650, 33, 0]), ([500, 649, 33, 0], [700, 650, 33, 0]),
                                ([3, 90, 0, 0], [4, 600, 1, 0])):
        first.copy_(i32(new_first))
        lens.copy_(i32(new_lens))
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        other = step(stream=side, workspace=None, out=None)
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        assert torch.equal(out, other)
        ref, dev = omod.decode_attention(as_np(q), as_np(kc), as_np(vc), table.cpu().numpy(), new_lens, 0.1, 20.0,
                                         slopes.cpu().numpy(), new_first)
        check(out, ref, dev, torch.bfloat16, 700, f"replay {new_first}")
