"""GPU parity of paged_varlen_prefill_attn_fp8 (a chunk of new tokens over an E4M3 cache) against the
float64 oracle on the dequantized cache."""

import numpy as np
import pytest
import torch

import pagedattention_kv_cache_gb300 as pkv
from pagedattention_kv_cache_gb300 import _lib
from pagedattention_kv_cache_gb300 import metadata as md
from pagedattention_kv_cache_gb300 import workloads as wl
from oracle import fp8 as of8
from oracle import modified as omod

from _harness import as_np
from _modified import SCORE, check, i32

pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 1.0 / 64, 3.0 / 256
CACHED, NEW = [0, 16, 0, 130, 300, 5], [1, 40, 129, 0, 260, 3]


def _codes(shape, gen, scale):
    return torch.from_numpy(of8.quantize(torch.randn(shape, generator=gen).bfloat16().float().numpy(), scale))


class Case:
    def __init__(self, seed, cached, new, *, block_size=16, hq=8, hkv=2, d=128, q_scale=1.0):
        rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.new, self.bs, self.hq, self.hkv, self.d, self.scale = new, block_size, hq, hkv, d, d ** -0.5
        self.totals = [c + n for c, n in zip(cached, new)]
        blocks = sum(-(-n // block_size) for n in self.totals) + 5
        self.tables = wl._assign_blocks(rng, self.totals, block_size, blocks)
        self.table = i32(md.table_matrix(self.tables))
        self.kc, self.vc = [_codes((blocks, block_size, hkv, d), gen, s) for s in (K_SCALE, V_SCALE)]
        self.q = (torch.randn(sum(new), hq, d, generator=gen) * q_scale).bfloat16()
        self.cu_q, self.cu_k = i32([0] + np.cumsum(new).tolist()), i32([0] + np.cumsum(self.totals).tolist())

    def poison(self):
        """The E4M3 NaN in every slot that holds no key of a sequence."""
        seen = torch.zeros(self.kc.shape[:2], dtype=torch.bool)
        for blocks, total in zip(self.tables, self.totals):
            for t in range(total):
                seen[blocks[t // self.bs], t % self.bs] = True
        self.kc[~seen], self.vc[~seen] = 0x7F, 0xFF

    def reference(self, causal=True):
        return omod.prefill_attention(as_np(self.q), self.cu_q.tolist(), self.cu_k.tolist(), self.scale,
                                      k_cache=of8.dequantize(self.kc.numpy(), K_SCALE),
                                      v_cache=of8.dequantize(self.vc.numpy(), V_SCALE), block_tables=self.table.numpy(),
                                      causal=causal)

    def call(self, causal=True, **kw):
        return pkv.paged_varlen_prefill_attn_fp8(self.q.cuda(), self.kc.cuda(), self.vc.cuda(), self.table.cuda(),
                                                 self.cu_q.cuda(), self.cu_k.cuda(), max(self.new), max(self.totals),
                                                 self.scale, K_SCALE, V_SCALE, causal=causal, **kw)

    def compare(self, causal=True, label="", **kw):
        ref, dev = self.reference(causal)
        self.poison()
        out = self.call(causal, **kw)
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        check(out, ref, dev, torch.float16, max(self.totals), label)
        return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,hkv", [(1, 3), (2, 2), (4, 1), (8, 1)])
@pytest.mark.parametrize("block_size", [16, 24, 256])
def test_every_group_and_head_dim(d, group, hkv, block_size):
    Case(group + d + block_size, CACHED, NEW, block_size=block_size, hq=group * hkv, hkv=hkv, d=d).compare()


@pytest.mark.parametrize("block_size", [1, 4, 5, 8, 32, 64, 100, 128, 384])
def test_block_sizes(block_size):
    Case(block_size, CACHED, NEW, block_size=block_size, d=64 if block_size % 5 == 0 else 128).compare()


def test_full_attention():
    for d in (64, 128):
        Case(d, CACHED, NEW, d=d).compare(causal=False)


# q far outside f16's range either way: each row is scaled by a power of two, and a row of zeros stays one
@pytest.mark.parametrize("q_scale", [0.0, 1e-37, 1e-30, 1e-6, 30.0, 3e4, 1e9, 1e36])
def test_q_magnitudes(q_scale):
    c = Case(61, [40, 0], [130, 20], q_scale=q_scale)
    c.q[5] = 0
    c.scale = c.d ** -0.5 * (min(1.0, 3.0 / q_scale) if q_scale else 1.0)  # scores of a few units
    c.compare(label=f"q x {q_scale}")


# the decode kernel's rows: a short chunk, and one decoded token per sequence
@pytest.mark.parametrize("q_scale", [1e-37, 1e9, 1e36])
def test_q_magnitudes_on_the_decode_kernel(q_scale):
    c = Case(75, [1500, 700, 40], [2, 1, 1], q_scale=q_scale)
    c.scale = c.d ** -0.5 * min(1.0, 3.0 / q_scale)  # scores of a few units
    assert pkv.chunk_workspace_bytes(3, c.hq, c.hkv, c.d, 2, 1502) > 0
    c.compare(label=f"chunk, q x {q_scale}")
    ref, dev = c.reference()
    out = pkv.paged_decode_attn_fp8(c.q[1:].cuda(), c.kc.cuda(), c.vc.cuda(), c.table.cuda(), i32(c.totals).cuda(), c.scale,
                                    K_SCALE, V_SCALE)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    check(out, ref[1:], dev[1:], torch.float16, 1502, f"decode, q x {q_scale}")


def test_codes_of_every_value():
    # every finite E4M3 code (subnormals among them) as K and as V
    codes = torch.tensor([x for x in range(256) if x & 0x7F != 0x7F], dtype=torch.uint8)
    c = Case(62, [0], [254], hkv=1, hq=2)
    gen = torch.Generator().manual_seed(1)
    for cache in (c.kc, c.vc):
        cache.copy_(codes[torch.randint(0, 254, cache.shape, generator=gen)])
    c.scale = 2e-4 / K_SCALE  # codes reach 448: scores of a few units
    c.compare()


@pytest.mark.parametrize("block_size", [16, 24, 256])
@pytest.mark.parametrize("group,hkv,new", [(1, 8, [4, 1, 8, 3, 0, 2]), (2, 8, [4, 1, 2, 3, 0, 4]), (2, 3, [4, 1, 2, 3, 0, 4]),
                                           (4, 2, [2, 1, 2, 0, 1, 2]), (8, 1, [1, 1, 1, 0, 1, 1])])
def test_short_chunks_on_the_decode_kernel(block_size, group, hkv, new):
    # drafted tokens after ragged histories, split over the SMs and merged
    c = Case(63, [1000, 17, 0, 255, 511, 2000], new, hq=group * hkv, hkv=hkv, block_size=block_size)
    assert pkv.chunk_workspace_bytes(6, c.hq, hkv, 128, max(new), 2004) > 0
    c.compare(label="causal")
    c.compare(causal=False, label="full")
    ws = pkv.chunk_workspace(6, c.hq, hkv, 128, max(new), 2004)
    a = c.compare(workspace=ws)
    assert torch.equal(a, c.compare(workspace=ws)) and int(ws[:65536].count_nonzero()) == 0


def test_short_chunks_of_more_sequences_than_threads():
    rng = np.random.default_rng(4)
    cached, new = rng.integers(0, 40, size=400).tolist(), rng.integers(0, 5, size=400).tolist()
    cached[7], cached[390] = 3000, 1500
    Case(70, cached, new, hq=4, hkv=2).compare()


def test_more_than_eight_kv_heads():
    Case(71, [100, 0, 700], [40, 130, 2], hq=12, hkv=12).compare()
    Case(72, [2000, 3], [2, 1], hq=48, hkv=12).compare()


def test_nan_reaches_only_the_rows_that_see_it():
    for new in (70, 4):  # the prefill kernel, and the decode kernel
        c = Case(73, [1500], [new], hq=2, hkv=1)
        ref, dev = c.reference()
        pos = 1500 + new - 3  # a NaN key that the last three rows see
        c.kc[c.tables[0][pos // 16], pos % 16, 0, 5] = 0x7F
        c.q[1, 0, 9] = float("nan")
        out = c.call()
        torch.cuda.synchronize()
        bad = torch.isnan(out).all(-1)
        want = torch.zeros(new, 2, dtype=torch.bool)
        want[new - 3:], want[1, 0] = True, True
        assert torch.equal(bad.cpu(), want)
        keep = ~want.numpy()
        check(out[~bad], ref[keep], dev[keep], torch.float16, 1600)


def test_captured_without_a_workspace():
    # the call's own workspace comes from the graph's pool, and its counters are zeroed in the graph
    for new in (60, 3):
        c = Case(74, [3000, 40], [new, 2], block_size=64, hq=4, hkv=2)
        q, kc, vc, table, cu_q, cu_k = [x.cuda() for x in (c.q, c.kc, c.vc, c.table, c.cu_q, c.cu_k)]
        call = lambda: pkv.paged_varlen_prefill_attn_fp8(q, kc, vc, table, cu_q, cu_k, new, 3000 + new, c.scale,  # noqa: E731
                                                         K_SCALE, V_SCALE)
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


def test_short_chunk_through_the_c_abi_without_its_workspace():
    # with no workspace, or one that is too small, the prefill kernel runs it
    c = Case(68, [1300, 17], [4, 2], hq=4, hkv=2)
    ref, dev = c.reference()
    q, kc, vc, table, cu_q, cu_k = [x.cuda() for x in (c.q, c.kc, c.vc, c.table, c.cu_q, c.cu_k)]
    small = torch.zeros(65536, dtype=torch.uint8, device="cuda")
    for ws, n in ((None, 0), (small.data_ptr(), small.numel())):
        out = torch.empty_like(q)
        st = _lib.load().pkv_paged_varlen_prefill_attn_fp8(
            out.data_ptr(), q.data_ptr(), kc.data_ptr(), vc.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), 4, 1304,
            table.data_ptr(), table.shape[1], 2, 6, 4, 2, 128, 16, kc.shape[0], c.scale, K_SCALE, V_SCALE, 1, ws, n,
            torch.cuda.current_stream().cuda_stream)
        assert st == _lib.OK
        torch.cuda.synchronize()
        check(out, ref, dev, torch.float16, 1304)
    assert pkv.device_error() == 0


def test_wide_chunks_of_drafted_tokens():
    # 1 to 8 drafted tokens with G = 2: more rows than a short chunk
    Case(63, [1000, 17, 0, 255, 511, 2000], [4, 1, 8, 3, 5, 2], hq=16, hkv=8, block_size=256).compare()


def test_split_key_ranges():
    c = Case(64, [6000, 3000], [70, 33], block_size=64, hq=4, hkv=2)
    assert pkv.prefill_workspace_bytes(2, 4, 2, 128, 70) > 0
    a = c.compare(label="split")
    c.compare(workspace=False, label="not split")
    ws = pkv.prefill_workspace(2, 4, 2, 128, 70)
    for _ in range(3):
        assert torch.equal(a, c.compare(workspace=ws))
    assert int(ws[:65536].count_nonzero()) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,workspace", [(9, False), (9, None), (4, None)])
def test_one_dominant_key_before_a_long_flat_tail(d, new, workspace):
    # key 0 scores 17.4, every other key 0: a tail key's weight is 2^-25.1 of the largest, 131072 of them
    # 0.36 % of the mass, and only they have a value.  A weight enters P V as f16 in units in which the row's
    # largest is 2^7 or more, so it is off by 2^-11 of itself or, as a subnormal, by 2^-25 of those units: 2^-32
    # of the largest weight
    tail = 131072
    c = Case(76, [tail], [new], block_size=256, hq=2, hkv=2, d=d)
    codes = torch.zeros_like(c.kc)
    codes[c.tables[0][0], 0, :, 3] = 0x7E  # 448 K_SCALE = 7
    c.kc, c.vc = codes, torch.full_like(c.vc, 0x7E)  # 448 V_SCALE = 5.25
    c.vc[c.tables[0][0], 0] = 0
    c.q.zero_()
    c.q[..., 3] = 1.0
    c.scale = 17.4 / 7
    ref, dev = c.reference()
    out = c.call(workspace=workspace)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    keys = tail + new
    allowed = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 * 1.01 + SCORE) * dev + keys * 2.0 ** -32 * 5.25 + keys * 2.0 ** -24 * ref
    assert 0.018 < ref.min() and (np.abs(out.double().cpu().numpy() - ref) <= allowed).all()


def test_pool_past_32_bit_offsets():
    bs, hkv, d, hq = 256, 8, 128, 16
    blocks = (1 << 32) // (bs * hkv * d) + 40
    gen = torch.Generator().manual_seed(3)
    ids = [blocks - 1, 3, blocks - 17]
    small = [_codes((3, bs, hkv, d), gen, s) for s in (K_SCALE, V_SCALE)]
    pools = [torch.zeros(blocks, bs, hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for pool, s in zip(pools, small):
        pool[ids] = s.cuda()
    q = torch.randn(40, hq, d, generator=gen).bfloat16()
    out = pkv.paged_varlen_prefill_attn_fp8(q.cuda(), *pools, i32([ids]).cuda(), i32([0, 40]).cuda(), i32([0, 600]).cuda(),
                                            40, 600, 0.1, K_SCALE, V_SCALE)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    ref, dev = omod.prefill_attention(as_np(q), [0, 40], [0, 600], 0.1, k_cache=of8.dequantize(small[0].numpy(), K_SCALE),
                                      v_cache=of8.dequantize(small[1].numpy(), V_SCALE), block_tables=np.arange(3)[None])
    check(out, ref, dev, torch.float16, 600)


def test_bad_cu_seqlens_and_pages_raise_bits():
    c = Case(65, [0, 16, 16], [20, 20, 20])
    ref, dev = c.reference()

    def call(cu_q, cu_k, max_q, table):
        pkv.device_error(reset=True)
        out = torch.full_like(c.q, 7.0).cuda()
        pkv.paged_varlen_prefill_attn_fp8(c.q.cuda(), c.kc.cuda(), c.vc.cuda(), table.cuda(), i32(cu_q).cuda(),
                                          i32(cu_k).cuda(), max_q, 64, c.scale, K_SCALE, V_SCALE, out=out)
        return pkv.device_error(), out

    for cu_q, cu_k, max_q in (([0, 20, 40, 61], [0, 20, 56, 92], 21), ([-1, 20, 40, 60], [0, 20, 56, 92], 21),
                              ([0, 20, 40, 60], [0, 20, 56, 92], 19), ([0, 20, 40, 60], [0, 19, 56, 92], 20),
                              ([0, 20, 40, 60], [0, 20, 56, 200], 20)):
        assert call(cu_q, cu_k, max_q, c.table)[0] == _lib.DERR_LEN_RANGE, (cu_q, cu_k, max_q)
    short = Case(69, [0, 16, 16], [2, 2, 2])  # the decode kernel's own checks
    for cu_q, cu_k, max_q in (([0, 2, 4, 7], [0, 2, 20, 38], 3), ([-1, 2, 4, 6], [0, 2, 20, 38], 3),
                              ([0, 2, 4, 6], [0, 2, 20, 38], 1), ([0, 2, 4, 6], [0, 1, 20, 38], 2),
                              ([0, 2, 4, 6], [0, 2, 20, 100], 2)):
        out = torch.full_like(short.q, 7.0).cuda()
        pkv.paged_varlen_prefill_attn_fp8(short.q.cuda(), short.kc.cuda(), short.vc.cuda(), short.table.cuda(),
                                          i32(cu_q).cuda(), i32(cu_k).cuda(), max_q, 2000, c.scale, K_SCALE, V_SCALE, out=out)
        assert pkv.device_error() == _lib.DERR_LEN_RANGE, (cu_q, cu_k, max_q)
        assert cu_k[-1] < 100 or torch.all(out[4:] == 7.0)  # a skipped sequence's rows are left alone
    bad = c.table.clone()
    bad[1, 0], bad[1, 2] = -1, c.kc.shape[0]
    bits, out = call([0, 20, 40, 60], [0, 20, 56, 92], 20, bad)
    assert bits == _lib.DERR_BLOCK_RANGE
    check(out[:20], ref[:20], dev[:20], torch.float16, 36)
    check(out[40:], ref[40:], dev[40:], torch.float16, 36)


def test_binding_refusals():
    c = Case(66, [0, 16], [8, 8])
    q, kc, vc, table, cu_q, cu_k = [x.cuda() for x in (c.q, c.kc, c.vc, c.table, c.cu_q, c.cu_k)]

    def call(q=q, kc=kc, vc=vc, table=table, ks=1.0, **kw):
        return pkv.paged_varlen_prefill_attn_fp8(q, kc, vc, table, cu_q, cu_k, 8, 24, 0.1, ks, 1.0, **kw)

    with pytest.raises(TypeError, match="E4M3"):
        call(kc=kc.float(), vc=vc.float())
    with pytest.raises(TypeError, match="E4M3"):
        call(kc=kc.view(torch.float8_e5m2), vc=vc.view(torch.float8_e5m2))
    with pytest.raises(TypeError, match="q must be"):
        call(q=q.float())
    with pytest.raises(ValueError, match="block_tables rows"):
        call(table=table[:1].contiguous())
    with pytest.raises(ValueError, match="head_dim differs"):
        call(kc=kc[..., :64].contiguous(), vc=vc[..., :64].contiguous())
    for ks in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(_lib.PagedKVError):
            call(ks=ks)
    with pytest.raises(_lib.PagedKVError):  # G = 3
        call(q=torch.zeros(16, 6, 128, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(call(kc=kc.view(torch.float8_e4m3fn), vc=vc.view(torch.float8_e4m3fn)), call())
    assert pkv.device_error() == 0


def test_captured_and_on_another_stream():
    c = Case(67, [900, 40], [60, 30], block_size=64, hq=4, hkv=2)
    q, kc, vc, table, cu_q, cu_k = [x.cuda() for x in (c.q, c.kc, c.vc, c.table, c.cu_q, c.cu_k)]
    out, ws = torch.empty_like(q), pkv.prefill_workspace(2, 4, 2, 128, 60)

    def step(**kw):
        return pkv.paged_varlen_prefill_attn_fp8(q, kc, vc, table, cu_q, cu_k, 60, 960, c.scale, K_SCALE, V_SCALE,
                                                 **dict(dict(workspace=ws, out=out), **kw))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    gen = torch.Generator().manual_seed(9)
    for _ in range(2):
        c.q = torch.randn(c.q.shape, generator=gen).bfloat16()
        q.copy_(c.q)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        other = step(stream=side, workspace=None, out=None)
        torch.cuda.synchronize()
        assert pkv.device_error() == 0 and torch.equal(out, other)
        ref, dev = c.reference()
        check(out, ref, dev, torch.float16, 960)


def test_quantizing_store_then_chunks_then_decode():
    # a prompt in two chunks and a decoded token over one E4M3 cache, each against the oracle
    bs, hq, hkv, d = 16, 8, 2, 128
    gen = torch.Generator().manual_seed(50)
    k, v = [torch.randn(150, hkv, d, generator=gen).bfloat16() for _ in range(2)]
    q = torch.randn(150, hq, d, generator=gen).bfloat16()
    table = [7, 2, 9, 0, 4, 8, 1, 3, 6, 5]
    kc, vc = [torch.full((10, bs, hkv, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    kd, vd = of8.dequantize(of8.quantize(as_np(k), K_SCALE), K_SCALE), of8.dequantize(of8.quantize(as_np(v), V_SCALE), V_SCALE)
    ref, dev = omod.prefill_attention(as_np(q), [0, 150], [0, 150], d ** -0.5, k=kd, v=vd)
    done = 0
    for n in (100, 49):
        meta = md.prefill_metadata([table], [done], [n], bs, always_tables=True)
        gm, rows = md.to_device(meta, "cuda"), slice(done, done + n)
        pkv.kv_store_fp8(k[rows].cuda(), v[rows].cuda(), kc, vc, gm["slot_mapping"], K_SCALE, V_SCALE)
        out = pkv.paged_varlen_prefill_attn_fp8(q[rows].cuda(), kc, vc, gm["block_tables"], gm["cu_seqlens_q"],
                                                gm["cu_seqlens_k"], n, done + n, d ** -0.5, K_SCALE, V_SCALE)
        check(out, ref[rows], dev[rows], torch.float16, 150, f"chunk at {done}")
        done += n
    meta = md.to_device(md.decode_metadata([table], [150], bs), "cuda")
    pkv.kv_store_fp8(k[149:].cuda(), v[149:].cuda(), kc, vc, meta["slot_mapping"], K_SCALE, V_SCALE)
    out = pkv.paged_decode_attn_fp8(q[149:].cuda(), kc, vc, meta["block_tables"], meta["context_lens"], d ** -0.5, K_SCALE,
                                    V_SCALE)
    check(out, ref[149:], dev[149:], torch.float16, 150, "decoded token")
    assert pkv.device_error() == 0
