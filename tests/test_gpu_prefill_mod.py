"""GPU parity of paged_varlen_prefill_attn_mod (softcap, distance bias, document / window / prefix masks)
against the float64 oracle."""

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


class Case:
    """A chunk batch (cached and new tokens per sequence) with its tensors on the host."""

    def __init__(self, seed, cached, new, *, block_size=16, hq=8, hkv=2, d=128, q_scale=3.0, paged=True):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.cached, self.new, self.bs, self.d, self.hq, self.hkv, self.paged = cached, new, block_size, d, hq, hkv, paged
        totals = [c + n for c, n in zip(cached, new)]
        self.totals, self.total_q = totals, sum(new)
        self.q = (torch.randn(self.total_q, hq, d, generator=gen) * q_scale).bfloat16()
        self.cu_q, self.cu_k = i32([0] + np.cumsum(new).tolist()), i32([0] + np.cumsum(totals).tolist())
        self.scale = d ** -0.5
        if paged:
            blocks = sum(-(-n // block_size) for n in totals) + 5
            self.tables = wl._assign_blocks(rng, totals, block_size, blocks)
            self.table = i32(md.table_matrix(self.tables))
            self.kc, self.vc = [torch.randn(blocks, block_size, hkv, d, generator=gen).bfloat16() for _ in range(2)]
        else:
            self.k, self.v = [torch.randn(sum(totals), hkv, d, generator=gen).bfloat16() for _ in range(2)]

    def positions(self):
        return np.concatenate([np.arange(t - n, t) for t, n in zip(self.totals, self.new)] or [np.zeros(0)]).astype(np.int64)

    def keys(self):
        if self.paged:
            return dict(k_cache=self.kc, v_cache=self.vc, block_tables=self.table)
        return dict(k=self.k, v=self.v)

    def reference(self, causal, cap, slopes, first, prefix):
        keys = {n: (as_np(x) if x.dtype != torch.int32 else x.numpy()) for n, x in self.keys().items()}
        return omod.prefill_attention(as_np(self.q), self.cu_q.tolist(), self.cu_k.tolist(), self.scale, causal=causal,
                                      softcap=cap, slopes=slopes, first_keys=first, prefix_lens=prefix, **keys)

    def hide_unseen(self, first):
        """NaN past every sequence's keys and before the least first key of its rows; those blocks' ids invalid."""
        seen = torch.zeros(self.kc.shape[:2], dtype=torch.bool)
        row = 0
        for i, (blocks, total, n) in enumerate(zip(self.tables, self.totals, self.new)):
            lo = 0 if first is None or n == 0 else max(0, int(first[row:row + n].min()))
            for t in range(min(lo, total), total):
                seen[blocks[t // self.bs], t % self.bs] = True
            self.table[i, : min(lo, total) // self.bs] = 1 << 30
            row += n
        self.kc[~seen], self.vc[~seen] = float("nan"), float("nan")

    def call(self, causal=True, cap=0.0, slopes=None, first=None, prefix=None, **kw):
        return pkv.paged_varlen_prefill_attn_mod(
            self.q.cuda(), self.cu_q.cuda(), self.cu_k.cuda(), max(self.new), max(self.totals), self.scale, causal=causal,
            softcap=cap, alibi_slopes=cuda(slopes), first_keys=cuda(first), prefix_lens=cuda(prefix),
            **{n: x.cuda() for n, x in self.keys().items()}, **kw)

    def compare(self, causal=True, cap=0.0, alibi=False, first=None, prefix=None, hide=False, label="", **kw):
        slopes = slopes_of(self.hq) if alibi else None
        first = None if first is None else i32(np.asarray(first).tolist())
        prefix = None if prefix is None else i32(prefix)
        ref, dev = self.reference(causal, cap, slopes, first, prefix)
        if hide and self.paged:
            self.hide_unseen(first)
        out = self.call(causal, cap, slopes, first, prefix, **kw)
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        check(out, ref, dev, torch.bfloat16, max(self.totals), label)
        return out


CACHED, NEW = [0, 16, 0, 130, 300, 5], [1, 40, 129, 0, 260, 3]


def _call_args(case, kw):
    """Arguments of Case.compare as those of Case.call."""
    kw = dict(kw)
    if kw.pop("alibi", False):
        kw["slopes"] = slopes_of(case.hq)
    return {n: i32(np.asarray(x).tolist()) if n in ("first", "prefix") else x for n, x in kw.items()}


def _documents(case, seed, least=1):
    """First key of each row from random document starts of each sequence."""
    rng, out = np.random.default_rng(seed), []
    for total, n in zip(case.totals, case.new):
        cuts = np.concatenate([[0], np.sort(rng.integers(0, max(total, 1), size=max(least, total // 60)))])
        pos = np.arange(total - n, total)
        out.append(cuts[np.searchsorted(cuts, pos, side="right") - 1])
    return np.concatenate(out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,hkv", [(1, 3), (2, 2), (4, 1), (8, 1)])
@pytest.mark.parametrize("mods", ["cap", "alibi", "documents", "window", "prefix", "all"])
def test_every_group_and_modifier(d, group, hkv, mods):
    c = Case(group * 10 + d, CACHED, NEW, hq=group * hkv, hkv=hkv, d=d)
    kw = {"cap": dict(cap=50.0), "alibi": dict(alibi=True), "documents": dict(first=_documents(c, group)),
          "window": dict(first=c.positions() - 99), "prefix": dict(prefix=[0, 30, 200, 7, 301, -4]),
          "all": dict(cap=20.0, alibi=True, first=_documents(c, group + 1), prefix=[9, 56, 64, 7, 400, 0])}[mods]
    c.compare(hide=True, label=mods, **kw)


@pytest.mark.parametrize("block_size", [1, 4, 5, 8, 24, 64, 100, 128, 256, 384])
def test_block_sizes(block_size):
    c = Case(block_size, CACHED, NEW, block_size=block_size, d=64 if block_size % 5 == 0 else 128)
    c.compare(cap=30.0, alibi=True, first=_documents(c, 3), hide=True)


@pytest.mark.parametrize("d,group", [(64, 2), (128, 1), (128, 8)])
def test_packed_keys_and_full_attention(d, group):
    c = Case(70 + d, [0] * 4, [1, 300, 128, 77], hq=2 * group, hkv=2, d=d, paged=False)
    c.compare(cap=40.0, alibi=True, first=_documents(c, 5), label="packed")
    c.compare(causal=False, cap=40.0, alibi=True, label="packed, full")
    c.compare(causal=False, first=c.positions() - 50, label="packed, full, first keys")
    c = Case(80 + d, CACHED, NEW, hq=2 * group, hkv=2, d=d)
    c.compare(causal=False, cap=40.0, alibi=True, first=np.minimum(_documents(c, 6), 60), hide=True, label="paged, full")


@pytest.mark.parametrize("block_size", [16, 24, 256])
@pytest.mark.parametrize("group,hkv,new", [(1, 8, [4, 1, 8, 3, 0, 2]), (2, 3, [4, 1, 2, 3, 0, 4]), (4, 2, [2, 1, 2, 0, 1, 2]),
                                           (8, 1, [1, 1, 1, 0, 1, 1])])
@pytest.mark.parametrize("mods", ["cap", "alibi", "documents", "window", "prefix", "all", "nothing", "full"])
def test_short_chunks_on_the_decode_kernel(block_size, group, hkv, new, mods):
    c = Case(90 + group, [1000, 17, 0, 255, 511, 2000], new, hq=group * hkv, hkv=hkv, block_size=block_size)
    assert pkv.chunk_workspace_bytes(6, c.hq, hkv, 128, max(new), 2004) > 0
    kw = {"cap": dict(cap=50.0), "alibi": dict(alibi=True), "documents": dict(first=_documents(c, group)),
          "window": dict(first=c.positions() - 99), "prefix": dict(prefix=[0, 18, 200, 257, 301, -4], alibi=True),
          "all": dict(cap=20.0, alibi=True, first=_documents(c, group + 1), prefix=[1003, 56, 64, 7, 400, 0]),
          "nothing": dict(cap=50.0, first=c.positions() + np.arange(sum(new)) % 3 - 1),
          "full": dict(causal=False, alibi=True, cap=30.0, first=c.positions() - 40)}[mods]
    c.compare(label=mods, **kw)
    ws = pkv.chunk_workspace(6, c.hq, hkv, 128, max(new), 2004)
    a = c.compare(workspace=ws, hide=True, **kw)
    assert torch.equal(a, c.call(workspace=ws, **_call_args(c, kw)))
    assert int(ws[:65536].count_nonzero()) == 0


def test_short_chunks_of_more_sequences_than_threads():
    rng = np.random.default_rng(4)
    cached, new = rng.integers(0, 40, size=400).tolist(), rng.integers(0, 5, size=400).tolist()
    cached[7], cached[390] = 3000, 1500
    c = Case(43, cached, new, hq=4, hkv=2)
    c.compare(cap=20.0, alibi=True, first=c.positions() - 9, prefix=rng.integers(0, 50, size=400).tolist())


def test_more_than_eight_kv_heads():
    Case(44, [100, 0, 700], [40, 130, 2], hq=12, hkv=12).compare(cap=20.0, alibi=True)
    c = Case(45, [2000, 3], [2, 1], hq=48, hkv=12)
    c.compare(first=c.positions() - 700)


@pytest.mark.parametrize("mods", ["masked", "cap", "alibi", "both"])
@pytest.mark.parametrize("new", [70, 4])
def test_nan_reaches_only_the_rows_that_see_it(mods, new):
    c = Case(46, [1500], [new], hq=2, hkv=1)
    slopes = slopes_of(2) if mods in ("alibi", "both") else None
    cap = 20.0 if mods in ("cap", "both") else 0.0
    ref, dev = c.reference(True, cap, slopes, None, None)
    pos = 1500 + new - 3  # a NaN key that the last three rows see
    c.kc[c.tables[0][pos // 16], pos % 16, 0, 5] = float("nan")
    c.q[1, 0, 9] = float("nan")
    out = c.call(True, cap, slopes)
    torch.cuda.synchronize()
    bad = torch.isnan(out).all(-1)
    want = torch.zeros(new, 2, dtype=torch.bool)
    want[new - 3:], want[1, 0] = True, True
    assert torch.equal(bad.cpu(), want)
    keep = ~want.numpy()
    check(out[~bad], ref[keep], dev[keep], torch.bfloat16, 1600)


def test_short_chunk_of_sequences_without_a_key():
    c = Case(99, [2000, 30, 0], [2, 3, 1], hq=4, hkv=2)
    first = np.array([1 << 30, 1 << 30, 0, 5, 1 << 30, 1 << 30])
    out = c.compare(first=first)
    assert not out[:2].any() and not out[4:].any() and out[2:4].any()


def test_rows_that_see_nothing():
    c = Case(31, [0, 100], [200, 150])
    first = c.positions() + np.arange(350) % 3 - 1  # one key before, the own key, one past it
    c.compare(cap=50.0, first=first)
    first[:] = 1 << 30
    out = c.compare(first=first)
    assert torch.count_nonzero(out) == 0
    first = np.where(np.arange(350) < 200, 1 << 30, 0)  # a whole sequence without a key
    c.compare(first=first, alibi=True)
    first = np.full(350, -(1 << 31))
    first[::7] = 2**31 - 1
    c.compare(first=first)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mods", ["masked", "cap", "alibi", "both"])
def test_results_do_not_depend_on_what_shared_memory_held(d, mods):
    # narrow windows leave most of a tile's keys unread: whatever an earlier kernel left in their place, the result is
    # the same bit for bit.  (The fill: a prefill on every SM over keys of one value.)
    c = Case(50, [0, 1, 300, 2000], [433, 70, 45, 839], block_size=8, d=d)
    kw = {"masked": {}, "cap": dict(cap=30.0), "alibi": dict(alibi=True), "both": dict(cap=30.0, alibi=True)}[mods]
    args = _call_args(c, dict(kw, first=c.positions() - 2))
    n = 128 * 64
    cu = i32([0, n]).cuda()
    outs = []
    for value in (0.0, 1.0, -300.0, 3e38, float("nan"), float("inf")):
        k = torch.full((n, 8, d), value, dtype=torch.bfloat16, device="cuda")
        pkv.paged_varlen_prefill_attn(torch.ones_like(k), cu, cu, n, n, 0.1, k=k, v=k, workspace=False)
        outs.append(c.call(workspace=False, **args))
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    assert torch.isfinite(outs[0]).all() and all(torch.equal(outs[0], o) for o in outs[1:])
    c.compare(workspace=False, **kw, first=c.positions() - 2)


def test_first_keys_in_any_order():
    c = Case(32, [500, 0], [260, 300])
    rng = np.random.default_rng(0)
    c.compare(first=rng.integers(-10, 700, size=560), cap=10.0, alibi=True)


def test_prefix_longer_than_the_sequence_is_full_attention():
    c = Case(33, [0, 64], [190, 33])
    big = c.compare(prefix=[10**9, 10**9], alibi=True)
    full = c.compare(causal=False, alibi=True)
    assert torch.equal(big, full)


def test_no_modifier_matches_the_plain_call():
    c = Case(34, CACHED, NEW)
    out = c.compare()
    plain = pkv.paged_varlen_prefill_attn(c.q.cuda(), c.cu_q.cuda(), c.cu_k.cuda(), max(c.new), max(c.totals), c.scale,
                                          k_cache=c.kc.cuda(), v_cache=c.vc.cuda(), block_tables=c.table.cuda())
    assert torch.equal(out, plain)


@pytest.mark.parametrize("q_scale,cap", [(40.0, 5.0), (8.0, 20.0)])
def test_scores_around_and_far_beyond_the_cap(q_scale, cap):
    Case(35, [100, 0], [140, 60], q_scale=q_scale).compare(cap=cap)


@pytest.mark.parametrize("cap", [1e-30, 1e-3, 1.0, 300.0, 1e4, 1e6, 1e30])
def test_caps_of_every_size(cap):
    c = Case(41, [100, 0], [140, 60])
    c.compare(cap=cap)
    c.compare(cap=cap, alibi=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_scale", [1e36, 1e-36])
def test_distance_bias_at_scales_of_every_size(d, q_scale):
    # q times a power of ten and the scale divided by it: the scores, and what the bias adds to them, stay.  Rows see
    # keys some way ahead of them only, so every score they have is biased by 100 or more at the steepest slope
    c = Case(48, [0, 100, 2], [300, 270, 9], d=d, q_scale=q_scale)
    c.scale = d ** -0.5 * 3.0 / q_scale
    c.compare(causal=False, alibi=True, label="every key")
    c.compare(causal=False, alibi=True, first=c.positions() + 260, label="keys from 260 on")
    c.compare(causal=False, alibi=True, cap=20.0, first=c.positions() + 260, label="capped")


def test_scores_that_overflow_are_capped():
    # every product of a key has that key's sign and is beyond float32: the score is +-infinity, the capped score +-5
    c = Case(35, [100, 0], [140, 60], q_scale=1e30)
    c.q = c.q.abs().clamp_min(1e30)
    c.kc = c.kc.abs().clamp_min(1.0) * torch.sign(c.kc[..., :1].float()).bfloat16() * 1e9
    c.compare(cap=5.0)


@pytest.mark.parametrize("mods", ["cap", "alibi", "window", "all"])
def test_split_key_ranges(mods):
    # one sequence with a long history: its tiles run as several parts that are merged
    c = Case(36, [6000, 3000], [70, 33], block_size=64, hq=4, hkv=2)
    assert pkv.prefill_workspace_bytes(2, 4, 2, 128, 70) > 0
    kw = {"cap": dict(cap=50.0), "alibi": dict(alibi=True), "window": dict(first=c.positions() - 2500),
          "all": dict(cap=30.0, alibi=True, first=c.positions() - 4000, prefix=[6050, 10])}[mods]
    a = c.compare(label="split", **kw)
    c.compare(workspace=False, label="not split", **kw)
    ws = pkv.prefill_workspace(2, 4, 2, 128, 70)
    for _ in range(3):  # the counters are left at zero: the same workspace serves the next call, bit for bit
        assert torch.equal(a, c.compare(workspace=ws, **kw))
    assert int(ws[:65536].count_nonzero()) == 0
    assert torch.equal(a, c.compare(hide=True, **kw))


def test_rows_behind_the_last_sequence_are_left_alone():
    c = Case(37, [0, 20], [30, 9])
    out = torch.full((50, c.hq, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    first = i32([0] * 50)
    q = torch.cat([c.q, torch.zeros(11, c.hq, c.d, dtype=torch.bfloat16)])
    pkv.paged_varlen_prefill_attn_mod(q.cuda(), c.cu_q.cuda(), c.cu_k.cuda(), 30, 30, c.scale, softcap=9.0,
                                      first_keys=first.cuda(), out=out, **{n: x.cuda() for n, x in c.keys().items()})
    torch.cuda.synchronize()
    assert torch.all(out[39:] == 7.0)
    ref, dev = c.reference(True, 9.0, None, None, None)
    check(out[:39], ref, dev, torch.bfloat16, 30)


def test_bad_cu_seqlens_and_pages_raise_bits():
    c = Case(38, [0, 16, 16], [20, 20, 20])
    kw = {n: x.cuda() for n, x in c.keys().items()}
    ref, dev = c.reference(True, 20.0, None, None, None)

    def call(cu_q, cu_k, max_q, **more):
        pkv.device_error(reset=True)
        out = torch.full_like(c.q, 7.0).cuda()
        pkv.paged_varlen_prefill_attn_mod(c.q.cuda(), i32(cu_q).cuda(), i32(cu_k).cuda(), max_q, 64, c.scale, softcap=20.0,
                                          out=out, **dict(kw, **more))
        return pkv.device_error(), out

    for cu_q, cu_k, max_q in (([0, 20, 40, 61], [0, 20, 56, 92], 21), ([0, 20, 10, 60], [0, 20, 56, 92], 20),
                              ([-1, 20, 40, 60], [0, 20, 56, 92], 21), ([0, 20, 40, 60], [0, 20, 56, 92], 19),
                              ([0, 20, 40, 60], [0, 19, 56, 92], 20), ([0, 20, 40, 60], [0, 20, 56, 200], 20)):
        bits, _ = call(cu_q, cu_k, max_q)
        assert bits == _lib.DERR_LEN_RANGE, (cu_q, cu_k, max_q)
    bad = c.table.clone()
    bad[1, 0], bad[1, 2] = -1, c.kc.shape[0]
    bits, out = call([0, 20, 40, 60], [0, 20, 56, 92], 20, block_tables=bad.cuda())
    assert bits == _lib.DERR_BLOCK_RANGE
    check(out[:20], ref[:20], dev[:20], torch.bfloat16, 36)
    check(out[40:], ref[40:], dev[40:], torch.bfloat16, 36)


def test_pool_past_32_bit_offsets():
    bs, hkv, d, hq = 256, 8, 128, 16
    blocks = (1 << 31) // (bs * hkv * d) + 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = [torch.zeros(blocks, bs, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ids = [blocks - 1, 3, blocks - 17]
    for c in (kc, vc):
        c[ids] = torch.randn(3, bs, hkv, d, generator=gen, device="cuda").bfloat16()
    q = torch.randn(40, hq, d, generator=gen, device="cuda").bfloat16()
    cu_q, cu_k = i32([0, 40]), i32([0, 600])
    out = pkv.paged_varlen_prefill_attn_mod(q, cu_q.cuda(), cu_k.cuda(), 40, 600, 0.1, k_cache=kc, v_cache=vc,
                                            block_tables=i32([ids]).cuda(), softcap=20.0)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    ref, dev = omod.prefill_attention(as_np(q), [0, 40], [0, 600], 0.1, k_cache=as_np(kc[ids]), v_cache=as_np(vc[ids]),
                                      block_tables=np.arange(3)[None], softcap=20.0)
    check(out, ref, dev, torch.bfloat16, 600)


def test_binding_refusals():
    c = Case(39, [0, 16], [8, 8])
    q, cu_q, cu_k = c.q.cuda(), c.cu_q.cuda(), c.cu_k.cuda()
    kw = {n: x.cuda() for n, x in c.keys().items()}
    call = lambda **more: pkv.paged_varlen_prefill_attn_mod(q, cu_q, cu_k, 8, 24, 0.1, **dict(kw, **more))  # noqa: E731
    with pytest.raises(ValueError, match="first_keys must have shape"):
        call(first_keys=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="prefix_lens must have shape"):
        call(prefix_lens=torch.zeros(16, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="alibi_slopes must have shape"):
        call(alibi_slopes=torch.zeros(2, device="cuda"))
    with pytest.raises(_lib.PagedKVError):
        call(prefix_lens=torch.zeros(2, dtype=torch.int32, device="cuda"), causal=False)
    with pytest.raises(_lib.PagedKVError):
        call(softcap=float("nan"))
    with pytest.raises(ValueError, match="packed k and v"):
        call(block_tables=None)
    with pytest.raises(ValueError, match="head_dim differs"):
        call(k_cache=kw["k_cache"][..., :64].contiguous(), v_cache=kw["v_cache"][..., :64].contiguous())
    with pytest.raises(_lib.PagedKVError):  # workspace not 256-byte aligned
        call(workspace=torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")[16:])
    assert pkv.device_error() == 0


def test_captured_and_on_another_stream():
    c = Case(40, [900, 40], [60, 30], block_size=64, hq=4, hkv=2)
    q, cu_q, cu_k = c.q.cuda(), c.cu_q.cuda(), c.cu_k.cuda()
    kw = {n: x.cuda() for n, x in c.keys().items()}
    slopes, first = slopes_of(4).cuda(), i32([0] * 90).cuda()
    out = torch.empty_like(q)
    ws = pkv.prefill_workspace(2, 4, 2, 128, 60)

    def step(**more):
        return pkv.paged_varlen_prefill_attn_mod(q, cu_q, cu_k, 60, 960, c.scale, softcap=30.0, alibi_slopes=slopes,
                                                 first_keys=first, **{**kw, "workspace": ws, "out": out, **more})

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for window in (2000, 300, 1):
        first.copy_(i32((c.positions() - window + 1).tolist()))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        other = step(stream=side, workspace=None, out=None)
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        assert torch.equal(out, other)
        ref, dev = c.reference(True, 30.0, slopes.cpu(), c.positions() - window + 1, None)
        check(out, ref, dev, torch.bfloat16, 960, f"window {window}")


def test_store_then_chunks_then_decode():
    # a capped, windowed, distance-biased model served step by step: two chunks of a prompt and two decoded
    # tokens over one cache, each against the oracle
    bs, hq, hkv, d, cap, window = 16, 8, 2, 128, 25.0, 70
    gen = torch.Generator().manual_seed(50)
    k, v = [torch.randn(150, hkv, d, generator=gen).bfloat16() for _ in range(2)]
    q = (torch.randn(150, hq, d, generator=gen) * 3).bfloat16()
    slopes = slopes_of(hq)
    table = [7, 2, 9, 0, 4, 8, 1, 3, 6, 5]
    kc, vc = [torch.full((10, bs, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    first = np.maximum(0, np.arange(150) + 1 - window)
    ref, dev = omod.prefill_attention(as_np(q), [0, 150], [0, 150], d ** -0.5, k=as_np(k), v=as_np(v), softcap=cap,
                                      slopes=slopes, first_keys=first)
    done = 0
    for n in (100, 48):
        meta = md.prefill_metadata([table], [done], [n], bs, always_tables=True)
        gm = md.to_device(meta, "cuda")
        rows = slice(done, done + n)
        pkv.kv_store(k[rows].cuda(), v[rows].cuda(), kc, vc, gm["slot_mapping"])
        out = pkv.paged_varlen_prefill_attn_mod(
            q[rows].cuda(), gm["cu_seqlens_q"], gm["cu_seqlens_k"], n, done + n, d ** -0.5, k_cache=kc, v_cache=vc,
            block_tables=gm["block_tables"], softcap=cap, alibi_slopes=slopes.cuda(), first_keys=i32(first[rows].tolist()).cuda())
        check(out, ref[rows], dev[rows], torch.bfloat16, 150, f"chunk at {done}")
        done += n
    for t in (148, 149):
        meta = md.to_device(md.decode_metadata([table], [t + 1], bs), "cuda")
        pkv.kv_store(k[t:t + 1].cuda(), v[t:t + 1].cuda(), kc, vc, meta["slot_mapping"])
        out = pkv.paged_decode_attn_mod(q[t:t + 1].cuda(), kc, vc, meta["block_tables"], meta["context_lens"], d ** -0.5,
                                        softcap=cap, alibi_slopes=slopes.cuda(), first_keys=i32([int(first[t])]).cuda())
        check(out, ref[t:t + 1], dev[t:t + 1], torch.bfloat16, 150, f"token {t}")
    assert pkv.device_error() == 0
