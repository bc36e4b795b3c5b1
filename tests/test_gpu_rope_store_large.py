"""Rotating stores and 4-bit loads of calls large enough for the kernels that take many tokens: the sizes come from the
device's SM count, and each case says that it passes it.  Rotated values, codes and loaded values are exact (as in the
tests of small calls): bit for bit."""

import numpy as np
import pytest
import torch

import pagedattention_kv_cache_gb300 as pkv
from pagedattention_kv_cache_gb300 import metadata as md
from oracle import fp8 as of8
from oracle import q4 as oq

from _harness import as_np
from test_gpu_rope_store import T_K, T_V, _bf16

pytestmark = pytest.mark.gpu


def _past_the_rule(heads, d):
    """A number of tokens that is no multiple of anything and that the kernels for many tokens take."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = (sms * 1024 // (heads * (d // 16)) + 40) | 1
    assert n * heads * (d // 16) > sms * 1024
    return n


class Step:
    """Inputs of one call over n tokens, its cache, and the call."""

    def __init__(self, fmt, n, hq, hkv, d, rot, seed=1):
        self.fmt, self.n, self.hq, self.hkv, self.d = fmt, n, hq, hkv, d
        gen = torch.Generator().manual_seed(seed)
        self.dtype = torch.float32 if fmt == "f32" else torch.bfloat16
        self.q, self.k, self.v = [torch.randn(n, h, d, generator=gen).to(self.dtype).cuda() for h in (hq, hkv, hkv)]
        self.pos = torch.randint(0, 500, (n,), generator=gen, dtype=torch.int32).cuda()
        self.table = torch.from_numpy(md.rope_cos_sin(500, rot)).cuda()
        self.nb, self.bs = n // 8 + 1, 8
        self.slots = torch.randperm(self.nb * self.bs, generator=gen)[:n].int()
        self.slots[::7] = -1
        self.slots = self.slots.cuda()

    def cache(self):
        shape = (self.nb, self.bs, self.hkv, self.d)
        if self.fmt == "q4":
            return [pkv.q4_cache(self.nb, self.bs, self.hkv, self.d) for _ in range(2)]
        return [torch.zeros(shape, dtype=torch.uint8 if self.fmt == "e4m3" else self.dtype, device="cuda") for _ in range(2)]

    def run(self, pools, interleaved=False, q=None, **kw):
        args = (self.q if q is None else q, self.k, self.v, self.pos, self.table, *pools, self.slots)
        if self.fmt in ("f32", "bf16"):
            return pkv.kv_rope_store(*args, interleaved=interleaved, **kw)
        call = pkv.kv_rope_store_q4 if self.fmt == "q4" else pkv.kv_rope_store_fp8
        return call(*args, T_K, T_V, interleaved=interleaved, **kw)

    def check(self, out, pools, interleaved, tokens):
        """The given tokens against the definition."""
        pos, slots = self.pos.cpu().numpy()[tokens], self.slots.cpu().numpy()[tokens]
        table = self.table.cpu().numpy()
        want_q, want_k = [oq.rotate(as_np(x[tokens]), pos, table, interleaved) for x in (self.q, self.k)]
        kept = slots >= 0
        rows = [x.view(self.nb * self.bs, -1)[slots[kept]].cpu() for x in pools]
        if self.fmt == "f32":
            for got, want in ((as_np(out[tokens]), want_q), (rows[0].numpy().reshape(-1, self.hkv, self.d), want_k[kept])):
                # the terms are below 8 in magnitude (normal draws, |c|, |s| <= 1)
                assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -45 * 16).all()
            assert np.array_equal(rows[1].numpy().reshape(-1, self.hkv, self.d), as_np(self.v[tokens])[kept])
            return
        assert np.array_equal(as_np(out[tokens]), _bf16(want_q))
        for got, want, t in ((rows[0], _bf16(want_k)[kept], T_K), (rows[1], as_np(self.v[tokens])[kept], T_V)):
            if self.fmt == "bf16":
                assert np.array_equal(as_np(got).reshape(want.shape), want)
            elif self.fmt == "e4m3":
                assert np.array_equal(got.numpy().reshape(want.shape), of8.quantize(want, t))
            else:
                assert np.array_equal(got.numpy(), np.stack([oq.encode_row(x, t) for x in want]))


SIZES = [(5, 3, 96, 64), (40, 5, 96, 64), (7, 7, 32, 32), (16, 8, 128, 128), (9, 3, 64, 32), (2, 2, 512, 256)]


@pytest.mark.parametrize("hq,hkv,d,rot", SIZES)
@pytest.mark.parametrize("fmt", ["f32", "bf16", "e4m3", "q4"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_large_calls(fmt, hq, hkv, d, rot, interleaved):
    if fmt == "q4" and d not in (64, 128):
        pytest.skip("4-bit rows have heads of 64 or 128")
    n = _past_the_rule(hq + 2 * hkv, d)
    step = Step(fmt, n, hq, hkv, d, rot)
    pools = step.cache()
    out = step.run(pools, interleaved)
    assert pkv.device_error() == 0
    step.check(out, pools, interleaved, np.unique(np.concatenate([np.arange(20), np.arange(n - 10, n), np.arange(0, n, n // 30)])))
    unused = np.setdiff1d(np.arange(step.nb * step.bs), step.slots.cpu().numpy())
    for x in pools:
        assert not x.view(step.nb * step.bs, -1)[unused].any()


@pytest.mark.parametrize("fmt,hq,hkv,d,rot", [("bf16", 16, 8, 128, 128), ("bf16", 40, 5, 96, 64), ("bf16", 4, 2, 64, 64),
                                              ("f32", 16, 8, 128, 64), ("e4m3", 16, 8, 128, 128), ("q4", 8, 2, 64, 64)])
def test_large_calls_in_place_on_a_stream_and_captured(fmt, hq, hkv, d, rot):
    n = _past_the_rule(hq + 2 * hkv, d)
    step = Step(fmt, n, hq, hkv, d, rot)
    want_pools = step.cache()
    want = step.run(want_pools)
    # q turned where it lies
    pools, mine = step.cache(), step.q.clone()
    assert step.run(pools, q=mine, q_out=mine) is mine
    assert torch.equal(mine, want) and all(torch.equal(a, b) for a, b in zip(pools, want_pools))
    # on a stream of its own, while the current one is busy with what the call does not wait for
    pools, side = step.cache(), torch.cuda.Stream()
    mine = step.q.clone()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)
    given = step.run(pools, stream=side)
    again = step.run(pools, q=mine, q_out=mine, stream=side)
    side.synchronize()
    assert torch.equal(given, want) and torch.equal(again, want)
    assert all(torch.equal(a, b) for a, b in zip(pools, want_pools))
    # captured once, replayed on other tokens in the same buffers
    other = Step(fmt, n, hq, hkv, d, rot, seed=2)
    other_pools = other.cache()
    other_want = other.run(other_pools)
    pools, graph = step.cache(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step.run(pools)
    for a, b in ((step.q, other.q), (step.k, other.k), (step.v, other.v), (step.pos, other.pos), (step.slots, other.slots)):
        a.copy_(b)
    graph.replay()
    assert torch.equal(out, other_want) and all(torch.equal(a, b) for a, b in zip(pools, other_pools))
    assert pkv.device_error() == 0


@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 64), (5, 128), (8, 128)])
@pytest.mark.parametrize("t", [1.0, 3.0 / 256, 0.37, 2.0 ** -100, 1e30])
@pytest.mark.parametrize("many", [False, True])
def test_loads_are_exact(hkv, d, t, many):
    """(code - 8) * scale is exact, times T rounded to float32, rounded to bf16."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * 1024 // (2 * hkv * (d // 8)) + 33 if many else 50
    assert (n * 2 * hkv * (d // 8) > sms * 1024) == many
    gen = torch.Generator().manual_seed(n)
    pools = [torch.randint(0, 256, (n // 8 + 1, 8, oq.row_bytes(hkv, d)), generator=gen, dtype=torch.uint8) for _ in range(2)]
    slots = torch.randperm((n // 8 + 1) * 8, generator=gen)[:n].int()
    slots[::9] = -1
    got = pkv.kv_load_q4(*[x.cuda() for x in pools], slots.cuda(), t, t, hkv, d)
    assert pkv.device_error() == 0
    for x, pool in zip(got, pools):
        value = oq.values(pool.view(-1, pool.shape[2])[slots.long()].numpy(), hkv, d, 1.0).astype(np.float32)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(value * np.float32(t)).to(torch.bfloat16)
        want[slots < 0] = 0
        x = x.cpu()
        assert torch.equal(x.isnan(), want.isnan())
        assert torch.equal(x.nan_to_num(0.0, 1.0, -1.0), want.nan_to_num(0.0, 1.0, -1.0))
