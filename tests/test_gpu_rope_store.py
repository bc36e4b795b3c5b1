"""GPU parity of the rotating stores and of the 4-bit store and load.

The rotated element is correct to 2^-46 of its terms before one rounding to float32,
so a float32 result is within 2^-24 of its value plus 2^-45 of the terms, and a bf16
result is the rounding of that float32 (the oracle's float64 rounded the same two
ways), bit for bit.  Stores of quantized caches are bit-exact.
"""

import numpy as np
import pytest
import torch

import pagedattention_kv_cache_gb300 as pkv
from pagedattention_kv_cache_gb300 import _lib
from pagedattention_kv_cache_gb300 import metadata as md
from oracle import attention as oa
from oracle import fp8 as of8
from oracle import q4 as oq

from _harness import as_np

pytestmark = pytest.mark.gpu

T_K, T_V = 1.0 / 64, 3.0 / 256


def _bf16(x64) -> np.ndarray:
    """float64 rounded to float32, then to bf16."""
    return torch.from_numpy(np.asarray(x64).astype(np.float32)).to(torch.bfloat16).float().numpy()


def _inputs(seed, n, hq, hkv, d, dtype, fused=False, max_position=500, rot=None, base=10000.0):
    gen = torch.Generator().manual_seed(seed)
    qkv = torch.randn(n, hq + 2 * hkv, d, generator=gen).to(dtype).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, max_position, (n,), generator=gen, dtype=torch.int32)
    pos[0], pos[-1] = max_position - 1, 0
    table = md.rope_cos_sin(max_position, rot or d, base)
    return gen, q, k, v, pos, table


def _slots(gen, n, num_slots, skip):
    slots = torch.randperm(num_slots, generator=gen)[:n].int()
    slots[::skip] = -1
    return slots


SHAPES = [(7, 16, 8, 128, 128), (1, 1, 1, 64, 64), (33, 8, 1, 64, 32), (50, 6, 3, 128, 96), (300, 4, 4, 32, 32),
          (19, 40, 5, 96, 64), (5, 2, 2, 512, 256)]


@pytest.mark.parametrize("n,hq,hkv,d,rot", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_store_same_type(n, hq, hkv, d, rot, dtype, interleaved):
    gen, q, k, v, pos, table = _inputs(n + d, n, hq, hkv, d, dtype, fused=n % 2 == 1, rot=rot)
    nb, bs = n // 4 + 2, 8
    kc, vc = [torch.randn(nb, bs, hkv, d, generator=gen).to(dtype) for _ in range(2)]
    slots = _slots(gen, n, nb * bs, 5)
    gk, gv = kc.cuda(), vc.cuda()
    out = pkv.kv_rope_store(q, k, v, pos.cuda(), torch.from_numpy(table).cuda(), gk, gv, slots.cuda(),
                            interleaved=interleaved)
    assert pkv.device_error() == 0
    want_q, want_k = [oq.rotate(as_np(x), pos, table, interleaved) for x in (q, k)]
    got_q, got_k = as_np(out), as_np(gk).reshape(-1, hkv, d)
    kept = slots.numpy() >= 0
    rows = slots.numpy()[kept]
    if dtype == torch.bfloat16:
        assert np.array_equal(got_q, _bf16(want_q)) and np.array_equal(got_k[rows], _bf16(want_k[kept]))
    else:
        for got, want in ((got_q, want_q), (got_k[rows], want_k[kept])):
            # the terms are below 8 in magnitude (normal draws, |c|, |s| <= 1)
            assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -45 * 16).all()
    # v and every other slot, bit for bit
    _, wv = oa.kv_store(as_np(kc), as_np(vc), as_np(k), as_np(v), slots.numpy())
    assert np.array_equal(as_np(gv), wv)
    others = np.setdiff1d(np.arange(nb * bs), rows)
    assert np.array_equal(got_k[others], as_np(kc).reshape(-1, hkv, d)[others])


def test_far_positions_and_cancelling_terms():
    # float32's own a c - b s would be off by 2^-24 of the terms where they cancel
    n, d = 64, 64
    gen, q, k, v, _, _ = _inputs(3, n, 2, 2, d, torch.float32)
    pos = torch.arange(131072 - n, 131072, dtype=torch.int32)
    table = md.rope_cos_sin(131072, d, 1e6)
    rows = table[pos.numpy()]
    a = q[:, :, :32]
    q[:, :, 32:] = a * torch.from_numpy(rows[:, None, :32] / np.where(rows[:, None, 32:] == 0, 1, rows[:, None, 32:])).cuda()
    kc = torch.zeros(8, 8, 2, d, device="cuda")
    out = pkv.kv_rope_store(q, k, v, pos.cuda(), torch.from_numpy(table).cuda(), kc, kc.clone(),
                            torch.arange(n, dtype=torch.int32).cuda())
    want = oq.rotate(as_np(q), pos, table, False)
    terms = np.abs(as_np(q)).max()
    assert (np.abs(as_np(out) - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -45 * 2 * terms).all()


@pytest.mark.parametrize("n,hq,hkv,d,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_store_fp8(n, hq, hkv, d, rot, interleaved):
    gen, q, k, v, pos, table = _inputs(n + d, n, hq, hkv, d, torch.bfloat16, fused=n % 2 == 0, rot=rot)
    nb, bs = n // 4 + 2, 8
    kc, vc = [torch.randint(0, 256, (nb, bs, hkv, d), generator=gen, dtype=torch.uint8) for _ in range(2)]
    slots = _slots(gen, n, nb * bs, 4)
    gk, gv = kc.cuda(), vc.cuda()
    out = pkv.kv_rope_store_fp8(q, k, v, pos.cuda(), torch.from_numpy(table).cuda(), gk, gv, slots.cuda(), T_K, T_V,
                                interleaved=interleaved)
    assert pkv.device_error() == 0
    assert np.array_equal(as_np(out), _bf16(oq.rotate(as_np(q), pos, table, interleaved)))
    wk, wv = of8.kv_store_fp8(kc.numpy(), vc.numpy(), _bf16(oq.rotate(as_np(k), pos, table, interleaved)), as_np(v),
                              slots.numpy(), T_K, T_V)
    assert np.array_equal(gk.cpu().numpy(), wk) and np.array_equal(gv.cpu().numpy(), wv)


@pytest.mark.parametrize("t", [1.0, 3.0 / 256, 1e-30, 1e30])
@pytest.mark.parametrize("n", [70, 2500])
def test_fp8_codes_are_those_of_kv_store_fp8(t, n):
    """Every bf16 value of both signs, infinities and NaN, at scales that leave the quotient's range too."""
    hkv, d, hq = 8, 128, 2
    values = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    gen = torch.Generator().manual_seed(n)
    v = values[torch.randint(0, 65536, (n, hkv, d), generator=gen)]
    v.view(-1)[:65536] = values
    v = v.cuda()
    q, k = [torch.randn(n, h, d, generator=gen).to(torch.bfloat16).cuda() for h in (hq, hkv)]
    table = torch.from_numpy(md.rope_cos_sin(10, d, 1e4)).cuda()
    slots = torch.randperm(n, generator=gen).int().cuda()
    pools = [torch.zeros(n, 1, hkv, d, dtype=torch.uint8, device="cuda") for _ in range(4)]
    pkv.kv_rope_store_fp8(q, k, v, slots % 10, table, pools[0], pools[1], slots, t, t)
    pkv.kv_store_fp8(k, v, pools[2], pools[3], slots, t, t)
    assert torch.equal(pools[1], pools[3]) and pkv.device_error() == 0


Q4_SHAPES = [(7, 16, 8, 128, 128), (1, 1, 1, 64, 64), (33, 8, 1, 64, 32), (50, 6, 3, 128, 96), (31, 10, 5, 64, 64),
             (300, 2, 2, 128, 32)]


@pytest.mark.parametrize("n,hq,hkv,d,rot", Q4_SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_store_q4(n, hq, hkv, d, rot, interleaved):
    gen, q, k, v, pos, table = _inputs(n + d, n, hq, hkv, d, torch.bfloat16, fused=n % 2 == 0, rot=rot)
    nb, bs = n // 4 + 2, 8
    kc, vc = [torch.randint(0, 256, (nb, bs, oq.row_bytes(hkv, d)), generator=gen, dtype=torch.uint8) for _ in range(2)]
    slots = _slots(gen, n, nb * bs, 4)
    gk, gv = kc.cuda(), vc.cuda()
    out = pkv.kv_rope_store_q4(q, k, v, pos.cuda(), torch.from_numpy(table).cuda(), gk, gv, slots.cuda(), T_K, T_V,
                               interleaved=interleaved)
    assert pkv.device_error() == 0
    rotated = _bf16(oq.rotate(as_np(k), pos, table, interleaved))
    assert np.array_equal(as_np(out), _bf16(oq.rotate(as_np(q), pos, table, interleaved)))
    assert np.array_equal(gk.cpu().numpy(), oq.store(kc.numpy(), rotated, slots.numpy(), T_K))
    assert np.array_equal(gv.cpu().numpy(), oq.store(vc.numpy(), as_np(v), slots.numpy(), T_V))


MANY = [(1500, 16, 8, 128, 128, 3), (2100, 5, 3, 96, 64, 1), (900, 2, 2, 512, 256, 1), (1111, 40, 5, 64, 32, 2),
        (4100, 8, 1, 64, 64, 1), (1400, 7, 7, 32, 32, 1), (160000, 1, 1, 32, 32, 50)]


@pytest.mark.parametrize("n,hq,hkv,d,rot,every", MANY)
@pytest.mark.parametrize("fmt", ["f32", "bf16", "e4m3", "q4"])
def test_many_tokens_as_few_at_a_time(n, hq, hkv, d, rot, every, fmt):
    """Large calls, which take other kernels, give bit for bit what calls of 100 tokens give."""
    if fmt == "q4" and d not in (64, 128):
        pytest.skip("4-bit rows have heads of 64 or 128")
    dtype = torch.float32 if fmt == "f32" else torch.bfloat16
    gen, q, k, v, pos, table = _inputs(n, n, hq, hkv, d, dtype, fused=n % 2 == 0, rot=rot)
    q[5, 0, 3], k[6, 0, 1], k[7, 0, 0] = float("inf"), float("nan"), 3e38
    nb, bs = n // 8 + 2, 8
    slots = _slots(gen, n, nb * bs, 7)
    slots[n // 2], pos[n // 3] = nb * bs, 500
    row = oq.row_bytes(hkv, d) if fmt == "q4" else hkv * d * {"f32": 4, "bf16": 2, "e4m3": 1}[fmt]
    pools = [torch.randint(0, 120, (nb, bs, row), generator=gen, dtype=torch.uint8).cuda() for _ in range(2)]
    pools += [x.clone() for x in pools]
    table, pos, slots = torch.from_numpy(table).cuda(), pos.cuda(), slots.cuda()

    def call(kc, vc, a, b, interleaved, q_out):
        args = (q[a:b], k[a:b], v[a:b], pos[a:b], table)
        if fmt == "q4":
            pkv.kv_rope_store_q4(*args, kc, vc, slots[a:b], T_K, T_V, interleaved=interleaved, q_out=q_out)
            return
        kc, vc = [x if fmt == "e4m3" else x.view(dtype) for x in (kc, vc)]
        kc, vc = [x.view(nb, bs, hkv, d) for x in (kc, vc)]
        if fmt == "e4m3":
            pkv.kv_rope_store_fp8(*args, kc, vc, slots[a:b], T_K, T_V, interleaved=interleaved, q_out=q_out)
        else:
            pkv.kv_rope_store(*args, kc, vc, slots[a:b], interleaved=interleaved, q_out=q_out)

    pkv.device_error(reset=True)
    for interleaved in (False, True):
        whole, parts = torch.full((n, hq, d), 7.0, dtype=dtype).cuda(), torch.full((n, hq, d), 7.0, dtype=dtype).cuda()
        call(pools[0], pools[1], 0, n, interleaved, whole)
        assert pkv.device_error() == _lib.DERR_SLOT_RANGE | _lib.DERR_POSITION_RANGE
        near = [(a, min(n, a + 100)) for a in range(0, n, 100)][::every]
        for a, b in near:
            call(pools[2], pools[3], a, b, interleaved, parts[a:b])
        torch.cuda.synchronize()
        pkv.device_error(reset=True)
        rows = torch.cat([torch.arange(a, b) for a, b in near]).cuda()
        bits = torch.int32 if fmt == "f32" else torch.int16
        assert torch.equal(whole[rows].view(bits), parts[rows].view(bits))
        to = slots[rows]
        to = to[(to >= 0) & (to < nb * bs)].long()
        for x, y in ((0, 2), (1, 3)):
            assert torch.equal(pools[x].view(-1, row)[to], pools[y].view(-1, row)[to])


@pytest.mark.parametrize("hkv,d,n", [(8, 128, 1500), (1, 64, 12000), (3, 64, 4097)])
def test_many_rows_loaded(hkv, d, n):
    gen = torch.Generator().manual_seed(n)
    kc, vc = [torch.randint(0, 127, (n // 8 + 1, 8, oq.row_bytes(hkv, d)), generator=gen, dtype=torch.uint8).cuda()
              for _ in range(2)]
    slots = _slots(gen, n, (n // 8 + 1) * 8, 9).cuda()
    k, v = pkv.kv_load_q4(kc, vc, slots, T_K, T_V, hkv, d)
    for a in range(0, n, 300):
        part = pkv.kv_load_q4(kc, vc, slots[a:a + 300], T_K, T_V, hkv, d)
        assert torch.equal(k[a:a + 300], part[0]) and torch.equal(v[a:a + 300], part[1])
    assert pkv.device_error() == 0


@pytest.mark.parametrize("hkv,d", [(1, 64), (8, 128), (3, 64), (5, 128)])
@pytest.mark.parametrize("t", [1.0, 3.0 / 256, 0.37, 1e-30, 1e30])
def test_store_and_load_q4(hkv, d, t):
    gen = torch.Generator().manual_seed(hkv)
    n, nb, bs = 41, 9, 5
    k, v = [(torch.randn(n, hkv, d, generator=gen) * 10.0 ** torch.randint(-4, 5, (n, 1, 1), generator=gen)
             * (t if abs(np.log10(t)) > 20 else 1.0)).to(torch.bfloat16) for _ in range(2)]
    k[0, 0, :16] = 0.0
    k[1, 0, 3], k[1, 0, 17], k[2, 0, 5] = float("inf"), float("-inf"), float("nan")
    v[3, 0, 0:16] = 2.0 ** -120
    v[4] = -0.0
    kc, vc = [torch.randint(0, 256, (nb, bs, oq.row_bytes(hkv, d)), generator=gen, dtype=torch.uint8) for _ in range(2)]
    slots = _slots(gen, n, nb * bs, 6)
    gk, gv = kc.cuda(), vc.cuda()
    pkv.kv_store_q4(k.cuda(), v.cuda(), gk, gv, slots.cuda(), t, t)
    assert pkv.device_error() == 0
    wk, wv = oq.store(kc.numpy(), as_np(k), slots.numpy(), t), oq.store(vc.numpy(), as_np(v), slots.numpy(), t)
    assert np.array_equal(gk.cpu().numpy(), wk) and np.array_equal(gv.cpu().numpy(), wv)
    lk, lv = pkv.kv_load_q4(gk, gv, slots.cuda(), t, t, hkv, d)
    assert pkv.device_error() == 0 and lk.shape == k.shape
    for got, pool in ((lk, wk), (lv, wv)):
        with np.errstate(over="ignore"):
            want = _bf16(oq.values(pool.reshape(nb * bs, -1)[slots.numpy()], hkv, d, t))
        want[slots.numpy() < 0] = 0
        # the value times T is rounded to float32 before bf16: an element may fall on bf16's other neighbour only
        # where the exact value lies within 2^-23 of the middle, which the comparison allows as one bf16 step
        got = as_np(got)
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        assert same.mean() > 0.999
        assert (np.abs(got - want)[~same] <= 2.0 ** -7 * np.abs(want)[~same]).all()


def test_padding_tokens_bad_slots_and_bad_positions():
    n, hq, hkv, d, nb, bs = 9, 4, 2, 64, 3, 8
    gen, q, k, v, pos, table = _inputs(1, n, hq, hkv, d, torch.bfloat16, max_position=50)
    slots = torch.arange(n, dtype=torch.int32)
    slots[2], slots[3], slots[4] = -1, nb * bs, -2
    pos[5], pos[6] = 50, -1
    table_gpu = torch.from_numpy(table).cuda()
    kc, vc = [torch.full((nb, bs, oq.row_bytes(hkv, d)), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2)]
    q_out = torch.full_like(q, 7.0)
    pkv.device_error(reset=True)
    pkv.kv_rope_store_q4(q, k, v, pos.cuda(), table_gpu, kc, vc, slots.cuda(), T_K, T_V, q_out=q_out)
    assert pkv.device_error() == _lib.DERR_SLOT_RANGE | _lib.DERR_POSITION_RANGE
    good = [0, 1, 7, 8]
    flat = kc.view(-1, kc.shape[2]).cpu().numpy()
    rotated = _bf16(oq.rotate(as_np(k)[good], pos[good], table, False))
    for i, row in zip(good, rotated):
        assert np.array_equal(flat[i][:72], oq.encode_row(row, T_K)[:72])
    untouched = [i for i in range(nb * bs) if i not in good]
    assert (flat[untouched] == 0x5A).all() and (vc.view(-1, vc.shape[2]).cpu().numpy()[untouched] == 0x5A).all()
    assert (flat[:, 72:] == 0x5A).all()  # a row's unused bytes
    rows = good + [2, 3, 4]  # a padding token's q is rotated, a token of no position is skipped
    assert np.array_equal(as_np(q_out)[rows], _bf16(oq.rotate(as_np(q)[rows], pos[rows], table, False)))
    assert (as_np(q_out)[[5, 6]] == 7.0).all()
    pkv.kv_load_q4(kc, vc, slots.cuda(), T_K, T_V, hkv, d)
    assert pkv.device_error() == _lib.DERR_SLOT_RANGE


def test_in_place_given_stream_and_graph():
    n, hq, hkv, d = 12, 8, 2, 128
    gen, q, k, v, pos, table = _inputs(4, n, hq, hkv, d, torch.bfloat16)
    slots, pos, table = torch.arange(n, dtype=torch.int32).cuda(), pos.cuda(), torch.from_numpy(table).cuda()
    kc, vc = [pkv.q4_cache(2, 8, hkv, d) for _ in range(2)]
    want = pkv.kv_rope_store_q4(q, k, v, pos, table, kc, vc, slots, T_K, T_V)
    wk, wv = kc.clone(), vc.clone()
    side = torch.cuda.Stream()
    kc.zero_()
    vc.zero_()
    side.wait_stream(torch.cuda.current_stream())
    inplace = q.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = pkv.kv_rope_store_q4(inplace, k, v, pos, table, kc, vc, slots, T_K, T_V, q_out=inplace, stream=side)
    lk, lv = pkv.kv_load_q4(kc, vc, slots, T_K, T_V, hkv, d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got is inplace and torch.equal(got, want) and torch.equal(kc, wk) and torch.equal(vc, wv)
    ek, ev = pkv.kv_load_q4(kc, vc, slots, T_K, T_V, hkv, d)
    assert torch.equal(lk, ek) and torch.equal(lv, ev)
    # captured: new inputs in the same buffers
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkv.kv_rope_store_q4(q, k, v, pos, table, kc, vc, slots, T_K, T_V)
    q.copy_(q.flip(0).clone())
    pos.copy_(pos.flip(0).clone())
    kc.zero_()
    graph.replay()
    assert torch.equal(out, want.flip(0))
    want_k = kc.clone()
    kc.zero_()
    pkv.kv_rope_store_q4(q, k, v, pos, table, kc, vc, slots, T_K, T_V)
    assert torch.equal(kc, want_k) and pkv.device_error() == 0


def test_refusals_of_the_binding():
    n, hq, hkv, d = 4, 4, 2, 64
    gen, q, k, v, pos, table = _inputs(5, n, hq, hkv, d, torch.bfloat16)
    pos, table, slots = pos.cuda(), torch.from_numpy(table).cuda(), torch.arange(n, dtype=torch.int32).cuda()
    kc = torch.zeros(2, 8, hkv, d, dtype=torch.bfloat16, device="cuda")
    k4 = pkv.q4_cache(2, 8, hkv, d)

    def same(**kw):
        a = dict(q=q, k=k, v=v, pos=pos, table=table, kc=kc, vc=kc, slots=slots, q_out=None)
        a.update(kw)
        return pkv.kv_rope_store(a["q"], a["k"], a["v"], a["pos"], a["table"], a["kc"], a["vc"], a["slots"],
                                 q_out=a["q_out"])

    for kw in (dict(q=q.cpu()), dict(k=k[:3]), dict(v=v[:, :1]), dict(pos=pos[:3]), dict(slots=slots[:3]),
               dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(k=k[..., ::2]), dict(table=table[:, ::2]),
               dict(kc=kc[:1]), dict(kc=kc[..., :32].contiguous(), vc=kc[..., :32].contiguous()), dict(q_out=q[:2]),
               dict(q=q[:1].expand(n, hq, d))):
        with pytest.raises(ValueError):
            same(**kw)
    for kw in (dict(q=q.half()), dict(k=k.float()), dict(pos=pos.long()), dict(table=table.double()), dict(kc=kc.float()),
               dict(q_out=torch.empty(n, hq, d, device="cuda"))):
        with pytest.raises(TypeError):
            same(**kw)
    with pytest.raises(_lib.PagedKVError):
        same(table=table[:, :48].contiguous())
    with pytest.raises(TypeError):
        pkv.kv_rope_store_q4(q.float(), k.float(), v.float(), pos, table, k4, k4, slots, T_K, T_V)
    with pytest.raises(TypeError):
        pkv.kv_rope_store_fp8(q, k, v, pos, table, kc, kc, slots, T_K, T_V)
    with pytest.raises(ValueError):
        pkv.kv_rope_store_q4(q, k, v, pos, table, k4[..., :64].contiguous(), k4[..., :64].contiguous(), slots, T_K, T_V)
    with pytest.raises(_lib.PagedKVError):
        pkv.kv_store_q4(k, v, k4, k4.clone(), slots, 0.0, 1.0)
    with pytest.raises(ValueError):
        pkv.kv_load_q4(k4, k4, slots, T_K, T_V, hkv, 128)
    with pytest.raises(ValueError):
        pkv.q4_cache(2, 8, 2, 96)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
