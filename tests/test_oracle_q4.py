"""Pins of the 4-bit codec and the rotation oracle, and the refusals of the calls that use them (CPU)."""

import numpy as np
import pytest

from pagedattention_kv_cache_gb300 import _lib
from pagedattention_kv_cache_gb300 import metadata as md
from oracle import q4 as oq


def test_row_layout_by_hand():
    # one head of 64: 32 code bytes, 4 scale bytes, 12 of padding
    assert oq.row_bytes(1, 64) == 48 and oq.row_bytes(8, 128) == 576 and oq.row_bytes(3, 128) == 224
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :16] = np.arange(-8, 8)  # amax 8: scale e4m3(8 / 7) = 1.125
    x[0, 16] = 7.0                # scale 1, code 15
    row = oq.encode_row(x, 1.0)
    assert row[32] == 0x39 and row[33] == 0x38 and row[34] == 0 and row[35] == 0
    # -8 / 1.125 = -7.1, -7 / 1.125 = -6.2, -6 / 1.125 = -5.3 ...
    assert [int(b) for b in row[:8]] == [1 + 16 * 2, 3 + 16 * 4, 4 + 16 * 5, 6 + 16 * 7, 8 + 16 * 9, 10 + 16 * 11,
                                         12 + 16 * 12, 13 + 16 * 14]
    assert row[8] == 15 + 16 * 8 and set(row[9:32].tolist()) == {0x88}
    v = oq.values(row, 1, 64, 1.0)
    assert v[0, 0] == -7 * 1.125 and v[0, 15] == 6 * 1.125 and v[0, 16] == 7.0 and not v[0, 17:].any()


def test_codes_stop_at_the_ends_and_nan_shows():
    codes, scale = oq.encode_group([np.inf] + [1.0] * 15, 1.0)
    assert scale == 0x7E and codes[0] == 15 and codes[1] == 8  # 448: the largest scale
    codes, scale = oq.encode_group([np.nan] + [1.0] * 15, 1.0)
    assert scale & 0x7F == 0x7F and set(codes.tolist()) == {8}
    # a scale of half its exact size (subnormal): -1.49 of 2^-9 steps of 7 -> scale 2^-9, codes beyond -8 stop there
    codes, scale = oq.encode_group([-1.49 * 7 * 2.0 ** -9, 1.49 * 7 * 2.0 ** -9] + [0.0] * 14, 1.0)
    assert scale == 1 and codes[0] == 0 and codes[1] == 15
    assert oq.encode_group([0.0] * 16, 1.0)[1] == 0


@pytest.mark.parametrize("t", [1.0, 3.0 / 256, 0.37])
def test_round_trip_is_within_half_a_step(t):
    x = np.random.default_rng(0).standard_normal((50, 2, 64)).astype(np.float32)
    for i in range(50):
        row = oq.encode_row(x[i], t)
        v = oq.values(row, 2, 64, t)
        step = np.abs(x[i].reshape(2, 4, 16)).max(-1, keepdims=True) / 7
        # half a step of a scale that is off by at most 2^-4; the largest element may be 7 / (15 / 16) = 7.47 steps,
        # which rounds to 7
        assert (np.abs(v - x[i]).reshape(2, 4, 16) <= 0.5 * step * (1 + 2.0 ** -4) * 1.0001).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, table = rng.standard_normal((4, 2, 64)), md.rope_cos_sin(1000, 32)
    pos = np.array([0, 1, 999, 57])
    y = oq.rotate(x, pos, table, interleaved)
    a, b = (x[..., 0:32:2], x[..., 1:32:2]) if interleaved else (x[..., :16], x[..., 16:32])
    z = (a + 1j * b) * (table[pos, None, :16].astype(np.float64) + 1j * table[pos, None, 16:])
    ya, yb = (y[..., 0:32:2], y[..., 1:32:2]) if interleaved else (y[..., :16], y[..., 16:32])
    assert np.abs(ya - z.real).max() < 1e-14 and np.abs(yb - z.imag).max() < 1e-14
    assert np.array_equal(y[..., 32:], x[..., 32:]) and np.array_equal(y[0], x[0])


def test_rope_table():
    table = md.rope_cos_sin(5, 4, base=100.0)
    assert table.dtype == np.float32 and table.shape == (5, 4)
    assert np.array_equal(table[0], [1, 1, 0, 0])
    want = np.array([np.cos(3), np.cos(0.3), np.sin(3), np.sin(0.3)])
    assert np.abs(table[3] - want).max() <= 2.0 ** -24 * 1.01
    with pytest.raises(ValueError):
        md.rope_cos_sin(5, 3)


# ---------------------------------------------------------------- refusals: before any CUDA call, no pointer is followed

def _lib_or_skip():
    try:
        return _lib.load()
    except _lib.LibraryMissing:
        import pagedattention_kv_cache_gb300.build as build
        build.build()
        return _lib.load()


PTR = 4096


def test_row_bytes_of_the_library():
    lib = _lib_or_skip()
    for hkv in (1, 2, 3, 7, 8, 40):
        for d in (64, 128):
            assert lib.pkv_q4_row_bytes(hkv, d) == oq.row_bytes(hkv, d)
    assert lib.pkv_q4_row_bytes(0, 64) == 0 and lib.pkv_q4_row_bytes(2, 96) == 0


def _rope(**kw):
    a = dict(q_out=PTR, q=PTR * 2, qs=1024, k=PTR, ks=512, v=PTR, vs=512, pos=PTR, cs=PTR, maxp=100, rot=128, inter=0,
             kc=PTR, vc=PTR, slots=PTR, n=3, nb=4, bs=16, hq=8, hkv=4, d=128, fmt=_lib.CACHE_SAME, ksc=1.0, vsc=1.0,
             dt=_lib.BF16)
    a.update(kw)
    return _lib_or_skip().pkv_kv_rope_store(
        a["q_out"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["cs"], a["maxp"], a["rot"],
        a["inter"], a["kc"], a["vc"], a["slots"], a["n"], a["nb"], a["bs"], a["hq"], a["hkv"], a["d"], a["fmt"],
        a["ksc"], a["vsc"], a["dt"], None)


def test_rope_store_refuses_on_the_host():
    assert _rope(n=0) == _lib.OK
    for kw in (dict(q=None), dict(q_out=None), dict(k=None), dict(v=None), dict(pos=None), dict(cs=None),
               dict(kc=None), dict(vc=None), dict(slots=None), dict(n=-1), dict(nb=-1), dict(bs=0), dict(hq=0),
               dict(hkv=0), dict(d=0, rot=0), dict(rot=0), dict(rot=160), dict(maxp=-1), dict(inter=2), dict(qs=1016),
               dict(ks=504), dict(vs=0), dict(fmt=_lib.CACHE_E4M3, ksc=0.0), dict(fmt=_lib.CACHE_Q4, vsc=float("nan")),
               dict(fmt=_lib.CACHE_Q4, ksc=float("inf")), dict(q_out=PTR * 2, qs=2048), dict(nb=1 << 20, bs=1 << 20)):
        assert _rope(**kw) == _lib.EINVAL, kw
    for kw in (dict(dt=7), dict(fmt=3), dict(fmt=_lib.CACHE_E4M3, dt=_lib.F32), dict(fmt=_lib.CACHE_Q4, dt=_lib.F32),
               dict(rot=48), dict(d=144, rot=32, qs=4096, ks=4096, vs=4096), dict(fmt=_lib.CACHE_Q4, d=96, rot=96),
               dict(d=1024, qs=1 << 20, ks=1 << 20, vs=1 << 20)):
        assert _rope(**kw) == _lib.EUNSUPPORTED, kw
    for kw in (dict(q=PTR + 8), dict(q_out=PTR + 2), dict(k=PTR + 4), dict(v=PTR + 8), dict(kc=PTR + 8), dict(vc=PTR + 8),
               dict(cs=PTR + 4), dict(qs=1028), dict(ks=514), dict(vs=516)):
        assert _rope(**kw) == _lib.EALIGN, kw


def test_q4_store_and_load_refuse_on_the_host():
    lib = _lib_or_skip()
    ok = dict(k=PTR, v=PTR, kc=PTR, vc=PTR, s=PTR, n=3, nb=4, bs=16, hkv=2, d=128, ks=1.0, vs=1.0)
    for fn in (lib.pkv_kv_store_q4, lib.pkv_kv_load_q4):
        def call(**kw):
            a = dict(ok, **kw)
            return fn(a["k"], a["v"], a["kc"], a["vc"], a["s"], a["n"], a["nb"], a["bs"], a["hkv"], a["d"], a["ks"],
                      a["vs"], None)
        assert call(n=0) == _lib.OK
        for kw in (dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(s=None), dict(n=-1), dict(nb=-1),
                   dict(bs=0), dict(hkv=0), dict(d=0), dict(ks=0.0), dict(vs=-1.0), dict(ks=float("nan")),
                   dict(nb=1 << 20, bs=1 << 20)):
            assert call(**kw) == _lib.EINVAL, kw
        assert call(d=96) == _lib.EUNSUPPORTED
        for kw in (dict(k=PTR + 8), dict(v=PTR + 8), dict(kc=PTR + 8), dict(vc=PTR + 8)):
            assert call(**kw) == _lib.EALIGN, kw


def test_q4_attention_refuses_on_the_host():
    lib = _lib_or_skip()
    ok = dict(out=PTR, q=PTR, kc=PTR, vc=PTR, bt=PTR, mb=4, cl=PTR, B=2, hq=4, hkv=2, d=128, bs=16, nb=8, scale=0.1,
              ks=1.0, vs=1.0, splits=0)

    def decode(**kw):
        a = dict(ok, **kw)
        return lib.pkv_paged_decode_attn_q4(a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["cl"], a["B"], a["hq"],
                                            a["hkv"], a["d"], a["bs"], a["nb"], a["scale"], a["ks"], a["vs"],
                                            a["splits"], None, 0, None)

    def chunk(**kw):
        a = dict(ok, **kw)
        return lib.pkv_paged_varlen_prefill_attn_q4(a["out"], a["q"], a["kc"], a["vc"], a["cl"], a["cl"], 5, 50, a["bt"],
                                                    a["mb"], a["B"], 7, a["hq"], a["hkv"], a["d"], a["bs"], a["nb"],
                                                    a["scale"], a["ks"], a["vs"], a.get("causal", 1), None, 0, None)

    for call in (decode, chunk):
        assert call(B=0) == _lib.OK
        for kw in (dict(out=None), dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None), dict(cl=None), dict(B=-1),
                   dict(hq=3), dict(hkv=0), dict(bs=0), dict(mb=-1), dict(ks=0.0), dict(vs=float("nan")),
                   dict(ks=float("inf")), dict(mb=1 << 20, bs=1 << 20)):
            assert call(**kw) == _lib.EINVAL, kw
        for kw in (dict(d=96), dict(hq=6), dict(hq=32)):
            assert call(**kw) == _lib.EUNSUPPORTED, kw
        for kw in (dict(out=PTR + 8), dict(q=PTR + 8), dict(kc=PTR + 8), dict(vc=PTR + 8)):
            assert call(**kw) == _lib.EALIGN, kw
        for t in (2.0 ** 65, 2.0 ** -65, -1.0):
            assert call(ks=t) == _lib.EINVAL and call(vs=t) == _lib.EINVAL
    assert decode(splits=-1) == _lib.EINVAL and decode(hkv=16, hq=16) == _lib.EUNSUPPORTED
    assert chunk(causal=2) == _lib.EINVAL and chunk(scale=0.0) == _lib.EINVAL and chunk(scale=float("nan")) == _lib.EINVAL
