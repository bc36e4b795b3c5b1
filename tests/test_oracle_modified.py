"""Pins of the modified-score oracle (closed forms), and the host-side refusals of the entry points (CPU)."""

import ctypes
import os

import numpy as np
import pytest

from oracle import attention as oa
from oracle import modified as omod
from pagedattention_kv_cache_gb300 import _lib


def _pool(rng, blocks=12, bs=4, hkv=2, d=8):
    return rng.standard_normal((blocks, bs, hkv, d)), rng.standard_normal((blocks, bs, hkv, d))


def test_no_modifier_is_plain_attention():
    rng = np.random.default_rng(0)
    kc, vc = _pool(rng)
    tables, lens = np.array([[3, 1, 7], [2, 9, -1], [0, -1, -1]]), [11, 5, 0]
    q = rng.standard_normal((3, 4, 8))
    out, _ = omod.decode_attention(q, kc, vc, tables, lens, 0.3)
    assert np.allclose(out, oa.paged_decode_attention(q, kc, vc, tables, lens, 0.3), atol=1e-13)
    cu_q, cu_k = [0, 4, 6], [0, 11, 16]
    qp = rng.standard_normal((6, 4, 8))
    for causal in (True, False):
        out, _ = omod.prefill_attention(qp, cu_q, cu_k, 0.3, k_cache=kc, v_cache=vc, block_tables=tables, causal=causal)
        ref = oa.paged_prefill_attention(qp, cu_q, cu_k, 0.3, k_cache=kc, v_cache=vc, block_tables=tables, causal=causal)
        assert np.allclose(out, ref, atol=1e-13)


def test_cap_and_bias_closed_forms():
    # two keys with scores 6 and 0 and values 1 and 0: the output is the first key's weight
    keys, values = np.array([[6.0], [0.0]]), np.array([[1.0], [0.0]])
    w = lambda s0, s1: np.exp(s0) / (np.exp(s0) + np.exp(s1))  # noqa: E731
    out, dev = omod.head_rows([[1.0]], keys, values, 1.0, [1], [0], [2], softcap=2.0)
    assert np.isclose(out[0, 0], w(2 * np.tanh(3.0), 0.0), atol=1e-15)
    assert np.isclose(dev[0, 0], 2 * out[0, 0] * (1 - out[0, 0]), atol=1e-15)
    # the first key is one position away from the query, the second none
    out, _ = omod.head_rows([[1.0]], keys, values, 1.0, [1], [0], [2], slope=5.0)
    assert np.isclose(out[0, 0], w(6.0 - 5.0, 0.0), atol=1e-15)
    # the bias is added after the cap
    out, _ = omod.head_rows([[1.0]], keys, values, 1.0, [1], [0], [2], softcap=2.0, slope=5.0)
    assert np.isclose(out[0, 0], w(2 * np.tanh(3.0) - 5.0, 0.0), atol=1e-15)
    # a query before the key (a prefix) is as far from it as one behind
    a, _ = omod.head_rows([[0.0]], np.zeros((5, 1)), np.arange(5.0)[:, None], 1.0, [2], [0], [5], slope=0.7)
    assert np.isclose(a[0, 0], 2.0, atol=1e-15)


def test_masks_equal_attention_on_the_visible_part():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((20, 2, 8)), rng.standard_normal((20, 2, 8))
    q = rng.standard_normal((20, 4, 8))
    slopes = [0.5, 0.25, 0.125, 0.0625]
    # documents [0, 7), [7, 8), [8, 20) in one sequence: each as if alone
    first = np.repeat([0, 7, 8], [7, 1, 12])
    out, _ = omod.prefill_attention(q, [0, 20], [0, 20], 0.4, k=k, v=v, first_keys=first, slopes=slopes)
    cuts = [0, 7, 8, 20]
    alone, _ = omod.prefill_attention(q, cuts, cuts, 0.4, k=k, v=v, slopes=slopes)
    assert np.allclose(out, alone, atol=1e-13)
    # a prefix of 6 in a sequence of 20: its rows see all of it, the others are causal
    out, _ = omod.prefill_attention(q, [0, 20], [0, 20], 0.4, k=k, v=v, prefix_lens=[6])
    full, _ = omod.prefill_attention(q[:6], [0, 6], [0, 6], 0.4, k=k, v=v, causal=False)
    causal, _ = omod.prefill_attention(q, [0, 20], [0, 20], 0.4, k=k, v=v)
    assert np.allclose(out[:6], full, atol=1e-13) and np.allclose(out[6:], causal[6:], atol=1e-13)
    # rows that see nothing
    out, dev = omod.prefill_attention(q, [0, 20], [0, 20], 0.4, k=k, v=v, first_keys=np.full(20, 9))
    assert not out[:9].any() and not dev[:9].any() and out[9:].any(axis=(1, 2)).all()
    # a window in decode is a context that starts there
    kc, vc = k.reshape(5, 4, 2, 8), v.reshape(5, 4, 2, 8)
    table = np.arange(5)[None]
    out, _ = omod.decode_attention(q[:1], kc, vc, table, [18], 0.4, first_keys=[13])
    ref, _ = omod.prefill_attention(q[:1], [0, 1], [0, 5], 0.4, k=k[13:18], v=v[13:18])
    assert np.allclose(out, ref, atol=1e-13)
    out, _ = omod.decode_attention(q[:1], kc, vc, table, [18], 0.4, first_keys=[18])
    assert not out.any()


# ---------------------------------------------------------------- refusals, before any CUDA call

P = 4096  # aligned, never dereferenced


def _lib_built():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libpagedkv.so not built (run __graft_entry__.build())")
    return _lib.load()


def _decode(**kw):
    a = dict(out=P, q=P, kc=P, vc=P, bt=P, mb=4, cl=P, batch=2, hq=4, hkv=2, d=128, bs=16, nb=8, scale=0.1, cap=0.0,
             slopes=None, first=None, splits=1, ws=None, wsb=0, dtype=_lib.BF16)
    a.update(kw)
    return _lib_built().pkv_paged_decode_attn_mod(
        a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["cl"], a["batch"], a["hq"], a["hkv"], a["d"], a["bs"],
        a["nb"], ctypes.c_float(a["scale"]), ctypes.c_float(a["cap"]), a["slopes"], a["first"], a["splits"], a["ws"],
        a["wsb"], a["dtype"], None)


@pytest.mark.parametrize("change,status", [
    (dict(cap=-1.0), "EINVAL"), (dict(cap=float("nan")), "EINVAL"), (dict(cap=float("inf")), "EINVAL"),
    (dict(cap=1e-31), "EINVAL"), (dict(cap=1e31), "EINVAL"),
    (dict(out=None), "EINVAL"), (dict(hq=3), "EINVAL"), (dict(splits=-1), "EINVAL"), (dict(bs=0), "EINVAL"),
    (dict(d=96), "EUNSUPPORTED"), (dict(hkv=16, hq=16), "EUNSUPPORTED"), (dict(dtype=7), "EUNSUPPORTED"),
    (dict(q=P + 8), "EALIGN"), (dict(batch=0), "OK")])
def test_decode_mod_refusals(change, status):
    assert _decode(**change) == getattr(_lib, status)


def _prefill_mod(**kw):
    a = dict(out=P, q=P, k=None, v=None, kc=P, vc=P, cq=P, ck=P, mq=8, mk=8, bt=P, mb=4, batch=2, tq=9, tk=0, hq=4,
             hkv=2, d=128, bs=16, nb=8, causal=1, cap=0.0, slopes=None, first=None, prefix=None, ws=None, wsb=0,
             dtype=_lib.BF16, scale=0.1)
    a.update(kw)
    return _lib_built().pkv_paged_varlen_prefill_attn_mod(
        a["out"], a["q"], a["k"], a["v"], a["kc"], a["vc"], a["cq"], a["ck"], a["mq"], a["mk"], a["bt"], a["mb"],
        a["batch"], a["tq"], a["tk"], a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], ctypes.c_float(a["scale"]), a["causal"],
        ctypes.c_float(a["cap"]), a["slopes"], a["first"], a["prefix"], a["ws"], a["wsb"], a["dtype"], None)


@pytest.mark.parametrize("change,status", [
    (dict(cap=-1.0), "EINVAL"), (dict(cap=float("nan")), "EINVAL"), (dict(prefix=P, causal=0), "EINVAL"),
    (dict(scale=0.0), "EINVAL"), (dict(scale=-1.0), "EINVAL"), (dict(scale=float("nan")), "EINVAL"),
    (dict(scale=1e-39), "EINVAL"), (dict(cap=1e31), "EINVAL"),
    (dict(causal=2), "EINVAL"), (dict(bt=None), "EINVAL"), (dict(bt=None, k=P, v=P, tk=0), "EINVAL"),
    (dict(bs=0), "EINVAL"), (dict(nb=0), "EINVAL"), (dict(nb=1 << 30, bs=16), "EINVAL"), (dict(cq=None), "EINVAL"),
    (dict(hq=12, hkv=2), "EUNSUPPORTED"), (dict(d=80), "EUNSUPPORTED"), (dict(dtype=_lib.F32), "EUNSUPPORTED"),
    (dict(kc=P + 4), "EALIGN"), (dict(ws=P + 16, wsb=1 << 20), "EALIGN"), (dict(batch=0), "OK"), (dict(mq=0), "OK")])
def test_prefill_mod_refusals(change, status):
    assert _prefill_mod(**change) == getattr(_lib, status)


def _prefill_fp8(**kw):
    a = dict(out=P, q=P, kc=P, vc=P, cq=P, ck=P, mq=8, mk=8, bt=P, mb=4, batch=2, tq=9, hq=4, hkv=2, d=128, bs=16, nb=8,
             ks=1.0, vs=1.0, causal=1, ws=None, wsb=0, scale=0.1)
    a.update(kw)
    return _lib_built().pkv_paged_varlen_prefill_attn_fp8(
        a["out"], a["q"], a["kc"], a["vc"], a["cq"], a["ck"], a["mq"], a["mk"], a["bt"], a["mb"], a["batch"], a["tq"],
        a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], ctypes.c_float(a["scale"]), ctypes.c_float(a["ks"]),
        ctypes.c_float(a["vs"]), a["causal"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(ks=0.0), "EINVAL"), (dict(vs=float("nan")), "EINVAL"), (dict(ks=float("inf")), "EINVAL"),
    (dict(scale=float("inf")), "EINVAL"), (dict(bt=None), "EINVAL"), (dict(kc=None), "EINVAL"), (dict(causal=-1), "EINVAL"), (dict(mk=-1), "EINVAL"),
    (dict(hq=10, hkv=2), "EUNSUPPORTED"), (dict(d=96), "EUNSUPPORTED"), (dict(q=P + 2), "EALIGN"),
    (dict(tq=0), "OK"), (dict(batch=0), "OK")])
def test_prefill_fp8_refusals(change, status):
    assert _prefill_fp8(**change) == getattr(_lib, status)
