"""Attention with modified scores over a paged cache, in float64 numpy.

TEST INFRASTRUCTURE ONLY (see the package docstring).

With s = scale * q . k, query position p, key position t and query head h:
    s = c * tanh(s / c)        when a cap c > 0 is given
    s = s - slope[h] * |p - t| when slopes are given
    out = sum_t softmax(s)_t v_t over the keys the row sees, zeros when it sees none.
A row sees first <= t < nk with t <= p (causal) or t < prefix of its sequence.

Every function also returns, per output element, the weighted mean deviation
    dev = sum_t w_t |v_t - out|,  w the softmax weights:
a relative error of at most d in each weight moves the output by at most about
d * dev, which is what the parity tests' tolerances are built from.
"""

from __future__ import annotations

import numpy as np

from .attention import gather_tokens


def head_rows(q, keys, values, scale, positions, first, last, softcap=0.0, slope=0.0):
    """One head: q [R, D]; keys, values [T, D]; positions, first, last [R] (row sees first <= t < last)."""
    q, keys, values = (np.asarray(x, dtype=np.float64) for x in (q, keys, values))
    t = np.arange(keys.shape[0])[None, :]
    positions, first, last = (np.asarray(x, dtype=np.int64)[:, None] for x in (positions, first, last))
    seen = (t >= first) & (t < last)
    out = np.zeros(q.shape)
    dev = np.zeros(q.shape)
    for r in range(q.shape[0]):
        idx = np.flatnonzero(seen[r])
        if idx.size == 0:
            continue
        s = scale * (keys[idx] @ q[r])
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
        s = s - slope * np.abs(positions[r, 0] - idx)
        w = np.exp(s - s.max())
        w /= w.sum()
        out[r] = w @ values[idx]
        dev[r] = w @ np.abs(values[idx] - out[r])
    return out, dev


def decode_attention(q, k_cache, v_cache, block_tables, context_lens, scale, softcap=0.0, slopes=None, first_keys=None):
    """One query token per sequence, at position context_lens[b] - 1; returns (out, dev), each [B, Hq, D]."""
    B, hq, d = q.shape
    group = hq // k_cache.shape[2]
    out, dev = np.zeros((B, hq, d)), np.zeros((B, hq, d))
    for b in range(B):
        ctx = int(context_lens[b])
        lo = 0 if first_keys is None else max(0, int(first_keys[b]))
        if ctx == 0 or lo >= ctx:
            continue
        keys, values = gather_tokens(k_cache, block_tables[b], ctx), gather_tokens(v_cache, block_tables[b], ctx)
        for h in range(hq):
            o, e = head_rows(q[b, h][None], keys[:, h // group], values[:, h // group], scale, [ctx - 1], [lo], [ctx],
                             softcap, 0.0 if slopes is None else float(slopes[h]))
            out[b, h], dev[b, h] = o[0], e[0]
    return out, dev


def prefill_attention(q, cu_seqlens_q, cu_seqlens_k, scale, *, k_cache=None, v_cache=None, block_tables=None, k=None,
                      v=None, causal=True, softcap=0.0, slopes=None, first_keys=None, prefix_lens=None):
    """Chunk of new tokens per sequence (keys from the cache, or packed k / v); returns (out, dev), [total_q, Hq, D]."""
    total_q, hq, d = q.shape
    out, dev = np.zeros((total_q, hq, d)), np.zeros((total_q, hq, d))
    for i in range(len(cu_seqlens_q) - 1):
        q0, q1 = int(cu_seqlens_q[i]), int(cu_seqlens_q[i + 1])
        k0, k1 = int(cu_seqlens_k[i]), int(cu_seqlens_k[i + 1])
        nq, nk = q1 - q0, k1 - k0
        if nq == 0:
            continue
        if block_tables is not None:
            keys, values = gather_tokens(k_cache, block_tables[i], nk), gather_tokens(v_cache, block_tables[i], nk)
        else:
            keys, values = np.asarray(k[k0:k1], dtype=np.float64), np.asarray(v[k0:k1], dtype=np.float64)
        group = hq // keys.shape[1]
        pos = np.arange(nk - nq, nk)
        last = pos + 1 if causal else np.full(nq, nk)
        if prefix_lens is not None:
            last = np.maximum(last, min(int(prefix_lens[i]), nk))
        first = np.zeros(nq, dtype=np.int64) if first_keys is None else np.maximum(0, np.asarray(first_keys[q0:q1]))
        for h in range(hq):
            out[q0:q1, h], dev[q0:q1, h] = head_rows(q[q0:q1, h], keys[:, h // group], values[:, h // group], scale,
                                                     pos, first, last, softcap, 0.0 if slopes is None else float(slopes[h]))
    return out, dev
