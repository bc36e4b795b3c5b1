"""Python binding of the C ABI: argument marshalling only.

Each function takes torch tensors that already live on the current CUDA
device, checks device, dtype, shape and contiguity (a mismatch that would let
a kernel read or write out of bounds is a host-side error, raised before any
launch), and passes raw pointers and sizes to libpagedkv.so on the current
torch stream.  Every step of the path runs
in the library's CUDA kernels; nothing here computes.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}


def _dtype_code(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32 or bfloat16") from None


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype=None, ndim=None, device=None, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.get_device() != device.index:
        raise ValueError(f"{name} is on {t.device}, the other arguments on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _device(t: torch.Tensor, name: str) -> torch.device:
    """The device every argument of a call must be on: the current CUDA device, where the
    library launches its kernels."""
    _need(t, name)
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device} but the current CUDA device is cuda:{cur}")
    return t.device


# the current stream's handle without building a Stream object (2 us of a call's host time)
_current_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream",
                                 lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream, device: torch.device) -> int:
    if stream is None:
        return _current_stream_handle(device.index)
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    return stream.cuda_stream


def kv_store(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
             slot_mapping: torch.Tensor, stream=None) -> None:
    """Write k/v rows [N, Hkv, D] into k_cache/v_cache [blocks, bs, Hkv, D] at slot_mapping (-1 skips)."""
    dev = _device(k, "k")
    for name, t in (("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t, name, dtype=k.dtype, device=dev)
    _need(slot_mapping, "slot_mapping", dtype=torch.int32, ndim=1, device=dev)
    if k.dim() != 3 or v.shape != k.shape or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("expected k, v [N, Hkv, D] and caches [blocks, bs, Hkv, D]")
    if k_cache.shape[2:] != k.shape[1:] or slot_mapping.shape[0] != k.shape[0]:
        raise ValueError("k/v rows and the cache disagree on (Hkv, D), or slot_mapping length differs")
    nb, bs, hkv, d = k_cache.shape
    st = _lib.load().pkv_kv_store(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                                  k.shape[0], nb, bs, hkv, d, _dtype_code(k), _stream(stream, dev))
    _lib.check("pkv_kv_store", st)


def copy_blocks(k_caches: list[torch.Tensor], v_caches: list[torch.Tensor], block_pairs: torch.Tensor,
                stream=None) -> None:
    """Copy-on-write block copies: for each (src, dst) row of block_pairs (int32 [n, 2]),
    block dst of every layer's K and V pool becomes a copy of block src."""
    if len(k_caches) != len(v_caches) or not k_caches:
        raise ValueError("need one K and one V pool per layer")
    shape = k_caches[0].shape
    dev = _device(k_caches[0], "k_caches[0]")
    for t in list(k_caches) + list(v_caches):
        _need(t, "cache", device=dev)
        if t.shape != shape or t.dtype != k_caches[0].dtype:
            raise ValueError("every pool must have the same shape and dtype")
    _need(block_pairs, "block_pairs", dtype=torch.int32, ndim=2, device=dev)
    if block_pairs.shape[1] != 2:
        raise ValueError("block_pairs must be [n, 2]")
    L = len(k_caches)
    kp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k_caches])
    vp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v_caches])
    block_bytes = k_caches[0][0].numel() * k_caches[0].element_size()
    st = _lib.load().pkv_copy_blocks(kp, vp, L, _ptr(block_pairs), block_pairs.shape[0], shape[0], block_bytes,
                                     _stream(stream, dev))
    _lib.check("pkv_copy_blocks", st)


def kv_store_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 slot_mapping: torch.Tensor, k_scale: float, v_scale: float, stream=None) -> None:
    """Quantizing store: bf16 rows [N, Hkv, D] into E4M3 caches [blocks, bs, Hkv, D] (uint8 or
    float8_e4m3fn tensors) as e4m3(x / scale); slot -1 skips."""
    dev = _device(k, "k")
    _need(k, "k", dtype=torch.bfloat16, ndim=3)
    _need(v, "v", dtype=torch.bfloat16, ndim=3, device=dev)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t, name, ndim=4, device=dev)
        if t.element_size() != 1:
            raise TypeError(f"{name} must be a one-byte (E4M3) tensor")
    _need(slot_mapping, "slot_mapping", dtype=torch.int32, ndim=1, device=dev)
    if v.shape != k.shape or v_cache.shape != k_cache.shape or k_cache.shape[2:] != k.shape[1:]:
        raise ValueError("expected k, v [N, Hkv, D] and caches [blocks, bs, Hkv, D]")
    if slot_mapping.shape[0] != k.shape[0]:
        raise ValueError("slot_mapping length differs from the number of rows")
    nb, bs, hkv, d = k_cache.shape
    st = _lib.load().pkv_kv_store_fp8(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                                      k.shape[0], nb, bs, hkv, d, ctypes.c_float(k_scale),
                                      ctypes.c_float(v_scale), _stream(stream, dev))
    _lib.check("pkv_kv_store_fp8", st)


def paged_decode_attn_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                          k_scale: float, v_scale: float, *, num_splits: int = 0,
                          workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """Decode attention over an E4M3 cache with per-tensor scales; q / out bf16 [B, Hq, D]."""
    dev = _device(q, "q")
    _need(q, "q", dtype=torch.bfloat16, ndim=3)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t, name, ndim=4, device=dev)
        if t.element_size() != 1:
            raise TypeError(f"{name} must be a one-byte (E4M3) tensor")
    _need(block_tables, "block_tables", dtype=torch.int32, ndim=2, device=dev)
    _need(context_lens, "context_lens", dtype=torch.int32, ndim=1, device=dev)
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("inconsistent shapes between q, caches, block_tables and context_lens")
    handle = _stream(stream, dev)
    out, workspace, ws_ptr, ws_bytes = _buffers(stream, q, out, _decode_workspace_args, workspace, B, hq, d, num_splits, dev)
    st = _lib.load().pkv_paged_decode_attn_fp8(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), B, hq, hkv, d, bs, nb, ctypes.c_float(scale), ctypes.c_float(k_scale),
        ctypes.c_float(v_scale), num_splits, ws_ptr, ws_bytes, handle)
    _lib.check("pkv_paged_decode_attn_fp8", st)
    return out


def decode_workspace_bytes(batch: int, num_q_heads: int, head_dim: int, num_splits: int = 0) -> int:
    """Bytes of split workspace paged_decode_attn needs on the current device."""
    return int(_lib.load().pkv_paged_decode_workspace_bytes(batch, num_q_heads, head_dim, num_splits))


def decode_workspace(batch: int, num_q_heads: int, head_dim: int, num_splits: int = 0,
                     device=None) -> torch.Tensor | None:
    """Allocate a zero-filled workspace (uint8) for paged_decode_attn, or None when none is needed."""
    n = decode_workspace_bytes(batch, num_q_heads, head_dim, num_splits)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.cuda.current_device())


def paged_decode_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
                      num_splits: int = 0, workspace: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode attention through block tables; returns out [B, Hq, D] (same dtype as q).

    num_splits: 0 = automatic split over the context, S >= 1 = S equal parts.
    workspace: from decode_workspace(); allocated (zero-filled) when None.
    """
    dev = _device(q, "q")
    _need(q, "q", ndim=3)
    _need(k_cache, "k_cache", dtype=q.dtype, ndim=4, device=dev)
    _need(v_cache, "v_cache", dtype=q.dtype, ndim=4, device=dev)
    _need(block_tables, "block_tables", dtype=torch.int32, ndim=2, device=dev)
    _need(context_lens, "context_lens", dtype=torch.int32, ndim=1, device=dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("inconsistent shapes between q, caches, block_tables and context_lens")
    handle = _stream(stream, dev)
    out, workspace, ws_ptr, ws_bytes = _buffers(stream, q, out, _decode_workspace_args, workspace, B, hq, d, num_splits, dev)
    st = _lib.load().pkv_paged_decode_attn(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), B, hq, hkv, d, bs, nb, ctypes.c_float(scale), num_splits, ws_ptr, ws_bytes,
        _dtype_code(q), handle)
    _lib.check("pkv_paged_decode_attn", st)
    return out


def paged_verify_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
                      num_splits: int = 0, workspace: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Speculative-decoding verify attention: q [B, q_len, Hq, D], the last q_len context
    tokens of each sequence, each causally limited to its own position."""
    dev = _device(q, "q")
    _need(q, "q", ndim=4)
    _need(k_cache, "k_cache", dtype=q.dtype, ndim=4, device=dev)
    _need(v_cache, "v_cache", dtype=q.dtype, ndim=4, device=dev, shape=k_cache.shape)
    _need(block_tables, "block_tables", dtype=torch.int32, ndim=2, device=dev)
    _need(context_lens, "context_lens", dtype=torch.int32, ndim=1, device=dev)
    B, ql, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("inconsistent shapes between q, caches, block_tables and context_lens")
    handle = _stream(stream, dev)
    out, workspace, ws_ptr, ws_bytes = _buffers(stream, q, out, _decode_workspace_args, workspace, B, ql * hq, d, num_splits, dev)
    st = _lib.load().pkv_paged_verify_attn(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), B, ql, hq, hkv, d, bs, nb, ctypes.c_float(scale), num_splits, ws_ptr, ws_bytes,
        _dtype_code(q), handle)
    _lib.check("pkv_paged_verify_attn", st)
    return out


def paged_decode_attn_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
                              num_splits: int = 0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """paged_decode_attn for callers that cannot allocate: the split workspace is the
    library's fixed 8 MiB device array (calls on one device must not overlap)."""
    dev = _device(q, "q")
    _need(q, "q", ndim=3)
    _need(k_cache, "k_cache", dtype=q.dtype, ndim=4, device=dev)
    _need(v_cache, "v_cache", dtype=q.dtype, ndim=4, device=dev, shape=k_cache.shape)
    _need(block_tables, "block_tables", dtype=torch.int32, ndim=2, device=dev)
    _need(context_lens, "context_lens", dtype=torch.int32, ndim=1, device=dev)
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("inconsistent shapes between q, caches, block_tables and context_lens")
    handle = _stream(stream, dev)
    (out,) = _buffers(stream, q, out, tuple)
    st = _lib.load().pkv_paged_decode_attn_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), B, hq, hkv, d, bs, nb, ctypes.c_float(scale), num_splits, _dtype_code(q),
        handle)
    _lib.check("pkv_paged_decode_attn_noalloc", st)
    return out


def prefill_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                            max_seqlen_q: int) -> int:
    """Bytes of the optional split workspace of paged_varlen_prefill_attn (0: never splits)."""
    return int(_lib.load().pkv_paged_varlen_prefill_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim,
                                                                     max_seqlen_q))


def prefill_workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seqlen_q: int,
                      device=None) -> torch.Tensor | None:
    """A zero-filled workspace (uint8) for paged_varlen_prefill_attn, or None when none is needed."""
    n = prefill_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seqlen_q)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.cuda.current_device())


_prefill_ws: dict[int, torch.Tensor] = {}


def _cached_prefill_workspace(nbytes: int, device: torch.device) -> torch.Tensor:
    """One zero-filled workspace per device, grown on demand; the kernel leaves it zeroed."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    ws = _prefill_ws.get(idx)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _prefill_ws[idx] = ws
    return ws


def paged_varlen_prefill_attn(q: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                              max_seqlen_q: int, max_seqlen_k: int, scale: float, *,
                              k: torch.Tensor | None = None, v: torch.Tensor | None = None,
                              k_cache: torch.Tensor | None = None, v_cache: torch.Tensor | None = None,
                              block_tables: torch.Tensor | None = None, causal: bool = True,
                              workspace: torch.Tensor | bool | None = None,
                              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Packed varlen prefill attention; keys through block_tables (cache) or from packed k/v.

    workspace: None = a zero-filled workspace cached per device (calls that may
    overlap on different streams must pass their own), or with `stream` and in a captured
    graph one for this call; False = never split long query tiles; or a tensor from
    prefill_workspace().
    """
    dev = _device(q, "q")
    _need(q, "q", ndim=3)
    _need(cu_seqlens_q, "cu_seqlens_q", dtype=torch.int32, ndim=1, device=dev)
    _need(cu_seqlens_k, "cu_seqlens_k", dtype=torch.int32, ndim=1, device=dev)
    if cu_seqlens_k.shape != cu_seqlens_q.shape:
        raise ValueError("cu_seqlens_q and cu_seqlens_k lengths differ")
    B = cu_seqlens_q.shape[0] - 1
    total_q, hq, d = q.shape
    if block_tables is not None:
        _need(block_tables, "block_tables", dtype=torch.int32, ndim=2, device=dev)
        _need(k_cache, "k_cache", dtype=q.dtype, ndim=4, device=dev)
        _need(v_cache, "v_cache", dtype=q.dtype, ndim=4, device=dev, shape=k_cache.shape)
        nb, bs, hkv, d2 = k_cache.shape
        if d2 != d:
            raise ValueError("k_cache head_dim differs from q's")
        mb = block_tables.shape[1]
        total_k = 0
        if block_tables.shape[0] != B:
            raise ValueError("block_tables rows must equal the batch")
    else:
        if k is None or v is None:
            raise ValueError("without block_tables the packed k and v are required")
        _need(k, "k", dtype=q.dtype, ndim=3, device=dev)
        _need(v, "v", dtype=q.dtype, ndim=3, device=dev)
        hkv = k.shape[1]
        if k.shape[2] != d:
            raise ValueError("k head_dim differs from q's")
        nb = bs = mb = 0
        total_k = k.shape[0]
        if v.shape != k.shape:
            raise ValueError("k and v shapes differ")
    handle = _stream(stream, dev)
    if workspace is None:
        nbytes = prefill_workspace_bytes(B, hq, hkv, d, int(max_seqlen_q))
        if nbytes > 0 and stream is None and not torch.cuda.is_current_stream_capturing():
            workspace = _cached_prefill_workspace(nbytes, dev)
    else:
        nbytes = 0
        if workspace is not False:
            _need(workspace, "workspace", dtype=torch.uint8, device=dev)
    out, workspace, ws_ptr, ws_bytes = _buffers(stream, q, out, _workspace_args, workspace, nbytes, B, dev)
    st = _lib.load().pkv_paged_varlen_prefill_attn(
        _ptr(out), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_k), int(max_seqlen_q), int(max_seqlen_k), _ptr(block_tables), mb, B, total_q,
        total_k, hq, hkv, d, bs, nb, ctypes.c_float(scale), 1 if causal else 0, ws_ptr, ws_bytes,
        _dtype_code(q), handle)
    _lib.check("pkv_paged_varlen_prefill_attn", st)
    return out


def _buffers(stream, q: torch.Tensor, out, workspace_args, *args):
    """out (allocated when None) and the workspace_args(*args) of a call, allocated on the stream the call
    runs on (its pool, and the zero fill in its order)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _buffers(None, q, out, workspace_args, *args)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", dtype=q.dtype, device=q.device, shape=q.shape)
    return out, *workspace_args(*args)


def _workspace_args(workspace, nbytes: int, batch: int, device: torch.device):
    """(tensor, pointer, bytes) of a split workspace: the caller's, none (False), or one for this call."""
    if workspace is False or (workspace is None and nbytes == 0):
        return None, None, 0
    if workspace is None:
        # only the counter area must be zero; past 4096 sequences it may be longer than 64 KiB
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        (workspace if batch > 4096 else workspace.narrow(0, 0, min(nbytes, 65536))).zero_()
    else:
        _need(workspace, "workspace", device=device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _decode_workspace_args(workspace, batch: int, hq: int, d: int, num_splits: int, device):
    return _workspace_args(workspace, decode_workspace_bytes(batch, hq, d, num_splits) if workspace is None else 0,
                           batch * max(num_splits, 1), device)


def chunk_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seqlen_q: int,
                          max_seqlen_k: int) -> int:
    """Bytes of the workspace with which paged_varlen_prefill_attn_mod and _fp8 split these sizes (0: never)."""
    short = int(_lib.load().pkv_paged_short_chunk_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim,
                                                                  max_seqlen_q, max_seqlen_k))
    return max(short, prefill_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seqlen_q))


def chunk_workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seqlen_q: int,
                    max_seqlen_k: int, device=None) -> torch.Tensor | None:
    """A zero-filled workspace (uint8) for paged_varlen_prefill_attn_mod and _fp8, or None when none is needed."""
    n = chunk_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seqlen_q, max_seqlen_k)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.cuda.current_device())


def _chunk_workspace_args(workspace, batch: int, hq: int, hkv: int, d: int, max_q: int, max_k: int, paged: bool, device):
    """The workspace of a chunk call: the caller's if it is large enough for a short chunk, else one for this call."""
    short = 0
    if paged and max_q * hq <= 8 * hkv:
        short = int(_lib.load().pkv_paged_short_chunk_workspace_bytes(batch, hq, hkv, d, max_q, max_k))
    if short > 0 and (workspace is None or workspace is False or workspace.numel() * workspace.element_size() < short):
        return _workspace_args(None, short, batch, device)
    return _workspace_args(workspace, prefill_workspace_bytes(batch, hq, hkv, d, max_q) if workspace is None else 0,
                           batch, device)


def _need_modifiers(device, num_q_heads: int, alibi_slopes, first_keys, rows: int, prefix_lens=None, batch: int = 0):
    if alibi_slopes is not None:
        _need(alibi_slopes, "alibi_slopes", dtype=torch.float32, device=device, shape=(num_q_heads,))
    if first_keys is not None:
        _need(first_keys, "first_keys", dtype=torch.int32, device=device, shape=(rows,))
    if prefix_lens is not None:
        _need(prefix_lens, "prefix_lens", dtype=torch.int32, device=device, shape=(batch,))


def paged_decode_attn_mod(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
                          softcap: float = 0.0, alibi_slopes: torch.Tensor | None = None,
                          first_keys: torch.Tensor | None = None, num_splits: int = 0,
                          workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """paged_decode_attn with modified scores; returns out [B, Hq, D] (same dtype as q).

    softcap: scores become softcap * tanh(score / softcap) (0 = none).
    alibi_slopes: float32 [Hq]; head h's scores fall by alibi_slopes[h] per position of distance.
    first_keys: int32 [B]; keys before it are not seen (window, or the start of the document).
    workspace: from decode_workspace(); allocated (zero-filled) for the call when None.
    """
    dev = _device(q, "q")
    _need(q, "q", ndim=3)
    _need(k_cache, "k_cache", dtype=q.dtype, ndim=4, device=dev)
    _need(v_cache, "v_cache", dtype=q.dtype, ndim=4, device=dev, shape=k_cache.shape)
    _need(block_tables, "block_tables", dtype=torch.int32, ndim=2, device=dev)
    _need(context_lens, "context_lens", dtype=torch.int32, ndim=1, device=dev)
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("inconsistent shapes between q, caches, block_tables and context_lens")
    _need_modifiers(dev, hq, alibi_slopes, first_keys, B)
    handle = _stream(stream, dev)
    out, workspace, ws_ptr, ws_bytes = _buffers(stream, q, out, _decode_workspace_args, workspace, B, hq, d, num_splits,
                                                dev)
    st = _lib.load().pkv_paged_decode_attn_mod(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), B, hq, hkv, d, bs, nb, scale, softcap, _ptr(alibi_slopes),
        _ptr(first_keys), num_splits, ws_ptr, ws_bytes, _dtype_code(q), handle)
    _lib.check("pkv_paged_decode_attn_mod", st)
    return out


def paged_varlen_prefill_attn_mod(q: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                                  max_seqlen_q: int, max_seqlen_k: int, scale: float, *,
                                  k: torch.Tensor | None = None, v: torch.Tensor | None = None,
                                  k_cache: torch.Tensor | None = None, v_cache: torch.Tensor | None = None,
                                  block_tables: torch.Tensor | None = None, causal: bool = True,
                                  softcap: float = 0.0, alibi_slopes: torch.Tensor | None = None,
                                  first_keys: torch.Tensor | None = None, prefix_lens: torch.Tensor | None = None,
                                  workspace: torch.Tensor | bool | None = None,
                                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """paged_varlen_prefill_attn with modified scores; keys through block_tables (cache) or from packed k/v.

    softcap, alibi_slopes: as for paged_decode_attn_mod.
    first_keys: int32 [total_q]; the row does not see keys before it (document or window mask).
    prefix_lens: int32 [B]; every row of the sequence sees keys below it besides the causal ones.
    workspace: a tensor from chunk_workspace() (or prefill_workspace()); None = a zero-filled one
    for this call where a split needs it; False = never split long query tiles.  Short chunks
    (max_seqlen_q * Hq / Hkv <= 8 over a long cache) take one for the call where the given one is too small.
    """
    dev = _device(q, "q")
    _need(q, "q", ndim=3)
    _need(cu_seqlens_q, "cu_seqlens_q", dtype=torch.int32, ndim=1, device=dev)
    _need(cu_seqlens_k, "cu_seqlens_k", dtype=torch.int32, ndim=1, device=dev, shape=cu_seqlens_q.shape)
    if cu_seqlens_q.shape[0] < 1:
        raise ValueError("cu_seqlens_q must hold batch + 1 offsets")
    B = cu_seqlens_q.shape[0] - 1
    total_q, hq, d = q.shape
    if block_tables is not None:
        _need(block_tables, "block_tables", dtype=torch.int32, ndim=2, device=dev)
        _need(k_cache, "k_cache", dtype=q.dtype, ndim=4, device=dev)
        _need(v_cache, "v_cache", dtype=q.dtype, ndim=4, device=dev, shape=k_cache.shape)
        nb, bs, hkv, d2 = k_cache.shape
        mb, total_k = block_tables.shape[1], 0
        if block_tables.shape[0] != B:
            raise ValueError("block_tables rows must equal the batch")
    else:
        if k is None or v is None:
            raise ValueError("without block_tables the packed k and v are required")
        _need(k, "k", dtype=q.dtype, ndim=3, device=dev)
        _need(v, "v", dtype=q.dtype, ndim=3, device=dev, shape=k.shape)
        total_k, hkv, d2 = k.shape
        nb = bs = mb = 0
    if d2 != d:
        raise ValueError("the keys' head_dim differs from q's")
    _need_modifiers(dev, hq, alibi_slopes, first_keys, total_q, prefix_lens, B)
    handle = _stream(stream, dev)
    out, workspace, ws_ptr, ws_bytes = _buffers(stream, q, out, _chunk_workspace_args, workspace, B, hq, hkv, d,
                                                int(max_seqlen_q), int(max_seqlen_k), block_tables is not None, dev)
    st = _lib.load().pkv_paged_varlen_prefill_attn_mod(
        _ptr(out), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_k), int(max_seqlen_q), int(max_seqlen_k), _ptr(block_tables), mb, B, total_q,
        total_k, hq, hkv, d, bs, nb, scale, 1 if causal else 0, softcap,
        _ptr(alibi_slopes), _ptr(first_keys), _ptr(prefix_lens), ws_ptr, ws_bytes, _dtype_code(q), handle)
    _lib.check("pkv_paged_varlen_prefill_attn_mod", st)
    return out


def paged_varlen_prefill_attn_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, cu_seqlens_q: torch.Tensor,
                                  cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, scale: float,
                                  k_scale: float, v_scale: float, *, causal: bool = True,
                                  workspace: torch.Tensor | bool | None = None,
                                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Varlen prefill attention of new tokens over an E4M3 cache (uint8 or float8_e4m3fn tensors)
    with per-tensor scales; q / out bf16 [total_q, Hq, D].  The new rows are stored first
    (kv_store_fp8).  workspace: as for paged_varlen_prefill_attn_mod."""
    dev = _device(q, "q")
    _need(q, "q", dtype=torch.bfloat16, ndim=3)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t, name, ndim=4, device=dev, shape=k_cache.shape)
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise TypeError(f"{name} must hold E4M3 codes (uint8 or float8_e4m3fn)")
    _need(block_tables, "block_tables", dtype=torch.int32, ndim=2, device=dev)
    _need(cu_seqlens_q, "cu_seqlens_q", dtype=torch.int32, ndim=1, device=dev)
    _need(cu_seqlens_k, "cu_seqlens_k", dtype=torch.int32, ndim=1, device=dev, shape=cu_seqlens_q.shape)
    B = cu_seqlens_q.shape[0] - 1
    total_q, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("k_cache head_dim differs from q's")
    if block_tables.shape[0] != B:
        raise ValueError("block_tables rows must equal the batch")
    handle = _stream(stream, dev)
    out, workspace, ws_ptr, ws_bytes = _buffers(stream, q, out, _chunk_workspace_args, workspace, B, hq, hkv, d,
                                                int(max_seqlen_q), int(max_seqlen_k), True, dev)
    st = _lib.load().pkv_paged_varlen_prefill_attn_fp8(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_seqlen_q),
        int(max_seqlen_k), _ptr(block_tables), block_tables.shape[1], B, total_q, hq, hkv, d, bs, nb,
        scale, k_scale, v_scale, 1 if causal else 0, ws_ptr, ws_bytes,
        handle)
    _lib.check("pkv_paged_varlen_prefill_attn_fp8", st)
    return out


def device_error(reset: bool = True) -> int:
    """Read (and by default clear) the current device's error word; synchronises the device."""
    flags = ctypes.c_uint32(0)
    _lib.check("pkv_get_device_error", _lib.load().pkv_get_device_error(ctypes.byref(flags), 1 if reset else 0))
    return int(flags.value)
