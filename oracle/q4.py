"""Oracle for the 4-bit KV cache and the rotating store.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages fix neither; the readings taken here are the library's own
definitions.  4 bits: an element is (code - 8) * e4m3(scale byte) * T, one
scale byte per 16 elements of a head and one float T per tensor.  A token's row
is every head's code bytes (element 2i in the low nibble of byte i), then every
head's scale bytes, then padding to a multiple of 16 bytes.  Storing rounds
amax / (7 T) to E4M3 and x / (scale T) to the nearest code, ties to even, in
float32 arithmetic.  Rotation: the pair (a, b) becomes (a c - b s, b c + a s).
"""

from __future__ import annotations

import numpy as np

from . import fp8


def row_bytes(hkv: int, d: int) -> int:
    n = hkv * d // 2 + hkv * d // 16
    while n % 16:
        n += 1
    return n


def encode_group(x, t: float) -> tuple[np.ndarray, int]:
    """Sixteen codes and the scale byte of sixteen values."""
    x = np.asarray(x, dtype=np.float32)
    t = np.float32(t)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        largest = np.max(np.abs(x))  # (a NaN stays one)
        scale = int(fp8.e4m3_encode(np.float64(largest / np.float32(np.float32(7) * t))).item())
        step = np.float32(np.float32(fp8.e4m3_decode(np.uint8(scale))) * t)
        if not step > 0:
            return np.full(16, 8, dtype=np.uint8), scale
        ratio = (x / step).astype(np.float64)
    return (np.clip(np.rint(ratio), -8, 7) + 8).astype(np.uint8), scale


def encode_row(x, t: float) -> np.ndarray:
    """The bytes of one token's row [hkv, d] (padding bytes 0)."""
    hkv, d = np.shape(x)
    row = np.zeros(row_bytes(hkv, d), dtype=np.uint8)
    for h in range(hkv):
        for g in range(d // 16):
            codes, scale = encode_group(x[h][16 * g:16 * g + 16], t)
            for i in range(8):
                row[h * d // 2 + 8 * g + i] = codes[2 * i] + 16 * codes[2 * i + 1]
            row[hkv * d // 2 + h * d // 16 + g] = scale
    return row


def store(cache, x, slots, t: float) -> np.ndarray:
    """A copy of cache [nb, bs, row bytes] with the rows of x [n, hkv, d] at slots (-1 skips, padding kept)."""
    out = np.array(cache, dtype=np.uint8, copy=True)
    _, hkv, d = np.shape(x)
    used = hkv * d // 2 + hkv * d // 16
    for i, slot in enumerate(np.asarray(slots).tolist()):
        if slot == -1:
            continue
        block, offset = divmod(slot, out.shape[1])
        out[block, offset, :used] = encode_row(x[i], t)[:used]
    return out


def values(cache, hkv: int, d: int, t: float) -> np.ndarray:
    """float64 values [..., hkv, d] of rows [..., row bytes]."""
    cache = np.asarray(cache, dtype=np.uint8)
    codes = cache[..., :hkv * d // 2]
    nibbles = np.empty((*codes.shape[:-1], hkv * d), dtype=np.int64)
    nibbles[..., 0::2] = codes % 16
    nibbles[..., 1::2] = codes // 16
    scales = fp8.e4m3_decode(cache[..., hkv * d // 2:hkv * d // 2 + hkv * d // 16])
    out = (nibbles - 8) * (np.repeat(scales, 16, axis=-1) * float(np.float32(t)))
    return out.reshape(*cache.shape[:-1], hkv, d)


def rotate(x, positions, cos_sin, interleaved: bool) -> np.ndarray:
    """float64 x [n, heads, d] rotated by the float32 table's entries."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    half = cos_sin.shape[1] // 2
    for i, p in enumerate(np.asarray(positions).tolist()):
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            c, s = float(cos_sin[p, j]), float(cos_sin[p, half + j])
            out[i, :, a] = x[i, :, a] * c - x[i, :, b] * s
            out[i, :, b] = x[i, :, b] * c + x[i, :, a] * s
    return out
