"""Cases, plain forms and 64-bit definitions of three operators around a paged KV cache.

kv_rope_store, _fp8, _q4      rotates a step's q and k by position and stores k and v in the cache (f32, bf16, E4M3,
                              4 bits); kv_load_q4 reads stored 4-bit rows back as values
paged_decode_attn_q4          one query token per sequence over a 4-bit cache
paged_varlen_prefill_attn_q4  a chunk of new tokens per sequence over a 4-bit cache

Rotation of a head's first r elements, with c and s the cosines and sines of its position:
    y[i] = x[i] c[i] - x[j] s[i];  y[j] = x[j] c[i] + x[i] s[i]     j = i + r / 2, or neighbours (2i, 2i + 1)
rounded to float32 and then to x's type.  4 bits: an element is (code - 8) * E4M3 scale of its group of 16 * the
tensor's scale T; the group's scale is e4m3(amax / (7 T)), the codes round to the nearest even and stop at -8 and 7.
A token's row holds the code bytes of every KV head (low nibble first), then the scale bytes, padded to 16 bytes.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
K_SCALE, V_SCALE = 1.0 / 64, 3.0 / 256


def _append(name, cache, tokens, **kw):
    return dict(dict(name=name, op="append", cache=cache, tokens=tokens, pad=0, hq=16, hkv=8, d=128, bs=256, rot=128,
                     span=32768, decode=False, neighbours=False, fused=False), **kw)


def _decode(name, lens, **kw):
    return dict(dict(name=name, op="decode", lens=lens, hq=16, hkv=8, d=128, bs=256), **kw)


def _chunk(name, history, new, **kw):
    return dict(dict(name=name, op="chunk", history=history, new=new, hq=16, hkv=8, d=128, bs=256), **kw)


def _spread(seed, n, lo, hi):
    """n lengths of [lo, hi], as a text (a case holds plain values)."""
    rng = random.Random(seed)
    return " ".join(str(rng.randint(lo, hi)) for _ in range(n))


def _prefixes(seed, n, bs=256, chunk=512):
    """A batch resuming after prefix hits: totals of [256, 4096], up to half of each cached, up to `chunk` new tokens."""
    rng = random.Random(seed)
    hist, new = [], []
    for _ in range(n):
        total = rng.randint(256, 4096)
        hist.append(bs * rng.randint(0, total // 2 // bs))
        new.append(min(chunk, total - hist[-1]))
    return " ".join(map(str, hist)), " ".join(map(str, new))


def listed():
    hist, new = _prefixes(1004, 16)
    return [
        # one decode step of a small batch, padded to the captured graph's 8 rows: the call's latency
        _append("append_decode8", "bf16", "6", pad=2, decode=True),
        # one decode step of a large batch into an E4M3 cache, rows taken from the fused projection's output
        _append("append_decode256_fp8", "e4m3", "256", decode=True, fused=True),
        # the new tokens of a chunked-prefill batch into a 4-bit cache, read back as values
        _append("append_chunks_q4", "q4", new),
        # a float32 cache with narrow heads, half of each rotated, neighbouring pairs, ragged prompts
        _append("append_f32_partial", "f32", "1 333 700", hq=8, hkv=2, d=64, bs=24, rot=32, neighbours=True),
        # whole prompts of a large batch: HBM-bound
        _append("append_prompts_bf16", "bf16", " ".join(["4096"] * 16), fused=True),
        # one user's chat, one token: latency
        _decode("decode_one_q4", "777", bs=16),
        # a serving batch
        _decode("decode_batch32_q4", _spread(1002, 32, 128, 2048)),
        # a large serving batch: HBM-bound
        _decode("decode_batch256_q4", _spread(1003, 256, 1024, 8192)),
        # very long contexts, four query heads per KV head: split over the context
        _decode("decode_long_q4", "32768 65536 100000 131072", hq=32, bs=16),
        # four drafted tokens for each sequence of a batch
        _chunk("verify4_q4", _spread(17, 24, 1024, 8192), " ".join(["4"] * 24)),
        # chunked prefill of a batch with prefix hits
        _chunk("chunk_batch16_q4", hist, new),
        # narrow heads, one KV head, pages that no tile is a multiple of
        _chunk("chunk_ragged_d64_q4", "1000 0 37 513", "129 300 1 64", hq=8, hkv=1, d=64, bs=24),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "chunk"])
    hkv, g, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    common = dict(hq=hkv * g, hkv=hkv, d=d, bs=rng.choice([8, 16, 24, 32, 64, 100, 128, 256]))
    if op == "append":
        cache = rng.choice(["bf16", "bf16", "f32", "e4m3", "q4", "q4"])
        elements = 65536 * 32 * 128 // (2 if cache == "f32" else 1)
        most = min(65536, elements // ((g + 2) * hkv * d))
        common.update(rot=rng.choice([32, d, d]), span=rng.choice([4096, 32768, 131072]), neighbours=rng.random() < 0.3,
                      fused=rng.random() < 0.5, pad=rng.choice([0, 0, rng.randint(1, 9)]))
        if rng.random() < 0.4:
            return _append(None, cache, str(_log(rng, 1, 512)), decode=True, **common)
        n = _log(rng, 1, 16)
        top = _log(rng, 1, min(4096, most // n))
        return _append(None, cache, " ".join(str(rng.randint(max(1, top // 3), top)) for _ in range(n)), **common)
    if op == "decode":
        n = _log(rng, 1, 256)
        top = _log(rng, 1, min(131072, 1048576 // n))
        return _decode(None, " ".join(str(rng.randint(max(0, top // 8), top)) for _ in range(n)), **common)
    n = _log(rng, 1, 24)
    top = _log(rng, 1, 1024 if n > 4 else 2048)
    new = [rng.randint(max(1, top // 3), top) for _ in range(n)]
    far = rng.choice([0, _log(rng, 1, 65536 // n), _log(rng, 1, 65536 // n)])
    hist = [rng.randint(far // 3, far) for _ in range(n)]
    while sum(new) * (max(hist) + max(new)) * hkv * g > 200_000_000:  # below the largest listed chunks
        new = [max(1, x // 2) for x in new]
        hist = [x // 2 for x in hist]
    return _chunk(None, " ".join(map(str, hist)), " ".join(map(str, new)), **common)


# ------------------------------------------------------------------ what a case says (no tensors)

def _ints(text):
    return np.array([int(x) for x in text.split()], dtype=np.int64)


def _row_bytes(case):
    """Bytes of one token's K (or V) row in the 4-bit cache."""
    return -(-case["hkv"] * (case["d"] // 2 + case["d"] // 16) // 16) * 16


def _lengths(case):
    """New tokens and total keys of each sequence of an attention case."""
    if case["op"] == "decode":
        keys = _ints(case["lens"])
        return np.minimum(keys, 1), keys
    new, hist = _ints(case["new"]), _ints(case["history"])
    return new, hist + new


def _places(case, seed):
    """Positions and slots of an append's tokens (padding rows last), and the cache's blocks."""
    rng = np.random.default_rng(seed)
    counts, bs = _ints(case["tokens"]), case["bs"]
    if case["decode"]:  # a token of every sequence, wherever it stands
        counts = np.ones(int(counts.sum()), dtype=np.int64)
    position, slots, blocks = [], [], 0
    for n in counts:
        start = int(rng.integers(0, max(1, case["span"] - n)))
        p = start + np.arange(n)
        position.append(p)
        slots.append((p // bs - start // bs + blocks) * bs + p % bs)
        blocks += int(n + bs - 2) // bs + 1  # wherever the run starts
    order = rng.permutation(blocks + 2)
    slots = np.concatenate(slots)
    slots = order[slots // bs] * bs + slots % bs
    pad = np.full(case["pad"], -1)
    return np.concatenate([np.concatenate(position), 0 * pad]), np.concatenate([slots, pad]), blocks + 2


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        position, slots, _ = _places(case, 0)
        es = 4 if case["cache"] == "f32" else 2
        kept = int((slots >= 0).sum())
        row = {"q4": _row_bytes(case), "e4m3": hkv * d}.get(case["cache"], hkv * d * es)
        read = (len(slots) * hq + 2 * kept * hkv) * d * es + len(np.unique(position)) * case["rot"] * 4 + 8 * len(slots)
        written = len(slots) * hq * d * es + 2 * kept * row
        if case["cache"] == "q4":  # the rows read back
            read, written = read + 2 * kept * row, written + 2 * len(slots) * hkv * d * 2
        return {"bytes": read + written, "flops": 3 * (len(slots) * hq + kept * hkv) * case["rot"]}
    new, keys = _lengths(case)
    pairs = sum(int(n) * int(t) - int(n) * (int(n) - 1) // 2 for n, t in zip(new, keys))
    pages = int((-(-keys // case["bs"])).sum())
    return {"bytes": int(keys.sum()) * 2 * _row_bytes(case) + 2 * int(new.sum()) * hq * d * 2 + 4 * pages + 4 * len(keys),
            "flops": 4 * hq * d * pairs}


# ------------------------------------------------------------------ inputs

def _dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(DEV)


def _rows_q4(x, scale):
    """Rows [n, hkv, d] of bf16 as 4-bit rows [n, row bytes], in float32 arithmetic."""
    n, hkv, d = x.shape
    x = x.float().reshape(n, hkv, d // 16, 16)
    t = torch.tensor(scale, dtype=torch.float32, device=x.device)
    s = (x.abs().amax(-1) / (7 * t)).clamp(max=448.0).to(E4M3)
    step = (s.float() * t)[..., None]
    code = torch.where(step > 0, torch.round(x / step).clamp(-8, 7) + 8, torch.full_like(x, 8.0)).to(torch.uint8)
    code = code.reshape(n, hkv * d)
    code = code[:, 0::2] | (code[:, 1::2] << 4)
    parts = [code, s.view(torch.uint8).reshape(n, -1)]
    short = -(code.shape[1] + parts[1].shape[1]) % 16
    if short:
        parts.append(torch.zeros(n, short, dtype=torch.uint8, device=x.device))
    return torch.cat(parts, 1)


def _pool_q4(case, blocks, gen, scale):
    """A 4-bit pool [blocks, bs, row bytes] of normal values, made in pieces."""
    rows = blocks * case["bs"]
    pool = torch.empty(rows, _row_bytes(case), dtype=torch.uint8, device=DEV)
    for a in range(0, rows, 65536):
        n = min(65536, rows - a)
        x = torch.randn(n, case["hkv"], case["d"], generator=gen, device=DEV).to(torch.bfloat16)
        pool[a:a + n] = _rows_q4(x, scale)
    return pool.view(blocks, case["bs"], -1)


def _inputs(case, seed):
    """Everything that the definition takes, on the GPU, from the case and the seed alone."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    if case["op"] == "append":
        dtype = TYPES["f32" if case["cache"] == "f32" else "bf16"]
        position, slots, blocks = _places(case, seed)
        n = len(slots)
        s = {"case": case, "positions": _dev(position), "slots": _dev(slots), "neighbours": case["neighbours"]}
        if case["fused"]:  # views of the projection's rows
            qkv = torch.randn(n, hq + 2 * hkv, d, generator=gen, device=DEV).to(dtype)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = [torch.randn(n, h, d, generator=gen, device=DEV).to(dtype) for h in (hq, hkv, hkv)]
        angle = torch.arange(case["span"], device=DEV, dtype=torch.float64)[:, None] * torch.pow(
            1e6, -torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case["cache"] == "q4":
            s["k_cache"], s["v_cache"] = _pool_q4(case, blocks, gen, K_SCALE), _pool_q4(case, blocks, gen, V_SCALE)
        else:
            pools = [torch.randn(blocks, bs, hkv, d, generator=gen, device=DEV) for _ in range(2)]
            if case["cache"] == "e4m3":
                pools = [(x / t).clamp_(-448, 448).to(E4M3).view(torch.uint8) for x, t in zip(pools, (K_SCALE, V_SCALE))]
            else:
                pools = [x.to(dtype) for x in pools]
            s["k_cache"], s["v_cache"] = pools
        return s
    new, keys = _lengths(case)
    rng = np.random.default_rng(seed)
    need = -(-keys // bs)
    blocks = int(need.sum()) + 3
    order, at = rng.permutation(blocks), 0
    tables = np.full((len(keys), max(1, int(need.max()))), -1)
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    rows = len(keys) if case["op"] == "decode" else int(new.sum())
    s = {"case": case, "scale": d ** -0.5, "tables": _dev(tables), "max_q": int(new.max()), "max_k": int(keys.max()),
         "q": (torch.randn(rows, hq, d, generator=gen, device=DEV) * 3).to(torch.bfloat16),
         "k_cache": _pool_q4(case, blocks, gen, K_SCALE), "v_cache": _pool_q4(case, blocks, gen, V_SCALE)}
    if case["op"] == "decode":
        s["lens"] = _dev(keys)
    else:
        s["cu_q"], s["cu_k"] = _dev(np.concatenate([[0], np.cumsum(new)])), _dev(np.concatenate([[0], np.cumsum(keys)]))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        kept = torch.nonzero(s["slots"] >= 0)[:, 0]  # rows that are stored, for the plain form
        s["kept"], s["to"] = kept, s["slots"][kept].long()
    elif case["op"] == "chunk":  # where row j of sequence i lies among the padded rows, for the plain form
        new, _ = _lengths(case)
        s["flat"] = _dev(np.concatenate([i * s["max_q"] + np.arange(n) for i, n in enumerate(new)]), np.int64)
    if own and case["op"] != "append":  # the workspace that a serving program keeps from step to step
        import pagedattention_kv_cache_gb300 as pkv
        if case["op"] == "decode":
            s["workspace"] = pkv.decode_workspace(len(s["lens"]), case["hq"], case["d"])
        else:
            s["workspace"] = pkv.chunk_workspace(len(s["cu_q"]) - 1, case["hq"], case["hkv"], case["d"], s["max_q"],
                                                 s["max_k"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    return {"append": _plain_append, "decode": _plain_decode, "chunk": _plain_chunk}[s["case"]["op"]](s)


def _own(s):
    import pagedattention_kv_cache_gb300 as pkv
    case = s["case"]
    if case["op"] == "decode":
        return pkv.paged_decode_attn_q4(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"], K_SCALE,
                                        V_SCALE, case["hkv"], workspace=s["workspace"])
    if case["op"] == "chunk":
        return pkv.paged_varlen_prefill_attn_q4(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["cu_q"], s["cu_k"],
                                                s["max_q"], s["max_k"], s["scale"], K_SCALE, V_SCALE, case["hkv"],
                                                workspace=False if s["workspace"] is None else s["workspace"])
    args = (s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["k_cache"], s["v_cache"], s["slots"])
    if case["cache"] == "q4":
        q = pkv.kv_rope_store_q4(*args, K_SCALE, V_SCALE, interleaved=s["neighbours"])
        k, v = pkv.kv_load_q4(s["k_cache"], s["v_cache"], s["slots"], K_SCALE, V_SCALE, case["hkv"], case["d"])
        return {"q": q, "k": k, "v": v}
    if case["cache"] == "e4m3":
        q = pkv.kv_rope_store_fp8(*args, K_SCALE, V_SCALE, interleaved=s["neighbours"])
        return {"q": q, "k_cache": s["k_cache"].view(E4M3), "v_cache": s["v_cache"].view(E4M3)}
    q = pkv.kv_rope_store(*args, interleaved=s["neighbours"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _rotated(s, x, wide):
    """x [n, heads, d] rotated, in `wide` arithmetic, rounded to float32 and to x's type."""
    half = s["cos_sin"].shape[1] // 2
    table = s["cos_sin"][s["positions"].long()].to(wide)[:, None]
    c, t = table[..., :half], table[..., half:]
    y, rest = x[..., :2 * half].to(wide), x[..., 2 * half:]
    if s["neighbours"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * t, b * c + a * t], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:]
        y = torch.cat([a * c - b * t, b * c + a * t], -1)
    return torch.cat([y.float().to(x.dtype), rest], -1)


def _plain_append(s):
    cache = s["case"]["cache"]
    # quantized keys: 64 bits, since a value next to a border between two codes would change the code
    k = _rotated(s, s["k"], torch.float64 if cache in ("e4m3", "q4") else torch.float32)
    q = _rotated(s, s["q"], torch.float32)
    for name, x, t in (("k_cache", k, K_SCALE), ("v_cache", s["v"], V_SCALE)):
        rows, x = s[name].view(-1, *s[name].shape[2:]), x[s["kept"]]
        if cache == "q4":
            x = _rows_q4(x, t)
        elif cache == "e4m3":
            x = (x.float() / t).clamp(-448, 448).to(E4M3).view(torch.uint8)
        rows[s["to"]] = x
    if cache == "q4":
        out = {"q": q}
        for name, x, t in (("k", "k_cache", K_SCALE), ("v", "v_cache", V_SCALE)):
            full = torch.zeros(s["k"].shape, dtype=torch.bfloat16, device=q.device)
            row = s[x].view(-1, s[x].shape[-1])[s["to"]]
            full[s["kept"]] = _values(s["case"], row, t).to(torch.bfloat16)
            out[name] = full
        return out
    view = (lambda x: x.view(E4M3)) if cache == "e4m3" else (lambda x: x)
    return {"q": q, "k_cache": view(s["k_cache"]), "v_cache": view(s["v_cache"])}


def _values(case, rows, scale):
    """4-bit rows [..., row bytes] as float32 [..., hkv, d]."""
    hkv, d = case["hkv"], case["d"]
    code = rows[..., :hkv * d // 2]
    code = torch.stack([code & 15, code >> 4], -1).reshape(*rows.shape[:-1], hkv, d // 16, 16)
    s = rows[..., hkv * d // 2:hkv * (d // 2 + d // 16)].contiguous().view(E4M3).float()
    return ((code.float() - 8) * (s * scale).reshape(*rows.shape[:-1], hkv, d // 16, 1)).flatten(-2)


def _attend(s, q, seen):
    """q [n, rows, hq, d], seen [n, rows, keys] -> [n, rows, hq, d], all in float32."""
    case = s["case"]
    t = torch.arange(s["max_k"], device=q.device)
    blocks = s["tables"].long().clamp_min(0)[:, t // case["bs"]]
    k = _values(case, s["k_cache"][blocks, t % case["bs"]], K_SCALE)
    n, rows, hq, d = q.shape
    hkv = case["hkv"]
    q = q.float().reshape(n, rows, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    x = (q @ k.permute(0, 2, 3, 1)).reshape(n, hq, rows, -1) * s["scale"]
    del k
    x = x.masked_fill(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = x.sum(-1, keepdim=True)
    v = _values(case, s["v_cache"][blocks, t % case["bs"]], V_SCALE)
    out = (x.reshape(n, hkv, -1, x.shape[-1]) @ v.permute(0, 2, 1, 3)).reshape(n, hq, rows, d)
    return (out / torch.where(total > 0, total, torch.ones_like(total))).permute(0, 2, 1, 3)


def _plain_decode(s):
    t = torch.arange(s["max_k"], device=s["q"].device)
    return _attend(s, s["q"][:, None], (t < s["lens"].long()[:, None])[:, None])[:, 0].to(s["q"].dtype)


def _plain_chunk(s):
    new, keys = s["cu_q"].diff().long(), s["cu_k"].diff().long()
    r, t = torch.arange(s["max_q"], device=s["q"].device), torch.arange(s["max_k"], device=s["q"].device)
    rows = (s["cu_q"][:-1, None].long() + r).clamp_max(s["q"].shape[0] - 1)
    seen = t <= ((keys - new)[:, None] + r)[..., None]
    out = _attend(s, s["q"][rows], seen & (t < keys[:, None, None]))
    return out.reshape(-1, *out.shape[2:])[s["flat"]].to(s["q"].dtype)


# ------------------------------------------------------------------ the definition in 64 bits

def _decoded(case, rows, scale):
    """Values of 4-bit rows [n, row bytes], in 64 bits, head by head: [n, hkv, d]."""
    hkv, d = case["hkv"], case["d"]
    out = torch.empty(rows.shape[0], hkv, d, dtype=torch.float64, device=rows.device)
    for h in range(hkv):
        at = hkv * d // 2 + h * (d // 16)
        step = rows[:, at:at + d // 16].contiguous().view(E4M3).double().repeat_interleave(16, 1) * scale
        byte = rows[:, h * d // 2:(h + 1) * d // 2].long()
        out[:, h, 0::2] = (byte % 16 - 8) * step[:, 0::2]
        out[:, h, 1::2] = (byte // 16 - 8) * step[:, 1::2]
    return out


def _quantized(x, scale):
    """The values that a 4-bit row of x [n, hkv, d] stands for."""
    group = x.double().unflatten(-1, (-1, 16))
    largest = group.abs().max(-1, keepdim=True).values
    step = (largest / (7 * scale)).clamp(max=448).float().to(E4M3).double() * scale
    code = torch.clamp(torch.round(group / step), -8, 7)
    return torch.where(step == 0, torch.zeros_like(code), code * step).flatten(-2)


def _exact_append(case, s):
    def turned(x):
        x = x.double()
        half = case["rot"] // 2
        y = x.clone()
        p = s["positions"].long()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["neighbours"] else (i, i + half)
            c, t = s["cos_sin"][p, i].double()[:, None], s["cos_sin"][p, half + i].double()[:, None]
            y[..., a] = x[..., a] * c - x[..., b] * t
            y[..., b] = x[..., b] * c + x[..., a] * t
        return y

    slots, out = s["slots"].long(), {"q": turned(s["q"])}
    stored = slots >= 0
    for name, x, scale in (("k", turned(s["k"]), K_SCALE), ("v", s["v"].double(), V_SCALE)):
        if case["cache"] == "q4":
            x = _quantized(x.float().to(torch.bfloat16), scale)
            x[~stored] = 0
            out[name] = x
            continue
        pool = s[name + "_cache"]
        if case["cache"] == "e4m3":
            pool = pool.view(E4M3)
            x = (x.float().to(torch.bfloat16).double() / scale).clamp(-448, 448).float().to(E4M3).double()
        pool = pool.double()
        pool.view(-1, *pool.shape[2:])[slots[stored]] = x[stored]
        out[name + "_cache"] = pool
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    new, keys = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    group, first = case["hq"] // case["hkv"], 0
    pools = [s[x].view(-1, s[x].shape[-1]) for x in ("k_cache", "v_cache")]
    for i in range(len(keys)):
        n, total = int(new[i]), int(keys[i])
        row0 = i if case["op"] == "decode" else first
        first += n
        if n == 0 or total == 0:
            continue
        t = torch.arange(total, device=out.device)
        slot = s["tables"][i].long()[t // case["bs"]] * case["bs"] + t % case["bs"]
        k, v = _decoded(case, pools[0][slot], K_SCALE), _decoded(case, pools[1][slot], V_SCALE)
        hidden = t > (total - n + torch.arange(n, device=out.device))[:, None]
        for h in range(case["hq"]):
            score = s["q"][row0:row0 + n, h].double() @ k[:, h // group].T * case["d"] ** -0.5
            out[row0:row0 + n, h] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v[:, h // group]
    return out
