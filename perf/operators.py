"""Cases, plain forms and 64-bit definitions of three attention operators over a paged KV cache.

paged_decode_attn_mod          one query token per sequence; scores may be capped by a tanh, biased by
                               distance (one slope per query head) and cut at a first visible key
paged_varlen_prefill_attn_mod  a chunk of new tokens per sequence, the same modifiers, and a prefix
                               that every row sees besides the causal mask
paged_varlen_prefill_attn_fp8  a chunk of new tokens over an E4M3 cache with one scale for K, one for V

With s = scale * q . k, key t, query position p, query head h:
    s <- cap * tanh(s / cap)                      (cap > 0)
    s <- s - slope[h] * |p - t|                   (slopes given)
    t is seen when first[row] <= t and (t <= p or t < prefix[sequence])
    out = softmax(s over seen t) V, zeros for a row that sees nothing.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _decode(name, lens, **kw):
    return dict(dict(name=name, op="decode", lens=lens, hq=16, hkv=8, d=128, bs=256, type="bf16", cap=0.0, alibi=False,
                     window=0), **kw)


def _chunk(name, op, history, new, **kw):
    return dict(dict(name=name, op=op, history=history, new=new, hq=16, hkv=8, d=128, bs=256, paged=True, cap=0.0,
                     alibi=False, window=0, docs=0, prefix=0), **kw)


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
        # one user's chat, one token: the call's latency
        _decode("decode_one_capped", "777", bs=16, cap=50.0),
        # a serving batch of a model with a distance bias instead of positions
        _decode("decode_batch32_alibi", _spread(1002, 32, 128, 2048), alibi=True),
        # a float32 cache with narrow heads, ragged, a padding row, capped and biased at once
        _decode("decode_f32_d64", "0 1 4095 1500 33 2049 640 17", hq=8, hkv=2, d=64, bs=24, type="f32", cap=30.0, alibi=True),
        # very long contexts, scores capped: HBM-bound
        _decode("decode_long_capped", "32768 65536 100000 131072", hq=32, bs=16, cap=50.0),
        # the same contexts in a layer that sees only the last 4096 tokens
        _decode("decode_long_window", "32768 65536 100000 131072", hq=32, bs=16, cap=50.0, window=4096),
        # a short question after a prefix that all its rows see: latency of a small chunk
        _chunk("chunk_small_prefix", "mod", "96 0", "33 7", hq=8, hkv=2, d=64, bs=16, prefix=64),
        # chunked prefill of a batch with prefix hits, scores capped
        _chunk("chunk_batch16_capped", "mod", hist, new, cap=50.0),
        # several documents packed into one sequence, no cache yet, with a distance bias
        _chunk("packed_documents_alibi", "mod", "0", "8192", hq=16, hkv=4, docs=9, alibi=True, paged=False),
        # four drafted tokens for each sequence of a batch, checked over an E4M3 cache
        _chunk("fp8_verify4", "fp8", _spread(17, 24, 1024, 8192), " ".join(["4"] * 24)),
        # chunked prefill of a batch with prefix hits over an E4M3 cache
        _chunk("fp8_batch16", "fp8", hist, new),
        # narrow heads, one KV head, pages that no tile is a multiple of
        _chunk("fp8_ragged_d64", "fp8", "1000 0 37 513", "129 300 1 64", hq=8, hkv=1, d=64, bs=24),
        # a long document resumed: 16k tokens of history in E4M3
        _chunk("fp8_long_history", "fp8", "16384", "512"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "mod", "fp8"])
    hkv, g, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    bs = rng.choice([8, 16, 24, 32, 64, 100, 128, 256])
    common = dict(hq=hkv * g, hkv=hkv, d=d, bs=bs)
    cap = rng.choice([0.0, 0.0, 20.0, 30.0, 50.0])
    alibi, window = rng.random() < 0.4, rng.choice([0, 0, _log(rng, 1, 5000)])
    if op == "decode":
        n = _log(rng, 1, 96)
        top = _log(rng, 1, min(131072, 262144 // n))
        lens = [rng.randint(max(0, top // 8), top) for _ in range(n)]
        return _decode(None, " ".join(map(str, lens)), type=rng.choice(["bf16", "bf16", "f32"]), cap=cap, alibi=alibi,
                       window=window, **common)
    n = _log(rng, 1, 16)
    top = _log(rng, 1, 1024 if n > 4 else 2048)
    new = [rng.randint(max(1, top // 3), top) for _ in range(n)]
    far = rng.choice([0, _log(rng, 1, 16384 // n)])
    hist = [rng.randint(far // 3, far) for _ in range(n)]
    while sum(new) * (max(hist) + max(new)) * hkv * g > 200_000_000:  # below the largest listed cases
        new = [max(1, x // 2) for x in new]
        hist = [x // 2 for x in hist]
    hist, new = " ".join(map(str, hist)), " ".join(map(str, new))
    if op == "fp8":
        return _chunk(None, op, hist, new, **common)
    paged = rng.random() < 0.8
    return _chunk(None, op, hist if paged else " ".join(["0"] * n), new, paged=paged, cap=cap, alibi=alibi, window=window,
                  docs=rng.choice([0, 0, rng.randint(2, 12)]), prefix=rng.choice([0, 0, _log(rng, 1, 2000)]), **common)


# ------------------------------------------------------------------ what a case says (no tensors)

def _ints(text):
    return np.array([int(x) for x in text.split()], dtype=np.int64)


def _lengths(case):
    """New tokens and total keys of each sequence."""
    if case["op"] == "decode":
        keys = _ints(case["lens"])
        return np.minimum(keys, 1), keys
    new, hist = _ints(case["new"]), _ints(case["history"])
    return new, hist + new


def _first_keys(case, position, total):
    """First visible key of each query row of one sequence (window, or the start of its document)."""
    first = np.zeros_like(position)
    if case["window"]:
        first = np.maximum(first, position + 1 - case["window"])
    if case.get("docs"):
        cuts = np.sort(np.random.default_rng(total).integers(0, total, size=case["docs"]))  # starts of documents
        at = np.searchsorted(cuts, position, side="right")
        first = np.maximum(first, np.where(at > 0, cuts[np.maximum(at - 1, 0)], 0))
    return first


def _rows(case):
    """For each sequence: positions of its query rows, their first and one past their last visible key."""
    new, keys = _lengths(case)
    for n, total in zip(new, keys):
        position = np.arange(total - n, total)
        first = _first_keys(case, position, int(total)) if case["op"] != "fp8" else np.zeros_like(position)
        last = np.maximum(position + 1, min(case.get("prefix", 0), total))
        yield position, first, last


def work(case):
    es = {"decode": 4 if case.get("type") == "f32" else 2, "mod": 2, "fp8": 1}[case["op"]]
    qes = 4 if case.get("type") == "f32" else 2
    pairs = keys = rows = pages = 0
    for position, first, last in _rows(case):
        rows += len(position)
        if len(position):
            pairs += int(np.maximum(last - first, 0).sum())
            seen = max(0, int(last.max() - first.min()))
            keys += seen
            pages += -(-seen // case["bs"])
    heads = case["hq"] * case["d"]
    return {"bytes": keys * case["hkv"] * case["d"] * 2 * es + 2 * rows * heads * qes + 4 * pages,
            "flops": 4 * heads * pairs}


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """Everything that the definition takes, on the GPU, from the case and the seed alone."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    new, keys = _lengths(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    dtype = TYPES[case.get("type", "bf16")]
    dev32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    s = {"case": case, "scale": d ** -0.5, "cap": case["cap"], "causal": True, "max_q": int(max(new, default=0)),
         "max_k": int(max(keys, default=0))}
    rows = len(keys) if case["op"] == "decode" else int(new.sum())
    # scores of a few units either side, as trained heads give: the cap bends the larger ones
    s["q"] = (normal(rows, hq, d) * 3).to(dtype)
    if case["op"] != "decode" and not case["paged"]:
        s["k"], s["v"] = normal(int(keys.sum()), hkv, d).to(dtype), normal(int(keys.sum()), hkv, d).to(dtype)
    else:
        need = -(-keys // bs)
        blocks = int(need.sum()) + 3
        order = rng.permutation(blocks)
        tables = np.full((len(keys), max(1, int(need.max()))), -1)
        at = 0
        for i, n in enumerate(need):
            tables[i, :n] = order[at:at + n]
            at += n
        s["tables"] = dev32(tables)
        shape = (blocks, bs, hkv, d)
        if case["op"] == "fp8":
            s["k_scale"], s["v_scale"] = 1.0 / 64, 3.0 / 256
            s["k_cache"], s["v_cache"] = [(normal(*shape) / x).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                                          for x in (s["k_scale"], s["v_scale"])]
        else:
            s["k_cache"], s["v_cache"] = normal(*shape).to(dtype), normal(*shape).to(dtype)
    if case["op"] == "decode":
        s["lens"] = dev32(keys)
    else:
        s["cu_q"], s["cu_k"] = dev32(np.concatenate([[0], np.cumsum(new)])), dev32(np.concatenate([[0], np.cumsum(keys)]))
    s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=DEV) if case["alibi"] else None
    s["first"] = s["prefix"] = None
    if case["window"] or case.get("docs"):
        firsts = [f[0] if case["op"] == "decode" and len(f) else (f if case["op"] != "decode" else 0) for _, f, _ in _rows(case)]
        s["first"] = dev32(np.array(firsts) if case["op"] == "decode" else np.concatenate(firsts))
    if case.get("prefix"):
        s["prefix"] = dev32(np.minimum(case["prefix"], keys))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] != "decode":  # where row j of sequence i lies among the padded rows, for the plain form
        new, _ = _lengths(case)
        s["flat"] = torch.from_numpy(np.concatenate([i * s["max_q"] + np.arange(n) for i, n in enumerate(new)])).to(DEV)
    if own:  # the workspace that a serving program keeps from step to step
        import pagedattention_kv_cache_gb300 as pkv
        n = len(s["cu_q"]) - 1 if case["op"] != "decode" else len(s["lens"])
        if case["op"] == "decode":
            s["workspace"] = pkv.decode_workspace(n, case["hq"], case["d"])
        else:
            s["workspace"] = pkv.prefill_workspace(n, case["hq"], case["hkv"], case["d"], s["max_q"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    return _plain_decode(s) if s["case"]["op"] == "decode" else _plain_chunk(s)


def _own(s):
    import pagedattention_kv_cache_gb300 as pkv
    op = s["case"]["op"]
    if op == "decode":
        return pkv.paged_decode_attn_mod(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                                         softcap=s["cap"], alibi_slopes=s["slopes"], first_keys=s["first"],
                                         workspace=s["workspace"])
    workspace = False if s["workspace"] is None else s["workspace"]
    if op == "fp8":
        return pkv.paged_varlen_prefill_attn_fp8(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["cu_q"], s["cu_k"],
                                                 s["max_q"], s["max_k"], s["scale"], s["k_scale"], s["v_scale"],
                                                 workspace=workspace)
    return pkv.paged_varlen_prefill_attn_mod(s["q"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], s["scale"],
                                             k=s.get("k"), v=s.get("v"), k_cache=s.get("k_cache"),
                                             v_cache=s.get("v_cache"), block_tables=s.get("tables"), softcap=s["cap"],
                                             alibi_slopes=s["slopes"], first_keys=s["first"], prefix_lens=s["prefix"],
                                             workspace=workspace)


def _gathered(s, name):
    """Keys or values of every sequence in logical order, padded: [sequences, max keys, KV heads, d] in float32."""
    t = torch.arange(s["max_k"], device=DEV)
    if name in s:
        rows = s["cu_k"][:-1, None].long() + t
        return s[name][rows.clamp_max(s[name].shape[0] - 1)].float()
    cache = s[name + "_cache"]
    blocks = s["tables"].long().clamp_min(0)[:, t // cache.shape[1]]
    rows = cache[blocks, t % cache.shape[1]]
    if cache.dtype == torch.uint8:
        return rows.view(torch.float8_e4m3fn).float() * s[name + "_scale"]
    return rows.float()


def _attend(s, q, position, seen):
    """q [n, rows, hq, d], position [n, rows], seen [n, rows, keys] -> [n, rows, hq, d], all in float32."""
    k, v = _gathered(s, "k"), _gathered(s, "v")
    n, rows, hq, d = q.shape
    hkv = k.shape[2]
    q = q.float().reshape(n, rows, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    x = (q @ k.permute(0, 2, 3, 1)).reshape(n, hq, rows, -1) * s["scale"]
    if s["cap"] > 0:
        x = torch.tanh(x / s["cap"]) * s["cap"]
    if s["slopes"] is not None:
        t = torch.arange(x.shape[-1], device=DEV)
        x = x - s["slopes"][None, :, None, None] * (position[:, None, :, None] - t).abs()
    x = x.masked_fill(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = x.sum(-1, keepdim=True)
    out = x.reshape(n, hkv, -1, x.shape[-1]) @ v.permute(0, 2, 1, 3)
    out = out.reshape(n, hq, rows, d) / torch.where(total > 0, total, torch.ones_like(total))
    return out.permute(0, 2, 1, 3)


def _plain_decode(s):
    lens = s["lens"].long()[:, None]
    t = torch.arange(s["max_k"], device=DEV)
    seen = t < lens
    if s["first"] is not None:
        seen = seen & (t >= s["first"].long()[:, None])
    return _attend(s, s["q"][:, None], lens - 1, seen[:, None])[:, 0].to(s["q"].dtype)


def _plain_chunk(s):
    new, keys = s["cu_q"].diff().long(), s["cu_k"].diff().long()
    r, t = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    rows = (s["cu_q"][:-1, None].long() + r).clamp_max(s["q"].shape[0] - 1)
    position = (keys - new)[:, None] + r
    last = position + 1
    if s["prefix"] is not None:
        last = torch.maximum(last, s["prefix"].long()[:, None])
    seen = (t < last[..., None]) & (t < keys[:, None, None])
    if s["first"] is not None:
        seen = seen & (t >= s["first"].long()[rows][..., None])
    out = _attend(s, s["q"][rows], position, seen)
    return out.reshape(-1, *out.shape[2:])[s["flat"]].to(s["q"].dtype)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    group = case["hq"] // case["hkv"]
    row0 = key0 = 0
    for i, (position, first, last) in enumerate(_rows(case)):
        n, total = len(position), int(_lengths(case)[1][i])
        if case["op"] == "decode":
            row0 = i
        if n and total:
            t = np.arange(total)
            if "tables" in s:
                table = s["tables"][i].cpu().numpy()
                slot = torch.from_numpy(table[t // case["bs"]] * np.int64(case["bs"]) + t % case["bs"]).to(DEV)
                k, v = [s[x].reshape(-1, case["hkv"], case["d"])[slot] for x in ("k_cache", "v_cache")]
                if case["op"] == "fp8":
                    k, v = k.view(torch.float8_e4m3fn).double() * s["k_scale"], v.view(torch.float8_e4m3fn).double() * s["v_scale"]
            else:
                k, v = s["k"][key0:key0 + total], s["v"][key0:key0 + total]
            lo, hi, at = (torch.from_numpy(np.asarray(a)).to(DEV)[:, None] for a in (first, last, position))
            t = torch.from_numpy(t).to(DEV)
            hidden = (t < lo) | (t >= hi)
            for h in range(case["hq"]):
                score = s["q"][row0:row0 + n, h].double() @ k[:, h // group].double().T * case["d"] ** -0.5
                if case["cap"] > 0:
                    score = case["cap"] * torch.tanh(score / case["cap"])
                if case["alibi"]:
                    score = score - s["slopes"][h].double() * (at - t).abs().double()
                score = score.masked_fill(hidden, -math.inf)
                p = torch.nan_to_num(torch.softmax(score, -1), nan=0.0)
                out[row0:row0 + n, h] = p @ v[:, h // group].double()
        row0, key0 = row0 + n, key0 + total
    return out
