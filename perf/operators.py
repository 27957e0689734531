"""Measured calls of the cache-writing and score-modified attention operators.

Three operators of one serving path:

  rope_append    the queries and keys of new tokens are normalised per head
                 (optional), rotated to their positions (half or interleaved
                 pairs, the whole head or its first part) and the keys and
                 values quantised into their slots of the paged cache;
  prefill        a ragged batch of prompt chunks attends over that cache,
                 causally, with the score options below;
  decode_scored  one new token per sequence does.

Score options, for the query at position p and the key at position t:
  s = softmax_scale * <q, k>;   softcap c > 0: s <- c * tanh(s / c);
  slopes: s <- s - slope[head] * |p - t|;
  visible: t < seq_len, first_key <= t, t > p - window, and
           t <= p or t < prefix_len.

`own = False` computes them with elementary torch operations in fp32 (fp64
for the rotation's angles); `own = True` makes the framework's calls.
"""
import math
import random

import torch

own = False

BLOCK = 16
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the next token of a single stream: pure latency
        dict(name="rope_t1", op="rope_append", fmt="bf16", tokens=1, hkv=2, group=4, dim=128, rot=128,
             interleaved=False, norm=True, start=1000, factor=1.0),
        # one decode step of 255 sequences, FP8 cache, a quarter of the head rotated, scaled positions
        dict(name="rope_b255_fp8", op="rope_append", fmt="fp8", tokens=255, hkv=4, group=6, dim=256,
             rot=64, interleaved=True, norm=False, start=131072, factor=8.0),
        # a prompt of 8191 tokens with per-head norms, the repository's 24 / 4 heads of 256
        dict(name="rope_t8191", op="rope_append", fmt="bf16", tokens=8191, hkv=4, group=6, dim=256,
             rot=256, interleaved=False, norm=True, start=0, factor=1.0),
        # the largest write: 32768 tokens at far positions into an FP8 cache
        dict(name="rope_t32768_fp8", op="rope_append", fmt="fp8", tokens=32768, hkv=4, group=6, dim=256,
             rot=128, interleaved=False, norm=True, start=1000000, factor=4.0),
        # a short prompt alone
        dict(name="prefill_t97", op="prefill", fmt="bf16", batch=1, chunk=97, context=0, spread=0, hkv=2,
             group=4, dim=128, softcap=30.0, slopes=False, window=0, doc=0, prefix=0),
        # a ragged batch of prompts and chunks, capped scores in a sliding window
        dict(name="prefill_ragged8", op="prefill", fmt="bf16", batch=8, chunk=2048, context=6144, spread=5,
             hkv=4, group=6, dim=128, softcap=50.0, slopes=False, window=4096, doc=0, prefix=0),
        # packed documents with a bidirectional prefix and a distance bias, over an int8 cache
        dict(name="prefill_docs_int8", op="prefill", fmt="int8", batch=4, chunk=1531, context=517, spread=3,
             hkv=4, group=6, dim=256, softcap=0.0, slopes=True, window=0, doc=700, prefix=100),
        # the largest: a chunk of 4096 tokens of a 32K prompt, capped scores
        dict(name="prefill_t4096_ctx28k", op="prefill", fmt="bf16", batch=1, chunk=4096, context=28672,
             spread=0, hkv=4, group=6, dim=256, softcap=50.0, slopes=False, window=0, doc=0, prefix=0),
        # one sequence of 1000 keys, capped scores: latency
        dict(name="decode_b1_l1000", op="decode_scored", fmt="bf16", batch=1, keys=1000, spread=0, hkv=2,
             group=4, dim=128, softcap=30.0, slopes=False, window=0, doc=0),
        # the repository's int8 batch (1K to 32K keys) with capped scores and a distance bias
        dict(name="decode_b32_int8", op="decode_scored", fmt="int8", batch=32, keys=32768, spread=11, hkv=4,
             group=6, dim=256, softcap=50.0, slopes=True, window=0, doc=0),
        # a sliding-window layer of a long-context batch, FP8 cache
        dict(name="decode_b64_window_fp8", op="decode_scored", fmt="fp8", batch=64, keys=65536, spread=7,
             hkv=4, group=6, dim=256, softcap=50.0, slopes=False, window=4096, doc=0),
        # the repository's NVFP4 case: four sequences of 262144 keys, capped scores
        dict(name="decode_b4_l262k_nvfp4", op="decode_scored", fmt="nvfp4", batch=4, keys=262144, spread=0,
             hkv=4, group=6, dim=256, softcap=50.0, slopes=False, window=0, doc=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_append", "prefill", "decode_scored"])
    hkv, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 6, 8]), rng.choice([128, 256])
    if op == "rope_append":
        most = 32768 * 32 * 256 // (hkv * (group + 2) * dim)
        return dict(op=op, fmt=rng.choice(["bf16", "fp8"]), tokens=_log_int(rng, 1, min(most, 32768)), hkv=hkv,
                    group=group, dim=dim, rot=32 * rng.randint(1, dim // 32), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.5, start=_log_int(rng, 1, 1000000),
                    factor=rng.choice([1.0, 4.0, 8.0]))
    fmt = rng.choice(["bf16", "int8", "fp8", "nvfp4"])
    softcap = rng.choice([0.0, 20.0, 30.0, 50.0])
    slopes = rng.random() < 0.4
    window = _log_int(rng, 64, 8192) if rng.random() < 0.4 else 0
    if op == "prefill":
        batch = rng.choice([1, 2, 3, 5, 8])
        chunk = _log_int(rng, 2, 4096 if batch == 1 else 2048)
        most = 4096 * 32768 * 24 * 256 // (batch * chunk * hkv * group * dim) - chunk
        context = _log_int(rng, 1, max(1, min(28672, most, 32768 * 8 // batch))) - 1
        return dict(op=op, fmt=fmt, batch=batch, chunk=chunk, context=context,
                    spread=rng.randint(1, 1000) if batch > 1 else 0, hkv=hkv, group=group, dim=dim,
                    softcap=softcap, slopes=slopes, window=window,
                    doc=_log_int(rng, 50, 5000) if rng.random() < 0.3 else 0,
                    prefix=_log_int(rng, 8, 500) if rng.random() < 0.3 else 0)
    batch = _log_int(rng, 1, 128)
    most = 4 * 262144 * 4 * 256 // (batch * hkv * dim)
    return dict(op=op, fmt=fmt, batch=batch, keys=_log_int(rng, 1, max(1, min(262144, most))),
                spread=rng.randint(1, 1000) if batch > 1 else 0, hkv=hkv, group=group, dim=dim,
                softcap=softcap, slopes=slopes, window=window,
                doc=_log_int(rng, 50, 5000) if rng.random() < 0.2 else 0)


def _lengths(case):
    """(new tokens, keys in the cache) of every sequence; spread = 0: all the largest."""
    rng = random.Random(case["spread"])
    new, keys = [], []
    for b in range(case["batch"]):
        whole = b == 0 or not case["spread"]
        if case["op"] == "prefill":
            n = case["chunk"] if whole else _log_int(rng, 1, case["chunk"])
            c = case["context"] if whole else rng.randint(0, case["context"])
            new.append(n)
            keys.append(n + c)
        else:
            new.append(1)
            keys.append(case["keys"] if whole else _log_int(rng, max(1, case["keys"] // 32), case["keys"]))
    return new, keys


def _visible(case):
    """Query-key pairs that the masks leave, and the keys that some query sees."""
    pairs = seen = 0
    for n, k in zip(*_lengths(case)):
        p = torch.arange(k - n, k)
        lo, hi = torch.zeros_like(p), p + 1
        if case["window"]:
            lo = (p - case["window"] + 1).clamp(min=0)
        if case["doc"]:
            lo = torch.maximum(lo, p // case["doc"] * case["doc"])
        if case.get("prefix"):
            hi = torch.maximum(hi, torch.tensor(min(case["prefix"], k)))
        live = (hi - lo).clamp(min=0)
        pairs += int(live.sum())
        seen += int(hi.max() - lo.min())
    return pairs, seen


def _code_bytes(fmt, dim):
    """Bytes of one cached row of `dim` values with its scales."""
    return {"bf16": 2 * dim, "int8": dim + 2, "fp8": dim, "nvfp4": dim // 2 + dim // 16}[fmt]


def work(case):
    hq, hkv, dim = case["hkv"] * case["group"], case["hkv"], case["dim"]
    if case["op"] == "rope_append":
        t = case["tokens"]
        return {"bytes": t * (2 * hq * dim * 2 + 2 * hkv * (2 * dim + _code_bytes(case["fmt"], dim)) + 12),
                "flops": t * (hq + hkv) * (3 * case["rot"] + (4 * dim if case["norm"] else 0))}
    new, keys = _lengths(case)
    pairs, seen = _visible(case)
    return {"bytes": 2 * sum(new) * hq * dim * 2 + 2 * seen * hkv * _code_bytes(case["fmt"], dim)
            + 4 * sum(-(-k // BLOCK) for k in keys),
            "flops": 4 * pairs * hq * dim}


# ----------------------------------------------------------------- inputs

def _pool(fmt, nb, hkv, dim, gen):
    """Codes (and scales) of K and V with the values' usual spread, about N(0, 1)."""
    out = {}
    for x in ("k", "v"):
        shape = (nb, hkv, BLOCK, dim)
        out[x + "_scale"] = None
        if fmt == "bf16":
            out[x] = torch.randn(shape, device=DEV, generator=gen, dtype=torch.bfloat16)
        elif fmt == "fp8":
            out[x] = torch.randn(shape, device=DEV, generator=gen, dtype=torch.bfloat16).mul_(8.0).to(
                torch.float8_e4m3fn).view(torch.uint8)
        elif fmt == "int8":
            out[x] = torch.randn(shape, device=DEV, generator=gen, dtype=torch.bfloat16).mul_(40.0).clamp_(
                -127, 127).to(torch.int8)
            out[x + "_scale"] = (torch.rand(shape[:3], device=DEV, generator=gen) * 0.02 + 0.015).half()
        else:
            out[x] = torch.randint(0, 256, (nb, hkv, BLOCK, dim // 2), device=DEV, generator=gen,
                                   dtype=torch.uint8)
            out[x + "_scale"] = (torch.rand((nb, hkv, BLOCK, dim // 16), device=DEV, generator=gen) * 4 + 2).to(
                torch.float8_e4m3fn).view(torch.uint8)
    # per-tensor scales (NVFP4, FP8); the other formats do not use them
    out["global"] = {"fp8": 0.125, "nvfp4": 0.0625}.get(fmt, 1.0)
    return out


def prepare(case, seed):
    gen = torch.Generator(DEV)
    gen.manual_seed(seed)
    hkv, dim, hq = case["hkv"], case["dim"], case["hkv"] * case["group"]
    s = {"case": dict(case)}
    if case["op"] == "rope_append":
        t = case["tokens"]
        nb = -(-t // BLOCK) + 3
        # one row of the fused projection per token: the q, k and v heads side by side
        qkv = torch.randn((t, hq + 2 * hkv, dim), device=DEV, generator=gen, dtype=torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["positions"] = (torch.arange(t, device=DEV, dtype=torch.int32) + case["start"])
        slots = torch.randperm(nb, device=DEV, generator=gen)[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)
        s["slots"] = slots.reshape(-1)[:t].contiguous()
        if t >= 64:   # padded rows of the batch: nothing of theirs is written
            s["slots"][torch.randint(0, t, (t // 64,), device=DEV, generator=gen)] = -1
        i = torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-i / case["rot"]) / case["factor"]).float()
        s["attn_factor"] = 0.1 * math.log(case["factor"]) + 1.0
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"], s["k_norm"] = (1 + 0.2 * torch.randn((2, dim), device=DEV, generator=gen)).to(
                torch.bfloat16).unbind(0)
        s["eps"] = 1e-6
        dt = torch.bfloat16 if case["fmt"] == "bf16" else torch.uint8
        s["pool"] = {"k": torch.zeros((nb, hkv, BLOCK, dim), device=DEV, dtype=dt),
                     "v": torch.zeros((nb, hkv, BLOCK, dim), device=DEV, dtype=dt),
                     "k_scale": None, "v_scale": None, "global": 1.0 / 64 if case["fmt"] == "fp8" else 1.0}
        return s
    new, keys = _lengths(case)
    pages = [-(-k // BLOCK) for k in keys]
    nb = sum(pages) + 5
    s["pool"] = _pool(case["fmt"], nb, hkv, dim, gen)
    perm = torch.randperm(nb, device=DEV, generator=gen).to(torch.int32)
    s["tables"] = torch.zeros((case["batch"], max(pages)), device=DEV, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        s["tables"][b, :n] = perm[at:at + n]
        at += n
    s["seq_lens"] = torch.tensor(keys, device=DEV, dtype=torch.int32)
    s["max_keys"], s["max_new"] = max(keys), max(new)
    # queries a little wider than unit normal: scores of a few units, as trained heads have
    s["q"] = torch.randn((sum(new), hq, dim), device=DEV, generator=gen, dtype=torch.bfloat16).mul_(2.0)
    s["scale"] = 1.0 / math.sqrt(dim)
    s["slopes"] = s["first_key"] = s["prefix"] = None
    if case["slopes"]:
        s["slopes"] = torch.rand((hq,), device=DEV, generator=gen) * 0.05
    if case["op"] == "prefill":
        s["q_starts"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
        p = torch.cat([torch.arange(k - n, k) for n, k in zip(new, keys)])
        if case["prefix"]:
            s["prefix"] = torch.full((case["batch"],), case["prefix"], device=DEV, dtype=torch.int32)
    else:
        s["q"] = s["q"][:, None]   # [B, 1, Hq, D]
        p = torch.tensor(keys) - 1
    if case["doc"]:
        s["first_key"] = (p // case["doc"] * case["doc"]).to(torch.int32).to(DEV)
    return s


# ------------------------------------------------------- the plain forms

def _values(pool, x, fmt, tables):
    """Rows of `tables`' pages as fp32 [B, Hkv, keys, D], dequantised."""
    c = pool[x][tables.long()]                       # [B, pages, Hkv, 16, ...]
    if fmt == "bf16":
        v = c.float()
    elif fmt == "fp8":
        v = c.view(torch.float8_e4m3fn).float() * pool["global"]
    elif fmt == "int8":
        v = c.float() * pool[x + "_scale"][tables.long()].float()[..., None]
    else:
        lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=c.device)
        v = lut[torch.stack((c & 15, c >> 4), -1).long()].flatten(-2)
        sc = pool[x + "_scale"][tables.long()].view(torch.float8_e4m3fn).float()
        v = v * sc.repeat_interleave(16, -1) * pool["global"]
    return v.transpose(1, 2).flatten(2, 3)


def _plain_rope(s):
    c = s["case"]
    rot, f = c["rot"], c["fmt"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = ((g(angle) * s["attn_factor"]).float()[:, None] for g in (torch.cos, torch.sin))

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        head, tail = x[..., :rot], x[..., rot:]
        a, b = (head[..., 0::2], head[..., 1::2]) if c["interleaved"] else (head[..., :rot // 2], head[..., rot // 2:])
        a, b = a * cos - b * sin, a * sin + b * cos
        head = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((head, tail), -1)

    q = turned(s["q"], s["q_norm"]).bfloat16()
    rows = s["slots"] >= 0
    at = s["slots"][rows]
    for x, new in (("k", turned(s["k"], s["k_norm"])), ("v", s["v"].float())):
        if f == "bf16":
            code = new.bfloat16()
        else:
            code = (new / s["pool"]["global"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["pool"][x][at // BLOCK, :, at % BLOCK] = code[rows]
    return q


def _plain_attention(s):
    c = s["case"]
    hkv, dim = c["hkv"], c["dim"]
    batch = s["tables"].shape[0]
    k, v = (_values(s["pool"], x, c["fmt"], s["tables"]) for x in ("k", "v"))
    n = s["seq_lens"].long()
    if c["op"] == "prefill":   # the ragged rows, padded to the longest chunk
        starts = s["q_starts"].long()
        new = starts[1:] - starts[:-1]
        i = torch.arange(s["max_new"], device=DEV)
        live = i < new[:, None]
        row = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
        pos = n[:, None] - new[:, None] + i
        q, first = s["q"][row], s["first_key"][row].long() if s["first_key"] is not None else None
    else:
        live, pos, q = None, n[:, None] - 1, s["q"]
        first = s["first_key"].long()[:, None] if s["first_key"] is not None else None
    nq = q.shape[1]
    q = q.float().view(batch, nq, hkv, c["group"], dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.transpose(-1, -2)).view(batch, hkv, c["group"], nq, -1)
    x *= s["scale"]
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    t = torch.arange(k.shape[2], device=DEV)
    if s["slopes"] is not None:
        far = (pos[:, :, None] - t).abs().float()
        x -= s["slopes"].view(hkv, c["group"], 1, 1) * far[:, None, None]
    seen = t <= pos[:, :, None]
    if s["prefix"] is not None:
        seen = seen | (t < s["prefix"].long()[:, None, None])
    seen = seen & (t < n[:, None, None])
    if c["window"]:
        seen = seen & (t > pos[:, :, None] - c["window"])
    if first is not None:
        seen = seen & (t >= first[:, :, None])
    seen = seen[:, None, None]
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).view(batch, hkv, c["group"], nq, dim)
    o = o / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3).bfloat16()
    return o[live] if live is not None else o


# ------------------------------------------------------------------- run

def _cache(pa, s):
    p = s["pool"]
    return pa.KvCache(s["case"]["fmt"], p["k"], p["v"], p["k_scale"], p["v_scale"], p["global"], p["global"])


def run(s):
    c = s["case"]
    if own:
        from paged_kv_decode_07_gb300 import pa
    if c["op"] == "rope_append":
        if own:
            q = pa.rope_append(_cache(pa, s), s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                               interleaved=c["interleaved"], attn_factor=s["attn_factor"], q_norm=s["q_norm"],
                               k_norm=s["k_norm"], eps=s["eps"])
        else:
            q = _plain_rope(s)
        k, v = s["pool"]["k"], s["pool"]["v"]
        if c["fmt"] == "fp8":   # the values that the codes stand for (per-tensor scale apart)
            k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        return {"q": q, "k": k, "v": v}
    if not own:
        return {"out": _plain_attention(s)}
    score = pa.Score(softcap=c["softcap"], slopes=s["slopes"], window=c["window"], first_key=s["first_key"],
                     prefix_lens=s["prefix"])
    ws = s.get("workspace")   # kept from the first call on, as a serving program keeps it
    if c["op"] == "prefill":
        out, s["workspace"] = pa.prefill(_cache(pa, s), s["q"], s["q_starts"], s["tables"], s["seq_lens"], s["scale"],
                                         score=score, max_seq_len=s["max_keys"], workspace=ws)
    else:
        out, s["workspace"] = pa.decode_scored(_cache(pa, s), s["q"], s["tables"], s["seq_lens"], s["scale"],
                                               score=score, max_seq_len=s["max_keys"], workspace=ws)
    return {"out": out}


# ------------------------------------------------------------ in 64 bits

def _exact_rows(s, x, pages):
    """fp64 [Hkv, keys, D] of one sequence's pages, from the formats' definitions."""
    fmt, pool = s["case"]["fmt"], s["pool"]
    c = pool[x].index_select(0, pages.long())
    if fmt == "nvfp4":
        def e2m1(n):
            n = n.to(torch.int64)
            e, m = (n >> 1) & 3, (n & 1).double()
            mag = torch.where(e == 0, m * 0.5, (1 + m / 2) * torch.exp2((e - 1).double()))
            return torch.where(n >= 8, -mag, mag)
        d = torch.empty(c.shape[:3] + (2 * c.shape[3],), dtype=torch.float64, device=c.device)
        d[..., 0::2], d[..., 1::2] = e2m1(c & 15), e2m1(c >> 4)
        sc = pool[x + "_scale"].index_select(0, pages.long()).view(torch.float8_e4m3fn).double()
        d = (d.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2) * pool["global"]
    elif fmt == "int8":
        d = c.double() * pool[x + "_scale"].index_select(0, pages.long()).double().unsqueeze(-1)
    elif fmt == "fp8":
        d = c.view(torch.float8_e4m3fn).double() * pool["global"]
    else:
        d = c.double()
    return d.permute(1, 0, 2, 3).reshape(d.shape[1], -1, d.shape[3])


def _exact_attention(s):
    c = s["case"]
    new, keys = _lengths(c)
    q = s["q"].reshape(-1, c["hkv"], c["group"], c["dim"])
    out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    row = 0
    for b, (m, n) in enumerate(zip(new, keys)):
        pages = s["tables"][b, :-(-n // BLOCK)]
        k, v = (_exact_rows(s, x, pages)[:, :n] for x in ("k", "v"))
        p = torch.arange(n - m, n, device=DEV)[:, None]
        t = torch.arange(n, device=DEV)[None]
        hidden = t > p
        if c.get("prefix"):
            hidden &= t >= c["prefix"]
        if c["window"]:
            hidden |= p - t >= c["window"]
        if c["doc"]:
            hidden |= t < p // c["doc"] * c["doc"]
        for h in range(c["hkv"]):
            for g in range(c["group"]):
                x = q[row:row + m, h, g].double() @ k[h].T * s["scale"]
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][h * c["group"] + g].double() * (p - t).abs()
                x[hidden.expand_as(x)] = -math.inf
                x = (x - x.amax(1, keepdim=True).clamp(min=-1e300)).exp_()
                out[row:row + m, h, g] = x @ v[h] / x.sum(1, keepdim=True).clamp(min=1e-300)
        row += m
    return {"out": out.reshape(s["q"].shape)}


def _exact_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    z = torch.polar(torch.full_like(s["positions"], s["attn_factor"], dtype=torch.float64)[:, None].expand(-1, half).contiguous(),
                    torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + s["eps"]).sqrt() * w.double()
        pair = x[..., :c["rot"]].unflatten(-1, (half, 2) if c["interleaved"] else (2, half))
        if not c["interleaved"]:
            pair = pair.transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        if not c["interleaved"]:
            y = y.transpose(-1, -2)
        return torch.cat((y.flatten(-2), x[..., c["rot"]:]), -1)

    got = {"q": turned(s["q"], s["q_norm"])}
    at = s["slots"].clamp(min=0)
    kept = s["slots"] >= 0
    for x, y in (("k", turned(s["k"], s["k_norm"])), ("v", s["v"].double())):
        d = torch.zeros(s["pool"][x].shape, dtype=torch.float64, device=DEV)
        y = (y / s["pool"]["global"]).clamp(-448, 448) if c["fmt"] == "fp8" else y
        d[at[kept] // BLOCK, :, at[kept] % BLOCK] = y[kept]
        got[x] = d
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope_append" else _exact_attention(s)
