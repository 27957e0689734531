"""Measured calls of the operators of latent attention over a paged cache.

A token's keys and values of all heads come from one shared row: a latent of
512 values and a rotated part of 64.  Per head, W_K and W_V make 128 key and
128 value dims of the latent, and the rotated part joins every head's key:

  latent_append   the new tokens' latents are normalised (RMS, optional),
                  their rotated parts and those of the queries turned to
                  their positions, and the rows written to their slots (bf16,
                  or FP8 latents with one scale for the pool: a value is the
                  stored one times the scale, in both parts)
  latent_gather   cached rows of a ragged batch back as bf16 rows, the input
                  of the products with W_K and W_V
  latent_prefill  the expanded form: queries and keys of 128 + 64 dims and
                  values of 128, a head's own, in ragged chunks; causal with
                  the last query at the last key, or without a mask
  latent_decode   the absorbed form: W_K is in the query (512 + 64 dims), W_V
                  follows the attention, and every head reads the cached rows
                  themselves: scores over 576 dims, values the first 512; one
                  token of each sequence, or a few causal ones (verify)

`own = False` computes them with elementary torch operations in fp32 (fp64
for the rotation's angles); `own = True` makes the framework's calls.
"""
import math
import random

import torch

own = False

BLOCK = 16
LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the next token of a single stream: pure latency
        dict(name="append_t1", op="latent_append", fmt="bf16", tokens=1, heads=20, norm=True, interleaved=True,
             absorbed=True, start=1000, factor=1.0),
        # one decode step of 255 sequences, FP8 latents, scaled positions, queries beside their absorbed parts
        dict(name="append_b255_fp8", op="latent_append", fmt="fp8", tokens=255, heads=24, norm=True,
             interleaved=False, absorbed=True, start=131072, factor=8.0),
        # a prompt of 8191 tokens of 64 heads
        dict(name="append_t8191", op="latent_append", fmt="bf16", tokens=8191, heads=64, norm=True,
             interleaved=True, absorbed=False, start=0, factor=1.0),
        # the cached part of five short prompts, before it is expanded
        dict(name="gather_b5_fp8", op="latent_gather", fmt="fp8", batch=5, keys=1531, spread=3),
        # a long context before its expansion
        dict(name="gather_b4_l32k", op="latent_gather", fmt="bf16", batch=4, keys=32768, spread=0),
        # a short prompt alone
        dict(name="prefill_t97", op="latent_prefill", batch=1, chunk=97, context=0, spread=0, heads=20, causal=True),
        # a ragged batch of prompts and chunks
        dict(name="prefill_ragged8", op="latent_prefill", batch=8, chunk=2048, context=2048, spread=5, heads=32,
             causal=True),
        # the largest: a chunk of 4096 tokens over the 12288 before it and itself
        dict(name="prefill_t4096_ctx12k", op="latent_prefill", batch=1, chunk=4096, context=12288, spread=0,
             heads=32, causal=True),
        # one sequence of 1000 keys: latency
        dict(name="decode_b1_l1000", op="latent_decode", fmt="bf16", batch=1, q_len=1, keys=1000, spread=0, heads=20),
        # the repository's batch of 1K to 32K keys and its 24 heads
        dict(name="decode_b32", op="latent_decode", fmt="bf16", batch=32, q_len=1, keys=32768, spread=11, heads=24),
        # many heads on one row: as much work of the tensor cores as bytes; FP8 latents
        dict(name="decode_b64_h128_fp8", op="latent_decode", fmt="fp8", batch=64, q_len=1, keys=16384, spread=7,
             heads=128),
        # the repository's verify step: 8 new tokens after 65536, 24 heads
        dict(name="verify_q8_b4_ctx64k", op="latent_decode", fmt="bf16", batch=4, q_len=8, keys=65544, spread=0,
             heads=24),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["latent_append", "latent_gather", "latent_prefill", "latent_prefill", "latent_decode",
                     "latent_decode"])
    heads = rng.choice([1, 4, 8, 20, 24, 32, 40, 64, 96, 128])
    fmt = rng.choice(["bf16", "fp8"])
    if op == "latent_append":
        return dict(op=op, fmt=fmt, tokens=_log_int(rng, 1, min(16384, 8191 * 64 // heads)), heads=heads,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.5, absorbed=rng.random() < 0.5,
                    start=_log_int(rng, 1, 1000000), factor=rng.choice([1.0, 4.0, 8.0]))
    batch = _log_int(rng, 1, 64)
    if op == "latent_gather":
        return dict(op=op, fmt=fmt, batch=batch, keys=_log_int(rng, 1, 131072 // batch),
                    spread=rng.randint(1, 1000) if batch > 1 else 0)
    if op == "latent_prefill":
        heads, batch = min(heads, 64), min(batch, 8)
        chunk = _log_int(rng, 2, 4096 if batch == 1 else 2048)
        most = 4096 * 16384 * 32 // (batch * chunk * heads) - chunk
        context = _log_int(rng, 1, max(1, min(12288, most, 65536 // batch))) - 1
        return dict(op=op, batch=batch, chunk=chunk, context=context, spread=rng.randint(1, 1000) if batch > 1 else 0,
                    heads=heads, causal=rng.random() < 0.8)
    q_len = 1 if rng.random() < 0.6 else rng.randint(2, 8)
    most = min(524288, 4 * 65544 * 192 * 2 // (heads * q_len)) // batch
    return dict(op=op, fmt=fmt, batch=batch, q_len=q_len, keys=_log_int(rng, q_len, max(q_len, min(131072, most))),
                spread=rng.randint(1, 1000) if batch > 1 else 0, heads=heads)


def _lengths(case):
    """(new tokens, keys) of every sequence; spread = 0: all the largest."""
    rng = random.Random(case["spread"])
    new, keys = [], []
    for b in range(case["batch"]):
        whole = b == 0 or not case["spread"]
        if case["op"] == "latent_prefill":
            n = case["chunk"] if whole else _log_int(rng, 1, case["chunk"])
            new.append(n)
            keys.append(n + (case["context"] if whole else rng.randint(0, case["context"])))
        else:
            q = case.get("q_len", 1)
            new.append(q)
            keys.append(case["keys"] if whole else _log_int(rng, max(q, case["keys"] // 32), case["keys"]))
    return new, keys


def _row_bytes(fmt):
    return (2 * LATENT if fmt == "bf16" else LATENT) + 2 * ROPE


def work(case):
    if case["op"] == "latent_append":
        t, h = case["tokens"], case["heads"]
        return {"bytes": t * (2 * h * ROPE * 2 + 2 * (LATENT + ROPE) + _row_bytes(case["fmt"]) + 12),
                "flops": t * ((h + 1) * 3 * ROPE + (4 * LATENT if case["norm"] else 0))}
    new, keys = _lengths(case)
    if case["op"] == "latent_gather":
        return {"bytes": sum(keys) * (_row_bytes(case["fmt"]) + 2 * (LATENT + ROPE)), "flops": sum(keys) * LATENT}
    causal = case.get("causal", True)
    pairs = sum(m * n - (m * (m - 1) // 2 if causal else 0) for m, n in zip(new, keys))
    h = case["heads"]
    if case["op"] == "latent_prefill":
        return {"bytes": 2 * sum(new) * h * (NOPE + ROPE + VDIM) + 2 * sum(keys) * (h * (NOPE + VDIM) + ROPE),
                "flops": 2 * pairs * h * (NOPE + ROPE + VDIM)}
    return {"bytes": 2 * sum(new) * h * (2 * LATENT + ROPE) + sum(keys) * _row_bytes(case["fmt"])
            + 4 * sum(-(-k // BLOCK) for k in keys),
            "flops": 2 * pairs * h * (2 * LATENT + ROPE)}


# ----------------------------------------------------------------- inputs

def _pool(fmt, nb, gen):
    """Latents as a norm leaves them, about N(0, 1), and rotated parts a little wider."""
    c = torch.randn((nb, BLOCK, LATENT), device=DEV, generator=gen, dtype=torch.bfloat16)
    r = torch.randn((nb, BLOCK, ROPE), device=DEV, generator=gen, dtype=torch.bfloat16).mul_(1.5)
    if fmt == "bf16":
        return c, r, 1.0
    return c.mul_(8.0).to(torch.float8_e4m3fn).view(torch.uint8), r.mul_(8.0), 0.125


def prepare(case, seed):
    gen = torch.Generator(DEV)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, device=DEV, generator=gen, dtype=torch.bfloat16)
    s = {"case": dict(case)}
    if case["op"] == "latent_append":
        t, h = case["tokens"], case["heads"]
        nb = -(-t // BLOCK) + 3
        # the down-projection's rows: latent and rotated part side by side; the queries' rotated dims are the
        # last of each head's
        down = randn(t, LATENT + ROPE)
        s["latent"], s["rope"] = down[:, :LATENT], down[:, LATENT:]
        s["q"] = randn(t, h, NOPE + ROPE)[..., NOPE:]
        s["positions"] = torch.arange(t, device=DEV, dtype=torch.int32) + case["start"]
        slots = torch.randperm(nb, device=DEV, generator=gen)[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)
        s["slots"] = slots.reshape(-1)[:t].contiguous()
        if t >= 64:   # padded rows of the batch: nothing of theirs is written
            s["slots"][torch.randint(0, t, (t // 64,), device=DEV, generator=gen)] = -1
        i = torch.arange(0, ROPE, 2, device=DEV, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-i / ROPE) / case["factor"]).float()
        s["attn_factor"] = 0.1 * math.log(case["factor"]) + 1.0
        s["norm"] = (1 + 0.2 * torch.randn(LATENT, device=DEV, generator=gen)).bfloat16() if case["norm"] else None
        s["eps"] = 1e-6
        # decode: the turned part goes beside the absorbed one, in the query of latent_decode
        s["q_out"] = None
        if case["absorbed"]:
            s["q_out"] = torch.zeros((t, h, LATENT + ROPE), device=DEV, dtype=torch.bfloat16)[..., LATENT:]
        dt = torch.bfloat16 if case["fmt"] == "bf16" else torch.uint8
        s["pool"] = (torch.zeros((nb, BLOCK, LATENT), device=DEV, dtype=dt),
                     torch.zeros((nb, BLOCK, ROPE), device=DEV, dtype=torch.bfloat16),
                     1.0 if case["fmt"] == "bf16" else 1.0 / 64)
        return s
    new, keys = _lengths(case)
    starts = torch.tensor([0] + keys, device=DEV).cumsum(0).to(torch.int32)
    if case["op"] == "latent_prefill":
        t, n, h = sum(new), sum(keys), case["heads"]
        s["q"] = randn(t, h, NOPE + ROPE).mul_(1.5)
        kv = randn(n, h, NOPE + VDIM)   # one product makes a head's key and value dims
        s["k"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
        s["k_rope"] = randn(n, ROPE).mul_(1.5)
        s["q_starts"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
        s["kv_starts"] = starts
        s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
        return s
    pages = [-(-k // BLOCK) for k in keys]
    nb = sum(pages) + 5
    s["pool"] = _pool(case["fmt"], nb, gen)
    perm = torch.randperm(nb, device=DEV, generator=gen).to(torch.int32)
    s["tables"] = torch.zeros((case["batch"], max(pages)), device=DEV, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        s["tables"][b, :n] = perm[at:at + n]
        at += n
    s["max_keys"] = max(keys)
    if case["op"] == "latent_gather":
        s["starts"], s["rows"] = starts, sum(keys)
        return s
    s["seq_lens"] = torch.tensor(keys, device=DEV, dtype=torch.int32)
    # absorbed queries: scores of a few units, as trained heads have
    s["q"] = randn(case["batch"], case["q_len"], case["heads"], LATENT + ROPE)
    s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
    return s


# ------------------------------------------------------- the plain forms

def _values(s, pages):
    """fp32 rows [..., 576] of pages, as stored times the pool's scale."""
    c, r, g = s["pool"]
    c, r = c[pages], r[pages].float()
    c = c.float() if s["case"]["fmt"] == "bf16" else c.view(torch.float8_e4m3fn).float() * g
    return torch.cat((c, r * g), -1)


def _plain_append(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = ((f(angle) * s["attn_factor"]).float() for f in (torch.cos, torch.sin))

    def turned(x, cos, sin):
        x = x.float()
        a, b = (x[..., 0::2], x[..., 1::2]) if c["interleaved"] else (x[..., :ROPE // 2], x[..., ROPE // 2:])
        a, b = a * cos - b * sin, a * sin + b * cos
        return torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)

    q = turned(s["q"], cos[:, None], sin[:, None]).bfloat16()
    if s["q_out"] is not None:
        s["q_out"].copy_(q)
        q = s["q_out"]
    x = s["latent"].float()
    if s["norm"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["norm"].float()
    r = turned(s["rope"], cos, sin)
    pool, rpool, g = s["pool"]
    if c["fmt"] == "fp8":
        x = (x / g).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        r = r / g
    rows = s["slots"] >= 0
    at = s["slots"][rows]
    pool.view(-1, LATENT)[at] = x.to(pool.dtype)[rows]
    rpool.view(-1, ROPE)[at] = r.bfloat16()[rows]
    return q


def _plain_gather(s):
    starts = s["starts"].long()
    n = starts[1:] - starts[:-1]
    t = torch.arange(s["max_keys"], device=DEV)
    live = t < n[:, None]
    x = _values(s, s["tables"].long()).flatten(1, 2)[:, :s["max_keys"]][live].bfloat16()
    return x[:, :LATENT].contiguous(), x[:, LATENT:].contiguous()


def _softmax_mix(x, v):
    """softmax(x) v over the last axis of x, rows that see nothing 0."""
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _plain_prefill(s):
    new, keys = _lengths(s["case"])
    out, row, key = [], 0, 0
    for m, n in zip(new, keys):
        q = s["q"][row:row + m].float().transpose(0, 1)
        k = s["k"][key:key + n].float().permute(1, 2, 0)
        x = torch.matmul(q[..., :NOPE], k)
        x += torch.matmul(q[..., NOPE:], s["k_rope"][key:key + n].float().T)
        x *= s["scale"]
        if s["case"]["causal"]:
            t = torch.arange(n, device=DEV)
            x = x.masked_fill(t > t[n - m:, None], -math.inf)
        out.append(_softmax_mix(x, s["v"][key:key + n].float().transpose(0, 1)).transpose(0, 1).bfloat16())
        row, key = row + m, key + n
    return torch.cat(out)


def _plain_decode(s):
    b, q_len, h, _ = s["q"].shape
    kv = _values(s, s["tables"].long()).flatten(1, 2)[:, :s["max_keys"]]
    x = torch.matmul(s["q"].float().flatten(1, 2), kv.transpose(1, 2)).view(b, q_len, h, -1)
    x *= s["scale"]
    n = s["seq_lens"].long()[:, None] - q_len + 1 + torch.arange(q_len, device=DEV)   # keys a token sees
    t = torch.arange(kv.shape[1], device=DEV)
    x = x.masked_fill((t >= n[..., None])[:, :, None], -math.inf).flatten(1, 2)
    return _softmax_mix(x, kv[..., :LATENT]).view(b, q_len, h, LATENT).bfloat16()


# ------------------------------------------------------------------- run

def run(s):
    c = s["case"]
    if own:
        from paged_kv_decode_07_gb300 import pa
    if c["op"] == "latent_prefill":
        if not own:
            return {"out": _plain_prefill(s)}
        out, s["workspace"] = pa.latent_prefill(s["q"], s["k"], s["k_rope"], s["v"], s["q_starts"], s["kv_starts"],
                                                s["scale"], causal=c["causal"], workspace=s.get("workspace"))
        return {"out": out}
    if own:
        pool = pa.LatentCache(c["fmt"], *s["pool"])
    if c["op"] == "latent_append":
        if own:
            q = pa.latent_append(pool, s["latent"], s["rope"], s["positions"], s["slots"], s["inv_freq"], q=s["q"],
                                 q_out=s["q_out"], interleaved=c["interleaved"], attn_factor=s["attn_factor"],
                                 norm=s["norm"], eps=s["eps"])
        else:
            q = _plain_append(s)
        latent, rope, _ = s["pool"]
        if c["fmt"] == "fp8":   # the values that the codes stand for (per-tensor scale apart)
            latent = latent.view(torch.float8_e4m3fn)
        return {"q": q, "latent": latent, "rope": rope}
    if c["op"] == "latent_gather":
        latent, rope = pa.latent_gather(pool, s["tables"], s["starts"], s["rows"]) if own else _plain_gather(s)
        return {"latent": latent, "rope": rope}
    if not own:
        return {"out": _plain_decode(s)}
    # the workspace is kept from the first call on, as a serving program keeps it
    out, s["workspace"] = pa.latent_decode(pool, s["q"], s["tables"], s["seq_lens"], s["scale"],
                                           max_seq_len=s["max_keys"], workspace=s.get("workspace"))
    return {"out": out}


# ------------------------------------------------------------ in 64 bits

def _exact_pool(s, pages):
    """fp64 (latents [n, 512], rotated parts [n, 64]) of one sequence's pages."""
    c, r, g = s["pool"]
    c = c.index_select(0, pages.long()).reshape(-1, LATENT)
    c = c.double() if s["case"]["fmt"] == "bf16" else c.view(torch.float8_e4m3fn).double() * g
    return c, r.index_select(0, pages.long()).reshape(-1, ROPE).double() * g


def _exact_append(s):
    c = s["case"]
    half = ROPE // 2
    a = torch.outer(s["positions"].double(), s["inv_freq"].double())
    z = torch.polar(torch.full_like(a, s["attn_factor"]), a)

    def turned(x, z):
        pair = x.double().unflatten(-1, (half, 2) if c["interleaved"] else (2, half))
        if not c["interleaved"]:
            pair = pair.transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        return (y if c["interleaved"] else y.transpose(-1, -2)).flatten(-2)

    g = s["pool"][2]
    x = s["latent"].double()
    if s["norm"] is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / LATENT + s["eps"]).sqrt() * s["norm"].double()
    x, r = x / g, turned(s["rope"], z) / g
    if c["fmt"] == "fp8":
        x = x.clamp(-448, 448)
    got = {"q": turned(s["q"], z[:, None])}
    kept = s["slots"] >= 0
    for name, y, like in (("latent", x, s["pool"][0]), ("rope", r, s["pool"][1])):
        d = torch.zeros(like.shape, dtype=torch.float64, device=DEV)
        d.view(-1, d.shape[-1])[s["slots"][kept]] = y[kept]
        got[name] = d
    return got


def _exact_attention(q, k, v, scale, hidden):
    x = q @ k.T * scale
    if hidden is not None:
        x[hidden] = -math.inf
    x = (x - x.amax(1, keepdim=True).clamp(min=-1e300)).exp_()
    return x @ v / x.sum(1, keepdim=True).clamp(min=1e-300)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "latent_append":
        return _exact_append(s)
    new, keys = _lengths(case)
    if case["op"] == "latent_gather":
        rows = [_exact_pool(s, s["tables"][b, :-(-n // BLOCK)]) for b, n in enumerate(keys)]
        return {"latent": torch.cat([c[:n] for (c, _), n in zip(rows, keys)]),
                "rope": torch.cat([r[:n] for (_, r), n in zip(rows, keys)])}
    h = case["heads"]
    if case["op"] == "latent_prefill":
        out = torch.empty((sum(new), h, VDIM), dtype=torch.float64, device=DEV)
        row = key = 0
        for m, n in zip(new, keys):
            hidden = None
            if case["causal"]:
                hidden = torch.arange(n, device=DEV)[None] - torch.arange(n - m, n, device=DEV)[:, None] > 0
            k_rope = s["k_rope"][key:key + n].double()
            for i in range(h):
                k = torch.cat((s["k"][key:key + n, i].double(), k_rope), 1)
                out[row:row + m, i] = _exact_attention(s["q"][row:row + m, i].double(), k,
                                                       s["v"][key:key + n, i].double(), s["scale"], hidden)
            row, key = row + m, key + n
        return {"out": out}
    out = torch.empty(s["q"].shape[:3] + (LATENT,), dtype=torch.float64, device=DEV)
    m = case["q_len"]
    for b, n in enumerate(keys):
        c, r = _exact_pool(s, s["tables"][b, :-(-n // BLOCK)])
        c, k = c[:n], torch.cat((c, r), 1)[:n]
        for i in range(m):
            seen = max(n - m + 1 + i, 0)
            out[b, i] = _exact_attention(s["q"][b, i].double(), k[:seen], c[:seen], s["scale"], None) if seen else 0.0
    return {"out": out}
