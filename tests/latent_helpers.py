"""Plain 64-bit forms of latent attention and the bounds that the kernels'
outputs are held to.

Bound, per output element, as in score_helpers.  With p the exact softmax
weights and A = sum p |v|:
  * each weight is rounded once before it meets a value: relative eps_p (bf16
    2^-8, fp16 2^-11), so A * eps_p; an fp16 weight below 2^-14 is off by up to
    2^-25 instead, and weights are relative to a maximum that the row's largest
    score reaches or passes, never misses: + 2^-25 * sum |stored value| of the
    keys seen, over a sum of at least 1;
  * a score off by d changes the output by at most 2 d A.  A score's products
    are added in at most 36 matrix steps (576 dims), each off by 2^-22 of its
    sum at most: 36 * 2^-22 < 2^-16 of S, the largest sum |q k| * scale of the
    row; FP8 caches: queries and rotated parts below 2^-14 are held in fp16 to
    2^-25, + 2^-25 * scale * (sum |q| + sum |k|); + 2^-20 for the exponential;
  * the output is rounded once: 2^-8 |o| (bf16) or 2^-23 |o| (fp32).
"""
import math

import torch

DEV = "cuda"
EPS = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -11}
BF16, I32 = torch.bfloat16, torch.int32


def pool(fmt, nb, seed=0):
    """(latent, rope, scale) with values about N(0, 1)."""
    g = torch.Generator(DEV).manual_seed(seed)
    c = torch.randn((nb, 16, 512), device=DEV, generator=g)
    r = torch.randn((nb, 16, 64), device=DEV, generator=g)
    if fmt == "bf16":
        return c.bfloat16(), r.bfloat16(), 1.0
    return (c * 8).to(torch.float8_e4m3fn).view(torch.uint8), (r * 8).bfloat16(), 0.125


def values(fmt, latent, rope, scale):
    """fp64 stored rows [NB, 16, 576] (before the scale) and the scale."""
    c = latent.double() if fmt == "bf16" else latent.view(torch.float8_e4m3fn).double()
    return torch.cat((c, rope.double()), -1), scale


def poison(fmt, latent, rope, used):
    """NaN in every slot that `used` (bool [NB, 16]) leaves."""
    if fmt == "bf16":
        latent[~used] = math.nan
    else:
        latent[~used] = 0x7F
    rope[~used] = math.nan


def mix(x, see, v, vabs, d, eps_p, out_eps, stored):
    """softmax of x (masked by see) times v -> (out, lse, bound)."""
    x = torch.where(see, x, -math.inf)
    top = x.amax(1, keepdim=True).clamp(min=-1e300)
    p = torch.where(see, torch.exp(x - top), 0.0)
    s = p.sum(1, keepdim=True)
    w = p / s.clamp(min=1e-300)
    o, a = w @ v, w @ vabs
    bound = (eps_p + 2 * d) * a + out_eps * o.abs() + 1e-30
    if eps_p == EPS["fp8"]:
        bound = bound + 2.0 ** -25 * (see.double() @ stored) / s.clamp(min=1.0)
    lse = torch.where(s > 0, top + torch.log(s.clamp(min=1e-300)), -math.inf).squeeze(1)
    return o, lse, bound


def decode_reference(fmt, kv, q, lens, tables, scale, out_eps=2.0 ** -23, bad=()):
    """q [B, Q, H, 576]; bad: page ids to skip -> (out, lse, bound) fp64."""
    rows, g = kv
    B, Q, H, _ = q.shape
    out = torch.zeros((B, Q, H, 512), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        ids = tables[b, :-(-n // 16)].long()
        ok = (ids >= 0) & (ids < rows.shape[0])
        k = rows[ids.clamp(0, rows.shape[0] - 1)]
        k = torch.where(ok[:, None, None], k, 0.0).reshape(-1, 576)[:n]
        live = ok.repeat_interleave(16)[:n]
        for i in range(Q):
            see = live & (torch.arange(n, device=q.device) < n - Q + 1 + i)
            qq = q[b, i].double()
            kk = torch.where(see[:, None], k, 0.0)    # hidden keys may hold anything
            x = qq @ kk.T * (scale * g)
            d = 2.0 ** -16 * (qq.abs() @ kk.abs().T * abs(scale * g))
            if fmt == "fp8":
                d = d + 2.0 ** -25 * abs(scale * g) * (qq.abs().sum(1, keepdim=True) + kk.abs().sum(1)[None])
            d = d.amax(1, keepdim=True) + 2.0 ** -20
            c = kk[:, :512]
            o, l, e = mix(x, see.expand(H, n), c * g, c.abs() * g, d, EPS[fmt], out_eps, c.abs() * g)
            out[b, i], lse[b, i], bound[b, i] = o, l, e
    return out, lse, bound


def prefill_reference(q, kn, kr, v, new, keys, scale, causal=True, out_eps=2.0 ** -23):
    """The expanded form over packed rows -> (out [T, H, 128], lse, bound)."""
    T, H, _ = q.shape
    out = torch.zeros((T, H, 128), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    row = key = 0
    for m, n in zip(new, keys):
        if m and n:
            see = torch.ones((m, n), dtype=torch.bool, device=q.device)
            if causal:
                see = torch.arange(n, device=q.device)[None] <= torch.arange(n - m, n, device=q.device)[:, None]
            for h in range(H):
                k = torch.cat((kn[key:key + n, h].double(), kr[key:key + n].double()), 1)
                vv = v[key:key + n, h].double()
                qq = q[row:row + m, h].double()
                x = qq @ k.T * scale
                d = 2.0 ** -16 * (qq.abs() @ k.abs().T * abs(scale))
                d = torch.where(see, d, 0.0).amax(1, keepdim=True) + 2.0 ** -20
                o, l, e = mix(x, see, vv, vv.abs(), d, EPS["bf16"], out_eps, vv.abs())
                out[row:row + m, h], lse[row:row + m, h], bound[row:row + m, h] = o, l, e
        row, key = row + m, key + n
    return out, lse, bound


def tables_for(lens, extra=2, seed=0):
    """(block tables with unused entries far out of range, pool size)."""
    pages = [-(-max(n, 0) // 16) for n in lens]
    nb = sum(pages) + extra
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(I32)
    t = torch.full((len(lens), max(max(pages), 1)), 1 << 28, dtype=I32)
    at = 0
    for b, n in enumerate(pages):
        t[b, :n] = perm[at:at + n]
        at += n
    return t.to(DEV), nb


def used_slots(tables, lens, nb):
    u = torch.zeros(nb * 16, dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        t = torch.arange(max(n, 0), device=DEV)
        u[tables[b, t // 16].long() * 16 + t % 16] = True
    return u.view(nb, 16)


def starts_of(counts):
    return torch.tensor([0] + list(counts), device=DEV).cumsum(0).to(I32)


def within(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite output"
    worst = (err / bound.clamp(min=1e-30)).max() if err.numel() else 0.0
    assert (err <= bound).all(), f"{what}: error is {float(worst):.3g} of the bound (max abs {float(err.max()):.3g})"


def lse_within(got, ref, what="", most=2e-3):
    """off by the scores' error: sums |q k| * scale of at most about 120 here,
    2^-16 of it, and two logarithms' roundings"""
    got = got.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: lse finiteness"
    assert (got[~fin] == -math.inf).all()
    if fin.any():
        err = (got[fin] - ref[fin]).abs().max()
        assert err <= most, f"{what}: lse off by {float(err):.3g}"
