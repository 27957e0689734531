"""Plain 64-bit forms of the scored attention and of the rotated cache write,
and the bounds that the kernels' outputs are held to.

Attention bound, per output element.  With p the exact softmax weights and
A = sum p |v|:
  * each weight is rounded once before it meets V: relative eps_p
    (bf16 2^-8, fp16 2^-11, a bf16 pair 2^-16), so A * eps_p;
  * an fp16 weight below 2^-14 has the absolute step 2^-24 instead (weights
    are relative to the row's largest, so their sum is at least 1): 2^-25 per
    key times the value it multiplies, which for int8, whose row scale goes
    into the weight, is the code itself: + 2^-25 * sum |code| / sum(weights).
    With scales of 0.02 that is the larger term for weights below 0.003;
  * a score off by d changes every weight by the factor e^+-d and, after
    normalisation, the output by at most 2 d A.  d = 2^-18 * S for S the
    largest sum |q k| * scale of the row (at most 256 products in 16 matrix
    steps, each step's adder off by 2^-22 of its sum at most: 16 * 2^-22),
    plus 2^-19 * cap
    for the cap's exponential and reciprocal (each 2^-22 relative, times up
    to 2 cap), plus 2^-22 * slope * distance for the bias, plus 2^-20 for the
    weights' own exponential;
  * the output is rounded once: 2^-8 |o| (bf16) or 2^-23 |o| (fp32).
"""
import math

import torch

DEV = "cuda"
EPS_BF16, EPS_FP16, EPS_BF16_PAIR = 2.0 ** -8, 2.0 ** -11, 2.0 ** -16


def make_pool(fmt, nb, hkv, D, seed=0, poison=True):
    """A pool of the format with N(0, 1)-like values; -> (arrays, global)."""
    g = torch.Generator(DEV).manual_seed(seed)
    shape = (nb, hkv, 16, D)

    def one():
        x = torch.randn(shape, device=DEV, generator=g)
        if fmt == "bf16":
            return x.bfloat16(), None
        if fmt == "fp8":
            return (x * 8).to(torch.float8_e4m3fn).view(torch.uint8), None
        if fmt == "int8":
            return ((x * 40).clamp(-127, 127).round().to(torch.int8),
                    (torch.rand(shape[:3], device=DEV, generator=g) * 0.02 + 0.015).half())
        return (torch.randint(0, 256, (nb, hkv, 16, D // 2), device=DEV, generator=g).to(torch.uint8),
                (torch.rand((nb, hkv, 16, D // 16), device=DEV, generator=g) * 4 + 2).to(
                    torch.float8_e4m3fn).view(torch.uint8))
    k, ks = one()
    v, vs = one()
    return k, v, ks, vs, {"fp8": 0.125, "nvfp4": 0.0625}.get(fmt, 1.0)


_E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]


def values(fmt, codes, scales, glob):
    """fp64 values of a pool [NB, Hkv, 16, D]."""
    if fmt == "bf16":
        return codes.double()
    if fmt == "fp8":
        return codes.view(torch.float8_e4m3fn).double() * glob
    if fmt == "int8":
        return codes.double() * scales.double()[..., None]
    lut = torch.tensor(_E2M1, dtype=torch.float64, device=codes.device)
    x = lut[torch.stack((codes & 15, codes >> 4), -1).long()].flatten(-2)
    return x * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * glob


def tables_for(lens, extra=2, seed=0):
    """(block tables with unused entries far out of range, pool size)."""
    pages = [-(-max(n, 0) // 16) for n in lens]
    nb = sum(pages) + extra
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    t = torch.full((len(lens), max(max(pages), 1)), 1 << 28, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        t[b, :n] = perm[at:at + n]
        at += n
    return t.to(DEV), nb


def reference(kv_vals, q, new, lens, tables, scale, *, softcap=0.0, slopes=None, window=0,
              first_key=None, prefix=None, eps_p=EPS_BF16, out_eps=2.0 ** -23, v_unit=None):
    """v_unit [NB, Hkv, 16]: the int8 scales that go into fp16 weights.
    q [T, Hq, D]; -> (out fp64 [T, Hq, D], lse [T, Hq], bound [T, Hq, D])."""
    kd, vd = kv_vals
    T, Hq, D = q.shape
    hkv = kd.shape[1]
    G = Hq // hkv
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    row = 0
    for b, (m, n) in enumerate(zip(new, lens)):
        if m == 0 or n <= 0:
            row += m
            continue
        pg = tables[b, :-(-n // 16)].long()
        k = kd[pg].transpose(0, 1).reshape(hkv, -1, D)[:, :n]
        v = vd[pg].transpose(0, 1).reshape(hkv, -1, D)[:, :n]
        if v_unit is not None:
            u = v_unit[pg].transpose(0, 1).reshape(hkv, -1)[:, :n].double()
        pos = torch.arange(n - m, n, device=q.device)[:, None]
        t = torch.arange(n, device=q.device)[None]
        see = t <= pos
        if prefix is not None:
            see = see | (t < int(prefix[b]))
        if window:
            see = see & (t > pos - window)
        if first_key is not None:
            see = see & (t >= first_key[row:row + m].long()[:, None])
        see = see & (pos >= 0)
        for h in range(Hq):
            qq = q[row:row + m, h].double()
            x = qq @ k[h // G].T * scale
            d = 2.0 ** -18 * (qq.abs() @ k[h // G].abs().T * abs(scale))
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                d = d + 2.0 ** -19 * softcap
            if slopes is not None:
                far = slopes[h].double() * (pos - t).abs()
                x = x - far
                d = d + 2.0 ** -22 * far.abs()
            d = torch.where(see, d, 0.0).amax(1, keepdim=True) + 2.0 ** -20
            x = torch.where(see, x, -math.inf)
            top = x.amax(1, keepdim=True).clamp(min=-1e300)
            p = torch.exp(x - top)
            s = p.sum(1, keepdim=True)
            live = (s > 0).squeeze(1)
            w = p / s.clamp(min=1e-300)
            # hidden values may be anything: 0 weights must not meet them
            vv = torch.where(see.any(0)[:, None], v[h // G], 0.0)
            o = w @ vv
            out[row:row + m, h] = o
            bound[row:row + m, h] = (eps_p + 2 * d) * (w @ vv.abs()) + out_eps * o.abs() + 1e-30
            if eps_p == EPS_FP16:
                code = vv.abs() if v_unit is None else vv.abs() / u[h // G][:, None]
                bound[row:row + m, h] += 2.0 ** -25 * (see.double() @ code) / s.clamp(min=1.0)
            lse[row:row + m, h] = torch.where(live, (top + torch.log(s.clamp(min=1e-300))).squeeze(1), -math.inf)
        row += m
    return out, lse, bound


def within(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite output"
    worst = (err / bound.clamp(min=1e-30)).max() if err.numel() else 0.0
    assert (err <= bound).all(), f"{what}: error is {float(worst):.3g} of the bound (max abs {float(err.max()):.3g})"


def lse_within(got, ref, what=""):
    """lse = max + ln(sum): off by the scores' error (below 4e-4 for these
    inputs: |q k| scale sums of at most about 100, 2^-18 of it) and two
    logarithms' roundings."""
    got = got.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: lse finiteness"
    assert (got[~fin] == -math.inf).all()
    if fin.any():
        err = (got[fin] - ref[fin]).abs().max()
        assert err <= 5e-4, f"{what}: lse off by {float(err):.3g}"
