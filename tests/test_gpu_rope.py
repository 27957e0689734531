"""pa_rope_append (per-head RMS norm, position rotation and quantised cache
write) against its formula in 64 bits.

Bounds.  A rotated value x cos a - y sin a, from fp32 x and y: the norm is
off by at most 24 roundings (a sum of 256 positive squares: 16 in a lane and
4 shuffles, the mean, rsqrt, two products), 24 * 2^-24 < 2^-19 relative; the
angle by 2^-23 radians (a turn's fraction in fp32) and each sine by 2 ulp; two
products and a sum: together below 2^-18 * (|x| + |y|).  Then one rounding:
bf16 2^-8 relative; int8 half a step of the row's scale; E4M3 2^-4 relative
or half its smallest step 2^-10; E2M1 half the gap around the value, the row
of gaps being 0.5 below 2, 1 below 4, 2 below 6 (of the block's scale), and
values past 6 where the scale was rounded down by up to 2^-4.
"""
import math

import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import score_helpers as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = ["bf16", "int8", "fp8", "nvfp4"]


def empty_pool(fmt, nb, hkv, D, fill=0x33):
    def byte(*shape):
        return torch.full(shape, fill, dtype=torch.uint8, device=DEV)
    if fmt == "bf16":
        k, v = (byte(nb, hkv, 16, D * 2).view(torch.bfloat16) for _ in range(2))
        return pa.KvCache(fmt, k, v)
    if fmt == "int8":
        k, v = (byte(nb, hkv, 16, D).view(torch.int8) for _ in range(2))
        ks, vs = (byte(nb, hkv, 32).view(torch.float16) for _ in range(2))
        return pa.KvCache(fmt, k, v, ks, vs)
    if fmt == "fp8":
        return pa.KvCache(fmt, byte(nb, hkv, 16, D), byte(nb, hkv, 16, D), None, None, 1 / 64, 1 / 32)
    return pa.KvCache(fmt, byte(nb, hkv, 16, D // 2), byte(nb, hkv, 16, D // 2), byte(nb, hkv, 16, D // 16),
                      byte(nb, hkv, 16, D // 16), 1 / 256, 1 / 128)


def formula(x, pos, inv_freq, rot, il, factor, w, eps):
    """(rotated fp64, sum of the pair's magnitudes)."""
    x = x.double()
    if w is not None:
        x = x * w.double() / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    y, mag = x.clone(), x.abs()
    if rot:
        a = (pos.double()[:, None] * inv_freq.double())[:, None]
        c, s = torch.cos(a) * factor, torch.sin(a) * factor
        i, j = (slice(0, rot, 2), slice(1, rot, 2)) if il else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., i] * s + x[..., j] * c
        m = (x[..., i].abs() + x[..., j].abs()) * abs(factor)
        mag[..., i], mag[..., j] = m, m
    return y, 2.0 ** -18 * mag + 1e-30


def stored(kv, x):
    codes, sc, g = ((kv.k_cache, kv.k_scale, kv.k_global) if x == "k" else (kv.v_cache, kv.v_scale, kv.v_global))
    return S.values(kv.dtype, codes, sc, g), sc, g


def check_row(kv, x, at, ref, slack):
    """The pool's rows at slots `at` against fp64 rows [n, Hkv, D]."""
    got, sc, g = stored(kv, x)
    got = got[at // 16, :, at % 16]
    err = (got - ref).abs()
    if kv.dtype == "bf16":
        ok = err <= slack + 2.0 ** -8 * ref.abs()
    elif kv.dtype == "fp8":
        sat = ref.clamp(-448 * g, 448 * g)
        ok = (got - sat).abs() <= slack + torch.maximum(2.0 ** -4 * sat.abs(), torch.tensor(2.0 ** -10 * g))
    elif kv.dtype == "int8":
        s = sc[at // 16, :, at % 16].double()
        want = ref.abs().amax(-1) / 127
        assert ((s - want).abs() <= 2.0 ** -11 * want + slack.amax(-1) / 127 + 2.0 ** -25).all()
        ok = err <= slack + s[..., None] * (0.5 + 127 * 2.0 ** -11)
    else:
        s = sc[at // 16, :, at % 16].view(torch.float8_e4m3fn).double()          # [n, Hkv, D / 16]
        blk, sl = ref.unflatten(-1, (-1, 16)), slack.unflatten(-1, (-1, 16)).amax(-1)
        want = (blk.abs().amax(-1) / (6 * g)).clamp(max=448)
        assert ((s - want).abs() <= torch.maximum(2.0 ** -4 * want, torch.tensor(2.0 ** -10)) + sl / (6 * g)).all()
        t = (s * g).repeat_interleave(16, -1)
        u = ref.abs() / t.clamp(min=1e-30)
        half = torch.where(u < 2, 0.25, torch.where(u < 4, 0.5, 1.0))
        ok = err <= slack + t * torch.maximum(half, u - 6)
    assert ok.all(), f"{kv.dtype} {x}: {int((~ok).sum())} values beyond the rounding"


def run(fmt, T, hkv, G, D, rot, il, norm, start, seed=0, factor=1.0, slots=None, inplace=False):
    gen = torch.Generator(DEV).manual_seed(seed)
    hq = hkv * G
    qkv = torch.randn((T, hq + 2 * hkv, D), device=DEV, generator=gen, dtype=torch.bfloat16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    keep = qkv.clone()
    nb = -(-T // 16) + 3
    kv = empty_pool(fmt, nb, hkv, D)
    if slots is None:
        slots = torch.randperm(nb * 16, device=DEV, generator=gen)[:T]
    pos = (torch.arange(T, device=DEV) * 3 + start).to(torch.int32)
    inv, _ = pa.rope_frequencies(rot, device=DEV) if rot else (torch.empty(0, device=DEV), 1.0)
    wq = wk = None
    if norm:
        wq, wk = (1 + 0.3 * torch.randn((2, D), device=DEV, generator=gen)).bfloat16().unbind(0)
    before = [None if t is None else t.clone() for t in (kv.k_cache, kv.v_cache, kv.k_scale, kv.v_scale)]
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = pa.rope_append(kv, q, k, v, pos, slots, inv, interleaved=il, attn_factor=factor, q_norm=wq, k_norm=wk,
                         eps=1e-6, workspace=ws, q_out=q if inplace else None)
    torch.cuda.synchronize()
    q, k, v = keep[:, :hq], keep[:, hq:hq + hkv], keep[:, hq + hkv:]
    ref, slack = formula(q, pos, inv, rot, il, factor, wq, 1e-6)
    assert ((out.double() - ref).abs() <= slack + 2.0 ** -8 * ref.abs()).all()
    if inplace:
        assert torch.equal(qkv[:, hq:].view(torch.int16), keep[:, hq:].view(torch.int16))
    else:
        assert torch.equal(qkv.view(torch.int16), keep.view(torch.int16))
    ok = (slots >= 0) & (slots < nb * 16)
    at = slots[ok]
    ref, slack = formula(k, pos, inv, rot, il, factor, wk, 1e-6)
    check_row(kv, "k", at, ref[ok], slack[ok])
    check_row(kv, "v", at, v.double()[ok], torch.full_like(v, 1e-30, dtype=torch.float64)[ok])
    # everything else in the pool is as it was
    other = torch.ones(nb * 16, dtype=torch.bool, device=DEV)
    other[at] = False
    oth = other.view(nb, 16)
    for t, b in zip((kv.k_cache, kv.v_cache, kv.k_scale, kv.v_scale), before):
        if t is not None:
            x, y = (a.view(torch.uint8).reshape(nb, hkv, 16, -1).transpose(1, 2)[oth] for a in (t, b))
            assert torch.equal(x, y)
    return pa.read_error(ws)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 32), (128, 96), (256, 256), (256, 64), (256, 224), (128, 0)])
@pytest.mark.parametrize("fmt", FMTS)
def test_formats_layouts_and_parts_of_the_head(fmt, D, rot, il, norm):
    assert run(fmt, 21, 2, 3, D, rot, il, norm, 1000) == 0


@pytest.mark.parametrize("T", [1, 2, 3, 5, 64, 257, 2000])
@pytest.mark.parametrize("hkv,G", [(1, 1), (1, 7), (3, 2), (4, 6), (8, 8)])
def test_tokens_and_heads(T, hkv, G):
    assert run("bf16", T, hkv, G, 128, 128, False, True, 0, seed=T) == 0
    assert run("fp8", T, hkv, G, 256, 64, True, False, 0, seed=T) == 0


@pytest.mark.parametrize("start", [-5000, 0, 131072, 1000003, 2 ** 31 - 200])
@pytest.mark.parametrize("il", [False, True])
def test_far_and_negative_positions(start, il):
    assert run("bf16", 40, 2, 2, 128, 128, il, False, start, factor=1.2) == 0


def test_in_place_and_padded_and_bad_slots():
    assert run("bf16", 100, 2, 4, 128, 128, False, True, 5, inplace=True) == 0
    slots = torch.arange(40, device=DEV)
    slots[3], slots[20:25] = -1, -1
    assert run("int8", 40, 2, 4, 128, 64, False, True, 5, slots=slots) == 0
    slots[30], slots[31] = 10 ** 9, -2
    for fmt in FMTS:
        assert run(fmt, 40, 2, 4, 256, 64, True, True, 5, slots=slots) == pa.PA_ERRF_BAD_SLOT


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_without_rotation_the_codes_are_those_of_append(fmt, D):
    """No norm, no rotation: the fp32 rows are the bf16 ones, so every byte is
    pa_append_kv's (ties, saturation, zeros and tiny rows among them)."""
    gen = torch.Generator(DEV).manual_seed(3)
    T, hkv = 300, 2
    x = torch.randn((T, 2 * hkv, D), device=DEV, generator=gen)
    x[10:20] = torch.randint(-8, 9, (10, 2 * hkv, D), device=DEV, generator=gen) * 0.5
    x[20:24] *= 1e4
    x[24:28] *= 1e-6
    x[28] = 0
    x[29] = -0.0
    x[30:34] *= 1e-30
    x = x.bfloat16()
    a, b = empty_pool(fmt, 20, hkv, D), empty_pool(fmt, 20, hkv, D)
    slots = torch.randperm(320, device=DEV, generator=gen)[:T]
    pa.append_kv(a, x[:, :hkv].contiguous(), x[:, hkv:].contiguous(), slots)
    pa.rope_append(b, x[:, :0], x[:, :hkv], x[:, hkv:], torch.zeros(T, dtype=torch.int32, device=DEV), slots,
                   torch.empty(0, device=DEV))
    for s, t in zip((a.k_cache, a.v_cache, a.k_scale, a.v_scale), (b.k_cache, b.v_cache, b.k_scale, b.v_scale)):
        if s is not None:
            assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_empty_batch_and_norm_of_a_zero_row():
    kv = empty_pool("bf16", 2, 1, 128)
    z = torch.zeros((0, 4, 128), device=DEV, dtype=torch.bfloat16)
    inv, _ = pa.rope_frequencies(128, device=DEV)
    out = pa.rope_append(kv, z, z[:, :1], z[:, :1], torch.empty(0, dtype=torch.int32, device=DEV),
                         torch.empty(0, dtype=torch.int64, device=DEV), inv)
    assert out.shape == (0, 4, 128)
    x = torch.zeros((1, 1, 128), device=DEV, dtype=torch.bfloat16)
    w = torch.ones(128, device=DEV, dtype=torch.bfloat16)
    out = pa.rope_append(kv, x, x, x, torch.ones(1, dtype=torch.int32, device=DEV),
                         torch.zeros(1, dtype=torch.int64, device=DEV), inv, q_norm=w, k_norm=w, eps=1e-6)
    assert (out == 0).all()


def test_only_one_side_is_normalised():
    gen = torch.Generator(DEV).manual_seed(1)
    q = torch.randn((7, 4, 128), device=DEV, generator=gen, dtype=torch.bfloat16)
    k, v = q[:, :1] * 2, q[:, 1:2]
    inv, _ = pa.rope_frequencies(64, device=DEV)
    w = (torch.rand(128, device=DEV, generator=gen) + 0.5).bfloat16()
    pos, slots = torch.arange(7, device=DEV, dtype=torch.int32), torch.arange(7, device=DEV)
    for wq, wk in ((w, None), (None, w)):
        kv = empty_pool("bf16", 1, 1, 128)
        out = pa.rope_append(kv, q, k, v, pos, slots, inv, q_norm=wq, k_norm=wk)
        ref, slack = formula(q, pos, inv, 64, False, 1.0, wq, 1e-6)
        assert ((out.double() - ref).abs() <= slack + 2.0 ** -8 * ref.abs()).all()
        ref, slack = formula(k, pos, inv, 64, False, 1.0, wk, 1e-6)
        check_row(kv, "k", slots, ref, slack)


def test_capture_and_replay_on_another_stream():
    gen = torch.Generator(DEV).manual_seed(1)
    q = torch.randn((9, 6, 256), device=DEV, generator=gen, dtype=torch.bfloat16)
    k, v = q[:, :2].contiguous(), q[:, 2:4].contiguous()
    inv, _ = pa.rope_frequencies(256, device=DEV)
    pos, slots = torch.arange(9, device=DEV, dtype=torch.int32), torch.arange(9, device=DEV)
    kv = empty_pool("fp8", 1, 2, 256)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.rope_append(kv, q, k, v, pos, slots, inv, q_out=out)
    for step in (100, 70000):
        pos.add_(step)
        g.replay()
        torch.cuda.synchronize()
        ref, slack = formula(q, pos, inv, 256, False, 1.0, None, 0)
        assert ((out.double() - ref).abs() <= slack + 2.0 ** -8 * ref.abs()).all()
        ref, slack = formula(k, pos, inv, 256, False, 1.0, None, 0)
        check_row(kv, "k", slots, ref, slack)


def test_a_prompt_and_its_next_tokens():
    """rope_append -> prefill -> rope_append -> decode_scored, as a serving
    step makes them, against one dense 64-bit attention over everything."""
    gen = torch.Generator(DEV).manual_seed(5)
    hkv, G, D, rot = 2, 4, 128, 64
    hq = hkv * G
    lens, steps, window, cap = [100, 33], 3, 60, 20.0
    total = [n + steps for n in lens]
    tables, nb = S.tables_for(total)
    k0, v0, _, _, _ = S.make_pool("bf16", nb, hkv, D)
    kv = pa.KvCache("bf16", k0, v0)
    inv, att = pa.rope_frequencies(rot, scaling="yarn", factor=4.0, original_len=2048, device=DEV)
    wq, wk = (1 + 0.1 * torch.randn((2, D), device=DEV, generator=gen)).bfloat16().unbind(0)
    rows = [torch.randn((n, hq + 2 * hkv, D), device=DEV, generator=gen, dtype=torch.bfloat16) for n in total]
    slope = torch.linspace(0.01, 0.05, hq, device=DEV)
    sc = pa.Score(softcap=cap, window=window, slopes=slope)

    def slots_of(b, p):
        return tables[b, p // 16].long() * 16 + p % 16

    def write(parts, pos):
        x = torch.cat(parts)
        sl = torch.cat([slots_of(b, p) for b, p in enumerate(pos)])
        return pa.rope_append(kv, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], torch.cat(pos).to(torch.int32), sl,
                              inv, attn_factor=att, q_norm=wq, k_norm=wk)

    pos = [torch.arange(n, device=DEV) for n in lens]
    q = write([r[:n] for r, n in zip(rows, lens)], pos)
    starts = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device=DEV)
    out, ws = pa.prefill(kv, q, starts, tables, torch.tensor(lens, dtype=torch.int32, device=DEV), D ** -0.5,
                         score=sc, out_fp32=True)
    got = [[out[:lens[0]]], [out[lens[0]:]]]
    queries = [[q[:lens[0]]], [q[lens[0]:]]]
    for i in range(steps):
        pos = [torch.tensor([n + i], device=DEV) for n in lens]
        q = write([r[n + i:n + i + 1] for r, n in zip(rows, lens)], pos)
        o, ws = pa.decode_scored(kv, q[:, None], tables, torch.tensor([n + i + 1 for n in lens], dtype=torch.int32, device=DEV),
                                 D ** -0.5, score=sc, out_fp32=True, workspace=ws)
        for b in range(2):
            got[b].append(o[b])
            queries[b].append(q[b:b + 1])
    for b in range(2):
        x, p = rows[b], torch.arange(total[b], device=DEV)
        want_k, slack = formula(x[:, hq:hq + hkv], p, inv, rot, False, att, wk, 1e-6)
        check_row(kv, "k", slots_of(b, p), want_k, slack)
        want_q, slack = formula(x[:, :hq], p, inv, rot, False, att, wq, 1e-6)
        qs = torch.cat(queries[b])
        assert ((qs.double() - want_q).abs() <= slack + 2.0 ** -8 * want_q.abs()).all()
        ref, _, bound = S.reference((kv.k_cache.double(), kv.v_cache.double()), qs, [total[b]], [total[b]],
                                    tables[b:b + 1], D ** -0.5, softcap=cap, window=window, slopes=slope)
        S.within(torch.cat(got[b]), ref, bound)
