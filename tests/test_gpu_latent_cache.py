"""pa_latent_append (norm, rotation, rounding into slots) against its formula
in 64 bits, and pa_latent_gather.

Bounds.  The norm: a sum of 512 squares in 16 steps and 5 shuffles, the mean,
rsqrt and two products, 32 roundings of 2^-24: 2^-19 relative.  A rotated value
x cos a - y sin a: the angle to 2^-23 radians, each sine to 2 ulp, two products
and a sum: 2^-18 * (|x| + |y|).  Then one rounding: bf16 2^-8 relative, E4M3
2^-4 or half its smallest step 2^-10; FP8 caches hold the rotated part over the
scale, one more quotient of 2^-24.
"""
import math

import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import latent_helpers as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


def turned(x, pos, inv, il, factor):
    """(fp64 rows, sum of a pair's magnitudes); x [T, .., 64]."""
    x = x.double()
    a = pos.double()[:, None] * inv.double()
    a = a.view(a.shape[0], *([1] * (x.dim() - 2)), 32)
    c, s = torch.cos(a) * factor, torch.sin(a) * factor
    i, j = (slice(0, 64, 2), slice(1, 64, 2)) if il else (slice(0, 32), slice(32, 64))
    y, mag = torch.empty_like(x), torch.empty_like(x)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    mag[..., i] = mag[..., j] = (x[..., i].abs() + x[..., j].abs()) * abs(factor)
    return y, 2.0 ** -18 * mag + 1e-30


def make(fmt, T, H, norm, il, seed=0, start=0, factor=1.0, slots=None):
    g = torch.Generator(DEV).manual_seed(seed)
    rows = torch.randn((T, 576), device=DEV, generator=g).bfloat16()
    q = torch.randn((T, max(H, 1), 192), device=DEV, generator=g).bfloat16()[..., 128:]
    nb = -(-max(T, 1) // 16) + 3
    if slots is None:
        slots = torch.randperm(nb * 16, device=DEV, generator=g)[:T]
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    fill = torch.full((nb, 16, 1024 if fmt == "bf16" else 512), 0x33, dtype=torch.uint8, device=DEV).view(dt)
    rope = torch.full((nb, 16, 128), 0x33, dtype=torch.uint8, device=DEV).view(torch.bfloat16)
    kv = pa.LatentCache(fmt, fill.clone(), rope.clone(), 1.0 if fmt == "bf16" else 1.0 / 64)
    w = (1 + 0.3 * torch.randn(512, device=DEV, generator=g)).bfloat16() if norm else None
    pos = (torch.arange(T, device=DEV) * 3 + start).to(I32)
    inv, _ = pa.rope_frequencies(64, device=DEV)
    return rows, q, slots, kv, w, pos, inv


def check(fmt, T, H, norm, il, start=0, factor=1.0, slots=None, mode="new", seed=0):
    rows, q, slots, kv, w, pos, inv = make(fmt, T, H, norm, il, seed, start, factor, slots)
    before = (kv.latent.clone(), kv.rope.clone())
    src = q.clone()
    q_out = None
    if mode == "inplace":
        q_out = q
    elif mode == "slice":
        q_out = torch.full((T, H, 576), 7.0, device=DEV, dtype=torch.bfloat16)[..., 512:]
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    got = pa.latent_append(kv, rows[:, :512], rows[:, 512:], pos, slots, inv, q=q if H else None, q_out=q_out,
                           interleaved=il, attn_factor=factor, norm=w, eps=1e-6, workspace=ws)
    torch.cuda.synchronize()
    if H:
        ref, slack = turned(src, pos, inv, il, factor)
        assert ((got.double() - ref).abs() <= slack + 2.0 ** -8 * ref.abs()).all()
    else:
        assert got is None
    ok = (slots >= 0) & (slots < kv.latent.shape[0] * 16)
    at = slots[ok]
    x = rows[:, :512].double()
    if norm:
        x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    slack = 2.0 ** -19 * x.abs()
    lat = kv.latent.view(-1, 512)[at]
    if fmt == "bf16":
        assert ((lat.double() - x[ok]).abs() <= (slack + 2.0 ** -8 * x.abs())[ok]).all()
    else:
        y = (x / kv.scale).clamp(-448, 448)[ok]
        step = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10, device=DEV)) + slack[ok] / kv.scale
        assert ((lat.view(torch.float8_e4m3fn).double() - y).abs() <= step).all()
    ref, slack = turned(rows[:, 512:], pos, inv, il, factor)
    ref, slack = ref[ok] / kv.scale, (slack[ok] + 2.0 ** -23 * ref[ok].abs()) / kv.scale
    assert ((kv.rope.view(-1, 64)[at].double() - ref).abs() <= slack + 2.0 ** -8 * ref.abs()).all()
    # every other slot as it was
    rest = torch.ones(kv.latent.shape[0] * 16, dtype=torch.bool, device=DEV)
    rest[at] = False
    for now, was in ((kv.latent, before[0]), (kv.rope, before[1])):
        a, b = (t.contiguous().view(-1, t.shape[-1]).view(torch.uint8)[rest] for t in (now, was))
        assert torch.equal(a, b)
    return pa.read_error(ws)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("T,H,norm", [(1, 20, True), (1, 1, False), (7, 24, True), (65, 128, False), (300, 7, True),
                                      (33, 0, True)])
def test_append(fmt, il, T, H, norm):
    assert check(fmt, T, H, norm, il) == 0


@pytest.mark.parametrize("mode", ["inplace", "slice"])
def test_append_queries_in_place_and_beside_the_absorbed_part(mode):
    assert check("bf16", 40, 20, True, False, mode=mode) == 0


def test_append_leaves_the_rest_of_the_queries():
    rows, q, slots, kv, w, pos, inv = make("bf16", 19, 5, True, True)
    whole = torch.randn((19, 5, 576), device=DEV).bfloat16()
    keep = whole.clone()
    pa.latent_append(kv, rows[:, :512], rows[:, 512:], pos, slots, inv, q=q, q_out=whole[..., 512:], interleaved=True)
    assert torch.equal(whole[..., :512], keep[..., :512])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_append_padded_and_bad_slots(fmt):
    slots = torch.tensor([5, -1, 40, -1, 7, 1 << 40, -2], device=DEV)
    assert check(fmt, 7, 3, True, False, slots=slots) == pa.PA_ERRF_BAD_SLOT
    assert check(fmt, 7, 3, True, False, slots=torch.full((7,), -1, device=DEV)) == 0


def test_append_far_positions():
    assert check("bf16", 17, 3, False, True, start=2 ** 31 - 60, factor=1.3) == 0


def test_append_no_tokens():
    assert check("bf16", 0, 4, True, False) == 0


def test_append_other_stream_and_graph():
    rows, q, slots, kv, w, pos, inv = make("fp8", 33, 9, True, False)
    want = pa.latent_append(kv, rows[:, :512], rows[:, 512:], pos, slots, inv, q=q, norm=w)
    lat, rope = kv.latent.clone(), kv.rope.clone()
    kv.latent.zero_(), kv.rope.zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = pa.latent_append(kv, rows[:, :512], rows[:, 512:], pos, slots, inv, q=q, norm=w, stream=st)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(rope[slots // 16, slots % 16], kv.rope[slots // 16, slots % 16])
    gr = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(gr):
        pa.latent_append(kv, rows[:, :512], rows[:, 512:], pos, slots, inv, q=q, q_out=out, norm=w)
    kv.latent.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lat[slots // 16, slots % 16], kv.latent[slots // 16, slots % 16])


# ------------------------------------------------------------------- gather

def gather_ref(fmt, kv, tables, lens, firsts):
    vals, g = L.values(fmt, kv.latent, kv.rope, kv.scale)
    rows = []
    for b, (n, f) in enumerate(zip(lens, firsts)):
        t = torch.arange(f, f + n, device=DEV)
        rows.append(vals[tables[b, t // 16].long(), t % 16] * g)
    return torch.cat(rows).float().bfloat16() if rows else None


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[1], [0, 16, 17], [1000, 3, 0, 65], [5] * 40])
def test_gather(fmt, lens):
    tables, nb = L.tables_for([n + 9 for n in lens])
    kv = pa.LatentCache(fmt, *L.pool(fmt, nb))
    for firsts in ([0] * len(lens), [(3 * b) % 10 for b in range(len(lens))]):
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        first = torch.tensor(firsts, dtype=I32, device=DEV) if any(firsts) else None
        lat, rope = pa.latent_gather(kv, tables, L.starts_of(lens), sum(lens), first=first, workspace=ws)
        ref = gather_ref(fmt, kv, tables, lens, firsts)
        assert torch.equal(torch.cat((lat, rope), 1), ref)
        assert pa.read_error(ws) == 0


def test_gather_rows_of_no_sequence_and_bad_pages():
    lens = [20, 40]
    tables, nb = L.tables_for(lens)
    kv = pa.LatentCache("bf16", *L.pool("bf16", nb))
    tables[1, 1] = nb
    starts = torch.tensor([3, 23, 63], dtype=I32, device=DEV)
    lat = torch.full((70, 512), 5.0, device=DEV, dtype=torch.bfloat16)
    rope = torch.full((70, 64), 5.0, device=DEV, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    pa.latent_gather(kv, tables, starts, 70, latent_out=lat, rope_out=rope, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERRF_BAD_BLOCK_ID
    for t in (lat, rope):
        assert (t[:3] == 5).all() and (t[63:] == 5).all() and (t[39:55] == 0).all()
    tables[1, 1] = 0
    ok = gather_ref("bf16", kv, tables, lens, [0, 0])
    assert torch.equal(lat[3:39], ok[:36, :512]) and torch.equal(rope[55:63], ok[52:60, 512:])


def test_gather_flags():
    tables, nb = L.tables_for([16, 16])
    kv = pa.LatentCache("fp8", *L.pool("fp8", nb))
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)

    def flags(starts, first=None, n=32):
        f = None if first is None else torch.tensor(first, dtype=I32, device=DEV)
        lat, _ = pa.latent_gather(kv, tables, torch.tensor(starts, dtype=I32, device=DEV), n, first=f, workspace=ws)
        assert torch.isfinite(lat[:1].float()).all()
        return pa.read_error(ws)
    assert flags([0, 16, 32]) == 0
    assert flags([0, 16, 32], [0, -1]) == pa.PA_ERRF_NEG_LEN
    assert flags([0, 16, 32], [0, 1]) == pa.PA_ERRF_LEN_OVER_CAPACITY
    assert flags([0, 16, 40]) & pa.PA_ERRF_BAD_Q_START
    assert flags([0, 20, 10]) & pa.PA_ERRF_BAD_Q_START


def test_append_queries_with_the_heads_outermost():
    rows, q, slots, kv, w, pos, inv = make("bf16", 21, 6, True, True)
    want = pa.latent_append(kv, rows[:, :512], rows[:, 512:], pos, slots, inv, q=q)
    turned_ = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((6, 21, 64), device=DEV, dtype=torch.bfloat16).transpose(0, 1)
    got = pa.latent_append(kv, rows[:, :512], rows[:, 512:], pos, slots, inv, q=turned_, q_out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
