"""pa_latent_decode (absorbed) and pa_latent_prefill (expanded) against their
formulas in 64 bits; the bounds are derived in latent_helpers."""
import math

import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import latent_helpers as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32
SCALE = 192 ** -0.5


def decode_case(fmt, lens, Q, H, seed=0):
    tables, nb = L.tables_for(lens, seed=seed)
    kv = pa.LatentCache(fmt, *L.pool(fmt, nb, seed))
    vals = L.values(fmt, kv.latent.clone(), kv.rope.clone(), kv.scale)
    L.poison(fmt, kv.latent, kv.rope, L.used_slots(tables, lens, nb))
    q = torch.randn((len(lens), Q, H, 576), device=DEV, generator=torch.Generator(DEV).manual_seed(seed + 1)).bfloat16()
    return kv, vals, q, tables, torch.tensor(lens, dtype=I32, device=DEV)


def check_decode(fmt, lens, Q, H, seed=0, flags=0, **kw):
    kv, vals, q, tables, sl = decode_case(fmt, lens, Q, H, seed)
    o, lse, ws = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True, return_lse=True, **kw)
    ref, rl, bound = L.decode_reference(fmt, vals, q, lens, tables, SCALE)
    L.within(o, ref, bound, f"{fmt} {lens} {Q} {H}")
    L.lse_within(lse, rl)
    assert pa.read_error(ws) == flags
    ob, _ = pa.latent_decode(kv, q, tables, sl, SCALE, workspace=ws, **kw)
    assert torch.equal(ob, o.bfloat16())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[1], [16, 15, 17], [63, 64, 65], [127, 128, 129, 0], [1000]])
@pytest.mark.parametrize("H", [1, 20, 64, 128])
def test_decode(fmt, lens, H):
    check_decode(fmt, lens, 1, H)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("Q,H", [(2, 24), (8, 24), (16, 8), (3, 96), (2, 128), (16, 1), (5, 33)])
def test_verify(fmt, Q, H):
    check_decode(fmt, [200, Q, Q + 1, 65 + Q, 0], Q, H)


@pytest.mark.parametrize("H", [7, 40, 72, 100, 127])
def test_decode_odd_heads(H):
    check_decode("bf16", [333, 64], 1, H)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,Q,H", [([9000, 1, 700, 2500], 1, 24), ([70] * 200, 1, 16), ([20000], 1, 128),
                                      ([3000, 5000, 10], 4, 40)])
def test_decode_splits(fmt, lens, Q, H):
    check_decode(fmt, lens, Q, H, flags=0)


def test_decode_many_short_sequences():
    check_decode("bf16", [1 + (7 * i) % 90 for i in range(700)], 1, 8)


def test_verify_shorter_than_its_tokens():
    check_decode("bf16", [3, 100, 0], 5, 12, flags=pa.PA_ERRF_LEN_LT_QLEN)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_bad_pages_are_skipped(fmt):
    lens = [300, 70, 16]
    kv, vals, q, tables, sl = decode_case(fmt, lens, 2, 10)
    tables[0, 3] = -1
    tables[0, 18] = 1 << 30
    tables[2, 0] = kv.latent.shape[0]
    o, lse, ws = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True, return_lse=True)
    ref, rl, bound = L.decode_reference(fmt, vals, q, lens, tables, SCALE)
    L.within(o, ref, bound)
    L.lse_within(lse, rl)
    assert pa.read_error(ws) == pa.PA_ERRF_BAD_BLOCK_ID
    assert (o[2] == 0).all()


def test_length_flags():
    kv, vals, q, tables, sl = decode_case("bf16", [64, 64], 1, 4)
    o, ws = pa.latent_decode(kv, q, tables, torch.tensor([-5, 64], dtype=I32, device=DEV), SCALE, out_fp32=True)
    assert pa.read_error(ws) == pa.PA_ERRF_NEG_LEN and (o[0] == 0).all()
    o, ws = pa.latent_decode(kv, q, tables, torch.tensor([64, 65], dtype=I32, device=DEV), SCALE, out_fp32=True)
    assert pa.read_error(ws) == pa.PA_ERRF_LEN_OVER_CAPACITY
    ref, _, bound = L.decode_reference("bf16", vals, q, [64, 64], tables, SCALE)
    L.within(o, ref, bound)


def test_decode_nan_and_large_scores():
    """A NaN in a key reaches every row that sees it; scores of hundreds are exact softmaxes."""
    kv, vals, q, tables, sl = decode_case("bf16", [150, 90], 2, 9)
    o, ws = pa.latent_decode(kv, q * 40, tables, sl, SCALE, out_fp32=True)
    ref, _, bound = L.decode_reference("bf16", vals, q * 40, [150, 90], tables, SCALE)
    L.within(o, ref, bound)
    kv.latent[tables[0, 2], 5, 100] = math.nan
    o, ws = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True, workspace=ws)
    assert torch.isnan(o[0]).all() and torch.isfinite(o[1]).all()


def test_decode_increasing_scores():
    """The running maximum moves at every tile: keys aligned with the query, ever longer."""
    n, H = 1500, 24
    kv, _, q, tables, sl = decode_case("bf16", [n], 1, H)
    t = torch.arange(n, device=DEV)
    u = torch.randn(512, device=DEV)
    kv.latent[tables[0, t // 16].long(), t % 16] = (u * (t / 400.0)[:, None]).bfloat16()
    q[..., :512] = u.bfloat16()
    vals = L.values("bf16", torch.nan_to_num(kv.latent), torch.nan_to_num(kv.rope), 1.0)
    for sign in (1.0, -1.0):
        o, lse, _ = pa.latent_decode(kv, q, tables, sl, SCALE * sign, out_fp32=True, return_lse=True)
        ref, rl, bound = L.decode_reference("bf16", vals, q, [n], tables, SCALE * sign)
        L.within(o, ref, bound)
        L.lse_within(lse, rl, most=0.1)   # scores of up to 140 with sums |q k| of thousands


def test_decode_capture_streams_and_reuse():
    kv, vals, q, tables, sl = decode_case("bf16", [700, 33, 5000], 2, 20)
    want, ws = pa.latent_decode(kv, q, tables, sl, SCALE)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, _ = pa.latent_decode(kv, q, tables, sl, SCALE, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        pa.latent_decode(kv, q, tables, sl, SCALE, out=out, workspace=ws)
    for lens in ([700, 33, 5000], [1, 0, 4000], [16, 700, 2]):
        sl.copy_(torch.tensor(lens, dtype=I32))
        out.fill_(9.0)
        gr.replay()
        torch.cuda.synchronize()
        eager, _ = pa.latent_decode(kv, q, tables, sl, SCALE)
        nan = torch.isnan(eager)   # (a longer length reaches poisoned slots: NaN in both)
        assert torch.equal(torch.isnan(out), nan) and torch.equal(out[~nan], eager[~nan])


def test_decode_is_deterministic_and_leaves_inputs():
    kv, vals, q, tables, sl = decode_case("fp8", [9000, 400, 31], 1, 128)
    keep = [t.clone() for t in (q, kv.latent, tables, sl)]
    a, ws = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True)
    b, _ = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True, workspace=ws)
    assert torch.equal(a, b)
    assert all(torch.equal(x, y) for x, y in zip(keep, (q, kv.latent, tables, sl)))


def test_empty_batch_clears_the_flags():
    kv, _, q, tables, sl = decode_case("bf16", [64], 1, 4)
    _, ws = pa.latent_decode(kv, q, tables, torch.tensor([-1], dtype=I32, device=DEV), SCALE)
    assert pa.read_error(ws)
    o, _ = pa.latent_decode(kv, q[:0], tables[:0], sl[:0], SCALE, workspace=ws)
    assert o.shape == (0, 1, 4, 512) and pa.read_error(ws) == 0


# ------------------------------------------------------------------ expanded

def prefill_case(new, keys, H, seed=0, packed=True, extra_q=0, extra_k=0):
    g = torch.Generator(DEV).manual_seed(seed)

    def randn(*s):
        return torch.randn(s, device=DEV, generator=g).bfloat16()
    T, N = sum(new) + extra_q, sum(keys) + extra_k
    q = randn(T, H, 192)
    if packed:
        kv = randn(N, H, 256)
        kn, v = kv[..., :128], kv[..., 128:]
        kr = randn(N, 576)[:, 512:]
    else:
        kn, v, kr = randn(N, H, 128), randn(N, H, 128), randn(N, 64)
    return q, kn, kr, v


def check_prefill(new, keys, H, causal=True, flags=0, **kw):
    q, kn, kr, v = prefill_case(new, keys, H, **kw)
    qs, ks = L.starts_of(new), L.starts_of(keys)
    o, lse, ws = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, causal=causal, out_fp32=True, return_lse=True)
    ref, rl, bound = L.prefill_reference(q, kn, kr, v, new, keys, SCALE, causal)
    L.within(o, ref, bound, f"{new} {keys} {H} {causal}")
    L.lse_within(lse, rl)
    assert pa.read_error(ws) == flags
    ob, _ = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, causal=causal, workspace=ws)
    assert torch.equal(ob, o.bfloat16())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H", [1, 5])
@pytest.mark.parametrize("new,keys", [([1], [1]), ([97], [97]), ([128], [128]), ([129], [129]), ([257], [300]),
                                      ([1], [1000]), ([300], [2000]), ([7, 0, 130, 1], [7, 5, 400, 129]),
                                      ([64, 64], [64, 640])])
def test_prefill(new, keys, H, causal):
    check_prefill(new, keys, H, causal)


def test_prefill_separate_tensors_and_many_sequences():
    check_prefill([3, 200], [3, 333], 4, packed=False)
    new = [1 + (5 * i) % 40 for i in range(70)]
    check_prefill(new, [m + (11 * i) % 50 for i, m in enumerate(new)], 2)


def test_prefill_long():
    check_prefill([700, 64], [3000, 5000], 3)
    check_prefill([1500], [1500], 20)


def test_prefill_rows_without_keys():
    check_prefill([5, 150, 3], [2, 20, 3], 3, flags=pa.PA_ERRF_LEN_LT_QLEN)
    check_prefill([5, 9], [0, 9], 3)
    check_prefill([5, 9], [0, 0], 3)
    check_prefill([200, 9], [0, 3], 2, causal=False)


def test_prefill_rows_of_no_sequence_stay():
    new, keys, H = [33, 40], [50, 40], 3
    q, kn, kr, v = prefill_case(new, keys, H, extra_q=12, extra_k=200)
    qs = torch.tensor([4, 37, 77], dtype=I32, device=DEV)
    ks = torch.tensor([100, 150, 190], dtype=I32, device=DEV)
    kn[:100], v[:100], kr[:100] = math.nan, math.nan, math.nan
    kn[190:], v[190:], kr[190:] = math.nan, math.inf, math.nan
    q[:4], q[77:] = math.nan, math.nan
    out = torch.full((85, H, 128), 7.0, device=DEV)
    o, lse, ws = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, out=out, return_lse=True)
    assert (o[:4] == 7).all() and (o[77:] == 7).all()
    ref, rl, bound = L.prefill_reference(q[4:77], kn[100:190], kr[100:190], v[100:190], new, keys, SCALE)
    L.within(o[4:77], ref, bound)
    L.lse_within(lse[4:77], rl)
    assert pa.read_error(ws) == 0


def test_prefill_neighbours_may_hold_anything():
    """The next sequence's rows share a tile with this one's last keys."""
    new, keys, H = [30, 64, 3], [30, 64, 3], 2
    q, kn, kr, v = prefill_case(new, keys, H)
    v[30:94], kn[30:94] = math.nan, math.inf
    o, _ = pa.latent_prefill(q, kn, kr, v, L.starts_of(new), L.starts_of(keys), SCALE, out_fp32=True)
    ref, _, bound = L.prefill_reference(q[:30], kn[:30], kr[:30], v[:30], [30], [30], SCALE)
    L.within(o[:30], ref, bound)
    ref, _, bound = L.prefill_reference(q[94:], kn[94:], kr[94:], v[94:], [3], [3], SCALE)
    L.within(o[94:], ref, bound)
    assert torch.isnan(o[30:94]).all()


def test_prefill_bad_starts():
    q, kn, kr, v = prefill_case([20], [20], 2)
    _, ws = pa.latent_prefill(q, kn, kr, v, torch.tensor([0, 25], dtype=I32, device=DEV), L.starts_of([20]), SCALE)
    assert pa.read_error(ws) & pa.PA_ERRF_BAD_Q_START
    _, ws = pa.latent_prefill(q, kn, kr, v, L.starts_of([20]), torch.tensor([5, 2], dtype=I32, device=DEV), SCALE)
    assert pa.read_error(ws) & pa.PA_ERRF_BAD_Q_START


def test_prefill_chunks_join_by_their_lse():
    """A context in two parts without a mask and the chunk's own causal part, merged."""
    m, n, H = 100, 700, 4
    q, kn, kr, v = prefill_case([m], [n], H)
    parts = [(0, 300, False), (300, 600, False), (600, 700, True)]
    res = [pa.latent_prefill(q, kn[a:b], kr[a:b], v[a:b], L.starts_of([m]), L.starts_of([b - a]), SCALE, causal=c,
                             out_fp32=True, return_lse=True)[:2] for a, b, c in parts]
    o, lse = pa.merge(torch.stack([r[0] for r in res]).flatten(1, 2), torch.stack([r[1] for r in res]).flatten(1),
                      out_fp32=True, return_lse=True)
    ref, rl, bound = L.prefill_reference(q, kn, kr, v, [m], [n], SCALE)
    L.within(o.view(m, H, 128), ref, bound + 2.0 ** -18)
    L.lse_within(lse.view(m, H), rl)


def test_prefill_capture_and_streams():
    new, keys = [50, 260], [90, 400]
    q, kn, kr, v = prefill_case(new, keys, 4)
    qs, ks = L.starts_of(new), L.starts_of(keys)
    want, ws = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, _ = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, out=out, workspace=ws)
    out.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# --------------------------------------------------------------- as used

@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_prompt_and_its_next_tokens(fmt):
    """append, gather, expansion, prefill; then append and decode of the next two
    tokens, against attention over the cached rows in 64 bits."""
    T, H, more = 150, 6, 2
    g = torch.Generator(DEV).manual_seed(3)

    def randn(*s):
        return torch.randn(s, device=DEV, generator=g)
    wk, wv = (randn(H, 512, 128).mul(512 ** -0.5).bfloat16() for _ in range(2))
    rows = randn(T + more, 576).bfloat16()
    q = randn(T + more, H, 192).bfloat16()
    nb = 12
    kv = pa.LatentCache(fmt, torch.zeros((nb, 16, 512), device=DEV, dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8),
                        torch.zeros((nb, 16, 64), device=DEV, dtype=torch.bfloat16), 1.0 if fmt == "bf16" else 1 / 64)
    tables = torch.randperm(nb, device=DEV, generator=g).to(I32)[None]
    pos = torch.arange(T + more, device=DEV, dtype=I32)
    slots = (tables[0, pos.long() // 16] * 16 + pos % 16).long()
    inv, _ = pa.rope_frequencies(64, device=DEV)
    norm = (1 + 0.1 * randn(512)).bfloat16()
    kw = dict(interleaved=True, norm=norm)
    pa.latent_append(kv, rows[:T, :512], rows[:T, 512:], pos[:T], slots[:T], inv, q=q[:T, :, 128:],
                     q_out=q[:T, :, 128:], **kw)
    c, r = pa.latent_gather(kv, tables, L.starts_of([T]), T)
    kn, v = (torch.einsum("td,hde->the", c, w) for w in (wk, wv))
    out, _ = pa.latent_prefill(q[:T], kn, r, v, L.starts_of([T]), L.starts_of([T]), SCALE, out_fp32=True)
    nxt = []
    for t in range(T, T + more):
        absorbed = torch.empty((1, 1, H, 576), device=DEV, dtype=torch.bfloat16)
        pa.latent_append(kv, rows[t:t + 1, :512], rows[t:t + 1, 512:], pos[t:t + 1], slots[t:t + 1], inv,
                         q=q[t:t + 1, :, 128:], q_out=absorbed[0, ..., 512:], **kw)
        absorbed[0, 0, :, :512] = torch.einsum("he,hde->hd", q[t, :, :128], wk)
        o, ws = pa.latent_decode(kv, absorbed, tables, torch.tensor([t + 1], dtype=I32, device=DEV), SCALE,
                                 out_fp32=True)
        assert pa.read_error(ws) == 0
        q[t, :, 128:] = absorbed[0, 0, :, 512:]
        nxt.append(torch.einsum("hd,hde->he", o[0, 0].double(), wv.double()))
    vals, gscale = L.values(fmt, kv.latent, kv.rope, kv.scale)
    row = vals[tables[0].long()].reshape(-1, 576)[:T + more] * gscale
    k64 = torch.einsum("td,hde->the", row[:, :512], wk.double())
    v64 = torch.einsum("td,hde->the", row[:, :512], wv.double())
    want, _, bound = L.prefill_reference(q, k64, row[:, 512:], v64, [T + more], [T + more], SCALE)
    got = torch.cat((out.double(), torch.stack(nxt)))
    # rounded on the way: expanded keys and values or absorbed queries (2^-8 of sums of unit size, in the
    # scores times |q| ~ 14 and the scale 0.07: below 2^-6 a score), the gathered rows (2^-8)
    assert ((got - want).abs() <= bound + 2.0 ** -4).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_prefill_increasing_scores(sign):
    """Keys aligned with the queries and ever longer: scores pass the first tile's by hundreds (the second pass with
    a running maximum), in one sequence of two and for one head of two."""
    new, keys, H = [300, 40], [1300, 700], 2
    q, kn, kr, v = prefill_case(new, keys, H)
    u = torch.randn(128, device=DEV, generator=torch.Generator(DEV).manual_seed(9))
    q[:300, 1, :128] = u.bfloat16()
    kn[:1300, 1] = (sign * u * (torch.arange(1300, device=DEV) / 100.0 - 3)[:, None]).bfloat16()
    o, lse, ws = pa.latent_prefill(q, kn, kr, v, L.starts_of(new), L.starts_of(keys), SCALE * sign, out_fp32=True,
                                   return_lse=True)
    ref, rl, bound = L.prefill_reference(q, kn, kr, v, new, keys, SCALE * sign)
    L.within(o, ref, bound)
    L.lse_within(lse, rl, most=0.1)   # sums |q k| of thousands: 2^-16 of them
    ob, _ = pa.latent_prefill(q, kn, kr, v, L.starts_of(new), L.starts_of(keys), SCALE * sign, workspace=ws)
    assert torch.equal(ob, o.bfloat16()) and pa.read_error(ws) == 0


def test_prefill_negative_and_zero_scale():
    new, keys, H = [129, 5], [200, 300], 2
    q, kn, kr, v = prefill_case(new, keys, H)
    for scale in (-SCALE, 0.0):
        o, lse, _ = pa.latent_prefill(q, kn, kr, v, L.starts_of(new), L.starts_of(keys), scale, out_fp32=True,
                                      return_lse=True)
        ref, rl, bound = L.prefill_reference(q, kn, kr, v, new, keys, scale)
        L.within(o, ref, bound)
        L.lse_within(lse, rl)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_decode_negative_and_zero_scale(fmt):
    lens = [129, 5]
    kv, vals, q, tables, sl = decode_case(fmt, lens, 2, 20)
    for scale in (-SCALE, 0.0):
        o, lse, _ = pa.latent_decode(kv, q, tables, sl, scale, out_fp32=True, return_lse=True)
        ref, rl, bound = L.decode_reference(fmt, vals, q, lens, tables, scale)
        L.within(o, ref, bound)
        L.lse_within(lse, rl)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,keys,H", [([10], [9000], 3),            # few tiles: all in pieces
                                        ([300, 5, 0, 130], [5000, 40, 0, 2100], 4),
                                        ([2300], [2600], 16),         # a round and a little more: the last in pieces
                                        ([260] * 20, [1100] * 20, 4)])
def test_prefill_pieces(new, keys, H, causal):
    check_prefill(new, keys, H, causal)


def test_prefill_pieces_that_see_nothing_and_hold_anything():
    """Pieces of a causal tile that its first rows do not see, beside neighbours of NaN."""
    m, n, H = 256, 4090, 2
    q, kn, kr, v = prefill_case([m], [n], H, extra_k=200)
    kn[n:], v[n:], kr[n:] = math.nan, math.nan, math.nan
    o, lse, _ = pa.latent_prefill(q, kn, kr, v, L.starts_of([m]), L.starts_of([n]), SCALE, out_fp32=True, return_lse=True)
    ref, rl, bound = L.prefill_reference(q, kn, kr, v, [m], [n], SCALE)
    L.within(o, ref, bound + 2.0 ** -20)
    L.lse_within(lse, rl)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("Q,H", [(1, 16), (1, 24), (2, 64), (1, 128)])
def test_decode_scores_far_past_the_first_tile(fmt, Q, H):
    """Some rows of some sequences: a worker goes over its run again."""
    lens = [900, 40, 7000]
    kv, _, q, tables, sl = decode_case(fmt, lens, Q, H)
    u = torch.randn(512, device=DEV, generator=torch.Generator(DEV).manual_seed(5))
    n = lens[2]
    t = torch.arange(n, device=DEV)
    k = u * (t / 700.0)[:, None]
    kv.latent[tables[2, t // 16].long(), t % 16] = (k.bfloat16() if fmt == "bf16" else
                                                    (k * 8).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    q[2, :, ::3, :512] = u.bfloat16()
    rows, scale = L.values(fmt, kv.latent, kv.rope, kv.scale)
    o, lse, ws = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True, return_lse=True)
    ref, rl, bound = L.decode_reference(fmt, (torch.nan_to_num(rows), scale), q, lens, tables, SCALE)
    L.within(o, ref, bound)
    L.lse_within(lse, rl, most=0.5)   # sums |q k| * scale of up to 30,000: 2^-16 of them
    assert pa.read_error(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("Q,H", [(5, 128), (16, 128), (16, 100)])
def test_verify_many_groups(fmt, Q, H):
    """More than eight groups of rows: several sets of them walk the keys one after another."""
    check_decode(fmt, [Q + 3, 130, 0, 1500], Q, H)


@pytest.mark.parametrize("H", [1, 3])
def test_prefill_heads_before_tokens(H):
    """Queries, keys and values with the heads outermost, and a single head with strides of its own."""
    new, keys = [150, 3], [200, 90]
    q, kn, kr, v = prefill_case(new, keys, H, packed=False)
    qs, ks = L.starts_of(new), L.starts_of(keys)
    want, _ = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE)
    if H == 1:
        def turn(x):
            return torch.as_strided(x, x.shape, (x.stride(0), 24, 1))
    else:
        def turn(x):
            return x.transpose(0, 1).contiguous().transpose(0, 1)
    got, _ = pa.latent_prefill(turn(q), turn(kn), kr, turn(v), qs, ks, SCALE)
    assert torch.equal(got, want)


def test_prefill_one_token_of_one_key():
    q, kn, kr, v = prefill_case([1], [1], 2)
    o, _ = pa.latent_prefill(q[:, :1], kn[:, :1], kr, v[:, :1], L.starts_of([1]), L.starts_of([1]), SCALE)
    assert torch.equal(o, v[:, :1])


def test_two_workspaces_at_once():
    """Two calls on two streams with a workspace each."""
    kv, _, q, tables, sl = decode_case("bf16", [3000, 800], 1, 40)
    kv2, _, q2, tables2, sl2 = decode_case("fp8", [5000, 70], 1, 128, seed=4)
    want, want2 = pa.latent_decode(kv, q, tables, sl, SCALE)[0], pa.latent_decode(kv2, q2, tables2, sl2, SCALE)[0]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        x, _ = pa.latent_decode(kv, q, tables, sl, SCALE, stream=a)
        y, _ = pa.latent_decode(kv2, q2, tables2, sl2, SCALE, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(x, want) and torch.equal(y, want2)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("Q,H", [(1, 24), (2, 60)])
def test_bad_first_pages_before_low_scores(fmt, Q, H):
    """The first tile of a piece gives no maximum; the keys after it all score about -460."""
    lens = [200, 90]
    kv, vals, q, tables, sl = decode_case(fmt, lens, Q, H)
    one = torch.tensor(4.0 if fmt == "bf16" else 32.0, device=DEV)
    kv.latent[..., 0] = one.bfloat16() if fmt == "bf16" else one.to(torch.float8_e4m3fn).view(torch.uint8)
    vals[0][..., 0] = one.double()
    q[..., 0] = -1600.0
    tables[0, :2] = 1 << 30
    tables[1, 0] = -1
    o, lse, ws = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True, return_lse=True)
    ref, rl, bound = L.decode_reference(fmt, vals, q, lens, tables, SCALE)
    L.within(o, ref, bound)
    L.lse_within(lse, rl, most=0.02)   # sums |q k| * scale of about 600: 2^-16 of them
    assert (lse < -300).all() and pa.read_error(ws) == pa.PA_ERRF_BAD_BLOCK_ID


@pytest.mark.parametrize("n,at", [(300, 0), (2100, 0), (2100, 1024)])
def test_prefill_first_tile_of_minus_infinity(n, at):
    """128 keys score -inf, the first tile of a piece; the others about -460."""
    H = 2
    q, kn, kr, v = prefill_case([150], [n], H)
    q[..., 0] = 800.0
    kn[..., 0] = -8.0
    kn[at:at + 128, :, 0] = -math.inf
    o, lse, _ = pa.latent_prefill(q, kn, kr, v, L.starts_of([150]), L.starts_of([n]), SCALE, causal=False, out_fp32=True,
                                  return_lse=True)
    left = torch.cat((torch.arange(at), torch.arange(at + 128, n))).to(DEV)
    ref, rl, bound = L.prefill_reference(q, kn[left], kr[left], v[left], [150], [n - 128], SCALE, causal=False)
    L.within(o, ref, bound)
    L.lse_within(lse, rl, most=0.02)   # sums |q k| * scale of about 500: 2^-16 of them


@pytest.mark.parametrize("B,most,H", [(32, 480, 120), (70, 60, 80)])
def test_prefill_thousands_of_items(B, most, H):
    """More than 32 items for each CTA, of one and of two row tiles; some need a second pass."""
    new = [1 + (37 * i) % most for i in range(B)]
    keys = [m + (53 * i) % 200 for i, m in enumerate(new)]
    assert sum(-(-m // 256) for m in new) * H > 33 * 152
    q, kn, kr, v = prefill_case(new, keys, H)
    ks = [0] + torch.tensor(keys).cumsum(0).tolist()
    for b, h in ((2, 5), (11, 40), (B - 1, H - 1)):
        kn[ks[b] + 128:ks[b + 1], h] *= 200   # (where the sequence has a second tile)
    qs, kst = L.starts_of(new), L.starts_of(keys)
    o, lse, ws = pa.latent_prefill(q, kn, kr, v, qs, kst, SCALE, out_fp32=True, return_lse=True)
    ref, rl, bound = L.prefill_reference(q, kn, kr, v, new, keys, SCALE)
    L.within(o, ref, bound)
    L.lse_within(lse, rl, most=0.5)   # sums |q k| * scale of up to 30,000 there: 2^-16 of them
    assert pa.read_error(ws) == 0
    ob, _ = pa.latent_prefill(q, kn, kr, v, qs, kst, SCALE, workspace=ws)
    assert torch.equal(ob, o.bfloat16())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_decode_many_rows_of_several_pieces(fmt):
    """Rows enough for a warp each in the join, of four or five pieces."""
    check_decode(fmt, [2500 + 37 * i for i in range(20)], 1, 128)
