"""pa_prefill (ragged prompt chunks over the paged cache, with score options)
against the plain 64-bit form of tests/score_helpers.py."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import score_helpers as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = ["bf16", "int8", "fp8", "nvfp4"]
# how the weights are rounded before the product with V
EPS_P = {"bf16": S.EPS_BF16, "int8": S.EPS_FP16, "fp8": S.EPS_FP16, "nvfp4": S.EPS_FP16}


def build(fmt, new, lens, hkv, G, D, seed=0):
    tables, nb = S.tables_for(lens, seed=seed)
    k, v, ks, vs, g = S.make_pool(fmt, nb, hkv, D, seed)
    kv = pa.KvCache(fmt, k, v, ks, vs, g, g)
    gen = torch.Generator(DEV).manual_seed(seed + 1)
    q = (torch.randn((sum(new), hkv * G, D), device=DEV, generator=gen) * 2).bfloat16()
    starts = torch.tensor([0] + list(new), device=DEV).cumsum(0).to(torch.int32)
    return kv, q, starts, tables, torch.tensor(lens, dtype=torch.int32, device=DEV)


def vals(kv):
    return (S.values(kv.dtype, kv.k_cache, kv.k_scale, kv.k_global),
            S.values(kv.dtype, kv.v_cache, kv.v_scale, kv.v_global))


def check(fmt, new, lens, hkv, G, D, seed=0, flags=0, **opt):
    kv, q, starts, tables, sl = build(fmt, new, lens, hkv, G, D, seed)
    sc = pa.Score(softcap=opt.get("softcap", 0.0), slopes=opt.get("slopes"), window=opt.get("window", 0),
                  first_key=opt.get("first_key"), prefix_lens=opt.get("prefix"))
    scale = D ** -0.5
    out, lse, ws = pa.prefill(kv, q, starts, tables, sl, scale, score=sc, out_fp32=True, return_lse=True,
                              max_seq_len=max(max(lens), 1))
    assert pa.read_error(ws) == flags
    ref, rl, bound = S.reference(vals(kv), q, new, lens, tables, scale, eps_p=EPS_P[fmt],
                                 v_unit=kv.v_scale if fmt == "int8" else None, **opt)
    what = f"{fmt} new {new} lens {lens} hkv {hkv} G {G} D {D}"
    S.within(out, ref, bound, what)
    S.lse_within(lse, rl, what)
    b16, ws = pa.prefill(kv, q, starts, tables, sl, scale, score=sc, max_seq_len=max(max(lens), 1), workspace=ws)
    assert torch.equal(b16.view(torch.int16), out.bfloat16().view(torch.int16))


def slopes(hq):
    return torch.linspace(0.001, 0.06, hq, device=DEV)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_ragged_causal(fmt, D):
    check(fmt, [1, 63, 64, 65, 130, 17], [1, 63, 100, 65, 300, 512], 2, 4, D)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8])
def test_group_sizes(G):
    check("bf16", [37, 129, 5], [37, 400, 77], 2, G, 128, seed=G)
    check("fp8", [37, 129, 5], [37, 400, 77], 1, G, 256, seed=G)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 513])
def test_lengths_around_tiles(n):
    check("bf16", [n], [n], 1, 4, 128, seed=n)
    check("bf16", [min(n, 33)], [n], 1, 2, 256, seed=n)
    check("nvfp4", [min(n, 33)], [n], 1, 2, 256, seed=n)


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 256), ("int8", 256), ("nvfp4", 128), ("fp8", 256)])
@pytest.mark.parametrize("opt", ["cap", "bias", "window", "docs", "prefix", "all"])
def test_score_options(fmt, D, opt):
    new, lens, hkv, G = [70, 1, 200], [70, 333, 650], 2, 4
    o = {}
    if opt in ("cap", "all"):
        o["softcap"] = 5.0
    if opt in ("bias", "all"):
        o["slopes"] = slopes(hkv * G)
    if opt in ("window", "all"):
        o["window"] = 100
    if opt in ("docs", "all"):
        pos = torch.cat([torch.arange(n - m, n) for m, n in zip(new, lens)])
        o["first_key"] = (pos // 90 * 90).to(torch.int32).to(DEV)
    if opt in ("prefix", "all"):
        o["prefix"] = torch.tensor([50, 0, 500], dtype=torch.int32, device=DEV)
    check(fmt, new, lens, hkv, G, D, **o)


def test_window_of_one_and_wider_than_the_cache():
    check("bf16", [40], [200], 1, 2, 128, window=1)
    check("bf16", [40], [200], 1, 2, 128, window=2 ** 31 - 1)


def test_rows_that_see_nothing():
    """first_key beyond the query: output 0 and lse -inf, neighbours as ever."""
    new, lens = [50, 20], [150, 20]
    first = torch.zeros(70, dtype=torch.int32)
    first[10:14] = 1 << 30
    first[50:] = 25          # the whole second sequence
    check("bf16", new, lens, 2, 4, 128, first_key=first.to(DEV))
    check("int8", new, lens, 2, 3, 256, first_key=first.to(DEV))


@pytest.mark.parametrize("fmt", FMTS)
def test_few_rows_over_a_long_cache(fmt):
    """The key axis is split and joined."""
    check(fmt, [3], [9001], 1, 4, 256, softcap=30.0)
    check(fmt, [40, 1], [5000, 3333], 2, 2, 128, slopes=slopes(4), window=2500)


@pytest.mark.parametrize("fmt,D,hkv,G,new,lens", [
    ("bf16", 256, 8, 8, [320], [8300]),            # 160 row tiles: eight in a last round of pieces
    ("bf16", 128, 8, 8, [637, 3], [8250, 300]),    # 160 + 8
    ("int8", 256, 4, 6, [411, 0, 420], [411, 20, 8500]),   # ragged: 80 + 80
    ("nvfp4", 256, 1, 8, [1, 2500], [8300, 12600])])
def test_last_round_of_tiles_in_pieces(fmt, D, hkv, G, new, lens):
    """A little more row tiles than SMs: those of the last round are split and
    joined, rows of no sequence stay as they were."""
    kv, q, starts, tables, sl = build(fmt, new, lens, hkv, G, D)
    T = sum(new)
    qq = torch.cat((q, q[:3]))
    out = torch.full((T + 3, hkv * G, D), 7.0, device=DEV)
    sc = pa.Score(softcap=20.0, window=8200)
    out, lse, ws = pa.prefill(kv, qq, starts, tables, sl, D ** -0.5, score=sc, out=out, return_lse=True,
                              max_seq_len=max(lens))
    assert pa.read_error(ws) == 0 and (out[T:] == 7.0).all()
    ref, rl, bound = S.reference(vals(kv), q, new, lens, tables, D ** -0.5, softcap=20.0, window=8200,
                                 eps_p=EPS_P[fmt], v_unit=kv.v_scale if fmt == "int8" else None)
    S.within(out[:T], ref, bound)
    S.lse_within(lse[:T], rl)


def test_padded_and_empty_sequences_and_rows_behind_the_last():
    new, lens = [5, 0, 9, 0], [5, 40, 60, 0]
    kv, q, starts, tables, sl = build("bf16", new, lens, 2, 4, 128)
    T = 14 + 6   # six rows of no sequence
    q = torch.cat((q, torch.full((6,) + q.shape[1:], float("nan"), device=DEV, dtype=torch.bfloat16)))
    out = torch.full((T, 8, 128), 7.0, device=DEV)
    out, lse, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, out=out, return_lse=True, max_seq_len=60)
    assert pa.read_error(ws) == 0
    ref, _, bound = S.reference(vals(kv), q[:14], new, lens, tables, 0.1)
    S.within(out[:14], ref, bound)
    assert (out[14:] == 7.0).all()
    # the same where the key axis is split (one long sequence) and rows precede the first
    kv, q, starts, tables, sl = build("bf16", [4], [4000], 1, 1, 128)
    qq = torch.cat((q, q, q))
    out = torch.full((12, 1, 128), 7.0, device=DEV)
    pa.prefill(kv, qq, starts + 4, tables, sl, 0.1, out=out, max_seq_len=4000)
    ref, _, bound = S.reference(vals(kv), q, [4], [4000], tables, 0.1)
    S.within(out[4:8], ref, bound)
    assert (out[:4] == 7.0).all() and (out[8:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
def test_values_no_query_sees_may_be_anything(fmt):
    """NaN past the end, and before the window's first key."""
    new, lens, hkv, G, D = [20, 33], [301, 44], 2, 2, 128
    kv, q, starts, tables, sl = build(fmt, new, lens, hkv, G, D)
    clean = vals(kv)
    ref, rl, bound = S.reference(clean, q, new, lens, tables, 0.1, window=30, eps_p=EPS_P[fmt],
                                 v_unit=kv.v_scale.clone() if fmt == "int8" else None)
    for b, (m, n) in enumerate(zip(new, lens)):
        hidden = list(range(0, max(0, n - m - 29))) + list(range(n, -(-n // 16) * 16))
        for t in hidden:
            pg = int(tables[b, t // 16])
            for x, s in ((kv.k_cache, kv.k_scale), (kv.v_cache, kv.v_scale)):
                if fmt == "int8":
                    s[pg, :, t % 16] = float("nan")
                elif fmt == "bf16":
                    x[pg, :, t % 16] = float("nan")
                else:
                    x[pg, :, t % 16] = 0x7F
    out, lse, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, score=pa.Score(window=30), out_fp32=True,
                              return_lse=True, max_seq_len=301)
    S.within(out, ref, bound, fmt)
    S.lse_within(lse, rl)
    assert pa.read_error(ws) == 0


def test_scores_far_beyond_the_cap():
    """Products of +-30000 in one key: the cap's exponential overflows or
    vanishes and the score is the cap itself; without a cap the key takes all
    the weight or none."""
    kv, q, starts, tables, sl = build("bf16", [64], [200], 1, 2, 128)
    q[:, :, 0] = torch.where(torch.arange(64, device=DEV) % 2 == 0, 1.0, -1.0)[:, None].bfloat16()
    pg = int(tables[0, 3])
    kv.k_cache[pg, :, 5] = 0
    kv.k_cache[pg, :, 5, 0] = 30000.0
    for cap in (20.0, 0.0):
        out, ws = pa.prefill(kv, q, starts, tables, sl, 1.0, score=pa.Score(softcap=cap), out_fp32=True, max_seq_len=200)
        # the other keys' scores are sums |q k| of at most 400: errors 2^-18 of it
        ref, _, _ = S.reference(vals(kv), q, [64], [200], tables, 1.0, softcap=cap)
        assert torch.isfinite(out).all()
        big = vals(kv)[1].abs().max()
        assert ((out.double() - ref).abs() <= (2.0 ** -8 + 2 * (400 * 2.0 ** -18 + 2.0 ** -14)) * big).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("cap", [1e6, 1e15, 1e30])
def test_caps_far_above_the_scores_leave_them(fmt, cap):
    """cap tanh(s / cap) differs from s by s^3 / (3 cap^2): below 1e-5 for |s| < 300."""
    for bias in (None, slopes(4)):
        kv, q, starts, tables, sl = build(fmt, [70, 200], [400, 200], 2, 2, 128)
        sc = pa.Score(softcap=cap, slopes=bias)
        out, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, score=sc, out_fp32=True, max_seq_len=400)
        ref, _, bound = S.reference(vals(kv), q, [70, 200], [400, 200], tables, 0.1, slopes=bias, eps_p=EPS_P[fmt],
                                    v_unit=kv.v_scale if fmt == "int8" else None)
        S.within(out, ref, bound + 2e-5 * vals(kv)[1].abs().max())


def test_tiny_cap_averages_the_keys():
    """Every score is at most the cap: equal weights, also for a product of 0."""
    for fmt in ("bf16", "fp8"):
        kv, q, starts, tables, sl = build(fmt, [70, 3], [400, 200], 2, 2, 128)
        q[5, 1] = 0
        out, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, score=pa.Score(softcap=1e-40), out_fp32=True, max_seq_len=400)
        ref, _, bound = S.reference(vals(kv), q * 0, [70, 3], [400, 200], tables, 0.1, eps_p=EPS_P[fmt])
        S.within(out, ref, bound)


@pytest.mark.parametrize("hkv,G,B,most,earlier", [(1, 8, 33, 150, 60), (2, 3, 300, 40, 60), (1, 1, 1100, 3, 60),
                                                  (1, 2, 40, 3, 2000)])
def test_many_sequences(hkv, G, B, most, earlier):
    """More than 32: chunks of 0 to `most` tokens over 0 to `earlier` keys (2000: the
    keys are split); rows before the first and behind the last sequence stay as
    they were."""
    r = torch.Generator().manual_seed(B)
    new = [int(x) for x in torch.randint(0, most + 1, (B,), generator=r)]
    lens = [m + int(x) for m, x in zip(new, torch.randint(0, earlier + 1, (B,), generator=r))]
    kv, q, starts, tables, sl = build("bf16", new, lens, hkv, G, 128)
    T = sum(new)
    qq = torch.cat((q[:min(T, 300)], q, q[:3]))
    k = len(qq) - T - 3   # rows before the first
    out = torch.full((len(qq), hkv * G, 128), 7.0, device=DEV)
    out, lse, ws = pa.prefill(kv, qq, starts + k, tables, sl, 0.1, out=out, return_lse=True, max_seq_len=max(lens))
    assert pa.read_error(ws) == 0
    ref, rl, bound = S.reference(vals(kv), q, new, lens, tables, 0.1)
    S.within(out[k:k + T], ref, bound)
    S.lse_within(lse[k:k + T], rl)
    assert (out[:k] == 7.0).all() and (out[k + T:] == 7.0).all()
    wild = starts.clone()
    wild[-2] = T + 5
    _, ws = pa.prefill(kv, q, wild, tables, sl, 0.1, max_seq_len=max(lens))
    assert pa.read_error(ws) & pa.PA_ERRF_BAD_Q_START


def test_bad_block_ids_lengths_and_starts_are_flagged():
    kv, q, starts, tables, sl = build("bf16", [20, 30], [120, 64], 2, 2, 128)
    bad = tables.clone()
    bad[0, 3] = -7
    out, ws = pa.prefill(kv, q, starts, bad, sl, 0.1, out_fp32=True, max_seq_len=120)
    assert pa.read_error(ws) == pa.PA_ERRF_BAD_BLOCK_ID
    ref, _, bound = S.reference(vals(kv), q, [20, 30], [120, 64], tables, 0.1)
    S.within(out[20:], ref[20:], bound[20:])
    # the other sequence: as if the block's keys were hidden
    keep = torch.cat((torch.arange(48), torch.arange(64, 120))).to(DEV)
    kd, vd = (x[tables[0, :8].long()].transpose(0, 1).reshape(2, -1, 128) for x in vals(kv))
    for i in (0, 19):
        vis = keep[keep <= 100 + i]
        w = torch.softmax(q[i, 0].double() @ kd[0, vis].T * 0.1, -1)
        S.within(out[i, 0], w @ vd[0, vis], 2.0 ** -7 * (w @ vd[0, vis].abs()))
    _, ws = pa.prefill(kv, q, starts, tables, torch.tensor([-3, 64], dtype=torch.int32, device=DEV), 0.1, max_seq_len=120)
    assert pa.read_error(ws) == pa.PA_ERRF_NEG_LEN
    _, ws = pa.prefill(kv, q, starts, tables[:, :8].contiguous(), torch.tensor([4000, 64], dtype=torch.int32, device=DEV),
                       0.1, max_seq_len=4000)
    assert pa.read_error(ws) == pa.PA_ERRF_LEN_OVER_CAPACITY
    o, ws = pa.prefill(kv, q, starts, tables, torch.tensor([12, 64], dtype=torch.int32, device=DEV), 0.1,
                       out_fp32=True, max_seq_len=120)
    assert pa.read_error(ws) == pa.PA_ERRF_LEN_LT_QLEN
    assert (o[:8] == 0).all()          # positions below 0 see nothing
    ref, _, bound = S.reference(vals(kv), q, [20, 30], [12, 64], tables, 0.1)
    S.within(o[8:], ref[8:], bound[8:])
    wild = torch.tensor([0, 99, 50], dtype=torch.int32, device=DEV)
    _, ws = pa.prefill(kv, q, wild, tables, sl, 0.1, max_seq_len=120)
    assert pa.read_error(ws) & pa.PA_ERRF_BAD_Q_START


def test_same_as_verify_and_decode_on_their_shapes():
    """Eight new tokens per sequence are pa_verify's case, one is pa_decode's."""
    for m, call in ((8, pa.verify), (1, pa.decode)):
        lens = [200, 77, 1000]
        kv, q, starts, tables, sl = build("bf16", [m] * 3, lens, 2, 4, 128)
        out, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, out_fp32=True, max_seq_len=1000)
        other, _ = call(kv, q.view(3, m, 8, 128), tables, sl, 0.1, out_fp32=True, max_seq_len=1000)
        ref, _, bound = S.reference(vals(kv), q, [m] * 3, lens, tables, 0.1)
        S.within(out, ref, bound)
        S.within(other.reshape(out.shape), ref, bound)


def test_repeats_bit_for_bit_and_on_another_stream():
    kv, q, starts, tables, sl = build("bf16", [300, 5], [900, 2000], 2, 4, 128)
    a, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, max_seq_len=2000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, _ = pa.prefill(kv, q, starts, tables, sl, 0.1, max_seq_len=2000, stream=s)
    s.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
@pytest.mark.parametrize("new,lens", [([150, 40], [600, 300]), ([4, 2], [3000, 2500])])
def test_capture_and_replay_with_new_inputs(fmt, new, lens):
    kv, q, starts, tables, sl = build(fmt, new, lens, 1, 4, 128)
    out = torch.empty((sum(new), 4, 128), device=DEV)
    first = torch.zeros(sum(new), dtype=torch.int32, device=DEV)
    sc = pa.Score(softcap=20.0, window=500, first_key=first)
    _, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, score=sc, out=out, max_seq_len=max(lens))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.prefill(kv, q, starts, tables, sl, 0.1, score=sc, out=out, max_seq_len=max(lens), workspace=ws)
    for step in range(3):
        cur = [n - 10 * step for n in lens]
        sl.copy_(torch.tensor(cur, dtype=torch.int32))
        first.fill_(step)
        q.copy_(torch.randn(q.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(step)).bfloat16())
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref, _, bound = S.reference(vals(kv), q, new, cur, tables, 0.1, softcap=20.0, window=500,
                                    first_key=first, eps_p=EPS_P[fmt])
        S.within(out, ref, bound, f"{fmt} step {step}")
        assert pa.read_error(ws) == 0


def test_two_calls_at_once_with_their_own_workspaces():
    a = build("bf16", [200], [800], 2, 4, 128, seed=1)
    b = build("bf16", [3], [4000], 1, 4, 128, seed=2)
    oa, _ = pa.prefill(*a, 0.1, max_seq_len=800)
    ob, _ = pa.prefill(*b, 0.1, max_seq_len=4000)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        got.append((pa.prefill(*a, 0.1, max_seq_len=800, stream=s1), pa.prefill(*b, 0.1, max_seq_len=4000, stream=s2)))
    torch.cuda.synchronize()
    for (x, _), (y, _) in got:
        assert torch.equal(x.view(torch.int16), oa.view(torch.int16))
        assert torch.equal(y.view(torch.int16), ob.view(torch.int16))
