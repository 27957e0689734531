"""pa_decode_scored (one new token with capped, biased or windowed scores)
against the plain 64-bit form of tests/score_helpers.py."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import score_helpers as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = ["bf16", "int8", "fp8", "nvfp4"]
EPS_P = {"bf16": S.EPS_BF16_PAIR, "int8": S.EPS_FP16, "fp8": S.EPS_FP16, "nvfp4": S.EPS_FP16}


def build(fmt, lens, hkv, G, D, seed=0):
    tables, nb = S.tables_for(lens, seed=seed)
    k, v, ks, vs, g = S.make_pool(fmt, nb, hkv, D, seed)
    kv = pa.KvCache(fmt, k, v, ks, vs, g, g)
    gen = torch.Generator(DEV).manual_seed(seed + 1)
    q = (torch.randn((len(lens), 1, hkv * G, D), device=DEV, generator=gen) * 2).bfloat16()
    return kv, q, tables, torch.tensor(lens, dtype=torch.int32, device=DEV)


def vals(kv):
    return (S.values(kv.dtype, kv.k_cache, kv.k_scale, kv.k_global),
            S.values(kv.dtype, kv.v_cache, kv.v_scale, kv.v_global))


def check(fmt, lens, hkv, G, D, seed=0, kernel=0, **opt):
    kv, q, tables, sl = build(fmt, lens, hkv, G, D, seed)
    sc = pa.Score(softcap=opt.get("softcap", 0.0), slopes=opt.get("slopes"), window=opt.get("window", 0),
                  first_key=opt.get("first_key"))
    out, lse, ws = pa.decode_scored(kv, q, tables, sl, D ** -0.5, score=sc, out_fp32=True, return_lse=True,
                                    max_seq_len=max(max(lens), 1), kernel=kernel)
    assert pa.read_error(ws) == 0
    ref, rl, bound = S.reference(vals(kv), q[:, 0], [1] * len(lens), lens, tables, D ** -0.5, eps_p=EPS_P[fmt],
                                v_unit=kv.v_scale if fmt == "int8" else None, **opt)
    S.within(out[:, 0], ref, bound, f"{fmt} {lens} {hkv} {G} {D}")
    S.lse_within(lse[:, 0], rl)
    b16, _ = pa.decode_scored(kv, q, tables, sl, D ** -0.5, score=sc, max_seq_len=max(max(lens), 1), kernel=kernel)
    assert torch.equal(b16.view(torch.int16), out.bfloat16().view(torch.int16))


LENS = [1, 15, 16, 17, 300, 0, 1000, 2777]


def options(opt, lens, hq):
    o = {}
    if opt in ("cap", "all"):
        o["softcap"] = 5.0
    if opt in ("bias", "all"):
        o["slopes"] = torch.linspace(0.001, 0.06, hq, device=DEV)
    if opt in ("window", "all"):
        o["window"] = 70
    if opt in ("docs", "all"):
        o["first_key"] = torch.tensor([max(0, n - 40 - 7 * i) for i, n in enumerate(lens)], dtype=torch.int32, device=DEV)
    return o


@pytest.mark.parametrize("opt", ["plain", "cap", "bias", "window", "docs", "all"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_split_decode(fmt, D, opt):
    check(fmt, LENS, 2, 4, D, **options(opt, LENS, 8))


@pytest.mark.parametrize("opt", ["plain", "cap", "bias", "window", "docs", "all"])
@pytest.mark.parametrize("fmt", FMTS)
def test_single_launch_decode(fmt, opt):
    lens = [1000, 33]
    check(fmt, lens, 2, 4, 128, kernel=5, **options(opt, lens, 8))
    check(fmt, lens, 1, 6, 256, kernel=5, **options(opt, lens, 6))


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_group_sizes(G):
    check("bf16", [700, 40], 3, G, 256, softcap=20.0, slopes=torch.linspace(0.01, 0.05, 3 * G, device=DEV))
    check("nvfp4", [2700, 40], 1, G, 128, softcap=20.0, slopes=torch.linspace(0.01, 0.05, G, device=DEV))


@pytest.mark.parametrize("fmt,G,D", [("int8", 3, 256), ("fp8", 5, 128), ("nvfp4", 7, 256), ("bf16", 5, 256)])
def test_odd_groups_split_and_single_launch(fmt, G, D):
    o = dict(softcap=20.0, slopes=torch.linspace(0.01, 0.05, 2 * G, device=DEV), window=1800)
    check(fmt, [2700, 40, 1], 2, G, D, **o)
    check(fmt, [700, 40, 1], 2, G, D, kernel=5, **o)


@pytest.mark.parametrize("cap", [300.0, 1e6, 1e15, 1e30])
@pytest.mark.parametrize("kernel", [2, 5])
def test_caps_far_above_the_scores_leave_them(cap, kernel):
    """|s| < 15 here (unit queries, keys of 128 dims: norms of 11.3 +- 0.7):
    cap tanh(s / cap) differs from s by s^3 / (3 cap^2), 1.3e-2 at cap = 300 (bounded
    as a score's error, twice that of A) and below 2e-9 for the others."""
    kv, q, tables, sl = build("bf16", [700, 40], 2, 4, 128)
    q = torch.nn.functional.normalize(q.float(), dim=-1).bfloat16()
    out, _ = pa.decode_scored(kv, q, tables, sl, 1.0, score=pa.Score(softcap=cap), out_fp32=True, max_seq_len=700,
                              kernel=kernel)
    ref, _, bound = S.reference(vals(kv), q[:, 0], [1, 1], [700, 40], tables, 1.0, eps_p=EPS_P["bf16"])
    if cap < 1e4:
        A = vals(kv)[1].abs().max()
        bound = bound + 2 * 1.3e-2 * A
    S.within(out[:, 0], ref, bound)


def test_tiny_cap_averages_the_keys():
    """Every score is at most the cap: equal weights, also for a product of 0."""
    kv, q, tables, sl = build("bf16", [300, 40], 2, 4, 128)
    q[0, 0, 1] = 0
    out, _ = pa.decode_scored(kv, q, tables, sl, 0.1, score=pa.Score(softcap=1e-40), out_fp32=True, max_seq_len=300)
    ref, _, bound = S.reference(vals(kv), q[:, 0] * 0, [1, 1], [300, 40], tables, 0.1, eps_p=EPS_P["bf16"])
    S.within(out[:, 0], ref, bound)


@pytest.mark.parametrize("B,most", [(1, 9000), (3, 5000), (40, 1500), (1024, 90), (1100, 90)])
def test_plans_of_few_and_many_sequences(B, most):
    """Lengths of 0 to `most`; windows and documents leave some sequences a few
    blocks, some one, some none."""
    r = torch.Generator().manual_seed(B)
    lens = [int(x) for x in torch.randint(0, most + 1, (B,), generator=r)]
    lens[0] = most
    first = torch.tensor([n if i % 7 == 3 else max(0, n - 200 * (i % 5)) for i, n in enumerate(lens)],
                         dtype=torch.int32, device=DEV)
    check("bf16", lens, 2, 4, 128, kernel=2)
    check("fp8", lens, 2, 2, 128, kernel=2, window=1000, softcap=20.0)
    check("bf16", lens, 1, 4, 128, kernel=2, window=500, first_key=first)


@pytest.mark.parametrize("D", [128, 256])
def test_one_long_sequence_among_many(D):
    """Rows of hundreds of partials beside rows of one, two and none."""
    lens = [50] * 10 + [40000] + [300, 0, 260] * 10
    check("bf16", lens, 2, 4, D, softcap=30.0)
    check("fp8", lens, 2, 4, D, window=8000)    # 62 partials at most
    first = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
    first[10] = 50000          # and the long one sees nothing
    check("nvfp4", lens, 1, 7, D, first_key=first)


def test_equal_windows_fill_whole_rounds():
    """64 windows of 64 or 65 blocks, four of them not filled: items of one size in
    whole rounds of the resident CTAs; the header says which rule was taken."""
    lens = [3000 + 13 * i for i in range(60)] + [900, 1000, 17, 700]
    kv, q, tables, sl = build("fp8", lens, 4, 2, 128)
    out, lse, ws = pa.decode_scored(kv, q, tables, sl, 0.1, score=pa.Score(window=1024), out_fp32=True, return_lse=True,
                                    max_seq_len=max(lens), kernel=2)
    ref, rl, bound = S.reference(vals(kv), q[:, 0], [1] * 64, lens, tables, 0.1, window=1024, eps_p=EPS_P["fp8"])
    S.within(out[:, 0], ref, bound)
    S.lse_within(lse[:, 0], rl)
    _, items, W, _, resident = ws[:20].view(torch.int32).tolist()
    assert resident > 0 and W > 8 and items <= max(resident, 256 * -(-65 // W))


@pytest.mark.parametrize("fmt", FMTS)
def test_long_cache_with_window(fmt):
    check(fmt, [40000, 17, 9001], 2, 4, 256, window=1025, softcap=50.0)


def test_rows_that_see_nothing():
    lens = [100, 200, 2000]
    first = torch.tensor([100, 199, 1 << 30], dtype=torch.int32, device=DEV)   # none, one key, none
    check("bf16", lens, 2, 4, 128, first_key=first)
    check("int8", lens, 2, 4, 256, first_key=first)
    check("fp8", [100, 200], 1, 4, 256, kernel=5, first_key=first[:2])


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("kernel", [2, 5])
def test_keys_behind_the_window_may_be_anything(fmt, kernel):
    lens, W = [301, 90], 37
    kv, q, tables, sl = build(fmt, lens, 2, 4, 128)
    ref, rl, bound = S.reference(vals(kv), q[:, 0], [1, 1], lens, tables, 0.1, window=W, eps_p=EPS_P[fmt],
                                v_unit=kv.v_scale.clone() if fmt == "int8" else None)
    t2 = tables.clone()
    for b, n in enumerate(lens):
        for t in list(range(0, n - W)) + list(range(n, -(-n // 16) * 16)):
            pg = int(tables[b, t // 16])
            for x, s in ((kv.k_cache, kv.k_scale), (kv.v_cache, kv.v_scale)):
                if fmt == "int8":
                    s[pg, :, t % 16] = float("nan")
                elif fmt == "bf16":
                    x[pg, :, t % 16] = float("nan")
                else:
                    x[pg, :, t % 16] = 0x7F
        t2[b, :(n - W) // 16] = -1      # freed pages: never looked up
    out, lse, ws = pa.decode_scored(kv, q, t2, sl, 0.1, score=pa.Score(window=W), out_fp32=True, return_lse=True,
                                    max_seq_len=301, kernel=kernel)
    assert pa.read_error(ws) == 0
    S.within(out[:, 0], ref, bound)
    S.lse_within(lse[:, 0], rl)


@pytest.mark.parametrize("fmt", FMTS)
def test_plain_score_is_decode(fmt):
    kv, q, tables, sl = build(fmt, LENS, 2, 4, 256)
    a, la, _ = pa.decode(kv, q, tables, sl, 0.0625, out_fp32=True, return_lse=True, max_seq_len=2777)
    b, lb, _ = pa.decode_scored(kv, q, tables, sl, 0.0625, out_fp32=True, return_lse=True, max_seq_len=2777)
    assert torch.allclose(a, b, rtol=1e-5, atol=1e-6) and torch.allclose(la, lb, rtol=1e-6, atol=1e-6)


def test_errors_of_the_device_are_flagged():
    kv, q, tables, sl = build("bf16", [300, 200], 2, 4, 128)
    bad = tables.clone()
    bad[0, 17] = kv.k_cache.shape[0]
    sc = pa.Score(softcap=10.0, window=60)
    _, ws = pa.decode_scored(kv, q, bad, sl, 0.1, score=sc, max_seq_len=300)
    assert pa.read_error(ws) == pa.PA_ERRF_BAD_BLOCK_ID
    _, ws = pa.decode_scored(kv, q, tables, torch.tensor([-1, 10 ** 6], dtype=torch.int32, device=DEV), 0.1,
                             score=sc, max_seq_len=300)
    # the second length is clamped to the table's 19 entries, of which the last are unused ids
    assert pa.read_error(ws) == pa.PA_ERRF_NEG_LEN | pa.PA_ERRF_LEN_OVER_CAPACITY | pa.PA_ERRF_BAD_BLOCK_ID


@pytest.mark.parametrize("lens", [[1000, 300], [5000, 300]])
def test_capture_and_replay_with_new_inputs(lens):
    kv, q, tables, sl = build("fp8", lens, 2, 4, 256)
    out = torch.empty((2, 1, 8, 256), device=DEV)
    first = torch.zeros(2, dtype=torch.int32, device=DEV)
    sc = pa.Score(softcap=20.0, window=900, first_key=first)
    _, ws = pa.decode_scored(kv, q, tables, sl, 0.1, score=sc, out=out, max_seq_len=max(lens))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.decode_scored(kv, q, tables, sl, 0.1, score=sc, out=out, max_seq_len=max(lens), workspace=ws)
    for step in range(3):
        cur = [n - 10 * step for n in lens]
        sl.copy_(torch.tensor(cur, dtype=torch.int32))
        first.fill_(50 * step)
        q.copy_(torch.randn(q.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(step)).bfloat16())
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref, _, bound = S.reference(vals(kv), q[:, 0], [1, 1], cur, tables, 0.1, softcap=20.0, window=900,
                                    first_key=first, eps_p=EPS_P["fp8"])
        S.within(out[:, 0], ref, bound)
        assert pa.read_error(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "int8", "nvfp4"])
def test_wrong_caches_and_workspaces_are_refused_by_name(fmt):
    kv, q, tables, sl = build(fmt, [300, 200], 2, 4, 128)
    bad = [("v_cache", kv.v_cache[:, :1]), ("v_cache", kv.v_cache[:-1]), ("v_cache", kv.v_cache.cpu()),
           ("v_cache", kv.v_cache.transpose(0, 1).contiguous().transpose(0, 1)), ("v_cache", kv.v_cache.float()),
           ("k_cache", kv.k_cache[:, :, :8])]
    if fmt != "bf16":
        bad += [("k_scale", None), ("v_scale", kv.v_scale[:-1]), ("v_scale", kv.v_scale.float())]
    for name, t in bad:
        other = pa.KvCache(fmt, kv.k_cache, kv.v_cache, kv.k_scale, kv.v_scale, kv.k_global, kv.v_global)
        setattr(other, name, t)
        with pytest.raises(ValueError, match="cache|scale"):
            pa.decode_scored(other, q, tables, sl, 0.1, max_seq_len=300)
        starts = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
        with pytest.raises(ValueError, match="cache|scale"):
            pa.prefill(other, q[:, 0], starts, tables, sl, 0.1, max_seq_len=300)
    ws = torch.zeros((1 << 20, 2), dtype=torch.uint8, device=DEV)[:, 0]
    with pytest.raises(ValueError, match="workspace"):
        pa.decode_scored(kv, q, tables, sl, 0.1, max_seq_len=300, workspace=ws)


def test_one_token_rows_of_any_pitch_are_rotated():
    """With a single token no stride counts."""
    kv, q, tables, sl = build("bf16", [300], 2, 4, 128)
    x = torch.randn((1, 12 * 128 + 5), device=DEV).bfloat16()
    views = [x[:, i * 128 * n0:][:, :n * 128].view(1, n, 128) for i, n0, n in ((0, 1, 8), (8, 1, 2), (10, 1, 2))]
    pos = torch.tensor([7], dtype=torch.int32, device=DEV)
    slot = torch.tensor([3], dtype=torch.int64, device=DEV)
    inv, _ = pa.rope_frequencies(64, device=DEV)
    a = pa.rope_append(kv, *views, pos, slot, inv)
    b = pa.rope_append(kv, *(v.clone(memory_format=torch.contiguous_format) for v in views), pos, slot, inv)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
