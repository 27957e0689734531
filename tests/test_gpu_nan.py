"""NaN in queries and in visible keys and values reaches the rows that meet it
(output and lse), and no other, in pa_prefill and pa_decode_scored."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import score_helpers as S
from tests import test_gpu_prefill as P
from tests import test_gpu_scored as C

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def spoil_key(kv, page, row, head):
    """NaN in one key of one kv head."""
    if kv.dtype == "int8":
        kv.k_scale[page, head, row] = NAN
    elif kv.dtype == "bf16":
        kv.k_cache[page, head, row, 3] = NAN
    elif kv.dtype == "fp8":
        kv.k_cache[page, head, row, 3] = 0x7F
    else:
        kv.k_scale[page, head, row, 0] = 0x7F


def options(opt, hq):
    return dict(plain=dict(), cap=dict(softcap=30.0), bias=dict(slopes=P.slopes(hq)),
                both=dict(softcap=30.0, slopes=P.slopes(hq)))[opt]


# one pass, split keys, and (a kernel of each kind) a last round in pieces
SHAPES = [([200, 70], [700, 70], 2, 4), ([9, 2], [4000, 3000], 1, 4), ([320], [8300], 8, 8)]
KERNELS = [("bf16", 128), ("bf16", 256), ("int8", 256), ("fp8", 128), ("nvfp4", 256)]
CASES = [(f, D, o, s) for f, D in KERNELS for o in ("plain", "cap", "bias", "both") for s in (0, 1)]


@pytest.mark.parametrize("fmt,D,opt,shape", CASES + [("bf16", 256, "cap", 2), ("int8", 256, "plain", 2)])
def test_prompts(fmt, D, opt, shape):
    new, lens, hkv, G = SHAPES[shape]
    kv, q, starts, tables, sl = P.build(fmt, new, lens, hkv, G, D)
    o = options(opt, hkv * G)
    ref, rl, bound = S.reference(P.vals(kv), q, new, lens, tables, 0.1, eps_p=P.EPS_P[fmt],
                                 v_unit=kv.v_scale.clone() if fmt == "int8" else None, **o)
    # a query head of token 1, and a key that the last two tokens of the first sequence see
    # (position lens - 2), of kv head 0
    q[1, 1, 5] = NAN
    at = lens[0] - 2
    spoil_key(kv, int(tables[0, at // 16]), at % 16, 0)
    out, lse, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, score=pa.Score(**o), out_fp32=True, return_lse=True,
                              max_seq_len=max(lens))
    assert pa.read_error(ws) == 0
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
    bad[1, 1] = True
    bad[new[0] - 2:new[0], :G] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    S.within(out[~bad], ref[~bad], bound[~bad])
    S.lse_within(lse[~bad], rl[~bad])


@pytest.mark.parametrize("opt", ["plain", "cap", "both"])
@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 256), ("int8", 256), ("fp8", 128)])
def test_a_prompts_values(fmt, D, opt):
    """A NaN value of the first key, which every query sees: its dim of every row."""
    new, lens = [130], [500]
    kv, q, starts, tables, sl = P.build(fmt, new, lens, 2, 4, D)
    page = int(tables[0, 0])
    if fmt == "int8":
        kv.v_scale[page, 0, 0] = NAN
    elif fmt == "bf16":
        kv.v_cache[page, 0, 0, 7] = NAN
    else:
        kv.v_cache[page, 0, 0, 7] = 0x7F
    out, _ = pa.prefill(kv, q, starts, tables, sl, 0.1, score=pa.Score(**options(opt, 8)), out_fp32=True, max_seq_len=500)
    dims = range(D) if fmt == "int8" else [7]
    bad = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    bad[:, :4, list(dims)] = True
    assert torch.equal(out.isnan(), bad)


# planned and merged, merged by a warp a row (windows of many rows), one launch
DECODES = [([3000, 40, 700], 2, 2, {}), ([2000] * 40, 2, 2, dict(window=1000)), ([900, 300], 1, 5, {}), ([60, 9], 2, 5, {})]


@pytest.mark.parametrize("opt", ["plain", "cap", "both"])
@pytest.mark.parametrize("fmt,G,D", [("bf16", 4, 128), ("bf16", 3, 256), ("int8", 4, 256), ("fp8", 8, 128), ("nvfp4", 2, 256)])
@pytest.mark.parametrize("lens,hkv,kernel,extra", DECODES)
def test_scored_decode(fmt, G, D, opt, lens, hkv, kernel, extra):
    kv, q, tables, sl = C.build(fmt, lens, hkv, G, D)
    o = dict(options(opt, hkv * G), **extra)
    ref, rl, bound = S.reference(C.vals(kv), q[:, 0], [1] * len(lens), lens, tables, 0.1, eps_p=C.EPS_P[fmt],
                                 v_unit=kv.v_scale.clone() if fmt == "int8" else None, **o)
    # one query head of the last sequence, and a key of the first, of the last kv head
    q[-1, 0, 0, 5] = NAN
    at = lens[0] - 20
    spoil_key(kv, int(tables[0, at // 16]), at % 16, hkv - 1)
    out, lse, ws = pa.decode_scored(kv, q, tables, sl, 0.1, score=pa.Score(**o), out_fp32=True, return_lse=True,
                                    max_seq_len=max(lens), kernel=kernel)
    assert pa.read_error(ws) == 0
    bad = torch.zeros(out.shape[:1] + out.shape[2:3], dtype=torch.bool, device=DEV)
    bad[-1, 0] = True
    bad[0, (hkv - 1) * G:] = True
    assert out[:, 0][bad].isnan().all() and lse[:, 0][bad].isnan().all()
    S.within(out[:, 0][~bad], ref[~bad], bound[~bad])
    S.lse_within(lse[:, 0][~bad], rl[~bad])


@pytest.mark.parametrize("kernel", [2, 5])
def test_a_key_that_is_the_only_one_seen(kernel):
    """Every part of the row is empty or NaN."""
    lens = [700, 1]
    kv, q, tables, sl = C.build("bf16", lens, 2, 4, 128)
    for b, n in enumerate(lens):
        kv.k_cache[int(tables[b, (n - 1) // 16]), :, (n - 1) % 16] = NAN
    out, lse, _ = pa.decode_scored(kv, q, tables, sl, 0.1, score=pa.Score(window=1), return_lse=True, max_seq_len=700,
                                   kernel=kernel)
    assert out.isnan().all() and lse.isnan().all()
