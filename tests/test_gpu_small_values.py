"""int8 caches whose value rows have small, large and unequal scales.

A weight meets its value row's scale before it is rounded to fp16, normalised
by a power of two that puts the largest scale M of the keys at hand (a tile of
128 in a prompt, a block of 16 in decode) between 1 and 2^7.  Where the product
is below fp16's normal range its rounding is off by 2^-25 in those units, that
is by 2^-25 M of the value's own, times the code: per key 2^-25 M |code|, over
the weights' sum (the weights are relative to the row's largest, so it is at
least 1).  With equal scales that is 2^-25 |v|, whatever their size: the bound
of score_helpers with the unit scale / M in the place of the scale."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import score_helpers as S
from tests import test_gpu_prefill as P
from tests import test_gpu_scored as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


def unit(scale, tables, lens, keys):
    """scale / M of every row, M the largest of the sequence's `keys` aligned keys."""
    u = torch.ones(scale.shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        for k0 in range(0, n, keys):
            pg = tables[b, k0 // 16:-(-min(n, k0 + keys) // 16)].long()
            s = scale[pg].double()                       # [pages, Hkv, 16]
            at = k0 + torch.arange(len(pg), device=DEV)[:, None, None] * 16 + torch.arange(16, device=DEV)
            M = torch.where(at < n, s, 0.0).amax((0, 2), keepdim=True)
            u[pg] = s / M
    return u


def amplitudes(kv, tables, lens, kind):
    """Scales of the value rows: `kind` times those of unit values, or drawn apart by
    pages, by tiles of 128 keys, or by rows."""
    if not isinstance(kind, str):
        kv.v_scale.copy_((kv.v_scale.float() * kind).half())
        return
    gen = torch.Generator(DEV).manual_seed(9)
    for b, n in enumerate(lens):
        pages = tables[b, :-(-n // 16)].long()
        x = torch.randint(-12, 11, (len(pages), 1, 16), device=DEV, generator=gen).float()
        if kind == "pages":
            x = x[:, :, :1]
        elif kind == "tiles":
            x = x[::8, :, :1].repeat_interleave(8, 0)[:len(pages)]
        kv.v_scale[pages] = (kv.v_scale[pages].float() * torch.exp2(x)).half()


KINDS = [2e4, 1e-2, 1e-3, 1e-4, "pages", "tiles", "rows"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,lens,hkv,G,D", [([33, 3], [8192, 3000], 1, 4, 256),      # keys split
                                              ([130, 700], [2000, 1900], 4, 8, 256),   # one pass
                                              ([300, 1000], [300, 2100], 2, 8, 128)])
@pytest.mark.parametrize("opt", ["plain", "cap", "bias"])
def test_prompts(kind, new, lens, hkv, G, D, opt):
    kv, q, starts, tables, sl = P.build("int8", new, lens, hkv, G, D)
    amplitudes(kv, tables, lens, kind)
    o = dict(softcap=30.0) if opt == "cap" else dict(slopes=P.slopes(hkv * G)) if opt == "bias" else {}
    out, lse, ws = pa.prefill(kv, q, starts, tables, sl, D ** -0.5, score=pa.Score(**o), out_fp32=True,
                              return_lse=True, max_seq_len=max(lens))
    assert pa.read_error(ws) == 0
    ref, rl, bound = S.reference(P.vals(kv), q, new, lens, tables, D ** -0.5, eps_p=S.EPS_FP16,
                                 v_unit=unit(kv.v_scale, tables, lens, 128), **o)
    S.within(out, ref, bound, f"{kind} {new} {lens}")
    S.lse_within(lse, rl)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,hkv,G,D,kernel", [([8192, 17, 3000], 2, 4, 256, 2), ([32768], 1, 8, 128, 2),
                                                 ([1000, 40], 2, 6, 256, 5), ([900, 1], 2, 3, 128, 5)])
def test_scored_decode(kind, lens, hkv, G, D, kernel):
    kv, q, tables, sl = C.build("int8", lens, hkv, G, D)
    amplitudes(kv, tables, lens, kind)
    for o in (dict(), dict(softcap=30.0, window=2000)):
        out, lse, ws = pa.decode_scored(kv, q, tables, sl, D ** -0.5, score=pa.Score(**o), out_fp32=True,
                                        return_lse=True, max_seq_len=max(lens), kernel=kernel)
        assert pa.read_error(ws) == 0
        ref, rl, bound = S.reference(C.vals(kv), q[:, 0], [1] * len(lens), lens, tables, D ** -0.5, eps_p=S.EPS_FP16,
                                     v_unit=unit(kv.v_scale, tables, lens, 16), **o)
        S.within(out[:, 0], ref, bound, f"{kind} {lens} {o}")
        S.lse_within(lse[:, 0], rl)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,lens,hkv,G,D", [(4, [8192, 17, 3000], 2, 4, 256), (8, [5000, 900], 1, 6, 256), (3, [4000, 40], 2, 4, 128)])
def test_verify(kind, m, lens, hkv, G, D):
    kv, q, starts, tables, sl = P.build("int8", [m] * len(lens), lens, hkv, G, D)
    amplitudes(kv, tables, lens, kind)
    out, lse, ws = pa.verify(kv, q.view(len(lens), m, hkv * G, D), tables, sl, D ** -0.5, out_fp32=True, return_lse=True,
                             max_seq_len=max(lens))
    assert pa.read_error(ws) == 0
    ref, rl, bound = S.reference(P.vals(kv), q, [m] * len(lens), lens, tables, D ** -0.5, eps_p=S.EPS_FP16,
                                 v_unit=unit(kv.v_scale, tables, lens, 16))
    S.within(out.view(ref.shape), ref, bound, f"{kind} {lens}")
    S.lse_within(lse.view(rl.shape), rl)
