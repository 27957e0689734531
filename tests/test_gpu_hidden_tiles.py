"""pa_prefill on row tiles of which no row sees a key: output 0 and lse -inf,
bit for bit, call after call, and the other rows as ever."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import score_helpers as S
from tests.test_gpu_prefill import EPS_P, build, vals

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 256), ("int8", 128), ("fp8", 256), ("nvfp4", 128)])
def test_padded_sequences_with_rows(fmt, D, softcap, fp32):
    """Three of four sequences have no keys (seq_len 0) but rows of their own."""
    B, hkv, G = 28, 2, 4
    new = [75 + 3 * b for b in range(B)]
    lens = [m if b % 4 == 0 else 0 for b, m in enumerate(new)]
    kv, q, starts, tables, sl = build(fmt, new, lens, hkv, G, D)
    row = torch.cat([torch.full((m,), n > 0) for m, n in zip(new, lens)]).to(DEV)
    ref, rl, bound = S.reference(vals(kv), q, new, lens, tables, 0.1, softcap=softcap, eps_p=EPS_P[fmt],
                                 out_eps=2.0 ** -23 if fp32 else 2.0 ** -8,
                                 v_unit=kv.v_scale if fmt == "int8" else None)
    ws = first = None
    for _ in range(30):
        out = torch.full(q.shape, 7.0, device=DEV, dtype=torch.float32 if fp32 else torch.bfloat16)
        out, lse, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, score=pa.Score(softcap=softcap), out=out,
                                  return_lse=True, max_seq_len=256, workspace=ws)
        assert pa.read_error(ws) == 0
        assert (out[~row] == 0).all() and (lse[~row] == -torch.inf).all()
        first = out if first is None else first
        assert torch.equal(out, first)
    S.within(out, ref, bound, f"{fmt} {D}")
    S.lse_within(lse, rl)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("D", [128, 256])
def test_documents_that_hide_every_key(D, fp32):
    """first_key past the queries of whole tiles, beside tiles of the same sequence
    that see their own."""
    new, lens, hkv, G = [640, 200], [640, 250], 4, 4
    kv, q, starts, tables, sl = build("bf16", new, lens, hkv, G, D)
    first = torch.zeros(840, dtype=torch.int32)
    first[128:512] = 1 << 30
    first[640:] = 1 << 30
    first[512:640] = 512
    first = first.to(DEV)
    gone = first == 1 << 30
    ref, _, bound = S.reference(vals(kv), q, new, lens, tables, 0.1, first_key=first,
                                out_eps=2.0 ** -23 if fp32 else 2.0 ** -8)
    for _ in range(30):
        out = torch.full(q.shape, 7.0, device=DEV, dtype=torch.float32 if fp32 else torch.bfloat16)
        pa.prefill(kv, q, starts, tables, sl, 0.1, score=pa.Score(first_key=first), out=out, max_seq_len=250)
        assert (out[gone] == 0).all()
    S.within(out, ref, bound, str(D))
