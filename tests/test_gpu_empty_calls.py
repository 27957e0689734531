"""Calls without tokens or sequences leave a workspace whose flags are their own:
none, whatever an earlier call or the memory left there."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import test_gpu_prefill as P
from tests import test_gpu_scored as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


def flagged():
    """Arguments of a prompt of two sequences, and a workspace with its flag set."""
    kv, q, starts, tables, sl = P.build("bf16", [20, 30], [120, 64], 2, 4, 128)
    bad = tables.clone()
    bad[0, 3] = -7
    _, ws = pa.prefill(kv, q, starts, bad, sl, 0.1, max_seq_len=120)
    assert pa.read_error(ws) == pa.PA_ERRF_BAD_BLOCK_ID
    return (kv, q, starts, tables, sl), ws


def test_prompts_without_tokens_or_sequences():
    (kv, q, starts, tables, sl), ws = flagged()
    out, got = pa.prefill(kv, q[:0], starts * 0, tables, sl, 0.1, max_seq_len=120, workspace=ws)
    assert out.shape[0] == 0 and got.data_ptr() == ws.data_ptr() and pa.read_error(ws) == 0
    _, ws = flagged()
    out, got = pa.prefill(kv, q, starts[:1], tables[:0], sl[:0], 0.1, out=torch.full_like(q, 7.0), max_seq_len=120,
                          workspace=ws)
    assert (out == 7.0).all() and pa.read_error(ws) == 0
    # a workspace that the call makes itself, of memory that held something
    old = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    del old
    _, ws = pa.prefill(kv, q[:0], starts * 0, tables, sl, 0.1, max_seq_len=120)
    assert pa.read_error(ws) == 0


@pytest.mark.parametrize("fn", ["scored", "decode", "verify"])
def test_decode_without_sequences(fn):
    kv, q, tables, sl = C.build("bf16", [300, 200], 2, 4, 128)

    def call(n, t, ws):
        if fn == "scored":
            return pa.decode_scored(kv, q[:n], t, sl[:n], 0.1, score=pa.Score(softcap=9.0), max_seq_len=300, workspace=ws)
        x = q[:n] if fn == "decode" else q[:n].expand(-1, 4, -1, -1).contiguous()
        return (pa.decode if fn == "decode" else pa.verify)(kv, x, t, sl[:n], 0.1, max_seq_len=300, workspace=ws)
    bad = tables.clone()
    bad[0, 1] = -7
    ws = call(2, bad, None)[-1]
    assert pa.read_error(ws) == pa.PA_ERRF_BAD_BLOCK_ID
    call(0, tables[:0], ws)
    assert pa.read_error(ws) == 0


def test_captured():
    (kv, q, starts, tables, sl), ws = flagged()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.prefill(kv, q[:0], starts, tables, sl, 0.1, max_seq_len=120, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERRF_BAD_BLOCK_ID
    g.replay()
    torch.cuda.synchronize()
    assert pa.read_error(ws) == 0
