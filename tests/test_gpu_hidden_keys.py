"""Keys inside a prompt that no query sees: tokens that see nothing themselves
(padding inside a packed sequence, whose slots nothing was written to) between
documents that begin behind them.  Their slots may hold anything."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import score_helpers as S
from tests import test_gpu_prefill as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
NONE = 1 << 30


def spoil(kv, page, row):
    for x, s in ((kv.k_cache, kv.k_scale), (kv.v_cache, kv.v_scale)):
        if kv.dtype == "int8":
            s[page, :, row] = float("nan")
        elif kv.dtype == "bf16":
            x[page, :, row] = float("nan")
        elif kv.dtype == "fp8":
            x[page, :, row] = 0x7F
        else:
            s[page, :, row] = 0x7F


# lengths of documents and, negative, of the padding between them
LAYOUTS = {"one": [100, -50, 106], "edges": [64, -64, 1, -1, 63, -63, 2, -190, 200], "first": [-20, 40, -3, 77],
           "all": [-300], "fine": [1, -1] * 40 + [30]}


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 256), ("int8", 128), ("fp8", 256), ("nvfp4", 128)])
@pytest.mark.parametrize("G,earlier,opt", [(4, 45, "plain"), (1, 0, "cap"), (3, 200, "cap"), (6, 2000, "plain"),
                                           (8, 45, "window"), (2, 70, "prefix")])
def test_prompts(layout, fmt, D, G, earlier, opt):
    runs, hkv = LAYOUTS[layout], 2
    T = sum(abs(r) for r in runs)
    new, lens = [T, 40], [T + earlier, 40]
    kv, q, starts, tables, sl = P.build(fmt, new, lens, hkv, G, D)
    first, at = [], earlier
    for i, r in enumerate(runs):
        first += [NONE if r < 0 else 0 if i == 0 else at] * abs(r)
        at += abs(r)
    first = torch.tensor(first + [0] * 40, dtype=torch.int32, device=DEV)
    o = dict(first_key=first)
    if opt == "cap":
        o["softcap"] = 20.0
    if opt == "window":
        o["window"] = 33
    if opt == "prefix":
        o["prefix"] = torch.tensor([earlier + T // 2, 0], dtype=torch.int32, device=DEV)
    ref, rl, bound = S.reference(P.vals(kv), q, new, lens, tables, 0.1, eps_p=P.EPS_P[fmt],
                                 v_unit=kv.v_scale.clone() if fmt == "int8" else None, **o)
    pos, f, t = torch.arange(earlier, earlier + T), first[:T].cpu(), torch.arange(earlier + T)[:, None]
    end = torch.maximum(pos + 1, torch.tensor(earlier + T // 2 if opt == "prefix" else 0))
    lo = torch.maximum(f, pos - 32) if opt == "window" else f
    hidden = ~((t >= lo) & (t < end)).any(1)
    assert hidden.any()
    for k in hidden.nonzero().flatten().tolist():
        spoil(kv, int(tables[0, k // 16]), k % 16)
    sc = pa.Score(softcap=o.get("softcap", 0.0), window=o.get("window", 0), first_key=first, prefix_lens=o.get("prefix"))
    out, lse, ws = pa.prefill(kv, q, starts, tables, sl, 0.1, score=sc, out_fp32=True, return_lse=True, max_seq_len=max(lens))
    assert pa.read_error(ws) == 0
    S.within(out, ref, bound, f"{layout} {fmt} {D} {G}")
    S.lse_within(lse, rl)
