"""pa_latent_prefill where a CTA takes many items one after another, among them items that
copy queries and multiply nothing; against the formula in 64 bits."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import latent_helpers as L
from tests.test_gpu_latent_attention import SCALE, prefill_case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def check(new, keys, H, causal, repeats, seed=0):
    q, kn, kr, v = prefill_case(new, keys, H, seed=seed)
    qs, ks = L.starts_of(new), L.starts_of(keys)
    ref, rl, bound = L.prefill_reference(q, kn, kr, v, new, keys, SCALE, causal)
    ws = None
    for _ in range(repeats):
        o, lse, ws = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, causal=causal, out_fp32=True, return_lse=True,
                                       workspace=ws)
        L.within(o, ref, bound, f"{len(new)} sequences, {H} heads, causal {causal}")
        L.lse_within(lse, rl)
        assert pa.read_error(ws) == 0
        ob, _ = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, causal=causal, workspace=ws)
        assert torch.equal(ob, o.bfloat16())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,H", [(33, 24), (70, 9)])
def test_sequences_without_keys_among_many(B, H, causal):
    """Every third sequence has queries and no keys: its items only copy their queries."""
    new = [1 + (211 * i) % 520 for i in range(B)]
    keys = [0 if i % 3 == 1 else m + (97 * i) % 300 for i, m in enumerate(new)]
    assert sum(-(-m // 256) for m in new) * H > 3 * 152
    check(new, keys, H, causal, 3)


def test_all_but_one_without_keys():
    new = [200 + 3 * i for i in range(40)]
    check(new, [0] * 20 + [700] + [0] * 19, 16, False, 3)


@pytest.mark.parametrize("causal", [True, False])
def test_pieces_that_do_not_divide_the_keys(causal):
    """98 to 106 key tiles in 12 or 13 pieces, after a round of whole items: every piece has
    keys, so that every row of it has a sum."""
    new, keys, H = 1280, 13568, 32
    q, kn, kr, v = prefill_case([new], [keys], H)
    qs, ks = L.starts_of([new]), L.starts_of([keys])
    _, ws = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, causal=causal)
    ws.fill_(0xFF)
    o, lse, ws = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, causal=causal, out_fp32=True, return_lse=True, workspace=ws)
    # the workspace: 256 bytes, then for 152 x 256 rows 128 floats each, then their lse; rows of
    # [item][most pieces: 16][256]
    rows = 152 * 256
    part = ws[256 + rows * 512:256 + rows * 516].view(torch.float32)[:8 * 16 * 256].view(8, 16, 256)
    # heads in a group of 31, the items with the most keys first, then the last head's: the last
    # eight items' key tiles, in pieces of eight or more
    for item, tiles in enumerate([98, 98, 98, 106, 104, 102, 100, 98] if causal else [106] * 8):
        assert torch.isfinite(part[item, :tiles // 8]).all()
        assert torch.isnan(part[item, tiles // 8:]).all()   # (as they were)
    ref, rl, bound = L.prefill_reference(q, kn, kr, v, [new], [keys], SCALE, causal)
    L.within(o, ref, bound + 2.0 ** -20)
    L.lse_within(lse, rl)
    for _ in range(3):
        ob, _ = pa.latent_prefill(q, kn, kr, v, qs, ks, SCALE, causal=causal, workspace=ws)
        assert torch.equal(ob, o.bfloat16()) and pa.read_error(ws) == 0
