"""pa_latent_decode over an FP8 cache with rotated parts of any bf16 size."""
import pytest
import torch

from paged_kv_decode_07_gb300 import pa
from tests import latent_helpers as L
from tests.test_gpu_latent_attention import SCALE

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("size", [2.0 ** 17, 2.0 ** 100, 2.0 ** -30])
@pytest.mark.parametrize("Q,H", [(1, 16), (1, 24), (2, 64), (1, 128)])
def test_rotated_parts_of_any_size(Q, H, size):
    """A scale chosen for the latents says nothing of the rotated parts stored over it."""
    lens = [300, 70, 1, 0]
    tables, nb = L.tables_for(lens)
    g = torch.Generator(DEV).manual_seed(7)
    latent, _, _ = L.pool("fp8", nb)
    rope = (torch.randn((nb, 16, 64), device=DEV, generator=g) * size).bfloat16()
    kv = pa.LatentCache("fp8", latent, rope, 2.0 ** -6)
    q = torch.randn((len(lens), Q, H, 576), device=DEV, generator=g)
    q[..., 512:] *= 2.0 ** 6 / size     # scores of the usual size
    q = q.bfloat16()
    vals = L.values("fp8", latent.clone(), rope.clone(), kv.scale)
    L.poison("fp8", latent, rope, L.used_slots(tables, lens, nb))
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    o, lse, ws = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True, return_lse=True)
    # the bound of bf16 weights, which are the coarser ones, and what fp16 adds at its low end: to the
    # latents' queries (2^-25 of the two sums of magnitudes, in the scores) and to the weights (2^-25 a key)
    ref, rl, bound = L.decode_reference("bf16", vals, q, lens, tables, SCALE)
    sums = q[..., :512].double().abs().sum(-1).amax() + vals[0][..., :512].abs().sum(-1).amax()
    low = 2 * 2.0 ** -25 * SCALE * kv.scale * sums + 2.0 ** -25 * max(lens)
    L.within(o, ref, bound + low * vals[0][..., :512].abs().amax() * kv.scale, f"{Q} {H} {size}")
    L.lse_within(lse, rl)
    assert pa.read_error(ws) == (pa.PA_ERRF_LEN_LT_QLEN if Q > 1 else 0)   # (a sequence of one token)


def test_a_written_row_is_attended():
    """latent_append stores a rotated part of 200,000 steps; latent_decode attends over it."""
    g = torch.Generator(DEV).manual_seed(8)
    T, H = 40, 20
    kv = pa.LatentCache("fp8", torch.zeros((4, 16, 512), dtype=torch.uint8, device=DEV),
                        torch.zeros((4, 16, 64), dtype=torch.bfloat16, device=DEV), 2.0 ** -16)
    rows = torch.randn((T, 576), device=DEV, generator=g)
    rows[:, :512] *= 2.0 ** -13
    rows = (rows * 3).bfloat16()
    pos = torch.arange(T, device=DEV, dtype=torch.int32)
    inv, _ = pa.rope_frequencies(64, device=DEV)
    pa.latent_append(kv, rows[:, :512], rows[:, 512:], pos, pos.long(), inv)
    assert kv.rope.abs().max() > 2e5
    q = torch.randn((1, 1, H, 576), device=DEV, generator=g).bfloat16()
    tables = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    sl = torch.tensor([T], dtype=torch.int32, device=DEV)
    o, lse, _ = pa.latent_decode(kv, q, tables, sl, SCALE, out_fp32=True, return_lse=True)
    ref, rl, bound = L.decode_reference("fp8", L.values("fp8", kv.latent, kv.rope, kv.scale), q, [T], tables, SCALE)
    L.within(o, ref, bound)
    L.lse_within(lse, rl)


@pytest.mark.parametrize("fmt,nb", [("bf16", 300_000), ("fp8", 600_000)])
def test_pages_past_four_gigabytes(fmt, nb):
    """Rows written, read back and attended in the last pages of a pool of 4.9 GB."""
    T, H = 100, 20
    g = torch.Generator(DEV).manual_seed(4)
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    kv = pa.LatentCache(fmt, torch.zeros((nb, 16, 512), dtype=dt, device=DEV),
                        torch.zeros((nb, 16, 64), dtype=torch.bfloat16, device=DEV), 1.0 if fmt == "bf16" else 2.0 ** -6)
    tables = (nb - 1 - torch.randperm(7, device=DEV, generator=g)).to(torch.int32)[None]
    t = torch.arange(T, device=DEV)
    slots = tables[0, t // 16].long() * 16 + t % 16
    rows = torch.randn((T, 576), device=DEV, generator=g).bfloat16()
    inv, _ = pa.rope_frequencies(64, device=DEV)
    pa.latent_append(kv, rows[:, :512], rows[:, 512:], t.int(), slots, inv)
    # the same rows in the first pages of a small pool
    few = pa.LatentCache(fmt, kv.latent[:8].clone(), kv.rope[:8].clone(), kv.scale)
    ids = torch.arange(7, dtype=torch.int32, device=DEV)[None]
    pa.latent_append(few, rows[:, :512], rows[:, 512:], t.int(), t, inv)
    q = torch.randn((1, 1, H, 576), device=DEV, generator=g).bfloat16()
    sl = torch.tensor([T], dtype=torch.int32, device=DEV)
    for f in (lambda c, i: pa.latent_gather(c, i, L.starts_of([T]), T), lambda c, i: pa.latent_decode(c, q, i, sl, SCALE)[:1]):
        assert all(torch.equal(x, y) and x.any() for x, y in zip(f(kv, tables), f(few, ids)))
    assert not kv.latent[:1000].any()
