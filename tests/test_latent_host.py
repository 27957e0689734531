"""Host side of the latent-attention entry points (no GPU): refusals with
nothing launched, workspace sizes, the binding's own checks."""
import ctypes
import math

import pytest
import torch

from paged_kv_decode_07_gb300 import build as pabuild
from paged_kv_decode_07_gb300 import pa

FAKE = 1 << 20   # a 16-byte aligned non-null address; never dereferenced on the host
BAD, UNSUP = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    pabuild.build()
    return pa.lib()


def cache(**kw):
    d = dict(dtype=0, num_blocks=64, block_size=16, latent_dim=512, rope_dim=64, latent=FAKE, rope=FAKE,
             global_scale=1.0)
    d.update(kw)
    return pa._LatentCache(**d)


def new(**kw):
    d = dict(num_tokens=4, num_q_heads=6, latent=FAKE, rope=FAKE, q=FAKE, q_out=FAKE, latent_stride=576,
             rope_stride=576, q_stride=6 * 192, q_head_stride=192, q_out_stride=6 * 64, q_out_head_stride=64,
             positions=FAKE, slot_mapping=FAKE, interleaved=0, inv_freq=FAKE, attn_factor=1.0, norm=None, eps=1e-6)
    d.update(kw)
    return pa._LatentNew(**d)


def prefill(**kw):
    d = dict(batch=2, num_heads=4, num_tokens=10, num_keys=20, q=FAKE, k_nope=FAKE, k_rope=FAKE, v=FAKE,
             q_stride=4 * 192, q_head_stride=192, k_stride=1024, k_head_stride=256, k_rope_stride=64, v_stride=1024,
             v_head_stride=256, q_starts=FAKE, kv_starts=FAKE, causal=1, softmax_scale=0.07, out=FAKE, out_fp32=0,
             lse_out=None)
    d.update(kw)
    return pa._LatentPrefill(**d)


def problem(**kw):
    d = dict(batch=2, num_heads=20, q_len=1, q=FAKE, block_tables=FAKE, block_table_stride=8, seq_lens=FAKE,
             max_seq_len=128, softmax_scale=0.07, out=FAKE, out_fp32=0, lse_out=None)
    d.update(kw)
    return pa._LatentProblem(**d)


def ref(x):
    return None if x is None else ctypes.byref(x)


def append(L, kv=None, ws=None, **kw):
    return L.pa_latent_append(ref(kv or cache()), ref(new(**kw)), ws, None)


def gather(L, kv=None, tables=FAKE, stride=8, starts=FAKE, first=None, batch=2, rows=10, lat=FAKE, rope=FAKE, ws=None):
    return L.pa_latent_gather(ref(kv or cache()), tables, stride, starts, first, batch, rows, lat, rope, ws, None)


def expanded(L, ws=FAKE, ws_bytes=1 << 34, **kw):
    return L.pa_latent_prefill(ref(prefill(**kw)), ws, ws_bytes, None)


def decode(L, kv=None, ws=FAKE, ws_bytes=1 << 34, **kw):
    return L.pa_latent_decode(ref(kv or cache()), ref(problem(**kw)), ws, ws_bytes, None)


CACHES = [(dict(dtype=1), UNSUP), (dict(dtype=2), UNSUP), (dict(dtype=9), BAD), (dict(num_blocks=0), BAD),
          (dict(block_size=32), UNSUP), (dict(latent_dim=256), UNSUP), (dict(rope_dim=32), UNSUP),
          (dict(latent=None), BAD), (dict(rope=None), BAD), (dict(latent=FAKE + 8), BAD), (dict(rope=FAKE + 2), BAD),
          (dict(dtype=3, global_scale=math.nan), BAD), (dict(num_blocks=1 << 28), UNSUP)]


@pytest.mark.parametrize("kw,status", CACHES)
def test_caches_refused(L, kw, status):
    for f in (append, gather, decode):
        assert f(L, cache(**kw)) == status
    assert L.pa_latent_decode_workspace_bytes(ref(cache(**kw)), ref(problem())) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), BAD), (dict(num_q_heads=-1), BAD), (dict(latent=None), BAD), (dict(rope=None), BAD),
    (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(positions=None), BAD), (dict(slot_mapping=None), BAD),
    (dict(inv_freq=None), BAD), (dict(latent=FAKE + 8), BAD), (dict(rope=FAKE + 2), BAD), (dict(q=FAKE + 8), BAD),
    (dict(q_out=FAKE + 4), BAD), (dict(norm=FAKE + 2), BAD), (dict(positions=FAKE + 2), BAD),
    (dict(slot_mapping=FAKE + 4), BAD), (dict(latent_stride=580), BAD), (dict(rope_stride=-8), BAD),
    (dict(q_stride=7), BAD), (dict(q_head_stride=196), BAD), (dict(q_out_stride=32), BAD),
    (dict(q_out_head_stride=56), BAD), (dict(attn_factor=math.inf), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=math.nan), BAD), (dict(num_tokens=1 << 30), UNSUP)])
def test_append_refusals(L, kw, status):
    assert append(L, **kw) == status


def test_append_accepts_nothing(L):
    assert append(L, num_tokens=0, latent=None, rope=None, q=None, q_out=None, positions=None, slot_mapping=None) == 0
    assert append(L, ws=FAKE + 4) == BAD
    assert L.pa_latent_append(ref(cache()), None, None, None) == BAD
    assert L.pa_latent_append(None, ref(new()), None, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(tables=None), BAD), (dict(starts=None), BAD), (dict(lat=None), BAD), (dict(rope=None), BAD),
    (dict(stride=0), BAD), (dict(batch=-1), BAD), (dict(rows=-1), BAD), (dict(tables=FAKE + 2), BAD),
    (dict(starts=FAKE + 1), BAD), (dict(first=FAKE + 2), BAD), (dict(lat=FAKE + 8), BAD), (dict(rope=FAKE + 8), BAD),
    (dict(ws=FAKE + 4), BAD), (dict(batch=0), 0), (dict(rows=0), 0)])
def test_gather_refusals(L, kw, status):
    assert gather(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(num_heads=0), BAD), (dict(num_tokens=-1), BAD), (dict(num_keys=-1), BAD),
    (dict(softmax_scale=math.nan), BAD), (dict(q=None), BAD), (dict(k_nope=None), BAD), (dict(k_rope=None), BAD),
    (dict(v=None), BAD), (dict(q_starts=None), BAD), (dict(kv_starts=None), BAD), (dict(out=None), BAD),
    (dict(q=FAKE + 8), BAD), (dict(k_nope=FAKE + 2), BAD), (dict(k_rope=FAKE + 2), BAD), (dict(v=FAKE + 8), BAD),
    (dict(out=FAKE + 4), BAD), (dict(lse_out=FAKE + 2), BAD), (dict(q_stride=4 * 192 + 4), BAD),
    (dict(q_head_stride=0), BAD), (dict(k_stride=-8), BAD), (dict(k_head_stride=130), BAD),
    (dict(k_rope_stride=60), BAD), (dict(v_stride=4), BAD), (dict(v_head_stride=-128), BAD),
    (dict(num_tokens=1 << 30), UNSUP), (dict(num_tokens=1 << 26, num_heads=64), UNSUP)])
def test_prefill_refusals(L, kw, status):
    assert expanded(L, **kw) == status


def test_prefill_workspace(L):
    need = L.pa_latent_prefill_workspace_bytes(ref(prefill()))
    assert need >= 256
    assert expanded(L, ws=None) == BAD and expanded(L, ws=FAKE + 8) == BAD
    assert expanded(L, ws_bytes=need - 1) == pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert L.pa_latent_prefill_workspace_bytes(None) == 0
    assert L.pa_latent_prefill_workspace_bytes(ref(prefill(num_heads=0))) == 0
    assert L.pa_latent_prefill(None, FAKE, 1 << 30, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(num_heads=0), BAD), (dict(num_heads=129), UNSUP), (dict(q_len=0), BAD),
    (dict(q_len=17), UNSUP), (dict(max_seq_len=-1), BAD), (dict(softmax_scale=math.inf), BAD), (dict(q=None), BAD),
    (dict(block_tables=None), BAD), (dict(seq_lens=None), BAD), (dict(out=None), BAD), (dict(q=FAKE + 8), BAD),
    (dict(out=FAKE + 8), BAD), (dict(block_tables=FAKE + 2), BAD), (dict(seq_lens=FAKE + 1), BAD),
    (dict(lse_out=FAKE + 2), BAD), (dict(block_table_stride=0), BAD)])
def test_decode_refusals(L, kw, status):
    assert decode(L, **kw) == status


def test_decode_workspace(L):
    need = L.pa_latent_decode_workspace_bytes(ref(cache()), ref(problem()))
    assert need >= 256
    assert decode(L, ws=None) == BAD and decode(L, ws=FAKE + 8) == BAD
    assert decode(L, ws_bytes=need - 1) == pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert L.pa_latent_decode(ref(cache()), None, FAKE, 1 << 30, None) == BAD


def test_the_binding_names_what_it_refuses():
    bf, i32 = torch.bfloat16, torch.int32
    kv = pa.LatentCache("bf16", torch.zeros((4, 16, 512), dtype=bf), torch.zeros((4, 16, 64), dtype=bf))
    rows, ints = torch.zeros((2, 576), dtype=bf), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.latent_append(kv, rows[:, :512], rows[:, 512:], ints, ints.long(), torch.zeros(32))
    with pytest.raises(ValueError, match="CUDA device"):
        pa.latent_gather(kv, ints[None], ints, 2)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.latent_decode(kv, torch.zeros((1, 1, 4, 576), dtype=bf), ints[None], ints[:1], 0.1)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.latent_prefill(torch.zeros((2, 4, 192), dtype=bf), torch.zeros((2, 4, 128), dtype=bf), rows[:, 512:],
                          torch.zeros((2, 4, 128), dtype=bf), ints, ints, 0.1)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=64, block_table_stride=1 << 26), UNSUP),                           # 2^31 tiles of 32 keys
    (dict(batch=63, block_table_stride=1 << 26), pa.PA_ERR_WORKSPACE_TOO_SMALL),
    (dict(batch=16, block_table_stride=1 << 26, num_heads=128, q_len=16), UNSUP),   # four sets of groups
    (dict(batch=15, block_table_stride=1 << 26, num_heads=128, q_len=16), pa.PA_ERR_WORKSPACE_TOO_SMALL),
])
def test_decode_tiles_fit_32_bits(L, kw, status):
    assert L.pa_latent_decode(ref(cache()), ref(problem(**kw)), FAKE, 256, None) == status
    assert (L.pa_latent_decode_workspace_bytes(ref(cache()), ref(problem(**kw))) == 0) == (status == UNSUP)
