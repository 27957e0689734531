"""Host side of pa_rope_append, pa_prefill and pa_decode_scored (no GPU):
refusals with nothing launched, workspace sizes, rotary frequencies, and the
binding's own checks."""
import ctypes
import math

import pytest
import torch

from paged_kv_decode_07_gb300 import build as pabuild
from paged_kv_decode_07_gb300 import pa

FAKE = 1 << 20   # a 16-byte aligned non-null address; never dereferenced on the host


@pytest.fixture(scope="module")
def L():
    pabuild.build()
    return pa.lib()


def kv_struct(dtype=0, D=256, hkv=4, nb=128, bs=16):
    return pa._KvCache(dtype, nb, bs, hkv, D, FAKE, FAKE, FAKE, FAKE, 1.0, 1.0)


def rope_struct(**kw):
    d = dict(num_tokens=4, num_q_heads=24, q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, q_stride=24 * 256,
             k_stride=1024, v_stride=1024, q_out_stride=24 * 256, positions=FAKE, slot_mapping=FAKE,
             rot_dim=64, interleaved=0, inv_freq=FAKE, attn_factor=1.0, q_norm=None, k_norm=None, eps=1e-6)
    d.update(kw)
    return pa._Rope(**d)


def prefill_struct(**kw):
    d = dict(batch=2, num_q_heads=24, num_tokens=10, q=FAKE, q_starts=FAKE, block_tables=FAKE,
             block_table_stride=8, seq_lens=FAKE, max_seq_len=100, softmax_scale=0.06, out=FAKE,
             out_fp32=0, lse_out=None)
    d.update(kw)
    return pa._Prefill(**d)


def rope(L, kv=None, ws=None, **kw):
    return L.pa_rope_append(ctypes.byref(kv or kv_struct()), ctypes.byref(rope_struct(**kw)), ws, None)


def prefill(L, kv=None, score=None, ws=FAKE, ws_bytes=1 << 34, **kw):
    return L.pa_prefill(ctypes.byref(kv or kv_struct()), ctypes.byref(prefill_struct(**kw)),
                        None if score is None else ctypes.byref(score), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), pa.PA_ERR_INVALID_ARG), (dict(num_q_heads=-1), pa.PA_ERR_INVALID_ARG),
    (dict(q=None), pa.PA_ERR_INVALID_ARG), (dict(k=None), pa.PA_ERR_INVALID_ARG),
    (dict(v=None), pa.PA_ERR_INVALID_ARG), (dict(q_out=None), pa.PA_ERR_INVALID_ARG),
    (dict(positions=None), pa.PA_ERR_INVALID_ARG), (dict(slot_mapping=None), pa.PA_ERR_INVALID_ARG),
    (dict(inv_freq=None), pa.PA_ERR_INVALID_ARG), (dict(q=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(k=FAKE + 2), pa.PA_ERR_INVALID_ARG), (dict(q_norm=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(positions=FAKE + 1), pa.PA_ERR_INVALID_ARG), (dict(slot_mapping=FAKE + 4), pa.PA_ERR_INVALID_ARG),
    (dict(q_stride=24 * 256 + 4), pa.PA_ERR_INVALID_ARG), (dict(k_stride=1025), pa.PA_ERR_INVALID_ARG),
    (dict(v_stride=-8), pa.PA_ERR_INVALID_ARG), (dict(q_out_stride=256), pa.PA_ERR_INVALID_ARG),
    (dict(rot_dim=-32), pa.PA_ERR_INVALID_ARG), (dict(rot_dim=288), pa.PA_ERR_INVALID_ARG),
    (dict(rot_dim=48), pa.PA_ERR_UNSUPPORTED), (dict(rot_dim=33), pa.PA_ERR_UNSUPPORTED),
    (dict(attn_factor=math.nan), pa.PA_ERR_INVALID_ARG), (dict(eps=-1.0), pa.PA_ERR_INVALID_ARG),
    (dict(eps=math.inf), pa.PA_ERR_INVALID_ARG), (dict(num_tokens=1 << 30), pa.PA_ERR_UNSUPPORTED)])
def test_rope_refusals(L, kw, status):
    assert rope(L, **kw) == status


def test_rope_refuses_caches_and_accepts_an_empty_batch(L):
    assert rope(L, kv_struct(D=96)) == pa.PA_ERR_UNSUPPORTED
    assert rope(L, kv_struct(bs=32)) == pa.PA_ERR_UNSUPPORTED
    assert rope(L, ws=FAKE + 4) == pa.PA_ERR_INVALID_ARG
    assert rope(L, num_tokens=0, q=None, k=None, v=None, q_out=None, positions=None, slot_mapping=None) == pa.PA_OK
    assert L.pa_rope_append(ctypes.byref(kv_struct()), None, None, None) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), pa.PA_ERR_INVALID_ARG), (dict(num_tokens=-1), pa.PA_ERR_INVALID_ARG),
    (dict(num_q_heads=25), pa.PA_ERR_INVALID_ARG), (dict(num_q_heads=0), pa.PA_ERR_INVALID_ARG),
    (dict(num_q_heads=36), pa.PA_ERR_UNSUPPORTED), (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(q_starts=None), pa.PA_ERR_INVALID_ARG), (dict(block_tables=None), pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=None), pa.PA_ERR_INVALID_ARG), (dict(out=None), pa.PA_ERR_INVALID_ARG),
    (dict(out=FAKE + 8), pa.PA_ERR_INVALID_ARG), (dict(q_starts=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(block_table_stride=0), pa.PA_ERR_INVALID_ARG), (dict(softmax_scale=math.inf), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=-1), pa.PA_ERR_INVALID_ARG), (dict(num_tokens=1 << 28), pa.PA_ERR_UNSUPPORTED),
    (dict(ws=None), pa.PA_ERR_INVALID_ARG), (dict(ws=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(ws_bytes=100), pa.PA_ERR_WORKSPACE_TOO_SMALL), (dict(batch=0), pa.PA_OK), (dict(num_tokens=0), pa.PA_OK)])
def test_prefill_refusals(L, kw, status):
    assert prefill(L, **kw) == status


def test_prefill_refuses_too_many_heads(L):
    assert prefill(L, kv=kv_struct(hkv=65536), num_q_heads=65536) == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("score", [
    pa._Score(-1.0, 0, None, None, None), pa._Score(math.nan, 0, None, None, None),
    pa._Score(math.inf, 0, None, None, None), pa._Score(0.0, -1, None, None, None),
    pa._Score(0.0, 0, FAKE + 2, None, None), pa._Score(0.0, 0, None, FAKE + 1, None),
    pa._Score(0.0, 0, None, None, FAKE + 3)])
def test_score_refusals(L, score):
    assert prefill(L, score=score) == pa.PA_ERR_INVALID_ARG
    p = pa._Problem(2, 24, 1, FAKE, FAKE, 8, FAKE, 100, 0.06, FAKE, 0, None)
    assert L.pa_decode_scored(ctypes.byref(kv_struct()), ctypes.byref(p), ctypes.byref(score), None, FAKE, 1 << 30,
                              None) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kernel,G,status", [(1, 6, pa.PA_ERR_UNSUPPORTED), (3, 6, pa.PA_ERR_UNSUPPORTED),
                                             (4, 6, pa.PA_ERR_UNSUPPORTED), (0, 9, pa.PA_ERR_UNSUPPORTED),
                                             (9, 6, pa.PA_ERR_INVALID_ARG)])
def test_decode_scored_refusals(L, kernel, G, status):
    p = pa._Problem(2, 4 * G, 1, FAKE, FAKE, 8, FAKE, 100, 0.06, FAKE, 0, None)
    o = pa._Options(kernel, 0, 0, None, None, 0)
    assert L.pa_decode_scored(ctypes.byref(kv_struct()), ctypes.byref(p), None, ctypes.byref(o), FAKE, 1 << 30,
                              None) == status
    p.q_len = 2
    o.kernel = 0
    assert L.pa_decode_scored(ctypes.byref(kv_struct()), ctypes.byref(p), None, ctypes.byref(o), FAKE, 1 << 30,
                              None) == pa.PA_ERR_UNSUPPORTED


def test_prefill_workspace(L):
    def need(**kw):
        return L.pa_prefill_workspace_bytes(ctypes.byref(kv_struct()), ctypes.byref(prefill_struct(**kw)))
    assert need(num_tokens=100, max_seq_len=200) == 256              # one pass over the keys
    assert need(num_tokens=100000, max_seq_len=100000) < 21 << 20    # pieces of a last round at most
    split = need(num_tokens=4, max_seq_len=100000)
    assert 256 < split < 64 << 20
    assert need(num_q_heads=25) == 0 and need(batch=-1) == 0
    assert need(batch=0) == 256


def freqs(rot, **kw):
    inv, att = pa.rope_frequencies(rot, **kw)
    return inv.double(), att


def test_rope_frequencies(L):
    i = torch.arange(64, dtype=torch.float64)
    base, att = freqs(128, base=10000.0)
    want = 10000.0 ** (-2 * i / 128)
    assert att == 1.0 and ((base - want).abs() <= 2.0 ** -24 * want).all()
    lin, att = freqs(128, scaling="linear", factor=4.0)
    assert att == 1.0 and ((lin - want / 4).abs() <= 2.0 ** -24 * want).all()
    ntk, att = freqs(128, scaling="ntk", factor=8.0)
    assert att == 1.0 and ntk[0] == 1.0 and abs(ntk[-1] / (want[-1] / 8) - 1) < 1e-6
    yarn, att = freqs(128, scaling="yarn", factor=16.0, original_len=4096)
    assert abs(att - (0.1 * math.log(16.0) + 1)) < 1e-6
    turns = 4096 * want / (2 * math.pi)
    ratio = yarn / want
    assert (ratio[turns > 32 * 1.2] - 1).abs().max() < 1e-6        # fast pairs kept
    assert (ratio[turns < 1 / 1.2] - 1 / 16).abs().max() < 1e-6    # slow pairs interpolated
    mid = ratio[(turns < 32) & (turns > 1)]
    assert (mid[1:] <= mid[:-1]).all() and (mid < 1).any() and (mid > 1 / 16).any()


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, base=1.0),
                                dict(rot_dim=64, scaling="linear", factor=0.5),
                                dict(rot_dim=64, scaling="yarn", factor=4.0),
                                dict(rot_dim=64, scaling="yarn", factor=4.0, original_len=100, beta_fast=1.0),
                                dict(rot_dim=2, scaling="ntk", factor=2.0), dict(rot_dim=64, base=math.inf)])
def test_rope_frequencies_refusals(L, kw):
    with pytest.raises(pa.PaError):
        pa.rope_frequencies(**kw)
    with pytest.raises(ValueError):
        pa.rope_frequencies(64, scaling="cubic")


def _args(T=4, hq=8, hkv=2, D=128):
    z = torch.zeros
    kv = pa.KvCache("bf16", z((4, hkv, 16, D), dtype=torch.bfloat16), z((4, hkv, 16, D), dtype=torch.bfloat16))
    b16 = torch.bfloat16
    return kv, dict(q=z((T, hq, D), dtype=b16), k=z((T, hkv, D), dtype=b16), v=z((T, hkv, D), dtype=b16),
                    positions=z(T, dtype=torch.int32), slot_mapping=z(T, dtype=torch.int64), inv_freq=z(D // 2))


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros((4, 8, 128))), ("q", torch.zeros((4, 8, 64), dtype=torch.bfloat16)),
    ("k", torch.zeros((4, 1, 128), dtype=torch.bfloat16)), ("v", torch.zeros((3, 2, 128), dtype=torch.bfloat16)),
    ("k", torch.zeros((4, 128, 2), dtype=torch.bfloat16).transpose(1, 2)),
    ("positions", torch.zeros(4, dtype=torch.int64)), ("positions", torch.zeros(5, dtype=torch.int32)),
    ("slot_mapping", torch.zeros(4, dtype=torch.int32)), ("inv_freq", torch.zeros(64, dtype=torch.float64)),
    ("inv_freq", torch.zeros(128)[::2]), ("q_norm", torch.zeros(128)), ("k_norm", torch.zeros(64, dtype=torch.bfloat16)),
    ("q_out", torch.zeros((4, 8, 128)))])
def test_binding_refuses_wrong_tensors(L, name, bad):
    kv, args = _args()
    args[name] = bad
    with pytest.raises(ValueError, match=name):
        pa.rope_append(kv, **args)


def test_binding_refuses_wrong_attention_tensors(L):
    kv, a = _args()
    t, n, st = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(q=a["q"].float()), dict(q=a["q"][:, :, :64]), dict(q_starts=st.long()), dict(q_starts=st[:1]),
                dict(block_tables=t.long()), dict(seq_lens=n.long()), dict(out=a["q"].half()), dict(out=a["q"][:2]),
                dict(score=pa.Score(slopes=torch.zeros(7))), dict(score=pa.Score(first_key=n.repeat(3))),
                dict(score=pa.Score(prefix_lens=n.float()))):
        args = dict(q=a["q"], q_starts=st, block_tables=t, seq_lens=n, softmax_scale=0.1)
        args.update(bad)
        with pytest.raises(ValueError):
            pa.prefill(kv, **args)
    q = a["q"][:1, None]
    for bad in (dict(q=a["q"]), dict(seq_lens=n.repeat(2)), dict(score=pa.Score(first_key=n.repeat(2)))):
        args = dict(q=q, block_tables=t, seq_lens=n, softmax_scale=0.1)
        args.update(bad)
        with pytest.raises(ValueError):
            pa.decode_scored(kv, **args)
