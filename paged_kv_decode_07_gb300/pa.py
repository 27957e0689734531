"""ctypes binding of the C ABI in include/pa.h (argument marshalling only).

Every step of the attention runs in libpa.so's CUDA kernels; this module
only turns torch tensors into pointers and sizes, picks the current CUDA
stream, and allocates outputs / workspace with torch when the caller does
not pass them.  There is no fallback: if libpa.so is missing or a call
fails, it raises.  rope_append, prefill, decode_scored and the latent_ calls
do the same in the extension _pa_py (csrc/pa_py.cpp); here only what it
declines is looked at:
arguments to refuse by name, another stream, another device.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from dataclasses import dataclass
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpa.so")
EXT_PATH = os.path.join(HERE, "_pa_py.so")

PA_OK = 0
PA_ERR_INVALID_ARG = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_WORKSPACE_TOO_SMALL = -3
PA_ERR_CUDA = -4

PA_KV_BF16, PA_KV_INT8, PA_KV_NVFP4, PA_KV_FP8 = 0, 1, 2, 3
DTYPE_CODES = {"bf16": PA_KV_BF16, "int8": PA_KV_INT8, "nvfp4": PA_KV_NVFP4, "fp8": PA_KV_FP8}

PA_ERRF_BAD_BLOCK_ID = 0x1
PA_ERRF_LEN_OVER_CAPACITY = 0x2
PA_ERRF_NEG_LEN = 0x4
PA_ERRF_LEN_LT_QLEN = 0x8
PA_ERRF_WAIT_TIMEOUT = 0x10
PA_ERRF_PLAN_OVERFLOW = 0x20
PA_ERRF_BAD_SLOT = 0x40
PA_ERRF_BAD_Q_START = 0x80

ROPE_KINDS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}

PA_TEST_EXPIRE_WAIT = 0x1

EXPORTED = ("pa_workspace_bytes", "pa_decode", "pa_verify", "pa_merge", "pa_dequant_gather",
            "pa_append_kv", "pa_block_means", "pa_sparse_workspace_bytes", "pa_decode_sparse",
            "pa_decode_wo_workspace_bytes", "pa_decode_wo",
            "pa_rope_append", "pa_rope_frequencies", "pa_decode_scored",
            "pa_prefill_workspace_bytes", "pa_prefill", "pa_latent_append", "pa_latent_gather",
            "pa_latent_prefill_workspace_bytes", "pa_latent_prefill",
            "pa_latent_decode_workspace_bytes", "pa_latent_decode",
            "pa_read_error", "pa_status_string", "pa_version")


class PaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


class _KvCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_global_scale", ctypes.c_float), ("v_global_scale", ctypes.c_float)]


class _Problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("q_len", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("block_tables", ctypes.c_void_p), ("block_table_stride", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p), ("max_seq_len", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("out_fp32", ctypes.c_int32), ("lse_out", ctypes.c_void_p)]


class _Sparse(ctypes.Structure):
    _fields_ = [("sparse_block", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("max_sparse_blocks", ctypes.c_int32), ("means", ctypes.c_void_p),
                ("selected", ctypes.c_void_p)]


class _Wo(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("hidden", ctypes.c_int32), ("y", ctypes.c_void_p),
                ("y_fp32", ctypes.c_int32), ("k_split", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("slot_mapping", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("inv_freq", ctypes.c_void_p),
                ("attn_factor", ctypes.c_float), ("q_norm", ctypes.c_void_p),
                ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float)]


class _Score(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("alibi_slopes", ctypes.c_void_p), ("first_key", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p)]


class _Prefill(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_tokens", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("q_starts", ctypes.c_void_p), ("block_tables", ctypes.c_void_p),
                ("block_table_stride", ctypes.c_int32), ("seq_lens", ctypes.c_void_p),
                ("max_seq_len", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("out", ctypes.c_void_p), ("out_fp32", ctypes.c_int32),
                ("lse_out", ctypes.c_void_p)]


class _LatentCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("latent_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("latent", ctypes.c_void_p),
                ("rope", ctypes.c_void_p), ("global_scale", ctypes.c_float)]


class _LatentNew(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("latent", ctypes.c_void_p), ("rope", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("latent_stride", ctypes.c_int64),
                ("rope_stride", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("q_out_head_stride", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("slot_mapping", ctypes.c_void_p), ("interleaved", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p), ("attn_factor", ctypes.c_float),
                ("norm", ctypes.c_void_p), ("eps", ctypes.c_float)]


class _LatentPrefill(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_tokens", ctypes.c_int32), ("num_keys", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("k_nope", ctypes.c_void_p), ("k_rope", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("k_rope_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("q_starts", ctypes.c_void_p), ("kv_starts", ctypes.c_void_p),
                ("causal", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("out", ctypes.c_void_p), ("out_fp32", ctypes.c_int32),
                ("lse_out", ctypes.c_void_p)]


class _LatentProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("q_len", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("block_tables", ctypes.c_void_p), ("block_table_stride", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p), ("max_seq_len", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("out_fp32", ctypes.c_int32), ("lse_out", ctypes.c_void_p)]


class _Options(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("split_blocks", ctypes.c_int32),
                ("target_items", ctypes.c_int32), ("event_begin", ctypes.c_void_p),
                ("event_end", ctypes.c_void_p), ("test_flags", ctypes.c_int32)]


_lib = None
_ext = None


def library_path() -> str:
    return LIB_PATH


def lib():
    """Loads libpa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        P, i32 = ctypes.c_void_p, ctypes.c_int32
        L.pa_workspace_bytes.restype = ctypes.c_size_t
        L.pa_workspace_bytes.argtypes = [P, P, P]
        for fn in ("pa_decode", "pa_verify"):
            getattr(L, fn).restype = ctypes.c_int
            getattr(L, fn).argtypes = [P, P, P, P, ctypes.c_size_t, P]
        L.pa_merge.restype = ctypes.c_int
        L.pa_merge.argtypes = [P, P, i32, i32, i32, P, i32, P, P]
        L.pa_dequant_gather.restype = ctypes.c_int
        L.pa_dequant_gather.argtypes = [P, P, i32, P, i32, i32, P, P, P, P]
        L.pa_block_means.restype = ctypes.c_int
        L.pa_block_means.argtypes = [P, P, i32, P, P, i32, i32, i32, i32, P, P, P]
        L.pa_sparse_workspace_bytes.restype = ctypes.c_size_t
        L.pa_sparse_workspace_bytes.argtypes = [P, P, P, P]
        L.pa_decode_sparse.restype = ctypes.c_int
        L.pa_decode_sparse.argtypes = [P, P, P, P, P, ctypes.c_size_t, P]
        L.pa_decode_wo_workspace_bytes.restype = ctypes.c_size_t
        L.pa_decode_wo_workspace_bytes.argtypes = [P, P, P, P]
        L.pa_decode_wo.restype = ctypes.c_int
        L.pa_decode_wo.argtypes = [P, P, P, P, P, ctypes.c_size_t, P]
        L.pa_rope_append.restype = ctypes.c_int
        L.pa_rope_append.argtypes = [P, P, P, P]
        L.pa_rope_frequencies.restype = ctypes.c_int
        L.pa_rope_frequencies.argtypes = [i32, ctypes.c_double, i32, ctypes.c_double, i32,
                                          ctypes.c_double, ctypes.c_double, P, P]
        L.pa_decode_scored.restype = ctypes.c_int
        L.pa_decode_scored.argtypes = [P, P, P, P, P, ctypes.c_size_t, P]
        L.pa_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.pa_prefill_workspace_bytes.argtypes = [P, P]
        L.pa_prefill.restype = ctypes.c_int
        L.pa_prefill.argtypes = [P, P, P, P, ctypes.c_size_t, P]
        L.pa_latent_append.restype = ctypes.c_int
        L.pa_latent_append.argtypes = [P, P, P, P]
        L.pa_latent_gather.restype = ctypes.c_int
        L.pa_latent_gather.argtypes = [P, P, i32, P, P, i32, i32, P, P, P, P]
        L.pa_latent_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.pa_latent_prefill_workspace_bytes.argtypes = [P]
        L.pa_latent_prefill.restype = ctypes.c_int
        L.pa_latent_prefill.argtypes = [P, P, ctypes.c_size_t, P]
        L.pa_latent_decode_workspace_bytes.restype = ctypes.c_size_t
        L.pa_latent_decode_workspace_bytes.argtypes = [P, P]
        L.pa_latent_decode.restype = ctypes.c_int
        L.pa_latent_decode.argtypes = [P, P, P, ctypes.c_size_t, P]
        L.pa_append_kv.restype = ctypes.c_int
        L.pa_append_kv.argtypes = [P, P, P, i32, P, P, P]
        L.pa_read_error.restype = ctypes.c_int
        L.pa_read_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), P]
        L.pa_status_string.restype = ctypes.c_char_p
        L.pa_status_string.argtypes = [ctypes.c_int]
        L.pa_version.restype = ctypes.c_int
        L.pa_version.argtypes = []
        _lib = L
    return _lib


def _fast():
    """The extension, with the entry points of the loaded library."""
    global _ext
    if _ext is None:
        L = lib()
        if not os.path.exists(EXT_PATH):
            raise RuntimeError(
                f"{EXT_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        loader = importlib.machinery.ExtensionFileLoader("_pa_py", EXT_PATH)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_pa_py", loader))
        loader.exec_module(ext)
        ext.entry_points(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "pa_rope_append", "pa_prefill", "pa_prefill_workspace_bytes", "pa_decode_scored",
            "pa_workspace_bytes", "pa_latent_append", "pa_latent_gather", "pa_latent_prefill",
            "pa_latent_prefill_workspace_bytes", "pa_latent_decode",
            "pa_latent_decode_workspace_bytes")))
        _ext = ext
    return _ext


def status_string(status: int) -> str:
    return lib().pa_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class KvCache:
    """The paged KV pool (tensors on the device)."""
    dtype: str
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    k_global: float = 1.0
    v_global: float = 1.0
    block_size: int = 16

    @classmethod
    def from_workload(cls, wl):
        return cls(wl.dtype, wl.k_cache, wl.v_cache, wl.k_scale, wl.v_scale, wl.k_global,
                   wl.v_global)

    @property
    def head_dim(self) -> int:
        return int(self.k_cache.shape[3]) * (2 if self.dtype == "nvfp4" else 1)

    @property
    def num_kv_heads(self) -> int:
        return int(self.k_cache.shape[1])

    def struct(self) -> _KvCache:
        return _KvCache(DTYPE_CODES[self.dtype], int(self.k_cache.shape[0]), self.block_size,
                        self.num_kv_heads, self.head_dim, _ptr(self.k_cache), _ptr(self.v_cache),
                        _ptr(self.k_scale), _ptr(self.v_scale), float(self.k_global),
                        float(self.v_global))


def _options(kernel=0, split_blocks=0, target_items=0, events=None, test_flags=0):
    eb = ee = None
    if events is not None:
        eb = ctypes.c_void_p(events[0].cuda_event)
        ee = ctypes.c_void_p(events[1].cuda_event)
    return _Options(int(kernel), int(split_blocks), int(target_items), eb, ee, int(test_flags))


def _problem(kv: KvCache, q, block_tables, seq_lens, softmax_scale, out, lse, max_seq_len):
    B, Q, Hq, D = q.shape
    return _Problem(B, Hq, Q, _ptr(q), _ptr(block_tables), int(block_tables.shape[1]),
                    _ptr(seq_lens), int(max_seq_len), float(softmax_scale), _ptr(out),
                    1 if out.dtype == torch.float32 else 0, _ptr(lse))


def workspace_bytes(kv: KvCache, batch: int, q_len: int, num_q_heads: int, max_seq_len: int,
                    kernel=0, split_blocks=0, target_items=0) -> int:
    p = _Problem(batch, num_q_heads, q_len, None, None, 1, None, int(max_seq_len), 1.0, None, 0,
                 None)
    o = _options(kernel, split_blocks, target_items)
    return int(lib().pa_workspace_bytes(ctypes.byref(kv.struct()), ctypes.byref(p), ctypes.byref(o)))


def _attend(fn_name, kv, q, block_tables, seq_lens, softmax_scale, *, out=None, out_fp32=False,
            return_lse=False, max_seq_len=None, workspace=None, kernel=0, split_blocks=0,
            target_items=0, events=None, stream=None, test_flags=0):
    B, Q, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, Q, Hq, D), dtype=torch.float32 if out_fp32 else torch.bfloat16,
                          device=q.device)
    lse = torch.empty((B, Q, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    if max_seq_len is None:
        max_seq_len = int(block_tables.shape[1]) * kv.block_size
    opts = _options(kernel, split_blocks, target_items, events, test_flags)
    kvs = kv.struct()
    prob = _problem(kv, q, block_tables, seq_lens, softmax_scale, out, lse, max_seq_len)
    need = int(lib().pa_workspace_bytes(ctypes.byref(kvs), ctypes.byref(prob), ctypes.byref(opts)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = getattr(lib(), fn_name)(ctypes.byref(kvs), ctypes.byref(prob), ctypes.byref(opts),
                                 _ptr(workspace), workspace.numel(), _stream(stream))
    if st != PA_OK:
        raise PaError(fn_name, st)
    return (out, lse, workspace) if return_lse else (out, workspace)


def decode(kv: KvCache, q, block_tables, seq_lens, softmax_scale, **kw):
    """q bf16 [B, 1, Hq, D] -> (out [B, 1, Hq, D], [lse,] workspace)."""
    return _attend("pa_decode", kv, q, block_tables, seq_lens, softmax_scale, **kw)


def verify(kv: KvCache, q, block_tables, seq_lens, softmax_scale, **kw):
    """q bf16 [B, Q, Hq, D] (Q new tokens, causal) -> (out, [lse,] workspace)."""
    return _attend("pa_verify", kv, q, block_tables, seq_lens, softmax_scale, **kw)


def merge(part_out: torch.Tensor, part_lse: torch.Tensor, *, out_fp32=False, return_lse=False,
          stream=None):
    """part_out fp32 [S, R, D], part_lse fp32 [S, R] -> out [R, D] (+ lse [R])."""
    S, R, D = part_out.shape
    out = torch.empty((R, D), dtype=torch.float32 if out_fp32 else torch.bfloat16,
                      device=part_out.device)
    lse = torch.empty((R,), dtype=torch.float32, device=part_out.device) if return_lse else None
    st = lib().pa_merge(_ptr(part_out), _ptr(part_lse), S, R, D, _ptr(out), 1 if out_fp32 else 0,
                        _ptr(lse), _stream(stream))
    if st != PA_OK:
        raise PaError("pa_merge", st)
    return (out, lse) if return_lse else out


def dequant_gather(kv: KvCache, block_tables, seq_lens, max_len: int, workspace=None, stream=None):
    """-> (k, v) fp32 [B, Hkv, max_len, D] through the table, dequantised."""
    B = int(block_tables.shape[0])
    shape = (B, kv.num_kv_heads, max_len, kv.head_dim)
    k = torch.empty(shape, dtype=torch.float32, device=kv.k_cache.device)
    v = torch.empty(shape, dtype=torch.float32, device=kv.k_cache.device)
    st = lib().pa_dequant_gather(ctypes.byref(kv.struct()), _ptr(block_tables),
                                 int(block_tables.shape[1]), _ptr(seq_lens), B, int(max_len),
                                 _ptr(k), _ptr(v), _ptr(workspace), _stream(stream))
    if st != PA_OK:
        raise PaError("pa_dequant_gather", st)
    return k, v


def block_means(kv: KvCache, block_tables, seq_lens, sparse_block: int, max_sparse_blocks: int,
                first=None, count=0, means=None, workspace=None, stream=None):
    """Mean keys of sparse blocks first[b] .. first[b] + count - 1 (count 0 =
    all) of every sequence, fp32 [B, max_sparse_blocks, Hkv, D] (other
    entries untouched; a new tensor starts at 0)."""
    B = int(block_tables.shape[0])
    if means is None:
        means = torch.zeros((B, max_sparse_blocks, kv.num_kv_heads, kv.head_dim),
                            dtype=torch.float32, device=kv.k_cache.device)
    st = lib().pa_block_means(ctypes.byref(kv.struct()), _ptr(block_tables),
                              int(block_tables.shape[1]), _ptr(seq_lens), _ptr(first),
                              int(count), B, int(sparse_block), int(max_sparse_blocks), _ptr(means),
                              _ptr(workspace), _stream(stream))
    if st != PA_OK:
        raise PaError("pa_block_means", st)
    return means


def _sparse(means, sparse_block, top_k, selected):
    return _Sparse(int(sparse_block), int(top_k), int(means.shape[1]), _ptr(means), _ptr(selected))


def sparse_workspace_bytes(kv: KvCache, batch: int, num_q_heads: int, max_seq_len: int, means,
                           sparse_block: int, top_k: int, kernel=0) -> int:
    p = _Problem(batch, num_q_heads, 1, None, None, 1, None, int(max_seq_len), 1.0, None, 0, None)
    sp = _sparse(means, sparse_block, top_k, None)
    o = _options(kernel)
    return int(lib().pa_sparse_workspace_bytes(ctypes.byref(kv.struct()), ctypes.byref(p),
                                               ctypes.byref(sp), ctypes.byref(o)))


def decode_sparse(kv: KvCache, q, block_tables, seq_lens, softmax_scale, means, sparse_block: int,
                  top_k: int, *, out=None, out_fp32=False, return_lse=False, return_selected=False,
                  max_seq_len=None, workspace=None, kernel=0, split_blocks=0, target_items=0,
                  events=None, stream=None):
    """Block-sparse decode: q bf16 [B, 1, Hq, D]; means from block_means.
    Returns (out, [lse,] [selected int32 [B, Hkv, top_k],] workspace)."""
    B, Q, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, Q, Hq, D), dtype=torch.float32 if out_fp32 else torch.bfloat16,
                          device=q.device)
    lse = torch.empty((B, Q, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    sel = (torch.empty((B, kv.num_kv_heads, top_k), dtype=torch.int32, device=q.device)
           if return_selected else None)
    if max_seq_len is None:
        max_seq_len = min(int(block_tables.shape[1]) * kv.block_size,
                          int(means.shape[1]) * int(sparse_block))
    opts = _options(kernel, split_blocks, target_items, events)
    kvs = kv.struct()
    prob = _problem(kv, q, block_tables, seq_lens, softmax_scale, out, lse, max_seq_len)
    sp = _sparse(means, sparse_block, top_k, sel)
    need = int(lib().pa_sparse_workspace_bytes(ctypes.byref(kvs), ctypes.byref(prob),
                                               ctypes.byref(sp), ctypes.byref(opts)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = lib().pa_decode_sparse(ctypes.byref(kvs), ctypes.byref(prob), ctypes.byref(sp),
                                ctypes.byref(opts), _ptr(workspace), workspace.numel(),
                                _stream(stream))
    if st != PA_OK:
        raise PaError("pa_decode_sparse", st)
    res = [out]
    if return_lse:
        res.append(lse)
    if return_selected:
        res.append(sel)
    res.append(workspace)
    return tuple(res)


def decode_wo(kv: KvCache, q, block_tables, seq_lens, softmax_scale, w_o, *, y=None,
              y_fp32=False, out=None, return_lse=False, k_split=0, max_seq_len=None,
              workspace=None, kernel=0, split_blocks=0, target_items=0, events=None,
              stream=None):
    """Attention (q_len 1: decode, > 1: verify) and the output projection
    y = o . W_O in one call.  w_o bf16 [Hq * D, hidden]; returns (y
    [B * Q, hidden], [lse,] workspace); `out` (fp32 [B, Q, Hq, D]) receives o."""
    B, Q, Hq, D = q.shape
    hidden = int(w_o.shape[1])
    assert w_o.dtype == torch.bfloat16 and w_o.is_contiguous() and int(w_o.shape[0]) == Hq * D
    if y is None:
        y = torch.empty((B * Q, hidden), dtype=torch.float32 if y_fp32 else torch.bfloat16,
                        device=q.device)
    y_fp32 = y.dtype == torch.float32
    if out is not None:
        assert out.dtype == torch.float32
    lse = torch.empty((B, Q, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    if max_seq_len is None:
        max_seq_len = int(block_tables.shape[1]) * kv.block_size
    opts = _options(kernel, split_blocks, target_items, events)
    kvs = kv.struct()
    prob = _Problem(B, Hq, Q, _ptr(q), _ptr(block_tables), int(block_tables.shape[1]),
                    _ptr(seq_lens), int(max_seq_len), float(softmax_scale), _ptr(out), 1,
                    _ptr(lse))
    wo = _Wo(_ptr(w_o), hidden, _ptr(y), 1 if y_fp32 else 0, int(k_split))
    need = int(lib().pa_decode_wo_workspace_bytes(ctypes.byref(kvs), ctypes.byref(prob),
                                                  ctypes.byref(wo), ctypes.byref(opts)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = lib().pa_decode_wo(ctypes.byref(kvs), ctypes.byref(prob), ctypes.byref(wo),
                            ctypes.byref(opts), _ptr(workspace), workspace.numel(),
                            _stream(stream))
    if st != PA_OK:
        raise PaError("pa_decode_wo", st)
    return (y, lse, workspace) if return_lse else (y, workspace)


def append_kv(kv: KvCache, k_new, v_new, slot_mapping, workspace=None, stream=None):
    """Quantise-on-write of new tokens into the pool (in place).  k_new /
    v_new bf16 [T, Hkv, D]; slot_mapping int64 [T] (-1 = padded row)."""
    T = int(slot_mapping.shape[0])
    if T:
        assert k_new.dtype == torch.bfloat16 and v_new.dtype == torch.bfloat16
        assert slot_mapping.dtype == torch.int64
        assert tuple(k_new.shape) == (T, kv.num_kv_heads, kv.head_dim) == tuple(v_new.shape)
        assert k_new.is_contiguous() and v_new.is_contiguous() and slot_mapping.is_contiguous()
    st = lib().pa_append_kv(ctypes.byref(kv.struct()), _ptr(k_new), _ptr(v_new), T,
                            _ptr(slot_mapping), _ptr(workspace), _stream(stream))
    if st != PA_OK:
        raise PaError("pa_append_kv", st)


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: Optional[str] = None,
                     factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device="cpu"):
    """Inverse frequencies fp32 [rot_dim / 2] for rope_append and the factor
    its rotated pairs are scaled by.  scaling: None, "linear", "ntk" or
    "yarn" (needs original_len, the length the model was trained on)."""
    if scaling not in ROPE_KINDS:
        raise ValueError(f"scaling must be one of {list(ROPE_KINDS)}: got {scaling!r}")
    inv = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float32)
    att = ctypes.c_float(1.0)
    st = lib().pa_rope_frequencies(int(rot_dim), float(base), ROPE_KINDS[scaling], float(factor),
                                   int(original_len), float(beta_fast), float(beta_slow),
                                   _ptr(inv), ctypes.byref(att))
    if st != PA_OK:
        raise PaError("pa_rope_frequencies", st)
    return inv.to(device), float(att.value)


_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _need(t, name, dtype, shape, idx, strided=False):
    """Raises ValueError unless the tensor has this type, shape, device index
    (-1: the CPU) and layout.  strided: [tokens, heads, head_dim], the tokens
    any distance apart."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor: got {type(t).__name__}")
    if t.dtype is not dtype or t.shape != shape or t.get_device() != idx:
        where = "cpu" if idx < 0 else f"cuda:{idx}"
        raise ValueError(f"{name} must be {dtype} {list(shape)} on {where}: got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    if not t.is_contiguous():
        st = t.stride()
        if not strided or st[2] != 1 or (shape[1] > 1 and st[1] != shape[2]):
            raise ValueError(f"{name} must be contiguous{' within a token' if strided else ''}: "
                             f"got strides {st}")


def _need_cache(kv, idx):
    """The cache's arrays: one shape and element size (whatever the bytes are called)."""
    if idx < 0:
        raise ValueError("the KV cache must be on a CUDA device")
    k = kv.k_cache
    if k.dim() != 4:
        raise ValueError(f"k_cache must have four dimensions: got {list(k.shape)}")
    pages = (k.shape[0], k.shape[1], kv.block_size, k.shape[3])
    size = 2 if kv.dtype == "bf16" else 1
    arrays = [("k_cache", k, pages, size), ("v_cache", kv.v_cache, pages, size)]
    if kv.dtype == "int8":
        arrays += [("k_scale", kv.k_scale, pages[:3], 2), ("v_scale", kv.v_scale, pages[:3], 2)]
    elif kv.dtype == "nvfp4":
        blocks = pages[:3] + (pages[3] // 8,)
        arrays += [("k_scale", kv.k_scale, blocks, 1), ("v_scale", kv.v_scale, blocks, 1)]
    for name, t, shape, size in arrays:
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor: got {type(t).__name__}")
        if t.shape != shape or t.element_size() != size or t.get_device() != idx or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {list(shape)} of {size}-byte elements on "
                             f"cuda:{idx}: got {t.dtype} {list(t.shape)} on {t.device}")


def _need_out(out, shape, idx):
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.dtype not in (_F32, _BF16):
            raise ValueError("out must be a bf16 or fp32 tensor")
        _need(out, "out", out.dtype, shape, idx)


def _need_workspace(ws, idx):
    if ws is not None and (not isinstance(ws, torch.Tensor) or ws.get_device() != idx or
                           not ws.is_contiguous() or ws.nbytes < 256):
        raise ValueError(f"workspace must be a contiguous tensor of at least 256 bytes on cuda:{idx}")


def _elsewhere(idx, stream):
    """A context for a call that the extension declined although its tensors
    are as they should be: its stream or its device is not the current one
    (outputs are then allocated there too)."""
    if stream is not None:
        if stream.device.index != idx:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{idx}")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != idx:
        return torch.cuda.device(idx)
    raise ValueError("a number among the arguments is none, or out of range")


def rope_append(kv: KvCache, q, k, v, positions, slot_mapping, inv_freq, *, interleaved=False,
                attn_factor=1.0, q_norm=None, k_norm=None, eps=1e-6, q_out=None, workspace=None,
                stream=None):
    """Per-head RMS norm (q_norm / k_norm bf16 [D], optional) and position
    rotation of the new tokens' queries and keys, and the quantised write of
    their keys and values into the pool (in place), in one pass.

    q bf16 [T, Hq, D], k / v bf16 [T, Hkv, D]: contiguous within a token, any
    distance between tokens (slices of one fused projection).  positions
    int32 [T]; slot_mapping int64 [T] (-1 = padded row); inv_freq fp32
    [rot_dim / 2] (rope_frequencies).  Returns the rotated queries bf16
    [T, Hq, D]; q_out=q rotates them in place."""
    if stream is None:
        r = (_ext or _fast()).rope_append(
            DTYPE_CODES[kv.dtype], kv.block_size, kv.k_cache, kv.v_cache, kv.k_scale, kv.v_scale,
            kv.k_global, kv.v_global, q, k, v, positions, slot_mapping, inv_freq, interleaved,
            attn_factor, q_norm, k_norm, eps, q_out, workspace)
        if type(r) is int:
            raise PaError("pa_rope_append", r)
        if r is not None:
            return r
    T, Hq, D = q.shape
    idx, hkv = kv.k_cache.get_device(), kv.num_kv_heads
    _need(q, "q", _BF16, (T, Hq, kv.head_dim), idx, True)
    _need(k, "k", _BF16, (T, hkv, D), idx, True)
    _need(v, "v", _BF16, (T, hkv, D), idx, True)
    _need(positions, "positions", _I32, (T,), idx)
    _need(slot_mapping, "slot_mapping", _I64, (T,), idx)
    _need(inv_freq, "inv_freq", _F32, (inv_freq.numel(),), idx)
    for t, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if t is not None:
            _need(t, name, _BF16, (D,), idx)
    if q_out is not None:
        _need(q_out, "q_out", _BF16, (T, Hq, D), idx, True)
    _need_workspace(workspace, idx)
    _need_cache(kv, idx)
    with _elsewhere(idx, stream):
        return rope_append(kv, q, k, v, positions, slot_mapping, inv_freq, interleaved=interleaved,
                           attn_factor=attn_factor, q_norm=q_norm, k_norm=k_norm, eps=eps,
                           q_out=q_out, workspace=workspace)


@dataclass
class Score:
    """Score options of prefill and decode_scored (defaults: plain softmax).

    softcap c: s <- c tanh(s / c); slopes fp32 [Hq]: s <- s - slope |p - t|;
    window: the last `window` keys up to the query's own; first_key int32
    (per query token: [T] for prefill, [B] for decode): earlier keys are
    hidden; prefix_lens int32 [B] (prefill): the first prefix_lens[b] keys
    are visible to every query of the sequence."""
    softcap: float = 0.0
    slopes: Optional[torch.Tensor] = None
    window: int = 0
    first_key: Optional[torch.Tensor] = None
    prefix_lens: Optional[torch.Tensor] = None

    def _need(self, num_q_heads: int, tokens: int, batch: int, idx: int):
        for t, name, dt, n in ((self.slopes, "slopes", _F32, num_q_heads),
                               (self.first_key, "first_key", _I32, tokens),
                               (self.prefix_lens, "prefix_lens", _I32, batch)):
            if t is not None:
                _need(t, name, dt, (n,), idx)


_PLAIN = Score()


def decode_scored(kv: KvCache, q, block_tables, seq_lens, softmax_scale, *, score=None, out=None,
                  out_fp32=False, return_lse=False, max_seq_len=None, workspace=None, kernel=0,
                  split_blocks=0, target_items=0, events=None, stream=None):
    """decode with score options: q bf16 [B, 1, Hq, D] -> (out, [lse,]
    workspace).  A workspace that is too small is replaced."""
    sc = _PLAIN if score is None else score
    if stream is None:
        r = (_ext or _fast()).decode_scored(
            DTYPE_CODES[kv.dtype], kv.block_size, kv.k_cache, kv.v_cache, kv.k_scale, kv.v_scale,
            kv.k_global, kv.v_global, q, block_tables, seq_lens, softmax_scale, sc.softcap,
            sc.slopes, sc.window, sc.first_key, sc.prefix_lens, out, out_fp32, return_lse,
            max_seq_len, workspace, kernel, split_blocks, target_items,
            0 if events is None else events[0].cuda_event,
            0 if events is None else events[1].cuda_event)
        if type(r) is int:
            raise PaError("pa_decode_scored", r)
        if r is not None:
            return r
    B, Q, Hq, D = q.shape
    idx = kv.k_cache.get_device()
    _need(q, "q", _BF16, (B, 1, Hq, kv.head_dim), idx)
    _need(block_tables, "block_tables", _I32, (B, block_tables.shape[1]), idx)
    _need(seq_lens, "seq_lens", _I32, (B,), idx)
    _need_out(out, (B, 1, Hq, D), idx)
    sc._need(Hq, B, B, idx)
    _need_workspace(workspace, idx)
    _need_cache(kv, idx)
    with _elsewhere(idx, stream):
        return decode_scored(kv, q, block_tables, seq_lens, softmax_scale, score=score, out=out,
                             out_fp32=out_fp32, return_lse=return_lse, max_seq_len=max_seq_len,
                             workspace=workspace, kernel=kernel, split_blocks=split_blocks,
                             target_items=target_items, events=events)


def prefill(kv: KvCache, q, q_starts, block_tables, seq_lens, softmax_scale, *, score=None,
            out=None, out_fp32=False, return_lse=False, max_seq_len=None, workspace=None,
            stream=None):
    """Attention of a ragged batch of prompt chunks over the paged cache.

    q bf16 [T, Hq, D]; sequence b owns the rows q_starts[b] .. q_starts[b + 1]
    - 1 (q_starts int32 [B + 1]), the last of its seq_lens[b] keys; rows
    outside are left as they are.  Returns (out [T, Hq, D], [lse [T, Hq],]
    workspace).  A workspace that is too small is replaced."""
    sc = _PLAIN if score is None else score
    if stream is None:
        r = (_ext or _fast()).prefill(
            DTYPE_CODES[kv.dtype], kv.block_size, kv.k_cache, kv.v_cache, kv.k_scale, kv.v_scale,
            kv.k_global, kv.v_global, q, q_starts, block_tables, seq_lens, softmax_scale,
            sc.softcap, sc.slopes, sc.window, sc.first_key, sc.prefix_lens, out, out_fp32,
            return_lse, max_seq_len, workspace)
        if type(r) is int:
            raise PaError("pa_prefill", r)
        if r is not None:
            return r
    T, Hq, D = q.shape
    B = seq_lens.shape[0]
    idx = kv.k_cache.get_device()
    _need(q, "q", _BF16, (T, Hq, kv.head_dim), idx)
    _need(q_starts, "q_starts", _I32, (B + 1,), idx)
    _need(block_tables, "block_tables", _I32, (B, block_tables.shape[1]), idx)
    _need(seq_lens, "seq_lens", _I32, (B,), idx)
    _need_out(out, (T, Hq, D), idx)
    sc._need(Hq, T, B, idx)
    _need_workspace(workspace, idx)
    _need_cache(kv, idx)
    with _elsewhere(idx, stream):
        return prefill(kv, q, q_starts, block_tables, seq_lens, softmax_scale, score=score, out=out,
                       out_fp32=out_fp32, return_lse=return_lse, max_seq_len=max_seq_len,
                       workspace=workspace)


@dataclass
class LatentCache:
    """The paged cache of latent attention: one row a token for all heads.

    dtype "bf16": latent bf16 [NB, 16, 512], rope bf16 [NB, 16, 64]; "fp8":
    latent uint8 (E4M3 codes), rope bf16, a value being the stored one times
    scale in both.  A scale chosen for the latents (their largest over 448) does
    for both: the rotated part keeps bf16's range wherever it is read."""
    dtype: str
    latent: torch.Tensor
    rope: torch.Tensor
    scale: float = 1.0
    block_size: int = 16

    def struct(self) -> _LatentCache:
        return _LatentCache(DTYPE_CODES[self.dtype], int(self.latent.shape[0]), self.block_size,
                            int(self.latent.shape[2]), int(self.rope.shape[2]), _ptr(self.latent),
                            _ptr(self.rope), float(self.scale))

    def _need(self, idx):
        if idx < 0:
            raise ValueError("the latent cache must be on a CUDA device")
        c, r = self.latent, self.rope
        if c.dim() != 3 or r.dim() != 3:
            raise ValueError(f"latent and rope must have three dimensions: got {list(c.shape)}, {list(r.shape)}")
        size = 2 if self.dtype == "bf16" else 1
        shape = (c.shape[0], self.block_size, c.shape[2])
        if c.shape != shape or c.element_size() != size or not c.is_contiguous():
            raise ValueError(f"latent must be contiguous {list(shape)} of {size}-byte elements: got {c.dtype} "
                             f"{list(c.shape)}")
        _need(r, "rope", _BF16, (c.shape[0], self.block_size, r.shape[2]), idx)


def _need_strided(t, name, shape, idx):
    """bf16, the last dim contiguous, the others any distance apart."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor: got {type(t).__name__}")
    if t.dtype is not _BF16 or t.shape != shape or t.get_device() != idx or t.stride(-1) != 1:
        raise ValueError(f"{name} must be {_BF16} {list(shape)} on cuda:{idx} with contiguous rows: got {t.dtype} "
                         f"{list(t.shape)} on {t.device}, strides {t.stride()}")


def latent_append(kv: LatentCache, latent, rope, positions, slot_mapping, inv_freq, *, q=None, q_out=None,
                  interleaved=False, attn_factor=1.0, norm=None, eps=1e-6, workspace=None, stream=None):
    """RMS norm (norm bf16 [512], optional) of the new tokens' latents,
    position rotation of their rotated parts and of the queries', and the
    write into the cache (in place), in one pass.

    latent bf16 [T, 512], rope bf16 [T, 64], q bf16 [T, Hq, 64] (None: no
    queries): rows contiguous, any distance apart (slices of projections).
    positions int32 [T]; slot_mapping int64 [T] (-1 = padded row); inv_freq
    fp32 [32] (rope_frequencies(64)).  Returns the turned queries, in q_out if
    given: q itself, or the last 64 dims of latent_decode's query."""
    if stream is None:
        r = (_ext or _fast()).latent_append(
            DTYPE_CODES[kv.dtype], kv.block_size, kv.latent, kv.rope, kv.scale, latent, rope, positions,
            slot_mapping, inv_freq, q, q_out, interleaved, attn_factor, norm, eps, workspace)
        if r is True:
            return None
        if type(r) is int:
            raise PaError("pa_latent_append", r)
        if r is not None:
            return r
    idx = kv.latent.get_device()
    kv._need(idx)
    T, dims, half = latent.shape[0], kv.latent.shape[2], kv.rope.shape[2]
    _need_strided(latent, "latent", (T, dims), idx)
    _need_strided(rope, "rope", (T, half), idx)
    _need(positions, "positions", _I32, (T,), idx)
    _need(slot_mapping, "slot_mapping", _I64, (T,), idx)
    _need(inv_freq, "inv_freq", _F32, (half // 2,), idx)
    if norm is not None:
        _need(norm, "norm", _BF16, (dims,), idx)
    if q is not None:
        _need_strided(q, "q", (T, q.shape[1], half), idx)
        if q_out is not None:
            _need_strided(q_out, "q_out", tuple(q.shape), idx)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _need_workspace(workspace, idx)
    with _elsewhere(idx, stream):
        return latent_append(kv, latent, rope, positions, slot_mapping, inv_freq, q=q, q_out=q_out,
                             interleaved=interleaved, attn_factor=attn_factor, norm=norm, eps=eps,
                             workspace=workspace)


def latent_gather(kv: LatentCache, block_tables, starts, num_rows: int, *, first=None, latent_out=None,
                  rope_out=None, workspace=None, stream=None):
    """Cached rows as bf16 (latent [num_rows, 512], rope [num_rows, 64]): rows
    starts[b] .. starts[b + 1] - 1 (starts int32 [B + 1]) are sequence b's
    tokens from first[b] on (first int32 [B]; None: 0).  Rows of no sequence
    are left as they are."""
    if stream is None:
        r = (_ext or _fast()).latent_gather(
            DTYPE_CODES[kv.dtype], kv.block_size, kv.latent, kv.rope, kv.scale, block_tables, starts, num_rows,
            first, latent_out, rope_out, workspace)
        if type(r) is int:
            raise PaError("pa_latent_gather", r)
        if r is not None:
            return r
    idx = kv.latent.get_device()
    kv._need(idx)
    B = block_tables.shape[0]
    _need(block_tables, "block_tables", _I32, (B, block_tables.shape[1]), idx)
    _need(starts, "starts", _I32, (B + 1,), idx)
    if first is not None:
        _need(first, "first", _I32, (B,), idx)
    for t, name, d in ((latent_out, "latent_out", kv.latent.shape[2]), (rope_out, "rope_out", kv.rope.shape[2])):
        if t is not None:
            _need(t, name, _BF16, (num_rows, d), idx)
    _need_workspace(workspace, idx)
    with _elsewhere(idx, stream):
        return latent_gather(kv, block_tables, starts, num_rows, first=first, latent_out=latent_out,
                             rope_out=rope_out, workspace=workspace)


def latent_prefill(q, k_nope, k_rope, v, q_starts, kv_starts, softmax_scale, *, causal=True, out=None,
                   out_fp32=False, return_lse=False, workspace=None, stream=None):
    """The expanded form of latent attention over a ragged batch.

    q bf16 [T, H, 192] (128 dims and the 64 rotated ones), k_nope bf16 [N, H,
    128], k_rope bf16 [N, 64] (shared by the heads), v bf16 [N, H, 128]: rows
    contiguous, any distance apart.  Sequence b owns the query rows from
    q_starts[b] and the key rows from kv_starts[b] (int32 [B + 1]); causal: its
    last query is at its last key, else every query sees every key.  Returns
    (out [T, H, 128], [lse [T, H],] workspace); rows of no sequence are left
    as they are.  A workspace that is too small is replaced."""
    if stream is None:
        r = (_ext or _fast()).latent_prefill(q, k_nope, k_rope, v, q_starts, kv_starts, softmax_scale, causal,
                                             out, out_fp32, return_lse, workspace)
        if type(r) is int:
            raise PaError("pa_latent_prefill", r)
        if r is not None:
            return r
    idx = q.get_device()
    if idx < 0:
        raise ValueError("q must be on a CUDA device")
    T, H, N, B = q.shape[0], q.shape[1], k_nope.shape[0], q_starts.shape[0] - 1
    _need_strided(q, "q", (T, H, 192), idx)
    _need_strided(k_nope, "k_nope", (N, H, 128), idx)
    _need_strided(k_rope, "k_rope", (N, 64), idx)
    _need_strided(v, "v", (N, H, 128), idx)
    _need(q_starts, "q_starts", _I32, (B + 1,), idx)
    _need(kv_starts, "kv_starts", _I32, (B + 1,), idx)
    _need_out(out, (T, H, 128), idx)
    _need_workspace(workspace, idx)
    with _elsewhere(idx, stream):
        return latent_prefill(q, k_nope, k_rope, v, q_starts, kv_starts, softmax_scale, causal=causal, out=out,
                              out_fp32=out_fp32, return_lse=return_lse, workspace=workspace)


def latent_decode(kv: LatentCache, q, block_tables, seq_lens, softmax_scale, *, out=None, out_fp32=False,
                  return_lse=False, max_seq_len=None, workspace=None, stream=None):
    """The absorbed form of latent attention over the paged cache: q bf16 [B,
    Q, H, 576] (the query times W_K, 512 dims, beside its 64 rotated ones) of
    the last Q tokens of each sequence, causal among them -> (out [B, Q, H,
    512], [lse,] workspace).  A workspace that is too small is replaced.

    Over an FP8 cache q's 512 dims and the weights pass through fp16: q up to
    65,504 (past that the output is NaN), weights off by up to 2^-25 of the
    largest.  Over a bf16 one weights are rounded to bf16.  Keys that only some
    of the Q tokens see must be finite."""
    if stream is None:
        r = (_ext or _fast()).latent_decode(
            DTYPE_CODES[kv.dtype], kv.block_size, kv.latent, kv.rope, kv.scale, q, block_tables, seq_lens,
            softmax_scale, out, out_fp32, return_lse, max_seq_len, workspace)
        if type(r) is int:
            raise PaError("pa_latent_decode", r)
        if r is not None:
            return r
    idx = kv.latent.get_device()
    kv._need(idx)
    B, Q, H, _ = q.shape
    dims = int(kv.latent.shape[2])
    _need(q, "q", _BF16, (B, Q, H, dims + kv.rope.shape[2]), idx)
    _need(block_tables, "block_tables", _I32, (B, block_tables.shape[1]), idx)
    _need(seq_lens, "seq_lens", _I32, (B,), idx)
    _need_out(out, (B, Q, H, dims), idx)
    _need_workspace(workspace, idx)
    with _elsewhere(idx, stream):
        return latent_decode(kv, q, block_tables, seq_lens, softmax_scale, out=out, out_fp32=out_fp32,
                             return_lse=return_lse, max_seq_len=max_seq_len, workspace=workspace)


def read_error(workspace: torch.Tensor, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    st = lib().pa_read_error(_ptr(workspace), ctypes.byref(flags), _stream(stream))
    if st != PA_OK:
        raise PaError("pa_read_error", st)
    return int(flags.value)


def header(workspace: torch.Tensor):
    """(err, num_items, split_blocks, slots, resident) from the workspace
    header; resident is the count of CTAs the planner rounded the items to
    (0 when it did not round)."""
    h = workspace[:32].view(torch.int32).cpu().tolist()
    return tuple(h[:5])
