// pa_py.cpp -- the ordinary calls of rope_append, prefill, decode_scored and the
// latent operators from Python: argument checks, outputs and workspace, and the call of the C
// ABI, in one step.  For a batch of a few tokens the kernels take 3 to 10
// microseconds and the interpreted checks and packing took 15.
//
// Every function returns its result, or None where an argument is not what the
// plain call expects (the interpreted path in pa.py then names it), or the
// negative pa_status of a refused call.  The C entry points are handed over by
// pa.py, which has loaded the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pa.h"

namespace {

using at::Tensor;

decltype(&pa_rope_append) f_rope = nullptr;
decltype(&pa_prefill) f_prefill = nullptr;
decltype(&pa_prefill_workspace_bytes) f_prefill_ws = nullptr;
decltype(&pa_decode_scored) f_decode = nullptr;
decltype(&pa_workspace_bytes) f_decode_ws = nullptr;
decltype(&pa_latent_append) f_lappend = nullptr;
decltype(&pa_latent_gather) f_lgather = nullptr;
decltype(&pa_latent_prefill) f_lprefill = nullptr;
decltype(&pa_latent_prefill_workspace_bytes) f_lprefill_ws = nullptr;
decltype(&pa_latent_decode) f_ldecode = nullptr;
decltype(&pa_latent_decode_workspace_bytes) f_ldecode_ws = nullptr;

// an argument that must be a tensor (throws nothing: null if it is not)
const Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool is(const Tensor *t, at::ScalarType dt, at::IntArrayRef shape, int dev) {
  return t && t->scalar_type() == dt && t->is_cuda() && t->device().index() == dev && t->sizes() == shape &&
         t->is_contiguous();
}
// [tokens, heads, head_dim], the tokens any distance apart
bool is_rows(const Tensor *t, at::IntArrayRef shape, int dev) {
  return t && t->scalar_type() == at::kBFloat16 && t->is_cuda() && t->device().index() == dev &&
         t->sizes() == shape &&
         (t->is_contiguous() || (t->stride(2) == 1 && (shape[1] < 2 || t->stride(1) == shape[2])));
}
// None, or a tensor that `is`
bool opt(PyObject *o, const Tensor *&t, at::ScalarType dt, at::IntArrayRef shape, int dev) {
  t = nullptr;
  if (o == Py_None) return true;
  t = tensor(o);
  return is(t, dt, shape, dev);
}
bool is_workspace(const Tensor *t, int dev) {
  return t && t->is_cuda() && t->device().index() == dev && t->is_contiguous();
}
void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

// one of the cache's arrays: its shape and element size, whatever the bytes are called
bool is_pool(const Tensor *t, at::IntArrayRef shape, size_t bytes, int dev) {
  return t && t->is_cuda() && t->device().index() == dev && t->sizes() == shape && t->itemsize() == bytes &&
         t->is_contiguous();
}

// the KV cache's eight fields from args[0 ..]; the device index, or -1
int cache(PyObject *const *a, pa_kv_cache &kv) {
  const Tensor *k = tensor(a[2]), *v = tensor(a[3]);
  const Tensor *ks = a[4] == Py_None ? nullptr : tensor(a[4]), *vs = a[5] == Py_None ? nullptr : tensor(a[5]);
  if (!k || !v || (a[4] != Py_None && !ks) || (a[5] != Py_None && !vs)) return -1;
  if (!k->is_cuda() || k->dim() != 4 || k->size(0) > INT32_MAX) return -1;
  kv.dtype = (int32_t)PyLong_AsLong(a[0]);
  kv.num_blocks = (int32_t)k->size(0);
  kv.block_size = (int32_t)PyLong_AsLong(a[1]);
  kv.num_kv_heads = (int32_t)k->size(1);
  kv.head_dim = (int32_t)k->size(3) * (kv.dtype == PA_KV_NVFP4 ? 2 : 1);
  kv.k_cache = k->data_ptr();
  kv.v_cache = v->data_ptr();
  kv.k_scale = ptr(ks);
  kv.v_scale = ptr(vs);
  kv.k_global_scale = (float)PyFloat_AsDouble(a[6]);
  kv.v_global_scale = (float)PyFloat_AsDouble(a[7]);
  const int dev = k->device().index();
  const int64_t pages[4] = {k->size(0), k->size(1), kv.block_size, k->size(3)};
  const size_t bytes = kv.dtype == PA_KV_BF16 ? 2 : 1;
  if (!is_pool(k, pages, bytes, dev) || !is_pool(v, pages, bytes, dev)) return -1;
  if (kv.dtype == PA_KV_INT8 && (!is_pool(ks, {pages[0], pages[1], pages[2]}, 2, dev) ||
                                 !is_pool(vs, {pages[0], pages[1], pages[2]}, 2, dev)))
    return -1;
  if (kv.dtype == PA_KV_NVFP4) {
    const int64_t blocks[4] = {pages[0], pages[1], pages[2], pages[3] / 8};
    if (!is_pool(ks, blocks, 1, dev) || !is_pool(vs, blocks, 1, dev)) return -1;
  }
  return c10::cuda::current_device() == dev ? dev : -1;
}

// score options from args[0 .. 4]: softcap, slopes, window, first_key, prefix_lens
bool score(PyObject *const *a, pa_score &s, int64_t heads, int64_t tokens, int64_t batch, int dev) {
  const Tensor *sl, *fk, *pl;
  if (!opt(a[1], sl, at::kFloat, {heads}, dev) || !opt(a[3], fk, at::kInt, {tokens}, dev) ||
      !opt(a[4], pl, at::kInt, {batch}, dev))
    return false;
  s.softcap = (float)PyFloat_AsDouble(a[0]);
  const long long w = PyLong_AsLongLong(a[2]);
  if (PyErr_Occurred() || w < INT32_MIN || w > INT32_MAX) {
    PyErr_Clear();
    return false;
  }
  s.window = (int32_t)w;
  s.alibi_slopes = static_cast<const float *>(ptr(sl));
  s.first_key = static_cast<const int32_t *>(ptr(fk));
  s.prefix_lens = static_cast<const int32_t *>(ptr(pl));
  return true;
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType dt, const Tensor &like) {
  return at::empty(shape, like.options().dtype(dt));
}

// the caller's output (bf16 or fp32), or a new one
bool output(PyObject *o, Tensor &out, at::IntArrayRef shape, bool fp32, const Tensor &like, int dev) {
  if (o == Py_None) {
    out = fresh(shape, fp32 ? at::kFloat : at::kBFloat16, like);
    return true;
  }
  const Tensor *t = tensor(o);
  if (!t || (t->scalar_type() != at::kFloat && t->scalar_type() != at::kBFloat16)) return false;
  if (!is(t, t->scalar_type(), shape, dev)) return false;
  out = *t;
  return true;
}

// torch's exceptions (out of memory, ..) become Python's
template <typename F>
PyObject *guarded(F &&f) {
  HANDLE_TH_ERRORS
  return f();
  END_HANDLE_TH_ERRORS
}

PyObject *refused() {
  if (PyErr_Occurred()) PyErr_Clear();   // a number that is none: the interpreted path says so
  Py_RETURN_NONE;
}

// rope_append(cache x 8, q, k, v, positions, slot_mapping, inv_freq,
//             interleaved, attn_factor, q_norm, k_norm, eps, q_out, workspace)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    pa_kv_cache kv;
    if (n != 21) return refused();
    const int dev = cache(a, kv);
    if (dev < 0) return refused();
    const Tensor *q = tensor(a[8]), *k = tensor(a[9]), *v = tensor(a[10]), *pos = tensor(a[11]),
                 *slots = tensor(a[12]), *inv = tensor(a[13]);
    if (!q || q->dim() != 3 || !inv) return refused();
    const int64_t T = q->size(0), H = q->size(1), D = kv.head_dim, half = inv->numel();
    const int64_t kvs[3] = {T, kv.num_kv_heads, D};
    if (T > INT32_MAX || H > INT32_MAX || half > 4096) return refused();
    const Tensor *wq, *wk;
    if (!is_rows(q, {T, H, D}, dev) || !is_rows(k, kvs, dev) || !is_rows(v, kvs, dev) ||
        !is(pos, at::kInt, {T}, dev) || !is(slots, at::kLong, {T}, dev) || !is(inv, at::kFloat, {half}, dev) ||
        !opt(a[16], wq, at::kBFloat16, {D}, dev) || !opt(a[17], wk, at::kBFloat16, {D}, dev))
      return refused();
    Tensor out;
    if (a[19] == Py_None) {
      out = fresh({T, H, D}, at::kBFloat16, *q);
    } else {
      const Tensor *o = tensor(a[19]);
      if (!is_rows(o, {T, H, D}, dev)) return refused();
      out = *o;
    }
    const Tensor *ws = a[20] == Py_None ? nullptr : tensor(a[20]);
    if (a[20] != Py_None && (!is_workspace(ws, dev) || ws->nbytes() < 256)) return refused();
    pa_rope r;
    r.num_tokens = (int32_t)T;
    r.num_q_heads = (int32_t)H;
    r.q = q->data_ptr();
    r.k = k->data_ptr();
    r.v = v->data_ptr();
    r.q_out = out.data_ptr();
    r.q_stride = q->stride(0);
    r.k_stride = k->stride(0);
    r.v_stride = v->stride(0);
    r.q_out_stride = out.stride(0);
    r.positions = static_cast<const int32_t *>(pos->data_ptr());
    r.slot_mapping = static_cast<const int64_t *>(slots->data_ptr());
    r.rot_dim = (int32_t)(2 * half);
    r.interleaved = PyObject_IsTrue(a[14]);
    r.inv_freq = static_cast<const float *>(inv->data_ptr());
    r.attn_factor = (float)PyFloat_AsDouble(a[15]);
    r.q_norm = ptr(wq);
    r.k_norm = ptr(wk);
    r.eps = (float)PyFloat_AsDouble(a[18]);
    if (PyErr_Occurred()) return refused();
    const int st = f_rope(&kv, &r, ptr(ws), (pa_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    return st == PA_OK ? THPVariable_Wrap(std::move(out)) : PyLong_FromLong(st);
  });
}

// runs `call(ws, bytes)`, with a new workspace of `need()` bytes where the
// caller's is missing or too small
template <typename C, typename N>
int with_workspace(PyObject *arg, Tensor &ws, const Tensor &like, C &&call, N &&need, bool &ok) {
  ok = true;
  int st = PA_ERR_WORKSPACE_TOO_SMALL;
  if (arg != Py_None) {
    const Tensor *t = tensor(arg);
    if (!is_workspace(t, like.device().index())) {
      ok = false;
      return 0;
    }
    ws = *t;
    st = call(ws.data_ptr(), ws.nbytes());
  }
  if (st == PA_ERR_WORKSPACE_TOO_SMALL) {
    const int64_t bytes = std::max<int64_t>((int64_t)need(), 256);
    ws = at::empty({bytes}, like.options().dtype(at::kByte));
    st = call(ws.data_ptr(), (size_t)bytes);
  }
  return st;
}

PyObject *results(int st, Tensor &&out, Tensor &&lse, bool has_lse, Tensor &&ws) {
  if (st != PA_OK) return PyLong_FromLong(st);
  PyObject *r = PyTuple_New(has_lse ? 3 : 2);
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(std::move(out)));
  if (has_lse) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(std::move(lse)));
  PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(ws)));
  return r;
}

// prefill(cache x 8, q, q_starts, block_tables, seq_lens, scale, score x 5,
//         out, out_fp32, return_lse, max_seq_len, workspace)
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    pa_kv_cache kv;
    if (n != 23) return refused();
    const int dev = cache(a, kv);
    if (dev < 0) return refused();
    const Tensor *q = tensor(a[8]), *starts = tensor(a[9]), *tab = tensor(a[10]), *lens = tensor(a[11]);
    if (!q || q->dim() != 3 || !tab || tab->dim() != 2 || !lens || lens->dim() != 1) return refused();
    const int64_t T = q->size(0), H = q->size(1), D = kv.head_dim, B = lens->size(0), stride = tab->size(1);
    if (T > INT32_MAX || H > INT32_MAX || B > INT32_MAX - 1 || stride > INT32_MAX) return refused();
    if (!is(q, at::kBFloat16, {T, H, D}, dev) || !is(starts, at::kInt, {B + 1}, dev) ||
        !is(tab, at::kInt, {B, stride}, dev) || !is(lens, at::kInt, {B}, dev))
      return refused();
    pa_score sc;
    if (!score(a + 13, sc, H, T, B, dev)) return refused();
    Tensor out, lse, ws;
    if (!output(a[18], out, {T, H, D}, PyObject_IsTrue(a[19]), *q, dev)) return refused();
    const bool has_lse = PyObject_IsTrue(a[20]);
    if (has_lse) lse = fresh({T, H}, at::kFloat, *q);
    pa_prefill_problem p;
    p.batch = (int32_t)B;
    p.num_q_heads = (int32_t)H;
    p.num_tokens = (int32_t)T;
    p.q = q->data_ptr();
    p.q_starts = static_cast<const int32_t *>(starts->data_ptr());
    p.block_tables = static_cast<const int32_t *>(tab->data_ptr());
    p.block_table_stride = (int32_t)stride;
    p.seq_lens = static_cast<const int32_t *>(lens->data_ptr());
    const long long most = a[21] == Py_None ? (long long)stride * kv.block_size : PyLong_AsLongLong(a[21]);
    if (most > INT32_MAX || most < INT32_MIN) return refused();
    p.max_seq_len = (int32_t)most;
    p.softmax_scale = (float)PyFloat_AsDouble(a[12]);
    p.out = out.data_ptr();
    p.out_fp32 = out.scalar_type() == at::kFloat;
    p.lse_out = has_lse ? static_cast<float *>(lse.data_ptr()) : nullptr;
    if (PyErr_Occurred()) return refused();
    const pa_stream_t s = (pa_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    bool ok;
    const int st = with_workspace(
        a[22], ws, *q, [&](void *w, size_t b) { return f_prefill(&kv, &p, &sc, w, b, s); },
        [&]() { return f_prefill_ws(&kv, &p); }, ok);
    if (!ok) return refused();
    return results(st, std::move(out), std::move(lse), has_lse, std::move(ws));
  });
}

// decode_scored(cache x 8, q, block_tables, seq_lens, scale, score x 5, out,
//               out_fp32, return_lse, max_seq_len, workspace, kernel,
//               split_blocks, target_items, event_begin, event_end)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    pa_kv_cache kv;
    if (n != 27) return refused();
    const int dev = cache(a, kv);
    if (dev < 0) return refused();
    const Tensor *q = tensor(a[8]), *tab = tensor(a[9]), *lens = tensor(a[10]);
    if (!q || q->dim() != 4 || !tab || tab->dim() != 2) return refused();
    const int64_t B = q->size(0), H = q->size(2), D = kv.head_dim, stride = tab->size(1);
    if (B > INT32_MAX || H > INT32_MAX || stride > INT32_MAX) return refused();
    if (!is(q, at::kBFloat16, {B, 1, H, D}, dev) || !is(tab, at::kInt, {B, stride}, dev) ||
        !is(lens, at::kInt, {B}, dev))
      return refused();
    pa_score sc;
    if (!score(a + 12, sc, H, B, B, dev)) return refused();
    Tensor out, lse, ws;
    if (!output(a[17], out, {B, 1, H, D}, PyObject_IsTrue(a[18]), *q, dev)) return refused();
    const bool has_lse = PyObject_IsTrue(a[19]);
    if (has_lse) lse = fresh({B, 1, H}, at::kFloat, *q);
    pa_problem p;
    p.batch = (int32_t)B;
    p.num_q_heads = (int32_t)H;
    p.q_len = 1;
    p.q = q->data_ptr();
    p.block_tables = static_cast<const int32_t *>(tab->data_ptr());
    p.block_table_stride = (int32_t)stride;
    p.seq_lens = static_cast<const int32_t *>(lens->data_ptr());
    const long long most = a[20] == Py_None ? (long long)stride * kv.block_size : PyLong_AsLongLong(a[20]);
    if (most > INT32_MAX || most < INT32_MIN) return refused();
    p.max_seq_len = (int32_t)most;
    p.softmax_scale = (float)PyFloat_AsDouble(a[11]);
    p.out = out.data_ptr();
    p.out_fp32 = out.scalar_type() == at::kFloat;
    p.lse_out = has_lse ? static_cast<float *>(lse.data_ptr()) : nullptr;
    pa_options o = {};
    o.kernel = (int32_t)PyLong_AsLong(a[22]);
    o.split_blocks = (int32_t)PyLong_AsLong(a[23]);
    o.target_items = (int32_t)PyLong_AsLong(a[24]);
    o.event_begin = PyLong_AsVoidPtr(a[25]);   // 0: none
    o.event_end = PyLong_AsVoidPtr(a[26]);
    if (PyErr_Occurred()) return refused();
    const pa_stream_t s = (pa_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    bool ok;
    const int st = with_workspace(
        a[21], ws, *q, [&](void *w, size_t b) { return f_decode(&kv, &p, &sc, &o, w, b, s); },
        [&]() { return f_decode_ws(&kv, &p, &o); }, ok);
    if (!ok) return refused();
    return results(st, std::move(out), std::move(lse), has_lse, std::move(ws));
  });
}

// ------------------------------------------------------------ latent attention

// the latent cache's five fields from args[0 ..]; the device index, or -1
int latent_cache(PyObject *const *a, pa_latent_cache &kv) {
  const Tensor *c = tensor(a[2]), *r = tensor(a[3]);
  if (!c || !r || !c->is_cuda() || c->dim() != 3 || r->dim() != 3 || c->size(0) > INT32_MAX ||
      c->size(2) > INT32_MAX || r->size(2) > INT32_MAX)
    return -1;
  kv.dtype = (int32_t)PyLong_AsLong(a[0]);
  kv.num_blocks = (int32_t)c->size(0);
  kv.block_size = (int32_t)PyLong_AsLong(a[1]);
  kv.latent_dim = (int32_t)c->size(2);
  kv.rope_dim = (int32_t)r->size(2);
  kv.latent = c->data_ptr();
  kv.rope = r->data_ptr();
  kv.global_scale = (float)PyFloat_AsDouble(a[4]);
  const int dev = c->device().index();
  if (!is_pool(c, {kv.num_blocks, kv.block_size, kv.latent_dim}, kv.dtype == PA_KV_BF16 ? 2 : 1, dev) ||
      !is(r, at::kBFloat16, {kv.num_blocks, kv.block_size, kv.rope_dim}, dev))
    return -1;
  return c10::cuda::current_device() == dev ? dev : -1;
}
// a shape whose last dim is contiguous, the others any distance apart
bool is_strided(const Tensor *t, at::IntArrayRef shape, int dev) {
  return t && t->scalar_type() == at::kBFloat16 && t->is_cuda() && t->device().index() == dev &&
         t->sizes() == shape && t->stride(t->dim() - 1) == 1;
}
pa_stream_t stream_of(int dev) {
  return (pa_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
}
// a number that fits 32 bits; false (with no error set) otherwise
bool int32_of(PyObject *o, int32_t &v) {
  const long long x = PyLong_AsLongLong(o);
  if (x < INT32_MIN || x > INT32_MAX) return false;
  v = (int32_t)x;
  return true;
}

// latent_append(cache x 5, latent, rope, positions, slot_mapping, inv_freq, q,
//               q_out, interleaved, attn_factor, norm, eps, workspace)
// -> q_out, or True where there are no queries
PyObject *latent_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    pa_latent_cache kv;
    if (n != 17) return refused();
    const int dev = latent_cache(a, kv);
    if (dev < 0) return refused();
    const Tensor *c = tensor(a[5]), *r = tensor(a[6]), *pos = tensor(a[7]), *slots = tensor(a[8]),
                 *inv = tensor(a[9]), *norm;
    if (!c || c->dim() != 2) return refused();
    const int64_t T = c->size(0);
    if (T > INT32_MAX || !is_strided(c, {T, kv.latent_dim}, dev) || !is_strided(r, {T, kv.rope_dim}, dev) ||
        !is(pos, at::kInt, {T}, dev) || !is(slots, at::kLong, {T}, dev) ||
        !is(inv, at::kFloat, {kv.rope_dim / 2}, dev) || !opt(a[14], norm, at::kBFloat16, {kv.latent_dim}, dev))
      return refused();
    pa_latent_new x = {};
    Tensor out;
    if (a[10] != Py_None) {
      const Tensor *q = tensor(a[10]);
      if (!q || q->dim() != 3 || q->size(1) > INT32_MAX || !is_strided(q, {T, q->size(1), kv.rope_dim}, dev))
        return refused();
      if (a[11] == Py_None) {
        out = fresh(q->sizes(), at::kBFloat16, *q);
      } else {
        const Tensor *o = tensor(a[11]);
        if (!is_strided(o, q->sizes(), dev)) return refused();
        out = *o;
      }
      x.num_q_heads = (int32_t)q->size(1);
      x.q = q->data_ptr();
      x.q_out = out.data_ptr();
      x.q_stride = q->stride(0);
      x.q_head_stride = q->stride(1);
      x.q_out_stride = out.stride(0);
      x.q_out_head_stride = out.stride(1);
    } else if (a[11] != Py_None) {
      return refused();
    }
    const Tensor *ws = a[16] == Py_None ? nullptr : tensor(a[16]);
    if (a[16] != Py_None && (!is_workspace(ws, dev) || ws->nbytes() < 256)) return refused();
    x.num_tokens = (int32_t)T;
    x.latent = c->data_ptr();
    x.rope = r->data_ptr();
    x.latent_stride = c->stride(0);
    x.rope_stride = r->stride(0);
    x.positions = static_cast<const int32_t *>(pos->data_ptr());
    x.slot_mapping = static_cast<const int64_t *>(slots->data_ptr());
    x.interleaved = PyObject_IsTrue(a[12]);
    x.inv_freq = static_cast<const float *>(inv->data_ptr());
    x.attn_factor = (float)PyFloat_AsDouble(a[13]);
    x.norm = ptr(norm);
    x.eps = (float)PyFloat_AsDouble(a[15]);
    if (PyErr_Occurred()) return refused();
    const int st = f_lappend(&kv, &x, ptr(ws), stream_of(dev));
    if (st != PA_OK) return PyLong_FromLong(st);
    if (a[10] == Py_None) Py_RETURN_TRUE;
    return THPVariable_Wrap(std::move(out));
  });
}

// latent_gather(cache x 5, block_tables, starts, num_rows, first, latent_out,
//               rope_out, workspace)
PyObject *latent_gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    pa_latent_cache kv;
    if (n != 12) return refused();
    const int dev = latent_cache(a, kv);
    if (dev < 0) return refused();
    const Tensor *tab = tensor(a[5]), *starts = tensor(a[6]), *first;
    int32_t N;
    if (!tab || tab->dim() != 2 || !int32_of(a[7], N) || PyErr_Occurred()) return refused();
    const int64_t B = tab->size(0), stride = tab->size(1);
    if (N < 0) return PyLong_FromLong(PA_ERR_INVALID_ARG);
    if (B > INT32_MAX - 1 || stride > INT32_MAX || !is(tab, at::kInt, {B, stride}, dev) ||
        !is(starts, at::kInt, {B + 1}, dev) || !opt(a[8], first, at::kInt, {B}, dev))
      return refused();
    Tensor co, ro;
    const int64_t cs[2] = {N, kv.latent_dim}, rs[2] = {N, kv.rope_dim};
    for (int i = 0; i < 2; ++i) {
      PyObject *const o = a[9 + i];
      Tensor &t = i ? ro : co;
      if (o == Py_None) {
        t = fresh(i ? rs : cs, at::kBFloat16, *tab);
      } else {
        if (!is(tensor(o), at::kBFloat16, i ? rs : cs, dev)) return refused();
        t = *tensor(o);
      }
    }
    const Tensor *ws = a[11] == Py_None ? nullptr : tensor(a[11]);
    if (a[11] != Py_None && (!is_workspace(ws, dev) || ws->nbytes() < 256)) return refused();
    const int st = f_lgather(&kv, static_cast<const int32_t *>(tab->data_ptr()), (int32_t)stride,
                             static_cast<const int32_t *>(starts->data_ptr()),
                             static_cast<const int32_t *>(ptr(first)), (int32_t)B, N, co.data_ptr(), ro.data_ptr(),
                             ptr(ws), stream_of(dev));
    if (st != PA_OK) return PyLong_FromLong(st);
    PyObject *r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(co)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(ro)));
    return r;
  });
}

// latent_prefill(q, k_nope, k_rope, v, q_starts, kv_starts, scale, causal, out,
//                out_fp32, return_lse, workspace)
PyObject *latent_prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 12) return refused();
    const Tensor *q = tensor(a[0]), *kn = tensor(a[1]), *kr = tensor(a[2]), *v = tensor(a[3]), *qs = tensor(a[4]),
                 *ks = tensor(a[5]);
    if (!q || q->dim() != 3 || !q->is_cuda() || !kn || kn->dim() != 3 || !qs || qs->dim() != 1) return refused();
    const int dev = q->device().index();
    const int64_t T = q->size(0), H = q->size(1), N = kn->size(0), B = qs->size(0) - 1;
    if (c10::cuda::current_device() != dev || T > INT32_MAX || H > INT32_MAX || N > INT32_MAX || B < 0 ||
        B > INT32_MAX)
      return refused();
    if (!is_strided(q, {T, H, 192}, dev) || !is_strided(kn, {N, H, 128}, dev) || !is_strided(kr, {N, 64}, dev) ||
        !is_strided(v, {N, H, 128}, dev) || !is(qs, at::kInt, {B + 1}, dev) || !is(ks, at::kInt, {B + 1}, dev))
      return refused();
    Tensor out, lse, ws;
    if (!output(a[8], out, {T, H, 128}, PyObject_IsTrue(a[9]), *q, dev)) return refused();
    const bool has_lse = PyObject_IsTrue(a[10]);
    if (has_lse) lse = fresh({T, H}, at::kFloat, *q);
    pa_latent_prefill_problem p = {};
    p.batch = (int32_t)B;
    p.num_heads = (int32_t)H;
    p.num_tokens = (int32_t)T;
    p.num_keys = (int32_t)N;
    p.q = q->data_ptr();
    p.k_nope = kn->data_ptr();
    p.k_rope = kr->data_ptr();
    p.v = v->data_ptr();
    p.q_stride = q->stride(0);
    p.q_head_stride = q->stride(1);
    p.k_stride = kn->stride(0);
    p.k_head_stride = kn->stride(1);
    p.k_rope_stride = kr->stride(0);
    p.v_stride = v->stride(0);
    p.v_head_stride = v->stride(1);
    p.q_starts = static_cast<const int32_t *>(qs->data_ptr());
    p.kv_starts = static_cast<const int32_t *>(ks->data_ptr());
    p.softmax_scale = (float)PyFloat_AsDouble(a[6]);
    p.causal = PyObject_IsTrue(a[7]);
    p.out = out.data_ptr();
    p.out_fp32 = out.scalar_type() == at::kFloat;
    p.lse_out = has_lse ? static_cast<float *>(lse.data_ptr()) : nullptr;
    if (PyErr_Occurred()) return refused();
    const pa_stream_t s = stream_of(dev);
    bool ok;
    const int st = with_workspace(
        a[11], ws, *q, [&](void *w, size_t b) { return f_lprefill(&p, w, b, s); },
        [&]() { return f_lprefill_ws(&p); }, ok);
    if (!ok) return refused();
    return results(st, std::move(out), std::move(lse), has_lse, std::move(ws));
  });
}

// latent_decode(cache x 5, q, block_tables, seq_lens, scale, out, out_fp32,
//               return_lse, max_seq_len, workspace)
PyObject *latent_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    pa_latent_cache kv;
    if (n != 14) return refused();
    const int dev = latent_cache(a, kv);
    if (dev < 0) return refused();
    const Tensor *q = tensor(a[5]), *tab = tensor(a[6]), *lens = tensor(a[7]);
    if (!q || q->dim() != 4 || !tab || tab->dim() != 2) return refused();
    const int64_t B = q->size(0), Q = q->size(1), H = q->size(2), stride = tab->size(1);
    if (B > INT32_MAX || Q > INT32_MAX || H > INT32_MAX || stride > INT32_MAX) return refused();
    if (!is(q, at::kBFloat16, {B, Q, H, kv.latent_dim + kv.rope_dim}, dev) || !is(tab, at::kInt, {B, stride}, dev) ||
        !is(lens, at::kInt, {B}, dev))
      return refused();
    Tensor out, lse, ws;
    if (!output(a[9], out, {B, Q, H, kv.latent_dim}, PyObject_IsTrue(a[10]), *q, dev)) return refused();
    const bool has_lse = PyObject_IsTrue(a[11]);
    if (has_lse) lse = fresh({B, Q, H}, at::kFloat, *q);
    pa_latent_problem p = {};
    p.batch = (int32_t)B;
    p.num_heads = (int32_t)H;
    p.q_len = (int32_t)Q;
    p.q = q->data_ptr();
    p.block_tables = static_cast<const int32_t *>(tab->data_ptr());
    p.block_table_stride = (int32_t)stride;
    p.seq_lens = static_cast<const int32_t *>(lens->data_ptr());
    const long long most = a[12] == Py_None ? (long long)stride * kv.block_size : PyLong_AsLongLong(a[12]);
    if (most > INT32_MAX || most < INT32_MIN) return refused();
    p.max_seq_len = (int32_t)most;
    p.softmax_scale = (float)PyFloat_AsDouble(a[8]);
    p.out = out.data_ptr();
    p.out_fp32 = out.scalar_type() == at::kFloat;
    p.lse_out = has_lse ? static_cast<float *>(lse.data_ptr()) : nullptr;
    if (PyErr_Occurred()) return refused();
    const pa_stream_t s = stream_of(dev);
    bool ok;
    const int st = with_workspace(
        a[13], ws, *q, [&](void *w, size_t b) { return f_ldecode(&kv, &p, w, b, s); },
        [&]() { return f_ldecode_ws(&kv, &p); }, ok);
    if (!ok) return refused();
    return results(st, std::move(out), std::move(lse), has_lse, std::move(ws));
  });
}

// entry_points(the addresses of the C functions above, in the order of their declaration)
PyObject *entry_points(PyObject *, PyObject *args) {
  unsigned long long f[11];
  if (!PyArg_ParseTuple(args, "KKKKKKKKKKK", f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6, f + 7, f + 8, f + 9, f + 10))
    return nullptr;
  f_rope = reinterpret_cast<decltype(f_rope)>(f[0]);
  f_prefill = reinterpret_cast<decltype(f_prefill)>(f[1]);
  f_prefill_ws = reinterpret_cast<decltype(f_prefill_ws)>(f[2]);
  f_decode = reinterpret_cast<decltype(f_decode)>(f[3]);
  f_decode_ws = reinterpret_cast<decltype(f_decode_ws)>(f[4]);
  f_lappend = reinterpret_cast<decltype(f_lappend)>(f[5]);
  f_lgather = reinterpret_cast<decltype(f_lgather)>(f[6]);
  f_lprefill = reinterpret_cast<decltype(f_lprefill)>(f[7]);
  f_lprefill_ws = reinterpret_cast<decltype(f_lprefill_ws)>(f[8]);
  f_ldecode = reinterpret_cast<decltype(f_ldecode)>(f[9]);
  f_ldecode_ws = reinterpret_cast<decltype(f_ldecode_ws)>(f[10]);
  Py_RETURN_NONE;
}

#define PA_FAST(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PA_FAST("rope_append", rope),
    PA_FAST("prefill", prefill),
    PA_FAST("decode_scored", decode),
    PA_FAST("latent_append", latent_append),
    PA_FAST("latent_gather", latent_gather),
    PA_FAST("latent_prefill", latent_prefill),
    PA_FAST("latent_decode", latent_decode),
    {"entry_points", entry_points, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_py() { return PyModule_Create(&module); }
