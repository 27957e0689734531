// pa_py.cpp -- the ordinary calls of rope_append, prefill and decode_scored
// from Python: argument checks, outputs and workspace, and the call of the C
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

// entry_points(addresses of pa_rope_append, pa_prefill,
//              pa_prefill_workspace_bytes, pa_decode_scored, pa_workspace_bytes)
PyObject *entry_points(PyObject *, PyObject *args) {
  unsigned long long r, p, pw, d, dw;
  if (!PyArg_ParseTuple(args, "KKKKK", &r, &p, &pw, &d, &dw)) return nullptr;
  f_rope = reinterpret_cast<decltype(f_rope)>(r);
  f_prefill = reinterpret_cast<decltype(f_prefill)>(p);
  f_prefill_ws = reinterpret_cast<decltype(f_prefill_ws)>(pw);
  f_decode = reinterpret_cast<decltype(f_decode)>(d);
  f_decode_ws = reinterpret_cast<decltype(f_decode_ws)>(dw);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefill)), METH_FASTCALL, nullptr},
    {"decode_scored", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"entry_points", entry_points, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_py() { return PyModule_Create(&module); }
