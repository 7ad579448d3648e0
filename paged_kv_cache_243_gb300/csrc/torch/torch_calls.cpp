// The calls for drafted tokens straight from torch tensors: what PagedKVCache's methods check and marshal in
// Python, without Python. Those calls take 2 to 15 us on the device, and 7 to 18 of checks and
// marshalling in Python before they get there.
//
// Every function either makes its call, or returns NotImplemented without having done anything: for whatever
// is not exactly as the C entry point wants it (another type or device, a stride, a shape, a refused
// argument, memory that has to be made first). The method then goes its own way, which says what is wrong.
// The interpreter's lock is held throughout.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "pkv.h"

namespace {

decltype(&pkv_rotary_append) rotary_append_fn = nullptr;
decltype(&pkv_tree_attention) tree_attention_fn = nullptr;
decltype(&pkv_keep_tokens) keep_tokens_fn = nullptr;
PyObject* error_type = nullptr;   // error_type(status, where)

// What a cache keeps for these calls.
struct Handle {
  const pkv_cache* cache;
  c10::DeviceIndex device;
  PyObject* fit;       // workspaces by (stream, batch, query heads, splits, drafts)
  PyObject* acquire;   // the lock of those workspaces: its bound methods
  PyObject* release;
};

constexpr const char* kName = "paged_kv_cache.handle";

void drop(PyObject* capsule) {
  Handle* h = static_cast<Handle*>(PyCapsule_GetPointer(capsule, kName));
  if (!h) return;
  Py_XDECREF(h->fit);
  Py_XDECREF(h->acquire);
  Py_XDECREF(h->release);
  delete h;
}

PyObject* decline() { Py_RETURN_NOTIMPLEMENTED; }

// A tensor on the cache's device; NULL for None (with `ok`) and for anything else.
const at::Tensor* tensor(PyObject* o, const Handle* h, bool& ok) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_CheckExact(o)) {
    ok = false;
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.get_device() != h->device || t.layout() != c10::kStrided) {
    ok = false;
    return nullptr;
  }
  return &t;
}

bool shaped(const at::Tensor* t, c10::ScalarType type, c10::IntArrayRef shape) {
  return t && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
}
bool shaped_or_none(PyObject* o, const at::Tensor* t, c10::ScalarType type, c10::IntArrayRef shape) {
  return o == Py_None || shaped(t, type, shape);
}

template <class T>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

bool number(PyObject* o, long& v) {
  v = PyLong_Check(o) ? PyLong_AsLong(o) : -1;
  if (PyErr_Occurred()) PyErr_Clear();
  return PyLong_Check(o) && v >= 0 && v <= INT32_MAX;
}

bool type_of(c10::ScalarType t, pkv_dtype& d) {
  d = t == c10::kHalf ? PKV_F16 : t == c10::kBFloat16 ? PKV_BF16 : PKV_F32;
  return t == c10::kHalf || t == c10::kBFloat16 || t == c10::kFloat;
}

// Elements from a token of t [rows][tokens][heads][d] to the next; -1 where its strides are others than one distance
// between tokens and the heads side by side.
int64_t token_stride(const at::Tensor& t, int64_t rows, int64_t tokens, int64_t heads, int64_t d) {
  const auto s = t.strides();
  const int64_t step = tokens > 1 ? s[1] : rows > 1 ? s[0] : heads * d;
  return s[3] != 1 || (heads > 1 && s[2] != d) || (rows > 1 && tokens > 1 && s[0] != tokens * s[1]) ? -1 : step;
}

// A call that failed on the way to the device cannot be made again as if it had not begun.
PyObject* not_ok(pkv_status st, const char* where) {
  if (st != PKV_ERR_CUDA) return decline();
  PyObject* e = PyObject_CallFunction(error_type, "is", (int)st, where);
  if (!e) return nullptr;
  PyErr_SetObject(error_type, e);
  Py_DECREF(e);
  return nullptr;
}

// (handle, q, k_new, v_new, cos_sin, block_table, positions, rotary_positions, new_lens, interleaved, q_out, dev_status)
PyObject* rotary_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12) return decline();
  const Handle* h = static_cast<Handle*>(PyCapsule_GetPointer(a[0], kName));
  if (!h) return nullptr;
  try {
    bool ok = true;
    const at::Tensor *q = tensor(a[1], h, ok), *k = tensor(a[2], h, ok), *v = tensor(a[3], h, ok), *cs = tensor(a[4], h, ok),
                     *table = tensor(a[5], h, ok), *pos = tensor(a[6], h, ok), *turns = tensor(a[7], h, ok),
                     *lens = tensor(a[8], h, ok), *out = tensor(a[10], h, ok), *status = tensor(a[11], h, ok);
    if (!ok || !q || !k || !v || !cs || !table || q->dim() != 4 || k->dim() != 4 || v->dim() != 4 || cs->dim() != 2 ||
        table->dim() != 2)
      return decline();
    const int64_t B = k->size(0), T = k->size(1), H = h->cache->num_kv_heads, D = h->cache->head_dim, Hq = q->size(2);
    const int64_t kv[4] = {B, T, H, D}, qs[4] = {B, T, Hq, D}, rows[1] = {B}, each[2] = {B, T}, tab[2] = {B, table->size(1)};
    const auto type = k->scalar_type();
    pkv_dtype src;
    if (!type_of(type, src) || src == PKV_F32 || q->scalar_type() != type || v->scalar_type() != type ||
        k->sizes() != c10::IntArrayRef(kv) || v->sizes() != c10::IntArrayRef(kv) || q->sizes() != c10::IntArrayRef(qs) ||
        Hq == 0 || B == 0 || T == 0 || !shaped(cs, c10::kFloat, cs->sizes()) || !shaped(table, c10::kInt, tab) || !shaped(pos, c10::kInt, rows) ||
        !shaped_or_none(a[7], turns, c10::kInt, each) || !shaped_or_none(a[8], lens, c10::kInt, rows) ||
        !shaped_or_none(a[10], out, type, qs) || (a[11] != Py_None && !(status && status->scalar_type() == c10::kInt)) ||
        tab[1] > INT32_MAX || B > INT32_MAX || T > INT32_MAX || Hq > INT32_MAX || cs->size(0) > INT32_MAX ||
        cs->size(1) > INT32_MAX)
      return decline();
    const int64_t sq = token_stride(*q, B, T, Hq, D), sk = token_stride(*k, B, T, H, D), sv = token_stride(*v, B, T, H, D);
    if (sq < 0 || sk < 0 || sv < 0 || (a[9] != Py_True && a[9] != Py_False)) return decline();
    const c10::cuda::CUDAGuard on(h->device);
    at::Tensor made;
    if (!out) {
      made = at::detail::empty_cuda(qs, type, c10::Device(c10::kCUDA, h->device), std::nullopt);
      out = &made;
    }
    const pkv_status st = rotary_append_fn(
        h->cache, (int32_t)B, (int32_t)T, (int32_t)Hq, data<void>(q), data<void>(k), data<void>(v), src, sq, sk, sv,
        data<float>(cs), (int32_t)cs->size(0), (int32_t)cs->size(1), a[9] == Py_True, data<int32_t>(turns),
        data<int32_t>(table), (int32_t)tab[1], data<int32_t>(pos), data<int32_t>(lens), data<void>(out),
        data<int32_t>(status), c10::cuda::getCurrentCUDAStream(h->device).stream());
    if (st != PKV_OK) return not_ok(st, "rotary_append");
    if (!made.defined()) return Py_NewRef(a[10]);
    return THPVariable_Wrap(made);
  } catch (...) {
    PyErr_Clear();
    return decline();
  }
}

// (handle, q, block_table, seq_lens, mask, draft_lens, sm_scale, out, dtype of a new out (pkv_dtype), num_splits, dev_status)
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) return decline();
  const Handle* h = static_cast<Handle*>(PyCapsule_GetPointer(a[0], kName));
  if (!h) return nullptr;
  try {
    bool ok = true;
    const at::Tensor *q = tensor(a[1], h, ok), *table = tensor(a[2], h, ok), *lens = tensor(a[3], h, ok),
                     *mask = tensor(a[4], h, ok), *drafts = tensor(a[5], h, ok), *out = tensor(a[7], h, ok),
                     *status = tensor(a[10], h, ok);
    if (!ok || !q || !table || q->dim() != 4 || table->dim() != 2) return decline();
    const int64_t B = q->size(0), T = q->size(1), Hq = q->size(2), D = h->cache->head_dim, words = (T + 63) / 64;
    const int64_t qs[4] = {B, T, Hq, D}, rows[1] = {B}, tab[2] = {B, table->size(1)}, all[3] = {B, T, words};
    pkv_dtype qt, ot;
    long splits, made_type;
    if (B == 0 || T == 0 || T > 256 || !type_of(q->scalar_type(), qt) || !shaped(q, q->scalar_type(), qs) ||
        !shaped(table, c10::kInt, tab) || !shaped(lens, c10::kInt, rows) || !shaped_or_none(a[5], drafts, c10::kInt, rows) ||
        !(a[4] == Py_None || shaped(mask, c10::kLong, all) || shaped(mask, c10::kLong, c10::IntArrayRef(all + 1, 2))) ||
        (a[10] != Py_None && !(status && status->scalar_type() == c10::kInt)) || !number(a[9], splits) ||
        !number(a[8], made_type) || made_type > PKV_F32 || tab[1] > INT32_MAX || B > 1024 || Hq > INT32_MAX ||
        (out && (!type_of(out->scalar_type(), ot) || !shaped(out, out->scalar_type(), qs))))
      return decline();
    double scale = 1.0 / std::sqrt((double)D);
    if (a[6] != Py_None) {
      if (!PyFloat_Check(a[6])) return decline();
      scale = PyFloat_AS_DOUBLE(a[6]);
    }
    const c10::cuda::CUDAGuard on(h->device);
    // a captured call has memory of its own, which is made elsewhere
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) return decline();
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(h->device).stream();
    PyObject* key = Py_BuildValue("(nLLlL)", (Py_ssize_t)(intptr_t)stream, (long long)B, (long long)Hq, splits, (long long)T);
    if (!key) return nullptr;
    PyObject* kept = PyDict_GetItemWithError(h->fit, key);   // borrowed
    Py_DECREF(key);
    if (!kept || !THPVariable_CheckExact(kept)) {
      PyErr_Clear();
      return decline();
    }
    const at::Tensor ws = THPVariable_Unpack(kept);   // a reference of its own
    at::Tensor made;
    if (!out) {
      ot = (pkv_dtype)made_type;
      made = at::detail::empty_cuda(qs, ot == PKV_F16 ? c10::kHalf : ot == PKV_BF16 ? c10::kBFloat16 : c10::kFloat,
                                    c10::Device(c10::kCUDA, h->device), std::nullopt);
      out = &made;
    }
    // (nothing that could throw while the lock is held)
    const void* const q_at = data<void>(q);
    const int32_t *const table_at = data<int32_t>(table), *const lens_at = data<int32_t>(lens),
                  *const drafts_at = data<int32_t>(drafts);
    const int64_t* const mask_at = data<int64_t>(mask);
    void *const out_at = data<void>(out), *const ws_at = ws.data_ptr();
    int32_t* const status_at = data<int32_t>(status);
    const size_t ws_bytes = ws.nbytes();
    const int one_mask = mask && mask->dim() == 2;
    // threads take turns: a call's two launches follow one another on the stream
    PyObject* got = PyObject_CallOneArg(h->acquire, Py_False);
    if (!got) return nullptr;
    const bool mine = got == Py_True;
    Py_DECREF(got);
    if (!mine) return decline();
    const pkv_status st = tree_attention_fn(
        h->cache, (int32_t)B, (int32_t)T, (int32_t)Hq, q_at, qt, (float)scale, table_at, (int32_t)tab[1], lens_at, drafts_at,
        mask_at, one_mask, out_at, ot, (int32_t)splits, ws_at, ws_bytes, status_at, stream);
    PyObject* done = PyObject_CallNoArgs(h->release);
    if (!done) return nullptr;
    Py_DECREF(done);
    if (st != PKV_OK) return not_ok(st, "tree_attention");
    if (!made.defined()) return Py_NewRef(a[7]);
    return THPVariable_Wrap(made);
  } catch (...) {
    PyErr_Clear();
    return decline();
  }
}

// (handle, keep, keep_lens, block_table, first, dev_status)
PyObject* keep_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return decline();
  const Handle* h = static_cast<Handle*>(PyCapsule_GetPointer(a[0], kName));
  if (!h) return nullptr;
  try {
    bool ok = true;
    const at::Tensor *keep = tensor(a[1], h, ok), *lens = tensor(a[2], h, ok), *table = tensor(a[3], h, ok),
                     *first = tensor(a[4], h, ok), *status = tensor(a[5], h, ok);
    if (!ok || !keep || !table || keep->dim() != 2 || table->dim() != 2) return decline();
    const int64_t B = keep->size(0), K = keep->size(1), lists[2] = {B, K}, rows[1] = {B}, tab[2] = {B, table->size(1)};
    if (!shaped(keep, c10::kInt, lists) || !shaped_or_none(a[2], lens, c10::kInt, rows) || !shaped(table, c10::kInt, tab) ||
        !shaped(first, c10::kInt, rows) || (a[5] != Py_None && !(status && status->scalar_type() == c10::kInt)) ||
        B > INT32_MAX || K > INT32_MAX || tab[1] > INT32_MAX)
      return decline();
    const c10::cuda::CUDAGuard on(h->device);
    const pkv_status st = keep_tokens_fn(h->cache, (int32_t)B, (int32_t)K, data<int32_t>(keep), data<int32_t>(lens),
                                         data<int32_t>(table), (int32_t)tab[1], data<int32_t>(first), data<int32_t>(status),
                                         c10::cuda::getCurrentCUDAStream(h->device).stream());
    if (st != PKV_OK) return not_ok(st, "keep_tokens");
    Py_RETURN_NONE;
  } catch (...) {
    PyErr_Clear();
    return decline();
  }
}

// (address of the pkv_cache, device, workspaces, acquire, release); the cache outlives the handle
PyObject* handle(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || !PyDict_Check(a[2])) {
    PyErr_SetString(PyExc_TypeError, "handle(cache, device, workspaces, acquire, release)");
    return nullptr;
  }
  const void* cache = PyLong_AsVoidPtr(a[0]);
  const long device = PyLong_AsLong(a[1]);
  if (PyErr_Occurred()) return nullptr;
  Handle* h = new Handle{static_cast<const pkv_cache*>(cache), (c10::DeviceIndex)device, Py_NewRef(a[2]), Py_NewRef(a[3]),
                         Py_NewRef(a[4])};
  PyObject* c = PyCapsule_New(h, kName, drop);
  if (!c) delete h;
  return c;
}

// addresses of the library's entry points, in the order below, and the type of its errors
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind(rotary_append, tree_attention, keep_tokens, error)");
    return nullptr;
  }
  rotary_append_fn = reinterpret_cast<decltype(rotary_append_fn)>(PyLong_AsVoidPtr(a[0]));
  tree_attention_fn = reinterpret_cast<decltype(tree_attention_fn)>(PyLong_AsVoidPtr(a[1]));
  keep_tokens_fn = reinterpret_cast<decltype(keep_tokens_fn)>(PyLong_AsVoidPtr(a[2]));
  if (PyErr_Occurred()) return nullptr;
  Py_XDECREF(error_type);
  error_type = Py_NewRef(a[3]);
  Py_RETURN_NONE;
}

#define PKV_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PKV_FAST(rotary_append), PKV_FAST(tree_attention), PKV_FAST(keep_tokens), PKV_FAST(handle),
                         PKV_FAST(bind), {nullptr, nullptr, 0, nullptr}};
#undef PKV_FAST
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch() { return PyModule_Create(&module_def); }
