// Native part of the Python binding: the paged-cache calls in their plain form.
//
// A decode step's calls take the GPU a few microseconds, less than Python
// takes to look at their tensors: a windowed decode of four requests spent 31
// us in the binding (25 with its outputs and workspace given) around a library
// call of 6.  Here the same checks and allocations are made on the tensors'
// C++ objects.
//
// Each function handles the call whose tensors are all plain, contiguous, of
// the right types and sizes and on the current device, on the current stream,
// and returns None, having launched nothing, for every other one, also for
// one that the library refuses: the Python function then checks it in full,
// switches devices and streams, and names the argument that is wrong.  A
// library status past the refusals is returned as an int.
//
// Allocations and library calls run without the interpreter's lock: an
// allocation that frees cached memory waits for the GPU, a launch into a full
// queue waits for room in it, and what they wait for may be a host function on
// the stream that needs the lock.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mla.h"

namespace {

constexpr int64_t kPage = 64, kQk = 576, kV = 512, kFp4Row = 400;
constexpr int kMaxPages = ((1ll << 31) - 1) / kPage;

// The interpreter's lock given up for a scope.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// What a call's arguments have been found to be.  `ok` turns false at the
// first one that is not plain; nothing more is read then.
struct Call {
  PyObject* const* args;
  int device = -1;
  bool ok = true;

  Call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : args(a), ok(n == want) {
    if (ok) device = c10::cuda::current_device();
  }
  bool given(int i) const { return ok && args[i] != Py_None; }
  // tensor argument i of `dim` dimensions (-1: any); strided: rows may be apart
  const at::Tensor* tensor(int i, at::ScalarType type, int dim, bool strided = false) {
    if (!ok) return nullptr;
    if (!THPVariable_CheckExact(args[i])) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.defined() || t.layout() != at::kStrided || !t.device().is_cuda() || t.device().index() != device ||
        t.scalar_type() != type || (dim >= 0 && t.dim() != dim) || !(strided || t.is_contiguous())) {
      ok = false;
      return nullptr;
    }
    for (int64_t d = 0; d < t.dim(); ++d)
      if (t.size(d) > INT32_MAX) ok = false;
    return ok ? &t : nullptr;
  }
  void need(bool condition) { ok = ok && condition; }
  int integer(int i) {
    if (!ok) return 0;
    const long long v = PyLong_AsLongLong(args[i]);
    if ((v == -1 && PyErr_Occurred()) || v < INT32_MIN || v > INT32_MAX) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<int>(v);
  }
  float number(int i) {
    if (!ok) return 0;
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(v);
  }
  at::TensorOptions options(at::ScalarType type) const {
    return at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(device));
  }
  mla_stream_t stream() const {
    return reinterpret_cast<mla_stream_t>(
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
  }
  // output argument i: the tensor given, of exactly this shape, or none yet
  at::Tensor output(int i, at::ScalarType type, at::IntArrayRef shape) {
    if (!ok || args[i] == Py_None) return {};
    const at::Tensor* t = tensor(i, type, static_cast<int>(shape.size()));
    if (!t || t->sizes() != shape) {
      ok = false;
      return {};
    }
    return *t;
  }
  at::Tensor workspace(int i) {
    if (!ok || args[i] == Py_None) return {};
    if (!THPVariable_CheckExact(args[i])) {
      ok = false;
      return {};
    }
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    need(t.device().is_cuda() && t.device().index() == device && t.is_contiguous());
    return ok ? t : at::Tensor();
  }
  // a new tensor where none was given
  void fill(at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) const {
    if (!t.defined()) t = at::empty(shape, options(type));
  }
};

template <class T = void>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// Runs `body` (which returns a new reference or NULL for "not plain"); C++
// exceptions (an allocation that fails) become "not plain" too, and the Python
// function meets them in its turn.
template <class Body>
PyObject* guarded(Body body) {
  PyObject* r = nullptr;
  try {
    r = body();
  } catch (...) {
    r = nullptr;
  }
  if (r) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}
// NULL for a refusal, the status as an int for a failure
PyObject* failed(mla_status st) {
  if (st == MLA_ERR_INVALID_ARG || st == MLA_ERR_UNSUPPORTED || st == MLA_ERR_WORKSPACE) return nullptr;
  return PyLong_FromLong(st);
}
PyObject* tuple_of(std::initializer_list<const at::Tensor*> tensors) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor* x : tensors) {
    PyObject* o = THPVariable_Wrap(*x);
    if (!o) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// Paged cache at argument i with scales at argument k; sets is_fp8.
const at::Tensor* cache(Call& c, int i, int k, int* is_fp8, float** scales) {
  *scales = nullptr;
  if (!c.ok || !THPVariable_CheckExact(c.args[i])) {
    c.ok = false;
    return nullptr;
  }
  *is_fp8 = THPVariable_Unpack(c.args[i]).scalar_type() == at::kByte;
  const at::Tensor* kv = c.tensor(i, *is_fp8 ? at::kByte : at::kBFloat16, 4);
  const bool token = c.given(k);
  if (kv) c.need(kv->size(2) == 1 && kv->size(3) == (*is_fp8 ? (token ? 640 : 656) : kQk) && (*is_fp8 || !token));
  if (c.ok && token) {
    const at::Tensor* s = c.tensor(k, at::kFloat, -1);
    if (s) c.need(s->numel() == kv->size(0) * kv->size(1));
    if (c.ok) *scales = ptr<float>(*s);
  }
  return c.ok ? kv : nullptr;
}

// Paged cache of FP4 rows at argument i with nothing at argument k; NULL, and
// the call still plain, if its rows are others.
const at::Tensor* fp4_cache(Call& c, int i, int k) {
  if (!c.ok || !THPVariable_CheckExact(c.args[i])) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(c.args[i]);
  if (!t.defined() || t.scalar_type() != at::kByte || t.dim() != 4 || t.size(3) != kFp4Row) return nullptr;
  const at::Tensor* kv = c.tensor(i, at::kByte, 4);
  c.need(kv && kv->size(2) == 1 && !c.given(k));
  return c.ok ? kv : nullptr;
}

// (cache_lengths, new_tokens, free_pages, free_cursor, block_table, num_tokens, num_pages or None,
//  cache_seqlens, row_offsets, slot_map, next_cursor)
PyObject* assign_pages(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 11);
    const at::Tensor* in[5];
    for (int i = 0; i < 5; ++i) in[i] = c.tensor(i, at::kInt, i == 4 ? 2 : 1);
    if (!c.ok) return nullptr;
    mla_assign_pages_args a{};
    const int64_t batch = in[0]->size(0);
    a.num_tokens = c.integer(5);
    a.num_pages = c.given(6) ? c.integer(6) : kMaxPages;
    c.need(in[1]->size(0) == batch && in[4]->size(0) == batch && in[3]->size(0) == 1 && a.num_tokens >= 0);
    at::Tensor lens = c.output(7, at::kInt, {batch}), offsets = c.output(8, at::kInt, {batch + 1}),
               slots = c.output(9, at::kInt, {a.num_tokens}), cursor = c.output(10, at::kInt, {1});
    if (!c.ok) return nullptr;
    a.cache_lengths = ptr<int32_t>(*in[0]);
    a.new_tokens = ptr<int32_t>(*in[1]);
    a.batch = static_cast<int>(batch);
    a.free_pages = ptr<int32_t>(*in[2]);
    a.num_free = static_cast<int>(in[2]->size(0));
    a.free_cursor = ptr<int32_t>(*in[3]);
    a.block_table = ptr<int32_t>(*in[4]);
    a.block_table_stride = static_cast<int>(in[4]->size(1));
    const mla_stream_t stream = c.stream();
    mla_status st;
    {
      const Unlocked unlocked;
      c.fill(lens, at::kInt, {batch});
      c.fill(offsets, at::kInt, {batch + 1});
      c.fill(slots, at::kInt, {a.num_tokens});
      c.fill(cursor, at::kInt, {1});
      a.cache_seqlens = ptr<int32_t>(lens);
      a.row_offsets = ptr<int32_t>(offsets);
      a.slot_map = ptr<int32_t>(slots);
      a.next_cursor = ptr<int32_t>(cursor);
      st = mla_assign_pages(&a, stream);
    }
    return st == MLA_OK ? tuple_of({&lens, &offsets, &slots, &cursor}) : failed(st);
  });
}

// (latent, rope, slot_map, kvcache, kv_scales or None) -> True
PyObject* cache_store(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 5);
    const at::Tensor* latent = c.tensor(0, at::kBFloat16, 2, true);
    const at::Tensor* rope = c.tensor(1, at::kBFloat16, 2, true);
    const at::Tensor* slots = c.tensor(2, at::kInt, 1);
    mla_cache_store_args a{};
    const at::Tensor* fp4 = fp4_cache(c, 3, 4);
    const at::Tensor* kv = fp4 ? fp4 : cache(c, 3, 4, &a.is_fp8, &a.kv_scales);
    if (!c.ok) return nullptr;
    const int64_t tokens = latent->size(0);
    c.need(latent->size(1) == kV && rope->size(1) == kQk - kV && rope->size(0) == tokens && slots->size(0) == tokens &&
           latent->stride(1) == 1 && rope->stride(1) == 1);
    if (!c.ok) return nullptr;
    a.latent = ptr(*latent);
    a.latent_stride = tokens > 1 ? latent->stride(0) : kV;
    a.rope = ptr(*rope);
    a.rope_stride = tokens > 1 ? rope->stride(0) : kV;
    a.slot_map = ptr<int32_t>(*slots);
    a.num_tokens = static_cast<int>(tokens);
    a.kvcache = ptr(*kv);
    a.num_pages = static_cast<int>(kv->size(0));
    a.page_size = static_cast<int>(kv->size(1));
    const mla_stream_t stream = c.stream();
    mla_status st;
    {
      const Unlocked unlocked;
      if (fp4) {
        const mla_fp4_cache_store_args f{a.latent,     a.latent_stride, a.rope,      a.rope_stride, a.slot_map,
                                         a.num_tokens, a.kvcache,       a.num_pages, a.page_size};
        st = mla_fp4_cache_store(&f, stream);
      } else {
        st = mla_cache_store(&a, stream);
      }
    }
    if (st != MLA_OK) return failed(st);
    Py_RETURN_TRUE;
  });
}

// (kvcache, block_table, row_offsets, num_tokens, starts or None, kv_scales or None, out or None)
PyObject* cache_load(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 7);
    mla_cache_load_args a{};
    int is_fp8 = 0;
    float* scales = nullptr;
    const at::Tensor* fp4 = fp4_cache(c, 0, 5);
    const at::Tensor* kv = fp4 ? fp4 : cache(c, 0, 5, &is_fp8, &scales);
    const at::Tensor* table = c.tensor(1, at::kInt, 2);
    const at::Tensor* offsets = c.tensor(2, at::kInt, 1);
    a.num_tokens = c.integer(3);
    const at::Tensor* starts = c.given(4) ? c.tensor(4, at::kInt, 1) : nullptr;
    if (!c.ok) return nullptr;
    const int64_t batch = table->size(0);
    c.need(offsets->size(0) == batch + 1 && (!starts || starts->size(0) == batch) && a.num_tokens >= 0);
    at::Tensor out = c.output(6, at::kBFloat16, {a.num_tokens, kQk});
    if (!c.ok) return nullptr;
    a.kvcache = ptr(*kv);
    a.num_pages = static_cast<int>(kv->size(0));
    a.page_size = static_cast<int>(kv->size(1));
    a.format = fp4 ? MLA_CACHE_FP4 : scales ? MLA_CACHE_FP8_TOKEN : is_fp8 ? MLA_CACHE_FP8 : MLA_CACHE_BF16;
    a.kv_scales = scales;
    a.block_table = ptr<int32_t>(*table);
    a.block_table_stride = static_cast<int>(table->size(1));
    a.batch = static_cast<int>(batch);
    a.starts = starts ? ptr<int32_t>(*starts) : nullptr;
    a.row_offsets = ptr<int32_t>(*offsets);
    const mla_stream_t stream = c.stream();
    mla_status st;
    {
      const Unlocked unlocked;
      c.fill(out, at::kBFloat16, {a.num_tokens, kQk});
      a.out = ptr(out);
      st = mla_cache_load(&a, stream);
    }
    return st == MLA_OK ? THPVariable_Wrap(out) : failed(st);
  });
}

// What the decode calls share: q, kvcache (`kv`, checked by the caller),
// block_table and cache_seqlens at the given places, the common fields of their
// argument structs.
template <class Args>
const at::Tensor* decode_io(Call& c, Args* a, const at::Tensor* kv, int table, int lens) {
  const at::Tensor* q = c.tensor(0, at::kBFloat16, 4);
  const at::Tensor* bt = c.tensor(table, at::kInt, 2);
  const at::Tensor* sl = c.tensor(lens, at::kInt, 1);
  if (!c.ok) return nullptr;
  c.need(q->size(3) == kQk && bt->size(0) == q->size(0) && sl->size(0) == q->size(0));
  a->q = ptr(*q);
  a->batch = static_cast<int>(q->size(0));
  a->s_q = static_cast<int>(q->size(1));
  a->h_q = static_cast<int>(q->size(2));
  a->kvcache = ptr(*kv);
  a->num_pages = static_cast<int>(kv->size(0));
  a->page_size = static_cast<int>(kv->size(1));
  a->block_table = ptr<int32_t>(*bt);
  a->block_table_stride = static_cast<int>(bt->size(1));
  a->cache_seqlens = ptr<int32_t>(*sl);
  return c.ok ? q : nullptr;
}
// Outputs at arguments i and i + 1, the workspace at i + 2, then the library call.
template <class Args, class Run>
PyObject* decode_run(Call& c, Args* a, const at::Tensor& q, int i, size_t bytes, Run run) {
  const int64_t out_shape[] = {q.size(0), q.size(1), q.size(2), kV};
  const at::IntArrayRef rows(out_shape, 3);
  at::Tensor out = c.output(i, at::kBFloat16, out_shape), lse = c.output(i + 1, at::kFloat, rows);
  at::Tensor ws = c.workspace(i + 2);
  if (!c.ok) return nullptr;
  const mla_stream_t stream = c.stream();
  mla_status st;
  {
    const Unlocked unlocked;
    c.fill(out, at::kBFloat16, out_shape);
    c.fill(lse, at::kFloat, rows);
    c.fill(ws, at::kByte, {static_cast<int64_t>(bytes)});
    a->workspace = ptr(ws);
    a->workspace_bytes = ws.nbytes();
    a->out = ptr(out);
    a->lse = ptr<float>(lse);
    st = run(a, stream);
  }
  return st == MLA_OK ? tuple_of({&out, &lse}) : failed(st);
}

// (q, kvcache, block_table, cache_seqlens, sm_scale, window, sinks, kv_scales, out, lse, workspace)
PyObject* window_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 11);
    if (const at::Tensor* kv = fp4_cache(c, 1, 7)) {
      mla_fp4_decode_args a{};
      const at::Tensor* q = decode_io(c, &a, kv, 2, 3);
      a.sm_scale = c.number(4);
      a.window = c.integer(5);
      a.sinks = c.integer(6);
      size_t bytes = 0;
      if (!c.ok || mla_fp4_decode_workspace_size(a.batch, a.h_q, a.s_q, &bytes) != MLA_OK) return nullptr;
      return decode_run(c, &a, *q, 8, bytes, mla_fp4_decode);
    }
    mla_window_decode_args a{};
    float* scales = nullptr;
    const at::Tensor* kv = cache(c, 1, 7, &a.is_fp8, &scales);
    const at::Tensor* q = decode_io(c, &a, kv, 2, 3);
    a.kv_scales = scales;
    a.sm_scale = c.number(4);
    a.window = c.integer(5);
    a.sinks = c.integer(6);
    size_t bytes = 0;
    if (!c.ok || mla_window_decode_workspace_size(a.batch, a.h_q, a.s_q, a.is_fp8, &bytes) != MLA_OK) return nullptr;
    return decode_run(c, &a, *q, 8, bytes, mla_window_decode);
  });
}

// (q, kvcache, prefix_table, prefix_length, block_table, cache_seqlens, sm_scale, is_causal, kv_scales, out,
//  lse, workspace)
PyObject* shared_prefix_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 12);
    mla_shared_prefix_decode_args a{};
    float* scales = nullptr;
    const at::Tensor* kv = cache(c, 1, 8, &a.is_fp8, &scales);
    const at::Tensor* q = decode_io(c, &a, kv, 4, 5);
    a.kv_scales = scales;
    const at::Tensor* table = c.tensor(2, at::kInt, 1);
    const at::Tensor* length = c.tensor(3, at::kInt, 1);
    a.sm_scale = c.number(6);
    if (!c.ok || length->size(0) != 1) return nullptr;
    const int causal = PyObject_IsTrue(args[7]);
    if (causal < 0) return nullptr;
    a.prefix_table = ptr<int32_t>(*table);
    a.prefix_table_len = static_cast<int>(table->size(0));
    a.prefix_length = ptr<int32_t>(*length);
    a.is_causal = causal;
    size_t bytes = 0;
    if (mla_shared_prefix_decode_workspace_size(a.batch, a.h_q, a.s_q, a.prefix_table_len, a.is_fp8, &bytes) != MLA_OK)
      return nullptr;
    return decode_run(c, &a, *q, 9, bytes, mla_shared_prefix_decode);
  });
}

// (q, k_nope, k_rope, v, q_offsets, k_offsets, sm_scale, is_causal, out, lse, workspace)
PyObject* prompt_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 11);
    const at::Tensor* q = c.tensor(0, at::kBFloat16, 3, true);
    const at::Tensor* k = c.tensor(1, at::kBFloat16, 3, true);
    const at::Tensor* rope = c.tensor(2, at::kBFloat16, 2, true);
    const at::Tensor* v = c.tensor(3, at::kBFloat16, 3, true);
    const at::Tensor* qo = c.tensor(4, at::kInt, 1);
    const at::Tensor* ko = c.tensor(5, at::kInt, 1);
    mla_prompt_attention_args a{};
    a.sm_scale = c.number(6);
    if (!c.ok) return nullptr;
    a.is_causal = PyObject_IsTrue(args[7]);
    const int64_t rows = q->size(0), heads = q->size(1);
    c.need(a.is_causal >= 0 && q->size(2) == 192 && k->size(2) == 128 && v->sizes() == k->sizes() && rope->size(1) == 64 &&
           rope->size(0) == k->size(0) && q->stride(2) == 1 && k->stride(2) == 1 && v->stride(2) == 1 &&
           rope->stride(1) == 1 && qo->size(0) == ko->size(0) && qo->size(0) >= 2);
    const int64_t out_shape[] = {rows, heads, 128};
    const at::IntArrayRef lse_shape(out_shape, 2);
    at::Tensor out = c.output(8, at::kBFloat16, out_shape), lse = c.output(9, at::kFloat, lse_shape);
    at::Tensor ws = c.workspace(10);
    size_t bytes = 0;
    if (!c.ok || mla_prompt_attention_workspace_size(static_cast<int>(rows), static_cast<int>(k->size(0)), static_cast<int>(heads),
                                                     static_cast<int>(qo->size(0) - 1), &bytes) != MLA_OK)
      return nullptr;
    a.q = ptr(*q);
    a.q_stride = q->stride(0);
    a.q_head_stride = q->stride(1);
    a.num_q = static_cast<int>(rows);
    a.h_q = static_cast<int>(heads);
    a.k_nope = ptr(*k);
    a.k_nope_stride = k->stride(0);
    a.k_nope_head_stride = k->stride(1);
    a.k_rope = ptr(*rope);
    a.k_rope_stride = rope->stride(0);
    a.v = ptr(*v);
    a.v_stride = v->stride(0);
    a.v_head_stride = v->stride(1);
    a.num_k = static_cast<int>(k->size(0));
    a.h_kv = static_cast<int>(k->size(1));
    a.q_offsets = ptr<int32_t>(*qo);
    a.k_offsets = ptr<int32_t>(*ko);
    a.batch = static_cast<int>(qo->size(0) - 1);
    const mla_stream_t stream = c.stream();
    mla_status st;
    {
      const Unlocked unlocked;
      c.fill(out, at::kBFloat16, out_shape);
      c.fill(lse, at::kFloat, lse_shape);
      c.fill(ws, at::kByte, {static_cast<int64_t>(bytes)});
      a.workspace = ptr(ws);
      a.workspace_bytes = ws.nbytes();
      a.out = ptr(out);
      a.lse = ptr<float>(lse);
      st = mla_prompt_attention(&a, stream);
    }
    return st == MLA_OK ? tuple_of({&out, &lse}) : failed(st);
  });
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(assign_pages), ENTRY(cache_store), ENTRY(cache_load), ENTRY(prompt_attention),
                         ENTRY(window_decode), ENTRY(shared_prefix_decode),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mla_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_binding() { return PyModule_Create(&module); }
