// Marshalling of the many-request calls without the interpreter: their tensors
// are checked here and handed to the library's C entry points.  A decode step
// of a small model is a handful of calls of 2 to 8 us on the GPU, and the same
// checks in Python with a ctypes call take 10 us each.
//
// A function returns the library's status, or None for a call that it leaves
// to the Python path, which knows every case (another current device, stream
// objects) and words the errors.  Nothing is kept between calls.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstring>

#include "flashloop.h"

namespace {

decltype(&flashloop_paged_plan) plan_fn;
decltype(&flashloop_paged_kv_write) write_fn;
decltype(&flashloop_prompt_attn) prompt_fn;
decltype(&flashloop_paged_attn) attn_fn;

struct NotPlain {};

// The arguments of a call whose tensors lie on the current device.
struct Call {
  flashloop_paged_params p;
  int dev = -1;
  at::ScalarType type = at::kBFloat16;  // of params.dtype
  void* stream = nullptr;

  Call(PyObject* params, PyObject* first, PyObject* on_stream) {
    Py_buffer view;
    if (PyObject_GetBuffer(params, &view, PyBUF_SIMPLE) != 0) throw NotPlain();
    const bool fits = view.len == (Py_ssize_t)sizeof(p);
    if (fits) std::memcpy(&p, view.buf, sizeof(p));
    PyBuffer_Release(&view);
    if (!fits || p.dtype < FLASHLOOP_DTYPE_BF16 || p.dtype > FLASHLOOP_DTYPE_FP16) throw NotPlain();
    if (p.batch < 0 || p.max_tokens < 0 || p.max_blocks < 0) throw NotPlain();
    type = p.dtype == FLASHLOOP_DTYPE_FP16 ? at::kHalf : at::kBFloat16;
    const at::Tensor& t = tensor(first);
    if (!t.is_cuda()) throw NotPlain();
    dev = t.get_device();
    if (c10::cuda::current_device() != dev) throw NotPlain();
    if (on_stream == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    } else if (PyLong_CheckExact(on_stream)) {
      stream = PyLong_AsVoidPtr(on_stream);
      if (PyErr_Occurred()) throw NotPlain();
    } else {
      throw NotPlain();
    }
  }

  static const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) throw NotPlain();
    return THPVariable_Unpack(o);
  }

  // A contiguous vector of at least n elements.
  void* vec(PyObject* o, long long n, at::ScalarType of) const {
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != of || !t.is_cuda() || t.get_device() != dev || t.numel() < n || !t.is_contiguous()) throw NotPlain();
    return t.data_ptr();
  }
  int32_t* ints(PyObject* o, long long n) const { return static_cast<int32_t*>(vec(o, n, at::kInt)); }

  // The same in rows of `row` elements: flat, or its last dimensions make up a row.
  void* in_rows(PyObject* o, long long n, long long row, at::ScalarType of) const {
    const at::Tensor& t = tensor(o);
    long long size = 1;
    int64_t d = t.dim();
    while (size != row && d > 0) size *= t.size(--d);
    if (n > 0 && size != row && t.dim() > 1) throw NotPlain();
    return vec(o, n, of);
  }
  int32_t* table(PyObject* o) const {
    return static_cast<int32_t*>(in_rows(o, (long long)p.batch * p.max_blocks, p.max_blocks, at::kInt));
  }
  float* lse(PyObject* o) const {
    return o == Py_None ? nullptr : static_cast<float*>(in_rows(o, (long long)p.max_tokens * p.n_heads, p.max_tokens, at::kFloat));
  }

  // [tokens, heads, head_dim]; a dimension of one may have any stride.
  flashloop_rows rows(PyObject* o, long long heads, at::ScalarType of, bool written = false) const {
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != of || !t.is_cuda() || t.get_device() != dev || t.dim() != 3 || t.size(0) != p.max_tokens ||
        t.size(1) != heads || t.size(2) != p.head_dim || t.stride(2) != 1)
      throw NotPlain();
    const int64_t st = t.stride(0), sh = t.stride(1);
    if (written && ((st == 0 && t.size(0) > 1) || (sh == 0 && heads > 1))) throw NotPlain();
    return {t.data_ptr(), t.size(0) > 1 ? st : p.head_dim, heads > 1 ? sh : p.head_dim};
  }

  // [n_pages, page_size, n_kv_heads, head_dim]
  flashloop_pages pages(PyObject* o, bool written = false) const {
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || t.dim() != 4 || t.size(0) != p.n_pages ||
        t.size(1) != p.page_size || t.size(2) != p.n_kv_heads || t.size(3) != p.head_dim || t.stride(3) != 1)
      throw NotPlain();
    const int64_t sp = t.stride(0), st = t.stride(1), sh = t.stride(2);
    if (written && ((sp == 0 && t.size(0) > 1) || st == 0 || (sh == 0 && t.size(2) > 1))) throw NotPlain();
    return {t.data_ptr(), t.size(0) > 1 ? sp : p.head_dim, st, t.size(2) > 1 ? sh : p.head_dim};
  }
};

// `body` marshals and launches; what it does not take, and whatever torch throws at an unusual
// tensor, is the Python path's.
template <typename Body>
PyObject* run(Py_ssize_t n, Py_ssize_t want, Body body) {
  if (n != want) Py_RETURN_NONE;
  try {
    return PyLong_FromLong(body());
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

template <typename Fn>
int without_gil(Fn fn) {
  PyThreadState* state = PyEval_SaveThread();
  const int rc = fn();
  PyEval_RestoreThread(state);
  return rc;
}

PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 13, [&] {
    const Call c(a[0], a[1], a[12]);
    const long long B = c.p.batch, T = c.p.max_tokens;
    int32_t *kv = c.ints(a[1], B), *add = c.ints(a[2], B), *stack = c.ints(a[3], 0), *n_free = c.ints(a[4], 1);
    const long long capacity = std::min<long long>(Call::tensor(a[3]).numel(), 0x7fffffff);  // at most n_pages of it count
    int32_t *table = c.table(a[5]), *cu = c.ints(a[6], B + 1), *kv_out = c.ints(a[7], B);
    int32_t *slot = c.ints(a[8], T), *pos = c.ints(a[9], T), *left = c.ints(a[10], 1), *err = c.ints(a[11], 1);
    return without_gil([&] {
      return plan_fn(&c.p, kv, add, stack, (int32_t)capacity, n_free, table, cu, kv_out, slot, pos, left, err, c.stream);
    });
  });
}

PyObject* kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 8, [&] {
    const Call c(a[0], a[4], a[7]);
    const at::ScalarType from = Call::tensor(a[1]).scalar_type();
    if (from != c.type && from != at::kFloat) throw NotPlain();
    const flashloop_rows k = c.rows(a[1], c.p.n_kv_heads, from), v = c.rows(a[2], c.p.n_kv_heads, from);
    const int32_t* slots = c.ints(a[3], c.p.max_tokens);
    const flashloop_pages kc = c.pages(a[4], true), vc = c.pages(a[5], true);
    int32_t* err = c.ints(a[6], 1);
    const int32_t src = from == at::kFloat ? FLASHLOOP_DTYPE_FP32 : c.p.dtype;
    return without_gil([&] { return write_fn(&c.p, &k, &v, src, slots, &kc, &vc, err, c.stream); });
  });
}

PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 9, [&] {
    const Call c(a[0], a[1], a[8]);
    const flashloop_rows q = c.rows(a[1], c.p.n_heads, c.type), k = c.rows(a[2], c.p.n_kv_heads, c.type);
    const flashloop_rows v = c.rows(a[3], c.p.n_kv_heads, c.type), o = c.rows(a[5], c.p.n_heads, c.type, true);
    const int32_t* cu = c.ints(a[4], c.p.batch + 1ll);
    float* lse = c.lse(a[6]);
    int32_t* err = c.ints(a[7], 1);
    return without_gil([&] { return prompt_fn(&c.p, &q, &k, &v, cu, &o, lse, err, c.stream); });
  });
}

PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 12, [&] {
    const Call c(a[0], a[1], a[11]);
    const long long B = c.p.batch;
    const flashloop_rows q = c.rows(a[1], c.p.n_heads, c.type), o = c.rows(a[7], c.p.n_heads, c.type, true);
    const flashloop_pages kc = c.pages(a[2]), vc = c.pages(a[3]);
    const int32_t *table = c.table(a[4]), *kv = c.ints(a[5], B), *cu = c.ints(a[6], B + 1);
    float* lse = c.lse(a[8]);
    const at::Tensor& ws = Call::tensor(a[9]);
    if (!ws.is_cuda() || ws.get_device() != c.dev || !ws.is_contiguous()) throw NotPlain();
    void* scratch = ws.data_ptr();
    const size_t bytes = ws.nbytes();
    int32_t* err = c.ints(a[10], 1);
    return without_gil([&] { return attn_fn(&c.p, &q, &kc, &vc, table, kv, cu, &o, lse, scratch, bytes, err, c.stream); });
  });
}

// The addresses of the library's entry points, in the order of the functions here.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[4];
  for (int i = 0; i < 4; ++i) {
    at[i] = n == 4 ? PyLong_AsVoidPtr(a[i]) : nullptr;
    if (PyErr_Occurred()) return nullptr;
    if (!at[i]) {
      PyErr_SetString(PyExc_ValueError, "four addresses");
      return nullptr;
    }
  }
  plan_fn = reinterpret_cast<decltype(plan_fn)>(at[0]);
  write_fn = reinterpret_cast<decltype(write_fn)>(at[1]);
  prompt_fn = reinterpret_cast<decltype(prompt_fn)>(at[2]);
  attn_fn = reinterpret_cast<decltype(attn_fn)>(at[3]);
  Py_RETURN_NONE;
}

template <typename Fn>
PyCFunction fast(Fn fn) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn));
}

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
  static PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                                  {"plan", fast(plan), METH_FASTCALL, nullptr},
                                  {"write", fast(kv_write), METH_FASTCALL, nullptr},
                                  {"prompt", fast(prompt), METH_FASTCALL, nullptr},
                                  {"attn", fast(attn), METH_FASTCALL, nullptr},
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
  PyObject* m = PyModule_Create(&module);
  // the build and the import look for this text in the file
  if (m && PyModule_AddStringConstant(m, "built_for", FLASHLOOP_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
