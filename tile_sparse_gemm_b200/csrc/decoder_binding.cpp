// CPython extension over the C ABI's decoder-layer calls (include/patch.h) for
// the calls of a decode step.  Their kernels take 1.5 to 15 us, less than the
// same checks and the marshalling take in Python (14 us for rotary positions,
// 18 us for attention); here they take about 2 us beside the launch.
//
// Each function does the ordinary call: every argument as documented, on the
// current device and stream.  Anything else (another device, a wrong type or
// shape, a torch dispatch mode that watches allocations) makes it return None without having done anything, and the caller
// (decoder.py) takes its own way through the same checks, which name the fault.
// A status code other than PATCH_OK comes back as an int.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "patch.h"

namespace {

decltype(&patch_rope) rope_fn;
decltype(&patch_kv8_append) append_fn;
decltype(&patch_attn_kv8) attn_fn;
decltype(&patch_gemm4) gemm4_fn;

using at::ScalarType;
using at::Tensor;

int code_of(ScalarType t) {  // PATCH_DTYPE_*, -1: none
  return t == ScalarType::BFloat16 ? PATCH_DTYPE_BF16 : t == ScalarType::Half ? PATCH_DTYPE_FP16 : t == ScalarType::Float ? PATCH_DTYPE_FP32 : -1;
}

// What a call has been given so far; `ok` turns false at the first thing out of the ordinary.
struct Args {
  bool ok = true;
  c10::DeviceIndex device = -1;

  const Tensor* tensor(PyObject* o) {  // a CUDA tensor of the call's device (the first one's, which must be current)
    if (!ok || !THPVariable_Check(o)) return fail();
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) return fail();
    if (device < 0) device = t.get_device();
    if (t.get_device() != device) return fail();
    return &t;
  }
  const Tensor* tensor(PyObject* o, ScalarType type, int dim) {
    const Tensor* t = tensor(o);
    if (!t || t->scalar_type() != type || t->dim() != dim || !t->is_contiguous()) return fail();
    return t;
  }
  // rows of heads [T][H][D], elements in a row
  const Tensor* heads(PyObject* o, ScalarType type, patch_heads* h) {
    const Tensor* t = tensor(o);
    if (!t || t->scalar_type() != type || t->dim() != 3 || (t->stride(2) != 1 && t->size(2) > 1)) return fail();
    *h = {t->data_ptr(), t->size(1), t->stride(0), t->stride(1)};
    return t;
  }
  const Tensor* fail() {
    ok = false;
    return nullptr;
  }
  // ... and a torch dispatch mode, which would not see the outputs' allocation
  bool current() const {
    return ok && device == c10::cuda::current_device() && !c10::impl::TorchDispatchModeTLS::any_modes_set();
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
  int32_t* status(PyObject* o) {
    if (o == Py_None) return nullptr;
    const Tensor* t = tensor(o, ScalarType::Int, 1);
    return t ? static_cast<int32_t*>(t->data_ptr()) : nullptr;
  }
};

Tensor empty(const Args& a, at::IntArrayRef size, ScalarType type) {
  return at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, a.device), std::nullopt);
}
patch_heads heads_of(const Tensor& t) { return {t.data_ptr(), t.size(1), t.stride(0), t.stride(1)}; }

int layout_of(PyObject* o) {
  if (!PyUnicode_Check(o)) return -1;
  if (PyUnicode_CompareWithASCIIString(o, "half") == 0) return PATCH_ROPE_HALF;
  return PyUnicode_CompareWithASCIIString(o, "interleaved") == 0 ? PATCH_ROPE_INTERLEAVED : -1;
}

PyObject* code(patch_status_t st) { return PyLong_FromLong(st); }

// C++ exceptions (an allocation that fails) become Python's
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (q, k or None, positions, table, layout, backward, q_out or None, k_out or None, status or None) -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    patch_heads hq, hk, ho, hko;
    const int layout = n == 9 ? layout_of(o[4]) : -1;
    if (layout < 0 || !PyBool_Check(o[5])) Py_RETURN_NONE;
    const Tensor* q = a.tensor(o[0]);
    if (!q || code_of(q->scalar_type()) < 0 || !a.heads(o[0], q->scalar_type(), &hq)) Py_RETURN_NONE;
    const int64_t T = q->size(0), D = q->size(2);
    const ScalarType type = q->scalar_type();
    const Tensor* k = nullptr;
    if (o[1] != Py_None) {
      k = a.heads(o[1], type, &hk);
      if (!k || k->size(0) != T || k->size(2) != D) Py_RETURN_NONE;
    } else if (o[7] != Py_None) {
      Py_RETURN_NONE;
    }
    const Tensor *pos = a.tensor(o[2], ScalarType::Int, 1), *table = a.tensor(o[3], ScalarType::Float, 3);
    if (!pos || !table || pos->size(0) != T || table->size(2) != 2) Py_RETURN_NONE;
    int32_t* status = a.status(o[8]);
    Tensor q_new, k_new;
    if (o[6] != Py_None) {
      const Tensor* t = a.heads(o[6], type, &ho);
      if (!t || t->sizes() != q->sizes()) Py_RETURN_NONE;
    }
    if (o[7] != Py_None) {
      const Tensor* t = a.heads(o[7], type, &hko);
      if (!t || t->sizes() != k->sizes()) Py_RETURN_NONE;
    }
    if (!a.current()) Py_RETURN_NONE;
    if (o[6] == Py_None) ho = heads_of(q_new = empty(a, q->sizes(), type));
    if (k && o[7] == Py_None) hko = heads_of(k_new = empty(a, k->sizes(), type));
    const patch_status_t st =
        rope_fn(&hq, k ? &hk : nullptr, &ho, k ? &hko : nullptr, T, D, code_of(type),
                static_cast<const int32_t*>(pos->data_ptr()), static_cast<const float*>(table->data_ptr()),
                table->size(0), 2 * table->size(1), layout, o[5] == Py_True, status, a.stream());
    if (st != PATCH_OK) return code(st);
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, q_new.defined() ? THPVariable_Wrap(q_new) : Py_NewRef(o[6]));
    PyTuple_SET_ITEM(r, 1, k_new.defined() ? THPVariable_Wrap(k_new) : Py_NewRef(o[7]));
    return r;
  });
}

// cache tensors k, v, k_scale, v_scale at o[0 .. 3]
bool cache_of(Args& a, PyObject* const* o, patch_kv8_cache* c) {
  const Tensor* k = a.tensor(o[0], ScalarType::Float8_e4m3fn, 4);
  const Tensor* v = a.tensor(o[1], ScalarType::Float8_e4m3fn, 4);
  const Tensor *ks = a.tensor(o[2], ScalarType::Float, 2), *vs = a.tensor(o[3], ScalarType::Float, 2);
  if (!k || !v || !ks || !vs || v->sizes() != k->sizes() || ks->size(0) != k->size(0) || ks->size(1) != k->size(1) ||
      vs->sizes() != ks->sizes())
    return false;
  *c = {k->data_ptr(), v->data_ptr(), static_cast<float*>(ks->data_ptr()), static_cast<float*>(vs->data_ptr()),
        k->size(0), k->size(1), k->size(2), k->size(3)};
  return true;
}

// block table, lengths [batch] and row offsets [batch + 1] or None at o[0 .. 2]
struct Sequences {
  const int32_t *table, *lens, *cu;
  int64_t batch, max_pages;
};
bool sequences_of(Args& a, PyObject* const* o, Sequences* s) {
  const Tensor *bt = a.tensor(o[0], ScalarType::Int, 2), *lens = a.tensor(o[1], ScalarType::Int, 1);
  if (!bt || !lens || lens->size(0) != bt->size(0)) return false;
  *s = {static_cast<const int32_t*>(bt->data_ptr()), static_cast<const int32_t*>(lens->data_ptr()), nullptr,
        bt->size(0), bt->size(1)};
  if (o[2] != Py_None) {
    const Tensor* cu = a.tensor(o[2], ScalarType::Int, 1);
    if (!cu || cu->size(0) != s->batch + 1) return false;
    s->cu = static_cast<const int32_t*>(cu->data_ptr());
  }
  return true;
}

// (k, v, cache x 4, block_table, past_lens, cu_new or None, table or None, layout, status or None) -> 0
PyObject* append(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    patch_kv8_cache c;
    patch_heads hk, hv;
    Sequences s;
    const int layout = n == 12 ? layout_of(o[10]) : -1;
    if (layout < 0 || !cache_of(a, o + 2, &c)) Py_RETURN_NONE;
    const Tensor* k = a.tensor(o[0]);
    if (!k || code_of(k->scalar_type()) < 0 || k->scalar_type() == ScalarType::Float) Py_RETURN_NONE;
    k = a.heads(o[0], k->scalar_type(), &hk);
    const Tensor* v = k ? a.heads(o[1], k->scalar_type(), &hv) : nullptr;
    if (!v || k->sizes() != v->sizes() || k->size(1) != c.kv_heads || k->size(2) != c.head_dim ||
        !sequences_of(a, o + 6, &s))
      Py_RETURN_NONE;
    const Tensor* table = nullptr;
    if (o[9] != Py_None) {
      table = a.tensor(o[9], ScalarType::Float, 3);
      if (!table || table->size(2) != 2) Py_RETURN_NONE;
    }
    int32_t* status = a.status(o[11]);
    if (!a.current()) Py_RETURN_NONE;
    return code(append_fn(&hk, &hv, k->size(0), code_of(k->scalar_type()), &c, s.table, s.max_pages, s.lens, s.cu,
                          s.batch, table ? static_cast<const float*>(table->data_ptr()) : nullptr,
                          table ? table->size(0) : 0, table ? 2 * table->size(1) : 0, layout, status, a.stream()));
  });
}

// (q, cache x 4, block_table, kv_lens, cu_q or None, scale or None, causal, window, out or None, want_lse, workspace,
//  status or None, wait_limit_us) -> out or (out, lse)
PyObject* attn(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    patch_kv8_cache c;
    patch_heads hq, ho;
    Sequences s;
    if (n != 16 || !PyBool_Check(o[9]) || !PyLong_Check(o[10]) || !PyBool_Check(o[12]) || !PyLong_Check(o[15]) ||
        !cache_of(a, o + 1, &c))
      Py_RETURN_NONE;
    const Tensor* q = a.tensor(o[0]);
    if (!q || code_of(q->scalar_type()) < 0 || q->scalar_type() == ScalarType::Float) Py_RETURN_NONE;
    const ScalarType type = q->scalar_type();
    q = a.heads(o[0], type, &hq);
    if (!q || q->size(2) != c.head_dim || c.kv_heads < 1 || q->size(1) % c.kv_heads || !sequences_of(a, o + 5, &s))
      Py_RETURN_NONE;
    double scale = 1.0 / std::sqrt(double(c.head_dim));
    if (o[8] != Py_None) {
      if (!PyFloat_Check(o[8])) Py_RETURN_NONE;
      scale = PyFloat_AS_DOUBLE(o[8]);
    }
    const long long window = PyLong_AsLongLong(o[10]), limit = PyLong_AsLongLong(o[15]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    if (limit < 0) Py_RETURN_NONE;
    const Tensor* ws = a.tensor(o[13], ScalarType::Byte, 1);
    int32_t* status = a.status(o[14]);
    Tensor out, lse;
    if (o[11] != Py_None) {
      const Tensor* t = a.heads(o[11], type, &ho);
      if (!t || t->sizes() != q->sizes()) Py_RETURN_NONE;
    }
    if (!ws || !a.current()) Py_RETURN_NONE;
    if (o[11] == Py_None) ho = heads_of(out = empty(a, q->sizes(), type));
    if (o[12] == Py_True) lse = empty(a, {q->size(0), q->size(1)}, ScalarType::Float);
    const patch_status_t st =
        attn_fn(&hq, q->size(0), code_of(type), &c, s.table, s.max_pages, s.lens, s.cu, s.batch, float(scale),
                o[9] == Py_True, window, &ho, lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
                ws->data_ptr(), size_t(ws->numel()), status, a.stream(), uint64_t(limit));
    if (st != PATCH_OK) return code(st);
    PyObject* r = out.defined() ? THPVariable_Wrap(out) : Py_NewRef(o[11]);
    if (!lse.defined()) return r;
    PyObject* both = PyTuple_New(2);
    PyTuple_SET_ITEM(both, 0, r);
    PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(lse));
    return both;
  });
}

// (X, codes, scales, group, Y or None, status or None) -> Y
PyObject* gemm4(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    if (n != 6 || !PyLong_Check(o[3])) Py_RETURN_NONE;
    const long group = PyLong_AsLong(o[3]);
    if (group != 32 && group != 64 && group != 128) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    const Tensor *codes = a.tensor(o[1], ScalarType::Byte, 2), *scales = a.tensor(o[2]), *x = a.tensor(o[0]);
    if (!codes || !scales || !x || x->dim() != 2 || !x->is_contiguous() || scales->dim() != 2 || !scales->is_contiguous())
      Py_RETURN_NONE;
    const int st_code = code_of(scales->scalar_type()), xt = code_of(x->scalar_type());
    const int64_t N = codes->size(0), K = 2 * codes->size(1), M = x->size(0);
    if (st_code < 0 || st_code == PATCH_DTYPE_FP32 || xt < 0 || xt == PATCH_DTYPE_FP32 || K % group || x->size(1) != K ||
        scales->size(0) != N || scales->size(1) != K / group)
      Py_RETURN_NONE;
    int32_t* status = a.status(o[5]);
    const Tensor* y = nullptr;
    if (o[4] != Py_None) {
      y = a.tensor(o[4], x->scalar_type(), 2);
      if (!y || y->size(0) != M || y->size(1) != N) Py_RETURN_NONE;
    }
    if (!a.current()) Py_RETURN_NONE;
    Tensor fresh;
    if (!y) fresh = empty(a, {M, N}, x->scalar_type());
    const patch_weight4 w = {N, K, int32_t(group), st_code, codes->data_ptr(), scales->data_ptr()};
    const patch_status_t st = gemm4_fn(x->data_ptr(), M, xt, &w, y ? y->data_ptr() : fresh.data_ptr(), status, a.stream());
    if (st != PATCH_OK) return code(st);
    return y ? Py_NewRef(o[4]) : THPVariable_Wrap(fresh);
  });
}

// the library's entry points, as addresses: patch_rope, patch_kv8_append, patch_attn_kv8, patch_gemm4
PyObject* bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) p[i] = PyLong_AsVoidPtr(o[i]);
  if (PyErr_Occurred()) return nullptr;
  rope_fn = reinterpret_cast<decltype(rope_fn)>(p[0]);
  append_fn = reinterpret_cast<decltype(append_fn)>(p[1]);
  attn_fn = reinterpret_cast<decltype(attn_fn)>(p[2]);
  gemm4_fn = reinterpret_cast<decltype(gemm4_fn)>(p[3]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(bind), nullptr},   {"rope", FAST(rope), nullptr},   {"append", FAST(append), nullptr},
                         {"attn", FAST(attn), nullptr},   {"gemm4", FAST(gemm4), nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decoder_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decoder_binding() { return PyModule_Create(&module); }
