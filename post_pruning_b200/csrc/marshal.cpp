// Argument marshalling of the calls that are made once per token and layer
// (the 8-bit forward and the attention): tensors in, one call of the C ABI.
// The same checks as the Python functions of sgpt.py, which make up most of
// such a call's host time there. Nothing is computed here, and no argument
// error is reported: a call that is not plainly valid returns -1, and the
// Python function repeats the checks, raises or makes the call itself (as it
// makes every call where this module is not there).
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/sgpt.h"

namespace {

decltype(&sgpt_quant_tokens) f_quant_tokens = nullptr;
decltype(&sgpt_quant_tokens_silu) f_quant_tokens_silu = nullptr;
decltype(&sgpt_linear_i8) f_linear_i8 = nullptr;
decltype(&sgpt_attention) f_attention = nullptr;

constexpr auto kBf16 = at::kBFloat16, kF32 = at::kFloat, kI8 = at::kChar, kI32 = at::kInt;

// The operands of one call: tensors of one device, the current one.
struct Operands {
  const at::Tensor* t[8];
  bool ok = true;
  int device = -1;

  Operands(PyObject* const* args, int n) {
    device = c10::cuda::current_device();
    for (int i = 0; i < n && ok; ++i) {
      ok = THPVariable_Check(args[i]);
      if (!ok) break;
      t[i] = &THPVariable_Unpack(args[i]);
      ok = t[i]->is_cuda() && t[i]->get_device() == device && t[i]->layout() == at::kStrided;
    }
  }
  const at::Tensor& operator[](int i) const { return *t[i]; }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

bool is(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
  return t.scalar_type() == type && t.sizes().equals(at::IntArrayRef(shape)) && t.is_contiguous();
}
bool is_info(const at::Tensor& t) { return t.scalar_type() == kI32 && t.numel() >= 1; }

// bf16 [n, d] with contiguous rows: the row stride, or -1.
int64_t row_stride(const at::Tensor& t) {
  if (t.scalar_type() != kBf16 || t.dim() != 2 || t.stride(1) != 1) return -1;
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}
// bf16 [rows, heads, width] with consecutive heads: the row stride, or -1.
int64_t heads_stride(const at::Tensor& t) {
  if (t.scalar_type() != kBf16 || t.dim() != 3 || t.stride(2) != 1) return -1;
  if (t.stride(1) != t.size(2) && t.size(1) > 1) return -1;
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}
bool token_codes(const at::Tensor& q, const at::Tensor& scale, const at::Tensor& sums, int64_t n, int64_t d) {
  return is(q, kI8, {n, d}) && is(scale, kF32, {n}) && is(sums, kI32, {n});
}

template <class T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// Runs `call` (status >= 0, or -1: not plainly valid) without the GIL's holder
// waiting for a full launch queue, and lets no C++ exception out.
template <class F>
PyObject* answer(F&& call) {
  int status = -1;
  try {
    status = call();
  } catch (...) {
    status = -1;
  }
  return PyLong_FromLong(status);
}
template <class F, class... A>
int launch(F f, A... a) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = (int)f(a...);
  Py_END_ALLOW_THREADS
  return status;
}

PyObject* quant_tokens(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return answer([&]() -> int {
    if (nargs != 5 || !f_quant_tokens) return -1;
    const Operands o(args, 5);
    if (!o.ok) return -1;
    const int64_t ld = row_stride(o[0]);
    if (ld < 0 || !is_info(o[4])) return -1;
    const int64_t n = o[0].size(0), d = o[0].size(1);
    if (d > INT32_MAX || !token_codes(o[1], o[2], o[3], n, d)) return -1;
    return launch(f_quant_tokens, ptr<const uint16_t>(o[0]), n, (int)d, ld, ptr<int8_t>(o[1]), ptr<float>(o[2]),
                  ptr<int32_t>(o[3]), ptr<int>(o[4]), o.stream());
  });
}

PyObject* quant_tokens_silu(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return answer([&]() -> int {
    if (nargs != 6 || !f_quant_tokens_silu) return -1;
    const Operands o(args, 6);
    if (!o.ok) return -1;
    const int64_t ldg = row_stride(o[0]), ldu = row_stride(o[1]);
    if (ldg < 0 || ldu < 0 || !o[0].sizes().equals(o[1].sizes()) || !is_info(o[5])) return -1;
    const int64_t n = o[0].size(0), d = o[0].size(1);
    if (d > INT32_MAX || !token_codes(o[2], o[3], o[4], n, d)) return -1;
    return launch(f_quant_tokens_silu, ptr<const uint16_t>(o[0]), ptr<const uint16_t>(o[1]), n, (int)d, ldg, ldu,
                  ptr<int8_t>(o[2]), ptr<float>(o[3]), ptr<int32_t>(o[4]), ptr<int>(o[5]), o.stream());
  });
}

PyObject* linear_i8(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return answer([&]() -> int {
    if (nargs != 8 || !f_linear_i8 || !PyLong_CheckExact(args[7])) return -1;
    const Operands o(args, 7);
    if (!o.ok || !is_info(o[6]) || o[0].dim() != 2 || o[3].dim() != 2) return -1;
    int over = 0;
    const long qbits = PyLong_AsLongAndOverflow(args[7], &over);
    if (over || qbits < 2 || qbits > 8) return -1;
    const int64_t n = o[0].size(0), d_in = o[0].size(1), d_out = o[3].size(0);
    const bool bf16 = o[5].scalar_type() == kBf16;
    if (d_in > INT32_MAX || d_out > INT32_MAX || !token_codes(o[0], o[1], o[2], n, d_in)) return -1;
    if (!is(o[3], kI8, {d_out, d_in}) || !is(o[4], kF32, {d_out, 2}) || !is(o[5], bf16 ? kBf16 : kF32, {n, d_out}))
      return -1;
    return launch(f_linear_i8, ptr<const int8_t>(o[0]), ptr<const float>(o[1]), ptr<const int32_t>(o[2]), n,
                  ptr<const int8_t>(o[3]), ptr<const float>(o[4]), (int)qbits, (int)d_in, (int)d_out, ptr<void>(o[5]),
                  (int)bf16, ptr<int>(o[6]), o.stream());
  });
}

PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return answer([&]() -> int {
    if (nargs != 7 || !f_attention) return -1;
    const Operands o(args, 6);
    if (!o.ok || !is_info(o[5])) return -1;
    const at::Tensor &Q = o[0], &K = o[1], &V = o[2], &off = o[3], &O = o[4];
    const int64_t ldq = heads_stride(Q), ldk = heads_stride(K), ldv = heads_stride(V), ldo = heads_stride(O);
    if (ldq < 0 || ldk < 0 || ldv < 0 || ldo < 0) return -1;
    const int64_t n = Q.size(0), heads = Q.size(1), width = Q.size(2), kv = K.size(1);
    if (!O.sizes().equals(Q.sizes()) || !V.sizes().equals(K.sizes()) || K.size(0) != n || K.size(2) != width) return -1;
    if (off.scalar_type() != kI32 || off.dim() != 1 || off.size(0) < 1 || !off.is_contiguous()) return -1;
    if (heads > INT32_MAX || kv > INT32_MAX || width > INT32_MAX || off.size(0) > INT32_MAX) return -1;
    double scale = 1.0 / std::sqrt((double)width);
    if (args[6] != Py_None) {
      if (!PyFloat_CheckExact(args[6])) return -1;
      scale = PyFloat_AS_DOUBLE(args[6]);
    }
    return launch(f_attention, ptr<const uint16_t>(Q), ldq, ptr<const uint16_t>(K), ldk, ptr<const uint16_t>(V), ldv,
                  ptr<const int32_t>(off), (int)(off.size(0) - 1), n, (int)heads, (int)kv, (int)width, (float)scale,
                  ptr<uint16_t>(O), ldo, ptr<int>(o[5]), o.stream());
  });
}

// The addresses of the four C entries, in the order above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 4) {
    PyErr_SetString(PyExc_TypeError, "bind() takes four addresses");
    return nullptr;
  }
  void* a[4];
  for (int i = 0; i < 4; ++i) {
    a[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  f_quant_tokens = reinterpret_cast<decltype(f_quant_tokens)>(a[0]);
  f_quant_tokens_silu = reinterpret_cast<decltype(f_quant_tokens_silu)>(a[1]);
  f_linear_i8 = reinterpret_cast<decltype(f_linear_i8)>(a[2]);
  f_attention = reinterpret_cast<decltype(f_attention)>(a[3]);
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(quant_tokens), METHOD(quant_tokens_silu), METHOD(linear_i8), METHOD(attention),
                         METHOD(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

// With the torch it was compiled against: the binding takes it for that one only.
PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&module_def);
  if (m && PyModule_AddStringConstant(m, "torch_version", SGPT_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
