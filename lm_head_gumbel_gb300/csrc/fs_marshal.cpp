// fs_marshal.cpp -- argument marshalling of the operators of fs_vocab.h and
// fs_speculate.h for Python: tensors are checked and become device pointers, sizes
// and strides, results are allocated, and the C ABI is called.  No part of an
// operator is computed here.
//
// These calls take a few microseconds on the GPU at decode sizes.  Checked and
// allocated from Python, one cost 10 to 27 us of host time (a torch.empty there
// is 1.6 us, a call has up to six); here it is 5 to 14.
//
// bind() receives the addresses of the C entry points and the exception class;
// every function takes its arguments by position (the keyword interface is the
// Python side's) and raises that exception for refused arguments and for any
// status but FS_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <exception>
#include <string>

#include "fs_speculate.h"
#include "fs_vocab.h"

namespace {

struct Entries {
  decltype(&fs_logprobs) logprobs;
  decltype(&fs_logprobs_workspace_size) logprobs_size;
  decltype(&fs_logprobs_grad) grad;
  decltype(&fs_logprobs_grad_workspace_size) grad_size;
  decltype(&fs_embed) embed;
  decltype(&fs_embed_grad) embed_grad;
  decltype(&fs_embed_grad_workspace_size) embed_grad_size;
  decltype(&fs_quantize) quantize;
  decltype(&fs_matmul_fp8) matmul_fp8;
  decltype(&fs_probs) probs;
  decltype(&fs_verify) verify;
} g;
PyObject* g_error = nullptr;

// Thrown to leave a function with the Python error already set, or with a status
// to raise.
struct PythonError {};
struct Refused {
  int status;
  std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused{FS_ERR_INVALID_ARG, what}; }

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kLong: return "int64";
    case at::kFloat8_e4m3fn: return "float8_e4m3fn";
    default: return "int32";
  }
}

// Address of a contiguous vector of n elements.
void* vector(const char* name, PyObject* o, at::ScalarType type, int64_t n, c10::Device dev) {
  const at::Tensor& t = tensor(name, o);
  if (t.scalar_type() != type || t.device() != dev || t.dim() != 1 || t.size(0) != n ||
      !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + type_name(type) + " vector of " +
           std::to_string(n) + " on " + dev.str());
  return t.data_ptr();
}
void* vector_or_none(const char* name, PyObject* o, at::ScalarType type, int64_t n,
                     c10::Device dev) {
  return o == Py_None ? nullptr : vector(name, o, type, n, dev);
}

struct Matrix {
  void* data;
  int64_t ld;
};
// Address and row stride of an [n, d] matrix (of a single row: a stride that
// every check accepts).
Matrix matrix(const char* name, const at::Tensor& t, at::ScalarType type, int64_t n, int64_t d,
              c10::Device dev) {
  if (t.scalar_type() != type || t.device() != dev || t.dim() != 2 || t.size(0) != n ||
      t.size(1) != d || (t.stride(1) != 1 && d > 1))
    refuse(std::string(name) + " must be a " + type_name(type) + " matrix [" + std::to_string(n) +
           ", " + std::to_string(d) + "] with unit column stride on " + dev.str());
  return {t.data_ptr(), n > 1 ? t.stride(0) : std::max(t.stride(0), (d + 7) / 8 * 8)};
}

// A new tensor from torch's caching allocator, in the order of the call's stream (On).
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
  return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
}

// Makes a call's device and stream current while it is alive: the stream of a handle,
// or the device's current one for None.  What is allocated meanwhile belongs to that
// stream, so its memory has no other stream's work pending, and a workspace may be
// freed while the kernels still run.
class On {
 public:
  On(PyObject* stream, c10::Device dev) : device_(dev) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(dev.index());
    handle_ = current.stream();
    if (stream == Py_None) return;
    handle_ = reinterpret_cast<cudaStream_t>(static_cast<intptr_t>(integer(stream)));
    if (handle_ == current.stream()) return;
    // 0 and cudaStreamLegacy are the same stream, torch's default one.
    stream_.reset_stream(handle_ == nullptr || handle_ == cudaStreamLegacy
                             ? c10::cuda::getDefaultCUDAStream(dev.index())
                             : c10::cuda::getStreamFromExternal(handle_, dev.index()));
  }
  void* handle() const { return handle_; }

 private:
  c10::cuda::OptionalCUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard stream_;
  cudaStream_t handle_;
};

void check(const char* name, int status) {
  if (status != FS_OK) throw Refused{status, name};
}

// H [B, d] and W [V, d].
struct Head {
  int64_t B, d, V;
  c10::Device dev;
  Matrix h, w;
};
Head head(PyObject* ho, PyObject* wo) {
  const at::Tensor &H = tensor("H", ho), &W = tensor("W", wo);
  if (H.dim() != 2 || W.dim() != 2 || !H.is_cuda())
    refuse("H and W must be CUDA bfloat16 matrices");
  const int64_t B = H.size(0), d = H.size(1), V = W.size(0);
  const c10::Device dev = H.device();
  return {B, d, V, dev, matrix("H", H, at::kBFloat16, B, d, dev),
          matrix("W", W, at::kBFloat16, V, d, dev)};
}

struct Mask {
  void* data = nullptr;
  int64_t ld = 0;
};
Mask mask_of(PyObject* o, int64_t rows, int64_t V, c10::Device dev) {
  if (o == Py_None) return {};
  const at::Tensor& t = tensor("vocab_mask", o);
  if (t.scalar_type() != at::kInt || t.device() != dev || t.dim() != 2 || t.size(0) != rows ||
      t.size(1) < (V + 31) / 32 || t.stride(1) != 1)
    refuse("vocab_mask must be an int32 matrix [B, >= ceil(V/32)] on " + dev.str());
  // A stride below the row's words (0 for one mask expanded to all rows) is the
  // library's to refuse; a single row's is never used.
  return {t.data_ptr(), rows > 1 ? t.stride(0) : t.size(1)};
}
Mask mask_of(PyObject* o, const Head& s) { return mask_of(o, s.B, s.V, s.dev); }

struct Workspace {
  at::Tensor made;  // freed after the call: reused in the order of its stream (On)
  void* data = nullptr;
  size_t bytes = 0;
};
Workspace workspace_of(PyObject* o, size_t need, c10::Device dev) {
  Workspace w;
  if (o == Py_None) {
    if (need == 0) return w;
    w.made = empty({int64_t(need)}, at::kByte, dev);
    w.data = w.made.data_ptr();
    w.bytes = need;
    return w;
  }
  const at::Tensor& t = tensor("workspace", o);
  if (t.device() != dev || !t.is_contiguous())
    throw Refused{FS_ERR_WORKSPACE, "workspace must be a contiguous tensor on " + dev.str()};
  w.data = t.data_ptr();
  w.bytes = size_t(t.numel()) * t.element_size();
  return w;
}

// A result: the given tensor (checked by the caller), or a new one.
struct Result {
  PyObject* given;
  at::Tensor made;
  PyObject* wrap() const {
    if (given == nullptr) Py_RETURN_NONE;
    if (given != Py_None) {
      Py_INCREF(given);
      return given;
    }
    return THPVariable_Wrap(made);
  }
};
void* row_result(const char* name, Result& r, int64_t n, c10::Device dev) {
  if (r.given != Py_None) return vector(name, r.given, at::kFloat, n, dev);
  r.made = empty({n}, at::kFloat, dev);
  return r.made.data_ptr();
}
void* table_result(const char* name, Result& r, at::ScalarType type, int64_t n, int64_t k,
                   c10::Device dev) {
  if (r.given != Py_None) {
    const at::Tensor& t = tensor(name, r.given);
    const Matrix m = matrix(name, t, type, n, k, dev);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return m.data;
  }
  r.made = empty({n, k}, type, dev);
  return r.made.data_ptr();
}

PyObject* tuple_of(std::initializer_list<const Result*> results) {
  PyObject* t = PyTuple_New(Py_ssize_t(results.size()));
  if (t == nullptr) throw PythonError{};
  Py_ssize_t i = 0;
  for (const Result* r : results) {
    PyObject* o = r->wrap();
    if (o == nullptr) {
      Py_DECREF(t);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// Runs a call; nothing is thrown past it.
template <class Call>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, Call call) {
  if (g_error == nullptr || nargs != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or bind() not called");
    return nullptr;
  }
  try {
    return call();
  } catch (const PythonError&) {
  } catch (const Refused& r) {
    PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.what.c_str());
    if (e != nullptr) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// (H, W, tokens, K, temperature, vocab_mask, vocab_offset, out_logp, out_entropy,
//  out_lse, out_topk_idx, out_topk_logp, workspace, stream, flags)
// -> (logp, entropy, lse, topk_idx, topk_logp)
PyObject* py_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const Head s = head(a[0], a[1]);
    const int64_t K = integer(a[3]);
    if (K < 0 || K > FS_LOGPROBS_TOPK_MAX)
      refuse("K must be 0 to " + std::to_string(FS_LOGPROBS_TOPK_MAX));
    const Mask m = mask_of(a[5], s);
    const On on(a[13], s.dev);
    Result logp{a[2] == Py_None ? nullptr : a[7], {}}, entropy{a[8], {}}, lse{a[9], {}};
    Result idx{K > 0 ? a[10] : nullptr, {}}, top{K > 0 ? a[11] : nullptr, {}};
    fs_logprobs_args p = {};
    p.H = s.h.data;
    p.W = s.w.data;
    p.temperature =
        static_cast<const float*>(vector_or_none("temperature", a[4], at::kFloat, s.B, s.dev));
    p.vocab_mask = static_cast<const uint32_t*>(m.data);
    p.mask_ld = m.ld;
    p.tokens = static_cast<const int64_t*>(vector_or_none("tokens", a[2], at::kLong, s.B, s.dev));
    p.B = s.B;
    p.d = s.d;
    p.V = s.V;
    p.ldh = s.h.ld;
    p.ldw = s.w.ld;
    p.vocab_offset = integer(a[6]);
    p.K = K;
    if (logp.given) p.out_logp = static_cast<float*>(row_result("out_logp", logp, s.B, s.dev));
    p.out_entropy = static_cast<float*>(row_result("out_entropy", entropy, s.B, s.dev));
    p.out_lse = static_cast<float*>(row_result("out_lse", lse, s.B, s.dev));
    if (K > 0) {
      p.out_topk_idx =
          static_cast<int64_t*>(table_result("out_topk_idx", idx, at::kLong, s.B, K, s.dev));
      p.out_topk_logp =
          static_cast<float*>(table_result("out_topk_logp", top, at::kFloat, s.B, K, s.dev));
    }
    const Workspace ws = workspace_of(a[12], g.logprobs_size(s.B, s.V, K), s.dev);
    p.workspace = ws.data;
    p.workspace_bytes = ws.bytes;
    p.flags = uint32_t(integer(a[14]));
    check("fs_logprobs", g.logprobs(&p, on.handle()));
    return tuple_of({&logp, &entropy, &lse, &idx, &top});
  });
}

// A bf16 [n, d] gradient, made here with rows on 16-byte boundaries when None.
Matrix gradient(const char* name, Result& r, int64_t n, int64_t d, c10::Device dev) {
  if (r.given != Py_None) return matrix(name, tensor(name, r.given), at::kBFloat16, n, d, dev);
  const int64_t ld = (d + 7) / 8 * 8;
  r.made = empty({n, ld}, at::kBFloat16, dev);
  const Matrix m{r.made.data_ptr(), ld};
  if (ld != d) r.made = r.made.narrow(1, 0, d);
  return m;
}

// (H, W, tokens, lse, grad_logp, entropy, grad_entropy, temperature, vocab_mask,
//  vocab_offset, out_dH, out_dW, need_dH, need_dW, workspace, stream) -> (dH, dW)
PyObject* py_logprobs_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const Head s = head(a[0], a[1]);
    const bool need_dH = truth(a[12]), need_dW = truth(a[13]);
    if (!need_dH && !need_dW) refuse("neither dH nor dW is asked for");
    if (a[6] != Py_None && a[5] == Py_None) refuse("grad_entropy needs entropy");
    const Mask m = mask_of(a[8], s);
    const On on(a[15], s.dev);
    Result dH{need_dH ? a[10] : nullptr, {}}, dW{need_dW ? a[11] : nullptr, {}};
    fs_logprobs_grad_args p = {};
    p.H = s.h.data;
    p.W = s.w.data;
    p.temperature =
        static_cast<const float*>(vector_or_none("temperature", a[7], at::kFloat, s.B, s.dev));
    p.vocab_mask = static_cast<const uint32_t*>(m.data);
    p.mask_ld = m.ld;
    p.tokens = static_cast<const int64_t*>(vector("tokens", a[2], at::kLong, s.B, s.dev));
    p.lse = static_cast<const float*>(vector("lse", a[3], at::kFloat, s.B, s.dev));
    p.grad_logp = static_cast<const float*>(vector("grad_logp", a[4], at::kFloat, s.B, s.dev));
    if (a[6] != Py_None) {
      p.entropy = static_cast<const float*>(vector("entropy", a[5], at::kFloat, s.B, s.dev));
      p.grad_entropy =
          static_cast<const float*>(vector("grad_entropy", a[6], at::kFloat, s.B, s.dev));
    }
    p.B = s.B;
    p.d = s.d;
    p.V = s.V;
    p.ldh = s.h.ld;
    p.ldw = s.w.ld;
    p.vocab_offset = integer(a[9]);
    if (need_dH) {
      const Matrix r = gradient("out_dH", dH, s.B, s.d, s.dev);
      p.out_dH = r.data;
      p.lddh = r.ld;
    }
    if (need_dW) {
      const Matrix r = gradient("out_dW", dW, s.V, s.d, s.dev);
      p.out_dW = r.data;
      p.lddw = r.ld;
    }
    const Workspace ws = workspace_of(a[14], g.grad_size(s.B, s.d, s.V), s.dev);
    p.workspace = ws.data;
    p.workspace_bytes = ws.bytes;
    check("fs_logprobs_grad", g.grad(&p, on.handle()));
    return tuple_of({&dH, &dW});
  });
}

// FS_BF16 / FS_F32 of a table's type.
int element_code(const char* name, const at::Tensor& t) {
  const at::ScalarType s = t.scalar_type();
  if ((s != at::kBFloat16 && s != at::kFloat) || t.dim() != 2 || !t.is_cuda())
    refuse(std::string(name) + " must be a CUDA bfloat16 or float32 matrix");
  return s == at::kFloat ? FS_F32 : FS_BF16;
}

// (ids, E, scale, vocab_offset, out, stream) -> out
PyObject* py_embed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor& E = tensor("E", a[1]);
    const int code = element_code("E", E);
    const c10::Device dev = E.device();
    const int64_t V = E.size(0), d = E.size(1);
    const at::Tensor& ids = tensor("ids", a[0]);
    const int64_t N = ids.dim() == 1 ? ids.size(0) : -1;
    const auto* id = static_cast<const int64_t*>(vector("ids", a[0], at::kLong, N, dev));
    const Matrix e = matrix("E", E, E.scalar_type(), V, d, dev);
    const On on(a[5], dev);
    Result out{a[4], {}};
    Matrix o{nullptr, d};
    if (a[4] == Py_None) {
      out.made = empty({N, d}, E.scalar_type(), dev);
      o.data = out.made.data_ptr();
    } else {
      o = matrix("out", tensor("out", a[4]), E.scalar_type(), N, d, dev);
    }
    check("fs_embed", g.embed(id, N, e.data, V, d, e.ld, code, float(real(a[2])), integer(a[3]),
                              o.data, o.ld, on.handle()));
    return out.wrap();
  });
}

// (ids, dY, V, scale, vocab_offset, out, accumulate, make_fp32, workspace, stream)
// -> out; make_fp32: the type of a result made here (else dY's).
PyObject* py_embed_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor& dY = tensor("dY", a[1]);
    const int y_code = element_code("dY", dY);
    const c10::Device dev = dY.device();
    const int64_t N = dY.size(0), d = dY.size(1), V = integer(a[2]);
    const bool accumulate = truth(a[6]);
    const Matrix y = matrix("dY", dY, dY.scalar_type(), N, d, dev);
    const auto* id = static_cast<const int64_t*>(vector("ids", a[0], at::kLong, N, dev));
    const On on(a[9], dev);
    Result out{a[5], {}};
    if (a[5] == Py_None) {
      if (accumulate) refuse("accumulate needs out");
      if (V < 1) refuse("V must be positive");
      out.made = empty({V, d}, truth(a[7]) ? at::kFloat : dY.scalar_type(), dev);
    }
    const at::Tensor& dE = a[5] == Py_None ? out.made : tensor("out", a[5]);
    const int e_code = element_code("out", dE);
    const Matrix e = matrix("out", dE, dE.scalar_type(), V, d, dev);
    const Workspace ws = workspace_of(a[8], g.embed_grad_size(N, d), dev);
    check("fs_embed_grad",
          g.embed_grad(id, N, y.data, V, d, y.ld, y_code, float(real(a[3])), integer(a[4]), e.data,
                       e.ld, e_code, accumulate ? 1 : 0, ws.data, ws.bytes,
                       on.handle()));
    return out.wrap();
  });
}

// ---- fs_speculate.h ---------------------------------------------------------
at::ScalarType type_of(int code) { return code == FS_F32 ? at::kFloat : at::kBFloat16; }

// A result [n, d], given or made here with rows on 16-byte boundaries.
Matrix rows_result(const char* name, Result& r, at::ScalarType type, int64_t n, int64_t d,
                   c10::Device dev) {
  if (r.given != Py_None) return matrix(name, tensor(name, r.given), type, n, d, dev);
  const int64_t unit = type == at::kFloat8_e4m3fn ? 16 : 8;
  const int64_t ld = (d + unit - 1) / unit * unit;
  r.made = empty({n, ld}, type, dev);
  const Matrix m{r.made.data_ptr(), ld};
  if (ld != d) r.made = r.made.narrow(1, 0, d);
  return m;
}
// The element type of a result: the given tensor's, else the one asked for.
int result_code(const char* name, PyObject* given, PyObject* code) {
  return given == Py_None ? int(integer(code)) : element_code(name, tensor(name, given));
}

// (x, block_rows, out, out_scale, stream) -> (values, scale)
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor& x = tensor("x", a[0]);
    const int code = element_code("x", x);
    const c10::Device dev = x.device();
    const int64_t N = x.size(0), d = x.size(1), block = integer(a[1]);
    if (block != 1 && block != FS_FP8_BLOCK)
      refuse("block_rows must be 1 or " + std::to_string(FS_FP8_BLOCK));
    const Matrix m = matrix("x", x, x.scalar_type(), N, d, dev);
    const On on(a[4], dev);
    Result values{a[2], {}}, scale{a[3], {}};
    const Matrix v = rows_result("out", values, at::kFloat8_e4m3fn, N, d, dev);
    const int64_t rows = (N + block - 1) / block, cols = (d + FS_FP8_BLOCK - 1) / FS_FP8_BLOCK;
    Matrix s{nullptr, cols};
    if (a[3] == Py_None) {
      scale.made = empty({rows, cols}, at::kFloat, dev);
      s.data = scale.made.data_ptr();
    } else {
      s = matrix("out_scale", tensor("out_scale", a[3]), at::kFloat, rows, cols, dev);
    }
    check("fs_quantize", g.quantize(m.data, N, d, m.ld, code, int(block), v.data, v.ld,
                                    static_cast<float*>(s.data), s.ld, on.handle()));
    return tuple_of({&values, &scale});
  });
}

// (A, a_scale, W, w_scale, out, out_code, stream, flags) -> out
PyObject* py_matmul_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor &A = tensor("A", a[0]), &W = tensor("W", a[2]);
    if (A.dim() != 2 || W.dim() != 2 || !A.is_cuda())
      refuse("A and W must be CUDA float8_e4m3fn matrices");
    const c10::Device dev = A.device();
    fs_matmul_fp8_args p = {};
    p.M = A.size(0);
    p.d = A.size(1);
    p.V = W.size(0);
    const int64_t kb = (p.d + FS_FP8_BLOCK - 1) / FS_FP8_BLOCK;
    const Matrix m = matrix("A", A, at::kFloat8_e4m3fn, p.M, p.d, dev);
    const Matrix w = matrix("W", W, at::kFloat8_e4m3fn, p.V, p.d, dev);
    const Matrix as =
        matrix("a_scale", tensor("a_scale", a[1]), at::kFloat, p.M, kb, dev);
    const Matrix ws = matrix("w_scale", tensor("w_scale", a[3]), at::kFloat,
                             (p.V + FS_FP8_BLOCK - 1) / FS_FP8_BLOCK, kb, dev);
    const On on(a[6], dev);
    Result out{a[4], {}};
    p.out_dtype = result_code("out", a[4], a[5]);
    const Matrix o = rows_result("out", out, type_of(p.out_dtype), p.M, p.V, dev);
    p.A = m.data;
    p.lda = m.ld;
    p.a_scale = static_cast<const float*>(as.data);
    p.lda_scale = as.ld;
    p.W = w.data;
    p.ldw = w.ld;
    p.w_scale = static_cast<const float*>(ws.data);
    p.ldw_scale = ws.ld;
    p.out = o.data;
    p.ldo = o.ld;
    p.flags = uint32_t(integer(a[7]));
    check("fs_matmul_fp8", g.matmul_fp8(&p, on.handle()));
    return out.wrap();
  });
}

// (logits, temperature, vocab_mask, out, out_code, stream) -> out
PyObject* py_probs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor& x = tensor("logits", a[0]);
    fs_probs_args p = {};
    p.dtype = element_code("logits", x);
    const c10::Device dev = x.device();
    p.N = x.size(0);
    p.V = x.size(1);
    const Matrix m = matrix("logits", x, x.scalar_type(), p.N, p.V, dev);
    p.temperature =
        static_cast<const float*>(vector_or_none("temperature", a[1], at::kFloat, p.N, dev));
    const Mask mask = mask_of(a[2], p.N, p.V, dev);
    const On on(a[5], dev);
    Result out{a[3], {}};
    p.out_dtype = result_code("out", a[3], a[4]);
    const Matrix o = rows_result("out", out, type_of(p.out_dtype), p.N, p.V, dev);
    p.logits = m.data;
    p.ldl = m.ld;
    p.vocab_mask = static_cast<const uint32_t*>(mask.data);
    p.mask_ld = mask.ld;
    p.out = o.data;
    p.ldo = o.ld;
    check("fs_probs", g.probs(&p, on.handle()));
    return out.wrap();
  });
}

// A [B, n, V] tensor of `type` with unit stride along V.
const at::Tensor& positions(const char* name, PyObject* o, at::ScalarType type, int64_t B,
                            int64_t n, int64_t V, c10::Device dev) {
  const at::Tensor& t = tensor(name, o);
  if (t.scalar_type() != type || t.device() != dev || t.dim() != 3 || t.size(0) != B ||
      t.size(1) != n || t.size(2) != V || (t.stride(2) != 1 && V > 1))
    refuse(std::string(name) + " must be a " + type_name(type) + " tensor [" + std::to_string(B) +
           ", " + std::to_string(n) + ", " + std::to_string(V) + "] with unit stride along V on " +
           dev.str());
  return t;
}

// (p, draft_ids, u, q, out_ids, out_accepted, stream) -> (ids, accepted)
PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor& t = tensor("p", a[0]);
    if (t.dim() != 3 || !t.is_cuda() || t.size(1) < 1 ||
        (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat))
      refuse("p must be a CUDA bfloat16 or float32 tensor [B, K + 1, V]");
    const c10::Device dev = t.device();
    fs_verify_args p = {};
    p.dtype = t.scalar_type() == at::kFloat ? FS_F32 : FS_BF16;
    p.B = t.size(0);
    p.K = t.size(1) - 1;
    p.V = t.size(2);
    positions("p", a[0], t.scalar_type(), p.B, p.K + 1, p.V, dev);
    p.p = t.data_ptr();
    p.p_seq = t.stride(0);
    p.p_pos = t.stride(1);
    if (a[3] != Py_None && p.K > 0) {
      const at::Tensor& q = positions("q", a[3], t.scalar_type(), p.B, p.K, p.V, dev);
      p.q = q.data_ptr();
      p.q_seq = q.stride(0);
      p.q_pos = q.stride(1);
    }
    const Matrix ids = matrix("draft_ids", tensor("draft_ids", a[1]), at::kLong, p.B, p.K, dev);
    const Matrix u = matrix("u", tensor("u", a[2]), at::kFloat, p.B, p.K + 1, dev);
    const On on(a[6], dev);
    Result out{a[4], {}}, accepted{a[5], {}};
    Matrix o{nullptr, p.K + 1};
    if (a[4] == Py_None) {
      out.made = empty({p.B, p.K + 1}, at::kLong, dev);
      o.data = out.made.data_ptr();
    } else {
      o = matrix("out_ids", tensor("out_ids", a[4]), at::kLong, p.B, p.K + 1, dev);
    }
    if (a[5] == Py_None) {
      accepted.made = empty({p.B}, at::kLong, dev);
      p.out_accepted = accepted.made.data_ptr<int64_t>();
    } else {
      p.out_accepted = static_cast<int64_t*>(vector("out_accepted", a[5], at::kLong, p.B, dev));
    }
    p.draft_ids = static_cast<const int64_t*>(ids.data);
    p.ld_ids = ids.ld;
    p.u = static_cast<const float*>(u.data);
    p.ldu = u.ld;
    p.out_ids = static_cast<int64_t*>(o.data);
    p.ld_out = o.ld;
    check("fs_verify", g.verify(&p, on.handle()));
    return tuple_of({&out, &accepted});
  });
}

// bind(error class, address of each entry point in the order of Entries)
constexpr int kEntries = 11;
static_assert(sizeof(Entries) == kEntries * sizeof(void*), "one address each");
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kEntries + 1) {
    PyErr_Format(PyExc_TypeError, "bind takes the exception class and %d addresses", kEntries);
    return nullptr;
  }
  void* at[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return nullptr;
    }
  }
  std::memcpy(&g, at, sizeof(g));
  Py_INCREF(a[0]);
  Py_XDECREF(g_error);
  g_error = a[0];
  Py_RETURN_NONE;
}

template <PyObject* (*kFunction)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kFunction));
}

PyMethodDef g_methods[] = {
    {"bind", fast<py_bind>(), METH_FASTCALL, "Set the entry points and the exception class."},
    {"logprobs", fast<py_logprobs>(), METH_FASTCALL, "fs_logprobs"},
    {"logprobs_grad", fast<py_logprobs_grad>(), METH_FASTCALL, "fs_logprobs_grad"},
    {"embed", fast<py_embed>(), METH_FASTCALL, "fs_embed"},
    {"embed_grad", fast<py_embed_grad>(), METH_FASTCALL, "fs_embed_grad"},
    {"quantize", fast<py_quantize>(), METH_FASTCALL, "fs_quantize"},
    {"matmul_fp8", fast<py_matmul_fp8>(), METH_FASTCALL, "fs_matmul_fp8"},
    {"probs", fast<py_probs>(), METH_FASTCALL, "fs_probs"},
    {"verify", fast<py_verify>(), METH_FASTCALL, "fs_verify"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", FS_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
