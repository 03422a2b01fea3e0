// Python side of the operators around the grouped GEMM: argument checks and the call of the C
// entry point, without the interpreter in between.  A call costs the host about as much as the
// launch itself (decode-sized operators run for 2 to 5 us on the GPU).  The entry points' addresses come
// from the library the package loaded, so any build of it can be called.
//
// Every buffer is a CUDA tensor, a raw device address (int, unchecked) or None.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "bsfp8.h"

namespace {

decltype(&bsmx_quantize) f_quantize = nullptr;
decltype(&bsmx_rmsnorm_quant) f_rmsnorm_quant = nullptr;
decltype(&bsmx_swiglu_quant) f_swiglu_quant = nullptr;
decltype(&bsmx_moe_sort) f_moe_sort = nullptr;
decltype(&bsmx_moe_combine) f_moe_combine = nullptr;
decltype(&bsmx_moe_combine_backward) f_moe_combine_backward = nullptr;

// A set of scalar types, as bits.
constexpr uint64_t of(at::ScalarType t) {
  return static_cast<unsigned>(t) < 64 ? uint64_t{1} << static_cast<unsigned>(t) : 0;
}
constexpr uint64_t kBf16 = of(at::kBFloat16), kFp32 = of(at::kFloat), kInt32 = of(at::kInt);
constexpr uint64_t kAnyInput = kBf16 | kFp32 | of(at::kHalf);

// Reads the arguments of one call in order; the first failure sets a Python error, after which
// everything returns zeros.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t have, Py_ssize_t want) : next_(args) {
    if (have != want) fail("expected %zd arguments, got %zd", want, have);
  }
  bool ok() const { return !failed_; }

  int64_t integer() {
    PyObject* o = take();
    if (!o) return 0;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) failed_ = true;
    return v;
  }
  int int32() {
    const int64_t v = integer();
    if (ok() && (v > INT32_MAX || v < INT32_MIN)) fail("%lld does not fit 32 bits", (long long)v);
    return static_cast<int>(v);
  }
  float number() {
    PyObject* o = take();
    if (!o) return 0.0f;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) failed_ = true;
    return static_cast<float>(v);
  }

  // A buffer: its tensor is looked at by check() below once the sizes are known.
  struct Buffer {
    void* address = nullptr;
    const at::Tensor* tensor = nullptr;
  };
  Buffer buffer(const char* name) {
    Buffer b;
    PyObject* o = take();
    if (!o || o == Py_None) return b;
    if (PyLong_Check(o)) {
      b.address = PyLong_AsVoidPtr(o);
      if (!b.address && PyErr_Occurred()) failed_ = true;
    } else if (THPVariable_Check(o)) {
      b.tensor = &THPVariable_Unpack(o);
    } else {
      fail("%s must be a tensor, a device address or None", name);
    }
    return b;
  }

  // `types`: the scalar types allowed, 0 for any of `bytes` bytes.
  void check(Buffer& b, const char* name, int64_t count, uint64_t types, size_t bytes = 0) {
    if (!ok() || !b.tensor) return;
    const at::Tensor& t = *b.tensor;
    if (types ? !(types & of(t.scalar_type())) : t.element_size() != (int64_t)bytes)
      return fail("%s has an unsupported type%s", name,
                  types == kBf16 ? ": it must be bf16" : "");
    if (!t.is_cuda()) return fail("%s must be a CUDA tensor (device memory)", name);
    if (t.get_device() != device())
      return fail("%s is on GPU %d, not on the current device (%d)", name, (int)t.get_device(),
                  device());
    if (!t.is_contiguous()) return fail("%s must be contiguous (row-major)", name);
    if (t.numel() < count)
      return fail("%s holds %lld elements, needs %lld", name, (long long)t.numel(),
                  (long long)count);
    b.address = t.data_ptr();
  }

  // bsmx_type of an input: as given (>= 0), or its tensor's.
  int type_of(const Buffer& b, const char* name, int given, uint64_t allowed) {
    if (!ok()) return 0;
    int code = given;
    if (code < 0 && !b.tensor) {
      if (b.address) fail("%s is a raw address: its type has to be given", name);
      return 0;
    }
    if (code < 0) {
      const at::ScalarType t = b.tensor->scalar_type();
      code = t == at::kBFloat16 ? BSMX_BF16 : t == at::kHalf ? BSMX_FP16 : BSMX_FP32;
      if (!(allowed & of(t))) fail("%s has an unsupported type", name);
    }
    return code;
  }

  // The stream's argument, which resolve() turns into a stream once everything else holds.
  void stream() { stream_ = take(); }
  cudaStream_t resolve() {
    if (stream_ == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* const own =
        PyLong_Check(stream_) ? nullptr : PyObject_GetAttrString(stream_, "cuda_stream");
    void* const p = PyLong_Check(stream_) ? PyLong_AsVoidPtr(stream_)
                    : own                 ? PyLong_AsVoidPtr(own)
                                          : nullptr;
    Py_XDECREF(own);
    if (PyErr_Occurred()) failed_ = true;
    return static_cast<cudaStream_t>(p);
  }

  template <typename... T>
  void fail(const char* format, T... args) {
    if (!failed_) PyErr_Format(PyExc_ValueError, format, args...);
    failed_ = true;
  }

 private:
  // The current device, which the call runs on; -1 where there is none.
  int device() {
    c10::DeviceIndex d = -1;
    if (device_ == kUnasked) device_ = c10::cuda::GetDevice(&d) == cudaSuccess ? d : -1;
    return device_;
  }
  PyObject* take() { return failed_ ? nullptr : *next_++; }

  PyObject* const* next_;
  PyObject* stream_ = Py_None;
  static constexpr int kUnasked = -2;
  int device_ = kUnasked;
  bool failed_ = false;
};

using Buffer = Args::Buffer;

// Codes and scales of an operand of rows x K in `format`.
void check_operand(Args& a, int format, Buffer& q, Buffer& scales, int64_t rows, int64_t K) {
  const bool fp4 = format == BSMX_MXFP4 || format == BSMX_NVFP4;
  a.check(q, "q", rows * (fp4 ? K / 2 : K), 0, 1);
  if (format == BSMX_BLOCKWISE)
    a.check(scales, "scales", rows * (K / 128), kFp32);
  else
    a.check(scales, "scales", rows * (K / (format == BSMX_NVFP4 ? 16 : 32)), 0, 1);
}

// Gives the interpreter lock away while it lives: a launch may wait for room in the stream's
// queue, which a host callback that wants the lock may have to make.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* const state_;
};

template <typename F>
PyObject* status(Args& a, F&& call) {
  if (!a.ok()) return nullptr;
  const cudaStream_t stream = a.resolve();
  if (!a.ok()) return nullptr;
  bsfp8_status st;
  {
    Unlocked unlocked;
    st = call(stream);
  }
  return PyLong_FromLong(st);
}

// quantize(format, x_type, x, row_of_slot, top_k, q, scales, rows, out_rows, K, stream)
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 11);
  const int format = a.int32();
  int type = a.int32();
  Buffer x = a.buffer("x"), map = a.buffer("row_of_slot");
  const int top_k = a.int32();
  Buffer q = a.buffer("q"), scales = a.buffer("scales");
  const int64_t rows = a.integer(), out_rows = a.integer();
  const int K = a.int32();
  a.stream();
  type = a.type_of(x, "x", type, kAnyInput);
  a.check(x, "x", rows * K, type == BSMX_BF16 ? kBf16 : type == BSMX_FP16 ? of(at::kHalf) : kFp32);
  a.check(map, "row_of_slot", rows * top_k, kInt32);
  check_operand(a, format, q, scales, out_rows, K);
  return status(a, [&](cudaStream_t stream) {
    return f_quantize(format, type, x.address, static_cast<const int32_t*>(map.address), top_k,
                      q.address, scales.address, rows, out_rows, K, stream);
  });
}

// rmsnorm_quant(format, residual_type, x, residual, weight, eps, residual_out, y, q, scales,
//               rows, K, stream)
PyObject* rmsnorm_quant(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 13);
  const int format = a.int32();
  int type = a.int32();
  Buffer x = a.buffer("x"), residual = a.buffer("residual"), weight = a.buffer("weight");
  const float eps = a.number();
  Buffer out = a.buffer("residual_out"), y = a.buffer("y"), q = a.buffer("q"),
         scales = a.buffer("scales");
  const int64_t rows = a.integer();
  const int K = a.int32();
  a.stream();
  const bool in = residual.tensor || residual.address;
  type = a.type_of(in ? residual : out, in ? "residual" : "residual_out", type, kBf16 | kFp32);
  const uint64_t res = type == BSMX_FP32 ? kFp32 : kBf16;
  a.check(x, "x", rows * K, kBf16);
  a.check(residual, "residual", rows * K, res);
  a.check(weight, "weight", K, kBf16);
  a.check(out, "residual_out", rows * K, res);
  a.check(y, "y", rows * K, kBf16);
  if (q.tensor || q.address) check_operand(a, format, q, scales, rows, K);
  return status(a, [&](cudaStream_t stream) {
    return f_rmsnorm_quant(format, type, x.address, residual.address, weight.address, eps,
                           out.address, y.address, q.address, scales.address, rows, K, stream);
  });
}

// swiglu_quant(format, h, q, scales, rows, N, stream)
PyObject* swiglu_quant(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 7);
  const int format = a.int32();
  Buffer h = a.buffer("h"), q = a.buffer("q"), scales = a.buffer("scales");
  const int64_t rows = a.integer();
  const int N = a.int32();
  a.stream();
  a.check(h, "h", rows * 2 * N, kBf16);
  check_operand(a, format, q, scales, rows, N);
  return status(a, [&](cudaStream_t stream) {
    return f_swiglu_quant(format, h.address, q.address, scales.address, rows, N, stream);
  });
}

// moe_sort(topk_ids, offsets, row_of_slot, slot_of_row, workspace, workspace_bytes, rows, top_k,
//          num_experts, stream); workspace_bytes < 0: those of the tensor
PyObject* moe_sort(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 10);
  Buffer ids = a.buffer("topk_ids"), offsets = a.buffer("offsets"),
         row = a.buffer("row_of_slot"), slot = a.buffer("slot_of_row"),
         workspace = a.buffer("workspace");
  int64_t bytes = a.integer();
  const int64_t rows = a.integer();
  const int top_k = a.int32(), experts = a.int32();
  a.stream();
  const int64_t slots = rows * top_k;
  a.check(ids, "topk_ids", slots, kInt32);
  a.check(offsets, "offsets", (int64_t)experts + 2, kInt32);
  a.check(row, "row_of_slot", slots, kInt32);
  a.check(slot, "slot_of_row", slots, kInt32);
  if (a.ok() && workspace.tensor) {
    a.check(workspace, "workspace", 0, 0, workspace.tensor->element_size());
    if (bytes < 0) bytes = workspace.tensor->numel() * workspace.tensor->element_size();
  }
  if (bytes < 0 && workspace.address)
    a.fail("workspace is a raw address: workspace_bytes has to be given");
  if (bytes < 0) bytes = 0;
  return status(a, [&](cudaStream_t stream) {
    return f_moe_sort(static_cast<const int32_t*>(ids.address),
                      static_cast<int32_t*>(offsets.address), static_cast<int32_t*>(row.address),
                      static_cast<int32_t*>(slot.address), workspace.address, bytes, rows, top_k,
                      experts, stream);
  });
}

// moe_combine(C, row_of_slot, weights, residual, out, rows, in_rows, top_k, N, stream)
PyObject* moe_combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 10);
  Buffer C = a.buffer("C"), row = a.buffer("row_of_slot"), weights = a.buffer("weights"),
         residual = a.buffer("residual"), out = a.buffer("out");
  const int64_t rows = a.integer(), in_rows = a.integer();
  const int top_k = a.int32(), N = a.int32();
  a.stream();
  a.check(C, "C", in_rows * N, kBf16);
  a.check(row, "row_of_slot", rows * top_k, kInt32);
  a.check(weights, "weights", rows * top_k, kFp32);
  a.check(residual, "residual", rows * N, kBf16);
  a.check(out, "out", rows * N, kBf16);
  return status(a, [&](cudaStream_t stream) {
    return f_moe_combine(C.address, static_cast<const int32_t*>(row.address),
                         static_cast<const float*>(weights.address), residual.address,
                         out.address, rows, in_rows, top_k, N, stream);
  });
}

// moe_combine_backward(d_out, C, row_of_slot, weights, dC, d_weights, rows, in_rows, top_k, N,
//                      stream)
PyObject* moe_combine_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 11);
  Buffer d_out = a.buffer("d_out"), C = a.buffer("C"), row = a.buffer("row_of_slot"),
         weights = a.buffer("weights"), dC = a.buffer("dC"), d_weights = a.buffer("d_weights");
  const int64_t rows = a.integer(), in_rows = a.integer();
  const int top_k = a.int32(), N = a.int32();
  a.stream();
  a.check(d_out, "d_out", rows * N, kBf16);
  a.check(C, "C", in_rows * N, kBf16);
  a.check(row, "row_of_slot", rows * top_k, kInt32);
  a.check(weights, "weights", rows * top_k, kFp32);
  a.check(dC, "dC", in_rows * N, kBf16);
  a.check(d_weights, "d_weights", rows * top_k, kFp32);
  return status(a, [&](cudaStream_t stream) {
    return f_moe_combine_backward(
        d_out.address, C.address, static_cast<const int32_t*>(row.address),
        static_cast<const float*>(weights.address), dC.address,
        static_cast<float*>(d_weights.address), rows, in_rows, top_k, N, stream);
  });
}

// current_stream(): the raw stream torch launches on
PyObject* current_stream(PyObject*, PyObject*) {
  return PyLong_FromVoidPtr(c10::cuda::getCurrentCUDAStream().stream());
}

// bind(addresses): the entry points, in the order below
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 6);
  void* p[6];
  for (void*& q : p) q = reinterpret_cast<void*>(a.integer());
  if (!a.ok()) return nullptr;
  f_quantize = reinterpret_cast<decltype(f_quantize)>(p[0]);
  f_rmsnorm_quant = reinterpret_cast<decltype(f_rmsnorm_quant)>(p[1]);
  f_swiglu_quant = reinterpret_cast<decltype(f_swiglu_quant)>(p[2]);
  f_moe_sort = reinterpret_cast<decltype(f_moe_sort)>(p[3]);
  f_moe_combine = reinterpret_cast<decltype(f_moe_combine)>(p[4]);
  f_moe_combine_backward = reinterpret_cast<decltype(f_moe_combine_backward)>(p[5]);
  Py_RETURN_NONE;
}

// No C++ exception passes into the interpreter.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* guarded_stream(PyObject* self, PyObject* none) {
  try {
    return current_stream(self, none);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef fast(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<F>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {fast<quantize>("quantize"),
                         fast<rmsnorm_quant>("rmsnorm_quant"),
                         fast<swiglu_quant>("swiglu_quant"),
                         fast<moe_sort>("moe_sort"),
                         fast<moe_combine>("moe_combine"),
                         fast<moe_combine_backward>("moe_combine_backward"),
                         fast<bind>("bind"),
                         {"current_stream", guarded_stream, METH_NOARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "bsfp8_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_bsfp8_binding() { return PyModule_Create(&module); }
