// The Python binding of the calls that a decode step issues between its large
// kernels: tensors checked, outputs allocated and the C ABI called without a line
// of Python in between (a norm of one token runs in 2.1 us, and took 12 to issue
// through ctypes; 3.1 to 5.4 from here, by its outputs). Marshalling only, as in the ctypes calls; the
// computation is in libfp8blk, whose functions are handed over by setup().
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <array>
#include <mutex>
#include <string>

#include "fp8blk.h"

namespace {

struct Functions {
  decltype(&fp8blk_status_string) status_string;
  decltype(&fp8blk_fp4_quant) fp4_quant;
  decltype(&fp8blk_fp4_dequant) fp4_dequant;
  decltype(&fp8blk_fp4_gemm) fp4_gemm;
  decltype(&fp8blk_fp4_linear) fp4_linear;
  decltype(&fp8blk_fp4_linear_workspace_bytes) fp4_linear_workspace_bytes;
  decltype(&fp8blk_residual_norm) residual_norm;
} lib;

PyObject* error_class = nullptr;  // Fp8BlkError
PyObject* buffers = nullptr;      // the package's workspaces: {(device, stream, name): uint8 tensor}
PyObject* new_buffer = nullptr;   // its _buffer(bytes, device, key, zeroed)

struct Refusal {
  std::string what;
};

[[noreturn]] void refuse(std::string what) { throw Refusal{std::move(what)}; }

// Runs a call: what it refuses becomes Fp8BlkError, what torch throws a torch error.
template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refusal& r) {
    PyErr_SetString(error_class, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return t;
}

void check_type(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
}

void check_device(const at::Tensor& t, int dev) {
  if (t.get_device() != dev) refuse("all tensors must be on one device");
}

struct Matrix {
  const at::Tensor* t;
  int64_t rows, cols, stride;
};

// A matrix whose rows are contiguous (they may lie apart).
Matrix rows_of(PyObject* o, at::ScalarType type, int dev, const char* name) {
  const at::Tensor& t = tensor(o, name);
  check_type(t, type, name);
  if (t.dim() != 2) refuse(std::string(name) + " must be a matrix");
  if (t.stride(1) != 1 && t.size(1) > 1) refuse(std::string(name) + ": the columns of a row must be contiguous");
  if (dev >= 0) check_device(t, dev);
  return {&t, t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1)};
}

// A contiguous tensor of a given shape.
const at::Tensor& plain(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int dev, const char* name) {
  const at::Tensor& t = tensor(o, name);
  check_type(t, type, name);
  if (t.sizes() != shape)
    refuse(std::string(name) + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  if (!t.is_contiguous()) refuse(std::string(name) + ": Input tensor must be contiguous");
  check_device(t, dev);
  return t;
}

// A new tensor of the current device (Issue, below), with memory of its own: straight
// from the allocator, 0.3 us of the host where at::empty takes 0.7.
at::Tensor make(at::IntArrayRef shape, at::ScalarType type) {
  size_t bytes = c10::elementSize(type);
  for (int64_t d : shape) bytes *= static_cast<size_t>(d);
  c10::Allocator* from = c10::cuda::CUDACachingAllocator::get();
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes, from->allocate(bytes),
                                                         from, /*resizable=*/true)),
      c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// The given output, or none.
at::Tensor given_output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like,
                        const char* name) {
  return o != Py_None ? plain(o, type, shape, like.get_device(), name) : at::Tensor();
}

// While tensors are allocated and kernels launched, on the device of `like`: the
// interpreter's lock is not held (either may wait, for memory or for room in the
// launch queue).
struct Issue {
  PyThreadState* state;
  c10::cuda::OptionalCUDAGuard guard;
  explicit Issue(const at::Tensor& like) : state(PyEval_SaveThread()) {
    try {
      if (c10::cuda::current_device() != like.get_device()) guard.set_device(like.device());
    } catch (...) {
      PyEval_RestoreThread(state);
      throw;
    }
  }
  Issue(const Issue&) = delete;
  ~Issue() { PyEval_RestoreThread(state); }
};

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}

int format(PyObject* o) {
  const int64_t v = integer(o);
  if (v != FP8BLK_FP4_E4M3 && v != FP8BLK_FP4_UE8M0) refuse("fmt must be FP4_E4M3 or FP4_UE8M0");
  return static_cast<int>(v);
}

std::array<int64_t, 5> scale_shape(int64_t rows, int64_t K, int fmt) {
  return {(rows + 127) / 128, K / (fmt == FP8BLK_FP4_E4M3 ? 64 : 128), 32, 4, 4};
}

void check_columns(int64_t K) {
  if (K % 128) refuse("Last dimension size must be divisible by block_size (block_size=128)");
}

// A 4-bit matrix: codes, scale tiles and row scales.
struct Operand {
  const at::Tensor* q;
  int64_t rows, K;
  const void* s;
  const float* g;
};

Operand operand(PyObject* q, PyObject* s, PyObject* g, int fmt, int dev, const char* name) {
  const std::string n(name);
  const at::Tensor& tq = tensor(q, name);
  check_type(tq, at::kByte, name);
  if (tq.dim() != 2 || !tq.is_contiguous()) refuse(n + " must be a contiguous matrix");
  if (dev >= 0) check_device(tq, dev);
  Operand o{&tq, tq.size(0), 2 * tq.size(1), nullptr, nullptr};
  check_columns(o.K);
  const auto shape = scale_shape(o.rows, o.K, fmt);
  const at::Tensor& ts = tensor(s, (n + "_s").c_str());
  if (ts.scalar_type() != at::kByte || !ts.is_contiguous() || ts.numel() != shape[0] * shape[1] * 512)
    refuse(n + "_s must be a contiguous uint8 tensor of shape " + shape_text(shape));
  check_device(ts, tq.get_device());
  o.s = ts.const_data_ptr();
  if (fmt == FP8BLK_FP4_E4M3) {
    if (g == Py_None) refuse(n + "_g: FP4_E4M3 needs row scales");
    o.g = plain(g, at::kFloat, {o.rows}, tq.get_device(), (n + "_g").c_str()).const_data_ptr<float>();
  }
  return o;
}

const void* data(const at::Tensor& t) { return t.const_data_ptr(); }

// Makes a call on the current stream of the device of `like`.
template <typename F>
void call(const at::Tensor& like, const char* what, F f) {
  const int status = f(reinterpret_cast<fp8blk_stream_t>(c10::cuda::getCurrentCUDAStream(like.get_device()).stream()));
  if (status) refuse(std::string(what) + ": " + lib.status_string(status) + " (status " + std::to_string(status) + ")");
}

// A new reference to a tuple of tensors (undefined: None).
PyObject* tuple(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    if (t->defined()) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(*t));
    else Py_INCREF(Py_None), PyTuple_SET_ITEM(r, i++, Py_None);
  }
  return r;
}

void count(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse("wrong number of arguments");
}

// ---- the calls --------------------------------------------------------------------

// x, fmt
PyObject* fp4_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    count(n, 2);
    const bool fp32 = THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).scalar_type() == at::kFloat;
    const Matrix x = rows_of(a[0], fp32 ? at::kFloat : at::kBFloat16, -1, "x");
    const int fmt = format(a[1]);
    check_columns(x.cols);
    at::Tensor q, s, g;
    const std::array<int64_t, 2> qs = {x.rows, x.cols / 2};
    const auto ss = scale_shape(x.rows, x.cols, fmt);
    const std::array<int64_t, 1> gs = {x.rows};
    {
      const Issue issue(*x.t);
      q = make(qs, at::kByte), s = make(ss, at::kByte);
      if (fmt == FP8BLK_FP4_E4M3) g = make(gs, at::kFloat);
      call(*x.t, "fp4_quant", [&](fp8blk_stream_t st) {
        return lib.fp4_quant(data(*x.t), fp32, x.stride, x.rows, x.cols, fmt, q.mutable_data_ptr(), s.mutable_data_ptr(),
                             g.defined() ? g.mutable_data_ptr<float>() : nullptr, st);
      });
    }
    return tuple({&q, &s, &g});
  });
}

// q, s, g, fmt, out
PyObject* fp4_dequant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    count(n, 5);
    const int fmt = format(a[3]);
    const Operand q = operand(a[0], a[1], a[2], fmt, -1, "q");
    at::Tensor out = given_output(a[4], {q.rows, q.K}, at::kBFloat16, *q.q, "out");
    {
      const Issue issue(*q.q);
      if (!out.defined()) out = make({q.rows, q.K}, at::kBFloat16);
      call(*q.q, "fp4_dequant", [&](fp8blk_stream_t st) {
        return lib.fp4_dequant(data(*q.q), q.s, q.g, q.rows, q.K, fmt, out.mutable_data_ptr(), st);
      });
    }
    return THPVariable_Wrap(out);
  });
}

// a, a_s, a_g, w, w_s, w_g, fmt, out
PyObject* fp4_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    count(n, 8);
    const int fmt = format(a[6]);
    const Operand x = operand(a[0], a[1], a[2], fmt, -1, "a");
    const Operand w = operand(a[3], a[4], a[5], fmt, x.q->get_device(), "w");
    if (x.K != w.K) refuse("a and w must share K");
    at::Tensor out = given_output(a[7], {x.rows, w.rows}, at::kBFloat16, *x.q, "out");
    {
      const Issue issue(*x.q);
      if (!out.defined()) out = make({x.rows, w.rows}, at::kBFloat16);
      call(*x.q, "fp4_gemm", [&](fp8blk_stream_t st) {
        return lib.fp4_gemm(data(*x.q), x.s, x.g, data(*w.q), w.s, w.g, out.mutable_data_ptr(), x.rows, w.rows, x.K, fmt,
                            st);
      });
    }
    return THPVariable_Wrap(out);
  });
}

// Two threads may call fp4_linear on one stream, whose workspace then holds the one's
// activations after the other's: the launches of a call go out together.
std::mutex linear_launches;

bool capturing(cudaStream_t stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  return cudaStreamIsCapturing(stream, &status) != cudaSuccess || status != cudaStreamCaptureStatusNone;
}

// x, w, w_s, w_g, fmt, out, ws
PyObject* fp4_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    count(n, 7);
    const Matrix x = rows_of(a[0], at::kBFloat16, -1, "x");
    const int dev = x.t->get_device(), fmt = format(a[4]);
    const Operand w = operand(a[1], a[2], a[3], fmt, dev, "w");
    if (x.cols != w.K) refuse("x and w must share K");
    at::Tensor out = given_output(a[5], {x.rows, w.rows}, at::kBFloat16, *x.t, "out");
    // The caller's workspace, or the one that the package keeps for the device and stream.
    uintptr_t at;
    size_t room;
    at::Tensor held;
    if (a[6] != Py_None) {
      held = tensor(a[6], "ws");
      if (!held.is_contiguous() || held.get_device() != dev)
        refuse("ws must be a contiguous tensor on the device of the inputs");
      at = reinterpret_cast<uintptr_t>(held.mutable_data_ptr());
      room = held.nbytes();
    } else {
      room = lib.fp4_linear_workspace_bytes(x.rows, w.rows, x.cols, fmt);
      const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
      THPObjectPtr key(Py_BuildValue("(iKs)", dev, static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(stream)),
                                     "fp4_linear"));
      if (!key) throw python_error();
      PyObject* kept = PyDict_GetItem(buffers, key.get());
      if (kept && static_cast<size_t>(THPVariable_Unpack(kept).numel()) >= room + 256 && !capturing(stream)) {
        held = THPVariable_Unpack(kept);
      } else {
        THPObjectPtr device(PyObject_GetAttrString(a[0], "device"));
        THPObjectPtr made(device ? PyObject_CallFunction(new_buffer, "nOOi", static_cast<Py_ssize_t>(room), device.get(),
                                                         key.get(), 0)
                                 : nullptr);
        if (!made) throw python_error();
        held = THPVariable_Unpack(made.get());
      }
      at = (reinterpret_cast<uintptr_t>(held.mutable_data_ptr()) + 255) & ~uintptr_t{255};
    }
    {
      const Issue issue(*x.t);
      if (!out.defined()) out = make({x.rows, w.rows}, at::kBFloat16);
      const std::lock_guard<std::mutex> together(linear_launches);
      call(*x.t, "fp4_linear", [&](fp8blk_stream_t st) {
        return lib.fp4_linear(data(*x.t), x.stride, data(*w.q), w.s, w.g, out.mutable_data_ptr(), x.rows, w.rows, x.cols,
                              fmt, reinterpret_cast<void*>(at), room, st);
      });
    }
    return THPVariable_Wrap(out);
  });
}

// y, x, norm_w, post_w, gate, residual_scale, eps, quant, scale_fmt, r
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    count(n, 10);
    const Matrix y = rows_of(a[0], at::kBFloat16, -1, "y");
    const int64_t T = y.rows, D = y.cols;
    const int dev = y.t->get_device();
    auto same = [&](const Matrix& m, const char* what) {
      if (m.rows != T || m.cols != D) refuse(what);
    };
    const void *x = nullptr, *tok = nullptr;
    const float *post = nullptr, *col = nullptr;
    int64_t x_stride = D, tok_stride = D;
    if (a[1] != Py_None) {
      const Matrix m = rows_of(a[1], at::kBFloat16, dev, "x");
      same(m, "x and y must have one shape");
      x = data(*m.t), x_stride = m.stride;
    }
    const float* norm = plain(a[2], at::kFloat, {D}, dev, "norm_w").const_data_ptr<float>();
    if (a[3] != Py_None) post = plain(a[3], at::kFloat, {D}, dev, "post_w").const_data_ptr<float>();
    if (a[4] != Py_None) {
      if (tensor(a[4], "gate").dim() == 1) {
        col = plain(a[4], at::kFloat, {D}, dev, "gate").const_data_ptr<float>();
      } else {
        const Matrix m = rows_of(a[4], at::kBFloat16, dev, "gate");
        same(m, "gate must be float32 [D] or bf16 [T, D]");
        tok = data(*m.t), tok_stride = m.stride;
      }
    }
    const float residual_scale = number(a[5]), eps = number(a[6]);
    int kind = FP8BLK_NORM_BF16, fmt = static_cast<int>(integer(a[8]));
    if (a[7] != Py_None) {
      if (PyUnicode_Check(a[7]) && PyUnicode_CompareWithASCIIString(a[7], "fp8") == 0) kind = FP8BLK_NORM_E4M3;
      else if (PyUnicode_Check(a[7]) && PyUnicode_CompareWithASCIIString(a[7], "fp4") == 0) kind = FP8BLK_NORM_E2M1;
      else refuse("quant must be None, \"fp8\" or \"fp4\"");
      check_columns(D);
      if (kind == FP8BLK_NORM_E2M1) fmt = format(a[8]);
    }
    at::Tensor r, h, s, g;
    const std::array<int64_t, 2> rs = {T, D}, bs = {T, D / 128};
    const std::array<int64_t, 1> gs = {T};
    if (a[9] != Py_None) r = plain(a[9], at::kBFloat16, rs, dev, "r");
    {
      const Issue issue(*y.t);
      if (!r.defined()) r = make(rs, at::kBFloat16);
      if (kind == FP8BLK_NORM_BF16) {
        h = make(rs, at::kBFloat16);
      } else if (kind == FP8BLK_NORM_E4M3) {
        h = make(rs, at::kFloat8_e4m3fn), s = make(bs, at::kFloat);
      } else {
        h = make({T, D / 2}, at::kByte), s = make(scale_shape(T, D, fmt), at::kByte);
        if (fmt == FP8BLK_FP4_E4M3) g = make(gs, at::kFloat);
      }
      call(*y.t, "residual_norm", [&](fp8blk_stream_t st) {
        return lib.residual_norm(data(*y.t), y.stride, x, x_stride, post, col, tok, tok_stride, residual_scale, norm, eps, T,
                                 D, kind, fmt, r.mutable_data_ptr(), h.mutable_data_ptr(),
                                 s.defined() ? s.mutable_data_ptr() : nullptr,
                                 g.defined() ? g.mutable_data_ptr<float>() : nullptr, st);
      });
    }
    PyObject* out = kind == FP8BLK_NORM_BF16   ? THPVariable_Wrap(h)
                    : kind == FP8BLK_NORM_E4M3 ? tuple({&h, &s})
                                               : tuple({&h, &s, &g});
    return Py_BuildValue("(NN)", THPVariable_Wrap(r), out);
  });
}

// addresses {name: int}, Fp8BlkError, the workspaces, _buffer
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) throw std::runtime_error("setup: wrong number of arguments");
    auto get = [&](auto& f, const char* name) {
      PyObject* v = PyDict_GetItemString(a[0], name);
      if (!v) throw std::runtime_error(std::string("setup: no ") + name);
      f = reinterpret_cast<std::decay_t<decltype(f)>>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(v)));
      if (PyErr_Occurred()) throw python_error();
    };
    get(lib.status_string, "fp8blk_status_string");
    get(lib.fp4_quant, "fp8blk_fp4_quant");
    get(lib.fp4_dequant, "fp8blk_fp4_dequant");
    get(lib.fp4_gemm, "fp8blk_fp4_gemm");
    get(lib.fp4_linear, "fp8blk_fp4_linear");
    get(lib.fp4_linear_workspace_bytes, "fp8blk_fp4_linear_workspace_bytes");
    get(lib.residual_norm, "fp8blk_residual_norm");
    for (int i = 1; i < 4; ++i) Py_INCREF(a[i]);
    error_class = a[1], buffers = a[2], new_buffer = a[3];
    Py_RETURN_NONE;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {{"setup", fast<setup>(), METH_FASTCALL, nullptr},
                         {"fp4_quant", fast<fp4_quant>(), METH_FASTCALL, nullptr},
                         {"fp4_dequant", fast<fp4_dequant>(), METH_FASTCALL, nullptr},
                         {"fp4_gemm", fast<fp4_gemm>(), METH_FASTCALL, nullptr},
                         {"fp4_linear", fast<fp4_linear>(), METH_FASTCALL, nullptr},
                         {"residual_norm", fast<residual_norm>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Checks, outputs and calls of libfp8blk.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
