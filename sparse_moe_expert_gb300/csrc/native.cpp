// CPython entry points of the short calls: argument checks, allocation of
// missing outputs and the C call in one step, for work that takes the device
// a few microseconds.  Written in Python they cost 11 to 21 us of host time per
// call (0.1 us for each attribute of a tensor, 3.4 us for the current stream,
// 1.5 us per allocation), here 4 to 8.
//
// Built against the installed torch next to libmoe_gb300.so, which it calls
// through the C ABI; binding.py has the documented functions.  A function
// returns its tensors, or the status code when the C call refuses; wrong
// tensors raise ValueError.  Nothing is retained between calls.  The arguments
// are read under the interpreter's lock, checks, allocation and the call run
// without it: a launch may wait for room in its stream's queue.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/moe_gb300.h"

namespace {

using at::Tensor;

// A refused argument; becomes ValueError.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

// A Python error is already set.
struct Raised {};

std::string shape_text(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

struct Args {
  PyObject* const* v;
  Py_ssize_t n;
  Py_ssize_t i = 0;

  PyObject* next() {
    if (i >= n) throw Refused("too few arguments");
    return v[i++];
  }
  // A tensor, or an undefined one for None where that is allowed.
  const Tensor& tensor(const char* name, bool optional = false) {
    static const Tensor none;
    PyObject* o = next();
    if (o == Py_None && optional) return none;
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  int64_t integer() {
    const long long x = PyLong_AsLongLong(next());
    if (x == -1 && PyErr_Occurred()) throw Raised();
    return x;
  }
  // An int for the C call, which checks its range.
  int i32() {
    const int64_t x = integer();
    if (x < INT32_MIN || x > INT32_MAX) throw Refused("integer argument out of range");
    return (int)x;
  }
  std::optional<int> optional_i32() {
    if (i < n && v[i] == Py_None) {
      ++i;
      return std::nullopt;
    }
    return i32();
  }
  double real() {
    const double x = PyFloat_AsDouble(next());
    if (x == -1.0 && PyErr_Occurred()) throw Raised();
    return x;
  }
  bool flag() {
    const int x = PyObject_IsTrue(next());
    if (x < 0) throw Raised();
    return x != 0;
  }
  std::optional<bool> optional_flag() {
    if (i < n && v[i] == Py_None) {
      ++i;
      return std::nullopt;
    }
    return flag();
  }
};

int dtype_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return MOE_DTYPE_F32;
  if (t.scalar_type() == at::kBFloat16) return MOE_DTYPE_BF16;
  throw Refused(std::string(name) + " must be float32 or bfloat16, got " + type_name(t.scalar_type()));
}

void need(const Tensor& t, at::ScalarType type, const char* name) {
  if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type)
    throw Refused(std::string(name) + " must be " + type_name(type) + ", got " +
                  type_name(t.scalar_type()));
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
}

void on_device(const Tensor& t, c10::Device dev, const char* name) {
  if (t.device() != dev) throw Refused(std::string(name) + " must be on " + dev.str());
}

void like(const Tensor& t, c10::IntArrayRef shape, at::ScalarType type, c10::Device dev,
          const char* name) {
  need(t, type, name);
  if (t.sizes() != shape)
    throw Refused(std::string(name) + " must have shape " + shape_text(shape) + ", got " +
                  shape_text(t.sizes()));
  on_device(t, dev, name);
}

void flat(const Tensor& t, int64_t least, c10::Device dev, const char* name) {
  need(t, at::kInt, name);
  if (t.numel() < least)
    throw Refused(std::string(name) + " must hold " + std::to_string(least) + " entries");
  on_device(t, dev, name);
}

// A contiguous fp32 or bf16 matrix of at least `rows` rows of `cols`.
void matrix(const Tensor& t, int64_t rows, int64_t cols, c10::Device dev, const char* name) {
  dtype_code(t, name);
  need(t, t.scalar_type(), name);
  if (t.dim() != 2 || t.size(0) < rows || t.size(1) != cols)
    throw Refused(std::string(name) + " must be [" + std::to_string(rows) + ", " +
                  std::to_string(cols) + "], got " + shape_text(t.sizes()));
  on_device(t, dev, name);
}

// Row stride of a 2D CUDA tensor of fp32 or bf16 with dense rows.
int64_t rows2d(const Tensor& t, const char* name) {
  if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
  dtype_code(t, name);
  if (t.dim() != 2) throw Refused(std::string(name) + " must have two dimensions");
  const int64_t T = t.size(0), E = t.size(1);
  if (E > 1 && t.stride(1) != 1) throw Refused(std::string(name) + " must have contiguous rows");
  if (T <= 1) return E;
  if (t.stride(0) < E) throw Refused(std::string(name) + " must have rows that do not overlap");
  return t.stride(0);
}

Tensor make(c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

int as_int(int64_t v, const char* what) {
  if (v < 0 || v > INT32_MAX) throw Refused(std::string(what) + " is too large");
  return (int)v;
}

template <typename T>
T* ptr(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

size_t scratch_bytes(const Tensor& t, c10::Device dev) {
  if (t.device() != dev || !t.is_contiguous())
    throw Refused("workspace must be a contiguous tensor on " + dev.str());
  return (size_t)t.nbytes();
}

// The stream that Python passed, if any.
struct StreamArg {
  bool given;
  moe_stream_t handle;

  explicit StreamArg(PyObject* o) : given(o != Py_None), handle(nullptr) {
    if (given) handle = PyLong_AsVoidPtr(o);
    if (given && !handle && PyErr_Occurred()) throw Raised();
  }
};

// The device and stream a call runs on: the handle that Python passed, or the
// device's current stream.  While it lives they are torch's current ones, so
// that what the call allocates belongs to its stream: a block that another
// stream gave up, and may still read, is not handed out to it.
struct OnStream {
  c10::cuda::CUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  moe_stream_t handle;

  OnStream(const StreamArg& s, c10::Device dev) : device(dev), handle(s.handle) {
    if (s.given)
      guard.reset_stream(
          c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), dev.index()));
    else
      handle = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  }
};

// f() without the interpreter's lock.
template <typename F>
moe_status_t unlocked(F&& f) {
  struct Release {
    PyThreadState* state = PyEval_SaveThread();
    ~Release() { PyEval_RestoreThread(state); }
  } release;
  return f();
}

PyObject* result(std::initializer_list<Tensor> ts) {
  PyObject* t = PyTuple_New((Py_ssize_t)ts.size());
  if (!t) throw Raised();
  Py_ssize_t i = 0;
  for (const Tensor& x : ts) {
    PyObject* o;
    if (x.defined()) {
      o = THPVariable_Wrap(x);
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    if (!o) {
      Py_DECREF(t);
      throw Raised();
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

PyObject* status(moe_status_t s) { return PyLong_FromLong((long)s); }

// logits, k, score, select_bias, n_groups, topk_groups, group_top, renormalize,
// scale, kmax (None: k), topk_ids, topk_w, k_dev, stream
PyObject* route_scored(Args a) {
  const Tensor& logits = a.tensor("logits");
  const int k = a.i32(), score = a.i32();
  const Tensor& bias = a.tensor("select_bias", true);
  const int n_groups = a.i32(), topk_groups = a.i32(), group_top = a.i32();
  const bool renorm = a.flag();
  const double scale = a.real();
  const int kmax = a.optional_i32().value_or(k);
  Tensor ids = a.tensor("topk_ids", true), w = a.tensor("topk_w", true),
         k_dev = a.tensor("k_dev", true);
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    const int64_t ld = rows2d(logits, "logits");
    const int T = as_int(logits.size(0), "T"), E = as_int(logits.size(1), "E");
    if (kmax < 0) return MOE_ERR_INVALID_ARG;
    const c10::Device dev = logits.device();
    const OnStream on(stream, dev);
    if (bias.defined()) like(bias, {E}, at::kFloat, dev, "select_bias");
    if (ids.defined()) like(ids, {T, kmax}, at::kInt, dev, "topk_ids");
    else ids = make({T, kmax}, at::kInt, dev);
    if (w.defined()) like(w, {T, kmax}, at::kFloat, dev, "topk_w");
    else w = make({T, kmax}, at::kFloat, dev);
    if (k_dev.defined()) like(k_dev, {1}, at::kInt, dev, "k_dev");
    else k_dev = make({1}, at::kInt, dev);
    return moe_route_scored(logits.data_ptr(), dtype_code(logits, "logits"), ld, ptr<float>(bias),
                            T, E, score, n_groups, topk_groups, group_top, k, kmax, renorm,
                            (float)scale, ptr<int32_t>(ids), ptr<float>(w), ptr<int32_t>(k_dev),
                            on.handle);
  });
  return s ? status(s) : result({ids, w, k_dev});
}

// logits, topk_ids, d_topk_w, expert_counts, score, k (None: kmax), renormalize,
// scale, balance_coef, z_coef, d_logits, losses, workspace, stream
PyObject* route_scored_backward(Args a) {
  const Tensor &logits = a.tensor("logits"), &ids = a.tensor("topk_ids"),
               &d_w = a.tensor("d_topk_w", true), &counts = a.tensor("expert_counts", true);
  const int score = a.i32();
  const std::optional<int> k = a.optional_i32();
  const bool renorm = a.flag();
  const double scale = a.real(), balance = a.real(), z = a.real();
  Tensor d_logits = a.tensor("d_logits", true), losses = a.tensor("losses", true),
         ws = a.tensor("workspace", true);
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    const int64_t ld = rows2d(logits, "logits");
    const int T = as_int(logits.size(0), "T"), E = as_int(logits.size(1), "E");
    const c10::Device dev = logits.device();
    if (ids.dim() != 2 || ids.size(0) != T) throw Refused("topk_ids must be [T, kmax]");
    const int kmax = as_int(ids.size(1), "kmax");
    like(ids, {T, kmax}, at::kInt, dev, "topk_ids");
    const OnStream on(stream, dev);
    if (d_w.defined()) like(d_w, {T, kmax}, at::kFloat, dev, "d_topk_w");
    if (counts.defined()) like(counts, {E}, at::kInt, dev, "expert_counts");
    int64_t ld_out = E;
    if (d_logits.defined()) {
      if (d_logits.scalar_type() != logits.scalar_type() || d_logits.sizes() != logits.sizes())
        throw Refused("d_logits must have the type and shape of logits");
      on_device(d_logits, dev, "d_logits");
      ld_out = rows2d(d_logits, "d_logits");
    } else {
      d_logits = make({T, E}, logits.scalar_type(), dev);
    }
    if (losses.defined()) like(losses, {2}, at::kFloat, dev, "losses");
    else losses = make({2}, at::kFloat, dev);
    if (!ws.defined())
      ws = make({(int64_t)moe_route_backward_workspace_size(E)}, at::kByte, dev);
    return moe_route_scored_backward(
        logits.data_ptr(), dtype_code(logits, "logits"), ld, ptr<int32_t>(ids), ptr<float>(d_w),
        ptr<int32_t>(counts), T, E, score, k.value_or(kmax), kmax, renorm, (float)scale,
        (float)balance, (float)z, d_logits.data_ptr(), ld_out, ptr<float>(losses), ws.data_ptr(),
        scratch_bytes(ws, dev), on.handle);
  });
  return s ? status(s) : result({d_logits, losses, ws});
}

// d_out, y, inv_pos, topk_w, k_dev, d_topk_w, d_y, need_d_y, stream
PyObject* combine_backward(Args a) {
  const Tensor &d_out = a.tensor("d_out"), &y = a.tensor("y"), &inv_pos = a.tensor("inv_pos"),
               &w = a.tensor("topk_w"), &k_dev = a.tensor("k_dev");
  Tensor d_w = a.tensor("d_topk_w", true), d_y = a.tensor("d_y", true);
  const bool need_d_y = a.flag();
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    need(d_out, at::kBFloat16, "d_out");
    if (d_out.dim() != 2) throw Refused("d_out must be [T, H]");
    const int T = as_int(d_out.size(0), "T"), H = as_int(d_out.size(1), "H");
    const c10::Device dev = d_out.device();
    const OnStream on(stream, dev);
    if (w.dim() != 2) throw Refused("topk_w must be [T, kmax]");
    const int kmax = as_int(w.size(1), "kmax");
    like(w, {T, kmax}, at::kFloat, dev, "topk_w");
    flat(inv_pos, (int64_t)T * kmax, dev, "inv_pos");
    matrix(y, (int64_t)T * kmax, H, dev, "y");
    like(k_dev, {1}, at::kInt, dev, "k_dev");
    if (d_w.defined()) like(d_w, {T, kmax}, at::kFloat, dev, "d_topk_w");
    else d_w = make({T, kmax}, at::kFloat, dev);
    if (d_y.defined()) like(d_y, y.sizes(), y.scalar_type(), dev, "d_y");
    else if (need_d_y) d_y = at::zeros_like(y);
    return moe_combine_backward(ptr<uint16_t>(d_out), y.data_ptr(), dtype_code(y, "y"),
                                ptr<int32_t>(inv_pos), ptr<float>(w), ptr<int32_t>(k_dev), T, kmax,
                                H, ptr<float>(d_w), ptr<void>(d_y), on.handle);
  });
  return s ? status(s) : result({d_w, d_y});
}

// x, adapter_ids, lora_a, lora_b, scales, base, out, epilogue, out_bf16 (None:
// by the base), topk_ids, sorted_assign, expert_offsets, x_by_token, workspace,
// stream
PyObject* lora_apply(Args a) {
  const Tensor &x = a.tensor("x"), &ad = a.tensor("adapter_ids"), &la = a.tensor("lora_a"),
               &lb = a.tensor("lora_b"), &scales = a.tensor("scales", true),
               &base = a.tensor("base", true);
  Tensor out = a.tensor("out", true);
  const int epilogue = a.i32();
  const std::optional<bool> out_bf16 = a.optional_flag();
  const Tensor &ids = a.tensor("topk_ids", true), &sorted = a.tensor("sorted_assign", true),
               &offsets = a.tensor("expert_offsets", true);
  const bool by_token = a.flag();
  Tensor ws = a.tensor("workspace", true);
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    need(x, at::kBFloat16, "x");
    const c10::Device dev = x.device();
    const OnStream on(stream, dev);
    if (la.dim() != 3 && la.dim() != 4) throw Refused("lora_a must be [n, R, K] or [n, E, R, K]");
    if (lb.dim() != la.dim()) throw Refused("lora_b does not match lora_a");
    const bool experts = la.dim() == 4;
    const int n = as_int(la.size(0), "adapters"), E = experts ? as_int(la.size(1), "E") : 1;
    const int R = as_int(la.size(-2), "R"), K = as_int(la.size(-1), "K");
    const int N = as_int(lb.size(-2), "N");
    need(la, at::kBFloat16, "lora_a");
    on_device(la, dev, "lora_a");
    if (experts) like(lb, {n, E, N, R}, at::kBFloat16, dev, "lora_b");
    else like(lb, {n, N, R}, at::kBFloat16, dev, "lora_b");
    if (ad.dim() != 1) throw Refused("adapter_ids must be [T]");
    const int T = as_int(ad.size(0), "T");
    like(ad, {T}, at::kInt, dev, "adapter_ids");
    int kmax = 1;
    if (sorted.defined() != ids.defined() || sorted.defined() != offsets.defined())
      throw Refused("expert rows need topk_ids, sorted_assign and expert_offsets");
    if (sorted.defined()) {
      if (ids.dim() != 2) throw Refused("topk_ids must be [T, kmax]");
      kmax = as_int(ids.size(1), "kmax");
      like(ids, {T, kmax}, at::kInt, dev, "topk_ids");
      like(offsets, {E + 1}, at::kInt, dev, "expert_offsets");
      flat(sorted, (int64_t)T * kmax, dev, "sorted_assign");
    }
    const int64_t rows = (int64_t)T * kmax;
    if (x.dim() != 2 || x.size(1) != K)
      throw Refused("x must be [rows, " + std::to_string(K) + "]");
    if (x.size(0) < (by_token ? T : rows)) throw Refused("x has too few rows");
    if (scales.defined()) like(scales, {n}, at::kFloat, dev, "scales");
    const bool swiglu = epilogue == MOE_EPILOGUE_SWIGLU;
    const int64_t cols = swiglu ? N / 2 : N;
    if (base.defined()) matrix(base, rows, N, dev, "base");
    if (out.defined()) {
      matrix(out, rows, cols, dev, "out");
    } else {
      at::ScalarType t = swiglu || !base.defined() ? at::kBFloat16 : base.scalar_type();
      if (out_bf16) t = *out_bf16 ? at::kBFloat16 : at::kFloat;
      out = make({rows, cols}, t, dev);
    }
    const int out_dt = dtype_code(out, "out");
    if (!ws.defined())
      ws = make({(int64_t)moe_lora_workspace_size(T, kmax, E, n, R)}, at::kByte, dev);
    return moe_lora_apply(
        ptr<uint16_t>(x), by_token, ptr<int32_t>(ad), ptr<int32_t>(ids), ptr<int32_t>(sorted),
        ptr<int32_t>(offsets), T, kmax, E, n, K, N, R, ptr<uint16_t>(la), ptr<uint16_t>(lb),
        ptr<float>(scales), ptr<void>(base), base.defined() ? dtype_code(base, "base") : out_dt,
        epilogue, out_dt, out.data_ptr(), ws.data_ptr(), scratch_bytes(ws, dev), on.handle);
  });
  return s ? status(s) : result({out, ws});
}

// C++ exceptions end here: refusals and torch's own errors become Python
// exceptions.
template <PyObject* (*F)(Args)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(Args{args, n});
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (!type) PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_RuntimeError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*F)(Args)>
PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>));
}

PyMethodDef methods[] = {
    {"route_scored", method<route_scored>(), METH_FASTCALL, nullptr},
    {"route_scored_backward", method<route_scored_backward>(), METH_FASTCALL, nullptr},
    {"combine_backward", method<combine_backward>(), METH_FASTCALL, nullptr},
    {"lora_apply", method<lora_apply>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
