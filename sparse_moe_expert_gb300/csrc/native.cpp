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
#include <vector>

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
    case at::kChar: return "torch.int8";
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
  if (ts.size() == 0) Py_RETURN_NONE;
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

// A result that may be an input itself (same type and rows) and otherwise may
// not share memory with it: kernels read a row whole before they write it.
void same_or_apart(const Tensor& out, const char* name, const Tensor& in, const char* other) {
  if (!out.defined() || !in.defined() || out.numel() == 0 || in.numel() == 0) return;
  const auto lo = [](const Tensor& t) { return reinterpret_cast<uintptr_t>(t.data_ptr()); };
  const auto hi = [&](const Tensor& t) {
    int64_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    return lo(t) + (uintptr_t)(last + 1) * t.element_size();
  };
  if (lo(out) >= hi(in) || lo(in) >= hi(out)) return;
  bool same = lo(out) == lo(in) && out.scalar_type() == in.scalar_type() && out.sizes() == in.sizes();
  for (int64_t i = 0; same && i < out.dim(); ++i)
    same = out.size(i) == 1 || out.stride(i) == in.stride(i);
  if (!same) throw Refused(std::string(name) + " overlaps " + other);
}

void apart(const Tensor& out, const char* name, const Tensor& in, const char* other) {
  if (!out.defined() || !in.defined() || out.numel() == 0 || in.numel() == 0) return;
  if (out.data_ptr() == in.data_ptr()) throw Refused(std::string(name) + " overlaps " + other);
  same_or_apart(out, name, in, other);
}

struct Named {
  const Tensor& t;
  const char* name;
};
// A caller's buffer that shares memory with none of the others.
void apart_from(const Tensor& out, const char* name, std::initializer_list<Named> others) {
  if (!out.defined()) return;
  for (const Named& o : others) apart(out, name, o.t, o.name);
}

// x's rows [T, H], of `type` if given; the row stride.
int64_t rows_like(const Tensor& t, int64_t T, int64_t H, c10::Device dev, const char* name) {
  const int64_t ld = rows2d(t, name);
  if (t.size(0) != T || t.size(1) != H)
    throw Refused(std::string(name) + " must be [" + std::to_string(T) + ", " + std::to_string(H) +
                  "], got " + shape_text(t.sizes()));
  on_device(t, dev, name);
  return ld;
}

void same_type(const Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    throw Refused(std::string(name) + " must be " + type_name(type) + ", got " +
                  type_name(t.scalar_type()));
}

// A weight or bias [n], fp32 or bf16; both of one type.
int vector_pair(const Tensor& w, const char* wn, const Tensor& b, const char* bn, int64_t n,
                c10::Device dev) {
  const Tensor& first = w.defined() ? w : b;
  if (!first.defined()) return MOE_DTYPE_F32;
  const int code = dtype_code(first, w.defined() ? wn : bn);
  if (w.defined()) like(w, {n}, first.scalar_type(), dev, wn);
  if (b.defined()) like(b, {n}, first.scalar_type(), dev, bn);
  return code;
}

// x, weight, bias, residual, eps, kind, out_bf16 (None: as x), need_stats, out,
// summed, mean, rstd, stream
PyObject* layer_norm(Args a) {
  const Tensor &x = a.tensor("x"), &w = a.tensor("weight", true), &bias = a.tensor("bias", true),
               &residual = a.tensor("residual", true);
  const double eps = a.real();
  const int kind = a.i32();
  const std::optional<bool> out_bf16 = a.optional_flag();
  const bool need_stats = a.flag();
  Tensor out = a.tensor("out", true), summed = a.tensor("summed", true),
         mean = a.tensor("mean", true), rstd = a.tensor("rstd", true);
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    const int64_t ld = rows2d(x, "x");
    const int T = as_int(x.size(0), "T"), H = as_int(x.size(1), "H");
    const c10::Device dev = x.device();
    const OnStream on(stream, dev);
    int64_t ld_r = 0;
    const at::ScalarType xt = x.scalar_type();
    if (residual.defined()) {
      ld_r = rows_like(residual, T, H, dev, "residual");
      same_type(residual, xt, "residual");
      if (summed.defined()) like(summed, {T, H}, xt, dev, "summed");
      else summed = make({T, H}, xt, dev);
    } else if (summed.defined()) {
      throw Refused("summed needs a residual");
    }
    const int wt = vector_pair(w, "weight", bias, "bias", H, dev);
    at::ScalarType ot = out.defined() ? out.scalar_type() : xt;
    if (out_bf16) ot = *out_bf16 ? at::kBFloat16 : at::kFloat;
    if (out.defined()) like(out, {T, H}, ot, dev, "out");
    else out = make({T, H}, ot, dev);
    const int out_code = dtype_code(out, "out");
    const bool layer = kind == MOE_NORM_LAYER;
    for (const Tensor* v : {&mean, &rstd})  // the caller's
      apart_from(*v, v == &mean ? "mean" : "rstd",
                 {{out, "out"}, {summed, "summed"}, {x, "x"}, {residual, "residual"}, {w, "weight"}, {bias, "bias"}});
    apart(mean, "mean", rstd, "rstd");
    if (mean.defined()) like(mean, {T}, at::kFloat, dev, "mean");
    else if (need_stats && layer) mean = make({T}, at::kFloat, dev);
    if (rstd.defined()) like(rstd, {T}, at::kFloat, dev, "rstd");
    else if (need_stats) rstd = make({T}, at::kFloat, dev);
    same_or_apart(out, "out", x, "x");
    same_or_apart(out, "out", residual, "residual");
    same_or_apart(summed, "summed", x, "x");
    same_or_apart(summed, "summed", residual, "residual");
    apart(out, "out", summed, "summed");
    for (const Tensor* v : {&w, &bias}) {  // read by every row
      apart(out, "out", *v, v == &w ? "weight" : "bias");
      apart(summed, "summed", *v, v == &w ? "weight" : "bias");
    }
    return moe_layer_norm(x.data_ptr(), dtype_code(x, "x"), ld, ptr<void>(residual), ld_r,
                          ptr<void>(w), ptr<void>(bias), wt, T, H, kind, (float)eps, out_code,
                          out.data_ptr(), ptr<void>(summed), ptr<float>(mean), ptr<float>(rstd),
                          on.handle);
  });
  return s ? status(s) : result({out, summed, mean, rstd});
}

// d_out, x, rstd, mean, weight, d_sum, kind, need_d_weight, need_d_bias, d_x,
// d_weight, d_bias, workspace, stream
PyObject* layer_norm_backward(Args a) {
  const Tensor &d = a.tensor("d_out"), &x = a.tensor("x"), &rstd = a.tensor("rstd"),
               &mean = a.tensor("mean", true), &w = a.tensor("weight", true),
               &d_sum = a.tensor("d_sum", true);
  const int kind = a.i32();
  const bool need_w = a.flag(), need_b = a.flag();
  Tensor d_x = a.tensor("d_x", true), d_w = a.tensor("d_weight", true),
         d_b = a.tensor("d_bias", true), ws = a.tensor("workspace", true);
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    const int64_t ld_x = rows2d(x, "x");
    const int T = as_int(x.size(0), "T"), H = as_int(x.size(1), "H");
    const c10::Device dev = x.device();
    const OnStream on(stream, dev);
    const at::ScalarType xt = x.scalar_type();
    const int64_t ld_d = rows_like(d, T, H, dev, "d_out");
    if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARG;
    if ((kind == MOE_NORM_LAYER) != mean.defined())
      throw Refused("mean belongs to the layer norm, and to it alone");
    if (mean.defined()) like(mean, {T}, at::kFloat, dev, "mean");
    like(rstd, {T}, at::kFloat, dev, "rstd");
    const int wt = vector_pair(w, "weight", Tensor(), "", H, dev);
    int64_t ld_s = 0;
    if (d_sum.defined()) {
      ld_s = rows_like(d_sum, T, H, dev, "d_sum");
      same_type(d_sum, xt, "d_sum");
    }
    if (d_x.defined()) like(d_x, {T, H}, xt, dev, "d_x");
    else d_x = make({T, H}, xt, dev);
    for (const Tensor* o : {&d_w, &d_b, &ws})  // the caller's
      apart_from(*o, o == &d_w ? "d_weight" : o == &d_b ? "d_bias" : "workspace",
                 {{d_x, "d_x"}, {d, "d_out"}, {x, "x"}, {d_sum, "d_sum"}, {w, "weight"}, {mean, "mean"}, {rstd, "rstd"}});
    apart(d_w, "d_weight", d_b, "d_bias");
    apart_from(ws, "workspace", {{d_w, "d_weight"}, {d_b, "d_bias"}});
    if (d_w.defined()) like(d_w, {H}, at::kFloat, dev, "d_weight");
    else if (need_w) d_w = make({H}, at::kFloat, dev);
    if (d_b.defined()) like(d_b, {H}, at::kFloat, dev, "d_bias");
    else if (need_b) d_b = make({H}, at::kFloat, dev);
    same_or_apart(d_x, "d_x", d, "d_out");
    same_or_apart(d_x, "d_x", x, "x");
    same_or_apart(d_x, "d_x", d_sum, "d_sum");
    apart(d_x, "d_x", w, "weight");
    apart(d_x, "d_x", mean, "mean");
    apart(d_x, "d_x", rstd, "rstd");
    if (!ws.defined() && (d_w.defined() || d_b.defined()))
      ws = make({(int64_t)moe_layer_norm_workspace_size(T, H)}, at::kByte, dev);
    return moe_layer_norm_backward(
        d.data_ptr(), dtype_code(d, "d_out"), ld_d, x.data_ptr(), dtype_code(x, "x"), ld_x,
        ptr<float>(mean), ptr<float>(rstd), ptr<void>(w), wt, ptr<void>(d_sum), ld_s, T, H,
        d_x.data_ptr(), ptr<float>(d_w), ptr<float>(d_b), ptr<void>(ws),
        ws.defined() ? scratch_bytes(ws, dev) : 0, on.handle);
  });
  return s ? status(s) : result({d_x, d_w, d_b, ws});
}

// The tensors of a list or tuple; none at all for None.
std::vector<Tensor> tensors(PyObject* o, const char* name, bool optional = false) {
  std::vector<Tensor> out;
  if (o == Py_None && optional) return out;
  PyObject* seq = PyList_Check(o) || PyTuple_Check(o) ? o : nullptr;
  if (!seq) throw Refused(std::string(name) + " must be a list of tensors");
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  out.reserve(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* t = PySequence_Fast_GET_ITEM(seq, i);
    if (!THPVariable_Check(t)) throw Refused(std::string(name) + " must hold tensors");
    out.push_back(THPVariable_Unpack(t));
  }
  return out;
}

void entries(const std::vector<Tensor>& ts, size_t n, const char* name) {
  if (ts.size() != n)
    throw Refused(std::string(name) + " must have " + std::to_string(n) + " entries, got " +
                  std::to_string(ts.size()));
}

// One of a list's tensors: dense, of this type, with n elements.
void item(const Tensor& t, int64_t n, at::ScalarType type, c10::Device dev, const char* name) {
  need(t, type, name);
  if (t.numel() != n)
    throw Refused(std::string(name) + " must hold " + std::to_string(n) + " elements, got " +
                  std::to_string(t.numel()));
  on_device(t, dev, name);
}

constexpr int64_t kStateBlock = 256;  // elements that share a scale of the 8-bit states

void eight_bit_states(moe_adamw_tensor_t& e, const Tensor& m, const Tensor& v, const Tensor& ms,
                      const Tensor& vs, int64_t n, c10::Device dev) {
  const int64_t blocks = (n + kStateBlock - 1) / kStateBlock;
  item(m, n, at::kChar, dev, "exp_avg");
  item(v, n, at::kByte, dev, "exp_avg_sq");
  item(ms, blocks, at::kFloat, dev, "exp_avg_scales");
  item(vs, blocks, at::kFloat, dev, "exp_avg_sq_scales");
  e.exp_avg_scale = ptr<float>(ms);
  e.exp_avg_sq_scale = ptr<float>(vs);
}

// params, grads, exp_avg, exp_avg_sq, exp_avg_scales, exp_avg_sq_scales, masters,
// step, lr, lr_dev, beta1, beta2, eps, weight_decay (a float or a list),
// grad_scale, stream
PyObject* adamw_step(Args a) {
  const std::vector<Tensor> params = tensors(a.next(), "params"), grads = tensors(a.next(), "grads"),
                            m = tensors(a.next(), "exp_avg"), v = tensors(a.next(), "exp_avg_sq"),
                            ms = tensors(a.next(), "exp_avg_scales", true),
                            vs = tensors(a.next(), "exp_avg_sq_scales", true),
                            masters = tensors(a.next(), "masters", true);
  const Tensor& step = a.tensor("step");
  const double lr = a.real();
  const Tensor& lr_dev = a.tensor("lr", true);
  const double beta1 = a.real(), beta2 = a.real(), eps = a.real();
  const size_t n = params.size();
  std::vector<float> decay(n);
  PyObject* wd = a.next();
  if (PyList_Check(wd) || PyTuple_Check(wd)) {
    if ((size_t)PySequence_Fast_GET_SIZE(wd) != n)
      throw Refused("weight_decay must be a number or have " + std::to_string(n) + " entries");
    for (size_t i = 0; i < n; ++i) {
      decay[i] = (float)PyFloat_AsDouble(PySequence_Fast_GET_ITEM(wd, i));
      if (PyErr_Occurred()) throw Raised();
    }
  } else {
    const double one = PyFloat_AsDouble(wd);
    if (PyErr_Occurred()) throw Raised();
    decay.assign(n, (float)one);
  }
  const Tensor& scale = a.tensor("grad_scale", true);
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    const c10::Device dev = step.device();
    like(step, {2}, at::kInt, dev, "step");
    const OnStream on(stream, dev);
    if (scale.defined()) item(scale, 1, at::kFloat, dev, "grad_scale");
    if (lr_dev.defined()) item(lr_dev, 1, at::kFloat, dev, "lr");
    const bool eight = !ms.empty() || !vs.empty() || (n > 0 && !m.empty() && m[0].scalar_type() == at::kChar);
    entries(grads, n, "grads");
    entries(m, n, "exp_avg");
    entries(v, n, "exp_avg_sq");
    if (eight) {
      entries(ms, n, "exp_avg_scales");
      entries(vs, n, "exp_avg_sq_scales");
    }
    if (!masters.empty()) entries(masters, n, "masters");
    std::vector<moe_adamw_tensor_t> table(n);
    for (size_t i = 0; i < n; ++i) {
      moe_adamw_tensor_t& e = table[i];
      const int64_t size = params[i].numel();
      dtype_code(params[i], "params");
      dtype_code(grads[i], "grads");
      item(params[i], size, params[0].scalar_type(), dev, "params");
      item(grads[i], size, grads[0].scalar_type(), dev, "grads");
      e = {params[i].data_ptr(), grads[i].data_ptr(), nullptr, m[i].data_ptr(), v[i].data_ptr(),
           nullptr, nullptr, size, decay[i]};
      if (!masters.empty()) {
        item(masters[i], size, at::kFloat, dev, "masters");
        e.master = ptr<float>(masters[i]);
      }
      if (eight) {
        eight_bit_states(e, m[i], v[i], ms[i], vs[i], size, dev);
      } else {
        item(m[i], size, at::kFloat, dev, "exp_avg");
        item(v[i], size, at::kFloat, dev, "exp_avg_sq");
      }
    }
    return moe_adamw_step(table.data(), (int)n, n ? dtype_code(params[0], "params") : MOE_DTYPE_F32,
                          n ? dtype_code(grads[0], "grads") : MOE_DTYPE_F32, eight ? 8 : 32, lr,
                          ptr<float>(lr_dev), beta1, beta2, eps, ptr<float>(scale),
                          ptr<int32_t>(step), on.handle);
  });
  return s ? status(s) : result({});
}

// params, grads: the checks of the gradients that adamw_step makes
PyObject* adamw_check(Args a) {
  const std::vector<Tensor> params = tensors(a.next(), "params"), grads = tensors(a.next(), "grads");
  unlocked([&] {
    entries(grads, params.size(), "grads");
    for (size_t i = 0; i < params.size(); ++i) {
      dtype_code(grads[i], "grads");
      item(grads[i], params[i].numel(), grads[0].scalar_type(), params[0].device(), "grads");
    }
    return MOE_OK;
  });
  return result({});
}

// exp_avg, exp_avg_sq, exp_avg_scales, exp_avg_sq_scales, stream
PyObject* adamw_values(Args a) {
  const std::vector<Tensor> m = tensors(a.next(), "exp_avg"), v = tensors(a.next(), "exp_avg_sq"),
                            ms = tensors(a.next(), "exp_avg_scales"),
                            vs = tensors(a.next(), "exp_avg_sq_scales");
  const StreamArg stream(a.next());
  Tensor out_m, out_v;
  if (m.empty()) throw Refused("exp_avg must not be empty");
  const moe_status_t s = unlocked([&] {
    const size_t n = m.size();
    entries(v, n, "exp_avg_sq");
    entries(ms, n, "exp_avg_scales");
    entries(vs, n, "exp_avg_sq_scales");
    const c10::Device dev = m[0].device();
    std::vector<moe_adamw_tensor_t> table(n);
    int64_t total = 0;
    for (size_t i = 0; i < n; ++i) {
      const int64_t size = m[i].numel();
      table[i] = {nullptr, nullptr, nullptr, m[i].data_ptr(), v[i].data_ptr(), nullptr, nullptr, size,
                  0.0f};
      eight_bit_states(table[i], m[i], v[i], ms[i], vs[i], size, dev);
      total += size;
    }
    const OnStream on(stream, dev);
    out_m = make({total}, at::kFloat, dev);
    out_v = make({total}, at::kFloat, dev);
    return moe_adamw_values(table.data(), (int)n, ptr<float>(out_m), ptr<float>(out_v), on.handle);
  });
  return s ? status(s) : result({out_m, out_v});
}

// Rows of a bf16 matrix that a tensor map can describe: 16-byte aligned rows.
int64_t mapped_rows(const Tensor& t, const char* name) {
  const int64_t ld = rows2d(t, name);
  same_type(t, at::kBFloat16, name);
  if (ld % 8 != 0 || reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 != 0)
    throw Refused(std::string(name) + " must have 16-byte aligned rows");
  return ld;
}

// x, w, bias, residual, activation, out, out_bf16 (None: bf16, or as residual),
// need_preact, preact, stream
PyObject* linear(Args a) {
  const Tensor &x = a.tensor("x"), &w = a.tensor("w"), &bias = a.tensor("bias", true),
               &residual = a.tensor("residual", true);
  const int act = a.i32();
  Tensor out = a.tensor("out", true);
  const std::optional<bool> out_bf16 = a.optional_flag();
  const bool need_preact = a.flag();
  Tensor preact = a.tensor("preact", true);
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    const int64_t ld = mapped_rows(x, "x");
    const c10::Device dev = x.device();
    const OnStream on(stream, dev);
    const int T = as_int(x.size(0), "T"), K = as_int(x.size(1), "K");
    if (w.dim() != 2 || w.size(1) != K) throw Refused("w must be [N, " + std::to_string(K) + "]");
    const int N = as_int(w.size(0), "N");
    like(w, {N, K}, at::kBFloat16, dev, "w");
    if (bias.defined()) like(bias, {N}, at::kFloat, dev, "bias");
    if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
    const int64_t cols = act == MOE_ACT_SWIGLU ? N / 2 : N;
    at::ScalarType ot = out.defined() ? out.scalar_type()
                        : residual.defined() ? residual.scalar_type() : at::kBFloat16;
    if (out_bf16) ot = *out_bf16 ? at::kBFloat16 : at::kFloat;
    if (residual.defined()) like(residual, {T, cols}, ot, dev, "residual");
    if (out.defined()) like(out, {T, cols}, ot, dev, "out");
    else out = make({T, cols}, ot, dev);
    const int out_code = dtype_code(out, "out");
    if (preact.defined()) like(preact, {T, N}, at::kBFloat16, dev, "preact");
    else if (need_preact) preact = make({T, N}, at::kBFloat16, dev);
    same_or_apart(out, "out", residual, "residual");
    for (const Tensor* o : {&out, &preact}) {
      const char* name = o == &out ? "out" : "preact";
      apart(*o, name, x, "x");
      apart(*o, name, w, "w");
      apart(*o, name, bias, "bias");
    }
    apart(preact, "preact", out, "out");
    apart(preact, "preact", residual, "residual");
    return moe_linear(ptr<uint16_t>(x), ld, ptr<uint16_t>(w), ptr<float>(bias), ptr<void>(residual), T,
                      K, N, act, out_code, out.data_ptr(), ptr<uint16_t>(preact), on.handle);
  });
  return s ? status(s) : result({out, preact});
}

// d_out, x, w, preact, activation, need_d_x, need_d_w, need_d_bias, d_x, d_w,
// d_w_bf16 (None: fp32), accumulate, d_bias, workspace, stream
PyObject* linear_backward(Args a) {
  const Tensor &d = a.tensor("d_out"), &x = a.tensor("x"), &w = a.tensor("w", true),
               &preact = a.tensor("preact", true);
  const int act = a.i32();
  const bool need_x = a.flag(), need_w = a.flag(), need_b = a.flag();
  Tensor d_x = a.tensor("d_x", true), d_w = a.tensor("d_w", true);
  const std::optional<bool> w_bf16 = a.optional_flag();
  const bool accumulate = a.flag();
  Tensor d_b = a.tensor("d_bias", true), ws = a.tensor("workspace", true), d_z;
  const StreamArg stream(a.next());
  const moe_status_t s = unlocked([&] {
    const int64_t ld_x = mapped_rows(x, "x");
    const c10::Device dev = x.device();
    const OnStream on(stream, dev);
    const int T = as_int(x.size(0), "T"), K = as_int(x.size(1), "K");
    if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
    if (d.dim() != 2) throw Refused("d_out must have two dimensions");
    // without w (no d_x) the gradient's width says how many features there are
    if (!w.defined() && (need_x || d_x.defined())) throw Refused("d_x needs w");
    if (w.defined() && (w.dim() != 2 || w.size(1) != K))
      throw Refused("w must be [N, " + std::to_string(K) + "]");
    const int N = as_int(w.defined() ? w.size(0) : d.size(1) * (act == MOE_ACT_SWIGLU ? 2 : 1), "N");
    if (w.defined()) like(w, {N, K}, at::kBFloat16, dev, "w");
    const int64_t cols = act == MOE_ACT_SWIGLU ? N / 2 : N;
    const int64_t ld_d = rows_like(d, T, cols, dev, "d_out");
    if (preact.defined()) like(preact, {T, N}, at::kBFloat16, dev, "preact");
    else if (act != MOE_ACT_NONE) throw Refused("preact is needed for the activation's gradient");
    if (d_x.defined()) like(d_x, {T, K}, at::kBFloat16, dev, "d_x");
    else if (need_x) d_x = make({T, K}, at::kBFloat16, dev);
    if (accumulate && !d_w.defined()) throw Refused("accumulate needs d_w");
    at::ScalarType wt = d_w.defined() ? d_w.scalar_type() : at::kFloat;
    if (w_bf16) wt = *w_bf16 ? at::kBFloat16 : at::kFloat;
    if (d_w.defined()) like(d_w, {N, K}, wt, dev, "d_w");
    else if (need_w) d_w = make({N, K}, wt, dev);
    const int w_code = d_w.defined() ? dtype_code(d_w, "d_w") : MOE_DTYPE_F32;
    if (d_b.defined()) like(d_b, {N}, at::kFloat, dev, "d_bias");
    else if (need_b) d_b = make({N}, at::kFloat, dev);
    for (const Tensor* o : {&d_x, &d_w, &d_b}) {
      const char* name = o == &d_x ? "d_x" : o == &d_w ? "d_w" : "d_bias";
      apart(*o, name, d, "d_out");
      apart(*o, name, x, "x");
      apart(*o, name, w, "w");
      apart(*o, name, preact, "preact");
    }
    apart(d_x, "d_x", d_w, "d_w");
    apart_from(d_b, "d_bias", {{d_x, "d_x"}, {d_w, "d_w"}});
    apart_from(ws, "workspace",
               {{d_x, "d_x"}, {d_w, "d_w"}, {d_b, "d_bias"}, {d, "d_out"}, {x, "x"}, {w, "w"}, {preact, "preact"}});
    // d_out is d_preact where it is bf16 with aligned rows and nothing was activated
    const bool direct = act == MOE_ACT_NONE && d.scalar_type() == at::kBFloat16 && ld_d % 8 == 0 &&
                        reinterpret_cast<uintptr_t>(d.data_ptr()) % 16 == 0;
    int64_t ld_z = 0;
    if (direct) {
      d_z = d;
    } else {
      ld_z = ((int64_t)N + 7) / 8 * 8;
      d_z = at::detail::empty_strided_cuda({T, N}, {ld_z, 1}, at::kBFloat16, dev);
    }
    if (!ws.defined() && d_b.defined())
      ws = make({(int64_t)moe_linear_backward_workspace_size(T, N, act)}, at::kByte, dev);
    return moe_linear_backward(d.data_ptr(), dtype_code(d, "d_out"), ld_d, ptr<uint16_t>(x), ld_x,
                               ptr<uint16_t>(w), ptr<uint16_t>(preact), T, K, N, act,
                               direct ? nullptr : ptr<uint16_t>(d_z), ld_z, ptr<uint16_t>(d_x),
                               ptr<void>(d_w), w_code, accumulate, ptr<float>(d_b), ptr<void>(ws),
                               ws.defined() ? scratch_bytes(ws, dev) : 0, on.handle);
  });
  if (s) return status(s);
  return result({d_x, d_w, d_b, d_z, ws});
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
    {"layer_norm", method<layer_norm>(), METH_FASTCALL, nullptr},
    {"layer_norm_backward", method<layer_norm_backward>(), METH_FASTCALL, nullptr},
    {"linear", method<linear>(), METH_FASTCALL, nullptr},
    {"linear_backward", method<linear_backward>(), METH_FASTCALL, nullptr},
    {"adamw_step", method<adamw_step>(), METH_FASTCALL, nullptr},
    {"adamw_check", method<adamw_check>(), METH_FASTCALL, nullptr},
    {"adamw_values", method<adamw_values>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
