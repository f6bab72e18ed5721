// block_binding.cpp — the Python binding of include/w4a4_block.h: checks of the
// tensors, allocation of the outputs that are not given, and the calls on the
// tensors' current stream.  No arithmetic.  It is compiled against torch
// because a call's host time is what a small call costs: through ctypes the
// marshalling of these argument lists took 5 to 8 us beside the launch's 3.
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "w4a4_block.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

PyObject* g_error = nullptr;  // the class of the library's errors

void check(const char* name, int status) {
  if (status == W4A4_OK) return;
  py::object e = py::reinterpret_borrow<py::object>(g_error)(name, status);
  PyErr_SetObject(g_error, e.ptr());
  throw py::error_already_set();
}

std::string text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

int dtype_of(at::ScalarType t) {
  if (t == at::kFloat) return W4A4_F32;
  if (t == at::kHalf) return W4A4_F16;
  throw py::type_error(std::string("unsupported dtype ") + c10::toString(t));
}

void on_device(const Tensor& t, const char* name, int64_t dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    throw py::value_error(std::string(name) + " must be a device tensor, on the device of the others");
}
int64_t device_index(const Tensor& t) {
  if (!t.is_cuda()) throw py::value_error("the tensors must be device tensors");
  return t.get_device();
}

// The row distance of a device matrix [M, C] with contiguous rows.  A single row's
// is C: the distance to a next row, which may be any (and off 16 bytes), is not used.
int64_t rows(const Tensor& t, const char* name, int64_t dev, int64_t M, int64_t C) {
  on_device(t, name, dev);
  if (t.dim() != 2 || t.size(0) != M || t.size(1) != C)
    throw py::value_error(std::string(name) + " must be " + text({M, C}) + ", not " + text(t.sizes()));
  if (C > 1 && t.stride(1) != 1) throw py::value_error(std::string(name) + " must have contiguous rows");
  if (M < 2) return C;
  if (t.stride(0) < C) throw py::value_error(std::string(name) + " must have rows that do not overlap");
  return t.stride(0);
}

// The address of a contiguous device tensor of this dtype and shape.
void* whole(const Tensor& t, const char* name, int64_t dev, at::ScalarType dtype, at::IntArrayRef shape) {
  on_device(t, name, dev);
  if (t.scalar_type() != dtype)
    throw py::type_error(std::string(name) + " must be " + c10::toString(dtype) + ", not " +
                         c10::toString(t.scalar_type()));
  if (t.sizes() != shape)
    throw py::value_error(std::string(name) + " must be " + text(shape) + ", not " + text(t.sizes()));
  if (!t.is_contiguous()) throw py::value_error(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

Tensor empty(const Tensor& like, at::IntArrayRef shape, at::ScalarType dtype) {
  return at::empty(shape, like.options().dtype(dtype));
}

void* stream_of(int64_t dev) {
  return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

Tensor adapter_add(const OptTensor& y, const Tensor& x, const Tensor& At, const Tensor& Bt,
                   const Tensor& index, const OptTensor& ranks, const OptTensor& scales, OptTensor out,
                   OptTensor workspace) {
  const int64_t dev = device_index(x);
  if (x.dim() != 2) throw py::value_error("x must be a matrix");
  if (At.dim() != 3 || Bt.dim() != 3)
    throw py::value_error("At must be [adapters, rank, K] and Bt [adapters, N, rank]");
  const at::ScalarType dt = x.scalar_type();
  const int64_t L = At.size(0), R = At.size(1), K = At.size(2), M = x.size(0), N = Bt.size(1);
  const int64_t ldx = rows(x, "x", dev, M, K);
  const void* at = whole(At, "At", dev, dt, {L, R, K});
  const void* bt = whole(Bt, "Bt", dev, dt, {L, N, R});
  const void* ix = whole(index, "index", dev, at::kInt, {M});
  const void* rk = ranks ? whole(*ranks, "ranks", dev, at::kInt, {L}) : nullptr;
  const void* sc = scales ? whole(*scales, "scales", dev, at::kFloat, {L}) : nullptr;
  const float* yp = nullptr;
  int64_t ldy = N, ldo = N;
  if (y) {
    if (y->scalar_type() != at::kFloat) throw py::type_error("y must be float32");
    ldy = rows(*y, "y", dev, M, N);
    yp = static_cast<const float*>(y->data_ptr());
  }
  const int xd = dtype_of(dt);
  const c10::DeviceGuard guard(x.device());
  if (out) {
    if (out->scalar_type() != at::kFloat) throw py::type_error("out must be float32");
    ldo = rows(*out, "out", dev, M, N);
  } else {
    out = empty(x, {M, N}, at::kFloat);
  }
  if (workspace) {
    on_device(*workspace, "workspace", dev);
    if (!workspace->is_contiguous()) throw py::value_error("workspace must be contiguous");
  } else {
    workspace = empty(x, {static_cast<int64_t>(w4a4_adapter_workspace_size(M, K, R))}, at::kByte);
  }
  check("adapter_add",
        w4a4_adapter_add(x.data_ptr(), xd, ldx, at, bt, L, R, static_cast<const int32_t*>(ix),
                         static_cast<const int32_t*>(rk), static_cast<const float*>(sc), M, N, K, yp, ldy,
                         static_cast<float*>(out->data_ptr()), ldo, workspace->data_ptr(),
                         workspace->nbytes(), stream_of(dev)));
  return *out;
}

std::pair<OptTensor, OptTensor> norm_residual(
    const OptTensor& h, const OptTensor& y, int post, const OptTensor& post_w, const OptTensor& post_b,
    const OptTensor& gate, int64_t gate_rows, double residual_scale, int pre, const OptTensor& pre_w,
    const OptTensor& pre_b, double offset, double eps, std::optional<at::ScalarType> x_dtype, OptTensor h_out,
    OptTensor x_out, bool want_h) {
  if (!h && !y) throw py::value_error("h or y must be given");
  const Tensor& ref = h ? *h : *y;
  const int64_t dev = device_index(ref);
  if (ref.dim() != 2) throw py::value_error("h and y must be matrices");
  const at::ScalarType dt = ref.scalar_type();
  const int64_t M = ref.size(0), C = ref.size(1);
  const int hd = dtype_of(dt), yd = y ? dtype_of(y->scalar_type()) : W4A4_F32;
  const int64_t ldh = h ? rows(*h, "h", dev, M, C) : C;
  const int64_t ldy = y ? rows(*y, "y", dev, M, C) : C;
  // One dtype for all parameters; the library refuses others than its own.
  std::optional<at::ScalarType> pt;
  auto param = [&](const OptTensor& t, const char* name) -> const void* {
    if (!t) return nullptr;
    if (!pt) pt = t->scalar_type();
    return whole(*t, name, dev, *pt, {C});
  };
  const void* pw = param(post_w, "post_weight");
  const void* pb = param(post_b, "post_bias");
  const void* qw = param(pre_w, "pre_weight");
  const void* qb = param(pre_b, "pre_bias");
  const int pd = !pt || *pt == at::kFloat ? W4A4_F32 : *pt == at::kHalf ? W4A4_F16 : -1;
  int64_t ldg = C;
  if (gate) {
    if (gate_rows < 1) throw py::value_error("gate_rows must be positive");
    ldg = rows(*gate, "gate", dev, M / gate_rows + (M % gate_rows != 0), C);
  }
  const int gd = gate ? dtype_of(gate->scalar_type()) : W4A4_F32;
  const c10::DeviceGuard guard(ref.device());
  int64_t ldho = C, ldx = C;
  if (h_out) {
    if (h_out->scalar_type() != dt) throw py::type_error("h_out must have h's dtype (y's without h)");
    ldho = rows(*h_out, "h_out", dev, M, C);
  } else if (want_h) {
    h_out = empty(ref, {M, C}, dt);
  }
  int xd = W4A4_F32;
  if (x_out) {
    xd = dtype_of(x_out->scalar_type());
    ldx = rows(*x_out, "x_out", dev, M, C);
  } else if (x_dtype) {
    xd = dtype_of(*x_dtype);
    x_out = empty(ref, {M, C}, *x_dtype);
  }
  check("norm_residual",
        w4a4_norm_residual(h ? h->data_ptr() : nullptr, hd, ldh, y ? y->data_ptr() : nullptr, yd, ldy, post,
                           pw, pb, gate ? gate->data_ptr() : nullptr, gd, ldg, gate_rows,
                           static_cast<float>(residual_scale), pre, qw, qb, pd, static_cast<float>(offset),
                           static_cast<float>(eps), M, C, h_out ? h_out->data_ptr() : nullptr, ldho,
                           x_out ? x_out->data_ptr() : nullptr, xd, ldx, stream_of(dev)));
  return {h_out, x_out};
}

Tensor gated_activation(const Tensor& gate, const OptTensor& up, int act, at::ScalarType out_dtype,
                        OptTensor out) {
  const int64_t dev = device_index(gate);
  if (gate.dim() != 2) throw py::value_error("gate must be a matrix");
  const int64_t M = gate.size(0), F = gate.size(1);
  const int64_t ldg = rows(gate, "gate", dev, M, F);
  const int gd = dtype_of(gate.scalar_type());
  int64_t ldu = F, ldo = F;
  if (up) {
    ldu = rows(*up, "up", dev, M, F);
    if (up->scalar_type() != gate.scalar_type()) throw py::type_error("gate and up must have one dtype");
  }
  const int od = dtype_of(out ? out->scalar_type() : out_dtype);
  const c10::DeviceGuard guard(gate.device());
  if (out)
    ldo = rows(*out, "out", dev, M, F);
  else
    out = empty(gate, {M, F}, out_dtype);
  check("gated_activation",
        w4a4_gated_activation(gate.data_ptr(), ldg, up ? up->data_ptr() : nullptr, ldu, gd, act, M, F,
                              out->data_ptr(), ldo, od, stream_of(dev)));
  return *out;
}

}  // namespace

PYBIND11_MODULE(_block, m) {
  m.def("set_error", [](py::object cls) { g_error = cls.release().ptr(); });
  m.def("adapter_add", &adapter_add);
  m.def("norm_residual", &norm_residual);
  m.def("gated_activation", &gated_activation);
}
