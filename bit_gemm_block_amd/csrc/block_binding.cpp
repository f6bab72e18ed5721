// block_binding.cpp — the Python binding of include/w4a4_block.h and
// include/w4a4_decode.h: checks of the tensors, allocation of the outputs that are
// not given, and the calls on the tensors' current stream.  No arithmetic.  It is
// compiled against torch because a call's host time is what a small call costs:
// through ctypes the marshalling of these argument lists took 5 to 8 us beside the
// launch's 3.
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <string>

#include "w4a4_block.h"
#include "w4a4_decode.h"

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

// ---- operators of a decoding step ---------------------------------------------

// The address of a given contiguous workspace, or of a new one.
void* workspace_of(OptTensor& workspace, const Tensor& like, size_t need, int64_t dev, size_t* bytes) {
  if (workspace) {
    on_device(*workspace, "workspace", dev);
    if (!workspace->is_contiguous()) throw py::value_error("workspace must be contiguous");
  } else if (need > 0) {
    workspace = empty(like, {static_cast<int64_t>(need)}, at::kByte);
  }
  *bytes = workspace ? workspace->nbytes() : 0;
  return workspace ? workspace->data_ptr() : nullptr;
}

Tensor qlinear_w4a16(const Tensor& x, const Tensor& wq, const Tensor& w_scale, int64_t w_group, int layout,
                     at::ScalarType out_dtype, OptTensor out, OptTensor workspace) {
  const int64_t dev = device_index(x);
  if (x.dim() != 2) throw py::value_error("x must be a matrix");
  const int64_t M = x.size(0), K = x.size(1);
  const int64_t ldx = rows(x, "x", dev, M, K);
  const int xd = dtype_of(x.scalar_type()), sd = dtype_of(w_scale.scalar_type());
  if (w_scale.dim() != (w_group > 0 ? 2 : 1))
    throw py::value_error("w_scale must be [N] or, with w_group, [N, K / w_group]");
  const int64_t N = w_scale.size(0);
  if (w_group > 0 && K % w_group != 0) throw py::value_error("w_group must divide K");
  const void* sw = w_group > 0 ? whole(w_scale, "w_scale", dev, w_scale.scalar_type(), {N, K / w_group})
                               : whole(w_scale, "w_scale", dev, w_scale.scalar_type(), {N});
  const int64_t wrows = layout == W4A4_WEIGHTS_ROWMAJOR ? N : (N + 15) / 16 * 16;
  const void* w = whole(wq, "wq", dev, at::kByte, {wrows, K / 2});
  const int od = dtype_of(out ? out->scalar_type() : out_dtype);
  const c10::DeviceGuard guard(x.device());
  int64_t ldo = N;
  if (out)
    ldo = rows(*out, "out", dev, M, N);
  else
    out = empty(x, {M, N}, out_dtype);
  size_t bytes = 0;
  void* ws = workspace_of(workspace, x, w4a16_qlinear_workspace_size(M, N, K), dev, &bytes);
  check("qlinear_w4a16", w4a16_qlinear_forward(x.data_ptr(), xd, ldx, static_cast<const uint8_t*>(w), layout, sw, sd, M,
                                               N, K, w_group, out->data_ptr(), od, ldo, ws, bytes, stream_of(dev)));
  return *out;
}

// The cache that four tensors make.
w4a4_cache cache_of(const Tensor& k, const Tensor& v, const Tensor& k_scale, const Tensor& v_scale, int bits,
                    int64_t dev) {
  if (k.dim() != 4) throw py::value_error("the cache's k must be [pages, heads, page_size, head_dim * bits / 8]");
  if (bits != 4 && bits != 8) throw py::value_error("bits must be 4 or 8");
  w4a4_cache c{};
  c.k = static_cast<uint8_t*>(whole(k, "the cache's k", dev, at::kByte, k.sizes()));
  c.v = static_cast<uint8_t*>(whole(v, "the cache's v", dev, at::kByte, k.sizes()));
  const at::IntArrayRef rows3 = k.sizes().slice(0, 3);
  c.k_scale = static_cast<float*>(whole(k_scale, "the cache's k_scale", dev, at::kFloat, rows3));
  c.v_scale = static_cast<float*>(whole(v_scale, "the cache's v_scale", dev, at::kFloat, rows3));
  c.pages = k.size(0);
  c.heads = k.size(1);
  c.page_size = k.size(2);
  c.head_dim = k.size(3) * 8 / bits;
  c.bits = bits;
  return c;
}

void cache_write(const Tensor& kc, const Tensor& vc, const Tensor& ks, const Tensor& vs, int bits, const Tensor& k,
                 const Tensor& v, const Tensor& slots) {
  const int64_t dev = device_index(kc);
  const w4a4_cache c = cache_of(kc, vc, ks, vs, bits, dev);
  if (k.dim() != 2) throw py::value_error("k and v must be matrices");
  const int64_t T = k.size(0), C = c.heads * c.head_dim;
  const int64_t ldk = rows(k, "k", dev, T, C), ldv = rows(v, "v", dev, T, C);
  if (k.scalar_type() != v.scalar_type()) throw py::type_error("k and v must have one dtype");
  const int dt = dtype_of(k.scalar_type());
  const void* ix = whole(slots, "slots", dev, at::kInt, {T});
  const c10::DeviceGuard guard(kc.device());
  check("cache_write", w4a4_cache_write(&c, k.data_ptr(), ldk, v.data_ptr(), ldv, dt, static_cast<const int32_t*>(ix),
                                        T, stream_of(dev)));
}

std::pair<OptTensor, OptTensor> cache_read(const Tensor& kc, const Tensor& vc, const Tensor& ks, const Tensor& vs,
                                           int bits, const Tensor& slots, at::ScalarType dtype, OptTensor k,
                                           OptTensor v, bool want_k, bool want_v) {
  const int64_t dev = device_index(kc);
  const w4a4_cache c = cache_of(kc, vc, ks, vs, bits, dev);
  if (slots.dim() != 1) throw py::value_error("slots must be a vector");
  const int64_t T = slots.size(0), C = c.heads * c.head_dim;
  const void* ix = whole(slots, "slots", dev, at::kInt, {T});
  const at::ScalarType dt = k ? k->scalar_type() : v ? v->scalar_type() : dtype;
  const int d = dtype_of(dt);
  const c10::DeviceGuard guard(kc.device());
  int64_t ld[2] = {C, C};
  auto take = [&](OptTensor& t, const char* name, bool want, int64_t* l) {
    if (t) {
      if (t->scalar_type() != dt) throw py::type_error("k and v must have one dtype");
      *l = rows(*t, name, dev, T, C);
    } else if (want) {
      t = empty(kc, {T, C}, dt);
    }
  };
  take(k, "k", want_k, &ld[0]);
  take(v, "v", want_v, &ld[1]);
  check("cache_read", w4a4_cache_read(&c, static_cast<const int32_t*>(ix), T, k ? k->data_ptr() : nullptr, ld[0],
                                      v ? v->data_ptr() : nullptr, ld[1], d, stream_of(dev)));
  return {k, v};
}

Tensor cache_attention(const Tensor& q, const Tensor& kc, const Tensor& vc, const Tensor& ks, const Tensor& vs,
                       int bits, const Tensor& tables, const Tensor& lengths, const OptTensor& q_start, int64_t max_q,
                       bool causal, const OptTensor& prefix_table, const OptTensor& prefix_length,
                       std::optional<double> scale, at::ScalarType out_dtype, OptTensor out, OptTensor workspace) {
  const int64_t dev = device_index(kc);
  const w4a4_cache c = cache_of(kc, vc, ks, vs, bits, dev);
  if (q.dim() != 2 || c.head_dim <= 0 || q.size(1) % c.head_dim != 0)
    throw py::value_error("q must be [tokens, heads * head_dim]");
  const int64_t T = q.size(0), C = q.size(1);
  const int64_t ldq = rows(q, "q", dev, T, C);
  const int qd = dtype_of(q.scalar_type());
  if (tables.dim() != 2) throw py::value_error("tables must be [sequences, pages]");
  const int64_t S = tables.size(0), width = tables.size(1);
  const void* tb = whole(tables, "tables", dev, at::kInt, {S, width});
  const void* ln = whole(lengths, "lengths", dev, at::kInt, {S});
  const void* qs = q_start ? whole(*q_start, "q_start", dev, at::kInt, {S + 1}) : nullptr;
  if (!q_start && (max_q != 1 || T < S))
    throw py::value_error("without q_start every sequence has one row of q, and max_q is 1");
  if (prefix_table.has_value() != prefix_length.has_value())
    throw py::value_error("prefix_table and prefix_length go together");
  int64_t P = 0;
  const void *pt = nullptr, *pl = nullptr;
  if (prefix_table) {
    if (prefix_table->dim() != 1) throw py::value_error("prefix_table must be a vector");
    P = prefix_table->size(0);
    pt = whole(*prefix_table, "prefix_table", dev, at::kInt, {P});
    pl = whole(*prefix_length, "prefix_length", dev, at::kInt, {1});
    if (P == 0) pt = pl = nullptr;  // an empty prefix
  }
  const int od = dtype_of(out ? out->scalar_type() : out_dtype);
  const c10::DeviceGuard guard(kc.device());
  int64_t ldo = C;
  if (out)
    ldo = rows(*out, "out", dev, T, C);
  else
    out = empty(q, {T, C}, out_dtype);
  size_t bytes = 0;
  void* ws = workspace_of(workspace, q, w4a4_cache_attention_workspace_size(&c, T, C / c.head_dim, S, width, max_q, P),
                          dev, &bytes);
  const double sc = scale ? *scale : 1.0 / std::sqrt(static_cast<double>(c.head_dim));
  check("cache_attention",
        w4a4_cache_attention(&c, q.data_ptr(), qd, ldq, T, C / c.head_dim, static_cast<const int32_t*>(tb), S, width,
                             static_cast<const int32_t*>(ln), static_cast<const int32_t*>(qs), max_q, causal,
                             static_cast<const int32_t*>(pt), P, static_cast<const int32_t*>(pl),
                             static_cast<float>(sc), out->data_ptr(), od, ldo, ws, bytes, stream_of(dev)));
  return *out;
}

}  // namespace

PYBIND11_MODULE(_block, m) {
  m.def("set_error", [](py::object cls) { g_error = cls.release().ptr(); });
  m.def("adapter_add", &adapter_add);
  m.def("norm_residual", &norm_residual);
  m.def("gated_activation", &gated_activation);
  m.def("qlinear_w4a16", &qlinear_w4a16);
  m.def("cache_write", &cache_write);
  m.def("cache_read", &cache_read);
  m.def("cache_attention", &cache_attention);
}
