// sequence.cpp -- host side of the sequence operators' binding (module _sequence):
// argument checks, views, results and workspaces, then one call of the C ABI.
//
// A single-token pass runs 3 to 10 us on the GPU.  The same checks and ctypes
// structures in Python took 30 to 60 us a call, so they are compiled: a call costs
// its argument parsing, one or two allocations and the launch.  Checks and messages
// are those of the other entry points: ValueError for shapes, devices, layouts and
// aliasing, TypeError for types, SDMError for what the library refuses.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <optional>
#include <string>
#include <vector>

#include "sdm.h"

namespace py = pybind11;
using at::Tensor;
using OptT = std::optional<Tensor>;

namespace {

std::string shape_str(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += std::to_string(s[i]) + (s.size() == 1 || i + 1 < s.size() ? "," : "") + (i + 1 < s.size() ? " " : "");
  return r + ")";
}
const char* dtype_str(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kLong: return "torch.int64";
    default: return at::toString(t);
  }
}

[[noreturn]] void bad_value(const std::string& m) { throw py::value_error(m); }
[[noreturn]] void bad_type(const std::string& m) { throw py::type_error(m); }

// SDMError for a library status, raised by the package's own check.
void check(int rc) {
  if (rc != SDM_OK) py::module_::import("sparse_memory_linear_scoring_b200.sdm").attr("_check")(rc);
}
[[noreturn]] void workspace_error() {
  py::object e = py::module_::import("sparse_memory_linear_scoring_b200.sdm").attr("SDMError")(
      int(SDM_ERR_WORKSPACE), "workspace too small, not contiguous or on another device");
  PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e.ptr())), e.ptr());
  throw py::error_already_set();
}

void expect(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type) {
  if (t.sizes() != shape)
    bad_value(std::string(name) + " has shape " + shape_str(t.sizes()) + ", expected " + shape_str(shape));
  if (t.scalar_type() != type)
    bad_type(std::string(name) + " has dtype " + dtype_str(t.scalar_type()) + ", expected " + dtype_str(type));
}
void expect(const OptT& t, const char* name, at::IntArrayRef shape, at::ScalarType type) {
  if (t) expect(*t, name, shape, type);
}

void four(const Tensor& t, const char* name, const char* layout) {
  if (t.dim() != 4)
    bad_value(std::string(name) + " must be " + layout + ", got shape " + shape_str(t.sizes()));
}
int in_type(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return SDM_DTYPE_F32;
  if (t.scalar_type() != at::kBFloat16)
    bad_type(std::string(name) + " has dtype " + dtype_str(t.scalar_type()) +
             ", expected torch.float32 or torch.bfloat16");
  return SDM_DTYPE_BF16;
}

int32_t i32(int64_t n, const char* what) {
  if (n < INT32_MIN || n > INT32_MAX) bad_value(std::string(what) + " is out of range");
  return int32_t(n);
}

// The tensors of a call: one device, dense where the library takes no strides.
enum Kind { kView, kDense };
struct Arg {
  const char* name;
  const Tensor* t;
  Kind kind;
};
struct Args {
  Arg a[12];
  int n = 0;
  void add(const char* name, const Tensor& t, Kind k = kView) { a[n++] = {name, &t, k}; }
  void add(const char* name, const OptT& t, Kind k = kDense) {
    if (t) a[n++] = {name, &*t, k};
  }
  c10::Device device() const {
    const c10::Device dev = a[0].t->device();
    for (int i = 0; i < n; ++i) {
      const Tensor& t = *a[i].t;
      if (!t.is_cuda()) bad_value("all tensors must be CUDA tensors (there is no CPU path)");
      if (t.device() != dev) bad_value("all tensors must be on one device");
      if (a[i].kind == kDense) {
        if (!t.is_contiguous()) bad_value(std::string(a[i].name) + " must be contiguous");
      } else if (t.dim() == 4 && t.size(3) > 1 && t.stride(3) != 1) {
        bad_value(std::string("the last axis of ") + a[i].name + " must be dense");
      }
    }
    return dev;
  }
  // The last `outs` arguments must not overlap themselves or any other argument.
  void apart(int outs) const {
    for (int i = n - outs; i < n; ++i) {
      const Tensor& o = *a[i].t;
      if (o.numel() == 0) continue;
      std::pair<int64_t, int64_t> ax[8];
      int m = 0;
      for (int k = 0; k < o.dim() && m < 8; ++k)
        if (o.size(k) > 1) ax[m++] = {o.stride(k), o.size(k)};
      std::sort(ax, ax + m);
      int64_t need = 0;
      for (int k = 0; k < m; ++k) {
        if (ax[k].first <= need) bad_value(std::string("rows of ") + a[i].name + " overlap");
        need += (ax[k].second - 1) * ax[k].first;
      }
      const auto so = span(o);
      for (int j = 0; j < n; ++j) {
        if (j == i || (j >= n - outs && j < i) || a[j].t->numel() == 0) continue;
        const auto st = span(*a[j].t);
        if (so.first < st.second && st.first < so.second)
          bad_value(std::string(a[i].name) + " overlaps " + a[j].name + "; outputs must not alias other tensors");
      }
    }
  }
  static std::pair<uintptr_t, uintptr_t> span(const Tensor& t) {
    int64_t m = 1;
    for (int k = 0; k < t.dim(); ++k) m += (t.size(k) - 1) * t.stride(k);
    const uintptr_t p = reinterpret_cast<uintptr_t>(t.const_data_ptr());
    return {p, p + size_t(m) * t.element_size()};
  }
};

// Device and stream of a call; allocations belong to the device's current stream.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  at::AutoDispatchBelowADInplaceOrView below;
  c10::Device dev;
  void* stream;
  explicit On(c10::Device d) : dev(d) {
    guard.set_device(d);
    stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
  }
  Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  }
  // Empty [B, H, T(, d)], token-major where t is.
  Tensor like(const Tensor& t) const {
    if (t.size(1) > 1 && t.size(2) > 1 && t.stride(2) > t.stride(1)) {
      std::vector<int64_t> s = t.sizes().vec();
      std::swap(s[1], s[2]);
      return empty(s, t.scalar_type()).transpose(1, 2);
    }
    return empty(t.sizes(), t.scalar_type());
  }
  Tensor workspace(size_t need, const OptT& given) const {
    if (!given) return empty({int64_t(need)}, at::kByte);
    if (given->device() != dev || given->nbytes() < need || !given->is_contiguous()) workspace_error();
    return *given;
  }
};

sdm_strides strides(const Tensor& t) {
  // the stride of an axis of one element says nothing and would hide alignment
  auto s = [&](int k) { return t.size(k) > 1 ? t.stride(k) : int64_t(0); };
  return {s(0), s(1), s(2)};
}
const sdm_strides kNone = {0, 0, 0};

const void* ptr(const Tensor& t) { return t.const_data_ptr(); }
const void* ptr(const OptT& t) { return t ? t->const_data_ptr() : nullptr; }
void* out(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }
void* out(const OptT& t) { return t ? t->data_ptr() : nullptr; }
template <typename P> const float* f32(const P& t) { return static_cast<const float*>(ptr(t)); }
template <typename P> float* f32_out(const P& t) { return static_cast<float*>(out(t)); }
const int32_t* lens(const OptT& t) { return static_cast<const int32_t*>(ptr(t)); }

// ---------------------------------------------------------------- convolution
sdm_conv_dims conv_dims(const Tensor& x, const Tensor& w, const OptT& bias, bool silu) {
  four(x, "x", "[B, H, T, d]");
  const int type = in_type(x, "x");
  if (w.dim() != 3) bad_value("w must be [H, d, K], got shape " + shape_str(w.sizes()));
  const int64_t H = x.size(1), d = x.size(3), K = w.size(2);
  expect(w, "w", {H, d, K}, x.scalar_type());
  expect(bias, "bias", {H, d}, x.scalar_type());
  return {i32(x.size(0), "B"), i32(H, "H"), i32(x.size(2), "T"), i32(d, "d"), i32(K, "K"), silu ? 1 : 0, type};
}

Tensor conv_forward(const Tensor& x, const Tensor& w, const OptT& bias, const OptT& state, bool silu,
                    const OptT& lengths, const OptT& y_) {
  const sdm_conv_dims d = conv_dims(x, w, bias, silu);
  const int64_t K1 = std::max(d.K - 1, 0);
  expect(state, "state", {d.B, d.H, K1, d.d}, x.scalar_type());
  expect(lengths, "lengths", {d.B}, at::kInt);
  expect(y_, "y", x.sizes(), x.scalar_type());
  Args a;
  a.add("x", x);
  a.add("w", w, kDense);
  a.add("bias", bias);
  a.add("lengths", lengths);
  a.add("state", state);
  a.add("y", y_, kView);
  const c10::Device dev = a.device();
  a.apart((state ? 1 : 0) + (y_ ? 1 : 0));
  On on(dev);
  const Tensor y = y_ ? *y_ : on.like(x);
  const sdm_strides sx = strides(x), sy = strides(y);
  check(sdm_conv_forward(ptr(x), ptr(w), ptr(bias), out(state), lens(lengths), out(y), &d, &sx, &sy, on.stream));
  return y;
}

py::dict conv_backward(const Tensor& x, const Tensor& w, const Tensor& dy, const OptT& bias,
                       const OptT& state0, const OptT& dstate, bool silu, const OptT& workspace) {
  const sdm_conv_dims d = conv_dims(x, w, bias, silu);
  const int64_t K1 = std::max(d.K - 1, 0);
  expect(dy, "dy", x.sizes(), x.scalar_type());
  expect(state0, "state0", {d.B, d.H, K1, d.d}, x.scalar_type());
  expect(dstate, "dstate", {d.B, d.H, K1, d.d}, at::kFloat);
  Args a;
  a.add("x", x);
  a.add("w", w, kDense);
  a.add("dy", dy);
  a.add("bias", bias);
  a.add("state0", state0);
  a.add("dstate", dstate);
  const c10::Device dev = a.device();
  const size_t need = sdm_conv_backward_workspace_bytes(&d);
  if (need == 0 || d.T == 0)  // the library says why
    check(sdm_conv_backward(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                            nullptr, &d, nullptr, nullptr, nullptr, nullptr, 0, nullptr));
  On on(dev);
  const Tensor dx = on.like(x), dw = on.empty({d.H, d.d, d.K}, at::kFloat);
  OptT db, ds;
  if (bias) db = on.empty({d.H, d.d}, at::kFloat);
  if (state0 || dstate) ds = on.empty({d.B, d.H, K1, d.d}, at::kFloat);
  const Tensor ws = on.workspace(need, workspace);
  const sdm_strides sx = strides(x), sdy = strides(dy), sdx = strides(dx);
  check(sdm_conv_backward(ptr(x), ptr(w), ptr(bias), ptr(state0), ptr(dy), f32(dstate), out(dx), f32_out(dw),
                          f32_out(db), f32_out(ds), &d, &sx, &sdy, &sdx, out(ws), ws.nbytes(), on.stream));
  py::dict g;
  g["x"] = dx;
  g["w"] = dw;
  if (db) g["bias"] = *db;
  if (ds) g["state"] = *ds;
  return g;
}

// ---------------------------------------------------------------- selective scan
sdm_ssm_dims ssm_dims(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& Bm,
                      const Tensor& Cm, const OptT& D) {
  four(x, "x", "[B, H, T, d_v]");
  const int type = in_type(x, "x");
  four(Bm, "Bm", "[B, G, T, d_k]");
  const int64_t B = x.size(0), H = x.size(1), T = x.size(2), P = x.size(3), G = Bm.size(1), N = Bm.size(3);
  expect(Bm, "Bm", {B, G, T, N}, x.scalar_type());
  expect(Cm, "Cm", {B, G, T, N}, x.scalar_type());
  expect(dt, "dt", {B, H, T}, at::kFloat);
  expect(A, "A", {H}, at::kFloat);
  expect(D, "D", {H}, at::kFloat);
  return {i32(B, "B"), i32(H, "H"), i32(G, "G"), i32(T, "T"), i32(N, "d_k"), i32(P, "d_v"), type};
}

Tensor ssm_forward(bool step, const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& Bm,
                   const Tensor& Cm, const Tensor& S, const OptT& D, const OptT& lengths, const OptT& y_,
                   const OptT& workspace) {
  const sdm_ssm_dims d = ssm_dims(x, dt, A, Bm, Cm, D);
  expect(S, "S", {d.B, d.H, d.d_v, d.d_k}, at::kFloat);
  expect(lengths, "lengths", {d.B}, at::kInt);
  expect(y_, "y", x.sizes(), x.scalar_type());
  Args a;
  a.add("x", x);
  a.add("dt", dt);
  a.add("A", A, kDense);
  a.add("Bm", Bm);
  a.add("Cm", Cm);
  a.add("D", D);
  a.add("lengths", lengths);
  a.add("S", S, kDense);
  a.add("y", y_, kView);
  const c10::Device dev = a.device();
  a.apart(y_ ? 2 : 1);
  On on(dev);
  const Tensor y = y_ ? *y_ : on.like(x);
  const sdm_ssm_views v = {strides(x), strides(dt), strides(Bm), strides(Cm), strides(y)};
  if (step) {
    check(sdm_ssm_step(ptr(x), f32(dt), f32(A), ptr(Bm), ptr(Cm), f32(D), f32_out(S), out(y), &d, &v, on.stream));
    return y;
  }
  const Tensor ws = on.workspace(sdm_ssm_workspace_bytes(&d), workspace);
  check(sdm_ssm_forward(ptr(x), f32(dt), f32(A), ptr(Bm), ptr(Cm), f32(D), f32_out(S), lens(lengths), out(y), &d,
                        &v, out(ws), ws.nbytes(), on.stream));
  return y;
}

py::dict ssm_backward(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& Bm, const Tensor& Cm,
                      const OptT& S0, const Tensor& dy, const OptT& dST, const OptT& D, const OptT& workspace) {
  const sdm_ssm_dims d = ssm_dims(x, dt, A, Bm, Cm, D);
  expect(dy, "dy", x.sizes(), x.scalar_type());
  expect(S0, "S0", {d.B, d.H, d.d_v, d.d_k}, at::kFloat);
  expect(dST, "dS_T", {d.B, d.H, d.d_v, d.d_k}, at::kFloat);
  Args a;
  a.add("x", x);
  a.add("dt", dt);
  a.add("A", A, kDense);
  a.add("Bm", Bm);
  a.add("Cm", Cm);
  a.add("S0", S0);
  a.add("dy", dy);
  a.add("dS_T", dST);
  a.add("D", D);
  const c10::Device dev = a.device();
  const size_t need = sdm_ssm_backward_workspace_bytes(&d);
  if (need == 0 || d.T == 0)  // the library says why
    check(sdm_ssm_backward(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                           nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, &d, nullptr, nullptr,
                           nullptr, 0, nullptr));
  On on(dev);
  const Tensor dx = on.like(x), ddt = on.like(dt), dA = on.empty({d.H}, at::kFloat), dB = on.like(Bm),
               dC = on.like(Cm), dS0 = on.empty({d.B, d.H, d.d_v, d.d_k}, at::kFloat);
  OptT dD;
  if (D) dD = on.empty({d.H}, at::kFloat);
  const Tensor ws = on.workspace(need, workspace);
  const sdm_ssm_views v = {strides(x), strides(dt), strides(Bm), strides(Cm), strides(dy)};
  const sdm_ssm_views gv = {strides(dx), strides(ddt), strides(dB), strides(dC), strides(dx)};
  check(sdm_ssm_backward(ptr(x), f32(dt), f32(A), ptr(Bm), ptr(Cm), f32(D), f32(S0), ptr(dy), f32(dST), out(dx),
                         f32_out(ddt), f32_out(dA), out(dB), out(dC), f32_out(dD), f32_out(dS0), &d, &v, &gv,
                         out(ws), ws.nbytes(), on.stream));
  py::dict g;
  g["x"] = dx;
  g["dt"] = ddt;
  g["A"] = dA;
  g["Bm"] = dB;
  g["Cm"] = dC;
  g["S0"] = dS0;
  if (dD) g["D"] = *dD;
  return g;
}

// ---------------------------------------------------------------- block attention
Tensor block_pool(const Tensor& k, const OptT& kc_, int64_t block, int64_t first) {
  four(k, "k", "[B, G, Tk, d]");
  const int type = in_type(k, "k");
  const int64_t B = k.size(0), G = k.size(1), Tk = k.size(2), d = k.size(3);
  const int64_t n = block > 0 ? Tk / block : 0;
  if (kc_) {
    if (kc_->dim() != 4 || kc_->size(2) < n)
      bad_value("kc must be [B, G, n >= " + std::to_string(n) + ", d], got shape " + shape_str(kc_->sizes()));
    expect(*kc_, "kc", {B, G, kc_->size(2), d}, k.scalar_type());
  } else if (first) {
    bad_value("first needs the kc that holds the blocks before it");
  }
  Args a;
  a.add("k", k);
  a.add("kc", kc_, kView);
  const c10::Device dev = a.device();
  a.apart(kc_ ? 1 : 0);
  const sdm_block_dims dims = {i32(B, "B"), i32(G, "G"), i32(G, "G"), 0, i32(Tk, "Tk"), i32(d, "d"),
                               i32(block, "block"), 1, type, 1.f};
  On on(dev);
  const Tensor kc = kc_ ? *kc_ : on.empty({B, G, n, d}, k.scalar_type());
  const sdm_block_views v = {kNone, strides(k), kNone, kNone, strides(kc)};
  check(sdm_block_pool(ptr(k), out(kc), i32(first, "first"), &dims, &v, on.stream));
  return kc;
}

Tensor block_select(const Tensor& q, const Tensor& kc, int64_t n_sel, int64_t block, std::optional<int64_t> Tk,
                    const OptT& lengths) {
  four(q, "q", "[B, H, Tq, d]");
  const int type = in_type(q, "q");
  four(kc, "kc", "[B, G, n, d]");
  const int64_t B = q.size(0), H = q.size(1), Tq = q.size(2), d = q.size(3), G = kc.size(1), n = kc.size(2);
  expect(kc, "kc", {B, G, n, d}, q.scalar_type());
  expect(lengths, "lengths", {B}, at::kInt);
  Args a;
  a.add("q", q);
  a.add("kc", kc);
  a.add("lengths", lengths);
  const c10::Device dev = a.device();
  const sdm_block_dims dims = {i32(B, "B"), i32(H, "H"), i32(G, "G"), i32(Tq, "Tq"),
                               i32(Tk ? *Tk : Tq, "Tk"), i32(d, "d"), i32(block, "block"), i32(n_sel, "n_sel"),
                               type, 1.f};
  On on(dev);
  const Tensor idx = on.empty({B, G, Tq, std::max<int64_t>(std::min<int64_t>(n_sel, 64), 0)}, at::kInt);
  const sdm_block_views v = {strides(q), kNone, kNone, kNone, strides(kc)};
  check(sdm_block_select(ptr(q), ptr(kc), i32(n, "n"), lens(lengths), static_cast<int32_t*>(out(idx)), &dims, &v,
                         on.stream));
  return idx;
}

sdm_block_dims block_dims(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& idx, int64_t block,
                          std::optional<double> scale, const OptT& lengths) {
  four(q, "q", "[B, H, Tq, d]");
  const int type = in_type(q, "q");
  four(k, "k", "[B, G, Tk, d]");
  const int64_t B = q.size(0), H = q.size(1), Tq = q.size(2), d = q.size(3), G = k.size(1), Tk = k.size(2);
  expect(k, "k", {B, G, Tk, d}, q.scalar_type());
  expect(v, "v", {B, G, Tk, d}, q.scalar_type());
  four(idx, "idx", "[B, G, Tq, n_sel]");
  expect(idx, "idx", {B, G, Tq, idx.size(3)}, at::kInt);
  expect(lengths, "lengths", {B}, at::kInt);
  return {i32(B, "B"), i32(H, "H"), i32(G, "G"), i32(Tq, "Tq"), i32(Tk, "Tk"), i32(d, "d"), i32(block, "block"),
          i32(idx.size(3), "n_sel"), type, scale ? float(*scale) : float(1.0 / std::sqrt(double(d)))};
}

py::object block_forward(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& idx, int64_t block,
                         std::optional<double> scale, const OptT& lengths, const OptT& o_, bool return_lse,
                         const OptT& workspace) {
  const sdm_block_dims dims = block_dims(q, k, v, idx, block, scale, lengths);
  expect(o_, "o", q.sizes(), q.scalar_type());
  Args a;
  a.add("q", q);
  a.add("k", k);
  a.add("v", v);
  a.add("idx", idx, kDense);
  a.add("lengths", lengths);
  a.add("o", o_, kView);
  const c10::Device dev = a.device();
  a.apart(o_ ? 1 : 0);
  On on(dev);
  const Tensor o = o_ ? *o_ : on.like(q);
  OptT lse;
  if (return_lse) lse = on.empty({q.size(0), q.size(1), q.size(2)}, at::kFloat);
  const sdm_block_views vw = {strides(q), strides(k), strides(v), strides(o), kNone};
  const Tensor ws = on.workspace(sdm_block_workspace_bytes(&dims), workspace);
  check(sdm_block_forward(ptr(q), ptr(k), ptr(v), static_cast<const int32_t*>(ptr(idx)), lens(lengths), out(o),
                          f32_out(lse), &dims, &vw, out(ws), ws.nbytes(), on.stream));
  if (return_lse) return py::make_tuple(o, *lse);
  return py::cast(o);
}

py::dict block_backward(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& idx, const Tensor& o,
                        const Tensor& lse, const Tensor& d_o, int64_t block, std::optional<double> scale,
                        const OptT& lengths, const OptT& workspace) {
  const sdm_block_dims dims = block_dims(q, k, v, idx, block, scale, lengths);
  expect(o, "o", q.sizes(), q.scalar_type());
  expect(d_o, "d_o", q.sizes(), q.scalar_type());
  expect(lse, "lse", {q.size(0), q.size(1), q.size(2)}, at::kFloat);
  Args a;
  a.add("q", q);
  a.add("k", k);
  a.add("v", v);
  a.add("idx", idx, kDense);
  a.add("o", o);
  a.add("lse", lse, kDense);
  a.add("d_o", d_o);
  a.add("lengths", lengths);
  const c10::Device dev = a.device();
  On on(dev);
  const Tensor dq = on.like(q), dk = on.like(k), dv = on.like(v);
  const Tensor ws = on.workspace(sdm_block_backward_workspace_bytes(&dims), workspace);
  const sdm_block_views vw = {strides(q), strides(k), strides(v), strides(o), kNone};
  const sdm_block_views gv = {strides(dq), strides(dk), strides(dv), strides(d_o), kNone};
  check(sdm_block_backward(ptr(q), ptr(k), ptr(v), static_cast<const int32_t*>(ptr(idx)), lens(lengths), ptr(o),
                           f32(lse), ptr(d_o), out(dq), out(dk), out(dv), &dims, &vw, &gv, out(ws), ws.nbytes(),
                           on.stream));
  py::dict g;
  g["q"] = dq;
  g["k"] = dk;
  g["v"] = dv;
  return g;
}

size_t ssm_workspace_bytes(int32_t B, int32_t H, int32_t G, int32_t T, int32_t d_k, int32_t d_v, int32_t type) {
  const sdm_ssm_dims d = {B, H, G, T, d_k, d_v, type};
  return sdm_ssm_workspace_bytes(&d);
}

}  // namespace

PYBIND11_MODULE(_sequence, m) {
  m.def("conv_forward", &conv_forward);
  m.def("conv_backward", &conv_backward);
  m.def("ssm_forward", &ssm_forward);
  m.def("ssm_backward", &ssm_backward);
  m.def("ssm_workspace_bytes", &ssm_workspace_bytes);
  m.def("block_pool", &block_pool);
  m.def("block_select", &block_select);
  m.def("block_forward", &block_forward);
  m.def("block_backward", &block_backward);
}
