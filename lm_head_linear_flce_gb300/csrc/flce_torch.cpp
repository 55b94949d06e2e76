// Python module over the C ABI's operators around the LM head: checks of the
// tensors, their outputs from torch's allocator, the call on torch's current
// stream.  Native because these are the calls of a decode step, where the host
// is the bound: one norm of one row takes 7 us this way, 18 us when the same
// steps are Python (ctypes).  Functions take their arguments by position (None
// where left out) and return tensors, or the C ABI's status when it is not 0;
// head_ops.py wraps them.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/flce.h"

namespace {

using at::Tensor;

constexpr int64_t kGroup = 128;  // columns that share a scale

// A tensor argument, or an undefined tensor for None.
Tensor arg(PyObject* o, const char* name) {
  if (o == Py_None) return Tensor();
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

void check_cuda(const Tensor& t, const char* name, int64_t device = -1) {
  TORCH_CHECK_VALUE(t.defined() && t.is_cuda(), name, " must be a CUDA tensor");
  TORCH_CHECK_VALUE(device < 0 || t.get_device() == device, name, " must be on cuda:", device,
                    ", got ", t.device());
}
void check_type(const Tensor& t, const char* name, at::ScalarType a, at::ScalarType b) {
  TORCH_CHECK_VALUE(t.scalar_type() == a || t.scalar_type() == b, name, " must be ", a,
                    a == b ? "" : " or ", a == b ? "" : at::toString(b), ", got ",
                    t.scalar_type());
}
// bf16 or float32, as the C ABI counts them.
flce_dtype check_float(const Tensor& t, const char* name) {
  check_type(t, name, at::kBFloat16, at::kFloat);
  return t.scalar_type() == at::kFloat ? FLCE_F32 : FLCE_BF16;
}

// t as rows of its last dimension (w elements) a constant distance apart: a
// view wherever the strides allow it.
struct Rows {
  Tensor keep;
  void* p = nullptr;
  int64_t ld = 0;
};
Rows rows(const Tensor& t, int64_t w) {
  Rows r{t, nullptr, w};
  if (!t.defined()) return Rows{};
  if (!t.is_contiguous()) {
    if (t.dim() != 2) r.keep = t.reshape({-1, w});
    const int64_t n = r.keep.size(0);
    if ((w > 1 && r.keep.stride(1) != 1) || (n > 1 && r.keep.stride(0) < w))
      r.keep = r.keep.contiguous();
    if (n > 1) r.ld = r.keep.stride(0);
  }
  r.p = r.keep.data_ptr();
  return r;
}
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// A caller's tensor to be written: autograd would take it for what it was.
void check_writable(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(!(c10::GradMode::is_enabled() && t.requires_grad()), name,
                    " requires a gradient, and the call has none");
}
// Tells autograd that a caller's tensor was written: what saved it for a backward
// then raises instead of using the new values.
void note_written(const Tensor& t) {
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

std::vector<int64_t> lead_and(const Tensor& t, int64_t last) {
  auto s = t.sizes().vec();
  s.back() = last;
  return s;
}
Tensor empty(at::IntArrayRef sizes, const Tensor& like, at::ScalarType type) {
  return at::empty(sizes, like.options().dtype(type));
}

struct OnDevice {
  c10::cuda::CUDAGuard guard;
  flce_stream_t stream;
  explicit OnDevice(const Tensor& t)
      : guard(t.device()),
        stream(reinterpret_cast<flce_stream_t>(
            c10::cuda::getCurrentCUDAStream(t.get_device()).stream())) {}
};

PyObject* wrap(Tensor t) {
  return t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None);
}
template <class... T>
PyObject* answer(flce_status st, T&&... t) {
  if (st != FLCE_OK) return PyLong_FromLong(st);
  PyObject* out = PyTuple_New(sizeof...(t));
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(out, i++, wrap(std::forward<T>(t))), ...);
  return out;
}

void check_count(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// What the norms share.
struct Norm {
  Tensor x, weight, residual, h, out;  // out: residual_out, if it is given
  flce_dtype type, weight_type;
  int64_t N, H;
  Rows xr, rr;

  // `name`: what the caller calls x
  Norm(PyObject* xo, PyObject* wo, PyObject* ro, const char* name = "x")
      : x(arg(xo, name)), weight(arg(wo, "weight")), residual(arg(ro, "residual")) {
    check_cuda(x, name);
    type = check_float(x, name);
    check_cuda(weight, "weight", x.get_device());
    weight_type = check_float(weight, "weight");
    H = x.dim() ? x.size(-1) : 0;
    TORCH_CHECK_VALUE(H > 0 && weight.dim() == 1 && weight.size(0) == H,
                      "expected ", name, " [..., H] and weight [H]");
    if (residual.defined()) {
      check_cuda(residual, "residual", x.get_device());
      check_type(residual, "residual", x.scalar_type(), x.scalar_type());
      TORCH_CHECK_VALUE(residual.sizes() == x.sizes(), "residual must have the shape of x");
    }
    N = x.numel() / H;
    xr = rows(x, H);
    rr = rows(residual, H);
    if (!weight.is_contiguous()) weight = weight.contiguous();
  }
  // Where the norm writes the sum: residual_out, or a new tensor if there is a residual.
  void sum_buffer(PyObject* o) {
    h = out = arg(o, "residual_out");
    if (h.defined()) {
      check_cuda(h, "residual_out", x.get_device());
      check_type(h, "residual_out", x.scalar_type(), x.scalar_type());
      TORCH_CHECK_VALUE(h.sizes() == x.sizes() && h.is_contiguous(),
                        "residual_out must be contiguous, with the shape of x");
      check_writable(h, "residual_out");
    } else if (residual.defined()) {
      h = empty(x.sizes(), x, x.scalar_type());
    }
  }
};

// (x, weight, eps, residual, residual_out) -> (y, h or None, rstd)
PyObject* rms_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 5);
  Norm m(a[0], a[1], a[3]);
  OnDevice on(m.x);
  m.sum_buffer(a[4]);
  Tensor y = empty(m.x.sizes(), m.x, m.x.scalar_type());
  Tensor rstd = empty(m.x.sizes().slice(0, m.x.dim() - 1), m.x, at::kFloat);
  const flce_status st = flce_rms_norm_forward(
      m.xr.p, m.xr.ld, m.rr.p, m.rr.ld, ptr(m.weight), m.N, m.H, static_cast<float>(number(a[2])),
      m.type, m.weight_type, ptr(y), ptr(m.h), static_cast<float*>(ptr(rstd)), on.stream);
  if (st == FLCE_OK) note_written(m.out);
  return answer(st, std::move(y), std::move(m.h), std::move(rstd));
  END_HANDLE_TH_ERRORS
}

// (x, weight, eps, residual, residual_out) -> (q, scale, h or None)
PyObject* rms_norm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 5);
  Norm m(a[0], a[1], a[3]);
  OnDevice on(m.x);
  m.sum_buffer(a[4]);
  Tensor q = empty(m.x.sizes(), m.x, at::kFloat8_e4m3fn);
  Tensor scale = empty(lead_and(m.x, (m.H + kGroup - 1) / kGroup), m.x, at::kFloat);
  const flce_status st = flce_rms_norm_fp8(
      m.xr.p, m.xr.ld, m.rr.p, m.rr.ld, ptr(m.weight), m.N, m.H, static_cast<float>(number(a[2])),
      m.type, m.weight_type, ptr(q), static_cast<float*>(ptr(scale)), ptr(m.h), on.stream);
  if (st == FLCE_OK) note_written(m.out);
  return answer(st, std::move(q), std::move(scale), std::move(m.h));
  END_HANDLE_TH_ERRORS
}

// (dy, h, weight, rstd, dh, need_dx, need_dweight) -> (dx or None, dweight or None)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 7);
  Norm m(a[1], a[2], Py_None, "h");
  const Tensor& h = m.x;
  Tensor dy = arg(a[0], "dy"), dh = arg(a[4], "dh"), rstd = arg(a[3], "rstd");
  const auto like_h = [&](Tensor& t, const char* name) {
    check_cuda(t, name, h.get_device());
    check_type(t, name, h.scalar_type(), h.scalar_type());
    TORCH_CHECK_VALUE(t.sizes() == h.sizes(), name, " must have the shape of h");
    if (!t.is_contiguous()) t = t.contiguous();
  };
  OnDevice on(h);
  like_h(dy, "dy");
  if (dh.defined()) like_h(dh, "dh");
  check_cuda(rstd, "rstd", h.get_device());
  check_type(rstd, "rstd", at::kFloat, at::kFloat);
  TORCH_CHECK_VALUE(rstd.sizes() == h.sizes().slice(0, h.dim() - 1) && rstd.is_contiguous(),
                    "rstd must be as flce_rms_norm returned it");
  Tensor dx, dw, ws;
  size_t nws = 0;
  if (PyObject_IsTrue(a[5])) dx = empty(h.sizes(), h, h.scalar_type());
  if (PyObject_IsTrue(a[6])) {
    dw = empty({m.H}, h, m.weight.scalar_type());
    nws = flce_rms_norm_workspace_size(m.N, m.H);
    ws = empty({static_cast<int64_t>(nws)}, h, at::kByte);
  }
  const flce_status st = flce_rms_norm_backward(
      ptr(dy), ptr(dh), m.xr.p, m.xr.ld, ptr(m.weight), static_cast<const float*>(ptr(rstd)), m.N,
      m.H, m.type, m.weight_type, ptr(dx), ptr(dw), ptr(ws), nws, on.stream);
  return answer(st, std::move(dx), std::move(dw));
  END_HANDLE_TH_ERRORS
}

// (x, block_rows) -> (q, scale)
PyObject* quantize_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 2);
  const Tensor x = arg(a[0], "x");
  const int64_t br = integer(a[1]);
  check_cuda(x, "x");
  const flce_dtype type = check_float(x, "x");
  TORCH_CHECK_VALUE(br == 1 || br == kGroup, "block_rows must be 1 or ", kGroup, ", got ", br);
  TORCH_CHECK_VALUE(x.dim() >= 1 && (br == 1 || x.dim() == 2) && x.size(-1) > 0,
                    "expected x [R, K]");
  const int64_t K = x.size(-1), gk = (K + kGroup - 1) / kGroup;
  OnDevice on(x);
  const Rows r = rows(x, K);
  Tensor q = empty(x.sizes(), x, at::kFloat8_e4m3fn);
  Tensor scale = br == 1 ? empty(lead_and(x, gk), x, at::kFloat)
                         : empty({(x.size(0) + br - 1) / br, gk}, x, at::kFloat);
  const flce_status st =
      flce_quantize_fp8(r.p, r.ld, x.numel() / K, K, type, static_cast<int>(br), ptr(q),
                        static_cast<float*>(ptr(scale)), on.stream);
  return answer(st, std::move(q), std::move(scale));
  END_HANDLE_TH_ERRORS
}

// (a, a_scale, b, b_scale, out type as the C ABI counts it) -> (y,)
PyObject* matmul_fp8(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 5);
  const Tensor a = arg(o[0], "a"), b = arg(o[2], "b");
  Tensor as = arg(o[1], "a_scale"), bs = arg(o[3], "b_scale");
  check_cuda(a, "a");
  check_type(a, "a", at::kFloat8_e4m3fn, at::kFloat8_e4m3fn);
  const int64_t dev = a.get_device();
  check_cuda(b, "b", dev);
  check_type(b, "b", at::kFloat8_e4m3fn, at::kFloat8_e4m3fn);
  check_cuda(as, "a_scale", dev);
  check_type(as, "a_scale", at::kFloat, at::kFloat);
  check_cuda(bs, "b_scale", dev);
  check_type(bs, "b_scale", at::kFloat, at::kFloat);
  TORCH_CHECK_VALUE(a.dim() >= 1 && b.dim() == 2 && a.size(-1) == b.size(1) && b.numel() > 0,
                    "expected a [..., K] and b [V, K]");
  const int64_t V = b.size(0), K = b.size(1), groups = (K + kGroup - 1) / kGroup;
  TORCH_CHECK_VALUE(as.sizes().equals(lead_and(a, groups)),
                    "a_scale must be [..., ceil(K / 128)], one row per row of a");
  TORCH_CHECK_VALUE(bs.dim() == 2 && bs.size(0) == (V + kGroup - 1) / kGroup &&
                        bs.size(1) == groups,
                    "b_scale must be [ceil(V / 128), ceil(K / 128)]");
  OnDevice on(a);
  Rows ar = rows(a, K), br = rows(b, K);
  // the kernels' 16-byte rows; a view that lacks them is copied
  const auto align = [&](Rows& r) {
    if (K % 16 == 0 && ((r.ld | reinterpret_cast<intptr_t>(r.p)) & 15)) {
      r.keep = r.keep.clone(at::MemoryFormat::Contiguous);
      r.p = r.keep.data_ptr();
      r.ld = K;
    }
  };
  align(ar);
  align(br);
  if (!as.is_contiguous()) as = as.contiguous();
  if (!bs.is_contiguous()) bs = bs.contiguous();
  const auto type = static_cast<flce_dtype>(integer(o[4]));
  const int64_t ld = (V + 7) / 8 * 8;
  Tensor y = empty(lead_and(a, ld), a, type == FLCE_F32 ? at::kFloat : at::kBFloat16);
  const flce_status st = flce_matmul_fp8(
      ar.p, ar.ld, static_cast<const float*>(ptr(as)), br.p, br.ld,
      static_cast<const float*>(ptr(bs)), a.numel() / K, V, K, ptr(y), ld, type, on.stream);
  return answer(st, ld == V ? std::move(y) : y.narrow(-1, 0, V));
  END_HANDLE_TH_ERRORS
}

// (logits, tokens, lengths, prompt_lengths, repetition, frequency, presence,
//  bias_ids, bias_values, allowed, out, out type or -1) -> (out,)
PyObject* process_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 12);
  const Tensor z = arg(a[0], "logits");
  check_cuda(z, "logits");
  const flce_dtype type = check_float(z, "logits");
  TORCH_CHECK_VALUE(z.dim() == 2 && z.size(1) > 0, "expected logits [B, V]");
  const int64_t B = z.size(0), V = z.size(1), dev = z.get_device(), want = integer(a[11]);
  OnDevice on(z);
  Tensor out = arg(a[10], "out");
  if (out.defined()) {
    check_cuda(out, "out", dev);
    check_float(out, "out");
    TORCH_CHECK_VALUE(out.dim() == 2 && out.size(0) == B && out.size(1) == V &&
                          (V == 1 || out.stride(1) == 1) && (B <= 1 || out.stride(0) >= V),
                      "out must be [B, V] with contiguous rows");
    TORCH_CHECK_VALUE(want < 0 || (want == FLCE_F32) == (out.scalar_type() == at::kFloat),
                      "out and out_dtype disagree");
    check_writable(out, "out");
  } else {
    out = empty({B, V}, z,
                want < 0 ? z.scalar_type() : want == FLCE_F32 ? at::kFloat : at::kBFloat16);
  }
  const flce_dtype out_type = check_float(out, "out");
  const Rows zr = rows(z, V);
  const auto is_id = [](const Tensor& t, const char* name) {
    check_type(t, name, at::kInt, at::kLong);
    return t.scalar_type() == at::kLong;
  };
  const Tensor tokens = arg(a[1], "tokens");
  Rows tr;
  int64_t L = 0;
  int t64 = 0;
  if (tokens.defined()) {
    check_cuda(tokens, "tokens", dev);
    t64 = is_id(tokens, "tokens");
    TORCH_CHECK_VALUE(tokens.dim() == 2 && tokens.size(0) == B, "tokens must be [B, L]");
    L = tokens.size(1);
    if (L > 0) tr = rows(tokens, L);
  } else {
    TORCH_CHECK_VALUE(a[2] == Py_None && a[3] == Py_None,
                      "lengths and prompt_lengths need tokens");
  }
  Tensor ids = arg(a[7], "bias_ids"), vals = arg(a[8], "bias_values");
  TORCH_CHECK_VALUE(ids.defined() == vals.defined(), "bias_ids and bias_values go together");
  int64_t nb = 0;
  int b64 = 0;
  if (ids.defined()) {
    check_cuda(ids, "bias_ids", dev);
    b64 = is_id(ids, "bias_ids");
    check_cuda(vals, "bias_values", dev);
    check_type(vals, "bias_values", at::kFloat, at::kFloat);
    TORCH_CHECK_VALUE(ids.dim() == 2 && ids.size(0) == B && vals.sizes() == ids.sizes(),
                      "bias_ids and bias_values must be [B, n]");
    nb = ids.size(1);
    if (!ids.is_contiguous()) ids = ids.contiguous();
    if (!vals.is_contiguous()) vals = vals.contiguous();
  }
  const Tensor allowed = arg(a[9], "allowed");
  Rows mr;
  if (allowed.defined()) {
    check_cuda(allowed, "allowed", dev);
    check_type(allowed, "allowed", at::kInt, at::kInt);
    TORCH_CHECK_VALUE(allowed.dim() == 2 && allowed.size(0) == B &&
                          allowed.size(1) >= (V + 31) / 32,
                      "allowed must be [B, ceil(V / 32)]");
    mr = rows(allowed, allowed.size(1));
  }
  const auto per_row = [&](int i, const char* name, at::ScalarType t) {
    Tensor v = arg(a[i], name);
    if (!v.defined()) return v;
    check_cuda(v, name, dev);
    check_type(v, name, t, t);
    TORCH_CHECK_VALUE(v.dim() == 1 && v.size(0) == B, name, " must be [B]");
    return v.is_contiguous() ? v : v.contiguous();
  };
  const Tensor len = per_row(2, "lengths", at::kInt), pl = per_row(3, "prompt_lengths", at::kInt),
               rep = per_row(4, "repetition_penalty", at::kFloat),
               freq = per_row(5, "frequency_penalty", at::kFloat),
               pres = per_row(6, "presence_penalty", at::kFloat);
  const flce_status st = flce_process_logits(
      zr.p, zr.ld, type, B, V, tr.p, tr.ld, t64, L, static_cast<const int32_t*>(ptr(len)),
      static_cast<const int32_t*>(ptr(pl)), static_cast<const float*>(ptr(rep)),
      static_cast<const float*>(ptr(freq)), static_cast<const float*>(ptr(pres)),
      nb ? ptr(ids) : nullptr, b64, nb ? static_cast<const float*>(ptr(vals)) : nullptr, nb,
      static_cast<const int32_t*>(mr.p), mr.ld, ptr(out), B > 1 ? out.stride(0) : V, out_type,
      on.stream);
  if (st == FLCE_OK && a[10] != Py_None) note_written(out);
  return answer(st, std::move(out));
  END_HANDLE_TH_ERRORS
}

#define FLCE_METHOD(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {FLCE_METHOD(rms_norm_forward), FLCE_METHOD(rms_norm_fp8),
                          FLCE_METHOD(rms_norm_backward), FLCE_METHOD(quantize_fp8),
                          FLCE_METHOD(matmul_fp8), FLCE_METHOD(process_logits),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_flce_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__flce_torch() { return PyModule_Create(&kModule); }
