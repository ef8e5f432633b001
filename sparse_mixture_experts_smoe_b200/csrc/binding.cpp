// binding.cpp -- the Python side of the routing, query/key norm and paged-cache calls:
// checks of their tensors, outputs and workspaces from torch's allocator on the current
// stream, and the call of the C entry point.  A decode step makes such a call every few
// microseconds, which is what checking fifteen tensors in Python takes: a step's cache
// append took 17 us of the host's time through ctypes.
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "smoe.h"

namespace py = pybind11;
using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

constexpr ScalarType F32 = at::kFloat, BF16 = at::kBFloat16, I32 = at::kInt, U8 = at::kByte;

std::string text(IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

[[noreturn]] void type_error(const std::string& m) { throw py::type_error(m); }
[[noreturn]] void value_error(const std::string& m) { throw py::value_error(m); }

void check(int rc) {
  if (rc == SMOE_OK) return;
  const py::object cls = py::module_::import("sparse_mixture_experts_smoe_b200").attr("SmoeError");
  const py::object e = cls(rc, smoe_last_error());
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

// A CUDA tensor of this type and shape on device dev, any strides.
void expect(const Tensor& t, const char* name, ScalarType dt, IntArrayRef shape, int dev) {
  const std::string n(name);
  if (!t.is_cuda()) type_error(n + " must be a CUDA tensor");
  if (t.scalar_type() != dt) type_error(n + " must be " + at::toString(dt) + ", got " + at::toString(t.scalar_type()));
  if (t.sizes() != shape) value_error(n + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (t.get_device() != dev)
    value_error(n + " is on cuda:" + std::to_string(t.get_device()) + ", not on cuda:" + std::to_string(dev));
}
void* at(const Tensor& t, const char* name, ScalarType dt, IntArrayRef shape, int dev) {
  expect(t, name, dt, shape, dev);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t.data_ptr();
}
template <typename V = void>
V* opt(const OptTensor& t, const char* name, ScalarType dt, IntArrayRef shape, int dev) {
  return t ? (V*)at(*t, name, dt, shape, dev) : nullptr;
}

// A matrix whose rows may lie apart.
struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};
Rows rows_of(const Tensor& t, const char* name, ScalarType dt, int64_t n, int64_t width, int dev) {
  const int64_t shape[2] = {n, width};
  expect(t, name, dt, shape, dev);
  if (width > 1 && t.stride(1) != 1) value_error(std::string(name) + " must have unit stride inside its rows");
  return {t.data_ptr(), n > 1 ? t.stride(0) : width};
}
void matrix(const Tensor& t, const char* name) {
  if (!t.is_cuda() || t.dim() != 2) type_error(std::string(name) + " must be a CUDA tensor of two dimensions");
}
smoe_dtype dtype_of(const Tensor& t) {
  if (t.scalar_type() == BF16) return SMOE_BF16;
  if (t.scalar_type() == F32) return SMOE_F32;
  type_error(std::string("unsupported dtype ") + at::toString(t.scalar_type()));
}
int as_int(int64_t v, const char* name) {
  if (v < 0 || v > 0x7fffffff) value_error(std::string(name) + " is out of range");
  return (int)v;
}

Tensor make(IntArrayRef shape, ScalarType dt, int dev) {
  return at::detail::empty_cuda(shape, dt, at::Device(at::kCUDA, (at::DeviceIndex)dev), std::nullopt);
}
// The given output, checked, or a new one.
void* out(OptTensor& t, const char* name, ScalarType dt, IntArrayRef shape, int dev) {
  if (t) return at(*t, name, dt, shape, dev);
  t = make(shape, dt, dev);
  return t->data_ptr();
}
// Refuses a given output (contiguous) that shares memory with the rows of an input: outputs
// are written while inputs are still read.
void apart(const OptTensor& out, const char* name, const Tensor& in, const char* input) {
  if (!out || out->numel() == 0 || in.numel() == 0) return;
  const bool rows = in.dim() == 2 && in.size(0) > 1;
  const uintptr_t o = (uintptr_t)out->data_ptr(), i = (uintptr_t)in.data_ptr(), oe = o + out->nbytes();
  const uintptr_t step = rows ? (uintptr_t)in.stride(0) * in.element_size() : 0;
  const uintptr_t width = (rows ? in.size(1) : in.numel()) * in.element_size();
  const uintptr_t last = rows ? in.size(0) - 1 : 0;
  if (oe <= i || o >= i + last * step + width) return;
  // the first row that ends behind the output's start
  const uintptr_t r = o < i + width || step == 0 ? 0 : (o - i - width) / step + 1;
  if (i + r * step < oe) value_error(std::string(name) + " must not overlap " + input);
}
void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((at::DeviceIndex)dev).stream(); }
// The device that a call's tensors are on is current while it runs.
struct On {
  int dev;
  c10::cuda::CUDAGuard guard;
  explicit On(const Tensor& t) : dev(t.get_device()), guard((at::DeviceIndex)dev) {}
};

// ---------------------------------------------------------------------------
std::pair<Tensor, Tensor> route_select(const Tensor& logits, const OptTensor& bias, OptTensor idx, OptTensor gates,
                                       int k, int score, bool renorm, float scale, int groups, int top_groups,
                                       int group_top) {
  matrix(logits, "logits");
  const smoe_dtype dt = dtype_of(logits);
  const On on(logits);
  const int64_t T = logits.size(0), E = logits.size(1);
  const Rows x = rows_of(logits, "logits", logits.scalar_type(), T, E, on.dev);
  const float* b = opt<float>(bias, "bias", F32, {E}, on.dev);
  if (k < 1 || k > SMOE_MAX_TOPK)  // refused before outputs of that size are made
    check(smoe_route_select(x.p, as_int(x.ld, "the row stride of logits"), b, as_int(T, "T"), as_int(E, "E"), k, score,
                            renorm, scale, groups, top_groups, group_top, dt, nullptr, nullptr, nullptr));
  const int64_t shape[2] = {T, k};
  apart(idx, "topk_idx", logits, "logits");
  apart(gates, "gates", logits, "logits");
  void* i = out(idx, "topk_idx", I32, shape, on.dev);
  void* g = out(gates, "gates", F32, shape, on.dev);
  check(smoe_route_select(x.p, as_int(x.ld, "the row stride of logits"), b, as_int(T, "T"), as_int(E, "E"), k, score,
                          renorm, scale, groups, top_groups, group_top, dt, (int32_t*)i, (float*)g,
                          stream_of(on.dev)));
  return {*idx, *gates};
}

Tensor route_select_bwd(const Tensor& logits, const Tensor& idx, const Tensor& gates, const Tensor& dgates,
                        OptTensor dlogits, int score, bool renorm, float scale) {
  matrix(logits, "logits");
  matrix(idx, "topk_idx");
  const smoe_dtype dt = dtype_of(logits);
  const On on(logits);
  const int64_t T = logits.size(0), E = logits.size(1), k = idx.size(1);
  const Rows x = rows_of(logits, "logits", logits.scalar_type(), T, E, on.dev);
  const int64_t shape[2] = {T, k}, full[2] = {T, E};
  void* i = at(idx, "topk_idx", I32, shape, on.dev);
  void* g = at(gates, "gates", F32, shape, on.dev);
  void* dg = at(dgates, "dgates", F32, shape, on.dev);
  apart(dlogits, "dlogits", logits, "logits");
  apart(dlogits, "dlogits", idx, "topk_idx");
  apart(dlogits, "dlogits", gates, "gates");
  apart(dlogits, "dlogits", dgates, "dgates");
  void* dl = out(dlogits, "dlogits", logits.scalar_type(), full, on.dev);
  check(smoe_route_select_bwd(x.p, as_int(x.ld, "the row stride of logits"), (int32_t*)i, (float*)g, (float*)dg,
                              as_int(T, "T"), as_int(E, "E"), as_int(k, "k"), score, renorm, scale, dt, dl,
                              stream_of(on.dev)));
  return *dlogits;
}

// ---------------------------------------------------------------------------
struct QkCall {
  int64_t T = 0, dh = 0, wide_q = 0, wide_k = 0;
  ScalarType dt = F32;
  smoe_qk_desc desc{};
};
// Sizes of a call on q rows, k rows or both, from the one that is there.
QkCall qk_call(const OptTensor& q, const OptTensor& k, int kslots, int q_heads, int kv_heads, bool norm,
               bool interleaved, float eps) {
  if (kslots < 1 || q_heads < 1 || kv_heads < 1) value_error("kslots, q_heads and kv_heads must be at least 1");
  if (!q && !k) value_error("q and k are both None");
  const Tensor& ref = k ? *k : *q;
  matrix(ref, k ? "k" : "q");
  QkCall c;
  const int64_t rows = ref.size(0), width = ref.size(1), heads = k ? kv_heads : q_heads;
  if (!k && rows % kslots)
    value_error("q has " + std::to_string(rows) + " rows, not a multiple of kslots = " + std::to_string(kslots));
  if (width % heads)
    value_error("rows of " + std::to_string(width) + " values do not divide into " + std::to_string(heads) + " heads");
  c.T = k ? rows : rows / kslots;
  c.dh = width / heads;
  c.wide_q = q_heads * c.dh;
  c.wide_k = kv_heads * c.dh;
  c.dt = ref.scalar_type();
  c.desc = {as_int(c.T, "T"), kslots, q_heads, kv_heads, as_int(c.dh, "head_dim"), dtype_of(ref), norm, interleaved,
            eps};
  return c;
}

// The same, but for an output that is its input.
void apart_or_same(const OptTensor& out, const char* name, const Tensor& in, const char* input) {
  if (out && out->data_ptr() == in.data_ptr() && in.is_contiguous() && out->nbytes() == in.nbytes()) return;
  apart(out, name, in, input);
}

std::pair<OptTensor, OptTensor> qk_norm_rope_fwd(const OptTensor& q, const OptTensor& k, const OptTensor& slots,
                                                 const OptTensor& positions, const OptTensor& inv_freq,
                                                 const OptTensor& wq, const OptTensor& wk, OptTensor q_out,
                                                 OptTensor k_out, int kslots, int q_heads, int kv_heads, bool norm,
                                                 bool interleaved, float eps) {
  const QkCall c = qk_call(q, k, kslots, q_heads, kv_heads, norm, interleaved, eps);
  const On on(k ? *k : *q);
  if ((!q && q_out) || (!k && k_out)) value_error("an output without its input");
  if (q) apart_or_same(q_out, "q_out", *q, "q");
  if (k) apart_or_same(k_out, "k_out", *k, "k");
  if (q && k) {
    apart(q_out, "q_out", *k, "k");
    apart(k_out, "k_out", *q, "q");
  }
  Rows x, y;
  void *xo = nullptr, *yo = nullptr;
  if (q) {
    const int64_t shape[2] = {c.T * kslots, c.wide_q};
    x = rows_of(*q, "q", c.dt, shape[0], shape[1], on.dev);
    xo = out(q_out, "q_out", c.dt, shape, on.dev);
  }
  if (k) {
    const int64_t shape[2] = {c.T, c.wide_k};
    y = rows_of(*k, "k", c.dt, shape[0], shape[1], on.dev);
    yo = out(k_out, "k_out", c.dt, shape, on.dev);
  }
  check(smoe_moa_qk_norm_rope_fwd(&c.desc, x.p, x.ld, y.p, y.ld,
                                  opt<int32_t>(slots, "sorted_slot", I32, {c.T * kslots}, on.dev),
                                  opt<int32_t>(positions, "positions", I32, {c.T}, on.dev),
                                  opt<float>(inv_freq, "inv_freq", F32, {c.dh / 2}, on.dev),
                                  opt<float>(wq, "wq", F32, {c.dh}, on.dev), opt<float>(wk, "wk", F32, {c.dh}, on.dev),
                                  xo, yo, stream_of(on.dev)));
  return {q_out, k_out};
}

std::tuple<OptTensor, OptTensor, OptTensor, OptTensor> qk_norm_rope_bwd(
    const OptTensor& dq_out, const OptTensor& dk_out, const OptTensor& q, const OptTensor& k, const OptTensor& slots,
    const OptTensor& positions, const OptTensor& inv_freq, const OptTensor& wq, const OptTensor& wk, int kslots,
    int q_heads, int kv_heads, bool norm, bool interleaved, float eps) {
  const QkCall c = qk_call(dq_out, dk_out, kslots, q_heads, kv_heads, norm, interleaved, eps);
  const On on(dk_out ? *dk_out : *dq_out);
  const float* w1 = opt<float>(wq, "wq", F32, {c.dh}, on.dev);
  const float* w2 = opt<float>(wk, "wk", F32, {c.dh}, on.dev);
  OptTensor dq, dk, dwq, dwk;
  Rows dx, dy, x, y;
  void *ox = nullptr, *oy = nullptr, *ow = nullptr, *ov = nullptr;
  const int64_t wide[1] = {c.dh};
  if (dq_out) {
    const int64_t shape[2] = {c.T * kslots, c.wide_q};
    dx = rows_of(*dq_out, "dq_out", c.dt, shape[0], shape[1], on.dev);
    if (norm && !q) value_error("the norm's backward needs q");
    if (norm) x = rows_of(*q, "q", c.dt, shape[0], shape[1], on.dev);
    ox = out(dq, "dq", c.dt, shape, on.dev);
    if (w1) ow = out(dwq, "dwq", F32, wide, on.dev);
  }
  if (dk_out) {
    const int64_t shape[2] = {c.T, c.wide_k};
    dy = rows_of(*dk_out, "dk_out", c.dt, shape[0], shape[1], on.dev);
    if (norm && !k) value_error("the norm's backward needs k");
    if (norm) y = rows_of(*k, "k", c.dt, shape[0], shape[1], on.dev);
    oy = out(dk, "dk", c.dt, shape, on.dev);
    if (w2) ov = out(dwk, "dwk", F32, wide, on.dev);
  }
  OptTensor ws;
  int64_t bytes[1] = {0};
  void* wp = nullptr;
  if (ow || ov) {
    bytes[0] = (int64_t)smoe_moa_qk_norm_rope_bwd_workspace_size(&c.desc);
    wp = out(ws, "workspace", U8, bytes, on.dev);
  }
  check(smoe_moa_qk_norm_rope_bwd(&c.desc, dx.p, dx.ld, dy.p, dy.ld, x.p, x.ld, y.p, y.ld,
                                  opt<int32_t>(slots, "sorted_slot", I32, {c.T * kslots}, on.dev),
                                  opt<int32_t>(positions, "positions", I32, {c.T}, on.dev),
                                  opt<float>(inv_freq, "inv_freq", F32, {c.dh / 2}, on.dev), w1, w2, ox, oy,
                                  (float*)ow, (float*)ov, wp, (size_t)bytes[0], stream_of(on.dev)));
  return {dq, dk, dwq, dwk};
}

// ---------------------------------------------------------------------------
smoe_kv_cache kv_cache(const Tensor& k, const Tensor& v, const Tensor& table, const Tensor& lens, const OptTensor& k_scale,
                       const OptTensor& v_scale, bool written, int dev) {
  if (!k_scale != !v_scale) value_error("k_scale and v_scale go together");
  const ScalarType dt = k_scale ? U8 : BF16;
  const IntArrayRef shape = k.sizes();
  int64_t st[2][3];
  for (int i = 0; i < 2; ++i) {
    const Tensor& t = i ? v : k;
    const char* name = i ? "v_cache" : "k_cache";
    expect(t, name, dt, shape, dev);
    if (shape[3] > 1 && t.stride(3) != 1) value_error(std::string(name) + " must have unit stride inside a head");
    for (int j = 0; j < 3; ++j) {
      st[i][j] = shape[j] > 1 ? t.stride(j) : 0;  // one place: its stride is of no account
      if (written && st[i][j] == 0 && shape[j] > 1)
        value_error(std::string(name) + " is written and must not be an expanded tensor");
    }
  }
  matrix(table, "block_table");
  const int64_t B = table.size(0), pages = table.size(1);
  const Rows tab = rows_of(table, "block_table", I32, B, pages, dev);
  const IntArrayRef scales = shape.slice(0, 3);
  smoe_kv_cache c{};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.k_scale = opt<float>(k_scale, "k_scale", F32, scales, dev);
  c.v_scale = opt<float>(v_scale, "v_scale", F32, scales, dev);
  c.block_table = (const int32_t*)tab.p;
  c.seq_lens = (const int32_t*)at(lens, "seq_lens", I32, {B}, dev);
  c.k_page_stride = st[0][0]; c.k_token_stride = st[0][1]; c.k_head_stride = st[0][2];
  c.v_page_stride = st[1][0]; c.v_token_stride = st[1][1]; c.v_head_stride = st[1][2];
  c.table_stride = tab.ld;
  c.num_pages = as_int(shape[0], "num_pages");
  c.page_size = as_int(shape[1], "page_size");
  c.max_pages = as_int(pages, "max_pages");
  c.B = as_int(B, "B");
  c.kv_heads = as_int(shape[2], "kv_heads");
  c.head_dim = as_int(shape[3], "head_dim");
  return c;
}
void cache_tensor(const Tensor& t) {
  if (!t.is_cuda() || t.dim() != 4)
    type_error("k_cache must be a [num_pages, page_size, kv_heads, head_dim] CUDA tensor");
}

OptTensor cache_append(const OptTensor& q, const Tensor& k, const Tensor& v, const Tensor& k_cache,
                       const Tensor& v_cache, const Tensor& table, const Tensor& lens, const OptTensor& slots,
                       const OptTensor& starts, const OptTensor& inv_freq, const OptTensor& wq, const OptTensor& wk,
                       const OptTensor& k_scale, const OptTensor& v_scale, OptTensor q_out, int kslots, int q_heads,
                       bool norm, bool interleaved, float eps) {
  cache_tensor(k_cache);
  const On on(k_cache);
  const smoe_kv_cache c = kv_cache(k_cache, v_cache, table, lens, k_scale, v_scale, true, on.dev);
  if (c.k == c.v && k_cache.numel() > 0) value_error("k_cache and v_cache must not overlap");
  matrix(k, "k");
  const int64_t T = k.size(0), dh = c.head_dim;
  const Rows y = rows_of(k, "k", BF16, T, c.kv_heads * dh, on.dev);
  const Rows z = rows_of(v, "v", BF16, T, c.kv_heads * dh, on.dev);
  Rows x;
  void* xo = nullptr;
  if (q) {
    const int64_t shape[2] = {T * kslots, q_heads * dh};
    x = rows_of(*q, "q", BF16, shape[0], shape[1], on.dev);
    apart_or_same(q_out, "q_out", *q, "q");
    apart(q_out, "q_out", k, "k");
    apart(q_out, "q_out", v, "v");
    xo = out(q_out, "q_out", BF16, shape, on.dev);
  } else if (q_out) {
    value_error("q_out without q");
  }
  const smoe_qk_desc desc = {as_int(T, "T"), kslots, q_heads, c.kv_heads, c.head_dim, SMOE_BF16, norm, interleaved, eps};
  check(smoe_moa_cache_append(&desc, x.p, x.ld, y.p, y.ld, z.p, z.ld,
                              opt<int32_t>(slots, "sorted_slot", I32, {T * kslots}, on.dev),
                              opt<int32_t>(starts, "starts", I32, {c.B + 1}, on.dev),
                              opt<float>(inv_freq, "inv_freq", F32, {dh / 2}, on.dev),
                              opt<float>(wq, "wq", F32, {dh}, on.dev), opt<float>(wk, "wk", F32, {dh}, on.dev), &c, xo,
                              stream_of(on.dev)));
  return q_out;
}

std::pair<Tensor, Tensor> decode(const Tensor& q, const Tensor& k_cache, const Tensor& v_cache, const Tensor& table,
                                 const Tensor& lens, const OptTensor& slots, const OptTensor& k_scale,
                                 const OptTensor& v_scale, OptTensor o, OptTensor lse, int kslots, int q_heads) {
  cache_tensor(k_cache);
  const On on(k_cache);
  const smoe_kv_cache c = kv_cache(k_cache, v_cache, table, lens, k_scale, v_scale, false, on.dev);
  const int64_t shape[2] = {(int64_t)c.B * kslots, (int64_t)q_heads * c.head_dim}, heads[2] = {shape[0], q_heads};
  const Rows x = rows_of(q, "q", BF16, shape[0], shape[1], on.dev);
  const int32_t* s = opt<int32_t>(slots, "sorted_slot", I32, {shape[0]}, on.dev);
  apart(o, "o", q, "q");
  apart(lse, "lse", q, "q");
  void* op = out(o, "o", BF16, shape, on.dev);
  void* lp = out(lse, "lse", F32, heads, on.dev);
  const int64_t bytes[1] = {
      (int64_t)smoe_moa_decode_workspace_size(c.B, kslots, q_heads, c.kv_heads, c.head_dim)};
  const Tensor ws = make(bytes, U8, on.dev);
  check(smoe_moa_decode(x.p, x.ld, s, kslots, q_heads, &c, op, (float*)lp, ws.data_ptr(), (size_t)bytes[0],
                        stream_of(on.dev)));
  return {*o, *lse};
}

}  // namespace

// torch's own errors (out of memory, a lost device) reach Python as torch's classes.
#define DEF(name) m.def(#name, torch::wrap_pybind_function(name))
PYBIND11_MODULE(_binding, m) {
  DEF(route_select);
  DEF(route_select_bwd);
  DEF(qk_norm_rope_fwd);
  DEF(qk_norm_rope_bwd);
  DEF(cache_append);
  DEF(decode);
}
