// binding.cpp -- the serving and training calls around the prefill, from torch tensors to
// the C ABI of libmoba (include/moba.h).
//
// It checks the tensors, allocates what the caller has not given, and passes pointers,
// strides and the current stream on, as the Python wrappers of the prefill do.  It is
// compiled because these calls are short: a decode step's append runs 6 us on the GPU, and
// the same checks in Python take 25 us.
#include <ATen/cuda/CUDAContext.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/extension.h>

#include <optional>
#include <string>
#include <tuple>

#include "moba.h"

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;
using Shape = std::vector<int64_t>;

namespace {

std::string show(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

std::string dtype_name(at::ScalarType t) {
  return "torch." + std::string(t == at::kBFloat16 ? "bfloat16" : t == at::kFloat ? "float32" : t == at::kInt ? "int32"
                                                                                                    : at::toString(t));
}

// One call's checks: every tensor on one CUDA device, of its type, shape and layout.
class Checks {
 public:
  explicit Checks(const char *fn) : fn_(fn) {}

  void rank(const char *name, const Tensor &t, int64_t n) const {
    if (t.dim() != n) fail(std::string(name) + " has " + std::to_string(t.dim()) + " dimensions, expected " + std::to_string(n));
    for (int64_t i = 0; i < n; ++i)   // (the C ABI counts in int; an expanded tensor can be longer)
      if (t.size(i) >= (int64_t(1) << 31)) fail(std::string(name) + " has shape " + show(t.sizes()) + ", beyond 32 bits");
  }

  // dt: the type, or at::ScalarType::Undefined for any.  shape null: any.
  void tensor(const char *name, const Tensor &t, at::ScalarType dt, bool contiguous, const Shape *shape = nullptr) {
    if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
    if (dt != at::ScalarType::Undefined && t.scalar_type() != dt)
      fail(std::string(name) + " must be " + dtype_name(dt) + ", not " + dtype_name(t.scalar_type()));
    if (contiguous && !t.is_contiguous()) fail(std::string(name) + " must be contiguous");
    if (shape && t.sizes() != at::IntArrayRef(*shape))
      fail(std::string(name) + " has shape " + show(t.sizes()) + ", expected " + show(*shape));
    const int i = t.get_device();
    if (dev_ < 0) dev_ = i;
    else if (i != dev_)
      fail("every tensor must be on cuda:" + std::to_string(dev_) + "; " + name + " is on cuda:" + std::to_string(i));
  }
  void tensor(const char *name, const MaybeTensor &t, at::ScalarType dt, bool contiguous, const Shape *shape = nullptr) {
    if (t) tensor(name, *t, dt, contiguous, shape);
  }

  moba_weight weight(const char *name, const MaybeTensor &t, int64_t d) {
    if (!t) return moba_weight{nullptr, 0};
    if (t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kFloat)
      fail(std::string(name) + " must be torch.bfloat16 or torch.float32, not " + dtype_name(t->scalar_type()));
    const Shape s{d};
    tensor(name, *t, at::ScalarType::Undefined, true, &s);
    return moba_weight{t->data_ptr(), t->scalar_type() == at::kFloat ? 1 : 0};
  }

  [[noreturn]] void fail(const std::string &what) const { throw py::value_error(std::string(fn_) + ": " + what); }
  int device() const { return dev_; }

 private:
  const char *fn_;
  int dev_ = -1;
};

// [batch, heads, N, d] (or, of three dimensions, with the strides named).
moba_tensor view4(const Checks &c, const Tensor &t) {
  if (t.stride(3) != 1) c.fail("the head dimension must be contiguous");
  return moba_tensor{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}
moba_tensor tokens(const Checks &c, const Tensor &t) {   // [tokens, heads, d]
  if (t.stride(2) != 1) c.fail("the head dimension must be contiguous");
  return moba_tensor{t.data_ptr(), 0, t.stride(1), t.stride(0)};
}
moba_tensor rows(const Checks &c, const Tensor &t) {     // [sequences, heads, d]
  if (t.stride(2) != 1) c.fail("the head dimension must be contiguous");
  return moba_tensor{t.data_ptr(), t.stride(0), t.stride(1), 0};
}
constexpr moba_tensor kNone{nullptr, 0, 0, 0};

Tensor make(at::IntArrayRef shape, at::ScalarType dt, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(dt).device(at::kCUDA, dev));
}
Tensor given(const MaybeTensor &t, at::IntArrayRef shape, at::ScalarType dt, int dev) {
  return t ? *t : make(shape, dt, dev);
}
size_t bytes(const Tensor &t) { return (size_t)t.numel() * t.element_size(); }
template <class T>
T *ptr(const MaybeTensor &t) {
  return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}
void *stream_of(int dev) { return at::cuda::getCurrentCUDAStream(dev).stream(); }

const auto kBF16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kAny = at::ScalarType::Undefined;

using Two = std::tuple<int, Tensor, Tensor>;

Two swa_fwd(const Tensor &q, const Tensor &k, const Tensor &v, int window, int sink, float scale,
            const MaybeTensor &out_, const MaybeTensor &lse_) {
  Checks c("swa_attn_fwd");
  c.rank("q", q, 4);
  c.rank("k", k, 4);
  const int64_t b = q.size(0), hq = q.size(1), N = q.size(2), d = q.size(3);
  const Shape ks{b, k.size(1), k.size(2), d}, os{b, hq, N, d}, ls{b, hq, N};
  c.tensor("q", q, kBF16, false);
  c.tensor("k", k, kBF16, false, &ks);
  c.tensor("v", v, kBF16, false, &ks);
  c.tensor("out", out_, kBF16, false, &os);
  c.tensor("lse", lse_, kF32, true, &ls);
  const c10::cuda::CUDAGuard guard(c.device());
  Tensor out = out_ ? *out_ : at::empty_like(q), lse = given(lse_, ls, kF32, c.device());
  const int rc = swa_sink_attn_fwd(view4(c, q), view4(c, k), view4(c, v), b, hq, k.size(1), N, k.size(2), d, window,
                                   sink, scale, view4(c, out), lse.data_ptr<float>(), stream_of(c.device()));
  return {rc, out, lse};
}

std::tuple<int, Tensor, Tensor, Tensor> swa_bwd(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &out,
                                                const Tensor &lse, const Tensor &dout, int window, int sink, float scale,
                                                const MaybeTensor &dq_, const MaybeTensor &dk_, const MaybeTensor &dv_,
                                                const MaybeTensor &workspace_) {
  Checks c("swa_attn_bwd");
  c.rank("q", q, 4);
  c.rank("k", k, 4);
  const int64_t b = q.size(0), hq = q.size(1), N = q.size(2), d = q.size(3), hkv = k.size(1);
  const Shape qs{b, hq, N, d}, ks{b, hkv, N, d}, ls{b, hq, N};
  c.tensor("q", q, kBF16, false);
  c.tensor("k", k, kBF16, false, &ks);
  c.tensor("v", v, kBF16, false, &ks);
  c.tensor("out", out, kBF16, false, &qs);
  c.tensor("lse", lse, kF32, true, &ls);
  c.tensor("dout", dout, kBF16, false, &qs);
  c.tensor("dq", dq_, kBF16, false, &qs);
  c.tensor("dk", dk_, kBF16, false, &ks);
  c.tensor("dv", dv_, kBF16, false, &ks);
  c.tensor("workspace", workspace_, kAny, true);
  const int dev = c.device();
  const c10::cuda::CUDAGuard guard(dev);
  Tensor dq = given(dq_, qs, kBF16, dev), dk = given(dk_, ks, kBF16, dev), dv = given(dv_, ks, kBF16, dev), ws;
  if (workspace_) {
    ws = *workspace_;
  } else {
    size_t n = 0;
    const int rc = swa_bwd_workspace_size(b, hq, hkv, N, d, window, sink, &n);
    if (rc) return {rc, dq, dk, dv};
    ws = make({(int64_t)n}, at::kByte, dev);
  }
  const int rc = swa_attn_bwd(view4(c, q), view4(c, k), view4(c, v), view4(c, out), view4(c, dout), lse.data_ptr<float>(),
                              b, hq, hkv, N, d, window, sink, scale, view4(c, dq), view4(c, dk), view4(c, dv),
                              ws.data_ptr(), bytes(ws), stream_of(dev));
  return {rc, dq, dk, dv};
}

// The checks of the angle tables; returns (rot, positions).
std::pair<int, int> angles(Checks &c, const Tensor &cos, const Tensor &sin) {
  c.rank("cos", cos, 2);
  const Shape s{cos.size(0), cos.size(1)};
  c.tensor("cos", cos, kF32, true);
  c.tensor("sin", sin, kF32, true, &s);
  return {(int)(2 * cos.size(1)), (int)cos.size(0)};
}

Two rope_fwd(const Tensor &q, const Tensor &k, const Tensor &cos, const Tensor &sin, const MaybeTensor &positions,
             const MaybeTensor &q_weight, const MaybeTensor &k_weight, float eps, bool interleaved,
             const MaybeTensor &q_out, const MaybeTensor &k_out) {
  Checks c("qk_norm_rope_fwd");
  c.rank("q", q, 4);
  c.rank("k", k, 4);
  const int64_t b = q.size(0), hq = q.size(1), N = q.size(2), d = q.size(3), hkv = k.size(1);
  const Shape qs{b, hq, N, d}, ks{b, hkv, N, d}, ps{b, N};
  c.tensor("q", q, kBF16, false);
  c.tensor("k", k, kBF16, false, &ks);
  const auto [rot, max_pos] = angles(c, cos, sin);
  c.tensor("positions", positions, kI32, true, &ps);
  const moba_weight wq = c.weight("q_weight", q_weight, d), wk = c.weight("k_weight", k_weight, d);
  c.tensor("q_out", q_out, kBF16, false, &qs);
  c.tensor("k_out", k_out, kBF16, false, &ks);
  const int dev = c.device();
  const c10::cuda::CUDAGuard guard(dev);
  Tensor qo = given(q_out, qs, kBF16, dev), ko = given(k_out, ks, kBF16, dev);
  const int rc = qk_norm_rope_fwd(view4(c, q), view4(c, k), cos.data_ptr<float>(), sin.data_ptr<float>(),
                                  ptr<int32_t>(positions), wq, wk, b, hq, hkv, N, d, rot, max_pos, interleaved, eps,
                                  view4(c, qo), view4(c, ko), stream_of(dev));
  return {rc, qo, ko};
}

std::tuple<int, Tensor, Tensor, MaybeTensor, MaybeTensor> rope_bwd(
    const Tensor &dq_out, const Tensor &dk_out, const Tensor &q, const Tensor &k, const Tensor &cos, const Tensor &sin,
    const MaybeTensor &positions, const MaybeTensor &q_weight, const MaybeTensor &k_weight, float eps, bool interleaved,
    const MaybeTensor &dq_, const MaybeTensor &dk_, const MaybeTensor &workspace_) {
  Checks c("qk_norm_rope_bwd");
  c.rank("dq_out", dq_out, 4);
  c.rank("dk_out", dk_out, 4);
  const int64_t b = dq_out.size(0), hq = dq_out.size(1), N = dq_out.size(2), d = dq_out.size(3), hkv = dk_out.size(1);
  const Shape qs{b, hq, N, d}, ks{b, hkv, N, d}, ps{b, N};
  c.tensor("dq_out", dq_out, kBF16, false);
  c.tensor("dk_out", dk_out, kBF16, false, &ks);
  c.tensor("q", q, kBF16, false, &qs);
  c.tensor("k", k, kBF16, false, &ks);
  const auto [rot, max_pos] = angles(c, cos, sin);
  c.tensor("positions", positions, kI32, true, &ps);
  const moba_weight wq = c.weight("q_weight", q_weight, d), wk = c.weight("k_weight", k_weight, d);
  c.tensor("dq", dq_, kBF16, false, &qs);
  c.tensor("dk", dk_, kBF16, false, &ks);
  c.tensor("workspace", workspace_, kAny, true);
  const int dev = c.device();
  const c10::cuda::CUDAGuard guard(dev);
  Tensor dq = given(dq_, qs, kBF16, dev), dk = given(dk_, ks, kBF16, dev);
  MaybeTensor dqw, dkw, ws = workspace_;
  if (wq.ptr) dqw = make({d}, kF32, dev);
  if (wk.ptr) dkw = make({d}, kF32, dev);
  if (!ws && (wq.ptr || wk.ptr)) {
    size_t n = 0;
    const int rc = qk_norm_rope_bwd_workspace_size(b, hq, hkv, N, d, &n);
    if (rc) return {rc, dq, dk, dqw, dkw};
    ws = make({(int64_t)n}, at::kByte, dev);
  }
  const int rc = qk_norm_rope_bwd(view4(c, dq_out), view4(c, dk_out), view4(c, q), view4(c, k), cos.data_ptr<float>(),
                                  sin.data_ptr<float>(), ptr<int32_t>(positions), wq, wk, b, hq, hkv, N, d, rot, max_pos,
                                  interleaved, eps, view4(c, dq), view4(c, dk), ptr<float>(dqw), ptr<float>(dkw),
                                  ptr<void>(ws), ws ? bytes(*ws) : 0, stream_of(dev));
  return {rc, dq, dk, dqw, dkw};
}

std::tuple<int, MaybeTensor> append(const Tensor &k, const Tensor &v, const Tensor &k_pages, const Tensor &v_pages,
                                    const Tensor &page_table, const Tensor &seq_lens, const MaybeTensor &cu_seqlens,
                                    const MaybeTensor &cos, const MaybeTensor &sin, const MaybeTensor &k_weight, float eps,
                                    bool interleaved, const MaybeTensor &q, const MaybeTensor &q_weight,
                                    const MaybeTensor &q_out_) {
  Checks c("kv_append");
  c.rank("k", k, 3);
  c.rank("k_pages", k_pages, 4);
  c.rank("page_table", page_table, 2);
  const int64_t T = k.size(0), hkv = k.size(1), d = k.size(2), pages = k_pages.size(0), page = k_pages.size(2);
  const int64_t batch = page_table.size(0), max_pages = page_table.size(1);
  const Shape vs{T, hkv, d}, pg{pages, hkv, page, d}, ls{batch}, cs{batch + 1};
  c.tensor("k", k, kBF16, false);
  c.tensor("v", v, kBF16, false, &vs);
  c.tensor("k_pages", k_pages, kBF16, false, &pg);
  c.tensor("v_pages", v_pages, kBF16, false, &pg);
  c.tensor("page_table", page_table, kI32, true);
  c.tensor("seq_lens", seq_lens, kI32, true, &ls);
  c.tensor("cu_seqlens", cu_seqlens, kI32, true, &cs);
  int rot = 0, max_pos = 0;
  if (cos.has_value() != sin.has_value()) c.fail("cos and sin come together");
  if (cos) std::tie(rot, max_pos) = angles(c, *cos, *sin);
  const moba_weight wq = c.weight("q_weight", q_weight, d), wk = c.weight("k_weight", k_weight, d);
  if (!q && (q_out_ || q_weight)) c.fail("q_out and q_weight need q");
  MaybeTensor q_out = q_out_;
  int64_t hq = 0;
  if (q) {
    c.rank("q", *q, 3);
    hq = q->size(1);
    const Shape qs{T, hq, d};
    c.tensor("q", *q, kBF16, false, &qs);
    c.tensor("q_out", q_out_, kBF16, false, &qs);
  }
  const int dev = c.device();
  const c10::cuda::CUDAGuard guard(dev);
  if (q && !q_out) q_out = make(q->sizes(), kBF16, dev);
  const int rc = kv_append(tokens(c, k), tokens(c, v), q ? tokens(c, *q) : kNone, ptr<int32_t>(cu_seqlens),
                           seq_lens.data_ptr<int32_t>(), page_table.data_ptr<int32_t>(), ptr<float>(cos), ptr<float>(sin),
                           wq, wk, batch, T, hq, hkv, d, rot, max_pos, interleaved, eps, page, pages, max_pages,
                           view4(c, k_pages), view4(c, v_pages), q_out ? tokens(c, *q_out) : kNone, stream_of(dev));
  return {rc, q_out};
}

Two decode(const Tensor &q, const Tensor &k_pages, const Tensor &v_pages, const Tensor &page_table,
           const Tensor &seq_lens, int window, int sink, float scale, const MaybeTensor &out_, const MaybeTensor &lse_,
           const MaybeTensor &workspace_) {
  Checks c("paged_decode_attn");
  c.rank("q", q, 3);
  c.rank("k_pages", k_pages, 4);
  c.rank("page_table", page_table, 2);
  const int64_t batch = q.size(0), hq = q.size(1), d = q.size(2);
  const int64_t pages = k_pages.size(0), hkv = k_pages.size(1), page = k_pages.size(2), max_pages = page_table.size(1);
  const Shape pg{pages, hkv, page, d}, ts{batch, max_pages}, bs{batch}, os{batch, hq, d}, ls{batch, hq};
  c.tensor("q", q, kBF16, false);
  c.tensor("k_pages", k_pages, kBF16, false, &pg);
  c.tensor("v_pages", v_pages, kBF16, false, &pg);
  c.tensor("page_table", page_table, kI32, true, &ts);
  c.tensor("seq_lens", seq_lens, kI32, true, &bs);
  c.tensor("out", out_, kBF16, false, &os);
  c.tensor("lse", lse_, kF32, true, &ls);
  c.tensor("workspace", workspace_, kAny, true);
  const int dev = c.device();
  const c10::cuda::CUDAGuard guard(dev);
  Tensor out = given(out_, os, kBF16, dev), lse = given(lse_, ls, kF32, dev), ws;
  if (workspace_) {
    ws = *workspace_;
  } else {
    size_t n = 0;
    const int rc = paged_decode_workspace_size(batch, hq, hkv, d, &n);
    if (rc) return {rc, out, lse};
    ws = make({(int64_t)n}, at::kByte, dev);
  }
  const int rc = paged_decode_attn(rows(c, q), view4(c, k_pages), view4(c, v_pages), page_table.data_ptr<int32_t>(),
                                   seq_lens.data_ptr<int32_t>(), batch, hq, hkv, d, page, pages, max_pages, window, sink,
                                   scale, rows(c, out), lse.data_ptr<float>(), ws.data_ptr(), bytes(ws), stream_of(dev));
  return {rc, out, lse};
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
  m.def("swa_fwd", &swa_fwd);
  m.def("swa_bwd", &swa_bwd);
  m.def("rope_fwd", &rope_fwd);
  m.def("rope_bwd", &rope_bwd);
  m.def("append", &append);
  m.def("decode", &decode);
}
