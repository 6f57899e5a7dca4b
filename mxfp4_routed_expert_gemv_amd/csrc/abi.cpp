// C-ABI entry points of libk3moe: argument validation (host only, before any
// launch), workspace carving and dispatch to the kernel launchers.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <string>
#include <vector>

#include "internal.h"

namespace k3 {

// One cache slot per device id; a slot is written with the same value by
// whichever thread gets there first, so concurrent first calls agree.
int cu_count() {
  constexpr int kSlots = 64;
  static std::atomic<int> cache[kSlots];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) dev = 0;
  const int slot = dev < kSlots ? dev : kSlots - 1;
  int cus = dev < kSlots ? cache[slot].load(std::memory_order_relaxed) : 0;
  if (cus > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      cus <= 0)
    cus = 256;
  if (dev < kSlots) cache[slot].store(cus, std::memory_order_relaxed);
  return cus;
}

namespace {

thread_local std::string g_last_error;

k3moe_status fail(k3moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
k3moe_status fail(k3moe_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

k3moe_status ok() {
  g_last_error.clear();
  return K3MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define K3_CHECK(expr)                         \
  do {                                         \
    k3moe_status st_ = (expr);                 \
    if (st_ != K3MOE_OK) return st_;           \
  } while (0)

k3moe_status check_shape(const k3moe_shape* s) {
  if (!s) return fail(K3MOE_EINVAL, "shape is NULL");
  if (s->T < 0 || s->d < 0 || s->f < 0 || s->E < 0 || s->k < 0 || s->n_shared < 0 ||
      s->f_shared < 0)
    return fail(K3MOE_EINVAL, "negative size in shape");
  if (s->x_dtype != K3MOE_F32 && s->x_dtype != K3MOE_BF16)
    return fail(K3MOE_EUNSUPPORTED, "x_dtype %d is not F32 or BF16", s->x_dtype);
  if (s->out_dtype != K3MOE_F32 && s->out_dtype != K3MOE_BF16)
    return fail(K3MOE_EUNSUPPORTED, "out_dtype %d is not F32 or BF16", s->out_dtype);
  if (s->router != K3MOE_ROUTER_SOFTMAX && s->router != K3MOE_ROUTER_SIGMOID &&
      s->router != K3MOE_ROUTER_SIGMOID_NORM)
    return fail(K3MOE_EUNSUPPORTED, "router %d is not one of K3MOE_ROUTER_*", s->router);
  if (s->act != K3MOE_ACT_EXACT && s->act != K3MOE_ACT_MXFP4)
    return fail(K3MOE_EUNSUPPORTED, "act %d is not one of K3MOE_ACT_*", s->act);
  if (s->act == K3MOE_ACT_MXFP4 && !(s->x_dtype == K3MOE_BF16 && s->d % 512 == 0 &&
                                     s->f % 512 == 0))
    return fail(K3MOE_EUNSUPPORTED,
                "MXFP4 activations need bf16 x, d %% 512 == 0 and f %% 512 == 0");
  if (s->routed_format != K3MOE_FMT_MXFP4 && s->routed_format != K3MOE_FMT_RVQ3)
    return fail(K3MOE_EUNSUPPORTED, "routed_format %d is not MXFP4 or RVQ3", s->routed_format);
  if (s->routed_format == K3MOE_FMT_RVQ3 && (s->d % 128 || s->f % 128))
    return fail(K3MOE_ESHAPE, "RVQ3 experts need d %% 128 == 0 and f %% 128 == 0");
  if (s->routed_format == K3MOE_FMT_RVQ3 && s->act != K3MOE_ACT_EXACT)
    return fail(K3MOE_EUNSUPPORTED, "MXFP4 activations are for MXFP4 experts");
  if (s->d < 32 || s->d > 16384 || s->d % 32)
    return fail(K3MOE_ESHAPE, "d = %d: need 32 <= d <= 16384, d %% 32 == 0", s->d);
  if (s->f < 32 || s->f > 16384 || s->f % 32)
    return fail(K3MOE_ESHAPE, "f = %d: need 32 <= f <= 16384, f %% 32 == 0", s->f);
  if (s->E < 1 || s->E > 1024) return fail(K3MOE_ESHAPE, "E = %d: need 1 <= E <= 1024", s->E);
  if (s->k < 1 || s->k > 64 || s->k > s->E)
    return fail(K3MOE_ESHAPE, "k = %d: need 1 <= k <= min(E, 64)", s->k);
  if (s->n_shared > 8) return fail(K3MOE_ESHAPE, "n_shared = %d: need <= 8", s->n_shared);
  if (s->n_shared > 0 && (s->f_shared < 32 || s->f_shared > 16384 || s->f_shared % 32))
    return fail(K3MOE_ESHAPE, "f_shared = %d: need 32 <= f_shared <= 16384, %% 32 == 0",
                s->f_shared);
  if (s->T * (int64_t)s->k >= (int64_t(1) << 31))
    return fail(K3MOE_ESHAPE, "T * k = %lld: need < 2^31", (long long)(s->T * s->k));
  return K3MOE_OK;
}

k3moe_status need_ptr(const void* p, const char* name) {
  if (!p) return fail(K3MOE_EINVAL, "%s is NULL", name);
  if (!aligned16(p)) return fail(K3MOE_EALIGN, "%s is not 16-byte aligned", name);
  return K3MOE_OK;
}

k3moe_status opt_ptr(const void* p, const char* name) {
  if (p && !aligned16(p)) return fail(K3MOE_EALIGN, "%s is not 16-byte aligned", name);
  return K3MOE_OK;
}

k3moe_status check_ws(void* ws, size_t have, size_t need) {
  if (need == 0) return K3MOE_OK;
  if (!ws) return fail(K3MOE_EWORKSPACE, "workspace is NULL; %zu bytes needed", need);
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(K3MOE_EALIGN, "workspace is not 256-byte aligned");
  if (have < need) return fail(K3MOE_EWORKSPACE, "workspace has %zu bytes; %zu needed", have, need);
  return K3MOE_OK;
}

k3moe_status check_routed_bank(const k3moe_shape& s, const k3moe_expert_bank* b) {
  if (!b) return fail(K3MOE_EINVAL, "expert bank is NULL");
  if (b->format != K3MOE_FMT_MXFP4 && b->format != K3MOE_FMT_RVQ3)
    return fail(K3MOE_EUNSUPPORTED, "routed experts must be MXFP4 or RVQ3 (format %d)",
                b->format);
  if (b->format != s.routed_format)
    return fail(K3MOE_EINVAL, "routed bank format %d differs from shape routed_format %d",
                b->format, s.routed_format);
  if (b->n_experts != s.E || b->d != s.d || b->f != s.f)
    return fail(K3MOE_EINVAL, "routed bank (n=%d, d=%d, f=%d) does not match shape (E=%d, d=%d, f=%d)",
                b->n_experts, b->d, b->f, s.E, s.d, s.f);
  K3_CHECK(need_ptr(b->w13, "routed.w13"));
  K3_CHECK(need_ptr(b->w13_scale, "routed.w13_scale"));
  K3_CHECK(need_ptr(b->w2, "routed.w2"));
  K3_CHECK(need_ptr(b->w2_scale, "routed.w2_scale"));
  return K3MOE_OK;
}

k3moe_status check_shared_bank(const k3moe_shape& s, const k3moe_expert_bank* b) {
  if (!b) return fail(K3MOE_EINVAL, "shared bank is NULL");
  if (b->format != K3MOE_FMT_BF16)
    return fail(K3MOE_EUNSUPPORTED, "shared experts must be BF16 (format %d)", b->format);
  if (b->n_experts != s.n_shared || b->d != s.d || b->f != s.f_shared)
    return fail(K3MOE_EINVAL, "shared bank (n=%d, d=%d, f=%d) does not match shape (n_shared=%d, d=%d, f_shared=%d)",
                b->n_experts, b->d, b->f, s.n_shared, s.d, s.f_shared);
  if (s.n_shared == 0) return K3MOE_OK;
  K3_CHECK(need_ptr(b->w13, "shared.w13"));
  K3_CHECK(need_ptr(b->w2, "shared.w2"));
  return K3MOE_OK;
}

k3moe_status check_bias(const k3moe_shape& s, const float* bias) {
  if (bias && s.router == K3MOE_ROUTER_SOFTMAX)
    return fail(K3MOE_EINVAL, "router_bias is given but the softmax router takes none");
  return opt_ptr(bias, "router_bias");
}

// Checks of the shared experts' training calls (T = 0 included).
k3moe_status check_train(const k3moe_shape* shape, const k3moe_expert_bank* bank) {
  K3_CHECK(check_shape(shape));
  K3_CHECK(check_shared_bank(*shape, bank));
  if (shape->n_shared == 0) return fail(K3MOE_EINVAL, "shape has no shared experts");
  if (shape->x_dtype != K3MOE_BF16)
    return fail(K3MOE_EUNSUPPORTED, "the shared experts train on bf16 x");
  if (shape->T > (int64_t(1) << 26))
    return fail(K3MOE_ESHAPE, "T = %lld: need <= 2^26", (long long)shape->T);
  return K3MOE_OK;
}

k3moe_status check_w4(const k3moe_w4_matrix* w, int64_t T, int32_t x_dtype, int32_t out_dtype,
                      bool glu) {
  if (!w) return fail(K3MOE_EINVAL, "w is NULL");
  if (T < 0 || w->n < 0 || w->k < 0 || w->group < 0) return fail(K3MOE_EINVAL, "negative size");
  if (x_dtype != K3MOE_F32 && x_dtype != K3MOE_BF16)
    return fail(K3MOE_EUNSUPPORTED, "x_dtype %d is not F32 or BF16", x_dtype);
  if (out_dtype != K3MOE_F32 && out_dtype != K3MOE_BF16)
    return fail(K3MOE_EUNSUPPORTED, "out_dtype %d is not F32 or BF16", out_dtype);
  if (T > (1 << 18)) return fail(K3MOE_ESHAPE, "T = %lld: need <= 2^18", (long long)T);
  if (w->n < 1 || w->n > (1 << 20)) return fail(K3MOE_ESHAPE, "n = %d: need 1 <= n <= 2^20", w->n);
  if (glu && w->n % 2) return fail(K3MOE_ESHAPE, "n = %d: the gated form needs an even n", w->n);
  if (w->group != 32 && w->group != 64 && (w->group < 128 || w->group % 128))
    return fail(K3MOE_ESHAPE, "group = %d: need 32, 64 or a multiple of 128", w->group);
  if (w->k < 1 || w->k > (1 << 20) || w->k % w->group)
    return fail(K3MOE_ESHAPE, "k = %d: need group <= k <= 2^20, k %% group == 0", w->k);
  if ((int64_t)w->n * w->k > (int64_t(1) << 36))
    return fail(K3MOE_ESHAPE, "n = %d, k = %d: need n * k <= 2^36", w->n, w->k);
  return K3MOE_OK;
}

// An operand's bytes; NULL or empty ones overlap nothing.
struct Region {
  const void* p;
  size_t bytes;
  const char* name;
};

bool meet(const Region& a, const Region& b) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && p < q + b.bytes && q < p + a.bytes;
}

// What a call writes must not touch what other workgroups still read or write.
template <size_t W, size_t R>
k3moe_status check_disjoint(const Region (&written)[W], const Region (&read)[R]) {
  for (size_t i = 0; i < W; ++i) {
    for (size_t j = 0; j < R; ++j)
      if (meet(written[i], read[j]))
        return fail(K3MOE_EINVAL, "%s overlaps %s", written[i].name, read[j].name);
    for (size_t j = 0; j < i; ++j)
      if (meet(written[i], written[j]))
        return fail(K3MOE_EINVAL, "%s overlaps %s", written[i].name, written[j].name);
  }
  return K3MOE_OK;
}

size_t dispatch_workspace(const k3moe_shape& s) {
  size_t need = 0;
  if (!permute_small_ok(s)) carve_permute(s, nullptr, &need);
  return need;
}

// Bytes of the operands that move between the tokens' and the experts' order.
struct RowBytes {
  size_t out, x, y, rows, pairs;   // one output element; x, y, the rows, a word per pair
  explicit RowBytes(const k3moe_shape& s) {
    const size_t in = s.x_dtype == K3MOE_F32 ? 4 : 2, P = (size_t)s.T * s.k;
    out = s.out_dtype == K3MOE_F32 ? 4 : 2;
    x = (size_t)s.T * s.d * in;
    y = (size_t)s.T * s.d * out;
    rows = P * s.d * in;
    pairs = 4 * P;
  }
};

k3moe_status check_w4_regions(const k3moe_w4_matrix& w, size_t x_bytes, const void* x,
                              const void* out, size_t out_bytes, const void* workspace,
                              size_t ws_bytes) {
  const size_t scales = (size_t)w.n * (w.k / w.group);
  const Region written[] = {{out, out_bytes, "out"}, {workspace, ws_bytes, "workspace"}};
  const Region read[] = {{x, x_bytes, "x"}, {w.codes, (size_t)w.n * (w.k / 2), "codes"},
                         {w.scale, 2 * scales, "scale"}, {w.zero, scales, "zero"}};
  return check_disjoint(written, read);
}

constexpr int kMaxTensors = 1 << 20;

struct Span {
  uintptr_t lo, hi;
  int32_t tensor;
  bool out;
};

// No clipped tensor's output may touch another tensor, or its own data other
// than exactly in place.
k3moe_status check_overlap(const k3moe_tensor* ts, int32_t n) {
  std::vector<Span> spans;
  spans.reserve(2 * (size_t)n);
  for (int32_t i = 0; i < n; ++i) {
    const k3moe_tensor& t = ts[i];
    if (t.numel == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(t.data), b = reinterpret_cast<uintptr_t>(t.out);
    const bool in_place = a == b && t.dtype == t.out_dtype;
    if (!in_place) spans.push_back({a, a + t.numel * (t.dtype == K3MOE_F32 ? 4u : 2u), i, false});
    spans.push_back({b, b + t.numel * (t.out_dtype == K3MOE_F32 ? 4u : 2u), i, true});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& p, const Span& q) { return p.lo < q.lo; });
  // against the span that reaches furthest so far, and the output that does
  uintptr_t any = 0, outs = 0;
  int32_t any_t = 0, out_t = 0;
  for (const Span& s : spans) {
    const bool hit = s.out ? s.lo < any : s.lo < outs;
    if (hit)
      return fail(K3MOE_EINVAL, "the out of tensor %d overlaps tensor %d",
                  s.out ? s.tensor : out_t, s.out ? any_t : s.tensor);
    if (s.hi > any) any = s.hi, any_t = s.tensor;
    if (s.out && s.hi > outs) outs = s.hi, out_t = s.tensor;
  }
  return K3MOE_OK;
}

// The workspace and, as the clipping writes it while tensors are still read, the
// norm touch no tensor.  (k3moe_grad_norm writes it after the last read.)
k3moe_status check_grad_regions(const k3moe_tensor* ts, int32_t n, bool clip, const float* norm,
                                const void* workspace, size_t ws_bytes) {
  const Region ws{workspace, ws_bytes, "workspace"}, nm{norm, sizeof(float), "norm"};
  if (meet(ws, nm)) return fail(K3MOE_EINVAL, "workspace overlaps norm");
  for (int32_t i = 0; i < n; ++i) {
    const k3moe_tensor& t = ts[i];
    const Region data{t.data, (size_t)t.numel * (t.dtype == K3MOE_F32 ? 4 : 2), "the data"};
    const Region out{clip ? t.out : nullptr, (size_t)t.numel * (t.out_dtype == K3MOE_F32 ? 4 : 2),
                     "the out"};
    for (const Region* r : {&data, &out}) {
      if (meet(ws, *r) || (clip && meet(nm, *r)))
        return fail(K3MOE_EINVAL, "%s overlaps %s of tensor %d", meet(ws, *r) ? ws.name : nm.name,
                    r->name, i);
    }
  }
  return K3MOE_OK;
}

k3moe_status check_grads(const k3moe_tensor* ts, int32_t n, const float* norm, bool clip) {
  if (n < 0 || n > kMaxTensors) return fail(K3MOE_EINVAL, "n = %d: need 0 <= n <= 2^20", n);
  if (n > 0 && !ts) return fail(K3MOE_EINVAL, "tensors is NULL");
  if (!norm) return fail(K3MOE_EINVAL, "norm is NULL");
  if (reinterpret_cast<uintptr_t>(norm) & 3u) return fail(K3MOE_EALIGN, "norm is not 4-byte aligned");
  for (int32_t i = 0; i < n; ++i) {
    const k3moe_tensor& t = ts[i];
    if (t.numel < 0 || t.numel > (int64_t(1) << 40))
      return fail(K3MOE_EINVAL, "tensor %d has %lld elements", i, (long long)t.numel);
    if (t.dtype != K3MOE_F32 && t.dtype != K3MOE_BF16)
      return fail(K3MOE_EUNSUPPORTED, "tensor %d: dtype %d is not F32 or BF16", i, t.dtype);
    if (clip && t.out_dtype != K3MOE_F32 && t.out_dtype != K3MOE_BF16)
      return fail(K3MOE_EUNSUPPORTED, "tensor %d: out_dtype %d is not F32 or BF16", i, t.out_dtype);
    if (t.numel == 0) continue;
    if (!t.data || (clip && !t.out)) return fail(K3MOE_EINVAL, "tensor %d has a NULL pointer", i);
    if ((reinterpret_cast<uintptr_t>(t.data) & (t.dtype == K3MOE_F32 ? 3u : 1u)) ||
        (clip && (reinterpret_cast<uintptr_t>(t.out) & (t.out_dtype == K3MOE_F32 ? 3u : 1u))))
      return fail(K3MOE_EALIGN, "tensor %d is not aligned to its elements", i);
  }
  return clip ? check_overlap(ts, n) : K3MOE_OK;
}

k3moe_status check_ortho(const k3moe_ortho* p) {
  if (!p) return fail(K3MOE_EINVAL, "the problem is NULL");
  if (p->batch < 1 || p->batch > 65535 || p->m < 1 || p->m > 32768 || p->n < 1 || p->n > 32768 ||
      (int64_t)p->batch * p->m * p->n > (int64_t(1) << 34))
    return fail(K3MOE_ESHAPE, "batch = %d, m = %d, n = %d: need 1 <= batch <= 65535, 1 <= m, n <= 32768, "
                "batch * m * n <= 2^34", p->batch, p->m, p->n);
  if (p->dtype != K3MOE_F32 && p->dtype != K3MOE_BF16)
    return fail(K3MOE_EUNSUPPORTED, "dtype %d is not F32 or BF16", p->dtype);
  if (p->steps < 1 || p->steps > 64) return fail(K3MOE_EINVAL, "steps = %d: need 1 <= steps <= 64", p->steps);
  if (!p->coefficients) return fail(K3MOE_EINVAL, "coefficients is NULL");
  if (!std::isfinite(p->scale)) return fail(K3MOE_EINVAL, "scale is not finite");
  if (!ortho_bounded(*p))
    return fail(K3MOE_EINVAL, "the coefficients let a singular value pass 1.4 before the last step");
  return K3MOE_OK;
}

size_t ortho_workspace(const k3moe_ortho& p) {
  size_t need = 0;
  if (ortho_small_ok(p)) carve_ortho_small(p, nullptr, &need);
  else carve_ortho(p, nullptr, &need);
  return need;
}

k3moe_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(K3MOE_EHIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
}

}  // namespace

// ----------------------------------------------------------------- workspace
RouteWs carve_route(const k3moe_shape& s, void* ws, size_t* bytes) {
  Carver c(ws);
  RouteWs r;
  r.logits = c.take<double>((size_t)s.T * s.E);
  r.lbound = c.take<float>((size_t)s.T * s.E);
  r.wnorm = use_mfma(s) ? c.take<float>((size_t)s.E) : nullptr;
  if (bytes) *bytes = c.off;
  return r;
}

PermuteWs carve_permute(const k3moe_shape& s, void* ws, size_t* bytes) {
  Carver c(ws);
  PermuteWs r;
  const int ch = permute_chunk_tokens(s.T, s.k);
  const size_t nchunks = (size_t)((s.T + ch - 1) / ch);
  // (what a batch needs serves a smaller one: larger chunks keep what the small ones take)
  r.chunk_base = c.take<int32_t>(std::max(nchunks, permute_least_chunks(s.T, s.k)) * s.E);
  if (bytes) *bytes = c.off;
  return r;
}

ExpertWs carve_gateup(const k3moe_shape& s, void* ws, size_t* bytes) {
  Carver c(ws);
  ExpertWs r;
  r.h = nullptr;
  r.xq = routed_scaled(s) ? c.take<uint8_t>(xq_bytes(s)) : nullptr;
  r.part = s.routed_format == K3MOE_FMT_RVQ3 ? c.take<float>(rvq_part_floats(s)) : nullptr;
  if (bytes) *bytes = c.off;
  return r;
}

ExpertWs carve_expert(const k3moe_shape& s, void* ws, size_t* bytes) {
  Carver c(ws);
  ExpertWs r;
  r.h = c.take<float>((size_t)s.T * s.k * s.f);
  r.xq = routed_scaled(s) ? c.take<uint8_t>(xq_bytes(s)) : nullptr;
  r.part = s.routed_format == K3MOE_FMT_RVQ3 ? c.take<float>(rvq_part_floats(s)) : nullptr;
  if (bytes) *bytes = c.off;
  return r;
}

SharedWs carve_shared(const k3moe_shape& s, void* ws, size_t* bytes) {
  Carver c(ws);
  SharedWs r;
  r.h = c.take<float>((size_t)s.T * s.n_shared * s.f_shared);
  if (bytes) *bytes = c.off;
  return r;
}

SharedTrainWs carve_shared_train(const k3moe_shape& s, bool backward, void* ws, size_t* bytes) {
  Carver c(ws);
  SharedTrainWs r;
  const size_t n = (size_t)shared_train_rows(s) * s.n_shared * s.f_shared;
  r.h = c.take<uint16_t>(n);
  r.dgu = backward ? c.take<uint16_t>(2 * n) : nullptr;
  r.part = c.take<float>(shared_train_part_floats(s, backward));
  if (bytes) *bytes = c.off;
  return r;
}

GradWs carve_grads(int n, void* ws, size_t* bytes) {
  Carver c(ws);
  GradWs r;
  r.partial = c.take<double>(grad_partials(n));
  r.total = c.take<double>(1);
  if (bytes) *bytes = c.off;
  return r;
}

LayerWs carve_layer(const k3moe_shape& s, void* ws, size_t* bytes) {
  Carver c(ws);
  LayerWs r;
  const size_t P = (size_t)s.T * s.k;
  r.topk_idx = c.take<int32_t>(P);
  r.topk_w = c.take<float>(P);
  r.counts = c.take<int32_t>(s.E);
  r.offsets = c.take<int32_t>((size_t)s.E + 1);
  r.sorted_pair = c.take<int32_t>(P);
  r.pair_pos = c.take<int32_t>(P);
  r.y_perm = c.take<float>(P * s.d);
  r.shared_y = s.n_shared > 0 ? c.take<float>((size_t)s.T * s.d) : nullptr;
  r.shared_h = s.n_shared > 0 ? carve_shared(s, c.base ? c.base + c.off : nullptr, nullptr).h
                              : nullptr;
  if (s.n_shared > 0) {
    size_t sh = 0;
    carve_shared(s, nullptr, &sh);
    c.off += sh;
  }
  size_t a = 0, b = 0, e = 0;
  carve_route(s, nullptr, &a);
  carve_permute(s, nullptr, &b);
  carve_expert(s, nullptr, &e);
  size_t m = a;
  if (b > m) m = b;
  if (e > m) m = e;
  r.scratch_bytes = m;
  r.scratch = c.take<char>(m);
  if (bytes) *bytes = c.off;
  return r;
}

// Validation of a whole-layer call, before anything is enqueued; *need
// receives the workspace bytes (0 for an empty batch).
k3moe_status layer_validate(const k3moe_shape* shape, const k3moe_layer_weights* weights,
                            const void* x, const void* out, const int32_t* diag, size_t* need) {
  *need = 0;
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (!weights) return fail(K3MOE_EINVAL, "weights is NULL");
  K3_CHECK(check_routed_bank(s, &weights->routed));
  K3_CHECK(check_shared_bank(s, &weights->shared));
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(weights->w_router, "w_router"));
  K3_CHECK(check_bias(s, weights->router_bias));
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(out, "out"));
  K3_CHECK(opt_ptr(diag, "diag"));
  carve_layer(s, nullptr, need);
  return K3MOE_OK;
}

namespace {
k3moe_status run_w4(const k3moe_w4_matrix* w, int64_t T, int32_t x_dtype, int32_t out_dtype,
                    const void* x, void* out, void* workspace, size_t workspace_bytes, void* stream,
                    bool glu) {
  K3_CHECK(check_w4(w, T, x_dtype, out_dtype, glu));
  if (T == 0) return ok();
  K3_CHECK(need_ptr(w->codes, "codes"));
  K3_CHECK(need_ptr(w->scale, "scale"));
  K3_CHECK(opt_ptr(w->zero, "zero"));
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(out, "out"));
  const size_t need = align256(w4_part_floats(*w, T) * sizeof(float));
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  K3_CHECK(check_w4_regions(*w, (size_t)T * w->k * (x_dtype == K3MOE_F32 ? 4 : 2), x, out,
                            (size_t)T * (glu ? w->n / 2 : w->n) * (out_dtype == K3MOE_F32 ? 4 : 2),
                            workspace, need));
  return hip_status(launch_w4(*w, T, x_dtype == K3MOE_F32, out_dtype == K3MOE_F32, glu, x, out,
                              static_cast<float*>(workspace), static_cast<hipStream_t>(stream)),
                    glu ? "k3moe_w4_glu launch" : "k3moe_w4_linear launch");
}
k3moe_status run_grads(const k3moe_tensor* tensors, int32_t n, bool clip, float max_norm,
                              float* norm, void* workspace, size_t workspace_bytes, void* stream,
                              const char* what) {
  try {
    K3_CHECK(check_grads(tensors, n, norm, clip));
  } catch (const std::bad_alloc&) {
    return fail(K3MOE_EINVAL, "no host memory for the list of %d tensors", n);
  }
  size_t need = 0;
  carve_grads(n, nullptr, &need);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  K3_CHECK(check_grad_regions(tensors, n, clip, norm, workspace, need));
  return hip_status(launch_grads(tensors, n, clip, max_norm, norm,
                                 carve_grads(n, workspace, nullptr),
                                 static_cast<hipStream_t>(stream)),
                    what);
}

}  // namespace

k3moe_status hip_failure(hipError_t e, const char* what) { return hip_status(e, what); }
k3moe_status shape_status(const k3moe_shape* shape) { return check_shape(shape); }
k3moe_status fail_status(k3moe_status st, const char* msg) { return fail(st, "%s", msg); }

k3moe_status workspace_too_small(size_t have, size_t need) {
  return fail(K3MOE_EWORKSPACE, "the call needs %zu bytes of workspace; %zu are available", need,
              have);
}

// The layer's stages on a validated call, with a workspace of at least
// k3moe_workspace_bytes(shape, K3MOE_OP_LAYER) bytes.
k3moe_status layer_run(const k3moe_shape& s, const k3moe_layer_weights& wts, const void* x,
                       void* out, int32_t* diag, void* workspace, hipStream_t st) {
  const k3moe_layer_weights* weights = &wts;
  const LayerWs L = carve_layer(s, workspace, nullptr);
  if (topk_shared_t1_ok(s) && shared_down_t1_ok(s)) {
    // One token: router logits; then the selection (which also writes the
    // permutation) beside the shared experts' gate/up; the routed experts;
    // the shared experts' down finishing each output with the combine.
    const RouteWs rws = carve_route(s, L.scratch, nullptr);
    PermOut perm;
    perm.counts = L.counts;
    perm.offsets = L.offsets;
    perm.sorted_pair = L.sorted_pair;
    perm.pair_pos = L.pair_pos;
    SharedWs sws;
    sws.h = L.shared_h;
    hipError_t e = launch_router_logits(s, x, static_cast<const uint16_t*>(weights->w_router),
                                        rws, st);
    if (e != hipSuccess) return hip_status(e, "k3moe_layer router");
    e = launch_topk_shared_t1(s, x, static_cast<const uint16_t*>(weights->w_router),
                              weights->router_bias, L.topk_idx, L.topk_w, diag, rws, perm,
                              weights->shared, sws.h, st);
    if (e != hipSuccess) return hip_status(e, "k3moe_layer top-k + shared gate/up");
    e = launch_expert_ffn(s, weights->routed, x, L.offsets, L.sorted_pair, L.y_perm,
                          carve_expert(s, L.scratch, nullptr), st);
    if (e != hipSuccess) return hip_status(e, "k3moe_layer routed experts");
    CombineArgs comb;
    comb.y_perm = L.y_perm;
    comb.pair_pos = L.pair_pos;
    comb.topk_w = L.topk_w;
    comb.out = out;
    comb.k = s.k;
    comb.out_bf16 = s.out_dtype == K3MOE_BF16;
    e = launch_shared_down_t1(s, weights->shared, sws, L.shared_y, st, comb);
    return hip_status(e, "k3moe_layer shared down + combine");
  }
  // One token: the top-k kernel also writes the (trivial) permutation.
  PermOut perm;
  if (s.T == 1) {
    perm.counts = L.counts;
    perm.offsets = L.offsets;
    perm.sorted_pair = L.sorted_pair;
    perm.pair_pos = L.pair_pos;
  }
  hipError_t e = launch_route(s, x, static_cast<const uint16_t*>(weights->w_router),
                              weights->router_bias, L.topk_idx, L.topk_w, nullptr, diag,
                              carve_route(s, L.scratch, nullptr), st, perm);
  if (e != hipSuccess) return hip_status(e, "k3moe_layer route");
  if (s.T != 1) {
    e = launch_permute(s, L.topk_idx, L.counts, L.offsets, L.sorted_pair, L.pair_pos, diag,
                       carve_permute(s, L.scratch, nullptr), st);
    if (e != hipSuccess) return hip_status(e, "k3moe_layer permute");
  }
  e = launch_expert_ffn(s, weights->routed, x, L.offsets, L.sorted_pair, L.y_perm,
                        carve_expert(s, L.scratch, nullptr), st);
  if (e != hipSuccess) return hip_status(e, "k3moe_layer routed experts");
  if (s.n_shared > 0 && !shared_mfma_ok(s)) {
    // the shared experts' down GEMV finishes each output with the combine
    CombineArgs comb;
    comb.y_perm = L.y_perm;
    comb.pair_pos = L.pair_pos;
    comb.topk_w = L.topk_w;
    comb.out = out;
    comb.k = s.k;
    comb.out_bf16 = s.out_dtype == K3MOE_BF16;
    SharedWs sws;
    sws.h = L.shared_h;
    e = launch_shared_ffn(s, weights->shared, x, L.shared_y, sws, st, comb);
    return hip_status(e, "k3moe_layer shared experts + combine");
  }
  if (s.n_shared > 0) {
    SharedWs sws;
    sws.h = L.shared_h;
    e = launch_shared_ffn(s, weights->shared, x, L.shared_y, sws, st);
    if (e != hipSuccess) return hip_status(e, "k3moe_layer shared experts");
  }
  e = launch_combine(s, L.y_perm, L.pair_pos, L.topk_w, s.n_shared > 0 ? L.shared_y : nullptr,
                     out, st);
  return hip_status(e, "k3moe_layer combine");
}

}  // namespace k3

using namespace k3;

extern "C" {

size_t k3moe_workspace_bytes(const k3moe_shape* shape, int op) {
  if (check_shape(shape) != K3MOE_OK) return 0;
  if (shape->T == 0) return 0;
  size_t n = 0;
  switch (op) {
    case K3MOE_OP_ROUTE: carve_route(*shape, nullptr, &n); break;
    case K3MOE_OP_PERMUTE: carve_permute(*shape, nullptr, &n); break;
    case K3MOE_OP_EXPERT_FFN: carve_expert(*shape, nullptr, &n); break;
    case K3MOE_OP_EXPERT_GATEUP: carve_gateup(*shape, nullptr, &n); break;
    case K3MOE_OP_SHARED_FFN: carve_shared(*shape, nullptr, &n); break;
    case K3MOE_OP_COMBINE: n = 0; break;
    case K3MOE_OP_LAYER: carve_layer(*shape, nullptr, &n); break;
    case K3MOE_OP_SHARED_TRAIN: carve_shared_train(*shape, false, nullptr, &n); break;
    case K3MOE_OP_SHARED_BACKWARD: carve_shared_train(*shape, true, nullptr, &n); break;
    case K3MOE_OP_DISPATCH: n = dispatch_workspace(*shape); break;
    case K3MOE_OP_ROUTE_BACKWARD: carve_route_back(*shape, nullptr, &n); break;
    default: return 0;
  }
  return n;
}

uint64_t k3moe_mxfp4_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return 0;
  return (uint64_t)rows * (uint64_t)cols * 17u / 32u;
}

int k3moe_path_class(const k3moe_shape* shape) {
  if (check_shape(shape) != K3MOE_OK) return K3MOE_PATH_GEMV;
  return use_mfma(*shape) ? K3MOE_PATH_MFMA : K3MOE_PATH_GEMV;
}

k3moe_status k3moe_route(const k3moe_shape* shape, const void* x, const void* w_router,
                         const float* router_bias, int32_t* topk_idx, float* topk_w,
                         float* logits, int32_t* diag, void* workspace, size_t workspace_bytes,
                         void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(w_router, "w_router"));
  K3_CHECK(check_bias(s, router_bias));
  K3_CHECK(need_ptr(topk_idx, "topk_idx"));
  K3_CHECK(need_ptr(topk_w, "topk_w"));
  K3_CHECK(opt_ptr(logits, "logits"));
  K3_CHECK(opt_ptr(diag, "diag"));
  size_t need = 0;
  carve_route(s, nullptr, &need);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const RouteWs ws = carve_route(s, workspace, nullptr);
  return hip_status(launch_route(s, x, static_cast<const uint16_t*>(w_router), router_bias,
                                 topk_idx, topk_w,
                                 logits, diag, ws, static_cast<hipStream_t>(stream)),
                    "k3moe_route launch");
}

k3moe_status k3moe_permute(const k3moe_shape* shape, const int32_t* topk_idx, int32_t* counts,
                           int32_t* offsets, int32_t* sorted_pair, int32_t* pair_pos,
                           int32_t* diag, void* workspace, size_t workspace_bytes, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(topk_idx, "topk_idx"));
  K3_CHECK(need_ptr(counts, "counts"));
  K3_CHECK(need_ptr(offsets, "offsets"));
  K3_CHECK(need_ptr(sorted_pair, "sorted_pair"));
  K3_CHECK(need_ptr(pair_pos, "pair_pos"));
  K3_CHECK(opt_ptr(diag, "diag"));
  size_t need = 0;
  carve_permute(s, nullptr, &need);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const PermuteWs ws = carve_permute(s, workspace, nullptr);
  return hip_status(launch_permute(s, topk_idx, counts, offsets, sorted_pair, pair_pos, diag, ws,
                                   static_cast<hipStream_t>(stream)),
                    "k3moe_permute launch");
}

k3moe_status k3moe_expert_ffn(const k3moe_shape* shape, const k3moe_expert_bank* bank,
                              const void* x, const int32_t* offsets, const int32_t* sorted_pair,
                              float* y, void* workspace, size_t workspace_bytes, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (!bank) return fail(K3MOE_EINVAL, "expert bank is NULL");
  if (bank->format == K3MOE_FMT_BF16) {
    // shared mode: every token through every expert of the bank, summed in order
    if (sorted_pair)
      return fail(K3MOE_EUNSUPPORTED, "a BF16 bank takes no sorted_pair (shared mode)");
    return k3moe_shared_ffn(shape, bank, x, y, workspace, workspace_bytes, stream);
  }
  K3_CHECK(check_routed_bank(s, bank));
  if (!sorted_pair)
    return fail(K3MOE_EUNSUPPORTED, "an MXFP4 bank needs sorted_pair (routed mode)");
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(offsets, "offsets"));
  K3_CHECK(need_ptr(sorted_pair, "sorted_pair"));
  K3_CHECK(need_ptr(y, "y"));
  size_t need = 0;
  carve_expert(s, nullptr, &need);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const ExpertWs ws = carve_expert(s, workspace, nullptr);
  return hip_status(launch_expert_ffn(s, *bank, x, offsets, sorted_pair, y, ws,
                                      static_cast<hipStream_t>(stream)),
                    "k3moe_expert_ffn launch");
}

k3moe_status k3moe_expert_gateup(const k3moe_shape* shape, const k3moe_expert_bank* bank,
                                 const void* x, const int32_t* offsets,
                                 const int32_t* sorted_pair, float* h, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  K3_CHECK(check_routed_bank(s, bank));
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(offsets, "offsets"));
  K3_CHECK(need_ptr(sorted_pair, "sorted_pair"));
  K3_CHECK(need_ptr(h, "h"));
  size_t need = 0;
  carve_gateup(s, nullptr, &need);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const ExpertWs ws = carve_gateup(s, workspace, nullptr);
  return hip_status(launch_expert_gateup(s, *bank, x, offsets, sorted_pair, h, ws,
                                         static_cast<hipStream_t>(stream)),
                    "k3moe_expert_gateup launch");
}

k3moe_status k3moe_expert_down(const k3moe_shape* shape, const k3moe_expert_bank* bank,
                               const float* h, const int32_t* offsets, float* y, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  K3_CHECK(check_routed_bank(s, bank));
  if (bank->format == K3MOE_FMT_RVQ3)
    return fail(K3MOE_EUNSUPPORTED,
                "the RVQ3 down product needs a workspace: use k3moe_expert_ffn");
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(h, "h"));
  K3_CHECK(need_ptr(offsets, "offsets"));
  K3_CHECK(need_ptr(y, "y"));
  return hip_status(launch_expert_down(s, *bank, h, offsets, y, static_cast<hipStream_t>(stream)),
                    "k3moe_expert_down launch");
}

k3moe_status k3moe_shared_ffn(const k3moe_shape* shape, const k3moe_expert_bank* bank,
                              const void* x, float* y, void* workspace, size_t workspace_bytes,
                              void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  K3_CHECK(check_shared_bank(s, bank));
  if (s.n_shared == 0) return fail(K3MOE_EINVAL, "shape has no shared experts");
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(y, "y"));
  size_t need = 0;
  carve_shared(s, nullptr, &need);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const SharedWs ws = carve_shared(s, workspace, nullptr);
  return hip_status(launch_shared_ffn(s, *bank, x, y, ws, static_cast<hipStream_t>(stream)),
                    "k3moe_shared_ffn launch");
}

k3moe_status k3moe_combine(const k3moe_shape* shape, const float* y_perm, const int32_t* pair_pos,
                           const float* topk_w, const float* shared_y, void* out, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(y_perm, "y_perm"));
  K3_CHECK(need_ptr(pair_pos, "pair_pos"));
  K3_CHECK(need_ptr(topk_w, "topk_w"));
  K3_CHECK(opt_ptr(shared_y, "shared_y"));
  K3_CHECK(need_ptr(out, "out"));
  return hip_status(launch_combine(s, y_perm, pair_pos, topk_w, shared_y, out,
                                   static_cast<hipStream_t>(stream)),
                    "k3moe_combine launch");
}

k3moe_status k3moe_layer(const k3moe_shape* shape, const k3moe_layer_weights* weights,
                         const void* x, void* out, int32_t* diag, void* workspace,
                         size_t workspace_bytes, void* stream) {
  size_t need = 0;
  K3_CHECK(layer_validate(shape, weights, x, out, diag, &need));
  if (shape->T == 0) return ok();
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  return layer_run(*shape, *weights, x, out, diag, workspace, static_cast<hipStream_t>(stream));
}

k3moe_status k3moe_shared_ffn_train(const k3moe_shape* shape, const k3moe_expert_bank* bank,
                                    const void* x, void* gu, void* y, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  K3_CHECK(check_train(shape, bank));
  const k3moe_shape& s = *shape;
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(gu, "gu"));
  K3_CHECK(need_ptr(y, "y"));
  size_t need = 0;
  carve_shared_train(s, false, nullptr, &need);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const size_t td = (size_t)s.T * s.d, tf = (size_t)s.T * s.n_shared * s.f_shared;
  const size_t w = (size_t)s.n_shared * s.f_shared * s.d * 2;
  const Region written[] = {{gu, 4 * tf, "gu"}, {y, td * (s.out_dtype == K3MOE_F32 ? 4 : 2), "y"},
                            {workspace, need, "workspace"}};
  const Region read[] = {{x, 2 * td, "x"}, {bank->w13, 2 * w, "w13"}, {bank->w2, w, "w2"}};
  K3_CHECK(check_disjoint(written, read));
  return hip_status(launch_shared_train(s, *bank, x, gu, y,
                                        carve_shared_train(s, false, workspace, nullptr),
                                        static_cast<hipStream_t>(stream)),
                    "k3moe_shared_ffn_train launch");
}

k3moe_status k3moe_shared_ffn_backward(const k3moe_shape* shape, const k3moe_expert_bank* bank,
                                       const void* x, const void* gu, const void* dy, void* dx,
                                       void* dw13, void* dw2, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  K3_CHECK(check_train(shape, bank));
  const k3moe_shape& s = *shape;
  hipStream_t st = static_cast<hipStream_t>(stream);
  K3_CHECK(opt_ptr(dx, "dx"));
  K3_CHECK(opt_ptr(dw13, "dw13"));
  K3_CHECK(opt_ptr(dw2, "dw2"));
  const size_t w = (size_t)s.n_shared * s.f_shared * s.d * 2, td = (size_t)s.T * s.d * 2;
  size_t need = 0;
  if (s.T > 0) {
    K3_CHECK(need_ptr(x, "x"));
    K3_CHECK(need_ptr(gu, "gu"));
    K3_CHECK(need_ptr(dy, "dy"));
    carve_shared_train(s, true, nullptr, &need);
    K3_CHECK(check_ws(workspace, workspace_bytes, need));
  }
  // (without outputs the workspace is not used either)
  const Region written[] = {{dx, td, "dx"}, {dw13, 2 * w, "dw13"}, {dw2, w, "dw2"},
                            {workspace, dx || dw13 || dw2 ? need : 0, "workspace"}};
  const Region read[] = {{x, td, "x"}, {gu, (size_t)s.T * s.n_shared * s.f_shared * 4, "gu"},
                         {dy, td, "dy"}, {bank->w13, 2 * w, "w13"}, {bank->w2, w, "w2"}};
  K3_CHECK(check_disjoint(written, read));
  if (s.T == 0) {
    hipError_t e = launch_zero(dw13, 2 * w, st);
    if (e == hipSuccess) e = launch_zero(dw2, w, st);
    return hip_status(e, "k3moe_shared_ffn_backward launch");
  }
  return hip_status(launch_shared_backward(s, *bank, x, gu, dy, dx, dw13, dw2,
                                           carve_shared_train(s, true, workspace, nullptr), st),
                    "k3moe_shared_ffn_backward launch");
}

size_t k3moe_w4_workspace_bytes(const k3moe_w4_matrix* w, int64_t T) {
  if (check_w4(w, T, K3MOE_BF16, K3MOE_BF16, false) != K3MOE_OK) return 0;
  return align256(w4_part_floats(*w, T) * sizeof(float));
}

k3moe_status k3moe_w4_linear(const k3moe_w4_matrix* w, int64_t T, int32_t x_dtype,
                             int32_t out_dtype, const void* x, void* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return run_w4(w, T, x_dtype, out_dtype, x, out, workspace, workspace_bytes, stream, false);
}

k3moe_status k3moe_w4_glu(const k3moe_w4_matrix* w, int64_t T, int32_t x_dtype,
                             int32_t out_dtype, const void* x, void* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return run_w4(w, T, x_dtype, out_dtype, x, out, workspace, workspace_bytes, stream, true);
}

size_t k3moe_grad_workspace_bytes(int32_t n) {
  if (n < 0 || n > kMaxTensors) return 0;
  size_t need = 0;
  carve_grads(n, nullptr, &need);
  return need;
}

k3moe_status k3moe_grad_norm(const k3moe_tensor* tensors, int32_t n, float* norm, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return run_grads(tensors, n, false, 0.0f, norm, workspace, workspace_bytes, stream,
                   "k3moe_grad_norm launch");
}

k3moe_status k3moe_grad_clip(const k3moe_tensor* tensors, int32_t n, float max_norm, float* norm,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.0f)) return fail(K3MOE_EINVAL, "max_norm is negative or NaN");
  return run_grads(tensors, n, true, max_norm, norm, workspace, workspace_bytes, stream,
                   "k3moe_grad_clip launch");
}

k3moe_status k3moe_dispatch(const k3moe_shape* shape, const void* x, const int32_t* topk_idx,
                            void* rows, int32_t* counts, int32_t* offsets, int32_t* sorted_pair,
                            int32_t* pair_pos, int32_t* diag, void* workspace,
                            size_t workspace_bytes, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(topk_idx, "topk_idx"));
  K3_CHECK(need_ptr(rows, "rows"));
  K3_CHECK(need_ptr(counts, "counts"));
  K3_CHECK(need_ptr(offsets, "offsets"));
  K3_CHECK(need_ptr(sorted_pair, "sorted_pair"));
  K3_CHECK(need_ptr(pair_pos, "pair_pos"));
  K3_CHECK(opt_ptr(diag, "diag"));
  const size_t need = dispatch_workspace(s);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const RowBytes b(s);
  const Region written[] = {{rows, b.rows, "rows"}, {counts, 4 * (size_t)s.E, "counts"},
                            {offsets, 4 * (size_t)s.E + 4, "offsets"}, {sorted_pair, b.pairs, "sorted_pair"},
                            {pair_pos, b.pairs, "pair_pos"}, {diag, 4 * K3MOE_DIAG_COUNT, "diag"},
                            {workspace, need, "workspace"}};
  const Region read[] = {{x, b.x, "x"}, {topk_idx, b.pairs, "topk_idx"}};
  K3_CHECK(check_disjoint(written, read));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (dispatch_small_ok(s))
    return hip_status(launch_dispatch_small(s, x, topk_idx, rows, counts, offsets, sorted_pair, pair_pos,
                                            diag, st),
                      "k3moe_dispatch launch");
  hipError_t e = launch_permute(s, topk_idx, counts, offsets, sorted_pair, pair_pos, diag,
                                carve_permute(s, workspace, nullptr), st);
  if (e == hipSuccess) e = launch_dispatch_rows(s, x, pair_pos, offsets, rows, st);
  return hip_status(e, "k3moe_dispatch launch");
}

k3moe_status k3moe_dispatch_backward(const k3moe_shape* shape, const void* drows,
                                     const int32_t* pair_pos, void* dx, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(drows, "drows"));
  K3_CHECK(need_ptr(pair_pos, "pair_pos"));
  K3_CHECK(need_ptr(dx, "dx"));
  const RowBytes b(s);
  const Region written[] = {{dx, b.y, "dx"}};
  const Region read[] = {{drows, b.rows, "drows"}, {pair_pos, b.pairs, "pair_pos"}};
  K3_CHECK(check_disjoint(written, read));
  return hip_status(launch_collect(s, drows, pair_pos, nullptr, nullptr, dx,
                                   static_cast<hipStream_t>(stream)),
                    "k3moe_dispatch_backward launch");
}

k3moe_status k3moe_collect(const k3moe_shape* shape, const void* rows, const int32_t* pair_pos,
                           const float* topk_w, const void* add, void* y, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (s.T == 0) return ok();
  K3_CHECK(need_ptr(rows, "rows"));
  K3_CHECK(need_ptr(pair_pos, "pair_pos"));
  K3_CHECK(need_ptr(topk_w, "topk_w"));
  K3_CHECK(opt_ptr(add, "add"));
  K3_CHECK(need_ptr(y, "y"));
  const RowBytes b(s);
  const Region written[] = {{y, b.y, "y"}};
  const Region read[] = {{rows, b.rows, "rows"}, {pair_pos, b.pairs, "pair_pos"},
                         {topk_w, b.pairs, "topk_w"}, {add, b.y, "add"}};
  K3_CHECK(check_disjoint(written, read));
  return hip_status(launch_collect(s, rows, pair_pos, topk_w, add, y,
                                   static_cast<hipStream_t>(stream)),
                    "k3moe_collect launch");
}

k3moe_status k3moe_collect_backward(const k3moe_shape* shape, const void* dy, const void* rows,
                                    const int32_t* pair_pos, const float* topk_w,
                                    const int32_t* offsets, void* drows, float* dw, void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  if (s.T == 0 || (!drows && !dw)) return ok();
  K3_CHECK(need_ptr(dy, "dy"));
  K3_CHECK(need_ptr(pair_pos, "pair_pos"));
  K3_CHECK(opt_ptr(drows, "drows"));
  K3_CHECK(opt_ptr(dw, "dw"));
  if (dw) K3_CHECK(need_ptr(rows, "rows"));
  if (drows) {
    K3_CHECK(need_ptr(topk_w, "topk_w"));
    K3_CHECK(need_ptr(offsets, "offsets"));
  }
  const RowBytes b(s);
  const Region written[] = {{drows, b.rows, "drows"}, {dw, b.pairs, "dw"}};
  const Region read[] = {{dy, b.y, "dy"}, {dw ? rows : nullptr, b.rows, "rows"},
                         {pair_pos, b.pairs, "pair_pos"}, {drows ? topk_w : nullptr, b.pairs, "topk_w"},
                         {drows ? offsets : nullptr, 4 * (size_t)s.E + 4, "offsets"}};
  K3_CHECK(check_disjoint(written, read));
  return hip_status(launch_collect_back(s, dy, rows, pair_pos, topk_w, offsets, drows, dw,
                                        static_cast<hipStream_t>(stream)),
                    "k3moe_collect_backward launch");
}

k3moe_status k3moe_route_backward(const k3moe_shape* shape, const void* x, const void* w_router,
                                  const int32_t* topk_idx, const float* topk_w, const float* dw,
                                  const float* logits, const int32_t* offsets,
                                  const int32_t* sorted_pair, const int32_t* pair_pos, void* dx,
                                  void* dw_router, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  K3_CHECK(check_shape(shape));
  const k3moe_shape& s = *shape;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  K3_CHECK(opt_ptr(dx, "dx"));
  K3_CHECK(opt_ptr(dw_router, "dw_router"));
  const RowBytes b(s);
  const size_t weights = (size_t)s.E * s.d;
  if (s.T == 0)
    return hip_status(launch_zero(dw_router, weights * b.out, st), "k3moe_route_backward launch");
  if (!dx && !dw_router) return ok();
  K3_CHECK(need_ptr(x, "x"));
  K3_CHECK(need_ptr(w_router, "w_router"));
  K3_CHECK(need_ptr(topk_idx, "topk_idx"));
  K3_CHECK(need_ptr(topk_w, "topk_w"));
  K3_CHECK(need_ptr(dw, "dw"));
  if (s.router == K3MOE_ROUTER_SIGMOID_NORM) K3_CHECK(need_ptr(logits, "logits"));
  else if (logits) return fail(K3MOE_EINVAL, "logits are given but this router's gradient takes none");
  K3_CHECK(need_ptr(offsets, "offsets"));
  K3_CHECK(need_ptr(sorted_pair, "sorted_pair"));
  K3_CHECK(need_ptr(pair_pos, "pair_pos"));
  size_t need = 0;
  carve_route_back(s, nullptr, &need);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const Region written[] = {{dx, b.x, "dx"}, {dw_router, weights * b.out, "dw_router"},
                            {workspace, need, "workspace"}};
  const Region read[] = {{x, b.x, "x"}, {w_router, 2 * weights, "w_router"},
                         {topk_idx, b.pairs, "topk_idx"}, {topk_w, b.pairs, "topk_w"},
                         {dw, b.pairs, "dw"}, {logits, 4 * (size_t)s.T * s.E, "logits"},
                         {offsets, 4 * (size_t)s.E + 4, "offsets"},
                         {sorted_pair, b.pairs, "sorted_pair"}, {pair_pos, b.pairs, "pair_pos"}};
  K3_CHECK(check_disjoint(written, read));
  return hip_status(launch_route_back(s, x, static_cast<const uint16_t*>(w_router), topk_idx, topk_w,
                                      dw, logits, offsets, sorted_pair, pair_pos, dx, dw_router,
                                      carve_route_back(s, workspace, nullptr), st),
                    "k3moe_route_backward launch");
}

size_t k3moe_orthogonalize_workspace_bytes(const k3moe_ortho* p) {
  return check_ortho(p) == K3MOE_OK ? ortho_workspace(*p) : 0;
}

k3moe_status k3moe_orthogonalize(const k3moe_ortho* p, const void* g, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  K3_CHECK(check_ortho(p));
  K3_CHECK(need_ptr(g, "g"));
  K3_CHECK(need_ptr(out, "out"));
  const size_t need = ortho_workspace(*p);
  K3_CHECK(check_ws(workspace, workspace_bytes, need));
  const size_t n = (size_t)p->batch * p->m * p->n, size = p->dtype == K3MOE_F32 ? 4 : 2;
  const bool in_place = g == out && p->dtype == K3MOE_BF16;
  const Region written[] = {{out, 2 * n, "out"}, {workspace, need, "workspace"}};
  const Region read[] = {{in_place ? nullptr : g, size * n, "g"}};
  K3_CHECK(check_disjoint(written, read));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return hip_status(ortho_small_ok(*p)
                        ? launch_ortho_small(*p, g, out, carve_ortho_small(*p, workspace, nullptr), st)
                        : launch_ortho(*p, g, out, carve_ortho(*p, workspace, nullptr), st),
                    "k3moe_orthogonalize launch");
}

const char* k3moe_status_str(k3moe_status status) {
  switch (status) {
    case K3MOE_OK: return "ok";
    case K3MOE_EINVAL: return "invalid argument";
    case K3MOE_ESHAPE: return "unsupported shape";
    case K3MOE_EALIGN: return "misaligned pointer";
    case K3MOE_EWORKSPACE: return "workspace missing or too small";
    case K3MOE_EUNSUPPORTED: return "unsupported dtype or weight format";
    case K3MOE_EHIP: return "HIP launch failed";
  }
  return "unknown status";
}

const char* k3moe_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
