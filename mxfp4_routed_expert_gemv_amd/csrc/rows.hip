// Rows moved to and from the experts' order, and the gradients of that and of
// the router.  With pos the sorted position of the (token, slot) pair:
//   dispatch       rows[pos(t, s)] = x[t]
//   its backward   dx[t] = sum over s of drows[pos(t, s)]
//   collect        y[t] = add[t] + sum over s of w[t][s] rows[pos(t, s)]
//   its backward   drows[pos(t, s)] = w[t][s] dy[t],  dw[t][s] = <dy[t], rows[pos(t, s)]>
//   router's       dl from dw (dlogit), dx[t] = sum over s of dl[t][s] W[e(t, s)],
//                  dW[e] = sum over e's pairs of dl x
// All but dW go token by token: a wave has 64 units of 8 elements (512 columns) of
// one token, so positions and weights are scalars, x or dy is read once, every
// access of a row is 1 KB in one piece (fp32: 2 KB), and a sum has one order.
// Nothing is reused but the token's own row: the bytes of the T k rows bound them.
#include <algorithm>

#include "internal.h"
#include "kern_common.h"

namespace k3 {
namespace {

struct f8 {
  float v[8];
};

template <bool F32>
__device__ __forceinline__ f8 load8(const void* base, size_t unit) {
  f8 r;
  if (F32) {
    const float4* p = static_cast<const float4*>(base) + 2 * unit;
    const float4 a = p[0], b = p[1];
    r = f8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  } else {
    const uint4 a = static_cast<const uint4*>(base)[unit];
    r = f8{{bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y), bf16_lo(a.z), bf16_hi(a.z),
            bf16_lo(a.w), bf16_hi(a.w)}};
  }
  return r;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
template <bool F32>
__device__ __forceinline__ void store8(void* base, size_t unit, const f8& r) {
  if (F32) {
    float4* p = static_cast<float4*>(base) + 2 * unit;
    p[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    p[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
  } else {
    static_cast<uint4*>(base)[unit] = make_uint4(pack2(r.v[0], r.v[1]), pack2(r.v[2], r.v[3]),
                                                 pack2(r.v[4], r.v[5]), pack2(r.v[6], r.v[7]));
  }
}
__device__ __forceinline__ f8 load8(const void* base, size_t unit, bool f32) {
  return f32 ? load8<true>(base, unit) : load8<false>(base, unit);
}
__device__ __forceinline__ void store8(void* base, size_t unit, const f8& r, bool f32) {
  if (f32) store8<true>(base, unit, r);
  else store8<false>(base, unit, r);
}

// Positions in use: offsets[E], whatever it holds inside 0 .. P.
__device__ __forceinline__ int64_t used_rows(const int32_t* offsets, int E, int64_t P) {
  const int64_t n = offsets[E];
  return n < 0 ? 0 : n > P ? P : n;
}

// ---- dispatch: x's 16-byte words, whatever their type.  Grid (pieces of a row,
// tokens in strides).
__global__ __launch_bounds__(512) void dispatch_rows(const uint4* __restrict__ x,
                                                     const int32_t* __restrict__ pair_pos,
                                                     const int32_t* __restrict__ offsets,
                                                     uint4* __restrict__ rows, int64_t T, int words,
                                                     int E, int k) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= words) return;
  const int64_t P = T * k;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    const uint4 v = x[t * words + u];
    const int32_t* pos = pair_pos + t * k;
    for (int s = 0; s < k; ++s) {
      const int p = pos[s];
      if (p >= 0 && p < P) rows[(size_t)p * words + u] = v;
    }
  }
  for (int64_t q = used_rows(offsets, E, P) + blockIdx.y; q < P; q += gridDim.y)
    rows[q * words + u] = make_uint4(0, 0, 0, 0);
}

// ---- a token's rows, weighted and summed
struct GatherArgs {
  const void* rows;          // [P][d] or, of the router's gradient, W [E][d] bf16
  const int32_t* pair_pos;   // [T][k]
  const float* w;            // [T][k], NULL: 1 everywhere
  const void* add;           // [T][d] in the output's type, or NULL
  void* out;                 // [T][d]
  int64_t T;
  int units, k, out_f32;     // units of 8 elements a row
  // the router's gradient
  const int32_t* idx;        // [T][k]
  const float* dw;           // [T][k]
  const float* logits;       // [T][E], for the renormalised sigmoid
  float* dl;                 // [T][k], written
  int E, router;
};

// The chosen experts' dL/dlogit from dL/dw, lane s for slot s (0 for a dropped
// pair, whose dw does not count).  With sig = sigmoid(logit):
//   softmax       w = e^l / sum e^l       dl_s = w_s (dw_s - sum w dw)
//   sigmoid       w = sig                 dl_s = dw_s w_s (1 - w_s)
//   renormalised  w = sig / sum sig       dl_s = w_s (1 - sig_s) (dw_s - sum w dw)
// 1 - sig is taken as sigmoid(-l), which keeps its bits where sig is near 1.
__device__ __forceinline__ float dlogit(const GatherArgs& g, int64_t t, int s, int e, bool there) {
  const float w = s < g.k ? g.w[t * g.k + s] : 0.0f;
  const float dw = there ? g.dw[t * g.k + s] : 0.0f;
  if (g.router == K3MOE_ROUTER_SIGMOID) return there ? dw * w * (1.0f - w) : 0.0f;
  const float mean = wave_sum(there ? w * dw : 0.0f);
  float v = w * (dw - mean);
  if (g.router == K3MOE_ROUTER_SIGMOID_NORM && there) v *= 1.0f / (1.0f + expf(g.logits[t * g.E + e]));
  return there ? v : 0.0f;
}

// G rows' loads are in flight at a time.  ROUTE: the router's gradient.
template <bool ROWS_F32, int G, bool ROUTE>
__global__ __launch_bounds__(512) void gather_sum(GatherArgs g) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  const int lane = threadIdx.x & 63;
  const int64_t P = g.T * g.k;
  const int64_t limit = ROUTE ? g.E : P;
  const bool in = u < g.units;
  const int uc = in ? u : g.units - 1;
  for (int64_t t = blockIdx.y; t < g.T; t += gridDim.y) {
    float dl = 0.0f;
    int e = -1;
    if (ROUTE) {
      const bool slot = lane < g.k;
      e = slot ? g.idx[t * g.k + lane] : -1;
      const int p = slot ? g.pair_pos[t * g.k + lane] : -1;
      const bool there = p >= 0 && e >= 0 && e < g.E;
      dl = dlogit(g, t, lane, e, there);
      e = there ? e : -1;
      if (u < 64 && slot) g.dl[t * g.k + lane] = dl;
      if (!g.out) continue;
    }
    f8 acc{};
    if (g.add) acc = load8(g.add, t * g.units + uc, g.out_f32);
    for (int s0 = 0; s0 < g.k; s0 += G) {
      int at[G];
      float w[G];
      f8 v[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int s = s0 + j < g.k ? s0 + j : g.k - 1;
        if (ROUTE) {
          at[j] = __builtin_amdgcn_readlane(e, s);
          w[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(dl), s));
        } else {
          at[j] = g.pair_pos[t * g.k + s];
          w[j] = g.w ? g.w[t * g.k + s] : 1.0f;
        }
        if (s0 + j >= g.k || at[j] >= limit) at[j] = -1;
      }
#pragma unroll
      for (int j = 0; j < G; ++j)
        v[j] = load8<ROWS_F32>(g.rows, (size_t)(at[j] < 0 ? 0 : at[j]) * g.units + uc);
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (at[j] >= 0 && w[j] != 0.0f) {
#pragma unroll
          for (int c = 0; c < 8; ++c) acc.v[c] = __builtin_fmaf(w[j], v[j].v[c], acc.v[c]);
        }
    }
    if (in) store8(g.out, t * g.units + u, acc, g.out_f32);
  }
}

// ---- collect's backward: kSlots slots of a token to a workgroup of 4 waves, which
// take the row's units in turn; the dot products' partial sums are added over the
// lanes, then over the waves in order.
constexpr int kSlots = 4;
template <bool ROWS_F32, bool DY_F32>
__global__ __launch_bounds__(256) void collect_back(const void* __restrict__ dy,
                                                    const void* __restrict__ rows,
                                                    const int32_t* __restrict__ pair_pos,
                                                    const float* __restrict__ topk_w,
                                                    const int32_t* __restrict__ offsets,
                                                    void* __restrict__ drows, float* __restrict__ dw,
                                                    int64_t T, int units, int E, int k) {
  __shared__ float part[4][kSlots];
  const int64_t P = T * k;
  const int s0 = blockIdx.x * kSlots, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    int at[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const bool slot = s0 + j < k;
      at[j] = slot ? pair_pos[t * k + s0 + j] : -1;
      if (at[j] >= P) at[j] = -1;
      w[j] = slot ? topk_w[t * k + s0 + j] : 0.0f;
      dot[j] = 0.0f;
    }
    for (int u = threadIdx.x; u < units; u += 256) {
      const f8 g = load8<DY_F32>(dy, t * units + u);
      f8 v[kSlots];
      if (dw) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          v[j] = load8<ROWS_F32>(rows, (size_t)(at[j] < 0 ? 0 : at[j]) * units + u);
      }
      if (drows) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (at[j] >= 0) {
            f8 r;
#pragma unroll
            for (int c = 0; c < 8; ++c) r.v[c] = w[j] * g.v[c];
            store8<ROWS_F32>(drows, (size_t)at[j] * units + u, r);
          }
      }
      if (dw) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
#pragma unroll
          for (int c = 0; c < 8; ++c) dot[j] = __builtin_fmaf(g.v[c], v[j].v[c], dot[j]);
      }
    }
    if (dw) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) dot[j] = wave_sum(dot[j]);
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j) part[wv][j] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < kSlots && s0 + (int)threadIdx.x < k) {
        const int j = threadIdx.x;
        const int p = pair_pos[t * k + s0 + j];
        const float d = ((part[0][j] + part[1][j]) + part[2][j]) + part[3][j];
        dw[t * k + s0 + j] = p >= 0 && p < P ? d : 0.0f;
      }
      __syncthreads();
    }
  }
  if (drows && blockIdx.x == 0) {
    const f8 zero{};
    for (int64_t q = used_rows(offsets, E, P) + blockIdx.y; q < P; q += gridDim.y)
      for (int u = threadIdx.x; u < units; u += 256) store8<ROWS_F32>(drows, q * units + u, zero);
  }
}

// ---- the router's weight gradient.  An expert's pairs are cut into chunks of
// kChunk; a wave has 512 columns of a chunk.  An expert of one chunk is done with
// it, the chunks of others leave fp32 sums that dw_join adds in order.
constexpr int kChunk = 256;
struct Chunk {
  int e, q0, q1, part;   // pairs q0 .. q1 of expert e; part: row of its sums, -1: none
};

// The list of chunks, at least one for every expert, by one workgroup: thread e
// places expert e's.
__global__ __launch_bounds__(1024) void plan_chunks(const int32_t* __restrict__ offsets, Chunk* list,
                                                    int2* joins, int E, int64_t P, int max_chunks) {
  __shared__ int sums[2][1024];
  const int e = threadIdx.x;
  auto at = [&](int i) {
    const int64_t o = offsets[i];
    return (int)(o < 0 ? 0 : o > P ? P : o);
  };
  int q0 = 0, n = 0;
  if (e < E) {
    q0 = at(e);
    n = at(e + 1) - q0;
    n = n < 0 ? 0 : n;
  }
  const int chunks = e < E ? (n > kChunk ? (n + kChunk - 1) / kChunk : 1) : 0;
  const int parts = chunks > 1 ? chunks : 0;
  sums[0][e] = chunks;
  sums[1][e] = parts;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int a = e >= o ? sums[0][e - o] : 0, b = e >= o ? sums[1][e - o] : 0;
    __syncthreads();
    sums[0][e] += a;
    sums[1][e] += b;
    __syncthreads();
  }
  const int first = sums[0][e] - chunks, part = sums[1][e] - parts;
  for (int c = 0; c < chunks && first + c < max_chunks; ++c)
    list[first + c] = Chunk{e, q0 + c * kChunk, min(q0 + (c + 1) * kChunk, q0 + n),
                            parts ? part + c : -1};
  if (e < E) joins[e] = make_int2(part, parts);
  for (int c = sums[0][1023] + e; c < max_chunks; c += 1024) list[c] = Chunk{-1, 0, 0, -1};
}

template <bool X_F32>
__global__ __launch_bounds__(256) void dw_chunks(const void* __restrict__ x,
                                                 const int32_t* __restrict__ sorted_pair,
                                                 const float* __restrict__ dl,
                                                 const Chunk* __restrict__ list,
                                                 float* __restrict__ part, void* __restrict__ dw,
                                                 int64_t T, int units, int k, int out_f32, int max_parts) {
  constexpr int G = 8;
  const int u = blockIdx.x * blockDim.x + threadIdx.x, lane = threadIdx.x & 63;
  const Chunk c = list[blockIdx.y];
  if (c.e < 0) return;
  const int64_t P = T * k;
  const int uc = u < units ? u : units - 1;
  f8 acc{};
  for (int b = c.q0; b < c.q1; b += 64) {
    // lane i has the token and weight of pair b + i
    int tok = 0;
    float w = 0.0f;
    if (b + lane < c.q1) {
      const int p = sorted_pair[b + lane];
      if (p >= 0 && p < P) {
        tok = (unsigned)p / (unsigned)k;
        w = dl[p];
      }
    }
    const int n = min(64, c.q1 - b);
    for (int i = 0; i < n; i += G) {
      f8 v[G];
      float wi[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int a = i + j < n ? i + j : n - 1;
        wi[j] = i + j < n ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), a)) : 0.0f;
        v[j] = load8<X_F32>(x, (size_t)__builtin_amdgcn_readlane(tok, a) * units + uc);
      }
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (wi[j] != 0.0f) {
#pragma unroll
          for (int q = 0; q < 8; ++q) acc.v[q] = __builtin_fmaf(wi[j], v[j].v[q], acc.v[q]);
        }
    }
  }
  if (u >= units) return;
  if (c.part < 0) store8(dw, (size_t)c.e * units + u, acc, out_f32);
  else if (c.part < max_parts) store8<true>(part, (size_t)c.part * units + u, acc);
}

__global__ __launch_bounds__(256) void dw_join(const float* __restrict__ part,
                                               const int2* __restrict__ joins, void* __restrict__ dw,
                                               int units, int out_f32, int max_parts) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x, e = blockIdx.y;
  const int2 j = joins[e];
  if (u >= units || j.y == 0) return;
  f8 acc{};
  for (int c = j.x; c < j.x + j.y && c < max_parts; ++c) {
    const f8 v = load8<true>(part, (size_t)c * units + u);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc.v[q] += v.v[q];
  }
  store8(dw, (size_t)e * units + u, acc, out_f32);
}

// Workgroups that cover a row of n lanes' pieces in waves: x of the grid and threads.
void cover(int n, int most, unsigned* pieces, unsigned* threads) {
  const int waves = (n + 63) / 64;
  *pieces = (waves + most - 1) / most;
  *threads = 64 * ((waves + *pieces - 1) / *pieces);
}
unsigned token_blocks(int64_t T) { return (unsigned)std::min<int64_t>(T, 65535); }

template <bool ROWS_F32, bool ROUTE>
hipError_t launch_gather(const GatherArgs& g, hipStream_t st) {
  unsigned pieces, threads;
  cover(g.units, 8, &pieces, &threads);
  const dim3 grid(pieces, token_blocks(g.T));
  if (g.k <= 2) gather_sum<ROWS_F32, 2, ROUTE><<<grid, threads, 0, st>>>(g);
  else if (g.k <= 4) gather_sum<ROWS_F32, 4, ROUTE><<<grid, threads, 0, st>>>(g);
  else if (g.k <= 8 || ROWS_F32) gather_sum<ROWS_F32, 8, ROUTE><<<grid, threads, 0, st>>>(g);
  else gather_sum<ROWS_F32, 16, ROUTE><<<grid, threads, 0, st>>>(g);
  return hipGetLastError();
}

int max_chunks(const k3moe_shape& s) { return (int)(s.E + s.T * s.k / kChunk); }
// An expert of more than kChunk pairs has at most twice its pairs / kChunk chunks.
int max_parts(const k3moe_shape& s) { return s.T > kChunk ? (int)(2 * (s.T * s.k / kChunk)) : 0; }

}  // namespace

RouteBackWs carve_route_back(const k3moe_shape& s, void* ws, size_t* bytes) {
  Carver c(ws);
  RouteBackWs w;
  w.dl = c.take<float>((size_t)s.T * s.k);
  w.chunks = c.take<int32_t>(4 * (size_t)max_chunks(s));
  w.joins = c.take<int32_t>(2 * (size_t)s.E);
  w.part = c.take<float>((size_t)max_parts(s) * s.d);
  if (bytes) *bytes = c.off;
  return w;
}

hipError_t launch_dispatch_rows(const k3moe_shape& s, const void* x, const int32_t* pair_pos,
                                const int32_t* offsets, void* rows, hipStream_t st) {
  const int words = s.d / (s.x_dtype == K3MOE_F32 ? 4 : 8);
  unsigned pieces, threads;
  cover(words, 8, &pieces, &threads);
  dispatch_rows<<<dim3(pieces, token_blocks(s.T)), threads, 0, st>>>(
      static_cast<const uint4*>(x), pair_pos, offsets, static_cast<uint4*>(rows), s.T, words, s.E, s.k);
  return hipGetLastError();
}

hipError_t launch_collect(const k3moe_shape& s, const void* rows, const int32_t* pair_pos,
                          const float* w, const void* add, void* out, hipStream_t st) {
  GatherArgs g{};
  g.rows = rows;
  g.pair_pos = pair_pos;
  g.w = w;
  g.add = add;
  g.out = out;
  g.T = s.T;
  g.units = s.d / 8;
  g.k = s.k;
  g.out_f32 = s.out_dtype == K3MOE_F32;
  return s.x_dtype == K3MOE_F32 ? launch_gather<true, false>(g, st) : launch_gather<false, false>(g, st);
}

hipError_t launch_collect_back(const k3moe_shape& s, const void* dy, const void* rows,
                               const int32_t* pair_pos, const float* w, const int32_t* offsets,
                               void* drows, float* dw, hipStream_t st) {
  if (!drows && !dw) return hipSuccess;
  const dim3 grid((s.k + kSlots - 1) / kSlots, token_blocks(s.T));
  auto run = [&](auto kernel) {
    kernel<<<grid, 256, 0, st>>>(dy, rows, pair_pos, w, offsets, drows, dw, s.T, s.d / 8, s.E, s.k);
  };
  const bool f = s.out_dtype == K3MOE_F32;
  if (s.x_dtype == K3MOE_F32) f ? run(collect_back<true, true>) : run(collect_back<true, false>);
  else f ? run(collect_back<false, true>) : run(collect_back<false, false>);
  return hipGetLastError();
}

hipError_t launch_route_back(const k3moe_shape& s, const void* x, const uint16_t* w_router,
                             const int32_t* idx, const float* w, const float* dw, const float* logits,
                             const int32_t* offsets, const int32_t* sorted_pair,
                             const int32_t* pair_pos, void* dx, void* dw_router,
                             const RouteBackWs& ws, hipStream_t st) {
  if (!dx && !dw_router) return hipSuccess;
  GatherArgs g{};
  g.rows = w_router;
  g.pair_pos = pair_pos;
  g.w = w;
  g.out = dx;
  g.T = s.T;
  g.units = s.d / 8;
  g.k = s.k;
  g.out_f32 = s.x_dtype == K3MOE_F32;
  g.idx = idx;
  g.dw = dw;
  g.logits = logits;
  g.dl = ws.dl;
  g.E = s.E;
  g.router = s.router;
  hipError_t e = launch_gather<false, true>(g, st);
  if (e != hipSuccess || !dw_router) return e;
  Chunk* list = reinterpret_cast<Chunk*>(ws.chunks);
  int2* joins = reinterpret_cast<int2*>(ws.joins);
  const int chunks = max_chunks(s), parts = max_parts(s);
  plan_chunks<<<1, 1024, 0, st>>>(offsets, list, joins, s.E, s.T * s.k, chunks);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  unsigned pieces, threads;
  cover(g.units, 4, &pieces, &threads);
  const int of32 = s.out_dtype == K3MOE_F32;
  for (int c0 = 0; c0 < chunks; c0 += 65535) {
    const dim3 grid(pieces, std::min(chunks - c0, 65535));
    if (s.x_dtype == K3MOE_F32)
      dw_chunks<true><<<grid, threads, 0, st>>>(x, sorted_pair, ws.dl, list + c0, ws.part, dw_router,
                                                s.T, g.units, s.k, of32, parts);
    else
      dw_chunks<false><<<grid, threads, 0, st>>>(x, sorted_pair, ws.dl, list + c0, ws.part, dw_router,
                                                 s.T, g.units, s.k, of32, parts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (parts > 0) {
    dw_join<<<dim3(pieces, s.E), threads, 0, st>>>(ws.part, joins, dw_router, g.units, of32, parts);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace k3
