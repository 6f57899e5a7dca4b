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
// Nothing is reused but the token's own row: the bytes of the T k rows bound them (d 7168,
// 16 slots, bf16: dispatch of 4096 tokens 195 us for 1.0 GB, collect of 16384 810 us for
// 4.2 GB, its backward at 4096 390 us for 1.9 GB, where a copy runs at 4.85 TB/s; fp32
// rows: dispatch back of 1000 tokens 92 us for 0.49 GB).  A few tokens are latency: 8 us
// for 37.  Rows are stored and read through the caches: non-temporal stores leave what
// reads the rows next to memory (dispatch and collect of 1000 tokens 112 us for 93) and are
// no faster by themselves while the rows fit the last-level cache (fp32 rows of 517 tokens:
// dispatch 62 us for 53, collect back 111 for 100; bf16 of 4096: 195 to 207 for 204 to 214,
// 393 for 391); non-temporal loads miss what the experts wrote last (collect of 37 tokens 12
// us for 8, dispatch back 101 for 92).
#include <algorithm>
#include <type_traits>

#include "chunk_plan.h"
#include "internal.h"
#include "kern_common.h"

namespace k3 {
namespace {

struct f8 {
  float v[8];
};

typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;

template <bool F32>
__device__ __forceinline__ f8 load8(const void* base, size_t unit) {
  f8 r;
  if (F32) {
    const f32x4_t* p = static_cast<const f32x4_t*>(base) + 2 * unit;
    const f32x4_t a = p[0], b = p[1];
    r = f8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  } else {
    const u32x4_t a = static_cast<const u32x4_t*>(base)[unit];
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
    f32x4_t* p = static_cast<f32x4_t*>(base) + 2 * unit;
    p[0] = f32x4_t{r.v[0], r.v[1], r.v[2], r.v[3]};
    p[1] = f32x4_t{r.v[4], r.v[5], r.v[6], r.v[7]};
  } else {
    static_cast<u32x4_t*>(base)[unit] = u32x4_t{pack2(r.v[0], r.v[1]), pack2(r.v[2], r.v[3]),
                                                pack2(r.v[4], r.v[5]), pack2(r.v[6], r.v[7])};
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
__global__ __launch_bounds__(512) void dispatch_rows(const u32x4_t* __restrict__ x,
                                                     const int32_t* __restrict__ pair_pos,
                                                     const int32_t* __restrict__ offsets,
                                                     u32x4_t* __restrict__ rows, int64_t T, int words,
                                                     int E, int k) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= words) return;
  const int64_t P = T * k;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    const u32x4_t v = x[t * words + u];
    const int32_t* pos = pair_pos + t * k;
    for (int s = 0; s < k; ++s) {
      const int p = pos[s];
      if (p >= 0 && p < P) rows[(size_t)p * words + u] = v;
    }
  }
  for (int64_t q = used_rows(offsets, E, P) + blockIdx.y; q < P; q += gridDim.y)
    rows[q * words + u] = u32x4_t{0, 0, 0, 0};
}

// ---- a token's rows, weighted and summed
struct GatherArgs {
  const void* rows;     // [limit][d]
  const int32_t* pos;   // [T][k] the rows
  const float* w;       // [T][k], NULL: 1 everywhere
  const void* add;      // [T][d] in the output's type, or NULL
  void* out;            // [T][d]
  int64_t T, limit;     // positions outside 0 .. limit are dropped
  int units, k;         // units of 8 elements a row
  int out_f32;
};

// G rows' loads are in flight at a time.  Grid (pieces of a row, tokens in strides);
// BY_PIECE: (tokens in strides of one to a wave, pieces of 512 columns), so that the
// chip works on one piece of the rows at a time: the router's weights, which many
// tokens read, then come from the L2s (T = 16384, 896 x 7168: 3.8 GB).
template <bool ROWS_F32, int G, bool BY_PIECE>
__global__ __launch_bounds__(512) void gather_sum(GatherArgs g) {
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int u = BY_PIECE ? blockIdx.y * 64 + (threadIdx.x & 63) : blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t step = BY_PIECE ? gridDim.x * 4 : gridDim.y;
  const bool in = u < g.units;
  const int uc = in ? u : g.units - 1;
  for (int64_t t = BY_PIECE ? blockIdx.x * 4 + wv : blockIdx.y; t < g.T; t += step) {
    f8 acc{};
    if (g.add) acc = load8(g.add, t * g.units + uc, g.out_f32);
    for (int s0 = 0; s0 < g.k; s0 += G) {
      int at[G];
      float w[G];
      f8 v[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int s = s0 + j < g.k ? s0 + j : g.k - 1;
        at[j] = g.pos[t * g.k + s];
        w[j] = g.w ? g.w[t * g.k + s] : 1.0f;
        if (s0 + j >= g.k || at[j] >= g.limit) at[j] = -1;
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
// lanes, then over the waves in order.  WAVE: a wave to a token instead, for rows of up
// to 1280 columns (5888 tokens, 6 slots, us so and with four waves: 192 columns 13, 27;
// 1056 43, 47; 2048 86, 72).
constexpr int kSlots = 4;
template <bool ROWS_F32, bool DY_F32, bool WAVE>
__global__ __launch_bounds__(256) void collect_back(const void* __restrict__ dy,
                                                    const void* __restrict__ rows,
                                                    const int32_t* __restrict__ pair_pos,
                                                    const float* __restrict__ topk_w,
                                                    const int32_t* __restrict__ offsets,
                                                    void* __restrict__ drows, float* __restrict__ dw,
                                                    int64_t T, int units, int E, int k) {
  __shared__ float part[4][kSlots];
  const int64_t P = T * k;
  constexpr int N = WAVE ? 64 : 256;   // threads to a token
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s0 = blockIdx.x * kSlots, tid = WAVE ? lane : threadIdx.x;
  const int64_t t0 = WAVE ? blockIdx.y * 4 + wv : blockIdx.y, step = WAVE ? gridDim.y * 4 : gridDim.y;
  for (int64_t t = t0; t < T; t += step) {
    int at[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const bool slot = s0 + j < k;
      at[j] = slot ? pair_pos[t * k + s0 + j] : -1;
      if (at[j] >= P) at[j] = -1;
      w[j] = slot && drows ? topk_w[t * k + s0 + j] : 0.0f;   // (topk_w may be NULL for dw alone)
      dot[j] = 0.0f;
    }
    for (int u = tid; u < units; u += N) {
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
      if (WAVE) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (lane == 0 && s0 + j < k) dw[t * k + s0 + j] = at[j] >= 0 ? dot[j] : 0.0f;
        continue;
      }
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
    for (int64_t q = used_rows(offsets, E, P) + t0; q < P; q += step)
      for (int u = tid; u < units; u += N) store8<ROWS_F32>(drows, q * units + u, zero);
  }
}

// ---- the router's gradient: first that of the chosen experts' logits, from dL/dw (0
// for a dropped pair, whose dw does not count).  With sig = sigmoid(logit):
//   softmax       w = e^l / sum e^l       dl_s = w_s (dw_s - sum w dw)
//   sigmoid       w = sig                 dl_s = dw_s w_s (1 - w_s)
//   renormalised  w = sig / sum sig       dl_s = w_s (1 - sig_s) (dw_s - sum w dw)
// 1 - sig is taken as sigmoid(-l), which keeps its bits where sig is near 1.
struct RouteArgs {
  const int32_t* idx;        // [T][k]
  const int32_t* pair_pos;   // [T][k]
  const float* w;            // [T][k]
  const float* dw;           // [T][k]
  const float* logits;       // [T][E], for the renormalised sigmoid
  const int32_t* offsets;    // [E + 1]
  float* dl;                 // [T][k]
  float* dl_sorted;          // [T k] at the pairs' positions
  int4* list;                // the chunks: expert, pairs q0 .. q1, row of the sums or -1
  int2* joins;               // [E] first row and number of the rows of an expert's sums
  int64_t T;
  int E, k, router, max_chunks;
};

// The router's weight gradient goes by chunks: an expert's pairs, kChunk to a chunk and
// a chunk at least.  An expert of one chunk is done with it, the chunks of others leave
// fp32 sums that dw_join adds in order.  The list is made by one workgroup, thread i
// placing experts 4 i .. 4 i + 3.  Offsets that do not ascend give experts without pairs:
// the chunks of others are at most max_chunks, whatever the offsets hold.
__device__ void plan_chunks(const RouteArgs& g) {
  __shared__ int wave[2][4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t P = g.T * g.k;
  auto at = [&](int i) {
    const int64_t o = g.offsets[i];
    return (int)(o < 0 ? 0 : o > P ? P : o);
  };
  int q0[4], n[4], c[4], sum[2] = {0, 0};
  bool falls = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = tid * 4 + j;
    q0[j] = e < g.E ? at(e) : 0;
    n[j] = e < g.E ? at(e + 1) - q0[j] : 0;
    falls |= n[j] < 0;
  }
  const bool none = __syncthreads_or(falls);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = tid * 4 + j;
    if (none) n[j] = 0;
    c[j] = e < g.E ? chunks_of(n[j]) : 0;
    sum[0] += c[j];
    sum[1] += c[j] > 1 ? c[j] : 0;
  }
  int first[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int incl = sum[h];
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    if (lane == 63) wave[h][tid >> 6] = incl;
    first[h] = incl - sum[h];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h)
    for (int w = 0; w < (tid >> 6); ++w) first[h] += wave[h][w];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = tid * 4 + j;
    if (e >= g.E) break;
    const int parts = c[j] > 1 ? c[j] : 0;
    for (int i = 0; i < c[j] && first[0] + i < g.max_chunks; ++i)
      g.list[first[0] + i] = make_int4(e, chunk_begin(q0[j], i), chunk_end(q0[j], n[j], i),
                                       parts ? first[1] + i : -1);
    g.joins[e] = make_int2(first[1], parts);
    first[0] += c[j];
    first[1] += parts;
  }
  const int all = wave[0][0] + wave[0][1] + wave[0][2] + wave[0][3];
  for (int i = all + tid; i < g.max_chunks; i += 256) g.list[i] = make_int4(-1, 0, 0, -1);
}

// The slots' dl of token t, lane s for slot s.
__device__ __forceinline__ float token_dl(const RouteArgs& g, int64_t t, int& e, int& pos, bool& there) {
  const int s = threadIdx.x & 63;
  const bool slot = s < g.k;
  const int64_t p = t * g.k + (slot ? s : 0);
  e = g.idx[p];
  pos = g.pair_pos[p];
  there = slot && pos >= 0 && pos < g.T * g.k && e >= 0 && e < g.E;
  const float w = there ? g.w[p] : 0.0f, dw = there ? g.dw[p] : 0.0f;
  if (g.router == K3MOE_ROUTER_SIGMOID) return there ? dw * w * (1.0f - w) : 0.0f;
  float v = w * (dw - wave_sum(w * dw));
  if (g.router == K3MOE_ROUTER_SIGMOID_NORM && there) v *= 1.0f / (1.0f + expf(g.logits[t * g.E + e]));
  return there ? v : 0.0f;
}

// A wave a token, and one workgroup for the list of chunks.
__global__ __launch_bounds__(256) void route_logits(RouteArgs g) {
  if (blockIdx.x == 0) return plan_chunks(g);
  const int s = threadIdx.x & 63;
  const int64_t step = (int64_t)(gridDim.x - 1) * 4;
  for (int64_t t = (int64_t)(blockIdx.x - 1) * 4 + (threadIdx.x >> 6); t < g.T; t += step) {
    int e, pos;
    bool there;
    const float v = token_dl(g, t, e, pos, there);
    if (s < g.k) g.dl[t * g.k + s] = v;
    if (there) g.dl_sorted[pos] = v;
  }
}

// Up to kFew tokens: everything in one launch, as each launch costs more than its work
// (of more tokens an expert may have too many pairs for one workgroup).  The first nx workgroups take a token's dx
// each, the others an expert's dW, whose pairs' dl they take from the tokens' weights
// again, a lane to a pair.  A wave has every fourth piece of 512 columns, kP at a time.
// (64 tokens, d 7168, 896 experts: 20 us in three launches; with a wave to a piece,
// which takes each dl 14 times, 18.6; here 12.)
constexpr int kFew = 64;
template <bool X_F32>
__global__ __launch_bounds__(256) void route_few(RouteArgs g, const void* __restrict__ x,
                                                 const void* __restrict__ w_router,
                                                 const int32_t* __restrict__ sorted_pair, void* __restrict__ dx,
                                                 void* __restrict__ dw_router, int units, int out_f32, int nx) {
  constexpr int G = 4, kP = 4;
  __shared__ float s_dl[kFew];
  __shared__ int s_row[kFew];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const bool tokens = (int)blockIdx.x < nx;
  const int at = tokens ? blockIdx.x : (int)blockIdx.x - nx;   // token or expert
  const int64_t P = g.T * g.k;
  int n;   // rows to add up, in s_row, times s_dl
  if (tokens) {
    n = g.k;
    if (wv == 0) {
      int e, pos;
      bool there;
      const float dl = token_dl(g, at, e, pos, there);
      s_dl[lane] = dl;
      s_row[lane] = there ? e : 0;
    }
  } else {
    auto offset = [&](int i) {
      const int64_t o = g.offsets[i];
      return (int)(o < 0 ? 0 : o > P ? P : o);
    };
    const int q0 = offset(at);
    n = min(max(offset(at + 1) - q0, 0), kFew);
    const int p = tid < n ? sorted_pair[q0 + tid] : -1;
    const bool in = p >= 0 && p < P;
    const int tok = in ? (unsigned)p / (unsigned)g.k : 0, pc = in ? p : 0;
    if (wv == 0) {
      const float w = g.w[pc], dw = g.dw[pc];
      float dl = dw * w * (1.0f - w);
      if (g.router != K3MOE_ROUTER_SIGMOID) {
        // (the sum in the order of slots: wave_sum's differs, and so may the last bits
        // of dl from dx's)
        constexpr int B = 8;
        float mean = 0.0f;
        for (int s0 = 0; s0 < g.k; s0 += B) {
          int e[B], pos[B];
          float ws[B], dws[B];
#pragma unroll
          for (int j = 0; j < B; ++j) {
            const int q = tok * g.k + min(s0 + j, g.k - 1);
            e[j] = g.idx[q];
            pos[j] = g.pair_pos[q];
            ws[j] = g.w[q];
            dws[j] = g.dw[q];
          }
#pragma unroll
          for (int j = 0; j < B; ++j)
            if (s0 + j < g.k && pos[j] >= 0 && pos[j] < P && e[j] >= 0 && e[j] < g.E)
              mean = __builtin_fmaf(ws[j], dws[j], mean);
        }
        dl = w * (dw - mean);
        if (g.router == K3MOE_ROUTER_SIGMOID_NORM) dl *= 1.0f / (1.0f + expf(g.logits[(size_t)tok * g.E + at]));
      }
      s_dl[tid] = in ? dl : 0.0f;
      s_row[tid] = tok;
    }
  }
  __syncthreads();
  const void* from = tokens ? w_router : x;
  const bool rows_f32 = X_F32 && !tokens;
  for (int u0 = wv * 64 + lane; u0 - lane < units; u0 += 256 * kP) {
    f8 acc[kP]{};
    for (int i = 0; i < n; i += G) {
      f8 v[G][kP];
      float w[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int a = min(i + j, n - 1);
        w[j] = i + j < n ? s_dl[a] : 0.0f;
        const size_t row = (size_t)s_row[a] * units;
#pragma unroll
        for (int c = 0; c < kP; ++c) v[j][c] = load8(from, row + min(u0 + 256 * c, units - 1), rows_f32);
      }
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (w[j] != 0.0f) {
#pragma unroll
          for (int c = 0; c < kP; ++c)
#pragma unroll
            for (int h = 0; h < 8; ++h) acc[c].v[h] = __builtin_fmaf(w[j], v[j][c].v[h], acc[c].v[h]);
        }
    }
#pragma unroll
    for (int c = 0; c < kP; ++c) {
      const int u = u0 + 256 * c;
      if (u >= units) continue;
      if (tokens) store8<X_F32>(dx, (size_t)at * units + u, acc[c]);
      else store8(dw_router, (size_t)at * units + u, acc[c], out_f32);
    }
  }
}

// dx for many tokens: a workgroup holds 64 columns of all of W in LDS (128 bytes an
// expert) and takes every gridDim.y-th group of tokens, eight to a wave, eight lanes to
// a token; a lane has one of the token's slots and eight of its columns.  (T = 16384,
// d 7168, 896 experts, 16 a token: from the L2s, row by row, 324 us.)
constexpr int kDxWaves = 16;
__global__ __launch_bounds__(64 * kDxWaves) void dx_columns(const uint4* __restrict__ w_router,
                                                            const int32_t* __restrict__ idx,
                                                            const float* __restrict__ dl,
                                                            void* __restrict__ dx, int64_t T, int units,
                                                            int E, int k, int out_f32) {
  constexpr int kZero = 1024;   // a row of zeros, for the slots whose dl is 0
  __shared__ uint4 sW[(kZero + 1) * 8];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, c = lane & 7;
  const int u = blockIdx.x * 8 + c;
  for (int i = threadIdx.x; i < E * 8; i += 64 * kDxWaves)
    sW[i] = w_router[(size_t)(i >> 3) * units + min((int)blockIdx.x * 8 + (i & 7), units - 1)];
  if (threadIdx.x < 8) sW[kZero * 8 + threadIdx.x] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  constexpr int kTokens = 8 * kDxWaves;   // of a workgroup at a time
  for (int64_t t0 = (int64_t)blockIdx.y * kTokens; t0 < T; t0 += (int64_t)gridDim.y * kTokens) {
    const int64_t t = t0 + wv * 8 + (lane >> 3), tc = t < T ? t : T - 1;
    f8 acc{};
    for (int s0 = 0; s0 < k; s0 += 8) {
      const bool slot = s0 + c < k;
      const int64_t p = tc * k + (slot ? s0 + c : 0);
      const int id = idx[p];
      const float v = dl[p];
      const float w = slot && id >= 0 && id < E ? v : 0.0f;
      const int e = w != 0.0f ? id : kZero;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int from = (lane & 56) + j;
        const float wj = __shfl(w, from, 64);
        const uint4 a = sW[__shfl(e, from, 64) * 8 + c];
        const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          acc.v[2 * h] = __builtin_fmaf(wj, bf16_lo(q[h]), acc.v[2 * h]);
          acc.v[2 * h + 1] = __builtin_fmaf(wj, bf16_hi(q[h]), acc.v[2 * h + 1]);
        }
      }
    }
    if (t < T && u < units) store8(dx, t * units + u, acc, out_f32);
  }
}

// dW of a chunk's C columns by a wave, C / 8 lanes to a row, so 512 / C pairs at a time.
//   512: a row's loads are 1 KB; for few tokens, whose x the L2s hold.
//    64: workgroups go by slices of 64 columns, XCD x through slices x, x + 8, ..,
//        so that an XCD works on one slice of x at a time, which its L2 holds.
// (16384 tokens, d 7168, 896 experts, 16 a token: 314 us on 64 columns, 555 on 512.)
template <bool X_F32, int C>
__global__ __launch_bounds__(256) void dw_chunks(const void* __restrict__ x,
                                                 const int32_t* __restrict__ sorted_pair,
                                                 const float* __restrict__ dl_sorted,
                                                 const int4* __restrict__ list,
                                                 float* __restrict__ part, void* __restrict__ dw,
                                                 int64_t T, int units, int k, int out_f32, int chunks,
                                                 int max_parts) {
  constexpr int L = C / 8, R = 64 / L, G = C == 512 ? 8 : 64 / R;   // lanes to a row, rows, loads in flight
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, row = lane / L;
  const int n_slices = (units + L - 1) / L, blocks = (chunks + 3) / 4;
  const int j = blockIdx.x >> 3;
  const int slice = (blockIdx.x & 7) + 8 * (j / blocks), at = j % blocks * 4 + wv;
  if (slice >= n_slices || at >= chunks) return;
  const int4 c = list[at];   // expert, first and last pair, row of the sums
  if (c.x < 0) return;
  const int u = slice * L + lane % L;
  const int64_t P = T * k;
  const int uc = u < units ? u : units - 1;
  f8 acc{};
  const unsigned end = c.z;
  for (unsigned b = c.y; b < end; b += 64) {   // (64 past the last pair may not fit an int)
    // lane i has the token and weight of pair b + i
    int tok = 0;
    float w = 0.0f;
    if (b + lane < end) {
      const int p = sorted_pair[b + lane];
      if (p >= 0 && p < P) {
        tok = (unsigned)p / (unsigned)k;
        w = dl_sorted[b + lane];
      }
    }
    const int n = (int)min(64u, end - b);
    for (int i = 0; i < n; i += G * R) {
      f8 v[G];
      float wi[G];
#pragma unroll
      for (int q = 0; q < G; ++q) {
        const int a = i + q * R + row;   // (those behind the last pair have weight 0)
        wi[q] = __shfl(w, a, 64);
        v[q] = load8<X_F32>(x, (size_t)__shfl(tok, a, 64) * units + uc);
      }
#pragma unroll
      for (int q = 0; q < G; ++q)
        if (wi[q] != 0.0f) {
#pragma unroll
          for (int h = 0; h < 8; ++h) acc.v[h] = __builtin_fmaf(wi[q], v[q].v[h], acc.v[h]);
        }
    }
  }
#pragma unroll
  for (int o = L; o < 64; o <<= 1)
#pragma unroll
    for (int h = 0; h < 8; ++h) acc.v[h] += __shfl_xor(acc.v[h], o, 64);
  if (u >= units || row != 0) return;
  if (c.w < 0) store8(dw, (size_t)c.x * units + u, acc, out_f32);
  else if (c.w < max_parts) store8<true>(part, (size_t)c.w * units + u, acc);
}

__global__ __launch_bounds__(256) void dw_join(const float* __restrict__ part,
                                               const int2* __restrict__ joins, void* __restrict__ dw,
                                               int units, int out_f32, int max_parts) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x, e = blockIdx.y;
  const int2 j = joins[e];
  if (u >= units || j.y == 0) return;
  constexpr int B = 4;   // loads in flight
  const int end = min(j.x + j.y, max_parts);
  f8 acc{};
  for (int c = j.x; c < end; c += B) {
    f8 v[B];
#pragma unroll
    for (int q = 0; q < B; ++q) v[q] = load8<true>(part, (size_t)min(c + q, end - 1) * units + u);
#pragma unroll
    for (int q = 0; q < B; ++q)
      if (c + q < end) {
#pragma unroll
        for (int h = 0; h < 8; ++h) acc.v[h] += v[q].v[h];
      }
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

template <bool ROWS_F32, bool BY_PIECE>
hipError_t launch_gather(const GatherArgs& g, hipStream_t st) {
  unsigned pieces, threads;
  cover(g.units, 8, &pieces, &threads);
  dim3 grid(pieces, token_blocks(g.T));
  if (BY_PIECE) {
    grid = dim3((unsigned)std::min<int64_t>((g.T + 3) / 4, 1 << 20), (g.units + 63) / 64);
    threads = 256;
  }
  if (g.k <= 2) gather_sum<ROWS_F32, 2, BY_PIECE><<<grid, threads, 0, st>>>(g);
  else if (g.k <= 4) gather_sum<ROWS_F32, 4, BY_PIECE><<<grid, threads, 0, st>>>(g);
  else if (g.k <= 8 || ROWS_F32) gather_sum<ROWS_F32, 8, BY_PIECE><<<grid, threads, 0, st>>>(g);
  else gather_sum<ROWS_F32, 16, BY_PIECE><<<grid, threads, 0, st>>>(g);
  return hipGetLastError();
}

// By the size of x: slices of 64 columns from 8 MB on.
template <bool X_F32>
hipError_t launch_dw(const k3moe_shape& s, const void* x, const int32_t* sorted_pair, const RouteBackWs& ws,
                     int chunks, int parts, void* dw, hipStream_t st) {
  const int units = s.d / 8, of32 = s.out_dtype == K3MOE_F32;
  const int4* list = reinterpret_cast<const int4*>(ws.chunks);
  const int64_t bytes = s.T * s.d * (X_F32 ? 4 : 2);
  const int lanes = bytes >= (8 << 20) ? 8 : 64;
  const int slices = ((units + lanes - 1) / lanes + 7) / 8;   // of an XCD
  const int most = (1 << 20) / slices * 4;                      // chunks of a launch (2^23 workgroups)
  for (int c0 = 0; c0 < chunks; c0 += most) {
    const int n = std::min(chunks - c0, most);
    auto run = [&](auto kernel) {
      kernel<<<8u * slices * ((n + 3) / 4), 256, 0, st>>>(x, sorted_pair, ws.dl_sorted, list + c0, ws.part, dw, s.T,
                                                          units, s.k, of32, n, parts);
    };
    if (lanes == 8) run(dw_chunks<X_F32, 64>);
    else run(dw_chunks<X_F32, 512>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int max_chunks(const k3moe_shape& s) { return most_chunks(s.E, s.T * s.k); }
int max_parts(const k3moe_shape& s) { return most_parts(s.T, s.T * s.k); }

}  // namespace

RouteBackWs carve_route_back(const k3moe_shape& s, void* ws, size_t* bytes) {
  Carver c(ws);
  RouteBackWs w{};
  if (s.T <= kFew) {   // (one launch, nothing kept)
    if (bytes) *bytes = 0;
    return w;
  }
  w.dl = c.take<float>((size_t)s.T * s.k);
  w.dl_sorted = c.take<float>((size_t)s.T * s.k);
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
      static_cast<const u32x4_t*>(x), pair_pos, offsets, static_cast<u32x4_t*>(rows), s.T, words, s.E, s.k);
  return hipGetLastError();
}

hipError_t launch_collect(const k3moe_shape& s, const void* rows, const int32_t* pair_pos,
                          const float* w, const void* add, void* out, hipStream_t st) {
  GatherArgs g{};
  g.rows = rows;
  g.pos = pair_pos;
  g.w = w;
  g.add = add;
  g.out = out;
  g.T = s.T;
  g.limit = s.T * s.k;
  g.units = s.d / 8;
  g.k = s.k;
  g.out_f32 = s.out_dtype == K3MOE_F32;
  return s.x_dtype == K3MOE_F32 ? launch_gather<true, false>(g, st) : launch_gather<false, false>(g, st);
}

hipError_t launch_collect_back(const k3moe_shape& s, const void* dy, const void* rows,
                               const int32_t* pair_pos, const float* w, const int32_t* offsets,
                               void* drows, float* dw, hipStream_t st) {
  if (!drows && !dw) return hipSuccess;
  const bool wave = s.d <= 1280;
  const dim3 grid((s.k + kSlots - 1) / kSlots, token_blocks(wave ? (s.T + 3) / 4 : s.T));
  auto run = [&](auto kernel) {
    kernel<<<grid, 256, 0, st>>>(dy, rows, pair_pos, w, offsets, drows, dw, s.T, s.d / 8, s.E, s.k);
  };
  const bool f = s.out_dtype == K3MOE_F32;
  auto pick = [&](auto rows_f32, auto dy_f32) {
    if (wave) run(collect_back<rows_f32, dy_f32, true>);
    else run(collect_back<rows_f32, dy_f32, false>);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (s.x_dtype == K3MOE_F32) f ? pick(Yes(), Yes()) : pick(Yes(), No());
  else f ? pick(No(), Yes()) : pick(No(), No());
  return hipGetLastError();
}

hipError_t launch_route_back(const k3moe_shape& s, const void* x, const uint16_t* w_router,
                             const int32_t* idx, const float* w, const float* dw, const float* logits,
                             const int32_t* offsets, const int32_t* sorted_pair,
                             const int32_t* pair_pos, void* dx, void* dw_router,
                             const RouteBackWs& ws, hipStream_t st) {
  if (!dx && !dw_router) return hipSuccess;
  RouteArgs a{};
  a.idx = idx;
  a.pair_pos = pair_pos;
  a.w = w;
  a.dw = dw;
  a.logits = logits;
  a.offsets = offsets;
  a.dl = ws.dl;
  a.dl_sorted = ws.dl_sorted;
  a.list = reinterpret_cast<int4*>(ws.chunks);
  a.joins = reinterpret_cast<int2*>(ws.joins);
  a.T = s.T;
  a.E = s.E;
  a.k = s.k;
  a.router = s.router;
  if (s.T <= kFew) {
    const int units = s.d / 8, nx = dx ? (int)s.T : 0, nw = dw_router ? s.E : 0;
    if (s.x_dtype == K3MOE_F32)
      route_few<true><<<nx + nw, 256, 0, st>>>(a, x, w_router, sorted_pair, dx, dw_router, units,
                                               s.out_dtype == K3MOE_F32, nx);
    else
      route_few<false><<<nx + nw, 256, 0, st>>>(a, x, w_router, sorted_pair, dx, dw_router, units,
                                                s.out_dtype == K3MOE_F32, nx);
    return hipGetLastError();
  }
  const int chunks = a.max_chunks = max_chunks(s), parts = max_parts(s);
  route_logits<<<1 + (unsigned)std::min<int64_t>((s.T + 3) / 4, 1 << 20), 256, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // (a workgroup of dx_columns reads E rows once, 3 us, and then T k of them from LDS)
  if (dx && s.T * s.k >= 16 * (int64_t)s.E && s.T >= 1024) {
    const int units = s.d / 8, slices = (units + 7) / 8;
    const int64_t groups = (s.T + 8 * kDxWaves - 1) / (8 * kDxWaves);
    const unsigned y = (unsigned)std::min<int64_t>(groups, std::max(1, 256 / slices));
    dx_columns<<<dim3(slices, y), 64 * kDxWaves, 0, st>>>(reinterpret_cast<const uint4*>(w_router), idx, ws.dl, dx,
                                                        s.T, units, s.E, s.k, s.x_dtype == K3MOE_F32);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else if (dx) {
    GatherArgs g{};
    g.rows = w_router;
    g.pos = idx;
    g.w = ws.dl;
    g.out = dx;
    g.T = s.T;
    g.limit = s.E;
    g.units = s.d / 8;
    g.k = s.k;
    g.out_f32 = s.x_dtype == K3MOE_F32;
    if ((e = launch_gather<false, true>(g, st)) != hipSuccess) return e;
  }
  if (!dw_router) return hipSuccess;
  e = s.x_dtype == K3MOE_F32 ? launch_dw<true>(s, x, sorted_pair, ws, chunks, parts, dw_router, st)
                             : launch_dw<false>(s, x, sorted_pair, ws, chunks, parts, dw_router, st);
  if (e != hipSuccess || parts == 0) return e;
  unsigned pieces, threads;
  cover(s.d / 8, 4, &pieces, &threads);
  dw_join<<<dim3(pieces, s.E), threads, 0, st>>>(ws.part, a.joins, dw_router, s.d / 8,
                                                 s.out_dtype == K3MOE_F32, parts);
  return hipGetLastError();
}

}  // namespace k3
