// The orthogonalised update (ortho.hip) of matrices whose short side is at most 128.
// The products of such a matrix fill no tiles, and a launch for each of them costs
// more than it computes.  Every step multiplies X by a polynomial of its own A = X X^T
// from the left, and A's next value follows from A alone, so X is needed only at both
// ends:
//   gram_parts   A_0 = X X^T, a piece of X's columns to a workgroup
//   iterate      P_k = a + b A_k + c A_k A_k,  A_k+1 = P_k A_k P_k, one workgroup a matrix
//   apply        P_4 ( .. P_1 (P_0 X)), 64 or 128 columns to a workgroup
// A holds squares of singular values: what A_0 lacks in bits a small one lacks twice,
// and a step multiplies it by a^2.  So every operand of these three has two fp16 parts
// (22 bits, three products each), and the host takes them only while the product of the
// a^2 is at most 2^15 (five of the usual steps: 19800); then a gradient with sixteen
// directions a hundred times its noise comes out 4e-4 off in norm, noise alone 1e-6.
// 128 x 2048: three launches for seventeen.
//
// A short side of 65 .. 128 beside a long one up to 256 goes to one launch instead,
// whatever the coefficients: `whole` takes the steps as ortho.hip does, with two parts of
// every operand here too.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "kern_common.h"
#include "dense_tile.h"

namespace k3 {
namespace {

using namespace dense;

constexpr float kScaleX = 32768.0f;   // 2^15, of X (at most 1.4)
constexpr float kScaleA = 16384.0f;   // 2^14, of A and P A (at most 1.96)

struct SmallArgs {
  const void* g;          // [batch][m][n]
  float* part;            // [batch][chunks][S][S] sums, in the tiles' lane order
  int* exps;              // [batch][chunks] the sums are of g / 2^exps
  uint16_t* poly;         // [batch][steps] both parts of every P, see poly_at
  float* norm;            // [batch][2] 1 / |g / 2^e| and e
  void* out;
  int rows, cols, tr;     // of X, the matrix taken wide; tr: g is its transpose
  int chunks, panels, steps;   // panels of a chunk
  float scale;
  float c[64][3];
};

// A power of two that takes P, at most |a| + 3.9, below 2^15.
__device__ __forceinline__ float poly_scale(float a) {
  const int q = (int)((__float_as_uint(fabsf(a) + 3.9f) >> 23) & 255) - 127;
  return ldexpf(1.0f, 14 - q);
}
// Where a P's part h has columns c .. of row r (c % 4 == 0): in the order of the
// fragments that apply reads, 1 KB each, [row block][32 columns][part][lane].
template <int S>
__device__ __forceinline__ int poly_at(int r, int c, int h) {
  return (((r >> 4) * (S / 32) + (c >> 5)) * 2 + h) * 512 + ((r & 15) + ((c >> 3) & 3) * 16) * 8 + (c & 4);
}
__device__ __forceinline__ uint32_t rest_f16(float a, float b, uint32_t hi) {
  const f16x2_t h = __builtin_bit_cast(f16x2_t, hi);
  return pack_f16(a - (float)h[0], b - (float)h[1]);
}

// A matrix of R rows x K columns in LDS, two parts of R K halves: panels of 64
// columns, each as an operand tile with the contraction along the rows of memory.
template <int R, int K>
struct Parts {
  static constexpr int kPart = R * K * 2, kBytes = 2 * kPart;
  using O = Operand<true, R>;
  __device__ static __forceinline__ void frags(const uint8_t* p, int rb, int k32, int ln, int lg, f16x8_t (&f)[2]) {
    const uint8_t* panel = p + (k32 >> 1) * O::kSlot;
    f[0] = __builtin_bit_cast(f16x8_t, O::frag(panel, rb, k32 & 1, ln, lg));
    f[1] = __builtin_bit_cast(f16x8_t, O::frag(panel + kPart, rb, k32 & 1, ln, lg));
  }
  // four columns c .. of row r (c % 4 == 0)
  __device__ static __forceinline__ void put_parts(uint8_t* p, int r, int c, uint2 h, uint2 l) {
    uint8_t* at = p + (c >> 6) * O::kSlot + r * 128 + ((((c >> 3) & 7) ^ ((r >> 1) & 7)) << 4) + (c & 4) * 2;
    *reinterpret_cast<uint2*>(at) = h;
    *reinterpret_cast<uint2*>(at + kPart) = l;
  }
  __device__ static __forceinline__ void put4(uint8_t* p, int r, int c, const float (&v)[4]) {
    const uint2 h = make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
    put_parts(p, r, c, h, make_uint2(rest_f16(v[0], v[1], h.x), rest_f16(v[2], v[3], h.y)));
  }
  // eight columns (c % 8 == 0)
  __device__ static __forceinline__ void put8(uint8_t* p, int r, int c, const float (&v)[8]) {
    uint8_t* at = p + (c >> 6) * O::kSlot + r * 128 + ((((c >> 3) & 7) ^ ((r >> 1) & 7)) << 4);
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = pack_f16(v[2 * j], v[2 * j + 1]);
      l[j] = rest_f16(v[2 * j], v[2 * j + 1], h[j]);
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(at + kPart) = make_uint4(l[0], l[1], l[2], l[3]);
  }
};

// Product q of the parts of a and b added to c (the least first; that of both second
// parts is left out).
template <int q>
__device__ __forceinline__ f32x4_t mfma(const f16x8_t (&a)[2], const f16x8_t (&b)[2], f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a[q == 0], b[q == 1], c, 0, 0, 0);
}

template <int N>
using Int = std::integral_constant<int, N>;

// acc += A B^T over K columns: MB x NB blocks of 16 x 16 from row blocks ra of A and
// rb of B; a lane holds row ln of A's block, columns 4 lg .. of B's.
template <typename M, int MB, int NB, int K>
__device__ __forceinline__ void multiply(const uint8_t* a, const uint8_t* b, int ra, int rb, f32x4_t (&acc)[MB][NB]) {
  const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  f16x8_t fa[2][MB][2], fb[2][NB][2];   // (the next 32 columns' fragments on their way)
  auto load = [&](int k) {
#pragma unroll
    for (int i = 0; i < MB; ++i) M::frags(a, ra + i, k, ln, lg, fa[k & 1][i]);
#pragma unroll
    for (int j = 0; j < NB; ++j) M::frags(b, rb + j, k, ln, lg, fb[k & 1][j]);
  };
  load(0);
#pragma unroll
  for (int k = 0; k < K / 32; ++k) {
    if (k + 1 < K / 32) load(k + 1);
    auto add = [&](auto q) {   // (of all blocks in turn: the next into the same sums has to wait)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma<q>(fb[k & 1][j], fa[k & 1][i], acc[i][j]);
    };
    add(Int<0>());
    add(Int<1>());
    add(Int<2>());
  }
}

// Eight elements i, i + step, .. of g, `in` of them (the others 0).  VEC: they are
// neighbours at 32 (bf16: 16) bytes, all of them in or none.  Every load is issued, of
// the first element where there is none, and nothing waits before get(): behind
// branches each would be waited for by itself.
template <bool F32, bool VEC>
struct Eight {
  static constexpr int kWords = !F32 && VEC ? 4 : 8;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* g, size_t i, size_t step, int in) {
    if (VEC) {
      const size_t at = in >= 8 ? i : 0;
#pragma unroll
      for (int q = 0; q < kWords / 4; ++q) {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const char*>(g) + at * (F32 ? 4 : 2) + 16 * q);
        w[4 * q] = a.x; w[4 * q + 1] = a.y; w[4 * q + 2] = a.z; w[4 * q + 3] = a.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const size_t at = j < in ? i + j * step : 0;
        w[j] = F32 ? static_cast<const uint32_t*>(g)[at] : static_cast<const uint16_t*>(g)[at];
      }
    }
  }
  __device__ __forceinline__ void get(int in, float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = F32 ? __uint_as_float(w[j]) : VEC ? (j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2])) : bf16_lo(w[j]);
      v[j] = j < in ? x : 0.0f;
    }
  }
};

// Workgroups of 1024 threads take 8192 elements of X at a time: kW columns.
template <int S>
struct Panel {
  static constexpr int kW = 8192 / S;
};

// ---- A's part of `panels` panels of X
template <int S, bool F32, bool VEC>
__global__ __launch_bounds__(1024) void gram_parts(SmallArgs g) {
  constexpr int kW = Panel<S>::kW, NB = S / 64;   // 4 x 4 waves, NB x NB blocks each
  using M = Parts<S, kW>;
  __shared__ __attribute__((aligned(16))) uint8_t x[M::kBytes];
  __shared__ float top[16];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const size_t first = (size_t)blockIdx.y * g.rows * g.cols;
  // row r of X and eight columns from u on; a row of memory to neighbouring lanes
  const int r = g.tr ? tid % S : tid / (kW / 8), u = (g.tr ? tid / S : tid % (kW / 8)) * 8;
  const size_t step = g.tr ? g.rows : 1;
  auto inside = [&](int panel) { return r < g.rows ? g.cols - (panel * kW + u) : 0; };
  auto load = [&](int panel, Eight<F32, VEC>& x8) {
    const int c = panel * kW + u;
    x8.load(g.g, first + (g.tr ? (size_t)c * g.rows + r : (size_t)r * g.cols + c), step, inside(panel));
  };
  const int p0 = blockIdx.x * g.panels, p1 = min(p0 + g.panels, (g.cols + kW - 1) / kW);
  Eight<F32, VEC> raw;
  float v[8], w[8], most = 0.0f;
  load(p0, raw);
  raw.get(inside(p0), v);
#pragma unroll
  for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(v[j]));
  for (int p = p0 + 1; p < p1; ++p) {
    load(p, raw);
    raw.get(inside(p), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(w[j]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
  if (lane == 0) top[wv] = most;
  __syncthreads();
  most = top[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) most = fmaxf(most, top[i]);
  // most < 2^e (zeros have the least e of all, an infinity goes on as it is)
  int e = most > 0.0f ? 0 : -1000;
  if (most > 0.0f && most < INFINITY) (void)frexpf(most, &e);
  f32x4_t acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int p = p0; p < p1; ++p) {
    if (p > p0) {
      load(p, raw);
      raw.get(inside(p), v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = ldexpf(v[j], 15 - e);
    if (p > p0) __syncthreads();
    M::put8(x, r, u, v);
    __syncthreads();
    multiply<M, NB, NB, kW>(x, x, (wv >> 2) * NB, (wv & 3) * NB, acc);
  }
  const size_t chunk = (size_t)blockIdx.y * g.chunks + blockIdx.x;
  if (tid == 0) g.exps[chunk] = e;
  f32x4_t* part = reinterpret_cast<f32x4_t*>(g.part) + chunk * (S * S / 4);
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int tile = ((wv >> 2) * NB + i) * (S / 16) + (wv & 3) * NB + j;
      part[tile * 64 + lane] = acc[i][j] * (1.0f / (kScaleX * kScaleX));
    }
}

// ---- the polynomials.  64: 4 x 4 waves of one block; 128: 2 x 4 waves of 4 x 2
// blocks (43 us for five steps when that was chosen; four waves of 4 x 4 50).
template <int S>
struct Waves {
  static constexpr int MB = S == 64 ? 1 : 4, NB = S == 64 ? 1 : 2;
  static constexpr int N = S / 16 / MB * (S / 16 / NB), kThreads = 64 * N;
};
template <int S>
__global__ __launch_bounds__(Waves<S>::kThreads) void iterate(SmallArgs g) {
  constexpr int MB = Waves<S>::MB, NB = Waves<S>::NB, N = Waves<S>::N;
  using M = Parts<S, S>;
  __shared__ __attribute__((aligned(16))) uint8_t sA[M::kBytes];
  __shared__ __attribute__((aligned(16))) uint8_t sP[M::kBytes];
  __shared__ float sums[N];
  __shared__ float coef[64][3];
  // (read at once and early: an argument of a kernel is far away)
  if (threadIdx.x < 3 * g.steps) (&coef[0][0])[threadIdx.x] = (&g.c[0][0])[threadIdx.x];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, ln = lane & 15, lg = lane >> 4;
  const int ra = wv / (S / 16 / NB) * MB, rb = wv % (S / 16 / NB) * NB;
  f32x4_t A[MB][NB], acc[MB][NB];
  auto zero = [&]() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };
  auto put = [&](uint8_t* to, float f, f32x4_t (&v)[MB][NB]) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const float q[4] = {v[i][j][0] * f, v[i][j][1] * f, v[i][j][2] * f, v[i][j][3] * f};
        M::put4(to, (ra + i) * 16 + ln, (rb + j) * 16 + lg * 4, q);
      }
  };
  // A_0: the parts in order, as multiples of the largest one's power of two
  const int* exps = g.exps + (size_t)blockIdx.x * g.chunks;
  int e = exps[0];
  for (int c = 1; c < g.chunks; ++c) e = max(e, exps[c]);
  const f32x4_t* part = reinterpret_cast<const f32x4_t*>(g.part) + (size_t)blockIdx.x * g.chunks * (S * S / 4);
  zero();
  for (int c = 0; c < g.chunks; ++c) {
    const float f = ldexpf(1.0f, 2 * (exps[c] - e));
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[i][j] += f * part[(size_t)c * (S * S / 4) + ((ra + i) * (S / 16) + rb + j) * 64 + lane];
  }
  float trace = 0.0f;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) trace += ra + i == rb + j && ln == lg * 4 + q ? acc[i][j][q] : 0.0f;
  trace = wave_sum(trace);
  if (lane == 0) sums[wv] = trace;
  __syncthreads();
  trace = sums[0];
#pragma unroll
  for (int i = 1; i < N; ++i) trace += sums[i];
  const float f = trace == 0.0f ? 0.0f : 1.0f / trace;
  if (threadIdx.x == 0) {
    g.norm[2 * blockIdx.x] = trace == 0.0f ? 0.0f : 1.0f / sqrtf(trace);
    g.norm[2 * blockIdx.x + 1] = (float)e;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) A[i][j] = acc[i][j] * f;
  put(sA, kScaleA, A);
  __syncthreads();
  uint16_t* poly = g.poly + (size_t)blockIdx.x * g.steps * 2 * S * S;
  for (int s = 0; s < g.steps; ++s, poly += 2 * S * S) {
    const float ca = coef[s][0], cb = coef[s][1], cc = coef[s][2] * (1.0f / (kScaleA * kScaleA));
    const float scale = poly_scale(ca);
    zero();
    multiply<M, MB, NB, S>(sA, sA, ra, rb, acc);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        float q[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool diagonal = ra + i == rb + j && ln == lg * 4 + r;
          q[r] = __builtin_fmaf(cc, acc[i][j][r], __builtin_fmaf(cb, A[i][j][r], diagonal ? ca : 0.0f)) * scale;
        }
        const int m = (ra + i) * 16 + ln, n = (rb + j) * 16 + lg * 4;
        M::put4(sP, m, n, q);
        const uint2 h = make_uint2(pack_f16(q[0], q[1]), pack_f16(q[2], q[3]));
        *reinterpret_cast<uint2*>(poly + poly_at<S>(m, n, 0)) = h;
        *reinterpret_cast<uint2*>(poly + poly_at<S>(m, n, 1)) =
            make_uint2(rest_f16(q[0], q[1], h.x), rest_f16(q[2], q[3], h.y));
      }
    if (s + 1 == g.steps) break;
    __syncthreads();
    const float back = 1.0f / scale;   // (a product of P and A has their scales)
    zero();
    multiply<M, MB, NB, S>(sP, sA, ra, rb, acc);
    __syncthreads();
    put(sA, back, acc);                // P A, in A's place
    __syncthreads();
    zero();
    multiply<M, MB, NB, S>(sP, sA, ra, rb, acc);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) A[i][j] = acc[i][j] * (back / kScaleA);
    __syncthreads();
    put(sA, kScaleA, A);
    __syncthreads();
  }
}

// Four values of row `row` of memory from column `col` on (col % 4 == 0), those inside.
__device__ __forceinline__ void put_row(uint16_t* o, int row, int col, const SmallArgs& g, uint2 q) {
  const int nr = g.tr ? g.cols : g.rows, nc = g.tr ? g.rows : g.cols;
  if (row >= nr || col >= nc) return;
  uint16_t* p = o + (size_t)row * nc + col;
  if (nc % 4 == 0) {
    *reinterpret_cast<uint2*>(p) = q;
  } else {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (col + r < nc) p[r] = (uint16_t)(w[r / 2] >> (r & 1 ? 16 : 0));
  }
}

// ---- kW columns of X through all polynomials.  X is kept transposed, [kW][S], as the
// products need it; a wave has 16 rows of P and four blocks of columns, and reads P's
// fragments from memory, kAhead steps before it needs them: the reads take longer than
// a step.
template <int S, bool F32, bool VEC>
__global__ __launch_bounds__(512) void apply(SmallArgs g) {
  constexpr int kW = Panel<S>::kW, K = S / 32, kAhead = 4, NB = 4;
  using M = Parts<kW, S>;
  __shared__ __attribute__((aligned(16))) uint8_t x[M::kBytes];
  __shared__ float unscale[64];   // of every step's P
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, ln = lane & 15, lg = lane >> 4;
  const size_t first = (size_t)blockIdx.y * g.rows * g.cols;
  const int n0 = blockIdx.x * kW;
  const int mb = wv % (S / 16), nb = wv / (S / 16) * NB;
  const uint16_t* poly = g.poly + (size_t)blockIdx.y * g.steps * 2 * S * S + mb * K * 1024 + lane * 8;
  f16x8_t fp[kAhead][K][2];
  auto load_p = [&](int s, f16x8_t (&f)[K][2]) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f[k][h] = *reinterpret_cast<const f16x8_t*>(poly + (size_t)s * 2 * S * S + (k * 2 + h) * 512);
  };
  const float norm = g.norm[2 * blockIdx.y], power = g.norm[2 * blockIdx.y + 1];
  // column c of X and eight rows from u on
  Eight<F32, VEC> raw[2];
  auto place = [&](int q, int& c, int& u) {
    const int i = tid + 512 * q;
    c = g.tr ? i / (S / 8) : i % kW;
    u = (g.tr ? i % (S / 8) : i / kW) * 8;
    return n0 + c < g.cols ? g.rows - u : 0;
  };
  const size_t stride = g.tr ? 1 : g.cols;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    int c, u;
    const int in = place(q, c, u);
    raw[q].load(g.g, first + (g.tr ? (size_t)(n0 + c) * g.rows + u : (size_t)u * g.cols + n0 + c), stride, in);
  }
#pragma unroll
  for (int j = 0; j < kAhead; ++j) load_p(min(j, g.steps - 1), fp[j]);
  if (tid < g.steps) unscale[tid] = 1.0f / poly_scale(g.c[tid][0]);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    int c, u;
    float v[8];
    const int in = place(q, c, u);
    raw[q].get(in, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = ldexpf(v[j], -(int)power) * (norm * kScaleX);
    M::put8(x, c, u, v);
  }
  __syncthreads();
  f32x4_t acc[NB];
  auto step = [&](int s, f16x8_t (&p)[K][2]) {
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      f16x8_t fx[NB][2];
#pragma unroll
      for (int j = 0; j < NB; ++j) M::frags(x, nb + j, k, ln, lg, fx[j]);
      auto add = [&](auto q) {   // a lane: column ln of the block, rows 4 lg ..
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[j] = mfma<q>(p[k], fx[j], acc[j]);
      };
      add(Int<0>());
      add(Int<1>());
      add(Int<2>());
    }
    if (s + kAhead < g.steps) load_p(s + kAhead, p);
    if (s + 1 == g.steps) return;
    const float back = unscale[s];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const float q[4] = {acc[j][0] * back, acc[j][1] * back, acc[j][2] * back, acc[j][3] * back};
      M::put4(x, (nb + j) * 16 + ln, mb * 16 + lg * 4, q);
    }
    __syncthreads();
  };
  for (int s = 0; s < g.steps; s += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (s + j < g.steps) step(s + j, fp[j]);
  }
  const float f = g.scale * (1.0f / kScaleX) * unscale[g.steps - 1];
  uint16_t* o = static_cast<uint16_t*>(g.out) + first;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{acc[j][0] * f, acc[j][1] * f}, bf16x2_t));
    const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{acc[j][2] * f, acc[j][3] * f}, bf16x2_t));
    uint2 q = make_uint2(a, b);
    // four values of one row of memory: rows of X there when it is g's transpose
    int row = n0 + (nb + j) * 16 + ln, col = mb * 16 + lg * 4;
    if (!g.tr) {
      q = transpose4(q, lane);
      row = mb * 16 + lg * 4 + (ln & 3);
      col = n0 + (nb + j) * 16 + (ln & ~3);
    }
    put_row(o, row, col, g, q);
  }
}

// ---- matrices of 65 .. 128 by up to 256: all steps as ortho.hip takes them, by one
// workgroup, X itself in fp32 in the registers of the waves that compute it: 64 rows x 64
// columns each of 2 x 4.  Every operand of a product has two fp16 parts: A's (then B's) in
// LDS, and beside them those of one half of X, 128 columns, at a time, as both halves'
// do not fit.  A wave has 32 columns of each half.  (256 x 128: 60 us, a step 10, of which
// LDS is busy 6.0 and the matrix cores 4.7; what is left are the nine barriers of a step.
// One part took 33 us and left the result 1.2e-3 off in norm beside its rounding to bf16,
// two 2e-8; all 64 blocks of the symmetric products for 36, and loads of single values of
// 128 x 256: 65 and 75 us.)
//
// Half of X, [128][128], serves as both operands: a row's eight columns for X X^T, and,
// read transposed, a column's eight rows for B X.  Row r's 32 bytes of columns 16 b .. are
// at block b ^ key, key = r mod 4 | (r / 8 mod 2) << 2, their two halves swapped where r
// has bit 2: eight rows' 16 bytes fall on distinct banks, and so do the eight lines of
// half a wave's transposing read.
constexpr int kBigL = 256, kHalf = 128;
struct HalfX {
  static constexpr int kPart = 128 * kHalf * 2, kBytes = 2 * kPart;
  __device__ static __forceinline__ int at(int r, int c) {   // byte of column c of row r (c % 4 == 0)
    const int key = (r & 3) | ((r >> 1) & 4);
    return r * (2 * kHalf) + (((c >> 4) ^ key) << 5) + ((((c >> 3) ^ (r >> 2)) & 1) << 4) + (c & 7) * 2;
  }
  __device__ static __forceinline__ void put4(uint8_t* x, int r, int c, f32x4_t v) {
    const uint2 h = make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
    *reinterpret_cast<uint2*>(x + at(r, c)) = h;
    *reinterpret_cast<uint2*>(x + kPart + at(r, c)) = make_uint2(rest_f16(v[0], v[1], h.x), rest_f16(v[2], v[3], h.y));
  }
  // rows 16 rb + ln, columns 32 k + 8 lg ..
  __device__ static __forceinline__ void rows(const uint8_t* x, int rb, int k, int ln, int lg, f16x8_t (&f)[2]) {
    const uint8_t* p = x + at(rb * 16 + ln, 32 * k + 8 * lg);
    f[0] = *reinterpret_cast<const f16x8_t*>(p);
    f[1] = *reinterpret_cast<const f16x8_t*>(p + kPart);
  }
  // columns 16 cb + ln, rows 32 k + 8 lg ..
  __device__ static __forceinline__ void columns(const uint8_t* x, int cb, int k, int ln, int lg, f16x8_t (&f)[2]) {
    const int r = 32 * k + 8 * lg + (ln >> 2);
    const uint8_t *p = x + at(r, cb * 16 + (ln & 3) * 4), *q = x + at(r + 4, cb * 16 + (ln & 3) * 4);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      union { s16x4_t w[2]; f16x8_t v; } u;
      u.w[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + h * kPart));
      u.w[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(q + h * kPart));
      f[h] = u.v;
    }
  }
};

// acc += MB x NB blocks' products over 128 columns: load_a(i, k, f) and load_b(j, k, f)
// give the two parts of row block i and column block j, elements 32 k ..
template <int MB, int NB, int N, typename LA, typename LB>
__device__ __forceinline__ void add_products(LA load_a, LB load_b, f32x4_t (&acc)[N]) {
  static_assert(N >= MB * NB, "a sum for every block");
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f16x8_t fa[MB][2], fb[NB][2];
#pragma unroll
    for (int i = 0; i < MB; ++i) load_a(i, k, fa[i]);
#pragma unroll
    for (int j = 0; j < NB; ++j) load_b(j, k, fb[j]);
    auto add = [&](auto q) {
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i * NB + j] = mfma<q>(fb[j], fa[i], acc[i * NB + j]);
    };
    add(Int<0>());
    add(Int<1>());
    add(Int<2>());
  }
}

// The 36 blocks of a symmetric product of 128 x 128 that lie on and over the diagonal: six
// waves have 2 x 2 of them over it, the last two the three of two squares of 2 x 2 on it
// each (so a SIMD has 8 or 10 where all 64 would be 16).
struct SymBlocks {
  static constexpr int kMost = 6;
  int wv;
  // squares of waves 0 .. 5: (0, 1) (0, 2) (0, 3) (1, 2) (1, 3) (2, 3)
  __device__ __forceinline__ int upper() const { return wv < 3 ? 0 : wv < 5 ? 1 : 2; }
  __device__ __forceinline__ int right() const { return wv < 3 ? wv + 1 : wv < 5 ? wv - 1 : 3; }
  // f(b, row block, column block, whether it lies over the diagonal) for the wave's blocks
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (wv < 6) {
      const int rb = 2 * upper(), cb = 2 * right();
#pragma unroll
      for (int b = 0; b < 4; ++b) f(b, rb + (b >> 1), cb + (b & 1), std::true_type());
      return;
    }
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const int at = 4 * (wv - 6) + 2 * d;
      f(3 * d, at, at, std::false_type());
      f(3 * d + 1, at, at + 1, std::true_type());
      f(3 * d + 2, at + 1, at + 1, std::false_type());
    }
  }
  // acc += rows' products with themselves; rows(rb, k, f) gives the parts of row block rb
  template <typename L>
  __device__ __forceinline__ void add(L rows, f32x4_t (&acc)[kMost]) const {
    if (wv < 6) {
      const int ra = 2 * upper(), rb = 2 * right();
      add_products<2, 2>([&](int i, int k, f16x8_t (&f)[2]) { rows(ra + i, k, f); },
                         [&](int j, int k, f16x8_t (&f)[2]) { rows(rb + j, k, f); }, acc);
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        f16x8_t f[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) rows(4 * (wv - 6) + 2 * d + i, k, f[i]);
        auto add = [&](auto q) {
          acc[3 * d] = mfma<q>(f[0], f[0], acc[3 * d]);
          acc[3 * d + 1] = mfma<q>(f[1], f[0], acc[3 * d + 1]);
          acc[3 * d + 2] = mfma<q>(f[1], f[1], acc[3 * d + 2]);
        };
        add(Int<0>());
        add(Int<1>());
        add(Int<2>());
      }
  }
};

template <bool F32>
__global__ __launch_bounds__(512) void whole(SmallArgs g) {
  constexpr int S = 128, MB = 4, NX = 4, NB = 2;   // blocks of a wave: rows, columns of X, of a half or of A
  using M = Parts<S, S>;
  __shared__ __attribute__((aligned(16))) uint8_t sX[HalfX::kBytes];
  __shared__ __attribute__((aligned(16))) uint8_t sA[M::kBytes];
  __shared__ double sums[8];
  __shared__ float coef[64][3];
  const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wv >> 2, wc = wv & 3;
  if (tid < 3 * g.steps) (&coef[0][0])[tid] = (&g.c[0][0])[tid];
  const size_t first = (size_t)blockIdx.x * g.rows * g.cols;
  // X, raw: rows 64 wr + 16 i + ln, columns 128 h + 32 wc + 16 j + 4 lg + r at j + 2 h
  f32x4_t x[MB][NX];
  auto row = [&](int i) { return (wr * MB + i) * 16 + ln; };
  auto column = [&](int j) { return (j >> 1) * kHalf + (wc * NB + (j & 1)) * 16 + lg * 4; };
  const uint32_t down = g.tr ? 1 : g.cols, right = g.tr ? g.rows : 1;
  const void* from = static_cast<const char*>(g.g) + first * (F32 ? 4 : 2);
  double sum = 0.0;
  if (!g.tr && g.cols % 4 == 0) {   // (four columns are neighbours, all of them in or none)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NX; ++j) {
        const uint32_t at = row(i) < g.rows && column(j) < g.cols ? row(i) * down + column(j) : 0;
        if (F32) {
          x[i][j] = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(from) + at);
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(from) + at);
          x[i][j] = f32x4_t{bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
        }
      }
  } else {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NX; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int m = row(i), n = column(j) + r;
          const uint32_t at = m < g.rows && n < g.cols ? m * down + n * right : 0;
          x[i][j][r] = F32 ? static_cast<const float*>(from)[at] : bf16_lo(static_cast<const uint16_t*>(from)[at]);
        }
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NX; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (row(i) >= g.rows || column(j) + r >= g.cols) x[i][j][r] = 0.0f;
        sum = fma((double)x[i][j][r], (double)x[i][j][r], sum);
      }
  sum = wave_sum(sum);
  if (lane == 0) sums[wv] = sum;
  __syncthreads();
  sum = sums[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) sum += sums[w];
  const double f = sum == 0.0 ? 0.0 : (double)kScaleX / sqrt(sum);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NX; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) x[i][j][r] = (float)((double)x[i][j][r] * f);
  // (X is 2^15 times itself, A too, B 2^14 times)
  const bool both = g.cols > kHalf;
  auto put_x = [&](int h) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) HalfX::put4(sX, row(i), column(j), x[i][2 * h + j]);
  };
  const SymBlocks sym{wv};
  auto put_a = [&](const f32x4_t (&v)[SymBlocks::kMost]) {   // those under the diagonal too
    sym.each([&](int b, int rb, int cb, auto over) {
      const uint2 h = make_uint2(pack_f16(v[b][0], v[b][1]), pack_f16(v[b][2], v[b][3]));
      const uint2 l = make_uint2(rest_f16(v[b][0], v[b][1], h.x), rest_f16(v[b][2], v[b][3], h.y));
      M::put_parts(sA, rb * 16 + ln, cb * 16 + lg * 4, h, l);
      if (over)   // (four neighbouring lanes have the same columns)
        M::put_parts(sA, cb * 16 + lg * 4 + (ln & 3), rb * 16 + (ln & ~3), transpose4(h, lane), transpose4(l, lane));
    });
  };
  auto x_rows = [&](int rb, int k, f16x8_t (&f)[2]) { HalfX::rows(sX, rb, k, ln, lg, f); };
  auto a_rows = [&](int rb, int k, f16x8_t (&f)[2]) { M::frags(sA, rb, k, ln, lg, f); };
  for (int s = 0;; ++s) {
    f32x4_t a[SymBlocks::kMost] = {};
    put_x(0);
    __syncthreads();
    const float ca = coef[s][0], cb = coef[s][1], cc = coef[s][2];
    sym.add(x_rows, a);
    if (both) {
      __syncthreads();
      put_x(1);
      __syncthreads();
      sym.add(x_rows, a);
    }
#pragma unroll
    for (int b = 0; b < SymBlocks::kMost; ++b) a[b] *= 1.0f / kScaleX;
    put_a(a);
    __syncthreads();
    f32x4_t aa[SymBlocks::kMost] = {};
    sym.add(a_rows, aa);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < SymBlocks::kMost; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) a[b][r] = __builtin_fmaf(cc * (0.5f / kScaleX), aa[b][r], 0.5f * cb * a[b][r]);
    put_a(a);   // B
    __syncthreads();
    // (the half of X that is in LDS first)
    auto half_step = [&](int h) {
      f32x4_t acc[MB * NB] = {};
      add_products<MB, NB>([&](int i, int k, f16x8_t (&f)[2]) { a_rows(wr * MB + i, k, f); },
                           [&](int j, int k, f16x8_t (&f)[2]) { HalfX::columns(sX, wc * NB + j, k, ln, lg, f); }, acc);
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            x[i][2 * h + j][r] = __builtin_fmaf(ca, x[i][2 * h + j][r], acc[i * NB + j][r] * (2.0f / kScaleX));
    };
    if (both) {
      half_step(1);
      __syncthreads();
      put_x(0);
      __syncthreads();
    }
    half_step(0);
    if (s + 1 == g.steps) break;
    __syncthreads();
  }
  const float scale = g.scale * (1.0f / kScaleX);
  uint16_t* o = static_cast<uint16_t*>(g.out) + first;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      const f32x4_t v = x[i][j] * scale;
      uint2 q = make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{v[0], v[1]}, bf16x2_t)),
                           __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{v[2], v[3]}, bf16x2_t)));
      int at = row(i), col = column(j);   // row and column of memory
      if (g.tr) {
        q = transpose4(q, lane);
        const int n = col + (ln & 3);
        col = at - (ln & 3);
        at = n;
      }
      put_row(o, at, col, g, q);
    }
}

int side(const k3moe_ortho& p) { return std::min(p.m, p.n) <= 64 ? 64 : 128; }

bool in_one(const k3moe_ortho& p) { return side(p) == 128 && std::max(p.m, p.n) <= kBigL; }

// Pieces of X's columns: one more costs `iterate` about half of what a panel costs
// `gram_parts`.
void split(const k3moe_ortho& p, int* chunks, int* panels) {
  const int n = (std::max(p.m, p.n) + 8192 / side(p) - 1) / (8192 / side(p));
  const int want = std::max(1, std::min(64, (int)std::ceil(std::sqrt(2.0 * n))));
  *panels = (n + want - 1) / want;
  *chunks = (n + *panels - 1) / *panels;
}

template <int S, bool F32>
hipError_t launch(const SmallArgs& a, int batch, hipStream_t st) {
  // gram_parts reads along X's rows, apply along its columns: one of them along memory
  const bool whole = (a.tr ? a.rows : a.cols) % 8 == 0;
  const dim3 parts(a.chunks, batch), panels((a.cols + Panel<S>::kW - 1) / Panel<S>::kW, batch);
  if (whole && !a.tr) gram_parts<S, F32, true><<<parts, 1024, 0, st>>>(a);
  else gram_parts<S, F32, false><<<parts, 1024, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  iterate<S><<<batch, Waves<S>::kThreads, 0, st>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (whole && a.tr) apply<S, F32, true><<<panels, 512, 0, st>>>(a);
  else apply<S, F32, false><<<panels, 512, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

bool ortho_small_ok(const k3moe_ortho& p) {
  if (std::min(p.m, p.n) > 128) return false;
  if (in_one(p)) return true;
  double grown = 1.0;
  for (int i = 0; i + 1 < p.steps; ++i) {
    const double a = p.coefficients[3 * i];
    grown *= std::max(1.0, a * a);
  }
  return grown <= 32768.0;
}

OrthoSmallWs carve_ortho_small(const k3moe_ortho& p, void* ws, size_t* bytes) {
  if (in_one(p)) {
    if (bytes) *bytes = 0;
    return OrthoSmallWs{};
  }
  int chunks, panels;
  split(p, &chunks, &panels);
  const size_t ss = (size_t)side(p) * side(p), b = p.batch;
  Carver c(ws);
  OrthoSmallWs w;
  w.part = c.take<float>(b * chunks * ss);
  w.exps = c.take<int>(b * chunks);
  w.poly = c.take<uint16_t>(b * p.steps * 2 * ss);
  w.norm = c.take<float>(2 * b);
  if (bytes) *bytes = c.off;
  return w;
}

hipError_t launch_ortho_small(const k3moe_ortho& p, const void* g, void* out, const OrthoSmallWs& ws, hipStream_t st) {
  SmallArgs a{};
  a.g = g;
  a.part = ws.part;
  a.exps = ws.exps;
  a.poly = ws.poly;
  a.norm = ws.norm;
  a.out = out;
  a.rows = std::min(p.m, p.n);
  a.cols = std::max(p.m, p.n);
  a.tr = p.m > p.n;
  split(p, &a.chunks, &a.panels);
  a.steps = p.steps;
  a.scale = p.scale;
  for (int i = 0; i < p.steps; ++i)
    for (int j = 0; j < 3; ++j) a.c[i][j] = p.coefficients[3 * i + j];
  if (in_one(p)) {
    if (p.dtype == K3MOE_F32) whole<true><<<p.batch, 512, 0, st>>>(a);
    else whole<false><<<p.batch, 512, 0, st>>>(a);
    return hipGetLastError();
  }
  if (p.dtype == K3MOE_F32) return side(p) == 64 ? launch<64, true>(a, p.batch, st) : launch<128, true>(a, p.batch, st);
  return side(p) == 64 ? launch<64, false>(a, p.batch, st) : launch<128, false>(a, p.batch, st);
}

}  // namespace k3
