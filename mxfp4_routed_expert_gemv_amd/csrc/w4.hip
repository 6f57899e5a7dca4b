// Products with 4-bit weights and group scales, for the few tokens of a
// decoding step: out = x W^T with W[r][j] = (q[r][j] - z[r][j / g]) s[r][j / g],
// and the gated form silu(x Wg^T) * (x Wu^T).
//
// The weights are read once, 16 bytes per lane, and feed
// v_mfma_f32_16x16x32_bf16 from registers: 16 weight rows per fragment against
// up to 16 activation rows.  A code q becomes the bf16 value 16 + q by one
// shift and one and-or (0x4180 | q << 3), so per scale group and weight row
//   sum (q - z) x = sum (16 + q) x - (16 + z) sum x,
// with sum x from the same instruction against ones.  All products are exact
// and the sums fp32; the subtraction amplifies their rounding by about
// 24 / 4.6 (the offset over the codes' spread).  An infinity or NaN among a
// group's terms would come out of that difference as NaN whatever its sign, so
// a wave whose sums are not finite repeats its slice with the weights (q - z) s
// themselves, as two exact bf16 parts, which follows the definition.
//
// fp32 activations are three exact bf16 parts (the top 8 significant bits, the
// next 8, the rest), each an activation row of its own, summed at the end.
#include "internal.h"
#include "kern_common.h"

namespace k3 {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;

constexpr int kWaves = 8;   // waves per workgroup, splitting the contraction
constexpr int kBlk = 128;   // contraction elements per 16-byte load of a lane

struct W4Args {
  const uint8_t* codes;    // [n][k / 2]
  const uint16_t* scale;   // [n][k / group] bf16
  const uint8_t* zero;     // [n][k / group], or nullptr: 8
  const void* x;           // [T][k]
  void* out;
  int T, n, k, group, f;   // f: gated form, rows of the gate half; else n
  int out_f32;
};

// 4x4 transpose of dwords across the wave's four rows of 16 lanes: dword j of
// row g becomes dword g of row j.
__device__ __forceinline__ void transpose4(uint32_t (&v)[4]) {
  u32x2_t t;
  t = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false); v[0] = t.x; v[2] = t.y;
  t = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false); v[1] = t.x; v[3] = t.y;
  t = __builtin_amdgcn_permlane16_swap(v[0], v[1], false, false); v[0] = t.x; v[1] = t.y;
  t = __builtin_amdgcn_permlane16_swap(v[2], v[3], false, false); v[2] = t.x; v[3] = t.y;
}

// The 8 codes of a dword as 16 + q, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8_t codes_biased(uint32_t w) {
  uint4 r;
  r.x = ((w << 3) & 0x00780078u) | 0x41804180u;
  r.y = ((w >> 1) & 0x00780078u) | 0x41804180u;
  r.z = ((w >> 5) & 0x00780078u) | 0x41804180u;
  r.w = ((w >> 9) & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(bf16x8_t, r);
}
// The weights (q - z) s themselves in the same order, as two bf16 parts of one
// sign whose sum is exact: q - z has at most 8 significant bits, a bf16 scale 8,
// so the product 16.  Neither part is zero unless the weight is (a weight of 8
// bits is halved), and an infinite or NaN weight is both: a part times an
// infinity is what the weight times it is.
__device__ __forceinline__ void codes_exact(uint32_t w, int z, float s, bf16x8_t& hi, bf16x8_t& lo) {
  uint32_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int shift = 4 * (i >> 1) + 16 * (i & 1);
    const float v = (float)((int)((w >> shift) & 15u) - z) * s;
    const float top = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    const bool whole = !(fabsf(v - top) > 0.0f);   // 8 bits, or not finite
    const float a = whole ? 0.5f * v : top;
    h[i] = f32_to_bf16(a);
    l[i] = f32_to_bf16(whole ? a : v - top);
  }
  hi = __builtin_bit_cast(bf16x8_t, make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16,
                                               h[4] | h[5] << 16, h[6] | h[7] << 16));
  lo = __builtin_bit_cast(bf16x8_t, make_uint4(l[0] | l[1] << 16, l[2] | l[3] << 16,
                                               l[4] | l[5] << 16, l[6] | l[7] << 16));
}

// Part p (0, 1, 2) of an fp32 value as bf16 bits: the value is the sum of its
// three parts (an infinity or NaN is its first part's).
__device__ __forceinline__ uint32_t part_of(float v, int p) {
  const uint32_t u = __float_as_uint(v);
  const bool special = (u & 0x7F800000u) == 0x7F800000u;
  // a NaN whose payload lies in the low bits alone would truncate to infinity
  const uint32_t hi = special && (u & 0x007FFFFFu) ? u | 0x00400000u : u;
  if (p == 0) return hi >> 16;
  if (special) return 0;
  const float r1 = v - __uint_as_float(u & 0xFFFF0000u);
  const uint32_t u1 = __float_as_uint(r1);
  if (p == 1) return u1 >> 16;
  return __float_as_uint(r1 - __uint_as_float(u1 & 0xFFFF0000u)) >> 16;
}

// Activation row r of the workgroup (bf16: token r; fp32: part r % 3 of token
// r / 3), elements k .. k + 8, in the codes' order; zeros for rows past the
// last token and elements past the contraction.
template <bool F32X>
__device__ __forceinline__ bf16x8_t x_frag(const W4Args& g, int t0, int r, int k) {
  const int t = t0 + (F32X ? r / 3 : r);
  uint4 v = make_uint4(0, 0, 0, 0);
  if (t < g.T && k < g.k) {
    if (F32X) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(g.x) + (size_t)t * g.k + k);
      const float4 a = p[0], b = p[1];
      const int q = r % 3;
      v.x = part_of(a.x, q) | (part_of(b.x, q) << 16);
      v.y = part_of(a.y, q) | (part_of(b.y, q) << 16);
      v.z = part_of(a.z, q) | (part_of(b.z, q) << 16);
      v.w = part_of(a.w, q) | (part_of(b.w, q) << 16);
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.x) + (size_t)t * g.k + k);
      v.x = (w.x & 0xFFFFu) | (w.z << 16);
      v.y = (w.x >> 16) | (w.z & 0xFFFF0000u);
      v.z = (w.y & 0xFFFFu) | (w.w << 16);
      v.w = (w.y >> 16) | (w.w & 0xFFFF0000u);
    }
  }
  return __builtin_bit_cast(bf16x8_t, v);
}

// One wave's slice of the contraction (blocks wv, wv + kWaves, ...) for MB x 16
// activation rows and NF x 16 weight rows.  SG: 32-element steps per scale.
template <int MB, int NF, int SG, bool F32X, bool EXACT>
__device__ __forceinline__ void w4_slice(const W4Args& g, int t0, int wv, int ln, int lg,
                                         const int (&row)[NF], f32x4_t (&acc)[MB][NF]) {
  const f32x4_t nil = {0.f, 0.f, 0.f, 0.f};
  const int groups = g.k / g.group;
  bf16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = nil;
  const int nblk = (g.k + kBlk - 1) / kBlk;
#pragma unroll 1
  for (int blk = wv; blk < nblk; blk += kWaves) {
    const int k0 = blk * kBlk;
    uint32_t c[NF][4];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      // (the last block may end inside: those lanes read the row's last 16
      // bytes, against activations of zero)
      const int kk = min(k0 + 32 * lg, g.k - 32);
      const uint4 v = ldg16(g.codes + (size_t)row[f] * (g.k >> 1) + (kk >> 1));
      c[f][0] = v.x; c[f][1] = v.y; c[f][2] = v.z; c[f][3] = v.w;
      transpose4(c[f]);
    }
#pragma unroll
    for (int s = 0; s < 4 / SG; ++s) {
      const int gi = min((k0 + s * SG * 32) / g.group, groups - 1);
      float sc[NF];
      int z[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const size_t o = (size_t)row[f] * groups + gi;
        sc[f] = __uint_as_float((uint32_t)g.scale[o] << 16);
        z[f] = g.zero ? g.zero[o] : 8;
      }
      f32x4_t dot[MB][NF], sum[MB];
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        sum[m] = nil;
#pragma unroll
        for (int f = 0; f < NF; ++f) dot[m][f] = nil;
      }
#pragma unroll
      for (int j = s * SG; j < (s + 1) * SG; ++j) {
        bf16x8_t b[NF], b_lo[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          if (EXACT) codes_exact(c[f][j], z[f], sc[f], b[f], b_lo[f]);
          else b[f] = codes_biased(c[f][j]);
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          const bf16x8_t a = x_frag<F32X>(g, t0, m * 16 + ln, k0 + 32 * j + 8 * lg);
          if (!EXACT) sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, sum[m], 0, 0, 0);
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            if (EXACT) dot[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b_lo[f], dot[m][f], 0, 0, 0);
            dot[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[f], dot[m][f], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const float off = -(float)(16 + z[f]);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[m][f][r] = EXACT ? acc[m][f][r] + dot[m][f][r]
                                 : __builtin_fmaf(sc[f], __builtin_fmaf(off, sum[m][r], dot[m][f][r]),
                                                  acc[m][f][r]);
      }
    }
  }
}

// Workgroup (blockIdx.x, blockIdx.y): 16 NF weight rows (gated form: 8 NF gate
// rows and the matching up rows) x the tokens of 16 MB activation rows.
template <int MB, int NF, int SG, bool F32X, bool GLU>
__global__ __launch_bounds__(64 * kWaves) void w4_kernel(W4Args g) {
  constexpr int TOK = F32X ? 16 * MB / 3 : 16 * MB;   // tokens per workgroup
  constexpr int NB = GLU ? 8 * NF : 16 * NF;          // outputs per token
  static_assert(!GLU || NF % 2 == 0, "gate and up fragments come in pairs");
  __shared__ float red[kWaves][16 * MB][16 * NF + 1];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, ln = lane & 15, lg = lane >> 4;
  const int t0 = blockIdx.y * TOK, n0 = blockIdx.x * NB;
  int row[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f)   // (rows past the last are read as it, and not stored)
    row[f] = GLU ? min(n0 + (f % (NF / 2)) * 16 + ln, g.f - 1) + (f >= NF / 2 ? g.f : 0)
                 : min(n0 + f * 16 + ln, g.n - 1);
  f32x4_t acc[MB][NF];
  w4_slice<MB, NF, SG, F32X, false>(g, t0, wv, ln, lg, row, acc);
  bool bad = false;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r) bad |= !(fabsf(acc[m][f][r]) < INFINITY);
  if (__any(bad)) w4_slice<MB, NF, SG, F32X, true>(g, t0, wv, ln, lg, row, acc);
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[wv][m * 16 + lg * 4 + r][f * 16 + ln] = acc[m][f][r];
  __syncthreads();
  // sum over the waves in order (and over an fp32 value's parts, largest first)
  const int tn = min(TOK, g.T - t0);
  for (int i = threadIdx.x; i < tn * NB; i += 64 * kWaves) {
    const int t = i / NB, c = i - t * NB;
    if (n0 + c >= (GLU ? g.f : g.n)) continue;
    float v[GLU ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (GLU ? 2 : 1); ++h) {
      float sum = 0.f;
#pragma unroll
      for (int p = 0; p < (F32X ? 3 : 1); ++p)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += red[w][F32X ? t * 3 + p : t][c + h * NB];
      v[h] = sum;
    }
    const float o = GLU ? silu_mul(v[0], v[GLU ? 1 : 0]) : v[0];
    const size_t at = (size_t)(t0 + t) * (GLU ? g.f : g.n) + n0 + c;
    if (g.out_f32) static_cast<float*>(g.out)[at] = o;
    else static_cast<uint16_t*>(g.out)[at] = f32_to_bf16(o);
  }
}

template <int MB, int NF, int SG, bool F32X, bool GLU>
hipError_t launch5(const W4Args& g, hipStream_t st) {
  constexpr int TOK = F32X ? 16 * MB / 3 : 16 * MB, NB = GLU ? 8 * NF : 16 * NF;
  const dim3 grid(((GLU ? g.f : g.n) + NB - 1) / NB, (g.T + TOK - 1) / TOK);
  w4_kernel<MB, NF, SG, F32X, GLU><<<grid, 64 * kWaves, 0, st>>>(g);
  return hipGetLastError();
}
template <int MB, int NF, bool F32X, bool GLU>
hipError_t launch4(const W4Args& g, hipStream_t st) {
  if (g.group == 32) return launch5<MB, NF, 1, F32X, GLU>(g, st);
  if (g.group == 64) return launch5<MB, NF, 2, F32X, GLU>(g, st);
  return launch5<MB, NF, 4, F32X, GLU>(g, st);   // a multiple of 128
}
template <bool F32X, bool GLU>
hipError_t launch2(const W4Args& g, hipStream_t st) {
  const long rows = (long)g.T * (F32X ? 3 : 1);
  if (rows <= (F32X ? 15 : 16)) return launch4<1, 2, F32X, GLU>(g, st);
  return launch4<4, 2, F32X, GLU>(g, st);
}

}  // namespace

hipError_t launch_w4(const k3moe_w4_matrix& w, int64_t T, bool x_f32, bool out_f32, bool glu,
                     const void* x, void* out, hipStream_t st) {
  W4Args g;
  g.codes = static_cast<const uint8_t*>(w.codes);
  g.scale = static_cast<const uint16_t*>(w.scale);
  g.zero = static_cast<const uint8_t*>(w.zero);
  g.x = x;
  g.out = out;
  g.T = (int)T;
  g.n = w.n;
  g.k = w.k;
  g.group = w.group;
  g.f = glu ? w.n / 2 : w.n;
  g.out_f32 = out_f32;
  if (x_f32) return glu ? launch2<true, true>(g, st) : launch2<true, false>(g, st);
  return glu ? launch2<false, true>(g, st) : launch2<false, false>(g, st);
}

}  // namespace k3
