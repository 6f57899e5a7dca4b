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
// 24 / 4.6 (the offset over the codes' spread), and more where x has a mean.  With
// fp32 x and outputs it is therefore taken after every 32 weights, before the sums
// have grown: the error is 0.8 to 1.7 times that of a plain fp32 product (4096 terms,
// x of spread 1 and mean 0 to 20), against 1.6 to 7.5 with one subtraction per group of
// 128, for 3 to 12 % of the time (5 tokens gated 2 x 2049 x 7168 13.0 -> 13.5 us, 64
// tokens 8192 x 4096 30.3 -> 33.3).  With bf16 x or outputs, whose own rounding is
// 2^-8, it is taken once per scale of a block.  An infinity or NaN among a
// group's terms would come out of that difference as NaN whatever its sign, so
// a wave whose sums are not finite repeats its slice with the weights (q - z) s
// themselves, as two exact bf16 parts, which follows the definition.
//
// What bounds them, at one token 7168 x 4096, group 128 (15 MB from HBM): 7.0 us, of
// which a launch is 2.3 and the codes at a large copy's rate 3.2; 16384 x 16384
// (134 MB and scales) 38.8 us, 3.6 TB/s.  From about 32 tokens on what a CU has to bring of x
// into LDS weighs more than the weights.
//
// fp32 activations enter as three exact bf16 parts (the top 8 significant bits,
// the next 8, the rest), one instruction each into the same sums.
#include <algorithm>

#include "internal.h"
#include "kern_common.h"
#include "grouped.h"

namespace k3 {
namespace {

using grouped::wait_lds;
using grouped::wait_vmem;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;

constexpr int kBlk = 128;   // contraction elements per 16-byte load of a lane

struct W4Args {
  const uint8_t* codes;    // [n][k / 2]
  const uint16_t* scale;   // [n][k / group] bf16
  const uint8_t* zero;     // [n][k / group], or nullptr: 8
  const void* x;           // [T][k]
  void* out;
  int T, n, k, f;          // f: gated form, rows of the gate half; else n
  int groups;              // scales of a row
  uint32_t per_group;      // blocks / (group / 128) = umulhi(blocks, per_group); 0: group 128
  int out_f32;
  float* part;             // more than 16 tokens: partial sums [splits][T][n]
  int splits, per_split;   // pieces of the contraction, blocks of a piece
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

// The 8 codes of a dword as 16 + q, in order: of byte b, the low nibble sits at
// bits 3 .. 6 of w << 3's byte b, the high one there in w >> 1's.
__device__ __forceinline__ bf16x8_t codes_biased(uint32_t w) {
  const uint32_t lo = w << 3, hi = w >> 1;
  uint4 r;   // (0x0C selects a zero byte; the second operand's bytes are 0 .. 3)
  r.x = (__builtin_amdgcn_perm(hi, lo, 0x0C040C00u) & 0x00780078u) | 0x41804180u;
  r.y = (__builtin_amdgcn_perm(hi, lo, 0x0C050C01u) & 0x00780078u) | 0x41804180u;
  r.z = (__builtin_amdgcn_perm(hi, lo, 0x0C060C02u) & 0x00780078u) | 0x41804180u;
  r.w = (__builtin_amdgcn_perm(hi, lo, 0x0C070C03u) & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(bf16x8_t, r);
}
// The weights (q - z) s themselves, as two bf16 parts of one
// sign whose sum is exact: q - z has at most 8 significant bits, a bf16 scale 8,
// so the product 16.  Neither part is zero unless the weight is (a weight of 8
// bits is halved), and an infinite or NaN weight is both: a part times an
// infinity is what the weight times it is.
__device__ __forceinline__ void codes_exact(uint32_t w, int z, float s, bf16x8_t& hi, bf16x8_t& lo) {
  uint32_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = (float)((int)((w >> (4 * i)) & 15u) - z) * s;
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

// Eight activations as fragments whose sum is exact: bf16 as they are; fp32 as the top
// 8 significant bits, the next 8 and the rest.
// SPECIAL: an infinity or NaN is every part, and no part is zero unless the
// value is, so that a part times an infinite weight is what the value times it
// is (otherwise an infinity or NaN is the first part's alone or all of them).
template <bool F32X, bool SPECIAL>
__device__ __forceinline__ void x_frags(const uint4* x, bf16x8_t (&out)[F32X ? 3 : 1]) {
  if constexpr (F32X) {
    const uint4 a = x[0], b = x[1];
    const uint32_t in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = __uint_as_float(in[i]);
      const float hi = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u), r1 = v - hi;
      const float mid = __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u), lo = r1 - mid;
      float q[3] = {hi, mid, lo};
      if (SPECIAL) {
        if (!(fabsf(v) < INFINITY)) {
          q[0] = q[1] = q[2] = v != v ? __uint_as_float(0x7FC00000u) : v;
        } else if (r1 == 0.0f) {
          q[0] = 0.5f * v; q[1] = q[2] = 0.25f * v;
        } else if (lo == 0.0f) {
          q[1] = q[2] = 0.5f * r1;
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) p[k][i] = __float_as_uint(q[k]);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      out[k] = __builtin_bit_cast(
          bf16x8_t, make_uint4(__builtin_amdgcn_perm(p[k][1], p[k][0], 0x07060302u),
                               __builtin_amdgcn_perm(p[k][3], p[k][2], 0x07060302u),
                               __builtin_amdgcn_perm(p[k][5], p[k][4], 0x07060302u),
                               __builtin_amdgcn_perm(p[k][7], p[k][6], 0x07060302u)));
  } else {
    out[0] = __builtin_bit_cast(bf16x8_t, x[0]);
  }
}

// The weights' side of one 128-element block, as loaded.
template <int NF, int SG>
struct Codes {
  uint4 c[NF];               // 32 codes per lane: elements 32 lg .. + 32 of row ln
  uint16_t s[4 / SG][NF];    // a scale for every SG steps of 32 elements
  uint8_t z[4 / SG][NF];
};

// A lane's rows: fragment f's weight row, and its token.
template <int NF>
struct Rows {
  int row[NF], tok, lg;
};

// The scale of step group s (of SG steps) of block blk in a row's list.
template <int SG>
__device__ __forceinline__ int group_of(const W4Args& g, int blk, int s) {
  return SG < 4 ? min(blk * (4 / SG) + s, g.groups - 1)
                : (g.per_group ? (int)__umulhi((uint32_t)blk, g.per_group) : blk);
}

// (lanes past the contraction read its last 32 elements, which no step uses)
template <int NF, int SG>
__device__ __forceinline__ void load_codes(const W4Args& g, int blk, const Rows<NF>& r,
                                           Codes<NF, SG>& b) {
  const int kc = min(blk * kBlk + 32 * r.lg, g.k - 32);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    b.c[f] = ldg16(g.codes + (size_t)r.row[f] * (g.k >> 1) + (kc >> 1));
#pragma unroll
    for (int s = 0; s < 4 / SG; ++s) {
      const size_t o = (size_t)r.row[f] * g.groups + group_of<SG>(g, blk, s);
      b.s[s][f] = g.scale[o];
      b.z[s][f] = g.zero ? g.zero[o] : 8;
    }
  }
}

// The activations of one block: step j of lane (ln, lg) is row ln, elements
// 32 j + 8 lg .. + 8.
template <bool F32X>
struct Acts {
  uint4 v[4][F32X ? 2 : 1];
};
template <bool F32X, int NF>
__device__ __forceinline__ void load_acts(const W4Args& g, int blk, const Rows<NF>& r, Acts<F32X>& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const size_t o = (size_t)r.tok * g.k + min(blk * kBlk + 32 * j, g.k - 32) + 8 * r.lg;
    const uint8_t* p = static_cast<const uint8_t*>(g.x) + o * (F32X ? 4 : 2);
    b.v[j][0] = ldg16(p);
    if constexpr (F32X) b.v[j][1] = ldg16(p + 16);
  }
}

// A wave's blocks (blk0, blk0 + step, ... below blk1) with the weights
// themselves: for sums that are not finite.
template <int NF, int SG, bool F32X>
__device__ __noinline__ void w4_slice_exact(const W4Args g, int blk0, int blk1, int step,
                                            const Rows<NF> rows, f32x4_t (&acc)[NF]) {
  constexpr int XP = F32X ? 3 : 1;
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int blk = blk0; blk < blk1; blk += step) {
    Codes<NF, SG> c;
    load_codes<NF, SG>(g, blk, rows, c);
    uint32_t t[NF][4];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      t[f][0] = c.c[f].x; t[f][1] = c.c[f].y; t[f][2] = c.c[f].z; t[f][3] = c.c[f].w;
      transpose4(t[f]);
    }
    Acts<F32X> x;
    load_acts<F32X, NF>(g, blk, rows, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (blk * kBlk + 32 * j >= g.k) break;
      bf16x8_t a[XP];
      x_frags<F32X, true>(x.v[j], a);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        bf16x8_t hi, lo;
        codes_exact(t[f][j], c.z[j / SG][f], bf16_lo(c.s[j / SG][f]), hi, lo);
#pragma unroll
        for (int p = 0; p < XP; ++p) {
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], lo, acc[f], 0, 0, 0);
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], hi, acc[f], 0, 0, 0);
        }
      }
    }
  }
}

// ---- few tokens.  A workgroup's W waves split the contraction in blocks of 128
// (wave w takes blocks w, w + W, ...); a wave copies its blocks into a ring of D
// slots of its own by LDS-DMA, so that D blocks of every wave are in flight
// whatever the registers hold, and no wave waits for another before the sum at
// the end.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// LDS-DMA copies from base + off: lane i's 16 bytes (dword; two bytes, one byte, as
// a dword) land at lds + 16 i (4 i).
__device__ __forceinline__ void dma_b128(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma_b32(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma_u16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ushort %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma_u8(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

// Slot of a block, for RC tokens and 16 NF weight rows:
//   codes  [16 NF rows][4 units of 16 bytes], unit u of row r at u ^ code_swz(r)
//   x      [RC rows][16 (fp32: 32) units], unit u of row r at u ^ (r mod 16)
//   scale  [4 / SG][16 NF] dwords, then zero the same; WIDE (groups of 32, four of
//     them a block at a time, whose addresses are then whole dwords): scale [16 NF]
//     [4] bf16, then zero [16 NF][4] bytes, half of the copies or less (64 tokens
//     7168 x 4096: 18.4 us against 20.8; 32 tokens 16384 x 4096: 26.1, 30.0)
// The permutations spread the 16 rows of a fragment read over the LDS banks.
template <int RC, int NF, int SG, bool F32X, bool WIDE>
struct Slot {
  static_assert(!WIDE || SG == 1, "four scales a block");
  static constexpr int kRow = F32X ? 512 : 256;             // bytes of x per token
  static constexpr int kX = NF * 1024, kS = kX + RC * kRow;
  static constexpr int kVals = WIDE ? 2 * 16 * NF : 4 / SG * 16 * NF;   // dwords of scales
  static constexpr int kZeros = WIDE ? 16 * NF : kVals;
  static constexpr int NS = (kVals + 63) / 64, NZ = (kZeros + 63) / 64;   // copies
  static constexpr int kZ = kS + NS * 256, kBytes = kZ + NZ * 256;
  static constexpr int NX = RC * kRow / 1024;               // copies of x
  static constexpr int kCopies = NF + NX + NS + NZ;
};
// Scales, and 16 + zero points negated, of a row's four groups of 32.
__device__ __forceinline__ void wide_values(const uint8_t* scale, const uint8_t* zero, bool has_zero,
                                            float (&sc)[4], float (&off)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(scale);
  const uint32_t z = has_zero ? *reinterpret_cast<const uint32_t*>(zero) : 0x08080808u;
  sc[0] = bf16_lo(w.x); sc[1] = bf16_hi(w.x); sc[2] = bf16_lo(w.y); sc[3] = bf16_hi(w.y);
#pragma unroll
  for (int s = 0; s < 4; ++s) off[s] = -(float)(16 + (z >> (8 * s) & 255u));
}
__device__ __forceinline__ int code_swz(int r) { return ((r >> 1) & 2) ^ ((r >> 3) & 1) * 3; }

// Workgroup blockIdx.x: 16 NF weight rows (gated form: 8 NF gate
// rows and the matching up rows) x RC tokens.  The offset is taken off after every FS
// steps of 32.
template <int W, int D, int RC, int NF, int SG, int FS, bool F32X, bool WIDE, bool GLU>
__global__ __launch_bounds__(64 * W) void w4_kernel(W4Args g) {
  using L = Slot<RC, NF, SG, F32X, WIDE>;
  constexpr int NB = GLU ? 8 * NF : 16 * NF;   // outputs per token
  constexpr int XP = F32X ? 3 : 1, MB = (RC + 15) / 16;   // fragments of tokens
  static_assert(!GLU || NF % 2 == 0, "gate and up fragments come in pairs");
  static_assert(RC * (16 * NF + 1) * 4 <= D * L::kBytes, "a wave's sums fit its ring");
  __shared__ __attribute__((aligned(16))) uint8_t ring[W][D * L::kBytes];
  const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_out = GLU ? g.f : g.n;
  const int n0 = blockIdx.x * NB, tn = g.T;
  // row of the workgroup's row i (rows past the last are read as it, and not stored)
  auto weight_row = [&](int i) {
    const int f = i >> 4, first = n0 + (GLU ? f % (NF / 2) : f) * 16;
    return min(first + (i & 15), n_out - 1) + (GLU && f >= NF / 2 ? g.f : 0);
  };

  // ---- copies: offsets from the wave's first block, in the arrays' rows
  const int kb = g.k >> 1;   // bytes of a row of codes
  uint32_t oc[NF], ox[L::NX], os[L::NS], oz[L::NZ];
  int kc[NF], kx[L::NX], vs[L::NS];
  const int row_lo = weight_row(0);
  const size_t up_rows = GLU ? (size_t)g.f : 0;   // fragments of the up half start there
#pragma unroll
  for (int c = 0; c < NF; ++c) {
    const int r = lane >> 2;
    kc[c] = ((lane & 3) ^ code_swz(r)) * 32;
    oc[c] = (uint32_t)(weight_row(c * 16 + r) - row_lo - (GLU && c >= NF / 2 ? g.f : 0)) * (uint32_t)kb;
  }
#pragma unroll
  for (int c = 0; c < L::NX; ++c) {
    constexpr int U = L::kRow / 16;   // units per token
    const int i = c * 64 + lane, r = i / U, u = (i % U) ^ (r & 15);
    kx[c] = u * (F32X ? 4 : 8);
    ox[c] = (uint32_t)min(r, tn - 1) * (uint32_t)g.k;
  }
  // (in scales from the first row's; the up half's rows are further than the gate's)
  auto scale_row = [&](int i) {
    const uint32_t r = (uint32_t)(weight_row(i) - row_lo - (GLU && (i >> 4) >= NF / 2 ? g.f : 0));
    return (r + (GLU && (i >> 4) >= NF / 2 ? (uint32_t)up_rows : 0u)) * (uint32_t)g.groups;
  };
#pragma unroll
  for (int c = 0; c < L::NS; ++c) {
    const int i = min(c * 64 + lane, L::kVals - 1);
    vs[c] = WIDE ? (i & 1) * 2 : i / (16 * NF);
    os[c] = scale_row(WIDE ? i >> 1 : i % (16 * NF));
  }
#pragma unroll
  for (int c = 0; c < L::NZ; ++c)
    oz[c] = WIDE ? scale_row(min(c * 64 + lane, 16 * NF - 1)) : os[c];
  const uint32_t my = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)ring[wv];
  const int nblk = (g.k + kBlk - 1) / kBlk;
  const uint8_t* const zeros = g.zero ? g.zero : reinterpret_cast<const uint8_t*>(g.scale);
  auto issue = [&](int b, int slot) {
    if (b >= nblk) return;
    const int k0 = b * kBlk;
    const uint32_t to = __builtin_amdgcn_readfirstlane(my + slot * L::kBytes);
    const int left = g.k - 32 - k0;   // codes past the row's end: its last 32, not used
#pragma unroll
    for (int c = 0; c < NF; ++c)
      dma_b128(g.codes + ((size_t)row_lo + (GLU && c >= NF / 2 ? up_rows : 0)) * kb + (k0 >> 1),
               oc[c] + (uint32_t)(min(kc[c], left) >> 1), to + c * 1024);
    const uint8_t* x = static_cast<const uint8_t*>(g.x) + (size_t)k0 * (F32X ? 4 : 2);
#pragma unroll
    for (int c = 0; c < L::NX; ++c)
      dma_b128(x, (ox[c] + (uint32_t)min(kx[c], g.k - (F32X ? 4 : 8) - k0)) * (F32X ? 4 : 2),
               to + L::kX + c * 1024);
    const uint16_t* const s_lo = g.scale + (size_t)row_lo * g.groups;
    const uint8_t* const z_lo = zeros + (size_t)row_lo * g.groups;
    if constexpr (WIDE) {
#pragma unroll
      for (int c = 0; c < L::NS; ++c)
        dma_b32(s_lo, (os[c] + (uint32_t)(b * 4 + vs[c])) * 2, to + L::kS + c * 256);
#pragma unroll
      for (int c = 0; c < L::NZ; ++c) dma_b32(z_lo, oz[c] + (uint32_t)(b * 4), to + L::kZ + c * 256);
    } else {
#pragma unroll
      for (int c = 0; c < L::NS; ++c) {
        const uint32_t o = os[c] + (uint32_t)(SG < 4 ? min(b * (4 / SG) + vs[c], g.groups - 1)
                                                     : group_of<SG>(g, b, 0));
        dma_u16(s_lo, o * 2, to + L::kS + c * 256);
        dma_u8(z_lo, o, to + L::kZ + c * 256);
      }
    }
  };

  const f32x4_t nil = {0.f, 0.f, 0.f, 0.f};
  f32x4_t acc[MB][NF];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = nil;
  bf16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;
#pragma unroll
  for (int q = 0; q < D; ++q) issue(wv + q * W, q);
  int slot = 0;
#pragma unroll 1
  for (int blk = wv; blk < nblk; blk += W) {
    // (towards the end fewer are in flight: wait for all)
    if (blk + (D - 1) * W < nblk) wait_vmem<(D - 1) * L::kCopies>();
    else wait_vmem<0>();
    const uint8_t* at = ring[wv] + slot * L::kBytes;
    uint32_t c[NF][4];
    uint4 x[MB][4][F32X ? 2 : 1];
    float sc[NF][4 / SG], off[NF][4 / SG];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const uint4 v = *reinterpret_cast<const uint4*>(at + f * 1024 + ln * 64 + ((lg ^ code_swz(ln)) << 4));
      c[f][0] = v.x; c[f][1] = v.y; c[f][2] = v.z; c[f][3] = v.w;
      if constexpr (WIDE) {
        const int r = f * 16 + ln;
        wide_values(at + L::kS + r * 8, at + L::kZ + r * 4, g.zero, sc[f], off[f]);
      } else {
#pragma unroll
        for (int s = 0; s < 4 / SG; ++s) {
          const int i = ((s * NF + f) * 16 + ln) * 4;
          sc[f][s] = bf16_lo(*reinterpret_cast<const uint32_t*>(at + L::kS + i));
          const int z = g.zero ? *reinterpret_cast<const int*>(at + L::kZ + i) : 8;
          off[f][s] = -(float)(16 + z);
        }
      }
    }
    const int xr = ln & (RC - 1);   // (rows past RC repeat one of them)
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < (F32X ? 2 : 1); ++h) {
          const int u = F32X ? 8 * j + 2 * lg + h : 4 * j + lg;
          x[m][j][h] = *reinterpret_cast<const uint4*>(at + L::kX + (m * 16 + xr) * L::kRow + ((u ^ xr) << 4));
        }
    // the slot is in registers: its next block may come
    wait_lds();
    issue(blk + D * W, slot);
    slot = slot == D - 1 ? 0 : slot + 1;
#pragma unroll
    for (int f = 0; f < NF; ++f) transpose4(c[f]);
#pragma unroll
    for (int s = 0; s < 4 / FS; ++s) {
      if (blk * kBlk + s * FS * 32 >= g.k) break;
      f32x4_t sum[MB], dot[MB][NF];
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        sum[m] = nil;
#pragma unroll
        for (int f = 0; f < NF; ++f) dot[m][f] = nil;
      }
#pragma unroll
      for (int j = s * FS; j < (s + 1) * FS; ++j) {
        bf16x8_t w[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) w[f] = codes_biased(c[f][j]);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          bf16x8_t a[XP];
          x_frags<F32X, false>(x[m][j], a);
#pragma unroll
          for (int p = 0; p < XP; ++p) {
            sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], ones, sum[m], 0, 0, 0);
#pragma unroll
            for (int f = 0; f < NF; ++f)
              dot[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], w[f], dot[m][f], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[m][f][r] = __builtin_fmaf(sc[f][s * FS / SG],
                                          __builtin_fmaf(off[f][s * FS / SG], sum[m][r], dot[m][f][r]),
                                          acc[m][f][r]);
    }
  }
  bool bad = false;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        bad |= m * 16 + lg * 4 + r < tn && !(fabsf(acc[m][f][r]) < INFINITY);
  if (__any(bad)) {
    Rows<NF> rows;
    rows.lg = lg;
#pragma unroll
    for (int f = 0; f < NF; ++f) rows.row[f] = weight_row(f * 16 + ln);
#pragma unroll 1
    for (int m = 0; m < MB; ++m) {
      rows.tok = min(m * 16 + ln, tn - 1);
      f32x4_t again[NF];   // (acc's own address would keep it out of registers)
      w4_slice_exact<NF, SG, F32X>(g, wv, nblk, W, rows, again);
#pragma unroll
      for (int q = 0; q < MB; ++q)
        if (q == m) {
#pragma unroll
          for (int f = 0; f < NF; ++f) acc[q][f] = again[f];
        }
    }
  }
  // ---- the waves' sums, each in its own ring (nothing is in flight to it any more)
  float* red = reinterpret_cast<float*>(ring[wv]);
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = m * 16 + lg * 4 + r;
        if (t < tn) red[t * (16 * NF + 1) + f * 16 + ln] = acc[m][f][r];
      }
  __syncthreads();
  for (int i = threadIdx.x; i < tn * NB; i += 64 * W) {
    const int t = i / NB, col = i - t * NB;
    if (n0 + col >= n_out) continue;
    float v[GLU ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (GLU ? 2 : 1); ++h) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w)
        sum += reinterpret_cast<const float*>(ring[w])[t * (16 * NF + 1) + col + h * NB];
      v[h] = sum;
    }
    const float o = GLU ? silu_mul(v[0], v[GLU ? 1 : 0]) : v[0];
    const size_t at = (size_t)t * n_out + n0 + col;
    if (g.out_f32) static_cast<float*>(g.out)[at] = o;
    else static_cast<uint16_t*>(g.out)[at] = f32_to_bf16(o);
  }
}

// ---- more tokens.  Here the activations are the larger operand of a workgroup, so
// its 8 waves share them: 128 weight rows, 16 MB tokens and one of
// g.splits pieces of the contraction, whose fp32 sums w4_finish adds in order.  A
// step takes two blocks of 128: waves 0 .. 3 the first, 4 .. 7 the second, 32 rows
// each, so that a fragment of x read from LDS and its sum serve two fragments of
// weights; the two halves are added through LDS at the end.  One ring of steps, one
// barrier a step.
template <int MB, int SG, bool F32X, bool WIDE>
struct TileSlot {
  static constexpr int kRow = F32X ? 512 : 256;        // bytes of x per token and block
  static constexpr int XC = 16 * MB * kRow / 8192;     // copies of x per wave and block
  static constexpr int kX = 8192, kBlock = kX + 16 * MB * kRow;   // codes, then x
  // scales: [two blocks][4 / SG][128 rows] dwords, then zero the same; WIDE: [two
  // blocks][128 rows][4] bf16, then zero [two blocks][128 rows][4] bytes
  static constexpr int kVals = WIDE ? 512 : 2 * (4 / SG) * 128, kZeros = WIDE ? 256 : kVals;
  static constexpr int kS = 2 * kBlock, kZ = kS + kVals * 4, kBytes = kZ + kZeros * 4;
  static constexpr int kCopies = 2 * (1 + XC) + (WIDE ? 2 : kVals / 256);
  static constexpr int kStages = (160 << 10) / kBytes < 3 ? (160 << 10) / kBytes : 3;
  static_assert(XC * 8192 == 16 * MB * kRow && kStages >= 2, "whole copies, two steps in LDS");
};

template <int MB, int SG, int FS, bool F32X, bool WIDE>
__global__ __launch_bounds__(512) void w4_tile(W4Args g) {
  using L = TileSlot<MB, SG, F32X, WIDE>;
  constexpr int XP = F32X ? 3 : 1, kStages = L::kStages;
  constexpr int kRed = 132;   // (a row of the sums; 4 rows apart: 16 banks)
  static_assert(16 * MB * kRed * 4 <= kStages * L::kBytes, "the sums fit the ring");
  __shared__ __attribute__((aligned(16))) uint8_t ring[kStages * L::kBytes];
  const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wk = wv >> 2, wn = wv & 3;
  const int t0 = blockIdx.z * (16 * MB), n0 = blockIdx.x * 128, tn = min(16 * MB, g.T - t0);
  if (n0 >= g.n) return;
  const int nblk = (g.k + kBlk - 1) / kBlk;
  const int b0 = blockIdx.y * g.per_split, b1 = min(b0 + g.per_split, nblk);
  const int steps = (b1 - b0 + 1) >> 1;
  const int last = g.n - 1 - n0;   // rows past it: read as it, not stored
  const int kb = g.k >> 1;
  const int cr = lane >> 2, ck = ((lane & 3) ^ code_swz(cr)) * 32;
  const uint32_t oc = (uint32_t)min(wv * 16 + cr, last) * (uint32_t)kb;
  uint32_t ox[L::XC];
  int kx[L::XC];
#pragma unroll
  for (int c = 0; c < L::XC; ++c) {
    constexpr int U = L::kRow / 16;
    const int i = (wv * L::XC + c) * 64 + lane, r = i / U, u = (i % U) ^ (r & 15);
    kx[c] = u * (F32X ? 4 : 8);
    ox[c] = (uint32_t)min(r, tn - 1) * (uint32_t)g.k;
  }
  const uint8_t* const codes = g.codes + (size_t)n0 * kb;
  const uint16_t* const scale = g.scale + (size_t)n0 * g.groups;
  const uint8_t* const zero = g.zero ? g.zero + (size_t)n0 * g.groups
                                     : reinterpret_cast<const uint8_t*>(scale);
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)ring;
  auto issue = [&](int step, int slot) {
    if (step >= steps) return;
    const uint32_t to = __builtin_amdgcn_readfirstlane(base + slot * L::kBytes);
    // (an odd piece's second block: its last again, which no wave uses)
    auto block = [&](int h) { return min(b0 + 2 * step + h, b1 - 1); };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k0 = block(h) * kBlk;
      dma_b128(codes + (k0 >> 1), oc + (uint32_t)(min(ck, g.k - 32 - k0) >> 1),
               to + h * L::kBlock + wv * 1024);
      const uint8_t* x = static_cast<const uint8_t*>(g.x) + ((size_t)t0 * g.k + k0) * (F32X ? 4 : 2);
#pragma unroll
      for (int c = 0; c < L::XC; ++c)
        dma_b128(x, (ox[c] + (uint32_t)min(kx[c], g.k - (F32X ? 4 : 8) - k0)) * (F32X ? 4 : 2),
                 to + h * L::kBlock + L::kX + (wv * L::XC + c) * 1024);
    }
    // scales and zeros, 64 of one block's and group's a copy: with 4 copies of each
    // waves 0 .. 3 make the scales', the others the zeros'
    auto value = [&](int c, bool z) {
      const int q = c >> 1, b = block(q / (4 / SG)), s = q % (4 / SG);
      const uint32_t o = (uint32_t)min((c & 1) * 64 + lane, last) * (uint32_t)g.groups +
                         (uint32_t)group_of<SG>(g, b, s);
      if (z) dma_u8(zero, o, to + L::kZ + c * 256);
      else dma_u16(scale, o * 2, to + L::kS + c * 256);
    };
    if constexpr (WIDE) {
      // wave w: scales 64 w .. + 64 (dwords) of the two blocks', zeros 64 (w mod 4)
      // .. + 64 (every one twice, so that each wave has the same copies in flight)
      const uint32_t r = (uint32_t)min((wv & 3) * 32 + (lane >> 1), last);
      dma_b32(scale, (r * g.groups + (uint32_t)(block(wv >> 2) * 4 + (lane & 1) * 2)) * 2,
              to + L::kS + wv * 256);
      const int c = wv & 3;
      dma_b32(zero, (uint32_t)min((c & 1) * 64 + lane, last) * (uint32_t)g.groups +
                        (uint32_t)(block(c >> 1) * 4), to + L::kZ + c * 256);
    } else if constexpr (L::kVals == 256) {
      if (wv < 4) value(wv, false);
      else value(wv - 4, true);
    } else {
#pragma unroll
      for (int c = 0; c < L::kVals / 512; ++c) {
        value(wv + 8 * c, false);
        value(wv + 8 * c, true);
      }
    }
  };
  const f32x4_t nil = {0.f, 0.f, 0.f, 0.f};
  f32x4_t acc[2][MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) acc[0][m] = acc[1][m] = nil;
  bf16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;
#pragma unroll
  for (int q = 0; q < kStages - 1; ++q) issue(q, q);
  int slot = 0;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    // this wave's copies of the step have landed and its reads of the one
    // before are done; past the barrier both hold for every wave
    wait_lds();
    if (step + kStages - 2 < steps) wait_vmem<(kStages - 2) * L::kCopies>();
    else wait_vmem<0>();
    grouped::wg_barrier();
    issue(step + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
    const uint8_t* const vals = ring + slot * L::kBytes;
    const uint8_t* const at = vals + wk * L::kBlock;
    slot = slot == kStages - 1 ? 0 : slot + 1;
    const int blk = b0 + 2 * step + wk;
    if (blk >= b1) continue;
    uint32_t c[2][4];
    float wsc[2][4], woff[2][4];   // WIDE: the block's four groups
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const uint4 v = *reinterpret_cast<const uint4*>(at + (wn * 2 + f) * 1024 + ln * 64 +
                                                      ((lg ^ code_swz(ln)) << 4));
      c[f][0] = v.x; c[f][1] = v.y; c[f][2] = v.z; c[f][3] = v.w;
      transpose4(c[f]);
      if constexpr (WIDE) {
        const int r = wk * 128 + wn * 32 + f * 16 + ln;
        wide_values(vals + L::kS + r * 8, vals + L::kZ + r * 4, g.zero, wsc[f], woff[f]);
      }
    }
#pragma unroll
    for (int s = 0; s < 4 / FS; ++s) {
      if (blk * kBlk + s * FS * 32 >= g.k) break;
      float sc[2], off[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        if constexpr (WIDE) {
          sc[f] = wsc[f][s];
          off[f] = woff[f][s];
          continue;
        }
        const int i = ((wk * (4 / SG) + s * FS / SG) * 128 + wn * 32 + f * 16 + ln) * 4;
        sc[f] = bf16_lo(*reinterpret_cast<const uint32_t*>(vals + L::kS + i));
        off[f] = -(float)(16 + (g.zero ? *reinterpret_cast<const int*>(vals + L::kZ + i) : 8));
      }
      f32x4_t sum[MB], dot[2][MB];
#pragma unroll
      for (int m = 0; m < MB; ++m) sum[m] = dot[0][m] = dot[1][m] = nil;
#pragma unroll
      for (int j = s * FS; j < (s + 1) * FS; ++j) {
        const bf16x8_t w[2] = {codes_biased(c[0][j]), codes_biased(c[1][j])};
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          uint4 xv[F32X ? 2 : 1];
#pragma unroll
          for (int h = 0; h < (F32X ? 2 : 1); ++h) {
            const int u = F32X ? 8 * j + 2 * lg + h : 4 * j + lg;
            xv[h] = *reinterpret_cast<const uint4*>(at + L::kX + (m * 16 + ln) * L::kRow + ((u ^ ln) << 4));
          }
          bf16x8_t a[XP];
          x_frags<F32X, false>(xv, a);
#pragma unroll
          for (int p = 0; p < XP; ++p) {
            sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], ones, sum[m], 0, 0, 0);
#pragma unroll
            for (int f = 0; f < 2; ++f)
              dot[f][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], w[f], dot[f][m], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[f][m][r] = __builtin_fmaf(sc[f], __builtin_fmaf(off[f], sum[m][r], dot[f][m][r]),
                                          acc[f][m][r]);
    }
  }
  bool bad = false;
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        bad |= m * 16 + lg * 4 + r < tn && !(fabsf(acc[f][m][r]) < INFINITY);
  if (__any(bad)) {
#pragma unroll 1
    for (int m = 0; m < MB; ++m) {
      Rows<2> rows;
      rows.lg = lg;
      rows.tok = t0 + min(m * 16 + ln, tn - 1);
#pragma unroll
      for (int f = 0; f < 2; ++f) rows.row[f] = n0 + min(wn * 32 + f * 16 + ln, last);
      f32x4_t again[2];
      w4_slice_exact<2, SG, F32X>(g, b0 + wk, b1, 2, rows, again);
#pragma unroll
      for (int q = 0; q < MB; ++q)
        if (q == m) { acc[0][q] = again[0]; acc[1][q] = again[1]; }
    }
  }
  // ---- the two halves: each wave hands over half of its tokens' sums and adds the
  // other's to the half it keeps (no copy is in flight into the ring any more)
  float* const red = reinterpret_cast<float*>(ring);
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MB; ++m)
    if ((m < MB / 2) == (wk == 1)) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          red[(m * 16 + lg * 4 + r) * kRed + wn * 32 + f * 16 + ln] = acc[f][m][r];
    }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MB; ++m)
    if ((m < MB / 2) == (wk == 0)) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = m * 16 + lg * 4 + r, n = wn * 32 + f * 16 + ln;
          if (t < tn && n <= last)
            g.part[((size_t)blockIdx.y * g.T + t0 + t) * g.n + n0 + n] = acc[f][m][r] + red[t * kRed + n];
        }
    }
}

// The pieces of a split contraction added in order, then the gated form's
// activation: one workgroup row a token, V consecutive outputs a thread.
template <bool GLU, int V>
__global__ __launch_bounds__(256) void w4_finish(W4Args g) {
  typedef __attribute__((ext_vector_type(V))) float vec_t;
  const int n_out = GLU ? g.f : g.n, n = (blockIdx.x * 256 + threadIdx.x) * V;
  const int64_t t = blockIdx.y;
  if (n >= n_out) return;
  const size_t piece = (size_t)g.T * g.n;
  const float* p = g.part + t * g.n + n;
  vec_t a = 0.f, b = 0.f;
#pragma unroll 4
  for (int s = 0; s < g.splits; ++s) {
    a += *reinterpret_cast<const vec_t*>(p + s * piece);
    if (GLU) b += *reinterpret_cast<const vec_t*>(p + s * piece + g.f);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float o = GLU ? silu_mul(a[i], b[i]) : a[i];
    if (g.out_f32) static_cast<float*>(g.out)[t * n_out + n + i] = o;
    else static_cast<uint16_t*>(g.out)[t * n_out + n + i] = f32_to_bf16(o);
  }
}

// Slots of a wave's ring: as many as the 160 KB of a CU hold, at most 4.  What
// counts is how many bytes a CU has in flight: one workgroup of 16 waves with a
// slot or two each reads faster than 8 waves with up to four (n x k, group, us from HBM:
// one token 7168 x 4096, 128: 7.0 against 7.8; gated 2 x 4096 x 7168: 11.0
// against 12.0; 16 tokens 7168 x 4096, 64: 9.1 against 9.8; 5 fp32 tokens gated
// 2 x 2049 x 7168, 64: 16.3 against 19.1), fp32 too, where the 16 waves' bound of
// 128 registers puts five to nine of them in scratch; only 32 workgroups of a
// short contraction lose (2 fp32 tokens 1024 x 1024, 32: 4.6 against 4.5).  16
// fp32 tokens do not fit with 16 waves; 8 there against 4: 19.3, 25.5
// (7168 x 7168).
template <int W, int RC, int NF, int SG, bool F32X, bool WIDE>
constexpr int ring_depth() {
  constexpr int n = (160 << 10) / (W * Slot<RC, NF, SG, F32X, WIDE>::kBytes);
  return n < 4 ? n : 4;
}

template <int W, int RC, int NF, int SG, int FS, bool F32X, bool WIDE, bool GLU>
hipError_t launch_fs(const W4Args& g, hipStream_t st) {
  constexpr int NB = GLU ? 8 * NF : 16 * NF;
  w4_kernel<W, ring_depth<W, RC, NF, SG, F32X, WIDE>(), RC, NF, SG, FS, F32X, WIDE, GLU>
      <<<((GLU ? g.f : g.n) + NB - 1) / NB, 64 * W, 0, st>>>(g);
  return hipGetLastError();
}
// (FS 1 for fp32 x and outputs: what it costs and brings is at the top)
template <int W, int RC, int NF, int SG, bool F32X, bool WIDE, bool GLU>
hipError_t launch_sg(const W4Args& g, hipStream_t st) {
  if constexpr (F32X && SG > 1)
    if (g.out_f32) return launch_fs<W, RC, NF, SG, 1, F32X, WIDE, GLU>(g, st);
  return launch_fs<W, RC, NF, SG, SG, F32X, WIDE, GLU>(g, st);
}
template <int W, int RC, int NF, bool F32X, bool GLU>
hipError_t launch(const W4Args& g, hipStream_t st) {
  const int group = g.k / g.groups;
  if (group == 32) return g.groups % 4 == 0 ? launch_sg<W, RC, NF, 1, F32X, true, GLU>(g, st)
                                            : launch_sg<W, RC, NF, 1, F32X, false, GLU>(g, st);
  if (group == 64) return launch_sg<W, RC, NF, 2, F32X, false, GLU>(g, st);
  return launch_sg<W, RC, NF, 4, F32X, false, GLU>(g, st);   // a multiple of 128
}
template <int MB, int SG, bool F32X, bool WIDE>
void launch_tile_sg(const W4Args& g, dim3 grid, hipStream_t st) {
  if constexpr (F32X && SG > 1)
    if (g.out_f32) {
      w4_tile<MB, SG, 1, F32X, WIDE><<<grid, 512, 0, st>>>(g);
      return;
    }
  w4_tile<MB, SG, SG, F32X, WIDE><<<grid, 512, 0, st>>>(g);
}
template <int MB, bool F32X, bool GLU>
hipError_t launch_tile(const W4Args& g, hipStream_t st) {
  // (a multiple of 8 along the weights: the token blocks of one set of rows run
  // on the same XCD, whose L2 then serves the codes)
  const dim3 grid(((g.n + 127) / 128 + 7) / 8 * 8, g.splits, (g.T + 16 * MB - 1) / (16 * MB));
  const int group = g.k / g.groups;
  if (group == 32 && g.groups % 4 == 0) launch_tile_sg<MB, 1, F32X, true>(g, grid, st);
  else if (group == 32) launch_tile_sg<MB, 1, F32X, false>(g, grid, st);
  else if (group == 64) launch_tile_sg<MB, 2, F32X, false>(g, grid, st);
  else launch_tile_sg<MB, 4, F32X, false>(g, grid, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int n_out = GLU ? g.f : g.n;
  if (n_out % 4 == 0)   // (whole 16-byte pieces of every row)
    w4_finish<GLU, 4><<<dim3((n_out + 1023) / 1024, g.T), 256, 0, st>>>(g);
  else
    w4_finish<GLU, 1><<<dim3((n_out + 255) / 256, g.T), 256, 0, st>>>(g);
  return hipGetLastError();
}

// Up to 16 tokens a workgroup always has all of them; the tiled kernel takes kChunk
// tokens at a time (so that its partial sums stay bounded).
constexpr int kFew = 16, kChunk = 256;

// Tokens of a workgroup of the tiled kernel.
int tile_tokens(int T, bool x_f32) { return x_f32 || T <= 32 ? 32 : 64; }
// Blocks of a piece of the contraction for a chunk of T tokens, a whole number of
// steps: at most one workgroup a CU (a second round of a few workgroups costs as
// much as the first).
int tile_piece(int n, int k, int T, bool x_f32) {
  const int tt = tile_tokens(T, x_f32);
  const int64_t wgs = (int64_t)((n + 127) / 128) * ((T + tt - 1) / tt);
  const int64_t pairs = (k + 2 * kBlk - 1) / (2 * kBlk), s = std::max<int64_t>(256 / wgs, 1);
  return (int)((pairs + s - 1) / s * 2);
}
int tile_splits(int n, int k, int T, bool x_f32) {
  const int per = tile_piece(n, k, T, x_f32) * kBlk;
  return (k + per - 1) / per;
}

// Up to 64 tokens (fp32: 32) may still go without a split contraction, whose
// partial sums and second launch cost 5 us: 32 weight rows a workgroup, which reads
// all of x.  It pays where those workgroups run in one round of the 256 CUs and x
// is short against what the split form writes, some n T sums (us, this form against
// the split one; 32 tokens x 4096: n 512 8.4, 8.9; 8192 11.2, 15.0; 8448 18.8, 17.1;
// 64 x 4096: n 512 12.6, 11.0; 3584 15.0, 15.7; 8192 16.6, 20.7; 64 x 7168: n 1024
// 18.8, 14.4; 8192 25.3, 24.5; 32 fp32 x 4096: n 2048 16.7, 12.7; 8192 20.7, 23.4).
bool one_round(const W4Args& g, bool x_f32) {
  const int64_t T = g.T <= 32 ? 32 : 64, x = T * g.k * (x_f32 ? 4 : 2);
  return g.T <= (x_f32 ? 32 : 64) && g.n <= 256 * 32 && x <= (256 << 10) + 64 * (int64_t)g.n;
}

template <bool F32X, bool GLU>
hipError_t launch_t(W4Args g, hipStream_t st) {
  if (g.T <= 4) return launch<16, 4, 2, F32X, GLU>(g, st);
  if (g.T <= 8) return launch<16, 8, 2, F32X, GLU>(g, st);
  if (g.T <= kFew) return launch<F32X ? 8 : 16, 16, 2, F32X, GLU>(g, st);
  if (one_round(g, F32X)) {
    if (g.T <= 32) return launch<8, 32, 2, F32X, GLU>(g, st);
    if constexpr (!F32X) return launch<8, 64, 2, F32X, GLU>(g, st);
  }
  const int T = g.T;
  const size_t out = (size_t)(GLU ? g.f : g.n) * (g.out_f32 ? 4 : 2);
  for (int t = 0; t < T; t += kChunk) {
    W4Args c = g;
    c.T = std::min(kChunk, T - t);
    c.x = static_cast<const uint8_t*>(g.x) + (size_t)t * g.k * (F32X ? 4 : 2);
    c.out = static_cast<uint8_t*>(g.out) + (size_t)t * out;
    c.splits = tile_splits(g.n, g.k, c.T, F32X);
    c.per_split = tile_piece(g.n, g.k, c.T, F32X);
    const hipError_t e = tile_tokens(c.T, F32X) == 32 ? launch_tile<2, F32X, GLU>(c, st)
                                                      : launch_tile<F32X ? 2 : 4, F32X, GLU>(c, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// Floats of the partial sums: the largest of a chunk's and the last, smaller
// chunk's, for bf16 x (fp32's workgroups of fewer tokens are no fewer, and so their
// pieces no more).
size_t w4_part_floats(const k3moe_w4_matrix& w, int64_t T) {
  if (T <= kFew) return 0;
  auto floats = [&](int64_t t) { return (size_t)tile_splits(w.n, w.k, (int)t, false) * t * w.n; };
  const int64_t rest = T % kChunk;
  return T < kChunk ? floats(T) : std::max(floats(kChunk), rest ? floats(rest) : 0);
}

hipError_t launch_w4(const k3moe_w4_matrix& w, int64_t T, bool x_f32, bool out_f32, bool glu,
                     const void* x, void* out, float* part, hipStream_t st) {
  W4Args g{};
  g.part = part;
  g.codes = static_cast<const uint8_t*>(w.codes);
  g.scale = static_cast<const uint16_t*>(w.scale);
  g.zero = static_cast<const uint8_t*>(w.zero);
  g.x = x;
  g.out = out;
  g.T = (int)T;
  g.n = w.n;
  g.k = w.k;
  g.groups = w.k / w.group;
  // (rounded up, exact for the at most 2^13 blocks of a row)
  const uint32_t blocks = (uint32_t)w.group / kBlk;
  g.per_group = blocks > 1 ? (uint32_t)(((uint64_t(1) << 32) + blocks - 1) / blocks) : 0;
  g.f = glu ? w.n / 2 : w.n;
  g.out_f32 = out_f32;
  if (x_f32) return glu ? launch_t<true, true>(g, st) : launch_t<true, false>(g, st);
  return glu ? launch_t<false, true>(g, st) : launch_t<false, false>(g, st);
}

}  // namespace k3
