// The orthogonalised update of a matrix by Newton-Schulz steps.  With X the matrix
// taken wide (s rows, l >= s columns; a tall one is transposed on its way in and
// out), scaled to Frobenius norm 1, a step is
//   A = X X^T          B = b A + c A A          X <- a X + B X
// which maps every singular value v to a v + b v^3 + c v^5 and leaves the singular
// vectors.  Three products of one kind, so one tile kernel (ortho_tile) runs them
// on v_mfma_f32_16x16x32_f16, both operands in LDS rings; A and A A are symmetric
// and only their tiles on and over the diagonal are computed, written twice.
//
// Operands are fp16 (11 bits), sums fp32.  The bound on singular values that the
// host derives from the coefficients fits all values into fp16 with fixed powers of
// two: 2^15 X, 2^15 A, 2^14 B.  X has a second fp16 part, its rounding's rest, for
// the term a X: a step multiplies a small singular value by a (3.4 for the usual
// coefficients), and what rounding X adds in directions where the update has little
// would grow along (relative error of the result for a gradient with sixteen
// directions ten times its noise, 512 x 1024: 1e-2 with one part, 3e-4 with two;
// for noise alone 1.5e-3, as much as the bf16 output's own rounding).  The last step,
// whose error nothing multiplies any more, does without.  The roundings inside the
// products do not need it for small singular values: they are relative to A and B, which
// are small where X is.  They are added again in every step, though: five of the usual
// steps end 1.7e-3 to 3.9e-3 off before the output's rounding, and only steps that settle
// (1.5, -0.5, 0) keep that for long.  Two parts everywhere would be three products for one.
//
// Matrices whose short side is at most 128 take the kernels of ortho_small.hip, but for
// coefficients that multiply its A too far (ortho_small_ok).
//
// Large matrices are bound by the products (2 x 4096 x 7168, us a step: A 209 to 214, with
// its finish 220 = 1.09 PFLOP/s of the half that is computed; B 131 to 145; X 406 to 450, of
// which some 30 us a round of tiles are its way out, X's two parts read and written at once
// by all CUs: the next row block's are requested ahead, and every other workgroup starts
// with a shorter piece).  Their matrix cores are busy 59 to 70 % of the time at 1.97 to 2.08
// GHz; the clock falls as they get busier (a library product of such values: 94 % at 1.67).
// 896 x 7168 takes 16 + 5, 9 and 25 us a step, half of it the start and way out of tiles of
// 14 stages; matrices of a few hundred rows 5 to 7 us a launch.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "kern_common.h"
#include "grouped.h"
#include "dense_tile.h"

namespace k3 {
namespace {

using namespace grouped;
using namespace dense;

constexpr float kScaleX = 32768.0f;   // 2^15, of X and of A; B has half of it

//   kGram   A:  M = N = s  K = l   a = b = X
//   kPoly   B:  M = N = s  K = s   a = b = A (its own transpose)
//   kStep   X:  M = s  N = l  K = s   a = B  b = X
//   kLast, kLastT   kStep into the output, as it is or transposed
enum Product { kGram, kPoly, kStep, kLast, kLastT };

struct OrthoArgs {
  const uint16_t* x;      // [batch][s][l] first parts
  uint16_t* xo;           // kStep: the next X's
  uint16_t* lo;           // [batch][s][l] second parts, replaced in place
  uint16_t* A;            // [batch][s][s]
  uint16_t* B;
  void* out;              // kLast: [batch][rows][cols], kLastT: [batch][cols][rows], bf16
  float* part;            // sums of the split tiles' pieces, in the waves' own order
  int s, l, batch;        // s and l in whole 64
  int rows, cols;         // the matrix's own
  int whole;              // tiles that one workgroup computes; the contraction of the others
  int pieces, k_piece;    // is split into pieces of k_piece elements (a multiple of kBK)
  int keep_lo;            // kStep: the next step takes second parts (the last does not)
  float ca, cb, cc, scale;
};

__device__ __forceinline__ float f16_lo(uint32_t w) {
  return (float)__builtin_bit_cast(f16x2_t, w)[0];
}
__device__ __forceinline__ float f16_hi(uint32_t w) {
  return (float)__builtin_bit_cast(f16x2_t, w)[1];
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

template <int P, int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN;
  static constexpr bool kSym = P == kGram || P == kPoly;
  static constexpr int MF = BM / 16 / WM, NF = BN / 16 / WN;
  static constexpr int NA = BM * 8 / 64 / NW, NB = BN * 8 / 64 / NW;   // copies per wave and stage
  using A = Operand<true, BM>;
  using B = Operand<kSym, BN>;
  static_assert(NA * 64 * NW == BM * 8 && NB * 64 * NW == BN * 8 && MF >= 1 && NF % 2 == 0, "whole copies");
  static_assert(!kSym || BM == BN, "square tiles of a symmetric product");
};

struct At {
  int b, m0, n0;
};

// Tiles in groups of 4 (symmetric products) or 8 rows of tiles, down the rows first,
// so that the workgroups of an XCD share both operands through its L2.
__host__ __device__ inline int sym_tiles(int n) { return n * (n + 1) / 2; }
template <typename C>
__device__ __forceinline__ At tile_at(const OrthoArgs& g, int it) {
  const int mt = (g.s + C::BM - 1) / C::BM;
  if (C::kSym) {
    const int per = sym_tiles(mt), b = it / per;
    int r = it - b * per, i0 = 0, rows, size;
    for (;;) {   // (mt / 4 steps at most)
      rows = min(4, mt - i0);
      size = sym_tiles(rows) + (mt - i0 - rows) * rows;
      if (r < size) break;
      r -= size;
      i0 += 4;
    }
    int i, j;
    if (r < sym_tiles(rows)) {   // columns of 1, 2, .. rows
      j = r >= 6 ? 3 : r >= 3 ? 2 : r >= 1 ? 1 : 0;
      i = r - sym_tiles(j);
    } else {
      r -= sym_tiles(rows);
      j = rows + r / rows;
      i = r % rows;
    }
    return At{b, (i0 + i) * C::BM, (i0 + j) * C::BN};
  }
  const int nt = (g.l + C::BN - 1) / C::BN, per = mt * nt, b = it / per;
  const int r = it - b * per, grp = r / (8 * nt), first = grp * 8, gsz = min(mt - first, 8);
  const int q = r - grp * 8 * nt, j = q / gsz;
  return At{b, (first + q - j * gsz) * C::BM, j * C::BN};
}

// ---- epilogue of a wave's fragments.  Two fragments side by side, their odd and even
// groups of 16 lanes exchanged, give a lane eight consecutive columns of its row; it
// reads A or X's two parts there, 16 bytes each (outside the matrix: at the origin).
struct Old {
  uint4 h, l;   // A, or X's parts
};
template <int P>
__device__ __forceinline__ Old load_old(const OrthoArgs& g, int b, int m16, int n_wave, int f) {
  const int lane = threadIdx.x & 63, lg = lane >> 4, m = m16 + (lane & 15);
  const int n = n_wave + (f + (lg & 1)) * 16 + (lg >> 1) * 8;
  Old o{};
  if (P == kPoly) {
    const uint32_t at = m < g.s && n < g.s ? (uint32_t)m * g.s + n : 0;
    o.h = *reinterpret_cast<const uint4*>(g.A + (size_t)b * g.s * g.s + at);
  } else if (P > kPoly) {
    const uint32_t at = m < g.s && n < g.l ? (uint32_t)m * g.l + n : 0;
    o.h = *reinterpret_cast<const uint4*>(g.x + (size_t)b * g.s * g.l + at);
    if (P == kStep) o.l = *reinterpret_cast<const uint4*>(g.lo + (size_t)b * g.s * g.l + at);
  }
  return o;
}

// Row block i (16 rows).
template <int P, int NF>
__device__ __forceinline__ void finish_row(const OrthoArgs& g, int b, int m16, int n_wave, f32x4_t (&acc)[NF],
                                           const Old (&old)[NF / 2]) {
  const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4, m = m16 + ln;
  const size_t ss = (size_t)g.s * g.s, sl = (size_t)g.s * g.l;
#pragma unroll
  for (int f = 0; f < NF; f += 2) {
    float v[8];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint32_t p = __float_as_uint(acc[f][r]), q = __float_as_uint(acc[f + 1][r]);
      exchange(p, q);
      v[r] = __uint_as_float(p);
      v[4 + r] = __uint_as_float(q);
    }
    const int n16 = n_wave + (f + (lg & 1)) * 16, n = n16 + (lg >> 1) * 8;
    if (P == kGram || P == kPoly) {
      // blocks of 16 x 16 under the diagonal are written by those over it
      const bool in = m < g.s && n < g.s && n16 >= m16;
      const size_t at = b * ss + (size_t)m * g.s + n;
      uint16_t* o = P == kGram ? g.A : g.B;
      if (P == kGram) {
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] *= 1.0f / kScaleX;
      } else {
        const uint4 a = old[f / 2].h;
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        const float hb = 0.5f * g.cb, hc = g.cc * (0.5f / kScaleX);
#pragma unroll
        for (int r = 0; r < 8; ++r)
          v[r] = __builtin_fmaf(hc, v[r], hb * (r & 1 ? f16_hi(w[r / 2]) : f16_lo(w[r / 2])));
      }
      const uint4 q = make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]),
                                 pack_f16(v[6], v[7]));
      // (the four lanes of a transpose have the same columns, and rows of one block)
      const uint2 t0 = transpose4(make_uint2(q.x, q.y), lane), t1 = transpose4(make_uint2(q.z, q.w), lane);
      if (in) *reinterpret_cast<uint4*>(o + at) = q;
      if (in && n16 > m16) {
        uint16_t* t = o + b * ss + (size_t)(n + (lane & 3)) * g.s + m16 + (ln & ~3);
        *reinterpret_cast<uint2*>(t) = t0;
        *reinterpret_cast<uint2*>(t + 4 * (size_t)g.s) = t1;
      }
    } else {
      const bool in = m < g.s && n < g.l;
      const size_t at = b * sl + (size_t)m * g.l + n;
      const uint4 h = old[f / 2].h, l = old[f / 2].l;
      const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        float x = r & 1 ? f16_hi(hw[r / 2]) : f16_lo(hw[r / 2]);
        if (P == kStep) x += r & 1 ? f16_hi(lw[r / 2]) : f16_lo(lw[r / 2]);
        v[r] = __builtin_fmaf(g.ca, x, v[r] * (2.0f / kScaleX));
      }
      if (P == kStep) {
        uint32_t ho[4], lo[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          ho[r] = pack_f16(v[2 * r], v[2 * r + 1]);
          lo[r] = pack_f16(v[2 * r] - f16_lo(ho[r]), v[2 * r + 1] - f16_hi(ho[r]));
        }
        if (in) {
          *reinterpret_cast<uint4*>(g.xo + at) = make_uint4(ho[0], ho[1], ho[2], ho[3]);
          if (g.keep_lo) *reinterpret_cast<uint4*>(g.lo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        continue;
      }
      uint4 q;
      q.x = pack_bf16(g.scale * v[0], g.scale * v[1]);
      q.y = pack_bf16(g.scale * v[2], g.scale * v[3]);
      q.z = pack_bf16(g.scale * v[4], g.scale * v[5]);
      q.w = pack_bf16(g.scale * v[6], g.scale * v[7]);
      uint16_t* o = static_cast<uint16_t*>(g.out) + (size_t)b * g.rows * g.cols;
      if (P == kLast) {
        if (m < g.rows && n < g.cols) {
          uint16_t* p = o + (size_t)m * g.cols + n;
          if (g.cols % 8 == 0) {
            *reinterpret_cast<uint4*>(p) = q;
          } else {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (n + r < g.cols) p[r] = (uint16_t)(w[r / 2] >> (r & 1 ? 16 : 0));
          }
        }
      } else {
        const int mm = m16 + (ln & ~3);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint2 t = transpose4(half ? make_uint2(q.z, q.w) : make_uint2(q.x, q.y), lane);
          const int nn = n + 4 * half + (lane & 3);
          if (nn >= g.cols || mm >= g.rows) continue;
          uint16_t* p = o + (size_t)nn * g.rows + mm;
          if (g.rows % 4 == 0) {
            *reinterpret_cast<uint2*>(p) = t;
          } else {
            const uint32_t w[2] = {t.x, t.y};
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (mm + r < g.rows) p[r] = (uint16_t)(w[r / 2] >> (r & 1 ? 16 : 0));
          }
        }
      }
    }
  }
}

// ---- the products.  The first g.whole items are tiles, the others pieces of the
// contraction of a tile each: their sums go to g.part, and ortho_finish adds them in
// order.
template <int P, int BM, int BN, int WM, int WN, int RING>
__global__ __launch_bounds__(64 * WM * WN) void ortho_tile(OrthoArgs g) {
  using C = Tile<P, BM, BN, WM, WN>;
  using OA = typename C::A;
  using OB = typename C::B;
  constexpr int MF = C::MF, NF = C::NF;
  __shared__ __attribute__((aligned(16))) uint8_t sA[RING * OA::kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t sB[RING * OB::kSlot];

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const int N = C::kSym ? g.s : g.l, K = P == kGram ? g.l : g.s;
  const int mt = (g.s + BM - 1) / BM, nt = (N + BN - 1) / BN;
  const int n_tiles = g.batch * (C::kSym ? sym_tiles(mt) : mt * nt);
  const int n_items = g.whole + (n_tiles - g.whole) * g.pieces;
  // A round takes the next gridDim.x items, its 8 contiguous pieces one to an XCD.
  // Every other workgroup takes the split tiles' round first, the others last, so that
  // half of them work on a tile while the tiles of the other half go to memory.
  const int G = gridDim.x, xcd = blockIdx.x & 7, wi = blockIdx.x >> 3;
  const int full = g.whole / G;
  bool early = false;
  auto item_of = [&](int r) {
    if (early && r <= full) r = r == 0 ? full : r - 1;
    const int64_t first = (int64_t)r * G;
    if (first >= n_items) return n_items;
    const int end = (int)min(first + G, (int64_t)n_items), piece = (end - (int)first + 7) >> 3;
    const int it = (int)first + xcd * piece + wi;
    return wi < piece && it < end ? it : n_items;
  };
  // (where it has an item of that round)
  early = (wi & 1) && g.whole % G == 0 && n_items - g.whole <= G && item_of(full) < n_items;
  auto span = [&](int it, int& k0, int& k1) {   // the item's tile
    if (it < g.whole) {
      k0 = 0;
      k1 = K;
      return tile_at<C>(g, it);
    }
    const int j = it - g.whole, t = j / g.pieces;
    k0 = (j - t * g.pieces) * g.k_piece;
    k1 = min(k0 + g.k_piece, K);
    return tile_at<C>(g, g.whole + t);
  };

  // ---- copies, as in the shared experts' products (K is a multiple of kBK)
  uint32_t va[C::NA], vb[C::NB];
  const uint16_t* opa = P == kGram ? g.x : P == kPoly ? g.A : g.B;
  const uint16_t* opb = P == kPoly ? g.A : g.x;
  const size_t lda = P == kGram ? g.l : g.s, ldb = P == kPoly ? g.s : g.l;
  const size_t sa_b = P == kGram ? (size_t)g.s * g.l : (size_t)g.s * g.s;
  const size_t sb_b = P == kPoly ? (size_t)g.s * g.s : (size_t)g.s * g.l;
  const uint32_t sa = kBK * 2, sb = C::kSym ? kBK * 2 : kBK * 2 * (uint32_t)ldb;   // bytes per stage
  uint64_t pa = 0, pb = 0;
  int c_rd = 0, c_k, c_end, c_it = item_of(0);
  auto setup = [&]() {
    const At t = span(c_it, c_k, c_end);
    pa = (uint64_t)(uintptr_t)(opa + t.b * sa_b + (size_t)t.m0 * lda + c_k);
    pb = (uint64_t)(uintptr_t)(opb + t.b * sb_b + (C::kSym ? (size_t)t.n0 * ldb + c_k
                                                         : (size_t)c_k * ldb + t.n0));
#pragma unroll
    for (int c = 0; c < C::NA; ++c) {
      int r, k;
      OA::unit((wv * C::NA + c) * 64 + lane, r, k);
      va[c] = t.m0 + r < g.s ? (uint32_t)(((size_t)r * lda + k) * 2) : kOut;
    }
#pragma unroll
    for (int c = 0; c < C::NB; ++c) {
      int r, k;
      OB::unit((wv * C::NB + c) * 64 + lane, r, k);
      const size_t e = C::kSym ? (size_t)r * ldb + k : (size_t)k * ldb + r;
      vb[c] = t.n0 + r < N ? (uint32_t)(e * 2) : kOut;
    }
  };
  auto copy = [&](int slot, int c) {
    const bool isa = c < C::NA;
    const int q = isa ? c : c - C::NA, n = isa ? C::NA : C::NB;
    const uint32_t to = lds_addr(isa ? sA : sB) +
                        (uint32_t)(slot * (isa ? OA::kSlot : OB::kSlot) + (wv * n + q) * 1024);
    dma16_buf(rsrc_of(isa ? pa : pb), isa ? va[q] : vb[q], to);
  };
  auto advance = [&]() {   // the copies' next stage
    c_k += kBK;
    pa += sa;
    pb += sb;
    if (c_k >= c_end) {
      c_it = item_of(++c_rd);
      if (c_it < n_items) {
        setup();
      } else {   // behind the last item: zeros, that nothing uses
        c_end = 0x7FFFFFFF;
#pragma unroll
        for (int c = 0; c < C::NA; ++c) va[c] = kOut;
#pragma unroll
        for (int c = 0; c < C::NB; ++c) vb[c] = kOut;
      }
    }
  };

  const int wm = wv / WN, wn = wv - wm * WN;
  bf16x8_t fa[MF], fb[NF], na[MF], nb[NF];
  f32x4_t acc[MF][NF];
  // MFMAs of fa, fb; reads of (slot, j) into na, nb; the copies into slot `to`
  // spread over the steps (to < 0: none)
  auto half = [&](int slot, int j, int to) {
    const uint8_t* ba = sA + slot * OA::kSlot;
    const uint8_t* bb = sB + slot * OB::kSlot;
    constexpr int kCp = (C::NA + C::NB + MF - 1) / MF;
    constexpr int kPer = (MF + NF + (MF > 2 ? MF - 2 : 1) - 1) / (MF > 2 ? MF - 2 : 1);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
#pragma unroll
      for (int r = i * kPer; r < (i + 1) * kPer && r < MF + NF; ++r) {
        if (r < NF) nb[r] = OB::frag(bb, wn * NF + r, j, ln, lg);
        else na[r - NF] = OA::frag(ba, wm * MF + r - NF, j, ln, lg);
      }
#pragma unroll
      for (int f = 0; f < NF; ++f)   // sums transposed: a lane holds 4 consecutive n of one m
        acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, fb[f]),
                                                           __builtin_bit_cast(f16x8_t, fa[i]), acc[i][f],
                                                           0, 0, 0);
      if (to >= 0) {
#pragma unroll
        for (int c = i * kCp; c < (i + 1) * kCp && c < C::NA + C::NB; ++c) copy(to, c);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) fa[i] = na[i];
#pragma unroll
    for (int f = 0; f < NF; ++f) fb[f] = nb[f];
  };
  if (c_it >= n_items) return;
  setup();
#pragma unroll
  for (int q = 0; q < RING; ++q) {
#pragma unroll
    for (int c = 0; c < C::NA + C::NB; ++c) copy(q, c);
    advance();
  }
  wait_vmem<(RING - 1) * (C::NA + C::NB)>();
  wg_barrier();
#pragma unroll
  for (int f = 0; f < NF; ++f) fb[f] = OB::frag(sB, wn * NF + f, 0, ln, lg);
#pragma unroll
  for (int i = 0; i < MF; ++i) fa[i] = OA::frag(sA, wm * MF + i, 0, ln, lg);
  int slot = 0;
  for (int rd = 0, it; (it = item_of(rd)) < n_items; ++rd) {
    int k0, k1;
    const At t = span(it, k0, k1);
    const int nst = (k1 - k0) / kBK;
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[i][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s = 0; s < nst; ++s) {
      half(slot, 1, -1);
      // this wave's reads of the slot are done and its copies of the next
      // stage have landed; past the barrier both hold for every wave
      wait_lds();
      wait_vmem<(RING - 2) * (C::NA + C::NB)>();
      wg_barrier();
      const int next = RING == 2 ? slot ^ 1 : slot == RING - 1 ? 0 : slot + 1;
      half(next, 0, slot);   // and the stage RING further on its way
      advance();
      slot = next;
    }
    if (it >= g.whole) {
      f32x4_t* p = reinterpret_cast<f32x4_t*>(g.part) + (size_t)(it - g.whole) * MF * NF * (64 * WM * WN);
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f) p[(i * NF + f) * (64 * WM * WN) + threadIdx.x] = acc[i][f];
    } else {
      // (what the next row block needs is on its way while one is finished, or a
      // tile's way out is one wait for memory after the other)
      Old old[2][NF / 2];
      auto load = [&](int i) {
#pragma unroll
        for (int f = 0; f < NF; f += 2)
          old[i & 1][f / 2] = load_old<P>(g, t.b, t.m0 + (wm * MF + i) * 16, t.n0 + wn * NF * 16, f);
      };
      load(0);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        if (i + 1 < MF) load(i + 1);
        __builtin_amdgcn_sched_barrier(0);
        finish_row<P, NF>(g, t.b, t.m0 + (wm * MF + i) * 16, t.n0 + wn * NF * 16, acc[i], old[i & 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

// The pieces of a split contraction added in order, and the epilogue: a workgroup
// for each row block of a tile's waves.
template <int P, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void ortho_finish(OrthoArgs g) {
  using C = Tile<P, BM, BN, WM, WN>;
  constexpr int MF = C::MF, NF = C::NF, kT = 64 * WM * WN;
  const int i = blockIdx.x % MF, tile = blockIdx.x / MF, wv = threadIdx.x >> 6;
  const At t = tile_at<C>(g, g.whole + tile);
  const f32x4_t* p = reinterpret_cast<const f32x4_t*>(g.part) +
                     ((size_t)tile * g.pieces * MF + i) * NF * kT + threadIdx.x;
  f32x4_t acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.pieces; ++s, p += (size_t)MF * NF * kT) {
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] += p[f * kT];
  }
  const int m16 = t.m0 + (wv / WN * MF + i) * 16, n_wave = t.n0 + wv % WN * NF * 16;
  Old old[NF / 2];
#pragma unroll
  for (int f = 0; f < NF; f += 2) old[f / 2] = load_old<P>(g, t.b, m16, n_wave, f);
  finish_row<P, NF>(g, t.b, m16, n_wave, acc, old);
}

// ---- the matrix on its way in.  Sums of squares, in fp64, of equal pieces of a
// matrix (one workgroup each), which scale_in adds in order.
constexpr int kMaxPieces = 256;
__device__ __forceinline__ float load_g(const void* g, size_t i, bool f32) {
  return f32 ? static_cast<const float*>(g)[i] : bf16_lo(static_cast<const uint16_t*>(g)[i]);
}

template <bool F32>
__global__ __launch_bounds__(256) void square_sums(const void* __restrict__ g, double* __restrict__ sums,
                                                   int64_t count, int64_t piece) {
  constexpr int W = F32 ? 4 : 8;   // elements in 16 bytes
  __shared__ double wave[4];
  const int64_t first = (int64_t)blockIdx.y * count;
  const int64_t lo = blockIdx.x * piece, hi = min(lo + piece, count);
  double a = 0.0;
  if (count % W == 0) {   // (then every matrix and piece starts at 16 bytes)
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(g) + first * (F32 ? 4 : 2));
    for (int64_t i = lo / W + threadIdx.x; i < hi / W; i += 256) {
      const uint4 q = p[i];
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (F32) {
          const double v = (double)__uint_as_float(w[j]);
          a = fma(v, v, a);
        } else {
          const double v = (double)bf16_lo(w[j]), u = (double)bf16_hi(w[j]);
          a = fma(v, v, a);
          a = fma(u, u, a);
        }
      }
    }
  } else {
    constexpr int U = 8;   // loads in flight
    for (int64_t i = lo + threadIdx.x; i < hi; i += 256 * U) {
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = load_g(g, first + min(i + 256 * u, hi - 1), F32);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + 256 * u < hi) a = fma((double)v[u], (double)v[u], a);
    }
  }
  a = wave_sum(a);
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x == 0)
    sums[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = ((wave[0] + wave[1]) + wave[2]) + wave[3];
}

// A 64 x 64 tile of X's two parts from g / |g| (0 for a matrix of zeros), zeros
// outside the matrix.  TR: X is g's transpose.
template <bool TR, bool F32>
__global__ __launch_bounds__(256) void scale_in(const void* __restrict__ g, const double* __restrict__ sums,
                                                uint16_t* __restrict__ hi, uint16_t* __restrict__ lo,
                                                int s, int l, int rows, int cols, int pieces) {
  __shared__ float t[64][65];
  __shared__ double wave[4];
  double a = wave_sum((int)threadIdx.x < pieces ? sums[(size_t)blockIdx.z * pieces + threadIdx.x] : 0.0);
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = a;
  __syncthreads();
  a = ((wave[0] + wave[1]) + wave[2]) + wave[3];
  const double f = a == 0.0 ? 0.0 : (double)kScaleX / sqrt(a);
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const size_t first = (size_t)blockIdx.z * rows * cols;
  // a thread's 16 elements: of X's row m0 + i (or, transposed, column n0 + i)
  const int c = (threadIdx.x & 15) * 4;
  const int nr = TR ? cols : rows, nk = TR ? rows : cols;   // g's rows and columns
  const int k = (TR ? m0 : n0) + c;
  float v[4][4];
  // (every load is issued, of the first element outside the matrix)
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = (TR ? n0 : m0) + (threadIdx.x >> 4) + 16 * q;
    const size_t at = first + (size_t)r * nk + k;
    if (nk % 4 == 0) {
      const size_t p = r < nr && k < nk ? at : 0;
      if (F32) {
        const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(g) + p);
        v[q][0] = x.x; v[q][1] = x.y; v[q][2] = x.z; v[q][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g) + p);
        v[q][0] = bf16_lo(x.x); v[q][1] = bf16_hi(x.x); v[q][2] = bf16_lo(x.y); v[q][3] = bf16_hi(x.y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[q][j] = load_g(g, r < nr && k + j < nk ? at + j : 0, F32);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int i = (threadIdx.x >> 4) + 16 * q, r = (TR ? n0 : m0) + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = r < nr && k + j < nk ? (float)((double)v[q][j] * f) : 0.0f;
      if (TR) t[c + j][i] = x; else t[i][c + j] = x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int i = (threadIdx.x >> 4) + 16 * q;
    uint32_t h[2], w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float x = t[i][c + 2 * j], y = t[i][c + 2 * j + 1];
      h[j] = pack_f16(x, y);
      w[j] = pack_f16(x - f16_lo(h[j]), y - f16_hi(h[j]));
    }
    const size_t at = (size_t)blockIdx.z * s * l + (size_t)(m0 + i) * l + n0 + c;
    *reinterpret_cast<uint2*>(hi + at) = make_uint2(h[0], h[1]);
    *reinterpret_cast<uint2*>(lo + at) = make_uint2(w[0], w[1]);
  }
}

// How a product runs: its tile, and how many of them are whole; the others are split
// into pieces of the contraction.
enum { kTile256, kTile128x256, kTile128, kTile64 };
struct Plan {
  int tile, whole, pieces, k_piece;
  size_t part;   // floats of the pieces' sums
};

struct Dims {
  int s, l, rows, cols, batch;   // rows <= cols: the matrix taken wide; s, l in whole 64
  bool tr;
  explicit Dims(const k3moe_ortho& p) {
    tr = p.m > p.n;
    rows = tr ? p.n : p.m;
    cols = tr ? p.m : p.n;
    s = (rows + 63) & ~63;
    l = (cols + 63) & ~63;
    batch = p.batch;
  }
};

int64_t tiles_of(int P, const Dims& d, int bm, int bn) {
  const int64_t mt = (d.s + bm - 1) / bm, nt = (d.l + bn - 1) / bn;
  return d.batch * (P <= kPoly ? mt * (mt + 1) / 2 : mt * nt);
}

// The tile and split that cost least, by what a 64-element stage and a tile's way out
// take (us) on 256 CUs.  A last round of a few tiles takes as long as a full one, so the tiles
// behind the last full round may be split: their pieces' sums go to memory and back
// (at 4.5 TB/s) and a second kernel adds them, 4 us.
Plan plan_product(int P, const Dims& d) {
  struct Kind {
    int bm, bn, slots;
    double stage, out;
  };
  constexpr Kind kinds[4] = {{256, 256, 256, 1.6, 9.0}, {128, 256, 256, 0.95, 4.6},
                             {128, 128, 256, 0.65, 2.7}, {64, 64, 768, 0.64, 1.9}};
  const int64_t nst = (P == kGram ? d.l : d.s) / kBK;
  double best = 1e30;
  Plan plan{};
  for (int k = 0; k < 4; ++k) {
    const Kind& c = kinds[k];
    if (P <= kPoly && c.bm != c.bn) continue;
    const int64_t n = tiles_of(P, d, c.bm, c.bn);
    // a round of `items` tiles or pieces of st stages; three 64 x 64 tiles share a CU
    auto round = [&](int64_t items, int64_t st) {
      const int64_t last = items % c.slots, full = items / c.slots;
      const double tail = k != 3 ? c.stage : last <= 256 ? 0.43 : last <= 512 ? 0.5 : 0.64;
      return full * (c.stage * st + c.out) + (last ? tail * st + c.out : 0.0);
    };
    double cost = round(n, nst);
    if (cost < best) best = cost, plan = Plan{k, (int)n, 1, 0, 0};
    const int64_t rest = n % c.slots, whole = n - rest;
    for (int64_t p = 2; rest && p <= 32 && 2 * p <= nst; ++p) {
      const int64_t per = (nst + p - 1) / p;
      if ((p - 1) * per >= nst || rest * p > 2 * c.slots) continue;
      const double bytes = 4.0 * rest * p * c.bm * c.bn;
      cost = round(whole, nst) + round(rest * p, per) + 4.0 + 2 * bytes / 4.5e6;
      if (cost < best)
        best = cost, plan = Plan{k, (int)whole, (int)p, (int)per * kBK, (size_t)rest * p * c.bm * c.bn};
    }
  }
  return plan;
}

template <int P, int BM, int BN, int WM, int WN, int RING>
hipError_t launch_tiles(const OrthoArgs& g, int64_t tiles, int grid, hipStream_t st) {
  constexpr int kT = 64 * WM * WN, MF = BM / 16 / WM;
  ortho_tile<P, BM, BN, WM, WN, RING><<<grid, kT, 0, st>>>(g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || tiles == g.whole) return e;
  ortho_finish<P, BM, BN, WM, WN><<<(unsigned)((tiles - g.whole) * MF), kT, 0, st>>>(g);
  return hipGetLastError();
}

template <int P>
hipError_t launch_product(const Dims& d, OrthoArgs g, hipStream_t st) {
  const Plan p = plan_product(P, d);
  const int cus = grouped_grid();
  g.whole = p.whole;
  g.pieces = p.pieces;
  g.k_piece = p.k_piece;
  switch (p.tile) {
    case kTile256: return launch_tiles<P, 256, 256, 2, 4, 2>(g, tiles_of(P, d, 256, 256), cus, st);
    case kTile128: return launch_tiles<P, 128, 128, 2, 4, 3>(g, tiles_of(P, d, 128, 128), cus, st);
    case kTile64: return launch_tiles<P, 64, 64, 2, 2, 3>(g, tiles_of(P, d, 64, 64), cus * 3, st);
  }
  if constexpr (P > kPoly) return launch_tiles<P, 128, 256, 2, 4, 3>(g, tiles_of(P, d, 128, 256), cus, st);
  return hipSuccess;   // (no plan of a symmetric product)
}

int pieces_of(const Dims& d) {
  const int64_t count = (int64_t)d.rows * d.cols;
  return (int)std::min<int64_t>(kMaxPieces, (count + 4095) / 4096);
}

}  // namespace

OrthoWs carve_ortho(const k3moe_ortho& p, void* ws, size_t* bytes) {
  const Dims d(p);
  const size_t sl = (size_t)d.batch * d.s * d.l, ss = (size_t)d.batch * d.s * d.s;
  Carver c(ws);
  OrthoWs w;
  w.sums = c.take<double>((size_t)d.batch * pieces_of(d));
  w.x[0] = c.take<uint16_t>(sl);
  w.x[1] = c.take<uint16_t>(p.steps > 1 ? sl : 0);
  w.lo = c.take<uint16_t>(sl);
  w.A = c.take<uint16_t>(ss);
  w.B = c.take<uint16_t>(ss);
  size_t part = 0;
  for (int P : {kGram, kPoly, kStep}) part = std::max(part, plan_product(P, d).part);
  w.part = c.take<float>(part);
  if (bytes) *bytes = c.off;
  return w;
}

// Whether fp16 holds 2^15 X, 2^15 X X^T and 2^14 B in every step, from |X| <= 1: the
// largest singular value that a step can leave is that of the polynomial on the
// interval before it.
bool ortho_bounded(const k3moe_ortho& p) {
  double top = 1.0;   // of the singular values
  for (int i = 0; i < p.steps; ++i) {
    const double a = p.coefficients[3 * i], b = p.coefficients[3 * i + 1], c = p.coefficients[3 * i + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    if (!(top <= 1.4)) return false;
    const double t = top * top;
    auto poly = [&](double y) { return std::fabs(b * y + c * y * y); };   // of B, y in 0 .. t
    double most = poly(t);
    if (c != 0.0 && -b / (2 * c) > 0.0 && -b / (2 * c) < t) most = std::max(most, poly(-b / (2 * c)));
    if (!(most <= 3.9)) return false;
    auto step = [&](double y) { return std::fabs(std::sqrt(y) * (a + b * y + c * y * y)); };
    double next = step(t);
    // a + 3 b y + 5 c y^2 = 0
    const double q = 9 * b * b - 20 * a * c;
    if (c == 0.0) {
      const double y = b == 0.0 ? -1.0 : -a / (3 * b);
      if (y > 0.0 && y < t) next = std::max(next, step(y));
    } else if (q >= 0.0) {
      for (double r : {std::sqrt(q), -std::sqrt(q)}) {
        const double y = (-3 * b + r) / (10 * c);
        if (y > 0.0 && y < t) next = std::max(next, step(y));
      }
    }
    top = next;
  }
  return std::isfinite(top);
}

hipError_t launch_ortho(const k3moe_ortho& p, const void* g, void* out, const OrthoWs& ws, hipStream_t st) {
  const Dims d(p);
  const int64_t count = (int64_t)d.rows * d.cols;
  const int pieces = pieces_of(d);
  const int64_t piece = ((count + pieces - 1) / pieces + 7) & ~int64_t(7);
  const bool f32 = p.dtype == K3MOE_F32;
  const dim3 sums(pieces, d.batch), tiles(d.l / 64, d.s / 64, d.batch);
  if (f32) square_sums<true><<<sums, 256, 0, st>>>(g, ws.sums, count, piece);
  else square_sums<false><<<sums, 256, 0, st>>>(g, ws.sums, count, piece);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  auto scale = [&](auto kernel) {
    kernel<<<tiles, 256, 0, st>>>(g, ws.sums, ws.x[0], ws.lo, d.s, d.l, d.rows, d.cols, pieces);
  };
  if (d.tr) f32 ? scale(scale_in<true, true>) : scale(scale_in<true, false>);
  else f32 ? scale(scale_in<false, true>) : scale(scale_in<false, false>);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  OrthoArgs a{};
  a.lo = ws.lo;
  a.A = ws.A;
  a.B = ws.B;
  a.out = out;
  a.part = ws.part;
  a.s = d.s;
  a.l = d.l;
  a.batch = d.batch;
  a.rows = d.rows;
  a.cols = d.cols;
  a.scale = p.scale / kScaleX;
  for (int i = 0; i < p.steps; ++i) {
    a.x = ws.x[i & 1];
    a.xo = ws.x[~i & 1];
    a.ca = p.coefficients[3 * i];
    a.cb = p.coefficients[3 * i + 1];
    a.cc = p.coefficients[3 * i + 2];
    a.keep_lo = i + 2 < p.steps;
    if ((e = launch_product<kGram>(d, a, st)) != hipSuccess) return e;
    if ((e = launch_product<kPoly>(d, a, st)) != hipSuccess) return e;
    if (i + 1 < p.steps) e = launch_product<kStep>(d, a, st);
    else e = d.tr ? launch_product<kLastT>(d, a, st) : launch_product<kLast>(d, a, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace k3
