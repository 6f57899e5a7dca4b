// The shared (dense, bf16) experts' training pass: the forward that keeps the
// pre-activations, and the backward.  S experts of width fs, F = S fs hidden
// features side by side:
//   forward   [g u] = x W13^T             h = g sigmoid(g) u        y = h W2^T
//   backward  dh = dy W2                  s = sigmoid(g)
//             du = dh g s                 dg = dh u s (1 + g (1 - s))
//             dx = [dg du] W13            dW13 = [dg du]^T x        dW2 = dy^T h
// Six matrix products of one kind, so one tile kernel (dense_tile) runs them
// all on v_mfma_f32_16x16x32_bf16; the products differ in which operand has
// its contraction along the rows of memory and in what the epilogue does with
// the fp32 sums: the gated activation is taken in the forward's epilogue from
// the gate and up sums of one wave, its derivative in the epilogue of dh.
// g, u (for the backward), h, dg, du and every output are rounded to bf16
// once, from fp32: they are operands of the next bf16 product.  Up to kRows tokens
// h, dg and du keep 15 bits or more, as two bf16 parts in two blocks of kRows rows: their
// products read the weights' every byte whatever the rows, and a rounding to 8 bits
// of so few values does not average out (an output's error of sqrt(2) of its own
// rounding alone, but up to twice that for one token of a small layer).  That costs
// nothing (T = 16 forward 46.7, backward 117 us; T = 17 46.6, 116).  Where the
// parts are rows of a product, its sums of a row and of the one kRows further are
// added; where they are contracted over, the other operand's rows are taken twice.
// From about 2000 tokens the matrix cores bound all six (d 7168, two experts of 2048,
// T = 16384: dx 1.37 ms = 1.40 PFLOP/s, dW13 and dW2 2.27 ms = 1.27, dh 0.86 ms =
// 1.12, whose epilogue moves 670 MB; the library's product of such sizes reaches 1.4
// to 1.5): they are busy 60 to 65 % of the time at the 1.95 GHz that this load
// leaves, what is missing being LDS reads and copies between them.  That is where the
// tiles fill whole rounds of the CUs; a last round of a few tiles takes as long as a
// full one (forward at T = 4096 539 us, 4097 654, 2500 447).  Below about 300
// tokens reading the weights (backward: and writing their gradients) bounds them:
// T = 1 forward 45 us for 176 MB, backward 115 us for 352 MB.
#include <algorithm>

#include "internal.h"
#include "kern_common.h"
#include "grouped.h"

namespace k3 {
namespace {

using namespace grouped;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kBK = 64;   // contraction elements per stage
constexpr int kRows = 16; // up to so many tokens h, dg and du have two parts

// The products.  M x N is the output, K the contraction:
//   kGateUp  M = T   N = F  K = d    a = x       b = w13 (gate and up rows of N features)
//   kDown    M = T   N = d  K = F    a = h       b = w2
//   kDHid    M = T   N = F  K = d    a = dy      b = w2
//   kDX      M = T   N = d  K = 2F   a = dgu     b = w13
//   kDW13    M = 2F  N = d  K = T    a = dgu     b = x
//   kDW2     M = d   N = F  K = T    a = dy      b = h
enum Product { kGateUp, kDown, kDHid, kDX, kDW13, kDW2 };

struct DenseArgs {
  const uint16_t* a;
  const uint16_t* b;
  const uint16_t* gu;   // kDHid: the kept pre-activations [T][S][2 fs]
  void* o0;             // kGateUp: gu; kDHid: dgu; else the product
  uint16_t* o1;         // kGateUp, kDHid: h [T][F]
  int T, d, fs, S;
  int out_f32;          // kDown: y in fp32
  int parts;            // T <= kRows: h and dgu are [2 kRows] rows, second parts from kRows on
  float* part;          // split contraction: partial sums [splits][M][columns]
  int splits, k_split;  // contraction elements per split (a multiple of kBK)
  int m_lo, m_hi;       // kDW2: the rows of M taken (m_lo a multiple of the tile's)
};

// A voffset past num_records: the copy writes zeros to LDS.  Every offset of
// an element inside a tile stays below 2^31 (at most two experts' matrices).
constexpr uint32_t kRecords = 0x80000000u;
constexpr uint32_t kOut = 0xFFFFFFF0u;

// Buffer descriptor over base p (wave-uniform).
__device__ __forceinline__ u32x4_t rsrc_of(uint64_t p) {
  u32x4_t r;
  r.x = __builtin_amdgcn_readfirstlane((uint32_t)p);
  r.y = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));   // 48-bit address, stride 0
  r.z = kRecords;
  r.w = 0x00020000u;
  return r;
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// LDS-DMA copy with a range check: lane i's 16 bytes at base + voff (zeros
// when voff is kOut) land at lds + 16 i.
__device__ __forceinline__ void dma16_buf(u32x4_t rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory", "m0");
}
#pragma clang diagnostic pop

// bf16 roundings (to nearest even, v_cvt_pk_bf16_f32) packed.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) float f2;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, bf16x2_t));
}
__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
  return make_uint2(pack2(a, b), pack2(c, d));
}

// sigmoid(g) from the hardware's exp2 and reciprocal: off by about |g| 2^-24
// of its value, far inside the bf16 rounding of everything made from it.  For g
// below -88 the exponential is +inf and the result 0, so g sigmoid(g) is -0
// there, never NaN.
__device__ __forceinline__ float sigmoid_fast(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// An operand tile of R rows (of M or N) x 64 contraction elements in LDS.
//   KC (contraction contiguous in memory): row r is 128 bytes; 16-byte unit u
//     of it sits at position u ^ ((r >> 1) & 7), so the 16 rows of a fragment
//     read fall on distinct 4-bank groups.
//   otherwise (rows contiguous): contraction element k is a line of 2 R bytes;
//     the 32 bytes of row block b (16 rows) sit at position b ^ key(k),
//     key = k mod 4 | (k / 8 mod 2) << 2, so the eight lines that half a wave's
//     transposing read touches fall on distinct 8-bank groups.
template <bool KC, int R>
struct Operand {
  static constexpr int kSlot = R * 128;
  static constexpr int kKeyMask = R / 16 >= 8 ? 7 : R / 16 - 1;
  static_assert(KC || R >= 32, "two row blocks at least");

  __device__ static __forceinline__ int key(int k) { return ((k & 3) | ((k >> 1) & 4)) & kKeyMask; }
  // Source row and first contraction element of LDS unit U (16 bytes) of a slot.
  __device__ static __forceinline__ void unit(int U, int& r, int& k) {
    if (KC) {
      r = U >> 3;
      k = ((U & 7) ^ ((r >> 1) & 7)) * 8;
    } else {
      constexpr int W = R / 8;
      k = U / W;
      const int p = U - k * W;
      r = (((p >> 1) ^ key(k)) << 4) + (p & 1) * 8;
    }
  }
  // Fragment of row block rb (16 rows), contraction half j: lane (ln, lg)
  // holds row ln, elements 32 j + 8 lg .. + 8.
  __device__ static __forceinline__ bf16x8_t frag(const uint8_t* base, int rb, int j, int ln, int lg) {
    if (KC) {
      const int r = rb * 16 + ln;
      return __builtin_bit_cast(
          bf16x8_t, *reinterpret_cast<const uint4*>(base + r * 128 + (((4 * j + lg) ^ ((r >> 1) & 7)) << 4)));
    }
    const int k = 32 * j + 8 * lg + (ln >> 2);
    const uint8_t* p = base + k * (R * 2) + ((rb ^ key(k)) << 5) + (ln & 3) * 8;
    union { s16x4_t h[2]; bf16x8_t v; } f;
    f.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p));
    f.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * R * 2));
    return f.v;
  }
};

template <int P, int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN;
  static constexpr bool A_KC = P == kGateUp || P == kDown || P == kDHid || P == kDX;
  static constexpr bool B_KC = P == kGateUp || P == kDown;
  static constexpr int MF = BM / 16 / WM, NF = BN / 16 / WN;
  static constexpr int NA = BM * 8 / 64 / NW, NB = BN * 8 / 64 / NW;   // copies per wave and stage
  static constexpr int kN = P == kGateUp ? BN / 2 : BN;               // outputs of N per tile
  using A = Operand<A_KC, BM>;
  using B = Operand<B_KC, BN>;
  static_assert(NA * 64 * NW == BM * 8 && NB * 64 * NW == BN * 8 && MF >= 1 && NF >= 1, "whole copies");
  static_assert(NF == 2 || NF % 4 == 0, "fragments (and pairs of gate and up) side by side");
};

// Column (row of w13) of hidden feature n's gate in [2 F]; its up is fs further.
__device__ __forceinline__ int gate_col(int n, int fs) { return n + n / fs * fs; }

// ---- epilogues.  A fragment's sums give a lane four consecutive columns of a row;
// two fragments side by side, their odd and even groups of 16 lanes exchanged, give
// it eight: lane group lg then has columns 8 (lg / 2) .. + 8 of fragment lg mod 2,
// a store is 16 bytes and a row's part of it 64 (with stores of 8 and 32 the
// backward took 8 % longer at T = 64 and 3 % at 16384).
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const auto t = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = t[0];
  b = t[1];
}
__device__ __forceinline__ uint4 pack8(f32x4_t a, f32x4_t b) {
  uint2 p = pack4(a[0], a[1], a[2], a[3]), q = pack4(b[0], b[1], b[2], b[3]);
  exchange(p.x, q.x);
  exchange(p.y, q.y);
  return make_uint4(p.x, p.y, q.x, q.y);
}
// v as two bf16 parts (the second once rounded): its top 8 bits and the rest.  Both
// have v's sign and neither is zero unless v is (a v of 8 bits is halved), and an
// infinity or NaN is both: a part times an infinity is what v times it is.
__device__ __forceinline__ float take_rest(float& v) {
  const float top = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u), d = v - top;
  const bool whole = !(fabsf(d) > 0.0f);   // 8 bits, or not finite
  v = whole ? 0.5f * v : top;
  return whole ? v : d;
}
__device__ __forceinline__ f32x4_t take_rest(f32x4_t& v) {
  f32x4_t l;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float x = v[r];
    l[r] = take_rest(x);
    v[r] = x;
  }
  return l;
}
__device__ __forceinline__ f32x4_t gated(f32x4_t ga, f32x4_t up) {
  f32x4_t h;
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = ga[r] * sigmoid_fast(ga[r]) * up[r];
  return h;
}
// The forward's gate and up sums of row m: columns n .. + 4, or, of two
// fragments, the lane's eight from n on.  FEW: T may be at most kRows.
template <bool FEW>
__device__ __forceinline__ void store_gateup(const DenseArgs& g, int m, int n, f32x4_t ga, f32x4_t up) {
  const int F = g.S * g.fs;
  f32x4_t h = gated(ga, up);
  if (FEW && g.parts) {
    const f32x4_t l = take_rest(h);
    *reinterpret_cast<uint2*>(g.o1 + (size_t)(m + kRows) * F + n) = pack4(l[0], l[1], l[2], l[3]);
  }
  uint16_t* gu = static_cast<uint16_t*>(g.o0) + (size_t)m * 2 * F + gate_col(n, g.fs);
  *reinterpret_cast<uint2*>(gu) = pack4(ga[0], ga[1], ga[2], ga[3]);
  *reinterpret_cast<uint2*>(gu + g.fs) = pack4(up[0], up[1], up[2], up[3]);
  *reinterpret_cast<uint2*>(g.o1 + (size_t)m * F + n) = pack4(h[0], h[1], h[2], h[3]);
}
template <bool FEW>
__device__ __forceinline__ void store_gateup(const DenseArgs& g, int m, int n, bool in, f32x4_t ga0,
                                             f32x4_t up0, f32x4_t ga1, f32x4_t up1) {
  const int F = g.S * g.fs;
  f32x4_t h0 = gated(ga0, up0), h1 = gated(ga1, up1);
  uint4 l{};
  if (FEW && g.parts) {
    const f32x4_t l0 = take_rest(h0), l1 = take_rest(h1);
    l = pack8(l0, l1);
  }
  const uint4 ga = pack8(ga0, ga1), up = pack8(up0, up1), h = pack8(h0, h1);
  if (!in) return;
  uint16_t* gu = static_cast<uint16_t*>(g.o0) + (size_t)m * 2 * F + gate_col(n, g.fs);
  *reinterpret_cast<uint4*>(gu) = ga;
  *reinterpret_cast<uint4*>(gu + g.fs) = up;
  *reinterpret_cast<uint4*>(g.o1 + (size_t)m * F + n) = h;
  if (FEW && g.parts) *reinterpret_cast<uint4*>(g.o1 + (size_t)(m + kRows) * F + n) = l;
}
// dh's sums v of row m: dg, du and h from the kept g and u (two bf16 values a word),
// or, of parts, their first and second parts.
template <bool FEW>
__device__ __forceinline__ void gate_grads(const float* v, uint32_t gw, uint32_t uw, bool parts,
                                           uint32_t (&out)[3], uint32_t (&low)[3]) {
  float d[2][3];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float ga = r ? bf16_hi(gw) : bf16_lo(gw), up = r ? bf16_hi(uw) : bf16_lo(uw);
    const float s = sigmoid_fast(ga), gs = ga * s;
    d[r][0] = v[r] * up * (s + gs * (1.0f - s));
    d[r][1] = v[r] * gs;
    d[r][2] = gs * up;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (FEW && parts) {
      const float l0 = take_rest(d[0][i]), l1 = take_rest(d[1][i]);
      low[i] = pack2(l0, l1);
    }
    out[i] = pack2(d[0][i], d[1][i]);
  }
}
template <bool FEW, int W, typename V>   // W words of two columns each
__device__ __forceinline__ void store_dhid_words(const DenseArgs& g, int m, int n, const float* v) {
  const int F = g.S * g.fs;
  const size_t o = (size_t)m * 2 * F + gate_col(n, g.fs);
  const V gw = *reinterpret_cast<const V*>(g.gu + o), uw = *reinterpret_cast<const V*>(g.gu + o + g.fs);
  V out[3], low[3];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    uint32_t a[3], b[3] = {0, 0, 0};
    gate_grads<FEW>(v + 2 * w, gw[w], uw[w], g.parts, a, b);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      out[i][w] = a[i];
      if (FEW) low[i][w] = b[i];
    }
  }
  auto put = [&](const V (&q)[3], int row) {
    uint16_t* o0 = static_cast<uint16_t*>(g.o0) + o + (size_t)row * 2 * F;
    *reinterpret_cast<V*>(o0) = q[0];
    *reinterpret_cast<V*>(o0 + g.fs) = q[1];
    *reinterpret_cast<V*>(g.o1 + (size_t)(m + row) * F + n) = q[2];
  };
  put(out, 0);
  if (FEW && g.parts) put(low, kRows);
}
template <bool FEW>
__device__ __forceinline__ void store_dhid(const DenseArgs& g, int m, int n, f32x4_t v) {
  const float a[4] = {v[0], v[1], v[2], v[3]};
  store_dhid_words<FEW, 2, u32x2_t>(g, m, n, a);
}
template <bool FEW>
__device__ __forceinline__ void store_dhid(const DenseArgs& g, int m, int n, bool in, f32x4_t v0,
                                           f32x4_t v1) {
  float v[8];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    uint32_t a = __float_as_uint(v0[r]), b = __float_as_uint(v1[r]);
    exchange(a, b);
    v[r] = __uint_as_float(a);
    v[4 + r] = __uint_as_float(b);
  }
  if (in) store_dhid_words<FEW, 4, u32x4_t>(g, m, n, v);
}
template <int P>
__device__ __forceinline__ size_t product_at(const DenseArgs& g, int m, int n, int N) {
  // dW2 [S][d][fs]: column n is feature n % fs of expert n / fs
  return P == kDW2 ? ((size_t)(n / g.fs) * g.d + m) * g.fs + n % g.fs : (size_t)m * N + n;
}
template <int P>
__device__ __forceinline__ void store_product(const DenseArgs& g, int m, int n, int N, f32x4_t v) {
  if (P == kDown && g.out_f32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(g.o0) + (size_t)m * N + n) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.o0) + product_at<P>(g, m, n, N)) =
        pack4(v[0], v[1], v[2], v[3]);
}

constexpr int kGM = 8;   // m-tiles per group of the item order

// Where a workgroup's items lie: rounds rd0 .. rd1 of G items each, of every
// round the wi-th item of XCD xcd's piece.
struct Items {
  int G, xcd, wi, rd0, rd1;
};

// The tiles of one product that `at` names.  SPLIT: an item is a tile and one of
// g.splits pieces of the contraction; its sums go to g.part, and split_finish adds
// the pieces in order.
template <int P, int BM, int BN, int WM, int WN, int RING, bool SPLIT>
__device__ __forceinline__ void run_tiles(const DenseArgs& g, const Items at, uint8_t* sA, uint8_t* sB) {
  using C = Tile<P, BM, BN, WM, WN>;
  using OA = typename C::A;
  using OB = typename C::B;
  constexpr int MF = C::MF, NF = C::NF;

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const int T = g.T, d = g.d, fs = g.fs, F = g.S * g.fs;
  const int M = P == kDW13 ? 2 * F : P == kDW2 ? g.m_hi : T;
  const int m_lo = P == kDW2 ? g.m_lo : 0;
  const int N = P == kGateUp || P == kDHid || P == kDW2 ? F : d;
  const int K = P == kGateUp || P == kDHid ? d : P == kDown ? F : P == kDX ? 2 * F
                                               : g.parts ? 2 * kRows : T;
  constexpr bool kFew = BM <= 128;   // (256 x 256 is no tile for the other products of few tokens)
  constexpr bool kPartRows = kFew && (P == kDown || P == kDX), kPartK = P == kDW13 || P == kDW2;
  const int a_rows = kPartRows && g.parts ? 2 * kRows : M;
  const int n_mt = (M - m_lo + BM - 1) / BM, n_nt = (N + C::kN - 1) / C::kN;
  const int n_cols = SPLIT ? n_nt * g.splits : n_nt;   // n-tiles, every split's in turn
  const int n_items = n_mt * n_cols;
  // This workgroup's item of round r (n_items: none).  A round takes the next G
  // items, its 8 contiguous pieces one to an XCD, the last round's shorter ones
  // too: the XCDs work on neighbouring tiles at any time, so what they all read
  // (a group's rows of A, all of B) stays in the last-level cache.
  auto item_of = [&](int r) {
    const int first = r * at.G, piece = (min(at.G, n_items - first) + 7) >> 3;
    const int it = first + at.xcd * piece + at.wi;
    return r < at.rd1 && first < n_items && at.wi < piece && it < min(first + at.G, n_items)
               ? it : n_items;
  };

  // Items: groups of kGM m-tiles, the m-tile fastest, then the n-tile, so the
  // workgroups of an XCD share both operands through its L2.
  auto item_tile = [&](int it, int& m0, int& n0, int& k0, int& k1) {
    const int per = kGM * n_cols, grp = it / per, first = grp * kGM;
    const int r = it - grp * per, gsz = min(n_mt - first, kGM), nt = r / gsz;
    const int sp = SPLIT ? nt / n_nt : 0;
    n0 = (nt - sp * n_nt) * C::kN;
    m0 = m_lo + (first + r - nt * gsz) * BM;
    k0 = SPLIT ? sp * g.k_split : 0;
    k1 = SPLIT ? min(k0 + g.k_split, K) : K;
    return sp;
  };

  // ---- copies: this wave's units of both operands, as byte offsets from the
  // tile's first element (kOut: outside the matrix), and that element's
  // address, which advances with the stage.
  uint32_t va[C::NA], vb[C::NB];
  const size_t lda = P == kGateUp || P == kDHid || P == kDW2 ? d : P == kDown ? F : 2 * F;
  const size_t ldb = P == kGateUp || P == kDX || P == kDW13 ? d : P == kDW2 ? F : fs;
  const uint32_t sa = C::A_KC ? kBK * 2 : kBK * 2 * (uint32_t)lda;   // bytes per stage
  const uint32_t sb = C::B_KC ? kBK * 2 : kBK * 2 * (uint32_t)ldb;
  uint64_t pa, pb;
  int c_rd = at.rd0, c_k, c_end;   // the copies' round, first contraction element and end
  int c_it = item_of(c_rd);
  int c_ko = 0;                      // kDown: c_k within its expert's features
  auto setup = [&]() {
    int m0, n0;
    item_tile(c_it, m0, n0, c_k, c_end);
    pa = (uint64_t)(uintptr_t)(g.a + (C::A_KC ? (size_t)m0 * lda + c_k : (size_t)c_k * lda + m0));
#pragma unroll
    for (int c = 0; c < C::NA; ++c) {
      int r, k;
      OA::unit((wv * C::NA + c) * 64 + lane, r, k);
      bool in = m0 + r < a_rows;
      if (kPartK && g.parts) {   // (one stage: k is the row)
        in = in && (k & (kRows - 1)) < T;
        if (P == kDW2) k &= kRows - 1;
      }
      const size_t e = C::A_KC ? (size_t)r * lda + k : (size_t)k * lda + r;
      va[c] = in ? (uint32_t)(e * 2) : kOut;
    }
    const int gc0 = gate_col(n0, fs);
    if (P == kDown) c_ko = c_k % fs;
    pb = (uint64_t)(uintptr_t)(
        g.b + (P == kGateUp ? (size_t)gc0 * d + c_k
               : P == kDHid ? (size_t)(n0 / fs) * d * fs + n0 % fs + (size_t)c_k * fs
               : P == kDown ? (size_t)(c_k / fs) * d * fs + (size_t)n0 * fs + c_ko
                            : (size_t)c_k * ldb + n0));
#pragma unroll
    for (int c = 0; c < C::NB; ++c) {
      int r, k;
      OB::unit((wv * C::NB + c) * 64 + lane, r, k);
      if (P == kGateUp) {
        // each wave's NF fragments: NF / 2 of gate rows, then the matching up rows
        const int w = r / (16 * NF), f = (r >> 4) % NF;
        const int n = n0 + w * (8 * NF) + (f % (NF / 2)) * 16 + (r & 15);
        const int row = gate_col(n, fs) + (f >= NF / 2 ? fs : 0) - gc0;
        vb[c] = n < N ? (uint32_t)(((size_t)row * d + k) * 2) : kOut;
      } else if (P == kDHid) {
        // the columns of several experts' matrices: expert s's starts s d fs further
        const int n = n0 + r;
        const size_t e = (size_t)(n / fs - n0 / fs) * d * fs + n % fs + (size_t)k * fs;
        vb[c] = n < N ? (uint32_t)((e - n0 % fs) * 2) : kOut;
      } else {
        bool in = n0 + r < N;
        if (kPartK && g.parts) {
          in = in && (k & (kRows - 1)) < T;
          if (P == kDW13) k &= kRows - 1;
        }
        const size_t e = C::B_KC ? (size_t)r * ldb + k : (size_t)k * ldb + r;
        vb[c] = in ? (uint32_t)(e * 2) : kOut;
      }
    }
  };
  // Copy c of the stage at c_k (A's units, then B's) into `slot`.
  auto copy = [&](int slot, int c) {
    const bool isa = c < C::NA;
    const int q = isa ? c : c - C::NA, n = isa ? C::NA : C::NB;
    const uint32_t to = lds_addr(isa ? sA : sB) +
                        (uint32_t)(slot * (isa ? OA::kSlot : OB::kSlot) + (wv * n + q) * 1024);
    int r, k;
    if (isa) OA::unit((wv * n + q) * 64 + lane, r, k); else OB::unit((wv * n + q) * 64 + lane, r, k);
    uint32_t v = isa ? va[q] : vb[q];
    uint64_t p = isa ? pa : pb;
    if (P == kDown && !isa) {
      // units past the end of expert c_k / fs's rows (fs may be 32: two ends)
      const uint32_t next = (uint32_t)(d - 1) * fs * 2;
      v += (c_ko + k >= fs ? next : 0u) + (c_ko + k >= 2 * fs ? next : 0u);
      v = vb[q] == kOut ? kOut : v;
    }
    dma16_buf(rsrc_of(p), c_k + kBK > c_end && c_k + k >= c_end ? kOut : v, to);
  };
  auto advance = [&]() {   // the copies' next stage
    c_k += kBK;
    pa += sa;
    pb += sb;
    if (P == kDown) {
      c_ko += kBK;
      while (c_ko >= fs) {   // into the next expert's matrix
        c_ko -= fs;
        pb += (uint64_t)(d - 1) * fs * 2;
      }
    }
    if (c_k >= c_end) {
      c_it = item_of(++c_rd);
      if (c_it < n_items) {
        setup();
      } else {   // behind the last item: zeros, that nothing uses
#pragma unroll
        for (int c = 0; c < C::NA; ++c) va[c] = kOut;
#pragma unroll
        for (int c = 0; c < C::NB; ++c) vb[c] = kOut;
      }
    }
  };

  const int wm = wv / WN, wn = wv - wm * WN;
  // Fragments of one 32-element half: a step's MFMAs use row block i of A and
  // every block of B; the next half's reads are spread over all but the last
  // two steps, so they have landed when its first MFMA issues.
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
        acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[f], fa[i], acc[i][f], 0, 0, 0);
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
  for (int rd = at.rd0, it; (it = item_of(rd)) < n_items; ++rd) {
    int m0, n0, k0, k1;
    const int sp = item_tile(it, m0, n0, k0, k1);
    const int nst = (k1 - k0 + kBK - 1) / kBK;
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
    // ---- epilogue: lane (ln, lg) holds m = m0 + 16 (wm MF + i) + ln, four n
    if constexpr (kPartRows) {
      static_assert(MF >= 2, "both parts of a row in one lane");
      if (g.parts) {   // (the first wave's rows 0 .. 15 and 16 .. 31)
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[0][f] += acc[1][f];
      }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = m0 + (wm * MF + i) * 16 + ln;
      if (m >= M) continue;
      if constexpr (SPLIT) {
        const int cols = P == kGateUp ? 2 * F : N;
        float* row = g.part + ((size_t)sp * M + m) * cols;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const int n = P == kGateUp ? n0 + wn * (8 * NF) + (f % (NF / 2)) * 16 + lg * 4
                                     : n0 + (wn * NF + f) * 16 + lg * 4;
          if (n >= N) continue;
          const int c = P == kGateUp ? gate_col(n, fs) + (f >= NF / 2 ? fs : 0) : n;
          *reinterpret_cast<f32x4_t*>(row + c) = acc[i][f];
        }
      } else if constexpr (P == kGateUp && NF == 2) {
        const int n = n0 + wn * 16 + lg * 4;
        if (n < N) store_gateup<kFew>(g, m, n, acc[i][0], acc[i][1]);
      } else if constexpr (P == kGateUp) {
#pragma unroll
        for (int f = 0; f < NF / 2; f += 2) {
          const int n = n0 + wn * (8 * NF) + (f + (lg & 1)) * 16 + (lg >> 1) * 8;
          store_gateup<kFew>(g, m, n, n < N, acc[i][f], acc[i][f + NF / 2], acc[i][f + 1],
                       acc[i][f + 1 + NF / 2]);
        }
      } else if (P == kDown && g.out_f32) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const int n = n0 + (wn * NF + f) * 16 + lg * 4;
          if (n < N) store_product<P>(g, m, n, N, acc[i][f]);
        }
      } else {
#pragma unroll
        for (int f = 0; f < NF; f += 2) {
          const int n = n0 + (wn * NF + f + (lg & 1)) * 16 + (lg >> 1) * 8;
          if constexpr (P == kDHid) {
            store_dhid<kFew>(g, m, n, n < N, acc[i][f], acc[i][f + 1]);
          } else {
            const uint4 v = pack8(acc[i][f], acc[i][f + 1]);
            if (n < N)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.o0) + product_at<P>(g, m, n, N)) = v;
          }
        }
      }
    }
  }
}

template <int P, int BM, int BN, int WM, int WN, int RING = 2, bool SPLIT = false>
__global__ __launch_bounds__(64 * WM * WN) void dense_tile(DenseArgs g) {
  __shared__ __attribute__((aligned(16))) uint8_t sA[RING * BM * 2 * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sB[RING * BN * 2 * kBK];
  const Items at{(int)gridDim.x, (int)blockIdx.x & 7, (int)blockIdx.x >> 3, 0, 1 << 30};
  run_tiles<P, BM, BN, WM, WN, RING, SPLIT>(g, at, sA, sB);
}

// dx (on XM x XN tiles), dW13 and dW2 in one launch: none depends on another, and
// none's tiles fill its last round of CUs.  kCUs workgroups for every n[p] rounds of product p, dx's
// first (they are the longest); a CU that has no dx tile, or is done with it, takes
// a workgroup of the next product.
constexpr int kCUs = 256;
struct GradArgs {
  DenseArgs g[3];
  int n[3], wgs[3];
};
template <int XM, int XN, int XRING, int BM, int BN, int RING, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void dense_grads(GradArgs a) {
  constexpr int kA = XRING * XM > RING * BM ? XRING * XM : RING * BM;
  constexpr int kB = XRING * XN > RING * BN ? XRING * XN : RING * BN;
  __shared__ __attribute__((aligned(16))) uint8_t sA[kA * 2 * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sB[kB * 2 * kBK];
  int wg = blockIdx.x;   // (every product's first is a multiple of 8, so wg & 7 is the XCD)
  auto items = [&](int p) {
    const int w = wg >> 3, r = w / (kCUs / 8) * a.n[p];
    return Items{kCUs, wg & 7, w % (kCUs / 8), r, r + a.n[p]};
  };
  if (wg < a.wgs[0]) return run_tiles<kDX, XM, XN, WM, WN, XRING, false>(a.g[0], items(0), sA, sB);
  wg -= a.wgs[0];
  if (wg < a.wgs[1]) return run_tiles<kDW13, BM, BN, WM, WN, RING, false>(a.g[1], items(1), sA, sB);
  wg -= a.wgs[1];
  run_tiles<kDW2, BM, BN, WM, WN, RING, false>(a.g[2], items(2), sA, sB);
}

// The pieces of a split contraction added in order, and the product's epilogue:
// one thread per row and four columns.
template <int P>
__global__ __launch_bounds__(256) void split_finish(DenseArgs g) {
  const int F = g.S * g.fs, M = g.T;
  const int N = P == kGateUp || P == kDHid ? F : g.d, cols = P == kGateUp ? 2 * F : N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int m = (int)(i / (N / 4)), n = (int)(i - (int64_t)m * (N / 4)) * 4;
  if (m >= M) return;
  const float* p = g.part + (size_t)m * cols + (P == kGateUp ? gate_col(n, g.fs) : n);
  f32x4_t a = {0.f, 0.f, 0.f, 0.f}, b = a;
  for (int s = 0; s < g.splits; ++s, p += (size_t)M * cols) {
    a += *reinterpret_cast<const f32x4_t*>(p);
    if (P == kGateUp) b += *reinterpret_cast<const f32x4_t*>(p + g.fs);
  }
  if constexpr (P == kGateUp) store_gateup<true>(g, m, n, a, b);
  else if constexpr (P == kDHid) store_dhid<true>(g, m, n, a);
  else store_product<P>(g, m, n, N, a);
}

__global__ __launch_bounds__(256) void zero_fill(uint4* p, size_t n16) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += (size_t)gridDim.x * 256)
    p[i] = make_uint4(0, 0, 0, 0);
}

// How a product runs: its tile and, for the smallest, the pieces its contraction
// is split into.
enum { kTile256, kTile128x256, kTile128, kTile64 };
struct Plan {
  int tile, splits, k_split;
};

// The tile whose rounds cost least, by what a 64-element stage was measured to
// take (us; d 7168, two experts of 2048, weights from HBM):
//   256 x 256, 2 slots, one workgroup a CU:    1.6;  the fastest from T = 2048 on
//     (gate/up 185 us there, against 208 on 128 x 256)
//   128 x 256, 3 slots, one workgroup a CU:    0.95;  gate/up 93 us at T = 517
//     (167 on 256 x 256, 120 on 128 x 128; 132 with 2 slots)
//   128 x 128, 3 slots, one workgroup a CU:    0.65;  dh 75 us at T = 1000 (108 on
//     128 x 256, 122 on 64 x 64)
//   64 x 64, 3 slots, three workgroups a CU:   0.43 (one a CU), 0.5 (two), 0.64;
//     gate/up 57 us at T = 200 (66 on 128 x 128; 92 with 2 slots)
// Where the outputs are few, the contraction is split, so that every CU loads a part
// of the weights: on 64 x 64 tiles below about 100 tokens, on the larger ones up to
// about 800 (forward at T = 128 59 us against 76 without a split on larger tiles,
// T = 256 80, 107; backward at T = 512 225, 247).  The sums of a piece then cost
// their way to memory and back, and a second kernel 5 us.
// A weight gradient's contraction can be a few tokens: there a tile's way out counts
// (us a round: 9, 4.6, 2.7, 1.9; both gradients at T = 64 65, 61, 63, 71).
constexpr double kPartUs = 1.6e-6;   // a partial sum written and read, 8 bytes
Plan plan_product(int P, const k3moe_shape& s) {
  const int64_t F = (int64_t)s.n_shared * s.f_shared, T = s.T, d = s.d;
  const int64_t M = P == kDW13 ? 2 * F : P == kDW2 ? d : T;
  const int64_t N = P == kGateUp || P == kDHid || P == kDW2 ? F : d;
  const int64_t K = P == kGateUp || P == kDHid ? d : P == kDown ? F : P == kDX ? 2 * F : T;
  const int64_t nst = (K + kBK - 1) / kBK, w = P == kGateUp ? 2 : 1;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N * w + bn - 1) / bn); };
  auto rounds = [](int64_t n, int64_t slots) { return (double)((n + slots - 1) / slots); };
  const int64_t t64 = tiles(64, 64);
  const bool dw = P == kDW13 || P == kDW2;
  double best = t64 <= 256 ? 0.43 * nst : t64 <= 512 ? 0.5 * nst
                           : rounds(t64, 768) * (0.64 * nst + (dw ? 1.9 : 0.0));
  Plan p{kTile64, 1, 0};
  if (!dw && t64 <= 384) {
    int64_t n = std::min<int64_t>(768 / t64, nst / 4);
    if (n > 1) {
      const int64_t per = (nst + n - 1) / n;
      n = (nst + per - 1) / per;
      const double c = 0.64 * per + 5.0 + kPartUs * n * M * N * w;
      if (c < best) {
        best = c;
        p.splits = (int)n;
        p.k_split = (int)(per * kBK);
      }
    }
  }
  auto consider = [&](int tile, int64_t t, double stage, double out) {
    const double c = rounds(t, 256) * (stage * nst + (dw ? out : 0.0));
    if (c < best) best = c, p = Plan{tile, 1, 0};
    // (dx shares its launch with the weight gradients, whose tiles fill its rounds)
    if (P == kDX || dw || t > 256) return;
    for (int64_t n = 2; n <= 8 && 4 * n <= nst; ++n) {
      const int64_t per = (nst + n - 1) / n;
      if ((n - 1) * per >= nst) continue;
      const double split = rounds(t * n, 256) * stage * per + 5.0 + kPartUs * n * M * N * w;
      if (split < best) best = split, p = Plan{tile, (int)n, (int)(per * kBK)};
    }
  };
  consider(kTile128, tiles(128, 128), 0.65, 2.7);
  consider(kTile128x256, tiles(128, 256), 0.95, 4.6);
  const double c256 = rounds(tiles(256, 256), 256) * (1.6 * nst + (dw ? 9.0 : 0.0));
  if (c256 <= best && (dw || T > kRows)) p = Plan{kTile256, 1, 0};
  return p;
}

// Both weight gradients on 256 x 256 tiles, in one launch whose rounds are all full:
// the rows of dW2 that do not fit go to 128 x 128 tiles, four times as many, in a
// launch of their own.  -1: two launches take no longer.  (T = 16384, d 7168, two
// experts of 2048: 896 and 448 tiles, 4 and 2 rounds; here 5 and 1024 rows of dW2 in
// one round of the small tiles: backward 4.31 ms against 4.39.)
int64_t tail_rows(const k3moe_shape& s) {
  if (plan_product(kDW13, s).tile != kTile256 || plan_product(kDW2, s).tile != kTile256) return -1;
  const int64_t F = (int64_t)s.n_shared * s.f_shared;
  const int64_t nd = (s.d + 255) / 256, nf = (F + 255) / 256, t13 = (2 * F + 255) / 256 * nd;
  const int64_t total = t13 + nd * nf, over = (total % kCUs + nf - 1) / nf;   // tile rows of dW2
  if (over >= nd) return -1;
  const int64_t rows = over == 0 ? 0 : s.d - (nd - over) * 256;
  auto rounds = [](int64_t n) { return (double)((n + kCUs - 1) / kCUs); };
  const double two = 1.6 * (rounds(t13) + rounds(nd * nf));
  const double one = 1.6 * (double)(total / kCUs) +
                     0.65 * rounds((rows + 127) / 128 * ((F + 127) / 128));
  return one < 0.98 * two ? rows : -1;
}

// Floats of the partial sums of a split product (0 when it is not split).
size_t part_floats(int P, const k3moe_shape& s) {
  const Plan p = plan_product(P, s);
  const size_t F = (size_t)s.n_shared * s.f_shared;
  const size_t cols = P == kGateUp ? 2 * F : P == kDHid ? F : (size_t)s.d;
  return p.splits > 1 ? (size_t)p.splits * s.T * cols : 0;
}

template <int P>
hipError_t launch_product(const k3moe_shape& s, DenseArgs g, float* part, hipStream_t st) {
  const Plan p = plan_product(P, s);
  const int cus = grouped_grid();
  if (p.splits > 1) {
    if constexpr (P != kDW13 && P != kDW2) {
      g.part = part;
      g.splits = p.splits;
      g.k_split = p.k_split;
      if (p.tile == kTile64) {
        dense_tile<P, 64, 64, 2, 2, 3, true><<<cus * 3, 256, 0, st>>>(g);
      } else if constexpr (P != kDX) {
        if (p.tile == kTile128) dense_tile<P, 128, 128, 2, 4, 3, true><<<cus, 512, 0, st>>>(g);
        else dense_tile<P, 128, 256, 2, 4, 3, true><<<cus, 512, 0, st>>>(g);
      }
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      const int64_t n = s.T * (P == kGateUp || P == kDHid ? (int64_t)g.S * g.fs : g.d) / 4;
      split_finish<P><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(g);
    }
  } else if (p.tile == kTile256) {
    dense_tile<P, 256, 256, 2, 4, 2><<<cus, 512, 0, st>>>(g);
  } else if (p.tile == kTile64) {
    dense_tile<P, 64, 64, 2, 2, 3><<<cus * 3, 256, 0, st>>>(g);
  } else if constexpr (P != kDX) {   // (dx on these tiles shares the weight gradients' launch)
    if (p.tile == kTile128x256) dense_tile<P, 128, 256, 2, 4, 3><<<cus, 512, 0, st>>>(g);
    else dense_tile<P, 128, 128, 2, 4, 3><<<cus, 512, 0, st>>>(g);
  }
  return hipGetLastError();
}

// The three gradients in one launch (g.o0 NULL: not wanted).  A workgroup takes as
// many of the short tiles as 48 stages make (16 on the smallest tiles, three to a
// CU), so that its start weighs little.
template <int XM, int XN, int XRING, int BM, int BN, int RING, int WM, int WN>
hipError_t launch_grads_tile(const k3moe_shape& s, const DenseArgs (&g)[3], hipStream_t st) {
  GradArgs a;
  const int64_t F = (int64_t)s.n_shared * s.f_shared, T = s.T, d = s.d;
  const int64_t M[3] = {T, 2 * F, d}, N[3] = {d, d, F}, K[3] = {2 * F, T, T};
  int64_t total = 0;
  for (int p = 0; p < 3; ++p) {
    a.g[p] = g[p];
    const int64_t rows = p == 2 ? g[p].m_hi : M[p];
    const int bm = p == 0 ? XM : BM, bn = p == 0 ? XN : BN;
    const int64_t items = (rows + bm - 1) / bm * ((N[p] + bn - 1) / bn);
    const int64_t rounds = (items + kCUs - 1) / kCUs, nst = (K[p] + kBK - 1) / kBK;
    const int64_t least = std::max<int64_t>((BM == 64 ? 16 : 48) / nst, 1);
    a.n[p] = (int)std::min(rounds, p == 0 ? rounds : p == 1 ? std::max(least, (rounds + 1) / 2) : least);
    a.wgs[p] = g[p].o0 ? (int)((rounds + a.n[p] - 1) / a.n[p] * kCUs) : 0;
    total += a.wgs[p];
  }
  if (total == 0) return hipSuccess;
  dense_grads<XM, XN, XRING, BM, BN, RING, WM, WN><<<(unsigned)total, 64 * WM * WN, 0, st>>>(a);
  return hipGetLastError();
}

DenseArgs dense_args(const k3moe_shape& s) {
  DenseArgs g{};
  g.T = (int)s.T;
  g.d = s.d;
  g.fs = s.f_shared;
  g.S = s.n_shared;
  g.parts = s.T <= kRows;
  g.m_hi = s.d;
  return g;
}

}  // namespace

int64_t shared_train_rows(const k3moe_shape& s) { return s.T <= kRows ? 2 * kRows : s.T; }

size_t shared_train_part_floats(const k3moe_shape& s, bool backward) {
  return backward ? std::max(part_floats(kDHid, s), part_floats(kDX, s))
                  : std::max(part_floats(kGateUp, s), part_floats(kDown, s));
}

hipError_t launch_shared_train(const k3moe_shape& s, const k3moe_expert_bank& b, const void* x,
                               void* gu, void* y, const SharedTrainWs& ws, hipStream_t st) {
  DenseArgs g = dense_args(s);
  g.a = static_cast<const uint16_t*>(x);
  g.b = static_cast<const uint16_t*>(b.w13);
  g.o0 = gu;
  g.o1 = ws.h;
  hipError_t e = launch_product<kGateUp>(s, g, ws.part, st);
  if (e != hipSuccess) return e;
  g = dense_args(s);
  g.a = ws.h;
  g.b = static_cast<const uint16_t*>(b.w2);
  g.o0 = y;
  g.out_f32 = s.out_dtype == K3MOE_F32;
  return launch_product<kDown>(s, g, ws.part, st);
}

hipError_t launch_shared_backward(const k3moe_shape& s, const k3moe_expert_bank& b, const void* x,
                                  const void* gu, const void* dy, void* dx, void* dw13, void* dw2,
                                  const SharedTrainWs& ws, hipStream_t st) {
  if (!dx && !dw13 && !dw2) return hipSuccess;
  const DenseArgs z = dense_args(s);
  DenseArgs g = z;
  g.a = static_cast<const uint16_t*>(dy);
  g.b = static_cast<const uint16_t*>(b.w2);
  g.gu = static_cast<const uint16_t*>(gu);
  g.o0 = ws.dgu;
  g.o1 = ws.h;
  hipError_t e = launch_product<kDHid>(s, g, ws.part, st);
  if (e != hipSuccess) return e;
  DenseArgs grads[3] = {z, z, z};
  grads[0].a = ws.dgu;
  grads[0].b = static_cast<const uint16_t*>(b.w13);
  grads[0].o0 = dx;
  grads[1].a = ws.dgu;
  grads[1].b = static_cast<const uint16_t*>(x);
  grads[1].o0 = dw13;
  grads[2].a = static_cast<const uint16_t*>(dy);
  grads[2].b = ws.h;
  grads[2].o0 = dw2;
  // One launch for the three: backward 244 us at T = 517 (275 in three launches), 1150
  // at 4096 (1175).  From four rounds of dx on a partly filled last round weighs
  // less than what a workgroup saves by going from tile to tile: 4.31 ms in launches
  // of their own at T = 16384 (4.50 in one); and without dx there is nothing to fill
  // the gaps with (T = 517 174 us against 179).
  // On 64 x 64 tiles one launch is worth it for smaller layers (tokens x d x fs x
  // experts: 4 x 256 x 128 16 us against 22; 128 x 4096 x 512 x 3, 4700 tiles: 42, 56;
  // 64 x 4096 x 1024 x 3, 9300 tiles: 55, 62; without dx, 16 x 4096 x 512 x 3: 33, 33);
  // where the weight gradients alone fill the chip they are faster on their own tiles,
  // beside a dx whose contraction is split (64 x 7168 x 2048 x 2, 21600 tiles: 127 us
  // against 140).
  const int tile = plan_product(kDX, s).tile;
  const int64_t dx_tiles = ((s.T + 255) / 256) * ((s.d + 255) / 256);
  const int64_t t64 = (s.T + 63) / 64, d64 = (s.d + 63) / 64,
                f64 = ((int64_t)s.n_shared * s.f_shared + 31) / 32;   // of 2 F
  const int64_t tiles64 = t64 * d64 + f64 * d64 + (f64 + 1) / 2 * d64;
  if (dx && tile == kTile256 && dx_tiles < 4 * kCUs)
    return launch_grads_tile<256, 256, 2, 256, 256, 2, 2, 4>(s, grads, st);
  if (dx && (tile == kTile128 || tile == kTile128x256)) {
    // (the weight gradients on 256 x 256 tiles, where there are some: T = 517 244 us
    // against 252 on dx's 128 x 256, 1000 357, 389; 2000 x 2048 x 1024, 96 tiles of
    // theirs, 70, 82; 1061 x 3616 x 128, 22 tiles, 43, 35)
    const int64_t d256 = (s.d + 255) / 256, f256 = ((int64_t)s.n_shared * s.f_shared + 127) / 128;
    if (d256 * f256 * 3 / 2 >= 64) return launch_grads_tile<128, 256, 3, 256, 256, 2, 2, 4>(s, grads, st);
    return launch_grads_tile<128, 256, 3, 128, 256, 3, 2, 4>(s, grads, st);
  }
  if (tile == kTile64 && tiles64 <= (dx ? 10240 : 4096))
    return launch_grads_tile<64, 64, 3, 64, 64, 3, 2, 2>(s, grads, st);
  if (dx && (e = launch_product<kDX>(s, grads[0], ws.part, st)) != hipSuccess) return e;
  if (const int64_t rows = dw13 && dw2 ? tail_rows(s) : -1; rows >= 0) {
    grads[0].o0 = nullptr;
    grads[2].m_hi = s.d - (int)rows;
    if ((e = launch_grads_tile<256, 256, 2, 256, 256, 2, 2, 4>(s, grads, st)) != hipSuccess || rows == 0) return e;
    grads[2].m_lo = grads[2].m_hi;
    grads[2].m_hi = s.d;
    dense_tile<kDW2, 128, 128, 2, 4, 3><<<grouped_grid(), 512, 0, st>>>(grads[2]);
    return hipGetLastError();
  }
  if (dw13 && (e = launch_product<kDW13>(s, grads[1], ws.part, st)) != hipSuccess) return e;
  return dw2 ? launch_product<kDW2>(s, grads[2], ws.part, st) : hipSuccess;
}

// The weight gradients of an empty batch.  (A fill kernel rather than a memset,
// so that a captured call holds kernels only.)
hipError_t launch_zero(void* p, size_t bytes, hipStream_t st) {
  if (!p || !bytes) return hipSuccess;
  zero_fill<<<(unsigned)std::min<size_t>((bytes / 16 + 255) / 256, 4096), 256, 0, st>>>(
      static_cast<uint4*>(p), bytes / 16);
  return hipGetLastError();
}

}  // namespace k3
