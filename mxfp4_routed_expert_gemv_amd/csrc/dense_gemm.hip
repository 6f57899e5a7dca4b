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
// once, from fp32: they are operands of the next bf16 product.
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
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kBK = 64;   // contraction elements per stage

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
};

// A voffset past num_records: the copy writes zeros to LDS.  Every offset of
// an element inside a tile stays below 2^31 (at most two experts' matrices).
constexpr uint32_t kRecords = 0x80000000u;
constexpr uint32_t kOut = 0xFFFFFFF0u;

__device__ __forceinline__ u32x4_t rsrc_of(const uint16_t* p) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  u32x4_t r;
  r.x = __builtin_amdgcn_readfirstlane((uint32_t)a);
  r.y = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xFFFFu);
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

// Four bf16 roundings packed.
__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
  uint2 p;
  p.x = (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
  p.y = (uint32_t)f32_to_bf16(c) | ((uint32_t)f32_to_bf16(d) << 16);
  return p;
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
  static_assert(P != kGateUp || NF % 2 == 0, "gate and up fragments come in pairs");
};

// Column (row of w13) of hidden feature n's gate in [2 F]; its up is fs further.
__device__ __forceinline__ int gate_col(int n, int fs) { return n + n / fs * fs; }

constexpr int kGM = 8;   // m-tiles per group of the item order

template <int P, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void dense_tile(DenseArgs g) {
  using C = Tile<P, BM, BN, WM, WN>;
  using OA = typename C::A;
  using OB = typename C::B;
  constexpr int MF = C::MF, NF = C::NF;
  __shared__ __attribute__((aligned(16))) uint8_t sA[2 * OA::kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t sB[2 * OB::kSlot];

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const int T = g.T, d = g.d, fs = g.fs, F = g.S * g.fs;
  const int M = P == kDW13 ? 2 * F : P == kDW2 ? d : T;
  const int N = P == kGateUp || P == kDHid || P == kDW2 ? F : d;
  const int K = P == kGateUp || P == kDHid ? d : P == kDown ? F : P == kDX ? 2 * F : T;
  const int nst = (K + kBK - 1) / kBK;
  const int n_mt = (M + BM - 1) / BM, n_nt = (N + C::kN - 1) / C::kN;
  const ItemRange ir = item_range((long)n_mt * n_nt);

  // Items: groups of kGM m-tiles, the m-tile fastest, then the n-tile, so the
  // workgroups of an XCD share both operands through its L2.
  auto item_tile = [&](long it, int& m0, int& n0) {
    const long per = (long)kGM * n_nt;
    const int grp = (int)(it / per), first = grp * kGM;
    const int r = (int)(it - grp * per), gsz = min(n_mt - first, kGM);
    const int nt = r / gsz;
    n0 = nt * C::kN;
    m0 = (first + r - nt * gsz) * BM;
  };

  // ---- copies: this wave's units of both operands, as byte offsets from the
  // tile's first element (kOut: outside the matrix), and the tile's base.
  uint32_t va[C::NA], vb[C::NB];
  int ka[C::NA], kb[C::NB];   // contraction element of each unit within the stage
  const uint16_t *pa, *pb;
  size_t sa, sb;              // elements a stage advances
  long c_it = ir.first;
  int c_st = 0;
  auto setup = [&]() {
    int m0, n0;
    item_tile(c_it, m0, n0);
    const size_t lda = P == kGateUp || P == kDHid || P == kDW2 ? d : P == kDown ? F : 2 * F;
    pa = g.a + (C::A_KC ? (size_t)m0 * lda : (size_t)m0);
    sa = C::A_KC ? (size_t)kBK : kBK * lda;
#pragma unroll
    for (int c = 0; c < C::NA; ++c) {
      int r, k;
      OA::unit((wv * C::NA + c) * 64 + lane, r, k);
      ka[c] = k;
      const size_t e = C::A_KC ? (size_t)r * lda + k : (size_t)k * lda + r;
      va[c] = m0 + r < M ? (uint32_t)(e * 2) : kOut;
    }
    const int gc0 = gate_col(n0, fs);
    const size_t ldb = P == kGateUp || P == kDX || P == kDW13 ? d : P == kDW2 ? F : fs;
    pb = g.b + (P == kGateUp ? (size_t)gc0 * d
                : P == kDHid ? (size_t)(n0 / fs) * d * fs + n0 % fs
                : C::B_KC    ? (size_t)n0 * ldb
                             : (size_t)n0);
    sb = C::B_KC ? (size_t)kBK : kBK * ldb;
#pragma unroll
    for (int c = 0; c < C::NB; ++c) {
      int r, k;
      OB::unit((wv * C::NB + c) * 64 + lane, r, k);
      kb[c] = k;
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
        // (kDown: the stage's expert and position are added in issue)
        const size_t e = C::B_KC ? (size_t)r * ldb + (P == kDown ? 0 : k) : (size_t)k * ldb + r;
        vb[c] = n0 + r < N ? (uint32_t)(e * 2) : kOut;
      }
    }
  };
  auto issue = [&](int slot) {
    if (c_it >= ir.end) return;
    const int k0 = c_st * kBK;
    const bool tail = k0 + kBK > K;
    const u32x4_t ra = rsrc_of(pa + (size_t)c_st * sa);
    const uint32_t la = lds_addr(sA) + (uint32_t)(slot * OA::kSlot + wv * (C::NA * 1024));
#pragma unroll
    for (int c = 0; c < C::NA; ++c)
      dma16_buf(ra, tail && k0 + ka[c] >= K ? kOut : va[c], la + c * 1024);
    const uint32_t lb = lds_addr(sB) + (uint32_t)(slot * OB::kSlot + wv * (C::NB * 1024));
    if (P == kDown) {
      // feature k0 + k is element (k0 + k) % fs of a row of expert (k0 + k) / fs
      const int e0 = k0 / fs;
      const u32x4_t rb = rsrc_of(pb + (size_t)e0 * d * fs);
#pragma unroll
      for (int c = 0; c < C::NB; ++c) {
        const int k = k0 - e0 * fs + kb[c], e = k / fs;
        const uint32_t o = (uint32_t)(((size_t)e * d * fs + (k - e * fs)) * 2);
        dma16_buf(rb, vb[c] == kOut || k0 + kb[c] >= K ? kOut : vb[c] + o, lb + c * 1024);
      }
    } else {
      const u32x4_t rb = rsrc_of(pb + (size_t)c_st * sb);
#pragma unroll
      for (int c = 0; c < C::NB; ++c)
        dma16_buf(rb, tail && k0 + kb[c] >= K ? kOut : vb[c], lb + c * 1024);
    }
    if (++c_st == nst) {
      c_st = 0;
      c_it += ir.step;
      if (c_it < ir.end) setup();
    }
  };

  const int wm = wv / WN, wn = wv - wm * WN;
  if (c_it < ir.end) setup();
  issue(0);
  int slot = 0;
  for (long it = ir.first; it < ir.end; it += ir.step) {
    int m0, n0;
    item_tile(it, m0, n0);
    f32x4_t acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[i][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s = 0; s < nst; ++s, slot ^= 1) {
      // this wave's copies of the stage have landed and its reads of the other
      // slot are done; past the barrier both hold for every wave
      wait_vmem<0>();
      wait_lds();
      wg_barrier();
      issue(slot ^ 1);
      const uint8_t* ba = sA + slot * OA::kSlot;
      const uint8_t* bb = sB + slot * OB::kSlot;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        bf16x8_t b[NF], a[2];
#pragma unroll
        for (int f = 0; f < NF; ++f) b[f] = OB::frag(bb, wn * NF + f, j, ln, lg);
        a[0] = OA::frag(ba, wm * MF, j, ln, lg);
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          if (i + 1 < MF) a[(i + 1) & 1] = OA::frag(ba, wm * MF + i + 1, j, ln, lg);
#pragma unroll
          for (int f = 0; f < NF; ++f)   // sums transposed: a lane holds 4 consecutive n of one m
            acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[f], a[i & 1], acc[i][f], 0, 0, 0);
        }
      }
    }
    // ---- epilogue: lane (ln, lg) holds m = m0 + 16 (wm MF + i) + ln, four n
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = m0 + (wm * MF + i) * 16 + ln;
      if (m >= M) continue;
      if constexpr (P == kGateUp) {
#pragma unroll
        for (int f = 0; f < NF / 2; ++f) {
          const int n = n0 + wn * (8 * NF) + f * 16 + lg * 4;
          if (n >= N) continue;
          const f32x4_t ga = acc[i][f], up = acc[i][f + NF / 2];
          uint16_t* gu = static_cast<uint16_t*>(g.o0) + (size_t)m * 2 * F + gate_col(n, fs);
          *reinterpret_cast<uint2*>(gu) = pack4(ga[0], ga[1], ga[2], ga[3]);
          *reinterpret_cast<uint2*>(gu + fs) = pack4(up[0], up[1], up[2], up[3]);
          *reinterpret_cast<uint2*>(g.o1 + (size_t)m * F + n) =
              pack4(silu_mul(ga[0], up[0]), silu_mul(ga[1], up[1]), silu_mul(ga[2], up[2]),
                    silu_mul(ga[3], up[3]));
        }
      } else {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const int n = n0 + (wn * NF + f) * 16 + lg * 4;
          if (n >= N) continue;
          const f32x4_t v = acc[i][f];
          if constexpr (P == kDHid) {
            const size_t o = (size_t)m * 2 * F + gate_col(n, fs);
            const uint2 gw = *reinterpret_cast<const uint2*>(g.gu + o);
            const uint2 uw = *reinterpret_cast<const uint2*>(g.gu + o + fs);
            const float ga[4] = {bf16_lo(gw.x), bf16_hi(gw.x), bf16_lo(gw.y), bf16_hi(gw.y)};
            const float up[4] = {bf16_lo(uw.x), bf16_hi(uw.x), bf16_lo(uw.y), bf16_hi(uw.y)};
            float dg[4], du[4], h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float s = 1.0f / (1.0f + expf(-ga[r]));
              // g s: for g < -88 e^-g is +inf and s is 0, the product -0, never NaN
              const float gs = ga[r] * s;
              h[r] = gs * up[r];
              du[r] = v[r] * gs;
              dg[r] = v[r] * up[r] * (s + gs * (1.0f - s));
            }
            uint16_t* o0 = static_cast<uint16_t*>(g.o0) + o;
            *reinterpret_cast<uint2*>(o0) = pack4(dg[0], dg[1], dg[2], dg[3]);
            *reinterpret_cast<uint2*>(o0 + fs) = pack4(du[0], du[1], du[2], du[3]);
            *reinterpret_cast<uint2*>(g.o1 + (size_t)m * F + n) = pack4(h[0], h[1], h[2], h[3]);
          } else if (P == kDown && g.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(g.o0) + (size_t)m * N + n) =
                make_float4(v[0], v[1], v[2], v[3]);
          } else {
            // dW2 [S][d][fs]: column n is feature n % fs of expert n / fs
            const size_t o = P == kDW2 ? ((size_t)(n / fs) * d + m) * fs + n % fs : (size_t)m * N + n;
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.o0) + o) = pack4(v[0], v[1], v[2], v[3]);
          }
        }
      }
    }
  }
}

__global__ __launch_bounds__(256) void zero_fill(uint4* p, size_t n16) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += (size_t)gridDim.x * 256)
    p[i] = make_uint4(0, 0, 0, 0);
}

template <int P>
hipError_t launch_product(const DenseArgs& g, hipStream_t st) {
  dense_tile<P, 128, 128, 2, 2><<<grouped_grid() * 2, 256, 0, st>>>(g);
  return hipGetLastError();
}

DenseArgs dense_args(const k3moe_shape& s) {
  DenseArgs g{};
  g.T = (int)s.T;
  g.d = s.d;
  g.fs = s.f_shared;
  g.S = s.n_shared;
  return g;
}

}  // namespace

hipError_t launch_shared_train(const k3moe_shape& s, const k3moe_expert_bank& b, const void* x,
                               void* gu, void* y, const SharedTrainWs& ws, hipStream_t st) {
  DenseArgs g = dense_args(s);
  g.a = static_cast<const uint16_t*>(x);
  g.b = static_cast<const uint16_t*>(b.w13);
  g.o0 = gu;
  g.o1 = ws.h;
  hipError_t e = launch_product<kGateUp>(g, st);
  if (e != hipSuccess) return e;
  g = dense_args(s);
  g.a = ws.h;
  g.b = static_cast<const uint16_t*>(b.w2);
  g.o0 = y;
  g.out_f32 = s.out_dtype == K3MOE_F32;
  return launch_product<kDown>(g, st);
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
  hipError_t e = launch_product<kDHid>(g, st);
  if (e != hipSuccess) return e;
  if (dx) {
    g = z;
    g.a = ws.dgu;
    g.b = static_cast<const uint16_t*>(b.w13);
    g.o0 = dx;
    e = launch_product<kDX>(g, st);
    if (e != hipSuccess) return e;
  }
  if (dw13) {
    g = z;
    g.a = ws.dgu;
    g.b = static_cast<const uint16_t*>(x);
    g.o0 = dw13;
    e = launch_product<kDW13>(g, st);
    if (e != hipSuccess) return e;
  }
  if (dw2) {
    g = z;
    g.a = static_cast<const uint16_t*>(dy);
    g.b = ws.h;
    g.o0 = dw2;
    e = launch_product<kDW2>(g, st);
  }
  return e;
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
