// Parts of the tiled 16-bit matrix products with both operands in LDS rings: the
// copies, the operand tiles' LDS layout and fragment reads, the lane exchange of
// the epilogues.  Used by the shared experts' training pass (bf16) and by the
// orthogonalised update (fp16): but for pack_f16, nothing here depends on the 16 bits'
// meaning.
#pragma once

#include "grouped.h"
#include "kern_common.h"

namespace k3 {
namespace dense {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kBK = 64;   // contraction elements per stage

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

// Swaps the odd 16-lane groups of a with the even ones of b.
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const auto t = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = t[0];
  b = t[1];
}

// 4 x 4 values of 16 bits, a row of them to each of four neighbouring lanes,
// transposed: lane j of the four gets the j-th value of every lane.
__device__ __forceinline__ uint2 transpose4(uint2 v, int lane) {
  const bool odd = lane & 1, upper = lane & 2;
  const uint32_t px = __builtin_amdgcn_mov_dpp((int)v.x, 0xB1, 0xF, 0xF, true);   // lane ^ 1
  const uint32_t py = __builtin_amdgcn_mov_dpp((int)v.y, 0xB1, 0xF, 0xF, true);
  const uint32_t x = odd ? (px >> 16) | (v.x & 0xFFFF0000u) : (v.x & 0xFFFFu) | (px << 16);
  const uint32_t y = odd ? (py >> 16) | (v.y & 0xFFFF0000u) : (v.y & 0xFFFFu) | (py << 16);
  const uint32_t qx = __builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true);     // lane ^ 2
  const uint32_t qy = __builtin_amdgcn_mov_dpp((int)y, 0x4E, 0xF, 0xF, true);
  return upper ? make_uint2(qy, y) : make_uint2(x, qx);
}

// Two values as fp16, to nearest even.  (The bits are opaque from here on: where the
// compiler sees a product in `a`, it may round it to fp16 in one step for one use of the
// result and through fp32 for another, and a second part taken from the one would not
// fit the other.)
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t w = __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b});
  asm volatile("" : "+v"(w));
  return w;
}

}  // namespace dense
}  // namespace k3
