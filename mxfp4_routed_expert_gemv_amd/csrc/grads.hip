// The global norm of a step's gradients and their clipping:
//   norm = sqrt(sum over all tensors of g^2),  out = g min(1, max_norm / norm).
// Reading the gradients bounds the norm (294 M bf16 elements: 104 us again and again,
// 5.6 TB/s, 118 in a pass by itself; no faster with four loads a thread in flight),
// the clipping that and its writes (into fp32: 400 us more, 4.4 TB/s; four loads a
// thread in flight 425, stores past the caches 500); for a list of small tensors the
// host, which builds the list.  The squares are summed in fp64, so no range or
// length of the tensors loses anything, and in a fixed order: every workgroup's
// partial sum has its own slot, one workgroup adds them up.  The list of tensors
// travels in the kernel arguments, kPerLaunch at a time, so a call needs no copy
// to the device and can be captured.
#include "internal.h"
#include "kern_common.h"

namespace k3 {
namespace {

constexpr int kPerLaunch = 120;     // tensors in one launch's arguments (below 4 KB)
constexpr int kUnit = 16384;        // elements per work item
constexpr int kMaxGrid = 2048;      // workgroups of a launch: partial sums per launch
constexpr int kVec = 8;             // elements per load
constexpr int64_t kMaxUnits = int64_t(1) << 30;   // work items of a launch

struct Entry {
  const void* in;
  void* out;
  int64_t n;
  int32_t unit0;     // the tensor's first work item in this launch
  int16_t in_f32, out_f32;
};
struct Table {
  Entry e[kPerLaunch];
  int count, units;
};
static_assert(sizeof(Table) <= 4000, "kernel arguments");

// Gradients may start at any element: loads and stores of 8 elements are only
// element-aligned.
struct __attribute__((packed, aligned(2))) Bf16x8 { uint32_t v[4]; };
struct __attribute__((packed, aligned(4))) F32x8 { float v[8]; };

__device__ __forceinline__ void load8(const Entry& e, int64_t i, float (&v)[kVec]) {
  if (e.in_f32) {
    const F32x8 w = *reinterpret_cast<const F32x8*>(static_cast<const float*>(e.in) + i);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = w.v[j];
  } else {
    const Bf16x8 w = *reinterpret_cast<const Bf16x8*>(static_cast<const uint16_t*>(e.in) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(w.v[j]);
      v[2 * j + 1] = bf16_hi(w.v[j]);
    }
  }
}
__device__ __forceinline__ float load1(const Entry& e, int64_t i) {
  return e.in_f32 ? static_cast<const float*>(e.in)[i]
                  : __uint_as_float((uint32_t)static_cast<const uint16_t*>(e.in)[i] << 16);
}

// Work item u of a launch: its tensor (the last whose first item is <= u).
__device__ __forceinline__ int tensor_of(const Table& t, int u) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].unit0 <= u) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(256) void sum_squares(Table t, double* __restrict__ partial) {
  __shared__ double s_wave[4];
  double sum = 0.0;
  for (int u = blockIdx.x; u < t.units; u += gridDim.x) {
    const Entry& e = t.e[tensor_of(t, u)];
    const int64_t a = (int64_t)(u - e.unit0) * kUnit, b = a + kUnit < e.n ? a + kUnit : e.n;
    for (int64_t i = a + threadIdx.x * kVec; i < b; i += 256 * kVec) {
      if (i + kVec <= b) {
        float v[kVec];
        load8(e, i, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum = __builtin_fma((double)v[j], (double)v[j], sum);
      } else {
        for (int64_t q = i; q < b; ++q) {
          const double v = load1(e, q);
          sum = __builtin_fma(v, v, sum);
        }
      }
    }
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) partial[blockIdx.x] = (s_wave[0] + s_wave[1]) + (s_wave[2] + s_wave[3]);
}

// The norm from n partial sums, in one order whatever workgroup does it.
__device__ __forceinline__ double norm_of(const double* __restrict__ partial, int n) {
  __shared__ double s_wave[4];
  double sum = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += 256) sum += partial[i];
  sum = wave_sum(sum);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = sum;
  __syncthreads();
  return sqrt((s_wave[0] + s_wave[1]) + (s_wave[2] + s_wave[3]));
}

// *norm, and the fp64 norm for scale_all.
__global__ __launch_bounds__(256) void finish_norm(const double* __restrict__ partial, int n,
                                                   float* norm, double* total) {
  const double v = norm_of(partial, n);
  if (threadIdx.x == 0) {
    *norm = (float)v;
    if (total) *total = v;
  }
}

// Scales the tensors; n > 0: every workgroup takes the norm from the n partial
// sums itself (the first one writes it), which a launch of its own would take
// longer for; n = 0: the norm is at partial[0].  The last items come first: the
// norm's pass read them last, so a part of them is still in the last-level cache.
__global__ __launch_bounds__(256) void scale_all(Table t, const double* __restrict__ partial, int n,
                                                 float max_norm, float* norm) {
  const double v = n > 0 ? norm_of(partial, n) : partial[0];
  if (n > 0 && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  // (a norm of infinities or NaN leaves the gradients as they are)
  const bool scaled = v < (double)INFINITY && v > (double)max_norm;
  const double factor = scaled ? (double)max_norm / v : 1.0;
  // Below fp32's normal range (a norm past max_norm 2^126) the factor has fewer bits in
  // fp32 than its products with such gradients can hold: they are taken in fp64 there,
  // and rounded once.
  const bool tiny = factor < 0x1p-126;
  const float f = (float)factor;
  auto times = [&](float g) { return tiny ? (float)((double)g * factor) : g * f; };
  for (int w = blockIdx.x; w < t.units; w += gridDim.x) {
    const int u = t.units - 1 - w;
    const Entry& e = t.e[tensor_of(t, u)];
    if (!scaled && e.in == e.out) continue;   // in place and not clipped: nothing to do
    const int64_t a = (int64_t)(u - e.unit0) * kUnit, b = a + kUnit < e.n ? a + kUnit : e.n;
    for (int64_t i = a + threadIdx.x * kVec; i < b; i += 256 * kVec) {
      if (i + kVec <= b) {
        float v[kVec];
        load8(e, i, v);
        if (scaled)
#pragma unroll
          for (int j = 0; j < kVec; ++j) v[j] = times(v[j]);
        if (e.out_f32) {
          F32x8 w;
#pragma unroll
          for (int j = 0; j < kVec; ++j) w.v[j] = v[j];
          *reinterpret_cast<F32x8*>(static_cast<float*>(e.out) + i) = w;
        } else {
          Bf16x8 w;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w.v[j] = (uint32_t)f32_to_bf16(v[2 * j]) | ((uint32_t)f32_to_bf16(v[2 * j + 1]) << 16);
          *reinterpret_cast<Bf16x8*>(static_cast<uint16_t*>(e.out) + i) = w;
        }
      } else {
        for (int64_t q = i; q < b; ++q) {
          const float v = scaled ? times(load1(e, q)) : load1(e, q);
          if (e.out_f32) static_cast<float*>(e.out)[q] = v;
          else static_cast<uint16_t*>(e.out)[q] = f32_to_bf16(v);
        }
      }
    }
  }
}

struct Batch {
  Table t;
  int next;   // first tensor of the next launch
};

// The next launch's table: tensors from i on, at most kPerLaunch, empty ones
// left out.
void fill_table(const k3moe_tensor* ts, int n, int i, Batch& b) {
  b.t.count = 0;
  int64_t units = 0;
  for (; i < n && b.t.count < kPerLaunch; ++i) {
    const k3moe_tensor& s = ts[i];
    if (s.numel == 0) continue;
    const int64_t u = (s.numel + kUnit - 1) / kUnit;
    if (units + u > kMaxUnits) break;
    Entry& e = b.t.e[b.t.count++];
    e.in = s.data;
    e.out = s.out;
    e.n = s.numel;
    e.unit0 = (int32_t)units;
    e.in_f32 = s.dtype == K3MOE_F32;
    e.out_f32 = s.out_dtype == K3MOE_F32;
    units += u;
  }
  b.t.units = (int)units;
  b.next = i;
}

}  // namespace

// One launch takes kPerLaunch non-empty tensors, or fewer where their work
// items would pass 2^30 (tensors are at most 2^40 elements: 2^26 items each).
size_t grad_partials(int n) { return ((size_t)n / 16 + 2) * kMaxGrid; }

hipError_t launch_grads(const k3moe_tensor* ts, int n, bool clip, float max_norm, float* norm,
                        const GradWs& ws, hipStream_t st) {
  Batch b;
  int slots = 0;
  for (int i = 0; i < n; i = b.next) {
    fill_table(ts, n, i, b);
    if (b.t.units == 0) continue;
    const int grid = b.t.units < kMaxGrid ? b.t.units : kMaxGrid;
    sum_squares<<<grid, 256, 0, st>>>(b.t, ws.partial + slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    slots += grid;
  }
  const bool fused = clip && slots > 0 && slots <= kMaxGrid;
  if (!fused) {
    finish_norm<<<1, 256, 0, st>>>(ws.partial, slots, norm, ws.total);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !clip) return e;
  }
  for (int i = 0; i < n; i = b.next) {
    fill_table(ts, n, i, b);
    if (b.t.units == 0) continue;
    scale_all<<<b.t.units < kMaxGrid ? b.t.units : kMaxGrid, 256, 0, st>>>(
        b.t, fused ? ws.partial : ws.total, fused ? slots : 0, max_norm, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace k3
