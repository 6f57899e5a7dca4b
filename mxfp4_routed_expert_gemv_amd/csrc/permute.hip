// Token -> expert counting sort, stable in pair order (pair p = t*k + slot).
//
// Every result is integer and exact.  A token's rank among the tokens routed
// to expert e is the popcount of the lower token bits of e's token mask, so
// every pair's sorted position is fixed without any ordering between threads.
// Slot s of a token takes part only when its id is in [0, E) and no earlier
// slot of the token holds the same id; a token then routes to each expert at
// most once, and "stable in pair order" is "tokens ascending within an
// expert".
//
// Small batches (T <= 256, T*k <= 4096): one workgroup does everything in LDS.
// Larger batches, three launches over chunks of CH tokens, a thread to a pair:
//   chunk_hist    per-chunk, per-expert pair counts (LDS atomics);
//   chunk_scan    per expert, exclusive scan over chunks (64 experts and 16 groups
//                 of chunks to a workgroup), and the counts;
//   chunk_scatter per chunk, the experts' offsets from the counts, positions =
//                 offset + pairs of the expert in earlier chunks + rank from the masks.
// All latency: 16 us at T = 4096, top 16 of 896 (54 with a thread to a token, chunks
// of 256 and one workgroup for the scan).
#include "internal.h"
#include "kern_common.h"

namespace k3 {
namespace {

constexpr int kSmallT = 256, kSmallPairs = 4096;

__device__ __forceinline__ bool valid_slot(const int32_t* row, int s, int E) {
  const int e = row[s];
  if (e < 0 || e >= E) return false;
  for (int q = 0; q < s; ++q)
    if (row[q] == e) return false;
  return true;
}

// Block-wide exclusive scan of one int per thread (blockDim.x == 1024).
__device__ __forceinline__ int block_excl_scan_1024(int v, int* sums, int* total) {
  const int tid = threadIdx.x;
  sums[tid] = v;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int add = tid >= o ? sums[tid - o] : 0;
    __syncthreads();
    sums[tid] += add;
    __syncthreads();
  }
  const int incl = sums[tid];
  *total = sums[1023];
  __syncthreads();
  return incl - v;
}

__device__ __forceinline__ void small_sort(const int32_t* __restrict__ idx, int32_t* __restrict__ counts,
                                           int32_t* __restrict__ offsets,
                                           int32_t* __restrict__ sorted_pair,
                                           int32_t* __restrict__ pair_pos, int32_t* __restrict__ diag,
                                           int T, int E, int k) {
  __shared__ int ids[kSmallPairs];
  __shared__ unsigned char valid[kSmallPairs];
  __shared__ int cnt[1024];
  __shared__ int sums[1024];
  __shared__ unsigned long long mask[1024][kSmallT / 64];
  const int tid = threadIdx.x;
  const int P = T * k;
  for (int p = tid; p < P; p += 1024) ids[p] = idx[p];
  cnt[tid] = 0;
  for (int i = tid; i < E * (kSmallT / 64); i += 1024) (&mask[0][0])[i] = 0ull;
  __syncthreads();
  int bad = 0;
  for (int p = tid; p < P; p += 1024) {
    const int t = p / k, s = p - t * k;
    const bool ok = valid_slot(ids + t * k, s, E);
    valid[p] = ok;
    if (ok) {
      atomicAdd(&cnt[ids[p]], 1);
      atomicOr(&mask[ids[p]][t >> 6], 1ull << (t & 63));
    } else {
      ++bad;
    }
  }
  if (bad && diag) atomicAdd(&diag[K3MOE_DIAG_BAD_EXPERT_IDS], bad);
  __syncthreads();
  const int c = tid < E ? cnt[tid] : 0;
  int total;
  const int excl = block_excl_scan_1024(c, sums, &total);
  if (tid < E) {
    counts[tid] = c;
    offsets[tid] = excl;
    cnt[tid] = excl;  // cnt now holds each expert's first position
  }
  if (tid == 0) offsets[E] = total;
  __syncthreads();
  for (int p = tid; p < P; p += 1024) {
    if (valid[p]) {
      const int e = ids[p], t = p / k, w = t >> 6;
      int rank = __popcll(mask[e][w] & ((1ull << (t & 63)) - 1ull));
      for (int q = 0; q < w; ++q) rank += __popcll(mask[e][q]);
      const int pos = cnt[e] + rank;
      sorted_pair[pos] = p;
      pair_pos[p] = pos;
    } else {
      pair_pos[p] = -1;
    }
  }
  for (int q = total + tid; q < P; q += 1024) sorted_pair[q] = -1;
}

__global__ __launch_bounds__(1024) void permute_small(const int32_t* __restrict__ idx,
                                                      int32_t* __restrict__ counts,
                                                      int32_t* __restrict__ offsets,
                                                      int32_t* __restrict__ sorted_pair,
                                                      int32_t* __restrict__ pair_pos,
                                                      int32_t* __restrict__ diag, int T, int E,
                                                      int k) {
  small_sort(idx, counts, offsets, sorted_pair, pair_pos, diag, T, E, k);
}

// The same, and the tokens' rows moved, in one launch: workgroup 0 sorts, workgroup
// t + 1 moves token t's row (its 16-byte words) and finds the places of its pairs by
// itself, as the valid pairs of lower experts and those of the same one in tokens
// before.  (4 tokens of 1 KB: 4.0 and 2.6 us and a launch between in two.)
__global__ __launch_bounds__(1024) void dispatch_small(const int32_t* __restrict__ idx,
                                                       const uint4* __restrict__ x,
                                                       uint4* __restrict__ rows,
                                                       int32_t* __restrict__ counts,
                                                       int32_t* __restrict__ offsets,
                                                       int32_t* __restrict__ sorted_pair,
                                                       int32_t* __restrict__ pair_pos,
                                                       int32_t* __restrict__ diag, int T, int E, int k,
                                                       int words) {
  if (blockIdx.x == 0) return small_sort(idx, counts, offsets, sorted_pair, pair_pos, diag, T, E, k);
  __shared__ int raw[kSmallPairs], ids[kSmallPairs];
  __shared__ int place[64], total;
  const int tid = threadIdx.x, lane = tid & 63, t0 = (int)blockIdx.x - 1, P = T * k;
  for (int p = tid; p < P; p += 1024) raw[p] = idx[p];
  if (tid < 64) place[tid] = 0;
  if (tid == 0) total = 0;
  __syncthreads();
  for (int p = tid; p < P; p += 1024) {
    const int t = p / k;
    ids[p] = valid_slot(raw + t * k, p - t * k, E) ? raw[p] : -1;
  }
  __syncthreads();
  // a wave counts for one slot at a time
  for (int s = tid >> 6; s <= k; s += 16) {   // (s == k: all valid pairs)
    const int e = s < k ? ids[t0 * k + s] : E;
    int n = 0;
    for (int p = lane; p < P; p += 64) {
      const int id = ids[p];
      n += id >= 0 && (id < e || (id == e && p < t0 * k));
    }
    n = wave_sum(n);
    if (lane == 0) (s < k ? place[s] : total) = e < 0 ? -1 : n;
  }
  __syncthreads();
  for (int u = tid; u < words; u += 1024) {
    const uint4 v = x[(size_t)t0 * words + u];
    for (int s = 0; s < k; ++s)
      if (place[s] >= 0) rows[(size_t)place[s] * words + u] = v;
  }
  for (int q = total + t0; q < P; q += T)   // behind the last pair's row
    for (int u = tid; u < words; u += 1024) rows[(size_t)q * words + u] = make_uint4(0, 0, 0, 0);
}

// Chunked path.  CH tokens per chunk; the chunk's id rows are staged in LDS with
// coalesced loads.
// Threads of a chunk's workgroup: those of the larger chunks fit a launch of 2^31 tokens.
template <int CH>
constexpr int chunk_threads() { return CH == 64 ? 1024 : 256; }

template <int CH>
__global__ __launch_bounds__(chunk_threads<CH>()) void chunk_hist(const int32_t* __restrict__ idx,
                                                  int32_t* __restrict__ chunk_base,
                                                  int32_t* __restrict__ diag, int64_t T, int E,
                                                  int k) {
  constexpr int N = chunk_threads<CH>();
  __shared__ int rows[kSmallPairs];  // CH * k <= 4096
  __shared__ int cnt[1024];
  const int64_t t0 = (int64_t)blockIdx.x * CH;
  const int np = (int)((T - t0) < CH ? (T - t0) : CH) * k;
  for (int i = threadIdx.x; i < np; i += N) rows[i] = idx[t0 * k + i];
  for (int e = threadIdx.x; e < E; e += N) cnt[e] = 0;
  __syncthreads();
  int bad = 0;
  for (int p = threadIdx.x; p < np; p += N) {
    const int t = p / k;
    if (valid_slot(rows + t * k, p - t * k, E)) atomicAdd(&cnt[rows[p]], 1);
    else ++bad;
  }
  if (bad && diag) atomicAdd(&diag[K3MOE_DIAG_BAD_EXPERT_IDS], bad);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += N) chunk_base[(size_t)blockIdx.x * E + e] = cnt[e];
}

// Lane l of wave g: expert 64 blockIdx + l, the g-th of 16 groups of chunks.
__global__ __launch_bounds__(1024) void chunk_scan(int32_t* __restrict__ chunk_base,
                                                   int32_t* __restrict__ counts, int nchunks,
                                                   int E) {
  __shared__ int sums[16][64];
  constexpr int B = 8;   // loads in flight
  const int l = threadIdx.x & 63, g = threadIdx.x >> 6, e = blockIdx.x * 64 + l;
  const int per = (nchunks + 15) / 16, c0 = g * per, c1 = min(c0 + per, nchunks);
  const bool in = e < E;
  const int32_t* at = chunk_base + (in ? e : 0);
  int sum = 0;
  for (int c = c0; c < c1; c += B) {
    int v[B];
#pragma unroll
    for (int u = 0; u < B; ++u) v[u] = at[(size_t)min(c + u, c1 - 1) * E];
#pragma unroll
    for (int u = 0; u < B; ++u) sum += c + u < c1 ? v[u] : 0;
  }
  sums[g][l] = sum;
  __syncthreads();
  int run = 0;
  for (int q = 0; q < g; ++q) run += sums[q][l];
  if (!in) return;
  if (g == 15) counts[e] = run + sum;
  for (int c = c0; c < c1; c += B) {
    int v[B];
#pragma unroll
    for (int u = 0; u < B; ++u) v[u] = at[(size_t)min(c + u, c1 - 1) * E];
#pragma unroll
    for (int u = 0; u < B; ++u)
      if (c + u < c1) {
        chunk_base[(size_t)(c + u) * E + e] = run;
        run += v[u];
      }
  }
}

template <int CH>
__global__ __launch_bounds__(chunk_threads<CH>()) void chunk_scatter(const int32_t* __restrict__ idx,
                                                     const int32_t* __restrict__ chunk_base,
                                                     const int32_t* __restrict__ counts,
                                                     int32_t* __restrict__ offsets,
                                                     int32_t* __restrict__ sorted_pair,
                                                     int32_t* __restrict__ pair_pos, int64_t T,
                                                     int E, int k) {
  constexpr int NW = CH / 64, N = chunk_threads<CH>(), EPT = 1024 / N;   // experts of a thread
  __shared__ int rows[kSmallPairs];  // CH * k <= 4096
  __shared__ int base[1024];
  __shared__ int wave[N / 64];
  __shared__ unsigned long long mask[1024][NW];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * CH;
  const int np = (int)((T - t0) < CH ? (T - t0) : CH) * k;
  for (int i = tid; i < np; i += N) rows[i] = idx[t0 * k + i];
  for (int i = tid; i < E * NW; i += N) (&mask[0][0])[i] = 0ull;
  // the experts' offsets: thread i has experts EPT i ..
  int c[EPT], before[EPT], sum = 0;
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int e = tid * EPT + j;
    c[j] = e < E ? counts[e] : 0;
    before[j] = e < E ? chunk_base[(size_t)blockIdx.x * E + e] : 0;
    sum += c[j];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o, 64);
    if ((tid & 63) >= o) incl += v;
  }
  if ((tid & 63) == 63) wave[tid >> 6] = incl;
  __syncthreads();
  int off = incl - sum, valid = 0;
#pragma unroll
  for (int w = 0; w < N / 64; ++w) {
    off += w < (tid >> 6) ? wave[w] : 0;
    valid += wave[w];
  }
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int e = tid * EPT + j;
    if (e < E) {
      base[e] = off + before[j];
      if (blockIdx.x == 0) offsets[e] = off;
    }
    off += c[j];
  }
  if (blockIdx.x == 0 && tid == 0) offsets[E] = valid;
  for (int p = tid; p < np; p += N) {
    const int t = p / k;
    if (valid_slot(rows + t * k, p - t * k, E)) atomicOr(&mask[rows[p]][t >> 6], 1ull << (t & 63));
  }
  __syncthreads();
  for (int p = tid; p < np; p += N) {
    const int t = p / k, word = t >> 6;
    const int64_t pair = t0 * k + p;
    if (valid_slot(rows + t * k, p - t * k, E)) {
      const int e = rows[p];
      int rank = __popcll(mask[e][word] & ((1ull << (t & 63)) - 1ull));
      for (int w = 0; w < word; ++w) rank += __popcll(mask[e][w]);
      const int pos = base[e] + rank;
      sorted_pair[pos] = (int32_t)pair;
      pair_pos[pair] = pos;
    } else {
      pair_pos[pair] = -1;
    }
  }
  // Positions past the last valid pair (only when ids were dropped) get -1.
  const int64_t P = T * k;
  for (int64_t q = valid + (int64_t)blockIdx.x * N + tid; q < P; q += (int64_t)gridDim.x * N)
    sorted_pair[q] = -1;
}

template <int CH>
hipError_t chunked(const k3moe_shape& s, const int32_t* idx, int32_t* counts, int32_t* offsets,
                   int32_t* sorted_pair, int32_t* pair_pos, int32_t* diag, const PermuteWs& ws,
                   hipStream_t st) {
  const int nchunks = (int)((s.T + CH - 1) / CH);
  chunk_hist<CH><<<nchunks, chunk_threads<CH>(), 0, st>>>(idx, ws.chunk_base, diag, s.T, s.E, s.k);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  chunk_scan<<<(s.E + 63) / 64, 1024, 0, st>>>(ws.chunk_base, counts, nchunks, s.E);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  chunk_scatter<CH><<<nchunks, chunk_threads<CH>(), 0, st>>>(idx, ws.chunk_base, counts, offsets, sorted_pair,
                                             pair_pos, s.T, s.E, s.k);
  return hipGetLastError();
}

}  // namespace

// Small chunks fill the chip; from 2^17 tokens there are enough of the larger ones,
// whose counts take a quarter of the memory (the workspace is smaller from 2^19 tokens on).
constexpr int64_t kLargeT = 1 << 17;
int permute_chunk_tokens(int64_t T, int k) { return k <= 16 && T >= kLargeT ? 256 : 64; }
size_t permute_least_chunks(int64_t T, int k) { return permute_chunk_tokens(T, k) == 256 ? kLargeT / 64 : 0; }

bool permute_small_ok(const k3moe_shape& s) { return s.T <= kSmallT && s.T * s.k <= kSmallPairs; }
// (each of the moving workgroups compares its token's ids with all: 4096 pairs of 256 x
// 7168 take 38 us so, 28 in two launches; 1024 pairs 15, 18)
bool dispatch_small_ok(const k3moe_shape& s) { return s.T <= kSmallT && s.T * s.k <= 1024; }

hipError_t launch_dispatch_small(const k3moe_shape& s, const void* x, const int32_t* idx, void* rows,
                                 int32_t* counts, int32_t* offsets, int32_t* sorted_pair,
                                 int32_t* pair_pos, int32_t* diag, hipStream_t st) {
  dispatch_small<<<1 + (unsigned)s.T, 1024, 0, st>>>(
      idx, static_cast<const uint4*>(x), static_cast<uint4*>(rows), counts, offsets, sorted_pair,
      pair_pos, diag, (int)s.T, s.E, s.k, s.d / (s.x_dtype == K3MOE_F32 ? 4 : 8));
  return hipGetLastError();
}

hipError_t launch_permute(const k3moe_shape& s, const int32_t* idx, int32_t* counts,
                          int32_t* offsets, int32_t* sorted_pair, int32_t* pair_pos,
                          int32_t* diag, const PermuteWs& ws, hipStream_t st) {
  if (permute_small_ok(s)) {
    permute_small<<<1, 1024, 0, st>>>(idx, counts, offsets, sorted_pair, pair_pos, diag,
                                      (int)s.T, s.E, s.k);
    return hipGetLastError();
  }
  if (permute_chunk_tokens(s.T, s.k) == 256)
    return chunked<256>(s, idx, counts, offsets, sorted_pair, pair_pos, diag, ws, st);
  return chunked<64>(s, idx, counts, offsets, sorted_pair, pair_pos, diag, ws, st);
}

}  // namespace k3
