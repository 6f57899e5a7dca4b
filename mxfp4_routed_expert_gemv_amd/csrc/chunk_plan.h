// How the router's weight gradient cuts an expert's pairs into chunks, for host and device.
#pragma once

#include <cstdint>

namespace k3 {

// Pairs of a chunk; an expert without pairs has a chunk too, which writes its zeros.
constexpr int kChunk = 256;

// Chunks of an expert of n pairs, 0 <= n < 2^31, and where chunk i of those from pair q0 on
// begins and ends (q0 + n < 2^31).
constexpr int chunks_of(int n) { return n > kChunk ? n / kChunk + (n % kChunk != 0) : 1; }
constexpr int chunk_begin(int q0, int i) { return q0 + i * kChunk; }
constexpr int chunk_end(int q0, int n, int i) {
  const int64_t most = (int64_t(i) + 1) * kChunk;
  return q0 + (most < n ? (int)most : n);
}

// Chunks of all experts at most, for P < 2^31 pairs, and of those that have several.  An
// expert of more than kChunk pairs (so of more than kChunk tokens) has at most twice its
// pairs / kChunk chunks.
constexpr int most_chunks(int E, int64_t P) { return (int)(E + P / kChunk); }
constexpr int most_parts(int64_t T, int64_t P) { return T > kChunk ? (int)(2 * (P / kChunk)) : 0; }

}  // namespace k3
