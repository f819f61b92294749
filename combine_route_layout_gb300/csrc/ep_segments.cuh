// The rows of all segments as equal pieces, for kernels whose CTAs go through them
// in turn: a CTA adds up the segments' pieces once, in shared memory, and finds a
// piece's place by binary search.
#pragma once

#include "ep_linear.cuh"

namespace ep {
namespace {

struct Piece {
  int64_t row;    // first pool row
  int rows;
  int group;
};

// Ints of shared memory for G groups: first piece and first row of each, one end.
constexpr int kSegmentInts = 3;

// Pieces of `per` rows of a segment. `count` goes up to INT32_MAX - 1024, so that with
// `per` rows more it passes an int.
__host__ __device__ inline int64_t pieces_of(int64_t count, int per) { return (count + per - 1) / per; }

// Pieces of all segments, at most: what a CTA's next one, a grid of them on, still fits.
constexpr int64_t kMostPieces = INT32_MAX - (1 << 20);

inline size_t segment_bytes(int G) { return (size_t)(kSegmentInts * G + 1) * sizeof(int); }

#ifdef __CUDACC__

// table: [G + 1] first pieces, then [G] first rows, then [G] counts. All threads of the
// CTA (at most 1024, whole warps); returns the number of pieces of `per` rows: none,
// with an error, where overlapping segments have more than kMostPieces.
__device__ __forceinline__ int segment_table(const LinearSegs& s, int per, int* table) {
  __shared__ int64_t sums[32];
  int* begins = table + s.G + 1;
  int* counts = begins + s.G;
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (s.G + threads - 1) / threads;
  const int g0 = threadIdx.x * each, g1 = min(s.G, g0 + each);
  int64_t mine = 0;
  for (int g = g0; g < g1; ++g) {
    int64_t b, c;
    segment_of(s, g, b, c);
    begins[g] = (int)b;
    counts[g] = (int)c;
    mine += pieces_of(c, per);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine;
  for (int w = 0; w < warp; ++w) before += sums[w];
  for (int g = g0; g < g1; ++g) {
    table[g] = (int)before;
    before += pieces_of(counts[g], per);
  }
  int64_t total = 0;
  for (int w = 0; w < threads / 32; ++w) total += sums[w];
  if (total > kMostPieces) {
    total = 0;
    if (threadIdx.x == 0) atomicOr(s.err, kErrSegment);
  }
  if (threadIdx.x == 0) table[s.G] = (int)total;
  __syncthreads();
  return (int)total;
}

__device__ __forceinline__ Piece piece_at(const LinearSegs& s, int per, const int* table, int piece) {
  int lo = 0, hi = s.G - 1;            // the last group that starts at or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table[mid] <= piece) lo = mid; else hi = mid - 1;
  }
  const int* begins = table + s.G + 1;
  const int in = (piece - table[lo]) * per;
  Piece p;
  p.group = lo;
  p.row = (int64_t)begins[lo] + in;
  p.rows = min(per, begins[s.G + lo] - in);
  return p;
}

#endif
}  // namespace
}  // namespace ep
