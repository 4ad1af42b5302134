// moda_packed.cuh -- how a CTA of the packed kernels finds its piece of work.
//
// A packed batch holds nseq sequences one behind the other: sequence s owns the token rows
// [cu[s], cu[s+1]) of N.  The lengths are known on the device alone, so the grid is sized
// by an upper bound and each CTA looks its piece up: sequence s has n_s = ceil(len_s / U)
// pieces of U tokens, piece p of a sequence costs about p + 1 (causal attention), and the
// pieces are numbered heaviest first over all sequences:
//   F(p) = sum_s max(0, n_s - p)   pieces whose index is at least p;
//   piece number c has the largest p with F(p) > c, and is the (c - F(p+1))-th sequence
//   with n_s > p.
// A binary search over p, each F a sum over the sequences by one warp; no plan has to be
// made, kept or passed, and a captured graph follows the lengths it finds when it runs.
// Every warp of the CTA runs the search by itself (the same reads, so the same answer),
// which needs no barrier; 64 sequences take well under a microsecond.
#pragma once

#include <stdint.h>

namespace moda {

struct PackedPiece {
  int first;  // first token row of the sequence
  int len;    // its length
  int p, n;   // piece index and number of pieces of this sequence
  bool found;
};

// Bounds of sequence s, clamped to [0, N); a sequence whose entries decrease or leave
// [0, N] is empty (and reported through `bad`).
__device__ __forceinline__ int packed_len(const int* cu, int s, int N, int& first, bool& bad) {
  const int a = __ldg(cu + s), e = __ldg(cu + s + 1);
  first = a;
  if (a < 0 || e < a || e > N) {
    bad = true;
    return 0;
  }
  return e - a;
}

// Piece number c (all 32 lanes call this together, with the same arguments).  With good bounds every
// count is below 2^31.  Where entries go back, sequences whose own bounds are good may overlap, and
// the counts may wrap around: what is found is then some piece of one of them, or none.
__device__ __forceinline__ PackedPiece packed_find(const int* cu, int nseq, int N, int U, int c) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  int first;
  auto pieces = [&](int s) { return (packed_len(cu, s, N, first, bad) + U - 1) / U; };
  // the first 32 sequences' counts stay in a register
  const int n0 = lane < nseq ? pieces(lane) : 0;
  auto total = [&](int p) {
    uint32_t t = max(0, n0 - p);
    for (int s = lane + 32; s < nseq; s += 32) t += max(0, pieces(s) - p);
    return __reduce_add_sync(0xffffffffu, t);
  };
  PackedPiece r{0, 0, 0, 0, false};
  int most = n0;
  for (int s = lane + 32; s < nseq; s += 32) most = max(most, pieces(s));
  most = __reduce_max_sync(0xffffffffu, most);
  if (__any_sync(0xffffffffu, bad) && threadIdx.x == 0) atomicOr(&g_error_word, kErrInternal);
  if (uint32_t(c) >= total(0)) return r;
  int lo = 0, hi = most;  // F(lo) > c >= F(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (total(mid) > uint32_t(c))
      lo = mid;
    else
      hi = mid;
  }
  // (below zero only where the counts have wrapped: then some lane still holds it)
  int rank = max(0, int(uint32_t(c) - total(lo + 1)));
  for (int s0 = 0; s0 < nseq; s0 += 32) {
    const int s = s0 + lane;
    const int n = s0 == 0 ? n0 : (s < nseq ? pieces(s) : 0);
    const uint32_t m = __ballot_sync(0xffffffffu, n > lo);
    const int here = __popc(m);
    if (rank < here) {
      // the lane that holds the rank-th of these sequences
      const bool mine = n > lo && __popc(m & ((1u << lane) - 1u)) == rank;
      const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      const int len = mine ? packed_len(cu, s, N, first, bad) : 0;
      r.first = __shfl_sync(0xffffffffu, first, src);
      r.len = __shfl_sync(0xffffffffu, len, src);
      r.n = __shfl_sync(0xffffffffu, n, src);
      r.p = lo;
      r.found = true;
      return r;
    }
    rank -= here;
  }
  return r;
}

// Upper bound of the number of pieces: each sequence has at most len / U + 1.
inline long long packed_pieces_bound(long long N, long long nseq, long long U) {
  return N / U + (nseq < N ? nseq : N);
}

// Rows [r0, r1) of a 128-row operand tile (128-byte swizzled regions, whose rows are
// contiguous) set to zero by one warp, for the tensor cores to read afterwards.  A row
// outside the sequence has weight zero, but zero times an infinity or a NaN is a NaN, so
// what lies there (another sequence, memory never written) must not enter a product.
__device__ __forceinline__ void zero_tile_rows(uint32_t tile, int regions, int r0, int r1) {
  const int lane = threadIdx.x & 31;
  for (int rg = 0; rg < regions; ++rg)
    for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
      sts128(tile + uint32_t(rg) * 16384u + uint32_t(i) * 16u, make_uint4(0u, 0u, 0u, 0u));
}
// ... and published to the asynchronous proxy through `bar` (one arrival).
__device__ __forceinline__ void publish_rows(uint32_t bar) {
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

}  // namespace moda
