// moda_evict.cu -- cutting a K/V cache down to its best entries, for B200 (sm_100a).
//
// What it computes, per sequence and KV head: of the len cached entries keep min(len, keep):
// the first `sinks`, the last `recent`, and of the rest those with the highest scores, ties to
// the lowest position; the kept entries' K, V and scores are copied to the new cache in their
// old order, and their old positions written down.
//
// What bounds it: the copy of the kept rows (HBM), once the selection is quick.  Two launches:
//   1. moda_evict_select_kernel: a radix selection.  A float's bits map to an integer of the
//      same order; protected entries get the largest integer, so that one selection of the
//      `keep` largest finds the whole set.  Three passes (11, 11 and 10 bits, from the top)
//      each count the keys that still match the prefix into 2048 bins and step into the bin
//      that holds the keep-th largest.  A row of scores is shared by a cluster of eight CTAs
//      (one CTA for short rows), which add their counts over distributed shared memory.  Then
//      each CTA writes its kept positions behind those of the CTAs before it: everything above
//      the threshold, and of the entries equal to it the first that still fit.
//   2. moda_evict_gather_kernel: the rows, 16 bytes a thread, every destination row its own
//      work item, so that the copy runs at the whole GPU's rate however the kept entries lie.
// Only counts go through atomics, so the result does not depend on their order.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "moda_internal.h"
#include "sm100.cuh"

namespace moda {

namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictBins = 2048;
// Rows of up to this many scores are one CTA's work; longer ones a cluster's.
constexpr int kEvictOneCta = 4096;

struct EvictArgs {
  const uint4 *k, *v;
  const float* score;
  const int* lengths;
  uint4 *k_out, *v_out;
  float* score_out;
  int *index, *lengths_out;
  int B, Hkv, S, keep, sinks, recent;
  int chunks;  // 16-byte chunks of a K or V row
};

__device__ __forceinline__ int evict_length(const EvictArgs& a, int b, bool report = false) {
  const int n = __ldg(a.lengths + b);
  if (report && (n < 0 || n > a.S)) atomicOr(&g_error_word, kErrInternal);
  return min(max(n, 0), a.S);
}

// An integer in the order of the float: -0 counts as 0, a NaN as less than everything.  (By
// its bits alone: arithmetic would flush a subnormal to zero.)
__device__ __forceinline__ uint32_t ordered(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Cluster of kCl CTAs (1 or 8) per (sequence, KV head); CTA `rank` holds the positions
// [rank * seg, (rank + 1) * seg).
template <int kCl>
__global__ void __launch_bounds__(kEvictThreads, 1) moda_evict_select_kernel(const EvictArgs a) {
  namespace cg = cooperative_groups;
  __shared__ __align__(16) int hist[3][kEvictBins];
  __shared__ int wsum[32], wsum2[32];
  __shared__ int found_bin, found_above;
  __shared__ int counts[2];  // this CTA's keys above the threshold, and equal to it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bg = blockIdx.x / kCl, rank = blockIdx.x % kCl;
  const int b = bg / a.Hkv;
  const int len = evict_length(a, b, rank == 0 && tid == 0 && bg % a.Hkv == 0);
  // the copying grid may be scheduled now: it waits for this grid's completion itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int want = min(len, a.keep);
  if (rank == 0 && tid == 0 && bg % a.Hkv == 0) a.lengths_out[b] = want;
  const int seg = ((len + kCl - 1) / kCl + 31) & ~31;
  const int p0 = min(len, rank * seg), p1 = min(len, p0 + seg);
  const float* const row = a.score + (long long)bg * a.S;
  int* const index = a.index + (long long)bg * a.keep;
  float* const score_out = a.score_out + (long long)bg * a.keep;
  if (len <= a.keep) {  // everything stays (the same decision in the whole cluster)
    for (int p = p0 + tid; p < p1; p += kEvictThreads) {
      index[p] = p;
      score_out[p] = row[p];
    }
    return;
  }
  const int last = len - a.recent;
  auto key_at = [&](int p) {
    return p < a.sinks || p >= last ? 0xffffffffu : ordered(__ldg(row + p));
  };
  auto cluster_wait = [&]() {
    if constexpr (kCl > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  };
  for (int i = tid; i < 3 * kEvictBins; i += kEvictThreads) (&hist[0][0])[i] = 0;
  __syncthreads();

  uint32_t prefix = 0;  // the threshold's bits found so far, from the top
  int need = want;      // how many of the keys that match the prefix are to be kept
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    const uint32_t above = pass == 0 ? 0u : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
    for (int p = p0 + tid; p < p1; p += kEvictThreads) {
      const uint32_t key = key_at(p);
      if ((key & above) == prefix) atomicAdd(&hist[pass][(key >> shift) & mask], 1);
    }
    cluster_wait();
    // thread t: bins 2047 - 2t and 2046 - 2t, so that a prefix sum runs from the top bin down
    const int hi_bin = kEvictBins - 1 - 2 * tid, lo_bin = hi_bin - 1;
    int n_hi = 0, n_lo = 0;
    if constexpr (kCl > 1) {
      cg::cluster_group cluster = cg::this_cluster();
#pragma unroll
      for (int r = 0; r < kCl; ++r) {
        const int2 x = *reinterpret_cast<const int2*>(
            cluster.map_shared_rank(&hist[pass][0], r) + lo_bin);
        n_lo += x.x;
        n_hi += x.y;
      }
    } else {
      n_hi = hist[pass][hi_bin];
      n_lo = hist[pass][lo_bin];
    }
    int incl = n_hi + n_lo;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int base = wsum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, base, o);
      if (lane >= o) base += v;
    }
    const int before_warp = __shfl_sync(0xffffffffu, base, warp ? warp - 1 : 0);
    const int before = (warp ? before_warp : 0) + incl - n_hi - n_lo;  // keys in higher bins
    // exactly one bin holds the need-th largest of the matching keys
    if (before < need && before + n_hi >= need) {
      found_bin = hi_bin;
      found_above = before;
    } else if (before + n_hi < need && before + n_hi + n_lo >= need) {
      found_bin = lo_bin;
      found_above = before + n_hi;
    }
    __syncthreads();
    prefix |= uint32_t(found_bin) << shift;
    need -= found_above;
    __syncthreads();
  }

  // positions above the threshold all stay, and the first `need` of those equal to it
  int gt = 0, eq = 0;
  for (int p = p0 + tid; p < p1; p += kEvictThreads) {
    const uint32_t key = key_at(p);
    gt += key > prefix;
    eq += key == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    wsum[warp] = gt;
    wsum2[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    const int g = __reduce_add_sync(0xffffffffu, wsum[lane]);
    const int e = __reduce_add_sync(0xffffffffu, wsum2[lane]);
    if (lane == 0) {
      counts[0] = g;
      counts[1] = e;
    }
  }
  cluster_wait();
  int at = 0, eq_before = 0;  // kept and equal keys of the CTAs before this one
  if constexpr (kCl > 1) {
    for (int r = 0; r < rank; ++r) {
      const int* c = cg::this_cluster().map_shared_rank(&counts[0], r);
      const int g = c[0], e = c[1];
      at += g + min(max(need - eq_before, 0), e);
      eq_before += e;
    }
    // (a CTA must not leave while another still reads its counts)
    cg::this_cluster().barrier_arrive();
  }
  for (int q0 = p0; q0 < p1; q0 += kEvictThreads) {
    const int p = q0 + tid;
    const uint32_t key = p < p1 ? key_at(p) : 0u;
    const bool is_gt = p < p1 && key > prefix, is_eq = p < p1 && key == prefix;
    const uint32_t bg_gt = __ballot_sync(0xffffffffu, is_gt);
    const uint32_t bg_eq = __ballot_sync(0xffffffffu, is_eq);
    if (lane == 0) {
      wsum[warp] = __popc(bg_gt);
      wsum2[warp] = __popc(bg_eq);
    }
    __syncthreads();
    // sums over the warps before this one, and over all of them
    const int g = wsum[lane], e = wsum2[lane];
    const int eq_w = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0);
    const int gt_w = __reduce_add_sync(0xffffffffu, lane < warp ? g : 0);
    const int eq_all = __reduce_add_sync(0xffffffffu, e);
    const int gt_all = __reduce_add_sync(0xffffffffu, g);
    const uint32_t below = (1u << lane) - 1u;
    const int eq_mine = eq_before + eq_w + __popc(bg_eq & below);  // equal keys before p
    if (is_gt || (is_eq && eq_mine < need)) {
      const int kept_eq = min(eq_mine, need) - min(eq_before, need);
      const int dst = at + gt_w + __popc(bg_gt & below) + kept_eq;
      index[dst] = p;
      score_out[dst] = row[p];
    }
    at += gt_all + min(eq_before + eq_all, need) - min(eq_before, need);
    eq_before += eq_all;
    __syncthreads();
  }
  if constexpr (kCl > 1) cg::this_cluster().barrier_wait();
}

// Destination rows in groups of kRows per thread, for loads in flight.
constexpr int kEvictRows = 4;
__global__ void __launch_bounds__(256) moda_evict_gather_kernel(const EvictArgs a, int groups) {
  // thread: chunk c of kEvictRows rows, K and V; rows of a block are `per` apart
  const int per = 256 / a.chunks, c = threadIdx.x % a.chunks, r = threadIdx.x / a.chunks;
  const int bg = blockIdx.x / groups;
  const int j0 = (blockIdx.x - bg * groups) * (per * kEvictRows) + r;
  const int n = min(evict_length(a, bg / a.Hkv), a.keep);
  const int* const index = a.index + (long long)bg * a.keep;
  // the selection's grid: wait for its completion
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long src = (long long)bg * a.S, dst = (long long)bg * a.keep;
  int at[kEvictRows];
#pragma unroll
  for (int i = 0; i < kEvictRows; ++i) at[i] = j0 + i * per < n ? index[j0 + i * per] : -1;
  uint4 x[kEvictRows], y[kEvictRows];
#pragma unroll
  for (int i = 0; i < kEvictRows; ++i)
    if (at[i] >= 0) {
      x[i] = ldg_nc_v4(a.k + (src + at[i]) * a.chunks + c);
      y[i] = ldg_nc_v4(a.v + (src + at[i]) * a.chunks + c);
    }
#pragma unroll
  for (int i = 0; i < kEvictRows; ++i)
    if (at[i] >= 0) {
      a.k_out[(dst + j0 + i * per) * a.chunks + c] = x[i];
      a.v_out[(dst + j0 + i * per) * a.chunks + c] = y[i];
    }
}

template <int kCl>
cudaError_t launch_select(const EvictArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.B) * a.Hkv * kCl);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moda_evict_select_kernel<kCl>, a);
}

}  // namespace

cudaError_t launch_evict(const EvictProblem& p, const void* k, const void* v, const float* score,
                         const int* lengths, void* k_out, void* v_out, float* score_out,
                         int* index, int* lengths_out, cudaStream_t stream, const char** why) {
  EvictArgs a;
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.score = score;
  a.lengths = lengths;
  a.k_out = static_cast<uint4*>(k_out);
  a.v_out = static_cast<uint4*>(v_out);
  a.score_out = score_out;
  a.index = index;
  a.lengths_out = lengths_out;
  a.B = p.B;
  a.Hkv = p.Hkv;
  a.S = p.S;
  a.keep = p.keep;
  a.sinks = p.sinks;
  a.recent = p.recent;
  a.chunks = p.d / 8;
  cudaError_t e = p.S <= kEvictOneCta ? launch_select<1>(a, stream) : launch_select<8>(a, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = "eviction's selection launch failed";
    return e;
  }
  const int rows = 256 / a.chunks * kEvictRows;  // destination rows of a block
  const int most = min(p.keep, p.S);
  const int groups = (most + rows - 1) / rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.B) * p.Hkv * groups);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, moda_evict_gather_kernel, a, groups);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) *why = "eviction's copy launch failed";
  return e;
}

}  // namespace moda
