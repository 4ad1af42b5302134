// moda_evict.cu -- cutting a K/V cache down to its best entries, for B200 (sm_100a).
//
// What it computes, per sequence and KV head: of the len cached entries keep min(len, keep):
// the first `sinks`, the last `recent`, and of the rest those with the highest scores, ties to
// the lowest position; the kept entries' K, V and scores are copied to the new cache in their
// old order, and their old positions written down.
//
// What bounds it: the copy of the kept rows (HBM), once the selection is quick (16 rows of 64K
// scores, 8192 kept, d = 128: 41.6 us from a graph; in the profiler the selection takes 20 and the copy
// 21 for 134 MB).  Two launches:
//   1. moda_evict_select_kernel: a radix selection.  A float's bits map to an integer of the
//      same order; protected entries get the largest integer, so that one selection of the
//      `keep` largest finds the whole set.  Four passes of 8 bits, from the top, each count the
//      keys that still match the prefix into 256 bins and step into the bin that holds the
//      keep-th largest.  A row of scores is shared by a cluster of eight CTAs (one CTA for short
//      rows), which add their counts over distributed shared memory.  The keys are read from
//      global memory once and stay in shared memory.  Then each warp, whose keys are a
//      contiguous run, writes its kept positions behind those of the warps and CTAs before it:
//      everything above the threshold, and of the entries equal to it the first that still fit.
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

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
// Rows of up to this many scores are one CTA's work; longer ones a cluster's.
constexpr int kEvictOneCta = 8192;
// Keys a CTA holds in shared memory (96 KB, so that two CTAs share an SM: with one CTA an SM
// the clusters of 16 rows did not all fit the GPU at once).  Longer rows are read from global
// memory in every pass.
constexpr int kEvictHeld = 24576;

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
// [rank * seg, (rank + 1) * seg), its warp w a contiguous sixteenth of them.
template <int kCl, bool kHeld>
__global__ void __launch_bounds__(kEvictThreads, 2) moda_evict_select_kernel(const EvictArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t held[];  // kHeld: this CTA's keys
  // kCopies counters per bin, by lane, for the counting itself: scores crowd in a few bins (many
  // are exactly zero), and the adds of one warp to one address come one after the other
  constexpr int kCopies = 8;
  __shared__ __align__(16) int tally[256 * kCopies];
  __shared__ int hist[4][256];
  __shared__ int wsum[kEvictWarps], wsum2[kEvictWarps];
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
  const int run = (((len + kCl - 1) / kCl + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  // this warp's positions [w0, w1)
  const long long first = ((long long)rank * kEvictWarps + warp) * run;
  const int w0 = int(min((long long)len, first)), w1 = int(min((long long)len, first + run));
  const float* const row = a.score + (long long)bg * a.S;
  int* const index = a.index + (long long)bg * a.keep;
  float* const score_out = a.score_out + (long long)bg * a.keep;
  if (len <= a.keep) {  // everything stays (the same decision in the whole cluster)
    for (int p = w0 + lane; p < w1; p += 32) {
      index[p] = p;
      score_out[p] = row[p];
    }
    return;
  }
  const int last = len - a.recent;
  auto make_key = [&](int p) {
    const uint32_t key = ordered(__ldg(row + p));
    return p < a.sinks || p >= last ? 0xffffffffu : key;
  };
  uint32_t* const mine = held + warp * run - w0;  // key of position p at mine[p]
  auto key_at = [&](int p) { return kHeld ? mine[p] : make_key(p); };
  auto cluster_wait = [&]() {
    if constexpr (kCl > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  };
  for (int i = tid; i < 256 * kCopies; i += kEvictThreads) tally[i] = 0;
  if constexpr (kHeld) {
    // (each warp reads and later uses only its own run)
#pragma unroll 8
    for (int p = w0 + lane; p < w1; p += 32) mine[p] = make_key(p);
  }
  __syncthreads();

  uint32_t prefix = 0;  // the threshold's bits found so far, from the top
  int need = want;      // how many of the keys that match the prefix are to be kept
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
#pragma unroll 4
    for (int p = w0 + lane; p < w1; p += 32) {
      const uint32_t key = key_at(p);
      if ((key & above) == prefix)
        atomicAdd(&tally[((key >> shift) & 255u) * kCopies + (lane & (kCopies - 1))], 1);
    }
    __syncthreads();
    if (tid < 256) {
      int4* const t4 = reinterpret_cast<int4*>(tally + tid * kCopies);
      const int4 x = t4[0], y = t4[1];
      hist[pass][tid] = (x.x + x.y) + (x.z + x.w) + (y.x + y.y) + (y.z + y.w);
      t4[0] = t4[1] = make_int4(0, 0, 0, 0);
    }
    cluster_wait();
    // thread t < 256: bin 255 - t, so that a prefix sum runs from the top bin down
    int n = 0, incl = 0;
    if (tid < 256) {
      if constexpr (kCl > 1) {
        cg::cluster_group cluster = cg::this_cluster();
#pragma unroll
        for (int r = 0; r < kCl; ++r) n += cluster.map_shared_rank(&hist[pass][0], r)[255 - tid];
      } else {
        n = hist[pass][255 - tid];
      }
      incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) wsum[warp] = incl;
    }
    __syncthreads();
    if (tid < 256) {
      const int before =
          incl - n + __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane & 7] : 0);
      // exactly one bin holds the need-th largest of the matching keys
      if (before < need && before + n >= need) {
        found_bin = 255 - tid;
        found_above = before;
      }
    }
    __syncthreads();
    prefix |= uint32_t(found_bin) << shift;
    need -= found_above;
  }

  // positions above the threshold all stay, and the first `need` of those equal to it
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int p = w0 + lane; p < w1; p += 32) {
    const uint32_t key = key_at(p);
    gt += key > prefix;
    eq += key == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  __syncthreads();  // (wsum's last readers)
  if (lane == 0) {
    wsum[warp] = gt;
    wsum2[warp] = eq;
  }
  __syncthreads();
  const int g = lane < kEvictWarps ? wsum[lane] : 0, e = lane < kEvictWarps ? wsum2[lane] : 0;
  if (warp == 0) {
    const int gs = __reduce_add_sync(0xffffffffu, g), es = __reduce_add_sync(0xffffffffu, e);
    if (lane == 0) {
      counts[0] = gs;
      counts[1] = es;
    }
  }
  // keys above and equal in the warps, then in the CTAs, before this one
  int gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? g : 0);
  int eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0);
  if constexpr (kCl > 1) {
    cg::this_cluster().sync();
    const int* c = cg::this_cluster().map_shared_rank(&counts[0], lane < rank ? lane : rank);
    gt_before += __reduce_add_sync(0xffffffffu, lane < rank ? c[0] : 0);
    eq_before += __reduce_add_sync(0xffffffffu, lane < rank ? c[1] : 0);
    // (a CTA must not leave while another still reads its counts)
    cg::this_cluster().barrier_arrive();
  }
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int q = w0; q < w1; q += 32) {
    const int p = q + lane;
    const uint32_t key = p < w1 ? key_at(p) : 0u;
    const float score = p < w1 ? __ldg(row + p) : 0.f;
    const uint32_t m_gt = __ballot_sync(0xffffffffu, p < w1 && key > prefix);
    const uint32_t m_eq = __ballot_sync(0xffffffffu, p < w1 && key == prefix);
    const int eq_mine = eq_before + __popc(m_eq & below);  // equal keys before p
    const bool is_eq = (m_eq >> lane) & 1u;
    if (((m_gt >> lane) & 1u) || (is_eq && eq_mine < need)) {
      const int dst = gt_before + __popc(m_gt & below) + min(eq_mine, need);
      index[dst] = p;
      score_out[dst] = score;
    }
    gt_before += __popc(m_gt);
    eq_before += __popc(m_eq);
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

template <int kCl, bool kHeld>
cudaError_t launch_select(const EvictArgs& a, cudaStream_t stream) {
  const int run = (((a.S + kCl - 1) / kCl + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.B) * a.Hkv * kCl);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = kHeld ? size_t(run) * kEvictWarps * 4 : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // (the limit of every call, not this one's size: calls may come from several threads)
  cudaError_t e = cudaFuncSetAttribute(moda_evict_select_kernel<kCl, kHeld>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kHeld ? kEvictHeld * 4 : 0);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, moda_evict_select_kernel<kCl, kHeld>, a);
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
  cudaError_t e = p.S <= kEvictOneCta       ? launch_select<1, true>(a, stream)
                  : (p.S + 7) / 8 <= kEvictHeld - 512 ? launch_select<8, true>(a, stream)
                                                      : launch_select<8, false>(a, stream);
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
