// moda_score.cu -- the attention weight that new queries give to each cached key, for B200
// (sm_100a).
//
// What it computes: for the newest N tokens of each sequence, whose log-sum-exp the attention
// has returned,
//   score_out[b,g,s] = score[b,g,s] + sum_{h in group g} sum_{i: s <= pos_i}
//                      exp(scale*<q[b,h,i], k[b,g,s]> - lse[b,h,i]),   pos_i = len_b - N + i.
// The weights are those of MoDA's joint softmax (hyper.ai summary of arXiv 2603.15619, section
// "Mixture-of-Depths Attention (MoDA)"): the share that went to depth entries is in lse.
//
// What bounds it: each key is read once and meets the G x N rows of its KV head.  Up to about
// 128 rows that is a stream of K from HBM; beyond, the exponentials take longer.  (8 caches of up
// to 64K keys, 16 heads, one token, from a graph: 68 us, 5.5 TB/s; 33 tokens over 2 caches of 5000,
// d = 64: 14.3 us, a CTA's own latency.  More than three row tiles read K again in another launch: the
// same 8 caches, 96 tokens 237 us, 128 tokens 334.)
//   The products are S^T = K Q^T: a key is a TMEM lane, so one thread owns one key and adds its
// weights up in a register, in a fixed order -- no reduction across threads, no atomics, the
// same bits every run.  The row tiles (up to three of 128 rows; more rows take more launches)
// stay in shared memory while K streams through a TMA ring.  The 128-key blocks of all
// sequences and KV heads are laid in one line and cut into equal shares, one per CTA,
// whatever the lengths are.  Two warpgroups take alternate blocks, two S buffers each.
//
// Warp roles (352 threads, one CTA per SM): warps 0-3 and 4-7 the weights, warp 8 TMA, warp 9
// tcgen05 issuer, warp 10 the rows' log-sum-exp (rows that carry no weight are zeroed, so that
// what lies there cannot become a NaN).  TMEM: S buffer (warpgroup w, i) at 256 w + 128 i.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "moda_internal.h"
#include "moda_packed.cuh"
#include "sm100.cuh"

namespace moda {

namespace {

constexpr int kScoreThreads = 352;
constexpr int kScoreCtas = 148;
constexpr int kScoreMaxTiles = 3;  // row tiles of one launch
constexpr int kScoreRegion = 16384;
constexpr int kScoreMaxStages = 12;
constexpr float kLog2eScore = 1.4426950408889634f;

template <int D>
struct ScoreCfg {
  static constexpr int kRegions = D / 64;
  static constexpr int kTile = kRegions * kScoreRegion;
  static constexpr int kOperands = 7 * 32768;  // row tiles, then the K ring
  static constexpr int kOffLse = kOperands;    // [kScoreMaxTiles * 128] fp32
  static constexpr int kOffBar = kOffLse + kScoreMaxTiles * 128 * 4;
  static constexpr int kSmemBytes = kOffBar + 320;
};

struct ScoreArgs {
  const float* score;
  float* score_out;
  const float* lse;  // [B][Hq][N]
  const int* lengths;
  int B, Hq, Hkv, G, N, S;
  int tok0, ntok;        // the query tokens of this launch
  int TQ, tiles, stages;  // tokens per row tile, row tiles, ring stages
  int copy_tail;         // also copy the scores behind each length (score_out != score)
  float scale_log2;
};

struct ScoreBars {
  uint64_t full[kScoreMaxStages], empty[kScoreMaxStages];
  uint64_t q_full, q_ready, q_empty;
  uint64_t s_full[2][2], s_free[2][2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ int score_length(const ScoreArgs& a, int b, bool report = false) {
  const int n = __ldg(a.lengths + b);
  if (report && (n < 0 || n > a.S)) atomicOr(&g_error_word, kErrInternal);
  return min(max(n, 0), a.S);
}
__device__ __forceinline__ int score_blocks(const ScoreArgs& a, int b) {
  return (score_length(a, b) + 127) / 128;
}

// A CTA's walk over its share of the key blocks, piece by piece: blocks [j0, j1) of KV head g
// of sequence b.
struct ScoreWalk {
  long long left;
  int b, g, j0, j1, len;
  __device__ __forceinline__ void clip(const ScoreArgs& a) {
    len = score_length(a, b);
    const int n = (len + 127) / 128;
    const long long want = left < n - j0 ? left : n - j0;
    j1 = j0 + int(want);
    left -= want;
  }
  __device__ __forceinline__ bool next(const ScoreArgs& a) {
    if (left <= 0) return false;
    if (++g == a.Hkv) {
      g = 0;
      do ++b;
      while (score_blocks(a, b) == 0);  // (more blocks are left, so one is not empty)
    }
    j0 = 0;
    clip(a);
    return true;
  }
};

__device__ __forceinline__ ScoreWalk score_first(const ScoreArgs& a, long long s, long long left) {
  const int lane = threadIdx.x & 31;
  ScoreWalk w;
  w.left = left;
  w.b = w.g = w.j0 = 0;
  long long before = 0;  // blocks of one KV head of the earlier sequences
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int mine = b0 + lane < a.B ? score_blocks(a, b0 + lane) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const bool past = b0 + lane < a.B && (before + incl) * a.Hkv > s;
    const uint32_t m = __ballot_sync(0xffffffffu, past);
    if (m) {
      const int src = __ffs(m) - 1;
      const int n = __shfl_sync(0xffffffffu, mine, src);
      const int at = __shfl_sync(0xffffffffu, incl, src) - n;
      const long long off = s - (before + at) * a.Hkv;
      w.b = b0 + src;
      w.g = int(off / n);
      w.j0 = int(off - (long long)w.g * n);
      break;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  w.clip(a);
  return w;
}

// This warpgroup's part of the scores behind each length, copied when score_out is not score:
// units of 1024 scores, one beside each key block (loaded before the block's weights are
// waited for and stored after them, so that it costs no time of its own), the rest at the end.
struct TailCopy {
  static constexpr int kEach = 8;  // scores per thread of a unit
  long long u, units;
  int per, at;
  __device__ __forceinline__ TailCopy(const ScoreArgs& a, int wg, int thread) {
    per = (a.S + 1023) / 1024;
    units = a.copy_tail ? (long long)a.B * a.Hkv * per : 0;
    u = 2ll * blockIdx.x + wg;
    at = thread;
  }
  template <typename F>
  __device__ __forceinline__ void each(const ScoreArgs& a, F f) const {
    const int bg = int(u / per), c = int(u - (long long)bg * per);
    const int lo = score_length(a, bg / a.Hkv);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int p = c * 1024 + i * 128 + at;
      if (p >= lo && p < a.S) f(i, (long long)bg * a.S + p);
    }
  }
  __device__ __forceinline__ void load(const ScoreArgs& a, float (&x)[kEach]) const {
    if (u < units) each(a, [&](int i, long long p) { x[i] = a.score[p]; });
  }
  __device__ __forceinline__ void store(const ScoreArgs& a, const float (&x)[kEach]) {
    if (u < units) each(a, [&](int i, long long p) { a.score_out[p] = x[i]; });
    u += 2 * gridDim.x;
  }
  __device__ __forceinline__ void rest(const ScoreArgs& a) {
    while (u < units) {
      float x[kEach];
      load(a, x);
      store(a, x);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kScoreThreads, 1)
    moda_score_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK, const ScoreArgs a) {
  using Cfg = ScoreCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicOr(&g_error_word, kErrInternal);
    return;
  }
  const uint32_t s0 = smem_u32(smem);
  const int nt = a.tiles, NS = a.stages;
  auto sQ = [&](int t) { return s0 + uint32_t(t) * Cfg::kTile; };
  auto sK = [&](int s) { return s0 + uint32_t(nt + s) * Cfg::kTile; };
  float* const lse2 = reinterpret_cast<float*>(smem + Cfg::kOffLse);
  ScoreBars* bars = reinterpret_cast<ScoreBars*>(smem + Cfg::kOffBar);
  static_assert(sizeof(ScoreBars) <= 320, "barrier space");
  volatile int* abort_flag = &bars->abort;
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  bool no_loads = false;
  if (warp == 8) {
    if (lane < 2) tma_prefetch_desc(lane ? &tmQ : &tmK);
    // test-only fault: issue no loads, so that every wait for them runs out
    no_loads = g_device_fault == kFaultForwardNoLoads;
  }
  long long n = 0;
  for (int b = lane; b < a.B; b += 32) n += score_blocks(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  const long long total = n * a.Hkv;
  const long long share = (total + kScoreCtas - 1) / kScoreCtas;
  const long long first = share * blockIdx.x;
  if (blockIdx.x == 0 && warp == 0)
    for (int b = lane; b < a.B; b += 32) score_length(a, b, true);
  if (first >= total) {  // no block for this CTA; its part of the tails is left
    TailCopy tail(a, threadIdx.x >> 7, threadIdx.x & 127);
    if (threadIdx.x < 256) tail.rest(a);
    return;
  }
  const ScoreWalk walk0 = score_first(a, first, min(share, total - first));

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(bars->full[s]), 1);
      mbar_init(bar(bars->empty[s]), 1);
    }
    mbar_init(bar(bars->q_full), 1);
    mbar_init(bar(bars->q_ready), 1);
    mbar_init(bar(bars->q_empty), 1 + 8);  // the products, and each weights warp (lse2)
    for (int w = 0; w < 2; ++w)
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(bars->s_full[w][i]), 1);
        mbar_init(bar(bars->s_free[w][i]), 4);
      }
    mbar_init(bar(bars->drain), 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 8) {
    // ------------------------------------------------------------ TMA
    if (lane == 0 && !no_loads) {
      int e = 0;
      ScoreWalk w = walk0;
      bool more = true;
      while (more && !*abort_flag) {
        for (int j = w.j0; j < w.j1; ++j, ++e) {
          const int s = e % NS;
          if (e >= NS && !mbar_wait(bar(bars->empty[s]), ((e / NS) - 1) & 1, abort_flag)) break;
          mbar_expect_tx(bar(bars->full[s]), Cfg::kTile);
          for (int rg = 0; rg < Cfg::kRegions; ++rg)
            tma_load_3d(sK(s) + rg * kScoreRegion, &tmK, bar(bars->full[s]), rg * 64, j * 128,
                        w.b * a.Hkv + w.g);
        }
        more = w.next(a);
      }
      if (*abort_flag)  // abort path: what was issued still lands; wait for it before exit
        for (int i = e > NS ? e - NS : 0; i < e; ++i)
          mbar_wait_drain(bar(bars->full[i % NS]), (i / NS) & 1);
    } else if (lane == 1 && !no_loads) {
      ScoreWalk w = walk0;
      int pc = 0;
      bool more = true;
      for (; more; ++pc, more = w.next(a)) {
        if (pc > 0 && !mbar_wait(bar(bars->q_empty), (pc - 1) & 1, abort_flag)) break;
        mbar_expect_tx(bar(bars->q_full), uint32_t(nt * Cfg::kRegions) * 128u * a.G * a.TQ);
        for (int t = 0; t < nt; ++t)
          for (int rg = 0; rg < Cfg::kRegions; ++rg)
            tma_load_4d(sQ(t) + rg * kScoreRegion, &tmQ, bar(bars->q_full), rg * 64, 0,
                        a.tok0 + t * a.TQ, w.b * a.Hkv + w.g);
      }
      if (*abort_flag && pc > 0) mbar_wait_drain(bar(bars->q_full), (pc - 1) & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ tcgen05 issuer
    // Blocks in pairs, one per warpgroup, and within a pair tile by tile, so that both
    // warpgroups always have a product to work on.
    if (elect_one()) {
      const int cols = (a.TQ * a.G + 15) & ~15;  // columns of a tile's S^T
      const uint32_t idesc = make_idesc_bf16(128, cols, 0, 0);
      ScoreWalk w = walk0;
      int e = 0, pc = 0;        // ring entry of block j0, piece
      uint32_t used[2] = {0, 0};  // units given to each warpgroup
      bool more = true;
      while (more && !*abort_flag) {
        mbar_wait(bar(bars->q_ready), pc & 1, abort_flag);
        for (int j = w.j0; j < w.j1 && !*abort_flag; j += 2) {
          const int nb = min(2, w.j1 - j);
          for (int t = 0; t < nt; ++t)
            for (int x = 0; x < nb; ++x) {
              const int en = e + (j - w.j0) + x, s = en % NS;
              // (the piece's first block always goes to warpgroup 0)
              if (t == 0) mbar_wait(bar(bars->full[s]), (en / NS) & 1, abort_flag);
              const uint32_t uo = used[x]++, i = uo & 1;
              if (uo >= 2) mbar_wait(bar(bars->s_free[x][i]), ((uo >> 1) - 1) & 1, abort_flag);
              tc_fence_after();
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks / 4) * kScoreRegion + (ks % 4) * 32;
                mma_ss(tmem + x * 256 + i * 128, make_sdesc_sw128(sK(s) + off, 16, 1024),
                       make_sdesc_sw128(sQ(t) + off, 16, 1024), idesc, ks > 0 ? 1u : 0u);
              }
              tc_commit(bar(bars->s_full[x][i]));
              if (t == nt - 1) tc_commit(bar(bars->empty[s]));
            }
        }
        tc_commit(bar(bars->q_empty));
        e += w.j1 - w.j0;
        ++pc;
        more = w.next(a);
      }
      if (*abort_flag) {
        tc_commit(bar(bars->drain));
        mbar_wait_drain(bar(bars->drain), 0);
      }
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ rows' log-sum-exp
    ScoreWalk w = walk0;
    int pc = 0;
    bool more = true;
    for (; more; ++pc, more = w.next(a)) {
      // (the tiles were reloaded only once the piece before was done with them and with lse2)
      if (!__all_sync(0xffffffffu, mbar_wait(bar(bars->q_full), pc & 1, abort_flag))) break;
      for (int t = 0; t < nt; ++t)
        for (int r0 = 0; r0 < a.TQ * a.G; r0 += 32) {
          const int r = r0 + lane, tok = r / a.G, i = a.tok0 + t * a.TQ + tok;
          const bool in = r < a.TQ * a.G && t * a.TQ + tok < a.ntok;
          float v = INFINITY;
          if (in && w.len - a.N + i >= 0) {  // (a query before the cache's start: no weight)
            const float x = __ldg(a.lse + ((long long)w.b * a.Hq + w.g * a.G + r - tok * a.G) * a.N + i);
            if (x != -INFINITY) v = x * kLog2eScore;  // -inf: a row that saw nothing
          }
          if (in) lse2[t * 128 + r] = v;
          // rows [.., ntok) without a weight, zeroed; the rows behind them are never summed
          const bool none = in && v == INFINITY;
          if (__any_sync(0xffffffffu, none))
            for (int z = 0; z < 32; ++z)
              if (__shfl_sync(0xffffffffu, none, z))
                zero_tile_rows(sQ(t), Cfg::kRegions, r0 + z, r0 + z + 1);
        }
      publish_rows(bar(bars->q_ready));
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ weights
    const int wg = warp >> 2;
    const int key = threadIdx.x & 127;  // TMEM lane = key of the block
    const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16) + wg * 256;
    ScoreWalk w = walk0;
    TailCopy tail(a, wg, key);
    uint32_t uo = 0;
    int pc = 0;
    bool more = true;
    for (; more; ++pc) {
      mbar_wait(bar(bars->q_ready), pc & 1, abort_flag);  // lse2
      const long long row = ((long long)w.b * a.Hkv + w.g) * a.S;
      for (int j = w.j0 + wg; j < w.j1; j += 2) {
        float moved[TailCopy::kEach];
        tail.load(a, moved);
        const int s = j * 128 + key;  // position of this thread's key
        const bool inside = s < w.len;
        const float old = inside ? a.score[row + s] : 0.f;  // (may be score_out)
        // query i sees the key iff s <= len - N + i: from token see on
        const int see = s - (w.len - a.N) - a.tok0;
        const bool masked = j * 128 + 127 > w.len - a.N + a.tok0;
        float2 sum = make_float2(0.f, 0.f);
        for (int t = 0; t < nt; ++t, ++uo) {
          mbar_wait(bar(bars->s_full[wg][uo & 1]), (uo >> 1) & 1, abort_flag);
          tc_fence_after();
          const uint32_t base = tS + (uo & 1) * 128;
          const int rows = min(a.TQ, a.ntok - t * a.TQ) * a.G;
          // first tile row whose token sees this key
          const int lo = masked ? (see - t * a.TQ) * a.G : 0;
          const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
          const float* const nl = lse2 + t * 128;
          int c0 = 0;
          for (; c0 + 32 <= rows; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(base + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 l4 = *reinterpret_cast<const float4*>(nl + c0 + c);
              float2 x = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sl2,
                               make_float2(-l4.x, -l4.y));
              float2 y = ffma2(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])),
                               sl2, make_float2(-l4.z, -l4.w));
              if (masked) {
                if (c0 + c < lo) x.x = -INFINITY;
                if (c0 + c + 1 < lo) x.y = -INFINITY;
                if (c0 + c + 2 < lo) y.x = -INFINITY;
                if (c0 + c + 3 < lo) y.y = -INFINITY;
              }
              sum = fadd2(sum, make_float2(ex2(x.x), ex2(x.y)));
              sum = fadd2(sum, make_float2(ex2(y.x), ex2(y.y)));
            }
          }
          for (; c0 < rows; c0 += 16) {  // the last, partly filled columns
            uint32_t v[16];
            tmem_ld16(base + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < rows && c0 + c >= lo)
                sum.x += ex2(fmaf(__uint_as_float(v[c]), a.scale_log2, -nl[c0 + c]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bars->s_free[wg][uo & 1]));
        }
        if (inside) a.score_out[row + s] = old + (sum.x + sum.y);
        tail.store(a, moved);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->q_empty));
      more = w.next(a);
    }
    tail.rest(a);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_score_d(const ScoreProblem& p, const void* q, const void* k, const float* lse,
                           const int* lengths, const float* score, float* score_out,
                           EncodeTiledFn encode, cudaStream_t stream, const char** why) {
  using Cfg = ScoreCfg<D>;
  const int G = p.Hq / p.Hkv;
  const cuuint64_t E = 2, BG = cuuint64_t(p.B) * p.Hkv;
  ScoreArgs a;
  a.lse = lse;
  a.lengths = lengths;
  a.B = p.B;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.G = G;
  a.N = p.N;
  a.S = p.S;
  a.TQ = min(p.N, 128 / G);
  a.scale_log2 = p.scale * kLog2eScore;
  CUtensorMap mQ, mK;
  cuuint32_t estr[4] = {1, 1, 1, 1};
  bool ok;
  {
    const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(G), cuuint64_t(p.N), BG};
    const cuuint64_t str[3] = {cuuint64_t(p.N) * D * E, cuuint64_t(D) * E,
                               cuuint64_t(G) * p.N * D * E};
    const cuuint32_t box[4] = {64, cuuint32_t(G), cuuint32_t(a.TQ), 1};
    ok = encode(&mQ, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, str, box,
                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  {
    const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(p.S), BG};
    const cuuint64_t str[2] = {cuuint64_t(D) * E, cuuint64_t(p.S) * D * E};
    const cuuint32_t box[3] = {64, 128, 1};
    ok = ok && encode(&mK, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(k), dims, str,
                      box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed for the score's tensors";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(moda_score_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg::kSmemBytes);
  if (e != cudaSuccess) {
    *why = "cudaFuncSetAttribute(max dynamic shared memory) failed";
    return e;
  }
  // up to kScoreMaxTiles row tiles a launch; each further launch adds to the one before
  const int step = kScoreMaxTiles * a.TQ;
  for (int t0 = 0; t0 < p.N && e == cudaSuccess; t0 += step) {
    a.tok0 = t0;
    a.ntok = min(step, p.N - t0);
    a.tiles = (a.ntok + a.TQ - 1) / a.TQ;
    a.stages = min(kScoreMaxStages, Cfg::kOperands / Cfg::kTile - a.tiles);
    a.score = t0 == 0 ? score : score_out;
    a.score_out = score_out;
    a.copy_tail = a.score != score_out;
    moda_score_kernel<D><<<kScoreCtas, kScoreThreads, Cfg::kSmemBytes, stream>>>(mQ, mK, a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) *why = "score launch failed";
  return e;
}

}  // namespace

cudaError_t launch_score(const ScoreProblem& p, const void* q, const void* k, const float* lse,
                         const int* lengths, const float* score, float* score_out,
                         EncodeTiledFn encode, cudaStream_t stream, const char** why) {
  return p.d == 128 ? launch_score_d<128>(p, q, k, lse, lengths, score, score_out, encode, stream,
                                          why)
                    : launch_score_d<64>(p, q, k, lse, lengths, score, score_out, encode, stream,
                                         why);
}

}  // namespace moda
