// moda_tree.cu -- attention of N drafted tokens per sequence over a ragged K/V cache, for
// B200 (sm_100a).
//
// The operator: the MoDA definition (hyper.ai summary of arXiv 2603.15619, section
// "Mixture-of-Depths Attention (MoDA)") for N new tokens per sequence that form a tree: a
// token sees every cached key of its sequence, its ancestors among the new tokens and
// itself, and its own L depth entries, in one joint softmax.  N = 1 is single-token decoding
// over caches of different lengths.  (The pages describe neither.)
//
// What bounds it (one B200, both launches, from a graph): 32 caches of 10K-32K keys, one token each,
// 16 heads in groups of 4, L = 48: 216 to 223 us, 6.6 TB/s; 61 drafts over 2 caches of up to 64K,
// 32 heads, L = 32: 140 to 147 us, 0.7 PFLOP/s and 2.9 TB/s, 11 of them the joining; 4 caches of
// 1000, one token, L = 24: 12.3 us, two launches' latency.
// Each cached K/V byte is needed once and serves the G x N rows of its KV
// head, so up to 128 rows the work is a stream from HBM and the tensor cores have the FLOPs
// to spare; from 128 to 256 rows both take about as long.
//
//   Tiles.  128 rows = TQ tokens x the G heads of one KV head, token-major, as in the
//   forward kernel.  With one tile per KV head the two softmax warpgroups take alternate key
//   blocks, each with its own running maximum, sum and accumulator, merged at the end; with
//   more tiles they take one tile each of a pair, and every block serves both.
//   Steps.  An item (sequence, KV head, tile or pair) is a list of 128-key steps: the depth
//   entries of its tokens (each row sees its own token's), the new tokens (each row sees its
//   ancestors), the cache blocks.  All run through one TMA ring into the tensor cores.
//   Split.  The steps of all items are laid in one line and cut into equal shares, one per
//   CTA, whatever the lengths are: a CTA may end one item and begin the next.  Where whole
//   CTAs per item leave shares hardly longer, each CTA has a part of one item instead
//   (TreePlan).  The lengths
//   are read on the device, so a captured graph follows them.  An item inside one CTA is
//   written directly; the pieces of a cut item go to the workspace as (maximum, sum, fp32
//   accumulator) and a second launch joins them, in the order of the steps.
//   Few rows (template flag kThin: up to 16 rows, d = 128).  One token of a group of 4 fills 4 of
//   the 128 rows, and the idle rest costs power and with it the clock, and the softmax's time.
//   Here the products are transposed, S^T = K Q^T and O^T = V^T P^T, with 16 columns for the
//   rows: an eighth of the products, and a thread holds one key instead of one row.  (Both sides'
//   times are at launch_tree.)
//   Prompts (template flag kPrompt).  The same machinery computes the packed forward of small
//   batches and of groups the forward kernel has no dense depth path for: an item is a tile (or
//   pair) of one sequence's tokens, its steps are the depth entries and the key blocks up to its
//   last token, and a CTA takes up to kPromptItems items one after the other.
//   Rows that must not be read as values (behind a cache's length, unused slots, tile rows no
//   entry fills) are zeroed in shared memory by warp 10 before the tensor cores see them: a
//   weight of zero times an infinity or a NaN is a NaN.
//
// Warp roles (352 threads, one CTA per SM): warps 0-3 and 4-7 softmax, warp 8 TMA (lane 0
// the ring, lane 1 the Q tiles), warp 9 tcgen05 issuer, warp 10 follows the ring and zeroes.
// TMEM columns: S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D,256+2D); few rows: S^T at
// 0 and 32, O^T at 64 and 96, 16 columns each.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "moda_internal.h"
#include "moda_packed.cuh"
#include "sm100.cuh"

namespace moda {

namespace {

constexpr int kTreeThreads = 352;
constexpr int kTreeCtas = 148;      // one CTA per SM of a B200
constexpr int kTreeMinShare = 2;    // steps of the smallest share
constexpr int kTreeRegion = 16384;  // 128 rows x 128 bytes, swizzled
constexpr float kLog2eTree = 1.4426950408889634f;
constexpr float kLn2Tree = 0.6931471805599453f;
constexpr float kTreeRescale = 8.0f;  // log2 units: O is rescaled only past 256x

// kThin: 0, or the rows (4 or 16) of the few-row form.
template <int D, bool kPair, int kThin>
struct TreeCfg {
  static constexpr int kRegions = D / 64;
  static constexpr int kTile = kRegions * kTreeRegion;
  static constexpr int kQTiles = kPair ? 2 : 1;
  static constexpr int kStages = D == 128 ? (kPair ? 5 : 6) : 10;
  // few rows: Q, and P^T of each warpgroup, are 16 rows of 128 bytes a region
  static constexpr int kQRegion = kThin ? 16 * 128 : kTreeRegion;
  static constexpr int kOffP = kRegions * kQRegion;
  static constexpr int kOffKV = kThin ? 3 * kOffP : kQTiles * kTile;
  static constexpr int kOffML = kOffKV + kStages * kTile;  // [2][128] float2
  static constexpr int kOffBar = kOffML + 2 * 128 * 8;
  static constexpr int kSmemBytes = kOffBar + 896;
};

struct TreeArgs {
  __nv_bfloat16* out;
  float* lse;
  float* ws_acc;  // [2 * kTreeCtas][rows][D]
  float* ws_ml;   // [2 * kTreeCtas][rows][2]: m (log2 units), l
  const int* parents;
  const int* lengths;
  int B, Hq, Hkv, G, N, S, L;
  int TQ, JC, ND;  // tokens per tile, depth entries per step, depth steps
  int nit;         // items per sequence: KV heads x tiles (or tile pairs)
  int nt;          // tiles (or tile pairs) per KV head
  int rows;        // rows of a workspace slot
  float scale_log2;
  // packed prompts (kPrompt): N is the row count of the token axis
  const int* cu;  // [nseq + 1] first rows of the sequences
  int nseq, causal;
  long long most;  // upper bound of the number of items
};

__device__ __forceinline__ int tree_length(const TreeArgs& a, int b, bool report = false) {
  const int n = __ldg(a.lengths + b);
  if (report && (n < 0 || n > a.S)) atomicOr(&g_error_word, kErrInternal);
  return min(max(n, 0), a.S);
}
// 128-key steps of each item of sequence b
__device__ __forceinline__ int tree_steps(const TreeArgs& a, int b) {
  return a.ND + 1 + (tree_length(a, b) + 127) / 128;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// How the steps are cut, the same in every CTA and in the joining kernel.
//   parts == 0: all items' steps in one line, `share` of them per CTA;
//   parts != 0: each item by itself into ceil(steps / share) equal parts, one per CTA, with the
//               smallest share for which the parts do not outnumber the CTAs.
// A CTA with two pieces drains the tensor cores, reads out and writes its accumulators twice,
// which costs about as much as kTreeSwitch steps: the second way is taken when its shares are
// at most that much longer.  (16 items of 10 steps: 80 CTAs of 2 steps; 16 of about 420 steps
// each: shares of 49 instead of 46.)
constexpr int kTreeSwitch = 3;
struct TreePlan {
  long long total, share;
  int parts;
  int n0;  // steps of an item of sequence `lane`, the first 32 sequences
  // CTAs of each item of a sequence with n steps per item, and the steps of each of them
  // (parts: the share then fits 32 bits, whose division is much the quicker one)
  __device__ __forceinline__ int ctas(int n) const {
    return int((unsigned(n) + unsigned(share) - 1u) / unsigned(share));
  }
  __device__ __forceinline__ int each(int n) const {
    const unsigned c = ctas(n);
    return int((unsigned(n) + c - 1u) / c);
  }
};

// (all lanes of a warp)
__device__ __forceinline__ TreePlan tree_plan(const TreeArgs& a) {
  const int lane = threadIdx.x & 31;
  TreePlan p;
  p.n0 = lane < a.B ? tree_steps(a, lane) : 0;
  int most = p.n0;
  if (a.B <= 32) {
    p.total = (long long)__reduce_add_sync(0xffffffffu, p.n0) * a.nit;
  } else {
    long long sum = p.n0;
    for (int b = lane + 32; b < a.B; b += 32) {
      const int n = tree_steps(a, b);
      sum += n;
      most = max(most, n);
    }
    p.total = warp_sum(sum) * a.nit;
  }
  p.share = (p.total + kTreeCtas - 1) / kTreeCtas;
  if (p.share < kTreeMinShare) p.share = kTreeMinShare;
  p.parts = 0;
  if ((long long)a.B * a.nit <= kTreeCtas) {
    most = __reduce_max_sync(0xffffffffu, most);
    // (a share of more than p.share + kTreeSwitch is not taken, so the search may end there)
    const int limit = min(int(p.share) + kTreeSwitch, most);
    for (int share = int(p.share); share <= limit; ++share) {
      int c = int((unsigned(p.n0) + unsigned(share) - 1u) / unsigned(share));
      for (int b = lane + 32; b < a.B; b += 32)
        c += int((unsigned(tree_steps(a, b)) + unsigned(share) - 1u) / unsigned(share));
      if (__reduce_add_sync(0xffffffffu, c) * a.nit <= kTreeCtas) {
        p.share = share;
        p.parts = 1;
        break;
      }
    }
  }
  return p;
}

// A CTA's walk over its share: piece by piece, each a run of steps of one item.
struct TreeWalk {
  long long left;      // steps left behind this piece
  int b, it;           // sequence and item of it (prompts: its first row, the KV head)
  int j0, j1, n, len;  // steps [j0, j1) of n, the sequence's cache length
  int t0;              // prompts: the item's first token in its sequence
  __device__ __forceinline__ void clip(const TreeArgs& a) {
    len = tree_length(a, b);
    n = a.ND + 1 + (len + 127) / 128;
    const long long want = left < n - j0 ? left : n - j0;
    j1 = j0 + int(want);
    left -= want;
  }
  __device__ __forceinline__ bool next(const TreeArgs& a) {
    if (left <= 0) return false;
    if (++it == a.nit) {
      it = 0;
      ++b;
    }
    j0 = 0;
    clip(a);
    return true;
  }
};

// Packed prompts: a CTA's items, a tile (or pair of tiles) of one sequence and KV head each.
// Item number c of all, heaviest first (packed_find), goes to the CTAs in turn and back, so
// that none gets the heavier one of every round; the CTA's warps find them side by side.
constexpr int kPromptItems = 32;
struct PromptItem {
  int row0, len, t0, g;  // len < 0: none
};

struct TreeBars {
  uint64_t full[10], empty[10], ready[10];  // ring: landed; released; zeroed where needed
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_half[2], p_full[2];
  uint64_t o_final, o_free;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  TreeWalk walk;                     // this CTA's first piece
  PromptItem items[kPromptItems];    // prompts: all of them
};

// This CTA's first piece (all lanes of a warp); left < 0: there is none.
__device__ __forceinline__ TreeWalk tree_first(const TreeArgs& a, const TreePlan& p) {
  const int lane = threadIdx.x & 31;
  // steps, or with parts CTAs, before this CTA's; counted per item of each sequence
  const long long s = p.parts ? blockIdx.x : p.share * blockIdx.x;
  TreeWalk w;
  w.left = p.parts ? 0 : min(p.share, p.total - s);
  long long before = 0;
  w.b = a.B;
  w.it = 0;
  w.j0 = 0;
  w.t0 = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int steps = b0 == 0 ? p.n0 : (b0 + lane < a.B ? tree_steps(a, b0 + lane) : 0);
    const int mine = p.parts ? p.ctas(steps) : steps;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const bool past = b0 + lane < a.B && (before + incl) * a.nit > s;
    const uint32_t m = __ballot_sync(0xffffffffu, past);
    if (m) {
      const int src = __ffs(m) - 1;
      const int n = __shfl_sync(0xffffffffu, mine, src);
      const int at = __shfl_sync(0xffffffffu, incl, src) - n;
      const long long off = s - (before + at) * a.nit;
      w.b = b0 + src;
      w.it = off >> 32 ? int(off / n) : int(unsigned(off) / unsigned(n));
      w.j0 = int(off - (long long)w.it * n);
      if (p.parts) {
        const int all = __shfl_sync(0xffffffffu, steps, src), each = p.each(all);
        w.left = min(each, all - w.j0 * each);
        w.j0 *= each;
      }
      break;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (w.b == a.B || w.left <= 0)
    w.left = -1;
  else
    w.clip(a);
  return w;
}

// Bits [lo, hi) of word w of a 128-bit row mask.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int w) {
  const int a = min(max(lo - 32 * w, 0), 32), e = min(max(hi - 32 * w, 0), 32);
  const uint32_t below_e = e == 32 ? 0xffffffffu : (1u << e) - 1u;
  const uint32_t below_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
  return below_e & ~below_a;
}

// The new tokens that token i sees: itself and its ancestors, as 128 bits.  A parent must
// come before its child and not be an unused slot; anything else ends the path there and is
// reported.
__device__ __forceinline__ void ancestor_bits(const int* par, int i, uint32_t (&vis)[4]) {
  vis[0] = vis[1] = vis[2] = vis[3] = 0u;
  auto set = [&](int c) {
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (c >> 5 == w) vis[w] |= 1u << (c & 31);
  };
  set(i);
  int cur = i, p = __ldg(par + i);
  if (p == -2) return;
  while (p >= 0 && p < cur) {
    const int up = __ldg(par + p);
    if (up == -2) break;
    set(p);
    cur = p;
    p = up;
  }
  if (p != -1) atomicOr(&g_error_word, kErrInternal);
}

// (all lanes of a warp)
__device__ __forceinline__ PromptItem prompt_item(const TreeArgs& a, int tokens, int round) {
  const int at = round & 1 ? int(gridDim.x) - 1 - int(blockIdx.x) : int(blockIdx.x);
  const int c = round * int(gridDim.x) + at;
  const PackedPiece pc = packed_find(a.cu, a.nseq, a.N, tokens, c / a.Hkv);
  return PromptItem{pc.first, pc.found ? pc.len : -1, pc.p * tokens, c % a.Hkv};
}

// Where an item's data lie.
struct TreeItem {
  int g, bg;     // KV head; batch index of the tensor maps
  int tok, key;  // rows of the first query token and of the first key
  int t0, ntok;  // first token of the item among its sequence's ntok
};

// OR of a predicate over the n threads of a named barrier.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(uint32_t(p))
      : "memory");
  return r != 0;
}

// The softmax warpgroups of the few-row form (N tokens x G heads <= kRows rows, one tile).  A
// thread is a key of the block: its lane of S^T holds that key's score of every row, so the
// exponentials are kRows a thread instead of 128 for each of a few rows, and the products are
// an eighth of the full tile's.  Each row keeps a reference m that all threads of the warpgroup
// share; it moves only when a score exceeds it by 2^kTreeRescale, which one barrier with an OR
// finds out, and l is summed per thread until the piece's end.
// P is rounded to bf16 as in the full form.
//   scratch: [2 warpgroups][4 warps][16] partial results, [2][16] (m, l), [2][16] ancestor bits
template <int D, int kRows>
__device__ __forceinline__ void thin_softmax(const TreeArgs& a, TreeBars* bars,
                                             const TreeWalk& walk0, uint32_t tmem, uint32_t sp,
                                             float* scratch) {
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  volatile int* abort_flag = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wg = warp >> 2, key = threadIdx.x & 127;  // key of the block; head dimension of O^T
  const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
  const uint32_t tS = tmem + lane_base + wg * 32, tO = tmem + lane_base + 64 + wg * 32;
  float* const red = scratch + wg * 64;                                // [4][16]
  float2* const ml = reinterpret_cast<float2*>(scratch + 128);        // [2][16]
  uint32_t* const anc = reinterpret_cast<uint32_t*>(scratch + 192) + wg * 16;
  const int rows = a.N * a.G;
  const uint32_t all = (1u << rows) - 1u;  // (rows <= 16)
  const uint32_t group = (1u << a.G) - 1u;
  // this key's place in P^T: row r is 128 bytes further, its 16-byte chunk swizzled by r % 8
  const uint32_t pcol = sp + uint32_t(key >> 6) * (16 * 128) + uint32_t(key & 7) * 2;
  const uint32_t chunk = uint32_t(key & 63) >> 3;
  TreeWalk w = walk0;
  int u = 0, pc = 0;
  bool more = true;
  for (; more; ++pc) {
    const int g = w.it;  // (one tile per KV head)
    const int* par = a.parents + (long long)w.b * a.N;
    float m[kRows], l[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
    bool has_o = false;
    for (int j = w.j0; j < w.j1; ++j) {
      if (((u + j - w.j0) & 1) != wg) continue;
      const int unit = u + j - w.j0;
      uint32_t see;  // rows that see this key
      if (j < a.ND) {
        const int tok = key / a.JC, e = j * a.JC + key - tok * a.JC;
        see = tok < a.N && e < a.L ? group << (tok * a.G) : 0u;
      } else if (j == a.ND) {
        if (key < a.N) {
          uint32_t vis[4];
          ancestor_bits(par, key, vis);
          anc[key] = vis[0];
        }
        named_bar_sync(2 + wg, 128);
        see = 0u;
        if (key < a.N)
          for (int t = 0; t < a.N; ++t)
            if ((anc[t] >> key) & 1u) see |= group << (t * a.G);
      } else {
        see = (j - a.ND - 1) * 128 + key < w.len ? 0xffffffffu : 0u;
      }
      see &= all;
      mbar_wait(bar(bars->s_full[wg]), (unit >> 1) & 1, abort_flag);
      tc_fence_after();
      uint32_t sv[16];
      tmem_ld16(tS, sv);
      tmem_wait_ld();
      float x[kRows];
      bool over = false;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        x[r] = (see >> r) & 1u ? __uint_as_float(sv[r]) * a.scale_log2 : -INFINITY;
        over = over || x[r] > m[r] + kTreeRescale;
      }
      if (named_bar_or(2 + wg, 128, over)) {
        // new references: the block's maxima
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float v = x[r];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
          if (lane == 0) red[(warp & 3) * 16 + r] = v;
        }
        named_bar_sync(2 + wg, 128);
        float f[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) f[r] = 1.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float n = fmaxf(fmaxf(fmaxf(red[r], red[16 + r]), fmaxf(red[32 + r], red[48 + r])),
                                m[r]);
          f[r] = ex2(m[r] - (n == -INFINITY ? 0.f : n));
          m[r] = n;
          l[r] *= f[r];
        }
        if (has_o) {  // every product of this warpgroup so far has finished (see the full form)
          uint32_t o[16];
          tmem_ld16(tO, o);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < 16; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r]);
          tmem_st16(tO, o);
          tmem_wait_st();
        }
      }
      has_o = true;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float p = ex2(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
        l[r] += p;
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(pcol + r * 128 + ((chunk ^ (r & 7)) << 4)),
                     "h"(bf16_bits(p))
                     : "memory");
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->p_full[wg]));
    }
    // ---- the piece's end: sums over the keys, both warpgroups' states merged
    const int units = w.j1 - w.j0;
    named_bar_sync(2 + wg, 128);  // (red's last readers)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
      if (lane == 0) red[(warp & 3) * 16 + r] = l[r];
    }
    named_bar_sync(2 + wg, 128);
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (key == r)
        ml[wg * 16 + r] = make_float2(m[r], red[r] + red[16 + r] + red[32 + r] + red[48 + r]);
    mbar_wait(bar(bars->o_final), pc & 1, abort_flag);
    tc_fence_after();
    named_bar_sync(1, 256);
    const bool whole = w.j0 == 0 && w.j1 == w.n;
    const bool use0 = units > 1 || (u & 1) == 0, use1 = units > 1 || (u & 1) == 1;
    uint32_t o0[16], o1[16];
    tmem_ld16(tmem + lane_base + 64, o0);
    tmem_ld16(tmem + lane_base + 96, o1);
    tmem_wait_ld();
    const int slot = 2 * int(blockIdx.x) + (pc > 0 ? 1 : 0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if ((r & 1) != wg || r >= rows) continue;
      const float2 x = ml[r], y = ml[16 + r];
      const float M = fmaxf(x.x, y.x), mu = M == -INFINITY ? 0.f : M;
      const float f0 = ex2(x.x - mu), f1 = ex2(y.x - mu);
      const float L = x.y * f0 + y.y * f1;
      const float v = (use0 ? f0 * __uint_as_float(o0[r]) : 0.f) +
                      (use1 ? f1 * __uint_as_float(o1[r]) : 0.f);
      const int tok = r / a.G, hl = r - tok * a.G;
      if (whole) {
        const long long row = ((long long)w.b * a.Hq + g * a.G + hl) * a.N + tok;
        const bool none = L == 0.f || __ldg(par + tok) == -2;
        a.out[row * D + key] = __float2bfloat16_rn(none ? 0.f : v / L);
        if (key == 0) a.lse[row] = none ? -INFINITY : (M + __log2f(L)) * kLn2Tree;
      } else {
        const long long wrow = (long long)slot * a.rows + r;
        a.ws_acc[wrow * D + key] = v;
        if (key == 0) *reinterpret_cast<float2*>(a.ws_ml + wrow * 2) = make_float2(M, L);
      }
    }
    named_bar_sync(1, 256);  // (the next piece writes the scratch again)
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(bars->o_free));
    u += units;
    more = w.next(a);
  }
}

template <int D, bool kPair, bool kPrompt, int kThin>
__global__ void __launch_bounds__(kTreeThreads, 1)
    moda_tree_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmKT,
                     const __grid_constant__ CUtensorMap tmVT,
                     const __grid_constant__ CUtensorMap tmKD,
                     const __grid_constant__ CUtensorMap tmVD, const TreeArgs a) {
  using Cfg = TreeCfg<D, kPair, kThin>;
  static_assert(!kThin || (D == 128 && !kPair && !kPrompt), "the few-row form");
  constexpr int NS = Cfg::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  // the joining grid may be scheduled now: it waits for this grid's completion itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the swizzled layouts need a 1024-byte aligned base, and there is no room to realign
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_error_word, kErrInternal);
    return;
  }
  const uint32_t s0 = smem_u32(smem);
  auto sQ = [&](int t) { return s0 + uint32_t(t) * Cfg::kTile; };
  auto sP = [&](int wg) { return s0 + uint32_t(wg + 1) * Cfg::kOffP; };  // (few rows)
  auto sKV = [&](int s) { return s0 + Cfg::kOffKV + uint32_t(s) * Cfg::kTile; };
  float2* const ml = reinterpret_cast<float2*>(smem + Cfg::kOffML);
  TreeBars* bars = reinterpret_cast<TreeBars*>(smem + Cfg::kOffBar);
  static_assert(sizeof(TreeBars) <= 896, "barrier space");
  volatile int* abort_flag = &bars->abort;
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool no_loads = false;
  if (warp == 8) {
    if (lane < 7) {
      const CUtensorMap* maps[7] = {&tmQ, &tmK, &tmV, &tmKT, &tmVT, &tmKD, &tmVD};
      tma_prefetch_desc(maps[lane]);
    }
    // test-only fault: issue no loads, so that every wait for them runs out
    no_loads = g_device_fault == kFaultForwardNoLoads;
  }

  // warp 0 finds this CTA's work (prompts: every warp an item) while others set up the barriers
  // and the tensor memory
  if constexpr (kPrompt) {
    for (int r = warp; r < kPromptItems; r += kTreeThreads / 32) {
      if ((long long)r * gridDim.x < a.most) {
        const PromptItem item = prompt_item(a, a.TQ * Cfg::kQTiles, r);
        if (lane == 0) bars->items[r] = item;
      } else if (lane == 0) {
        bars->items[r].len = -1;
      }
    }
  } else if (warp == 0) {
    const TreeWalk w = tree_first(a, tree_plan(a));
    if (blockIdx.x == 0)
      for (int b = lane; b < a.B; b += 32) tree_length(a, b, true);
    if (lane == 0) bars->walk = w;
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(bars->full[s]), 1);
      mbar_init(bar(bars->empty[s]), 2);  // the products that read it, and warp 10
      mbar_init(bar(bars->ready[s]), 1);
    }
    mbar_init(bar(bars->q_full), 1);
    mbar_init(bar(bars->q_empty), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(bars->s_full[t]), 1);
      mbar_init(bar(bars->p_half[t]), 4);  // one arrival a warp
      mbar_init(bar(bars->p_full[t]), 4);
    }
    mbar_init(bar(bars->o_final), 1);
    mbar_init(bar(bars->o_free), 8);
    mbar_init(bar(bars->drain), 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  // (Q rows past TQ*G never receive data: whatever lies there only makes rows of S, P and O
  // that nothing reads)
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // prompts: item `k` of this CTA as a piece; `left` counts the items behind it
  auto load_item = [&](TreeWalk& w, int k) {
    const PromptItem t = bars->items[k];
    w.b = t.row0;
    w.it = t.g;
    w.len = t.len;
    w.t0 = t.t0;
    w.j0 = 0;
    w.j1 = w.n =
        a.ND + ((a.causal ? min(t.len, t.t0 + a.TQ * Cfg::kQTiles) : t.len) + 127) / 128;
  };
  TreeWalk walk0;
  int items = 0;  // prompts: this CTA's items
  if constexpr (kPrompt) {
    while (items < kPromptItems && bars->items[items].len >= 0) ++items;
    walk0.left = items - 1;
    if (items > 0) load_item(walk0, 0);
  } else {
    walk0 = bars->walk;
  }
  auto next_piece = [&](TreeWalk& w) {
    if constexpr (kPrompt) {
      if (w.left <= 0) return false;
      --w.left;
      load_item(w, items - 1 - int(w.left));
      return true;
    } else {
      return w.next(a);
    }
  };
  if (walk0.left < 0) {  // no work for this CTA
    if (warp == 9) tmem_dealloc(tmem, 512);
    return;
  }
  constexpr int kOwn = kPrompt ? 0 : 1;  // steps of the new tokens' own keys
  auto item_of = [&](const TreeWalk& w) {
    TreeItem t;
    if constexpr (kPrompt) {
      t = TreeItem{w.it, w.it, w.b + w.t0, w.b, w.t0, w.len};
    } else {
      const int g = w.it / a.nt, t0 = (w.it - g * a.nt) * a.TQ * Cfg::kQTiles;
      t = TreeItem{g, w.b * a.Hkv + g, t0, 0, t0, a.N};
    }
    return t;
  };

  // Ring entries of a step: keys then values; a depth step of a tile pair has both tiles'
  // keys, then both tiles' values.
  auto wide = [&](int j) { return kPair && j < a.ND; };

  if (warp == 8) {
    // ------------------------------------------------------------ TMA
    if (lane == 0 && !no_loads) {
      int e = 0;
      TreeWalk w = walk0;
      bool more = true;
      while (more && !*abort_flag) {
        const TreeItem item = item_of(w);
        for (int j = w.j0; j < w.j1; ++j) {
          const int ne = wide(j) ? 4 : 2;
          bool ok = true;
          for (int u = 0; u < ne; ++u, ++e) {
            const int s = e % NS;
            if (e >= NS && !mbar_wait(bar(bars->empty[s]), ((e / NS) - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            const bool values = ne == 4 ? u >= 2 : u == 1;
            const uint32_t full = bar(bars->full[s]);
            if (j < a.ND) {
              mbar_expect_tx(full, uint32_t(Cfg::kRegions) * 128u * a.TQ * a.JC);
              for (int rg = 0; rg < Cfg::kRegions; ++rg)
                tma_load_4d(sKV(s) + rg * kTreeRegion, values ? &tmVD : &tmKD, full, rg * 64,
                            j * a.JC, item.tok + (ne == 4 && (u & 1) ? a.TQ : 0), item.bg);
            } else {
              mbar_expect_tx(full, Cfg::kTile);
              const bool tree = !kPrompt && j == a.ND;
              const CUtensorMap* map = tree ? (values ? &tmVT : &tmKT) : (values ? &tmV : &tmK);
              for (int rg = 0; rg < Cfg::kRegions; ++rg)
                tma_load_3d(sKV(s) + rg * kTreeRegion, map, full, rg * 64,
                            tree ? 0 : item.key + (j - a.ND - kOwn) * 128, item.bg);
            }
          }
          if (!ok) break;
        }
        more = next_piece(w);
      }
      if (*abort_flag)  // abort path: what was issued still lands; wait for it before exit
        for (int i = e > NS ? e - NS : 0; i < e; ++i)
          mbar_wait_drain(bar(bars->full[i % NS]), (i / NS) & 1);
    } else if (lane == 1 && !no_loads) {
      TreeWalk w = walk0;
      int pc = 0;  // piece
      bool more = true;
      for (; more; ++pc, more = next_piece(w)) {
        if (pc > 0 && !mbar_wait(bar(bars->q_empty), (pc - 1) & 1, abort_flag)) break;
        const TreeItem item = item_of(w);
        mbar_expect_tx(bar(bars->q_full),
                       uint32_t(Cfg::kQTiles * Cfg::kRegions) * 128u * a.G * a.TQ);
        for (int t = 0; t < Cfg::kQTiles; ++t)
          for (int rg = 0; rg < Cfg::kRegions; ++rg)
            tma_load_4d(sQ(t) + rg * Cfg::kQRegion, &tmQ, bar(bars->q_full), rg * 64, 0,
                        item.tok + t * a.TQ, item.bg);
      }
      if (*abort_flag && pc > 0) mbar_wait_drain(bar(bars->q_full), (pc - 1) & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ tcgen05 issuer
    // Units: (step) with the warpgroup alternating, or (step, tile) for a pair.  Order:
    // S(0) S(1) { PV(u) S(u+2) }: while one warpgroup turns its S into P the tensor cores
    // work for the other.  S(u+2) overwrites P(u), which PV(u), issued before it, has read.
    if (elect_one()) {
      // few rows: S^T = K Q^T (keys x rows), O^T = V^T P^T (d x rows; V is MN-major)
      constexpr uint32_t idesc_s = make_idesc_bf16(128, kThin ? 16 : 128, 0, 0);
      constexpr uint32_t idesc_o =
          kThin ? make_idesc_bf16(128, 16, 1, 0) : make_idesc_bf16(128, D, 0, 1);
      struct Cursor {
        TreeWalk w;
        int j, half, e, pc, u;  // step, tile of the pair, ring entry, piece, unit
        bool live;
      };
      Cursor cs{walk0, walk0.j0, 0, 0, 0, 0, true};
      Cursor cp = cs;
      auto advance = [&](Cursor& c) {
        ++c.u;
        if (kPair && c.half == 0) {
          c.half = 1;
          return;
        }
        c.half = 0;
        c.e += wide(c.j) ? 4 : 2;
        if (++c.j == c.w.j1) {
          c.live = next_piece(c.w);
          c.j = c.w.j0;
          ++c.pc;
        }
      };
      auto issue_s = [&](Cursor& c) {
        const int wg = c.u & 1;
        const bool two = wide(c.j);
        const int e = c.e + (two ? c.half : 0);
        if (c.j == c.w.j0 && c.half == 0) mbar_wait(bar(bars->q_full), c.pc & 1, abort_flag);
        mbar_wait(bar(bars->full[e % NS]), (e / NS) & 1, abort_flag);
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks / 4) * kTreeRegion + (ks % 4) * 32;
          if constexpr (kThin)
            mma_ss(tmem + wg * 32, make_sdesc_sw128(sKV(e % NS) + off, 16, 1024),
                   make_sdesc_sw128(sQ(0) + (ks / 4) * Cfg::kQRegion + (ks % 4) * 32, 16, 1024),
                   idesc_s, ks > 0 ? 1u : 0u);
          else
            mma_ss(tmem + wg * 128, make_sdesc_sw128(sQ(kPair ? c.half : 0) + off, 16, 1024),
                   make_sdesc_sw128(sKV(e % NS) + off, 16, 1024), idesc_s, ks > 0 ? 1u : 0u);
        }
        tc_commit(bar(bars->s_full[wg]));
        if (!kPair || two || c.half == 1) tc_commit(bar(bars->empty[e % NS]));
        if (c.j == c.w.j1 - 1 && (!kPair || c.half == 1)) tc_commit(bar(bars->q_empty));
        advance(c);
      };
      auto issue_pv = [&](Cursor& c) {
        const int wg = c.u & 1;
        const bool two = wide(c.j);
        const int e = c.e + (two ? 2 + c.half : 1);
        mbar_wait(bar(bars->ready[e % NS]), (e / NS) & 1, abort_flag);
        // the accumulators of the piece before have been read
        if (c.pc > 0 && c.j == c.w.j0 && c.half == 0)
          mbar_wait(bar(bars->o_free), (c.pc - 1) & 1, abort_flag);
        // this warpgroup's first product of the piece overwrites its accumulator
        const bool fresh = kPair ? c.j == c.w.j0 : c.j - c.w.j0 < 2;
        if constexpr (kThin) {
          mbar_wait(bar(bars->p_full[wg]), (c.u >> 1) & 1, abort_flag);
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ss(tmem + 64 + wg * 32,
                   make_sdesc_sw128(sKV(e % NS) + ks * 2048, kTreeRegion, 1024),
                   make_sdesc_sw128(sP(wg) + (ks / 4) * Cfg::kQRegion + (ks % 4) * 32, 16, 1024),
                   idesc_o, (ks > 0 || !fresh) ? 1u : 0u);
        } else {
          // keys [0, 64) as soon as their P is in, then the rest
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            mbar_wait(bar(half ? bars->p_full[wg] : bars->p_half[wg]), (c.u >> 1) & 1,
                      abort_flag);
            tc_fence_after();
#pragma unroll
            for (int kq = 0; kq < 4; ++kq) {
              const int ks = half * 4 + kq;
              mma_ts(tmem + 256 + wg * D, tmem + wg * 128 + ks * 8,
                     make_sdesc_sw128(sKV(e % NS) + ks * 2048, kTreeRegion, 1024), idesc_o,
                     (ks > 0 || !fresh) ? 1u : 0u);
            }
          }
        }
        if (!kPair || two || c.half == 1) tc_commit(bar(bars->empty[e % NS]));
        if (c.j == c.w.j1 - 1 && (!kPair || c.half == 1)) tc_commit(bar(bars->o_final));
        advance(c);
      };
      issue_s(cs);
      if (cs.live) issue_s(cs);
      while (cp.live && !*abort_flag) {
        issue_pv(cp);
        if (cs.live) issue_s(cs);
      }
      if (*abort_flag) {
        tc_commit(bar(bars->drain));
        mbar_wait_drain(bar(bars->drain), 0);
      }
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ rows that are no values
    // zeroes the `each` rows of every unused slot among the new tokens [t0, t1)
    auto zero_unused = [&](uint32_t tile, const int* par, int t0, int t1, int each) {
      for (int t = t0; t < t1; t += 32) {
        uint32_t unused =
            __ballot_sync(0xffffffffu, t + lane < t1 && __ldg(par + t + lane) == -2);
        for (; unused; unused &= unused - 1) {
          const int i = t - t0 + __ffs(unused) - 1;
          zero_tile_rows(tile, Cfg::kRegions, i * each, (i + 1) * each);
        }
      }
    };
    int e = 0;
    TreeWalk w = walk0;
    bool more = true, stop = false;
    while (more && !stop) {
      const TreeItem item = item_of(w);
      const int* par = kPrompt ? nullptr : a.parents + (long long)w.b * a.N;
      for (int j = w.j0; j < w.j1 && !stop; ++j) {
        const int ne = wide(j) ? 4 : 2;
        for (int u = 0; u < ne; ++u, ++e) {
          const int s = e % NS;
          stop = !__all_sync(0xffffffffu, mbar_wait(bar(bars->full[s]), (e / NS) & 1, abort_flag));
          if (stop) break;
          if (ne == 4 ? u >= 2 : u == 1) {
            if (j < a.ND) {
              // rows that no entry of a token fills, and the entries of unused slots
              const int t0 = item.t0 + (ne == 4 && (u & 1) ? a.TQ : 0);
              const int toks = min(a.TQ, max(0, item.ntok - t0));
              zero_tile_rows(sKV(s), Cfg::kRegions, toks * a.JC, 128);
              if constexpr (!kPrompt) zero_unused(sKV(s), par, t0, t0 + toks, a.JC);
            } else if (!kPrompt && j == a.ND) {
              zero_unused(sKV(s), par, 0, a.N, 1);
            } else {
              const int inside = w.len - (j - a.ND - kOwn) * 128;
              if (inside < 128) zero_tile_rows(sKV(s), Cfg::kRegions, inside, 128);
            }
          }
          publish_rows(bar(bars->ready[s]));
          if (lane == 0) mbar_arrive(bar(bars->empty[s]));
        }
      }
      more = next_piece(w);
    }
    __syncwarp();
  } else if constexpr (kThin != 0) {
    thin_softmax<D, kThin>(a, bars, walk0, tmem, sP(warp >> 2),
                           reinterpret_cast<float*>(smem + Cfg::kOffML));
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int wg = warp >> 2;
    const int r = threadIdx.x & 127;  // tile row
    const int tok = r / a.G, hl = r - tok * a.G;
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + wg * 128;
    const uint32_t tO = tmem + lane_base + 256 + wg * D;
    float m = -INFINITY, l = 0.f;  // this row's running maximum (log2 units) and sum
    bool has_o = false;
    // O is rescaled before the first half of P is published, since that half's product may
    // start at once.  (Every product of this warpgroup so far was issued before its S and has
    // finished.)
    auto rescale_o = [&](bool grow, float alpha) {
      if (__any_sync(0xffffffffu, grow && has_o)) {
        const float f = grow ? alpha : 1.f;
#pragma unroll 1
        for (int cc = 0; cc < D / 16; ++cc) {
          uint32_t o[16];
          tmem_ld16(tO + cc * 16, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st16(tO + cc * 16, o);
        }
      }
      has_o = true;
    };
    auto publish = [&](uint64_t& b) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    // P enters its product as bf16 (the products' operand type); l sums it unrounded.  Each
    // weight is then off by at most 2^-8 of itself, independently: over the measured cases out
    // differs from 64 bits by 2.1e-3 to 2.4e-3 of its size, where rounding out alone gives 1.7e-3.
    // A second product with what the rounding left would bring that back, for twice the work with V.
    // All 128 keys of a step.  Without a mask (a block inside the cache) every fourth pair of
    // exponentials is computed on the FMA pipe, as in the forward.
    auto full_step = [&](auto masked_c, const uint32_t (&vis)[4]) {
      constexpr bool kMasked = decltype(masked_c)::value;
      uint32_t s[128];
      tmem_ld32(tS + 0, &s[0]);
      tmem_ld32(tS + 32, &s[32]);
      tmem_ld32(tS + 64, &s[64]);
      tmem_ld32(tS + 96, &s[96]);
      tmem_wait_ld();
      if constexpr (kMasked) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (!((vis[c >> 5] >> (c & 31)) & 1u)) s[c] = __float_as_uint(-INFINITY);
      }
      float mx = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int c = 0; c < 128; c += 4) {
        mx = fmax3(mx, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        mx1 = fmax3(mx1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
      }
      const float m_cand = fmaxf(m, fmaxf(mx, mx1) * a.scale_log2);
      const bool grow = m_cand > m + kTreeRescale;
      const float m_new = grow ? m_cand : m;
      const float m_use = kMasked && m_new == -INFINITY ? 0.f : m_new;
      const float alpha = ex2(m - m_use);
      const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
      const float2 nm2 = make_float2(-m_use, -m_use);
      float2 ps = make_float2(0.f, 0.f);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 x = ffma2(make_float2(__uint_as_float(s[half * 64 + c]),
                                             __uint_as_float(s[half * 64 + c + 1])),
                                 sl2, nm2);
          const float2 p = !kMasked && (c / 2) % kExpFmaPeriod == kExpFmaPeriod - 1
                               ? exp2_fma2(x)
                               : make_float2(ex2(x.x), ex2(x.y));
          ps = fadd2(ps, p);
          pk[c / 2] = pack_bf16x2(p.x, p.y);
        }
        if (half == 0) rescale_o(grow, alpha);
        tmem_st32(tS + half * 32, pk);
        publish(half ? bars->p_full[wg] : bars->p_half[wg]);
      }
      l = l * alpha + (ps.x + ps.y);
      m = m_new;
    };
    // Keys of kW chunks of 32 from chunk q0 on (0 <= q0 <= 4 - kW), the only ones that some row
    // of the warp sees; P is zero elsewhere.
    auto window_step = [&](auto width_c, int q0, const uint32_t (&vis)[4]) {
      constexpr int kW = decltype(width_c)::value;
      uint32_t see[kW];
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        const int q = q0 + i;
        see[i] = q < 2 ? (q ? vis[1] : vis[0]) : (q > 2 ? vis[3] : vis[2]);
      }
      uint32_t s[32 * kW];
#pragma unroll
      for (int i = 0; i < kW; ++i) tmem_ld32(tS + 32 * (q0 + i), &s[32 * i]);
      tmem_wait_ld();
      float mx = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int c = 0; c < 32 * kW; ++c)
        if (!((see[c / 32] >> (c & 31)) & 1u)) s[c] = __float_as_uint(-INFINITY);
#pragma unroll
      for (int c = 0; c < 32 * kW; c += 4) {
        mx = fmax3(mx, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        mx1 = fmax3(mx1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
      }
      const float m_cand = fmaxf(m, fmaxf(mx, mx1) * a.scale_log2);
      const bool grow = m_cand > m + kTreeRescale;
      const float m_new = grow ? m_cand : m;
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = ex2(m - m_use);
      const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
      const float2 nm2 = make_float2(-m_use, -m_use);
      float2 ps = make_float2(0.f, 0.f);
      uint32_t pk[16 * kW];
#pragma unroll
      for (int c = 0; c < 32 * kW; c += 2) {
        const float2 x =
            ffma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2, nm2);
        const float2 p = make_float2(ex2(x.x), ex2(x.y));
        ps = fadd2(ps, p);
        pk[c / 2] = pack_bf16x2(p.x, p.y);
      }
      rescale_o(grow, alpha);
      uint32_t zero[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) zero[c] = 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q < q0 || q >= q0 + kW)
          tmem_st16(tS + 16 * q, zero);
        else if (kW == 1 || q == q0)
          tmem_st16(tS + 16 * q, &pk[0]);
        else
          tmem_st16(tS + 16 * q, &pk[16 * (kW - 1)]);
        if (q & 1) publish(q == 3 ? bars->p_full[wg] : bars->p_half[wg]);
      }
      l = l * alpha + (ps.x + ps.y);
      m = m_new;
    };
    // Any other step.  Most let a warp's rows see only keys inside 32 or 64 columns (a token's
    // depth entries, a small tree, the edge of a block): those alone are loaded and
    // exponentiated.
    auto masked_step = [&](const TreeWalk& w, int j, int ti, const int* par) {
      (void)par;
      uint32_t vis[4];
      if (j < a.ND) {
        const int lo = tok * a.JC, nv = min(a.JC, a.L - j * a.JC);
#pragma unroll
        for (int q = 0; q < 4; ++q) vis[q] = range_bits(lo, lo + nv, q);
      } else if (!kPrompt && j == a.ND) {
        vis[0] = vis[1] = vis[2] = vis[3] = 0u;
        if (tok < a.TQ && ti < a.N) ancestor_bits(par, ti, vis);
      } else {
        // keys of the block inside the sequence, and of a prompt (causal) up to the token
        const int end = kPrompt && a.causal ? min(ti + 1, w.len) : w.len;
        const int inside = end - (j - a.ND - kOwn) * 128;
#pragma unroll
        for (int q = 0; q < 4; ++q) vis[q] = range_bits(0, inside, q);
      }
      int q0 = 4, q1 = 0;  // chunks of 32 keys [q0, q1) hold all that the warp's rows see
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (__any_sync(0xffffffffu, vis[q] != 0u)) {
          q0 = min(q0, q);
          q1 = q + 1;
        }
      if (q1 - q0 > 2) {
        full_step(std::true_type{}, vis);
        return;
      }
      if (q1 - q0 == 2)
        window_step(std::integral_constant<int, 2>{}, q0, vis);
      else
        window_step(std::integral_constant<int, 1>{}, min(q0, 3), vis);
    };
    const uint32_t no_mask[4] = {0u, 0u, 0u, 0u};
    TreeWalk w = walk0;
    int u = 0;  // unit
    int pc = 0;
    bool more = true;
    // (no early way out: the warpgroups meet at named barriers; once a wait has failed every
    // later one returns at once)
    for (; more; ++pc) {
      const TreeItem item = item_of(w);
      const int t0 = item.t0 + (kPair ? wg * a.TQ : 0);
      const int ti = t0 + tok;  // this row's token
      const int* par = kPrompt ? nullptr : a.parents + (long long)w.b * a.N;
      const bool valid = tok < a.TQ && ti < item.ntok;
      // warps without a row in the tile only keep the barriers in step
      const bool active = (warp & 3) * 32 < min(a.TQ, item.ntok - t0) * a.G;
      // keys that every row of the tile sees
      const int sure = kPrompt && a.causal ? min(t0 + 1, w.len) : w.len;
      m = -INFINITY;
      l = 0.f;
      has_o = false;
      for (int j = w.j0; j < w.j1; ++j) {
        if (!kPair && ((u + j - w.j0) & 1) != wg) continue;
        const int unit = kPair ? u + 2 * (j - w.j0) + wg : u + j - w.j0;
        mbar_wait(bar(bars->s_full[wg]), (unit >> 1) & 1, abort_flag);
        tc_fence_after();
        if (active) {
          const int kbase = (j - a.ND - kOwn) * 128;
          if (j >= a.ND + kOwn && kbase + 128 <= sure)
            full_step(std::false_type{}, no_mask);
          else
            masked_step(w, j, ti, par);
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(bars->p_half[wg]));
            mbar_arrive(bar(bars->p_full[wg]));
          }
        }
      }
      // ---- the piece's end
      const int units = (w.j1 - w.j0) * Cfg::kQTiles;
      mbar_wait(bar(bars->o_final), pc & 1, abort_flag);
      tc_fence_after();
      const bool whole = kPrompt || (w.j0 == 0 && w.j1 == w.n);
      float m_all = m, l_all = l, f0 = 1.f, f1 = 0.f;
      constexpr int kCols = kPair ? D : D / 2;  // columns this thread writes
      const int col0 = kPair ? 0 : wg * kCols;
      if constexpr (!kPair) {
        ml[wg * 128 + r] = make_float2(m, l);
        named_bar_sync(1, 256);
        const float2 x = ml[r], y = ml[128 + r];
        named_bar_sync(1, 256);  // (the next piece writes them again)
        m_all = fmaxf(x.x, y.x);
        const float mu = m_all == -INFINITY ? 0.f : m_all;
        f0 = ex2(x.x - mu);
        f1 = ex2(y.x - mu);
        l_all = x.y * f0 + y.y * f1;
      }
      // which accumulators hold anything: with a single unit only its warpgroup's does
      const bool use0 = kPair || units > 1 || (u & 1) == 0;
      const bool use1 = !kPair && (units > 1 || (u & 1) == 1);
      if (active) {
        // an unused slot: zeros, -inf
        bool dead = false;
        if constexpr (!kPrompt) dead = valid && __ldg(par + ti) == -2;
        // (l = 0 only for a row that saw nothing)
        const float inv = whole ? ((dead || l_all == 0.f) ? 0.f : 1.f / l_all) : 1.f;
        const long long row =
            ((long long)(kPrompt ? 0 : w.b) * a.Hq + item.g * a.G + hl) * a.N +
            (kPrompt ? item.key : 0) + (valid ? ti : 0);
        // a cut item's first piece in a CTA's share has the share's first slot
        const int slot = 2 * int(blockIdx.x) + (pc > 0 ? 1 : 0);
        const long long wrow = (long long)slot * a.rows + (kPair ? wg * a.TQ * a.G : 0) + r;
#pragma unroll
        for (int cc = 0; cc < kCols / 32; ++cc) {
          uint32_t o[32], o1[32];
          if constexpr (kPair) {
            tmem_ld32(tO + cc * 32, o);
          } else {
            tmem_ld32(tmem + lane_base + 256 + col0 + cc * 32, o);
            tmem_ld32(tmem + lane_base + 256 + D + col0 + cc * 32, o1);
          }
          tmem_wait_ld();
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if constexpr (kPair) {
              v[i] = __uint_as_float(o[i]);
            } else {
              v[i] = (use0 ? f0 * __uint_as_float(o[i]) : 0.f) +
                     (use1 ? f1 * __uint_as_float(o1[i]) : 0.f);
            }
          }
          if (valid) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + col0 + cc * 32);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = inv == 0.f ? 0.f : v[q * 8 + i];
                dst[q] = pack8(x, inv);
              }
            } else {
              // 32 bytes a store: a row's columns come from one thread, so that a narrower
              // store would fill its sectors in two goes
              float* const dst = a.ws_acc + wrow * D + col0 + cc * 32;
#pragma unroll
              for (int q = 0; q < 4; ++q) stg256(dst + 8 * q, &v[8 * q]);
            }
          }
        }
        if (valid && (kPair || wg == 0)) {
          if (whole)
            a.lse[row] = (dead || l_all == 0.f) ? -INFINITY : (m_all + __log2f(l_all)) * kLn2Tree;
          else
            *reinterpret_cast<float2*>(a.ws_ml + wrow * 2) = make_float2(m_all, l_all);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->o_free));
      u += units;
      more = next_piece(w);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the items that were cut: one warp per row (sequence, head, token), a
// lane for every 32nd group of four columns.  Rows of items inside one CTA's share were
// written by it.
template <int D>
__global__ void __launch_bounds__(256) moda_tree_join_kernel(const TreeArgs a, int qtiles) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.Hq * a.N) return;
  const TreePlan plan = tree_plan(a);
  const int i = int(row % a.N);
  const int h = int(row / a.N % a.Hq), b = int(row / a.N / a.Hq);
  const int g = h / a.G, hl = h - g * a.G;
  const int n = tree_steps(a, b);
  const int tile = i / a.TQ, item = g * a.nt + tile / qtiles;
  long long before = 0;
  for (int x = lane; x < b; x += 32) {
    const int m = x < 32 ? plan.n0 : tree_steps(a, x);
    before += plan.parts ? plan.ctas(m) : m;
  }
  before = warp_sum(before) * a.nit;
  const int each = plan.parts ? plan.ctas(n) : n;
  const long long s = before + (long long)item * each;
  int c0, c1;  // the CTAs that hold this item
  if (plan.parts) {
    c0 = int(s);
    // (its parts that are not empty)
    c1 = c0 + (n + plan.each(n) - 1) / plan.each(n) - 1;
  } else {
    c0 = int(s / plan.share);
    c1 = int((s + n - 1) / plan.share);
  }
  // the pieces' grid: wait for its completion
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 == c1) return;
  const int r = (tile % qtiles) * a.TQ * a.G + (i - tile * a.TQ) * a.G + hl;
  auto slot_row = [&](int c) {
    return (long long)(2 * c + (!plan.parts && s > c * plan.share ? 1 : 0)) * a.rows + r;
  };
  float M = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, a.ws_ml[slot_row(c) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float Mu = M == -INFINITY ? 0.f : M;
  constexpr int kV = D / 32;  // columns per lane
  float acc[kV], den = 0.f;
#pragma unroll
  for (int v = 0; v < kV; ++v) acc[v] = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const long long wr = slot_row(c);
    const float2 x = *reinterpret_cast<const float2*>(a.ws_ml + wr * 2);
    const float f = ex2(x.x - Mu);
    den = fmaf(f, x.y, den);
    const float* p = a.ws_acc + wr * D + lane * kV;
    // (a piece in which the row saw nothing has weight zero)
    if constexpr (kV == 4) {
      const float4 y = *reinterpret_cast<const float4*>(p);
      acc[0] = fmaf(f, y.x, acc[0]);
      acc[1] = fmaf(f, y.y, acc[1]);
      acc[2] = fmaf(f, y.z, acc[2]);
      acc[3] = fmaf(f, y.w, acc[3]);
    } else {
      const float2 y = *reinterpret_cast<const float2*>(p);
      acc[0] = fmaf(f, y.x, acc[0]);
      acc[1] = fmaf(f, y.y, acc[1]);
    }
  }
  const bool none = den == 0.f || __ldg(a.parents + (long long)b * a.N + i) == -2;
  const float inv = none ? 0.f : 1.f / den;
#pragma unroll
  for (int v = 0; v < kV; ++v) acc[v] = none ? 0.f : acc[v] * inv;
  __nv_bfloat16* dst = a.out + row * D + lane * kV;
  if constexpr (kV == 4)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0], acc[1]);
  if (lane == 0) a.lse[row] = none ? -INFINITY : (Mu + __log2f(den)) * kLn2Tree;
}

struct TreeGeom {
  int TQ, JC, ND, tiles, nt, rows;
  bool pair;
};
TreeGeom tree_geom(int N, int G, int L) {
  TreeGeom t;
  t.TQ = min(N, 128 / G);
  t.JC = 128 / t.TQ;
  t.ND = (L + t.JC - 1) / t.JC;
  t.tiles = (N + t.TQ - 1) / t.TQ;
  t.pair = t.tiles > 1;
  t.nt = t.pair ? (t.tiles + 1) / 2 : 1;
  t.rows = t.TQ * G * (t.pair ? 2 : 1);
  return t;
}

template <int D, bool kPair, bool kPrompt, int kThin = 0>
cudaError_t launch_tree_d(const TreeProblem& p, const TreeGeom& tg, const TreeArgs& a,
                          const void* q, const void* k, const void* v, const void* kt,
                          const void* vt, const void* kd, const void* vd, EncodeTiledFn encode,
                          cudaStream_t stream, const char** why) {
  using Cfg = TreeCfg<D, kPair, kThin>;
  const cuuint64_t E = 2, BG = cuuint64_t(p.B) * p.Hkv;
  auto map = [&](CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                 const cuuint64_t* str, const cuuint32_t* box) {
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, str,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  CUtensorMap mQ, mK, mV, mKT, mVT, mKD, mVD;
  bool ok;
  {
    const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(a.G), cuuint64_t(p.N), BG};
    const cuuint64_t str[3] = {cuuint64_t(p.N) * D * E, cuuint64_t(D) * E,
                               cuuint64_t(a.G) * p.N * D * E};
    const cuuint32_t box[4] = {64, cuuint32_t(a.G), cuuint32_t(tg.TQ), 1};
    ok = map(&mQ, q, 4, dims, str, box);
  }
  auto keys = [&](CUtensorMap* m, const void* base, int rows) {
    const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(rows), BG};
    const cuuint64_t str[2] = {cuuint64_t(D) * E, cuuint64_t(rows) * D * E};
    const cuuint32_t box[3] = {64, 128, 1};
    return map(m, base, 3, dims, str, box);
  };
  ok = ok && keys(&mK, k, p.S) && keys(&mV, v, p.S);
  if (kPrompt) {
    mKT = mK;  // never loaded
    mVT = mV;
  } else {
    ok = ok && keys(&mKT, kt, p.N) && keys(&mVT, vt, p.N);
  }
  mKD = mK;  // never loaded when L == 0
  mVD = mV;
  if (p.L > 0) {
    const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(p.L), cuuint64_t(p.N), BG};
    const cuuint64_t str[3] = {cuuint64_t(D) * E, cuuint64_t(p.L) * D * E,
                               cuuint64_t(p.N) * p.L * D * E};
    const cuuint32_t box[4] = {64, cuuint32_t(tg.JC), cuuint32_t(tg.TQ), 1};
    ok = ok && map(&mKD, kd, 4, dims, str, box) && map(&mVD, vd, 4, dims, str, box);
  }
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed for the tree attention's tensors";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(moda_tree_kernel<D, kPair, kPrompt, kThin>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg::kSmemBytes);
  if (e != cudaSuccess) {
    *why = "cudaFuncSetAttribute(max dynamic shared memory) failed";
    return e;
  }
  // prompts: one CTA per SM takes item after item, up to kPromptItems each
  unsigned grid = kTreeCtas;
  if (kPrompt) {
    const long long each = (a.most + kPromptItems - 1) / kPromptItems;
    grid = unsigned(a.most < kTreeCtas ? a.most : (each > kTreeCtas ? each : kTreeCtas));
  }
  moda_tree_kernel<D, kPair, kPrompt, kThin><<<grid, kTreeThreads, Cfg::kSmemBytes, stream>>>(
      mQ, mK, mV, mKT, mVT, mKD, mVD, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = kPrompt ? "packed forward launch failed" : "tree attention launch failed";
    return e;
  }
  if (kPrompt) return e;
  // programmatic dependent launch: see the decode's combine step
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(((long long)p.B * p.Hq * p.N + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, moda_tree_join_kernel<D>, a, kPair ? 2 : 1);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) *why = "tree attention join launch failed";
  return e;
}

TreeArgs tree_args(const TreeProblem& p, const TreeGeom& t, void* out, float* lse) {
  TreeArgs a = {};
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.B = p.B;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.G = p.Hq / p.Hkv;
  a.N = p.N;
  a.S = p.S;
  a.L = p.L;
  a.TQ = t.TQ;
  a.JC = t.JC;
  a.ND = t.ND;
  a.nt = t.nt;
  a.nit = p.Hkv * t.nt;
  a.rows = t.rows;
  a.scale_log2 = p.scale * kLog2eTree;
  return a;
}

}  // namespace

size_t tree_workspace_bytes(const TreeProblem& p) {
  const TreeGeom t = tree_geom(p.N, p.Hq / p.Hkv, p.L);
  return size_t(2 * kTreeCtas) * t.rows * (p.d + 2) * 4;
}

cudaError_t launch_tree(const TreeProblem& p, const void* q, const void* k, const void* v,
                        const void* kt, const void* vt, const void* kd, const void* vd,
                        const int* parents, const int* lengths, void* out, float* lse,
                        void* workspace, EncodeTiledFn encode, cudaStream_t stream,
                        const char** why) {
  const TreeGeom t = tree_geom(p.N, p.Hq / p.Hkv, p.L);
  TreeArgs a = tree_args(p, t, out, lse);
  a.ws_acc = static_cast<float*>(workspace);
  a.ws_ml = a.ws_acc + size_t(2 * kTreeCtas) * t.rows * p.d;
  a.parents = parents;
  a.lengths = lengths;
  auto go = [&](auto d_c, auto pair_c) {
    return launch_tree_d<decltype(d_c)::value, decltype(pair_c)::value, false>(
        p, t, a, q, k, v, kt, vt, kd, vd, encode, stream, why);
  };
  using D128 = std::integral_constant<int, 128>;
  using D64 = std::integral_constant<int, 64>;
  // Few rows: the transposed products, with 4 rows' exponentials a thread or with 16.  (d = 64 has
  // no such form: its O^T would have 64 lanes.)  From a graph, 16 heads in groups of 4, 4-row form /
  // 16-row form / full tiles: one token (4 rows), 4 caches of 1000 keys with L = 24: 12.3 / 16.2 /
  // 15.9 us, 32 of 10K-32K with L = 48: 223 / 229 / 235; 4 tokens (16 rows), - / 16.4 / 16.4 and
  // - / 235 / 247.
  const int rows = p.N * (p.Hq / p.Hkv);
  if (p.d == 128 && rows <= 4)
    return launch_tree_d<128, false, false, 4>(p, t, a, q, k, v, kt, vt, kd, vd, encode, stream,
                                               why);
  if (p.d == 128 && rows <= 16)
    return launch_tree_d<128, false, false, 16>(p, t, a, q, k, v, kt, vt, kd, vd, encode, stream,
                                                why);
  if (p.d == 128)
    return t.pair ? go(D128{}, std::true_type{}) : go(D128{}, std::false_type{});
  return t.pair ? go(D64{}, std::true_type{}) : go(D64{}, std::false_type{});
}

// The forward kernel's pairs of tiles make better use of the tensor cores; single tiles (whose
// two warpgroups take alternate key blocks) are done sooner, and here a CTA goes on to its next
// tile with the loads already under way.  So single tiles are taken
//   - while their CTAs fit the GPU at once, smaller ones as long as that still holds: with few
//     tokens a tile, a depth step holds more of each token's entries (16 heads in groups of 4,
//     d = 128, L = 24: 411 tokens in 5 sequences 14.4 us, 17.4 in full tiles, against the forward
//     kernel's 22.5);
//   - for short sequences, about as long as a tile or shorter, in tiles of up to twice their
//     length (1500 tokens in 181: 60 us against 105; 4000 in 200: 99 against 135; 4000 in 64, mean
//     62: 85 against 79, so not there);
//   - for sequences of up to five tiles when each CTA gets several (12000 tokens in 200, d = 64,
//     L = 8: 94 us against 126; 16000 in 50, L = 0, mean 320: 136 against 123, so not there).
// Groups without a dense depth path in the forward kernel run here at any size: in pairs of
// tiles once single ones no longer fit and sequences are long (groups of 3, d = 64, L = 7: 5000
// tokens in 37 sequences 26 us in single tiles and 33 in pairs; 9000 in 30, 42 and 41).
// (From a graph; log-normal lengths, sigma 1.)  The mean is all that the host knows: where one
// sequence is much longer than the others, or slots of cu_seqlens are empty, the variant may be the
// slower one (one sequence of 64K tokens 15.3 ms, and 19.9 with 1023 empty slots behind it).
PromptTile prompt_tile(const Problem& p) {
  const int full = 128 / p.G;
  const int nseq = p.nseq < p.T ? p.nseq : p.T;
  auto pieces = [&](int tokens) { return packed_pieces_estimate(p, tokens); };
  const int mean = p.T / nseq;
  const bool dense = p.L == 0 || dense_depth_supported(p);
  int tokens = full;
  if (pieces(dense ? full : 2 * full) <= kTreeCtas) {
    while (tokens > 1 && pieces(tokens / 2) <= kTreeCtas) tokens /= 2;
    return PromptTile{tokens, false};
  }
  const bool single = dense ? 4 * mean <= 5 * full ||
                                  (mean <= 5 * full && pieces(full) >= 6 * kTreeCtas)
                            : mean <= 4 * full;
  if (!single) return dense ? PromptTile{0, false} : PromptTile{full, true};
  while (tokens > 8 && tokens / 2 >= 2 * mean) tokens /= 2;
  return PromptTile{tokens, false};
}

cudaError_t launch_prompt(const Problem& p, const PromptTile& tile, const void* q, const void* k,
                          const void* v, const void* kd, const void* vd, void* out, float* lse,
                          EncodeTiledFn encode, cudaStream_t stream, const char** why) {
  const TreeProblem tp{1, p.Hq, p.Hkv, p.T, p.T, p.L, p.d, p.scale};
  TreeGeom t;
  t.TQ = tile.tokens;
  t.JC = 128 / t.TQ;
  t.ND = (p.L + t.JC - 1) / t.JC;
  t.pair = tile.pair;
  t.tiles = t.nt = 1;
  t.rows = 0;  // (no workspace)
  TreeArgs a = tree_args(tp, t, out, lse);
  a.cu = p.cu;
  a.nseq = p.nseq;
  a.causal = p.causal;
  a.most = p.Hkv * packed_pieces_bound(p.T, p.nseq, t.TQ * (t.pair ? 2 : 1));
  auto go = [&](auto d_c, auto pair_c) {
    return launch_tree_d<decltype(d_c)::value, decltype(pair_c)::value, true>(
        tp, t, a, q, k, v, nullptr, nullptr, kd, vd, encode, stream, why);
  };
  using D128 = std::integral_constant<int, 128>;
  using D64 = std::integral_constant<int, 64>;
  if (p.d == 128)
    return t.pair ? go(D128{}, std::true_type{}) : go(D128{}, std::false_type{});
  return t.pair ? go(D64{}, std::true_type{}) : go(D64{}, std::false_type{});
}

}  // namespace moda
