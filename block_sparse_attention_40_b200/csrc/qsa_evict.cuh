// qsa_evict.cuh -- eviction from a decode cache by accumulated attention weight.
//
// k_block_weights: the attention weight that one decode query gives to each selected block (and
// to its own block), summed over the 24 heads and added to the cache's running weights.
// k_evict_select / k_evict_move: a sequence of more than `keep` complete blocks keeps its
// first `sinks`, its last `recent` and, of the rest, those of largest running weight (the lower
// block among equals), moved together in place and in order; the incomplete last block follows.

#pragma once

#include <cooperative_groups.h>

#include "qsa_common.cuh"

namespace qsa {

// ---------------------------------------------------------------------------------------
// Attention weights per block.  For each head, with the scaled logits x of the live tokens of
// the selected blocks and the own block,  w[blk] = sum_heads sum_{t in blk} e^(x_t - lse_h).
//
// One cluster of C CTAs per sequence; a warp takes tiles of 4 blocks (16 token rows) of one KV
// head.  A tile's logits are one 16 x 16 x 128 product (tokens x the group's 12 heads, padded
// to 16): warp MMAs, since 12 query rows would leave most of a tcgen05 tile empty and the
// kernel is bound by the keys' bytes (2 KB a block).  Keys go straight from global memory to the
// operand registers: the order of the 128 dims inside the product is free, so each lane's
// fragments are whole 16-byte words.  Every (block, head) pair leaves one number, the log2 of
// the sum of its 4 exponentials, in shared memory; the heads' totals are then joined over the
// CTA and the cluster (distributed shared memory) in a fixed order, and each block's weight
// is the sum over heads of 2^(block's log-sum - head's total): one pass over the keys and no
// second launch.
constexpr int kWtThreads = 256;
constexpr int kWtWarps = kWtThreads / 32;
constexpr int kWtMaxCluster = 16;

struct WeightArgs {
  const __nv_bfloat16* q;         // [B][24][128]
  const __nv_bfloat16* k_blocks;  // [pool pages][2][page blocks][4][128]
  const int32_t* len;             // [B]
  const int32_t* idx;             // [B][topk]
  const int32_t* cnt;             // [B]
  int32_t topk;
  int32_t cap_blocks;             // row length of mass
  float* mass;                    // [B][cap_blocks]
  Paging pg;
  DevStatus st;
};

__device__ __forceinline__ void mma_bf16_16816(float* c, const uint32_t* a, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Tiles (of 4 items) that a CTA of a cluster of c handles; items = selected blocks + own block.
__host__ __device__ constexpr int wt_tiles_per_cta(int topk, int c) {
  return ((topk + 1 + 3) / 4 + c - 1) / c;
}
__host__ __device__ constexpr int wt_smem_bytes(int topk, int c) {
  return wt_tiles_per_cta(topk, c) * 4 * (kHeads + 1) * 4;
}

// grid (C, B), clusters of (C, 1, 1)
__global__ void __launch_bounds__(kWtThreads) k_block_weights(WeightArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ float lse_sh[];                   // [local item][25]
  __shared__ float head_m[kHeads], head_s[kHeads];    // this CTA's max and sum per head
  __shared__ float head_lse[kHeads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int C = gridDim.x, rank = blockIdx.x, b = blockIdx.y;
  const int len = a.len[b];
  const int own = (len - 1) / kBlock;
  int n = a.cnt[b];
  const bool bad = len < 1 || own >= a.cap_blocks || n < 0 || n > a.topk;
  if (bad && tid == 0 && rank == 0) report_error(a.st, kErrDevice, 300);
  if (bad) n = 0;
  const int items = bad ? 0 : n + 1;
  const int per = wt_tiles_per_cta(a.topk, C) * 4;    // items per CTA
  const int i0 = rank * per, mine = max(0, min(per, items - i0));
  const int32_t* idx = a.idx + static_cast<int64_t>(b) * a.topk;
  // block of item i, -1 where it cannot be used (out of order or range)
  auto item_block = [&](int i) -> int {
    if (i == n) return own;
    const int x = idx[i];
    const int before = i > 0 ? idx[i - 1] : -1;
    return (x <= before || x < 0 || x >= own) ? -1 : x;
  };
  const int kv = warp & 1;
  // this KV head's queries as B fragments: n-tile 0 is heads 0..7, n-tile 1 heads 8..11
  uint4 qf[2][4];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int hd = nt * 8 + g;
      qf[nt][j] = make_uint4(0u, 0u, 0u, 0u);
      if (hd < kGroup)
        qf[nt][j] = *reinterpret_cast<const uint4*>(
            a.q + ((static_cast<int64_t>(b) * kHeads + kv * kGroup + hd) * kHeadDim + 32 * j + 8 * tq));
    }
  const float scale = 0.08838834764831845f * 1.4426950408889634f;   // 1/sqrt(128) in log2 units
  for (int tile = warp >> 1; tile * 4 < mine; tile += kWtWarps / 2) {
    uint4 kf[2][4];
    bool live[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int li = tile * 4 + (g >> 2) + 2 * half, tok = g & 3;
      int blk = -1;
      if (li < mine) {
        blk = item_block(i0 + li);
        if (blk < 0 && kv == 0 && (lane & 15) == 0) report_error(a.st, kErrDevice, 301);
      }
      live[half] = blk >= 0 && blk * kBlock + tok < len;
#pragma unroll
      for (int j = 0; j < 4; ++j) kf[half][j] = make_uint4(0u, 0u, 0u, 0u);
      if (live[half]) {
        const int64_t row = pool_kv_row(a.pg, b, kv, blk);
        if (row < 0) {   // reads as zeros, as in the decode attention
          if (tq == 0) report_error(a.st, kErrDevice, 302);
        } else {
          const uint4* kp = reinterpret_cast<const uint4*>(a.k_blocks + (row + tok) * kHeadDim) + tq;
#pragma unroll
          for (int j = 0; j < 4; ++j) kf[half][j] = kp[4 * j];
        }
      }
    }
    float acc[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a0[4] = {kf[0][j].x, kf[1][j].x, kf[0][j].y, kf[1][j].y};
      const uint32_t a1[4] = {kf[0][j].z, kf[1][j].z, kf[0][j].w, kf[1][j].w};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        mma_bf16_16816(acc[nt], a0, qf[nt][j].x, qf[nt][j].y);
        mma_bf16_16816(acc[nt], a1, qf[nt][j].z, qf[nt][j].w);
      }
    }
    // rows of one block sit in lanes that differ in bits 2 and 3: join its four tokens
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int half = e >> 1;
        const float x = live[half] ? acc[nt][e] * scale : -INFINITY;
        float m = x;
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        float s = x == -INFINITY ? 0.f : exp2f(x - m);
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        const int hd = nt * 8 + 2 * tq + (e & 1);
        const int li = tile * 4 + (g >> 2) + 2 * half;
        if ((g & 3) == 0 && hd < kGroup && li < mine)
          lse_sh[li * (kHeads + 1) + kv * kGroup + hd] = m + log2f(s);
      }
  }
  __syncthreads();
  // per head: this CTA's max and sum (one warp takes heads warp, warp + 8, ..)
  for (int hd = warp; hd < kHeads; hd += kWtWarps) {
    float m = -INFINITY;
    for (int i = lane; i < mine; i += 32) m = fmaxf(m, lse_sh[i * (kHeads + 1) + hd]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = 0.f;
    if (m > -INFINITY)
      for (int i = lane; i < mine; i += 32) s += exp2f(lse_sh[i * (kHeads + 1) + hd] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      head_m[hd] = m;
      head_s[hd] = s;
    }
  }
  cl.sync();
  if (tid < kHeads) {
    float m = -INFINITY;
    for (int c = 0; c < C; ++c) m = fmaxf(m, *cl.map_shared_rank(&head_m[tid], c));
    float s = 0.f;
    for (int c = 0; c < C; ++c) {
      const float mc = *cl.map_shared_rank(&head_m[tid], c);
      if (mc > -INFINITY) s += *cl.map_shared_rank(&head_s[tid], c) * exp2f(mc - m);
    }
    head_lse[tid] = m + log2f(s);
  }
  cl.sync();   // also: no CTA exits while another reads its shared memory
  for (int li = tid; li < mine; li += kWtThreads) {
    const int blk = item_block(i0 + li);
    if (blk < 0) continue;
    float w = 0.f;
#pragma unroll
    for (int hd = 0; hd < kHeads; ++hd) w += exp2f(lse_sh[li * (kHeads + 1) + hd] - head_lse[hd]);
    a.mass[static_cast<int64_t>(b) * a.cap_blocks + blk] += w;
  }
}

// ---------------------------------------------------------------------------------------
// Which blocks stay.  One CTA per sequence: a radix select (digits of 11, 11 and 10 bits, high
// to low, histograms in shared memory) finds the key of the last block that stays and how many
// blocks of exactly that key stay, then one ordered pass writes the kept blocks in ascending
// order.  A weight's key orders as the weight does; NaN counts below every number and -0 as 0.
constexpr int kEvThreads = 1024;
constexpr int kEvBins = 2048;

// What the select leaves for the move, per sequence (a CTA's worth of 32-bit words).
struct EvictMeta {
  int32_t count;   // blocks to place, the incomplete last one included; 0: nothing moves
  int32_t first;   // first place whose block comes from elsewhere
  int32_t whole;   // complete blocks kept
  int32_t old;     // blocks held before, the incomplete last one included
};

struct EvictArgs {
  int32_t* len;          // [B]
  float* mass;           // [B][cap_blocks]
  int32_t cap_blocks;
  int32_t batch;
  int32_t keep, sinks, recent;
  int32_t* kept;         // [B][keep] or null
  int32_t* src;          // [B][keep + 1] workspace: place j takes block src[j]
  EvictMeta* meta;       // [B] workspace
  uint4* k_blocks;       // pools, 64 units of 16 bytes a block (K, V), 8 (kbar)
  uint4* v_blocks;
  uint4* kbar;
  Paging pg;
  int32_t parts;         // column parts of a block that move independently
  DevStatus st;
};

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  return float_key(w + 0.f);
}

__global__ void __launch_bounds__(kEvThreads) k_evict_select(EvictArgs a) {
  __shared__ uint32_t hist[kEvBins];
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t sh_prefix, sh_need;
  __shared__ int sh_first;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x;
  const int len = a.len[b];
  const int nb = len / kBlock, tail = len % kBlock;
  const float* mass = a.mass + static_cast<int64_t>(b) * a.cap_blocks;
  int32_t* src = a.src + static_cast<int64_t>(b) * (a.keep + 1);
  int32_t* kept = a.kept != nullptr ? a.kept + static_cast<int64_t>(b) * a.keep : nullptr;
  if (len < 0 || nb > a.cap_blocks || nb <= a.keep) {   // nothing to cut (or a length out of range)
    if (tid == 0) {
      if (len < 0 || nb > a.cap_blocks) report_error(a.st, kErrDevice, 310);
      a.meta[b] = EvictMeta{0, 0, 0, 0};
    }
    if (kept != nullptr)
      for (int j = tid; j < a.keep; j += kEvThreads) kept[j] = j < nb ? j : -1;
    return;
  }
  const int lo = a.sinks, hi = nb - a.recent;            // candidates lo .. hi-1
  const uint32_t want = static_cast<uint32_t>(a.keep - a.sinks - a.recent);
  // key of the last candidate that stays (prefix) and how many of that key stay (need)
  if (tid == 0) {
    sh_prefix = 0u;
    sh_need = want;
  }
  const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
  for (int d = 0; d < 3 && want > 0; ++d) {
    for (int i = tid; i < kEvBins; i += kEvThreads) hist[i] = 0u;
    __syncthreads();
    const uint32_t prefix = sh_prefix, need = sh_need;
    const uint32_t bins = 1u << bits[d];
    for (int i0 = lo; i0 < hi; i0 += kEvThreads) {
      const int i = i0 + tid;
      uint32_t bin = 0xffffffffu;
      if (i < hi) {
        const uint32_t key = weight_key(mass[i]);
        if (d == 0 || (key >> (shift[d] + bits[d])) == prefix) bin = (key >> shift[d]) & (bins - 1);
      }
      // equal bins of a warp (runs of zero weight) count as one addition
      const uint32_t same = __match_any_sync(0xffffffffu, bin);
      if (bin != 0xffffffffu && lane == __ffs(same) - 1) atomicAdd(&hist[bin], __popc(same));
    }
    __syncthreads();
    // suffix counts, two bins a thread from the top: thread t has bins bins-1-2t, bins-2-2t
    const int b1 = static_cast<int>(bins) - 1 - 2 * tid, b0 = b1 - 1;
    const uint32_t h1 = b1 >= 0 ? hist[b1] : 0u, h0 = b0 >= 0 ? hist[b0] : 0u;
    uint32_t incl = h1 + h0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t base = 0;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    const uint32_t above = base + incl - h1 - h0;   // candidates in higher bins
    if (b1 >= 0 && above < need && above + h1 >= need) {
      sh_prefix = (prefix << bits[d]) | static_cast<uint32_t>(b1);
      sh_need = need - above;
    } else if (b0 >= 0 && above + h1 < need && above + h1 + h0 >= need) {
      sh_prefix = (prefix << bits[d]) | static_cast<uint32_t>(b0);
      sh_need = need - above - h1;
    }
    __syncthreads();
  }
  __syncthreads();
  const uint32_t last = sh_prefix, ties = sh_need;
  // ordered pass: a block before which m larger and e equal candidates stand takes place
  // sinks + m + min(e, ties)
  uint32_t done_gt = 0, done_eq = 0;
  if (tid == 0) sh_first = want > 0 ? hi : lo;   // becomes the first block that goes
  __syncthreads();
  for (int j = tid; j < a.sinks; j += kEvThreads) {
    src[j] = j;
    if (kept != nullptr) kept[j] = j;
  }
  for (int i0 = lo; i0 < hi && want > 0; i0 += kEvThreads) {
    const int i = i0 + tid;
    uint32_t gt = 0, eq = 0;
    if (i < hi) {
      const uint32_t key = weight_key(mass[i]);
      gt = key > last;
      eq = key == last;
    }
    // counts of both in one 32-bit scan (at most 1,024 of each)
    uint32_t incl = gt << 16 | eq;
    const uint32_t own = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t base = 0, total = 0;
    for (int w = 0; w < 32; ++w) {
      if (w == warp) base = total;
      total += warp_sum[w];
    }
    const uint32_t ex = base + incl - own;
    const uint32_t m = done_gt + (ex >> 16), e = done_eq + (ex & 0xffffu);
    if (gt || (eq && e < ties)) {
      const int place = lo + static_cast<int>(m + min(e, ties));
      src[place] = i;
      if (kept != nullptr) kept[place] = i;
    } else if (i < hi && done_gt + min(done_eq, ties) == static_cast<uint32_t>(i0 - lo)) {
      atomicMin(&sh_first, i);   // no block before this pass has gone
    }
    done_gt += total >> 16;
    done_eq += total & 0xffffu;
    __syncthreads();
  }
  for (int j = tid; j < a.recent; j += kEvThreads) {
    const int place = a.keep - a.recent + j;
    src[place] = hi + j;
    if (kept != nullptr) kept[place] = hi + j;
  }
  __syncthreads();
  if (tid == 0) {
    src[a.keep] = nb;
    a.meta[b] = EvictMeta{a.keep + (tail > 0), sh_first, a.keep, nb + (tail > 0)};
    a.len[b] = kBlock * a.keep + tail;
  }
}

// Moves the kept blocks together.  Place j takes block src[j] >= j and src is ascending, so a
// CTA that walks its places in order, a tile at a time, reads nothing that it has overwritten:
// the tile's loads (into registers) come before the barrier, its stores after it, and the next
// tile's sources lie beyond this tile's places.  Streams that are independent go to their own
// CTAs: K and V of each KV head, each cut into `parts` column ranges, the compressed keys and
// the weights.  Nothing before the first place that changes is touched.
constexpr int kMvThreads = 512;
constexpr int kMvUnits = 8;   // 16-byte units a thread holds

__global__ void __launch_bounds__(kMvThreads) k_evict_move(EvictArgs a) {
  const int tid = threadIdx.x, b = blockIdx.y;
  const EvictMeta m = a.meta[b];
  if (m.count == 0) return;
  const int32_t* src = a.src + static_cast<int64_t>(b) * (a.keep + 1);
  const int stream = blockIdx.x;
  if (stream < 4 * a.parts) {
    const int which = stream / a.parts, part = stream % a.parts, g = which & 1;
    uint4* pool = which < 2 ? a.k_blocks : a.v_blocks;
    const int upb = 64 / a.parts;   // units of a block in this stream (a power of two)
    const int64_t u_end = static_cast<int64_t>(m.count) * upb;
    auto unit = [&](int64_t blk, int u) -> uint4* {
      const int64_t row = pool_kv_row(a.pg, b, g, blk);
      return row < 0 ? nullptr : pool + row * 16 + part * upb + u;
    };
    for (int64_t u0 = static_cast<int64_t>(m.first) * upb; u0 < u_end;
         u0 += kMvThreads * kMvUnits) {
      uint4 x[kMvUnits];
#pragma unroll
      for (int i = 0; i < kMvUnits; ++i) {
        const int64_t u = u0 + i * kMvThreads + tid;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (u < u_end) {
          const uint4* p = unit(src[u / upb], static_cast<int>(u % upb));
          if (p != nullptr) x[i] = __ldcg(p);
          else if (stream == 0 && u % upb == 0) report_error(a.st, kErrDevice, 311);
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMvUnits; ++i) {
        const int64_t u = u0 + i * kMvThreads + tid;
        if (u < u_end) {
          uint4* p = unit(u / upb, static_cast<int>(u % upb));
          if (p != nullptr) __stcg(p, x[i]);
          else if (stream == 0 && u % upb == 0) report_error(a.st, kErrDevice, 312);
        }
      }
    }
  } else if (stream == 4 * a.parts) {
    const int64_t u_end = static_cast<int64_t>(m.whole) * 8;
    for (int64_t u0 = static_cast<int64_t>(m.first) * 8; u0 < u_end; u0 += kMvThreads * kMvUnits) {
      uint4 x[kMvUnits];
#pragma unroll
      for (int i = 0; i < kMvUnits; ++i) {
        const int64_t u = u0 + i * kMvThreads + tid;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (u < u_end) {
          const int64_t blk = pool_block(a.pg, b, src[u / 8]);
          if (blk >= 0) x[i] = __ldcg(a.kbar + blk * 8 + u % 8);
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMvUnits; ++i) {
        const int64_t u = u0 + i * kMvThreads + tid;
        if (u < u_end) {
          const int64_t blk = pool_block(a.pg, b, u / 8);
          if (blk >= 0) __stcg(a.kbar + blk * 8 + u % 8, x[i]);
        }
      }
    }
  } else {
    float* mass = a.mass + static_cast<int64_t>(b) * a.cap_blocks;
    for (int j0 = m.first; j0 < m.count; j0 += kMvThreads * kMvUnits) {
      float x[kMvUnits];
#pragma unroll
      for (int i = 0; i < kMvUnits; ++i) {
        const int j = j0 + i * kMvThreads + tid;
        x[i] = j < m.count ? __ldcg(mass + src[j]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMvUnits; ++i) {
        const int j = j0 + i * kMvThreads + tid;
        if (j < m.count) __stcg(mass + j, x[i]);
      }
    }
    __syncthreads();
    for (int j = m.count + tid; j < m.old; j += kMvThreads) mass[j] = 0.f;
  }
}

}  // namespace qsa
