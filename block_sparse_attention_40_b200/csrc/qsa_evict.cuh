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
// One cluster of C CTAs per sequence, each with a part of the selected blocks, whose places in the
// pool it looks up first.  A warp takes tiles of 4 blocks (16 token rows) of one KV head, the next
// tile's keys on their way.  A tile's logits are one 16 x 16 x 128 product (tokens x the group's
// 12 heads, padded to 16): warp MMAs, since 12 query rows would leave most of a tcgen05 tile empty
// and the kernel is bound by the keys' bytes (2 KB a block), or by latency where there are few.
// Keys go straight from global memory to the operand registers: the order of the 128 dims inside
// the product is free, so each lane's fragments are whole 16-byte words.  Every (block, head) pair
// leaves one number, the log2 of the sum of its 4 exponentials, in shared memory; the heads'
// totals are then joined over the CTA and the cluster (distributed shared memory) in a fixed
// order, and each block's weight is the sum over heads of 2^(block's log-sum - head's total): one
// pass over the keys and no second launch.  64 sequences of 32K tokens, 4,096-token pages: 21.3 us
// a call, 3.2 TB/s (the keys would take 10.4; 17.9 us where L2 holds them); one sequence: 8.8 us, all
// latency (idx -> page -> keys, two barriers of the cluster).
constexpr int kWtMaxCluster = 8;

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

// 2^x to 2 ulp (0 for -inf) and log2 x to 2^-22 (-inf for 0): a weight is off by as much
__device__ __forceinline__ float wt_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float wt_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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
// log-sums (rows of 25: without bank conflicts), logical blocks, places in the pool, running weights
__host__ __device__ constexpr int wt_smem_bytes(int topk, int c) {
  return wt_tiles_per_cta(topk, c) * 4 * (kHeads + 1 + 3) * 4;
}

// grid (C, B), clusters of (C, 1, 1)
template <int kWtThreads>
__global__ void __launch_bounds__(kWtThreads) k_block_weights(WeightArgs a) {
  constexpr int kWtWarps = kWtThreads / 32;
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ float lse_sh[];                   // [local item][25]
  __shared__ float head_m[kHeads], head_s[kHeads];    // this CTA's max and sum per head
  __shared__ float head_lse[kHeads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int C = gridDim.x, rank = blockIdx.x, b = blockIdx.y;
  const int per = wt_tiles_per_cta(a.topk, C) * 4;    // items per CTA: selected blocks, own block
  int32_t* blk_sh = reinterpret_cast<int32_t*>(lse_sh + per * (kHeads + 1));   // -1: not used
  int32_t* at_sh = blk_sh + per;                      // its K rows / 4 (KV head 0); -1: reads as zeros
  float* mass_sh = reinterpret_cast<float*>(at_sh + per);   // fetched here, added to at the end
  float* mass = a.mass + static_cast<int64_t>(b) * a.cap_blocks;
  pdl_wait();      // launched as a programmatic dependent of the caller's last kernel, which is done
  pdl_trigger();   // before any kernel behind this one starts
  const int len = a.len[b];
  const int own = (len - 1) / kBlock;
  int n = a.cnt[b];
  const bool bad = len < 1 || own >= a.cap_blocks || n < 0 || n > a.topk;
  if (bad && tid == 0 && rank == 0) report_error(a.st, kErrDevice, 300);
  if (bad) n = 0;
  const int items = bad ? 0 : n + 1;
  const int i0 = rank * per, mine = max(0, min(per, items - i0));
  const int32_t* idx = a.idx + static_cast<int64_t>(b) * a.topk;
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
  for (int li = tid; li < per; li += kWtThreads) {
    int blk = -1, at = -1;
    if (li < mine) {
      const int i = i0 + li;
      if (i == n) {
        blk = own;
      } else {
        // out of order or range: left out
        const int x = idx[i], before = i > 0 ? idx[i - 1] : -1;
        blk = (x <= before || x < 0 || x >= own) ? -1 : x;
        if (blk < 0) report_error(a.st, kErrDevice, 301);
      }
      if (blk >= 0) {
        mass_sh[li] = mass[blk];
        const int64_t row = pool_kv_row(a.pg, b, 0, blk);
        at = row < 0 ? -1 : static_cast<int32_t>(row / kBlock);
        if (row < 0) report_error(a.st, kErrDevice, 302);
      }
    }
    blk_sh[li] = blk;
    at_sh[li] = at;
  }
  __syncthreads();
  const float scale = 0.08838834764831845f * 1.4426950408889634f;   // 1/sqrt(128) in log2 units
  const int tiles = (mine + 3) / 4, step = kWtWarps / 2;
  auto fetch = [&](int tile, uint4 (*kf)[4]) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int li = tile * 4 + (g >> 2) + 2 * half;
      const int at = tile < tiles ? at_sh[li] : -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) kf[half][j] = make_uint4(0u, 0u, 0u, 0u);
      // tokens behind the last one are read too (the block's space is there) and masked below
      if (at >= 0) {
        const int64_t row = (static_cast<int64_t>(at) + kv * a.pg.page_blocks) * kBlock + (g & 3);
        const uint4* kp = reinterpret_cast<const uint4*>(a.k_blocks + row * kHeadDim) + tq;
#pragma unroll
        for (int j = 0; j < 4; ++j) kf[half][j] = kp[4 * j];
      }
    }
  };
  auto logits = [&](int tile, const uint4 (*kf)[4]) {
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
    for (int half = 0; half < 2; ++half) {
      const int li = tile * 4 + (g >> 2) + 2 * half;
      const int blk = blk_sh[li];
      const bool live = blk >= 0 && blk * kBlock + (g & 3) < len;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 2 * half; e < 2 * half + 2; ++e) {
          const float x = live ? acc[nt][e] * scale : -INFINITY;
          float m = x;
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          float s = x == -INFINITY ? 0.f : wt_exp2(x - m);
          s += __shfl_xor_sync(0xffffffffu, s, 4);
          s += __shfl_xor_sync(0xffffffffu, s, 8);
          const int hd = nt * 8 + 2 * tq + (e & 1);
          if ((g & 3) == 0 && hd < kGroup) lse_sh[li * (kHeads + 1) + kv * kGroup + hd] = m + wt_log2(s);
        }
    }
  };
  {
    uint4 ka[2][4], kb[2][4];
    int tile = warp >> 1;
    fetch(tile, ka);
    for (; tile < tiles; tile += 2 * step) {
      fetch(tile + step, kb);
      logits(tile, ka);
      if (tile + step >= tiles) break;
      fetch(tile + 2 * step, ka);
      logits(tile + step, kb);
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
      for (int i = lane; i < mine; i += 32) s += wt_exp2(lse_sh[i * (kHeads + 1) + hd] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      head_m[hd] = m;
      head_s[hd] = s;
    }
  }
  cl.sync();
  // the heads' totals over the cluster, a CTA a lane
  for (int hd = warp; hd < kHeads; hd += kWtWarps) {
    float mc = -INFINITY, s = 0.f;
    if (lane < C) {
      mc = *cl.map_shared_rank(&head_m[hd], lane);
      s = *cl.map_shared_rank(&head_s[hd], lane);
    }
    float m = mc;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    s = mc > -INFINITY ? s * wt_exp2(mc - m) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) head_lse[hd] = m + wt_log2(s);
  }
  __syncthreads();
  cl.barrier_arrive();   // this CTA has read the others' sums
  // four lanes to a block, six heads each
  for (int l0 = 0; l0 < mine; l0 += kWtThreads / 4) {
    const int li = l0 + (tid >> 2), h0 = (tid & 3) * (kHeads / 4);
    const int blk = li < mine ? blk_sh[li] : -1;
    float w = 0.f;
    if (blk >= 0)
#pragma unroll
      for (int hd = 0; hd < kHeads / 4; ++hd)
        w += wt_exp2(lse_sh[li * (kHeads + 1) + h0 + hd] - head_lse[h0 + hd]);
    w += __shfl_xor_sync(0xffffffffu, w, 1);
    w += __shfl_xor_sync(0xffffffffu, w, 2);
    if (blk >= 0 && (tid & 3) == 0) mass[blk] = mass_sh[li] + w;
  }
  cl.barrier_wait();   // no CTA exits while another reads its shared memory
}

// ---------------------------------------------------------------------------------------
// Which blocks stay.  A cluster of CTAs per sequence, each with a contiguous part of its blocks:
// a radix select (digits of 11, 11 and 10 bits, high to low; histograms in shared memory, summed
// over the cluster through distributed shared memory) finds the key of the last block that stays
// and how many blocks of exactly that key stay, then one ordered pass writes the kept blocks in
// ascending order.  A weight's key orders as the weight does; NaN counts below every number and
// -0 as 0.  Bound by latency (barriers of the CTA and the cluster, shared-memory atomics): a row of
// 2,047 weights 8.7 us, 16 rows of 16,383 15 us, one of 262,143 33 us.
constexpr int kEvThreads = 1024;
constexpr int kEvBins = 2048;
constexpr int kEvMaxCluster = 16;
constexpr int kMvPlaces = 16;   // places of a tile of the move
constexpr int kEvBatch = 4;     // consecutive weights of a thread

// What the select leaves for the move, per sequence.
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
  int32_t tiles;         // tiles of kMvPlaces places per sequence
  int32_t* loaded;       // [B][tiles] workspace: the tile's blocks have been read
  int32_t* before;       // [B][tiles + 1] workspace: kept blocks below the tile's first place
  int32_t* ticket;       // [1] workspace
  uint4* k_blocks;       // pools, 64 units of 16 bytes a block (K, V), 8 (kbar)
  uint4* v_blocks;
  uint4* kbar;
  Paging pg;
  DevStatus st;
  uint64_t wait_ns;      // limit of the move's waits
  int32_t fault;         // testing: sequence 0's first tile does not say that its blocks were read
};

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  return float_key(w + 0.f);
}

// Runs f(first index, keys, how many are in range) over i0 .. i1-1, kEvBatch consecutive weights
// a thread, all threads of the CTA together.  A part of one batch a thread stays in registers
// (`held`, from ev_hold); of a longer one the next batch is on its way meanwhile.
constexpr int kEvOnce = kEvThreads * kEvBatch;

__device__ __forceinline__ void ev_fetch(const float* mass, int base, int i1, float* x) {
  const int i = base + kEvBatch * static_cast<int>(threadIdx.x);
#pragma unroll
  for (int b = 0; b < kEvBatch; ++b) x[b] = i + b < i1 ? mass[i + b] : 0.f;
}

__device__ __forceinline__ void ev_hold(const float* mass, int i0, int i1, uint32_t* held) {
  float w[kEvBatch];
  ev_fetch(mass, i0, i1, w);
#pragma unroll
  for (int b = 0; b < kEvBatch; ++b) held[b] = weight_key(w[b]);
}

template <typename F>
__device__ __forceinline__ void ev_scan(const float* mass, int i0, int i1, const uint32_t* held,
                                        F&& f) {
  const int first = i0 + kEvBatch * static_cast<int>(threadIdx.x);
  if (i1 - i0 <= kEvOnce) {
    if (i0 < i1) f(first, held, i1 - first);
    return;
  }
  float w[2][kEvBatch];
  ev_fetch(mass, i0, i1, w[0]);
  for (int base = i0, i = first; base < i1; base += kEvOnce, i += kEvOnce) {
    ev_fetch(mass, base + kEvOnce, i1, w[1]);
    uint32_t key[kEvBatch];
#pragma unroll
    for (int b = 0; b < kEvBatch; ++b) key[b] = weight_key(w[0][b]);
    f(i, key, i1 - i);
#pragma unroll
    for (int b = 0; b < kEvBatch; ++b) w[0][b] = w[1][b];
  }
}

// Sum over the warps before this one of a value per warp, and over all 32 (in *total).
__device__ __forceinline__ uint32_t ev_warps_before(const uint32_t* warp_sum, int warp, int lane,
                                                    uint32_t* total) {
  uint32_t x = warp_sum[lane];
  const uint32_t own = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  *total = __shfl_sync(0xffffffffu, x, 31);
  return __shfl_sync(0xffffffffu, x - own, warp);
}

// grid (C, B), clusters of (C, 1, 1), C a power of two
__global__ void __launch_bounds__(kEvThreads, 1) k_evict_select(EvictArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  __shared__ uint32_t hist[kEvBins];   // this CTA's counts
  __shared__ uint32_t all[kEvBins];    // the cluster's (every CTA sums a slice for all)
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t sh_prefix, sh_need, sh_gt, sh_eq;
  __shared__ int sh_first;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.y;
  const int C = gridDim.x, rank = blockIdx.x;
  pdl_wait();      // the caller's last kernel
  pdl_trigger();   // the move's first CTAs wait beside these
  const int len = a.len[b];
  const int nb = len / kBlock, tail = len % kBlock;
  const float* mass = a.mass + static_cast<int64_t>(b) * a.cap_blocks;
  int32_t* src = a.src + static_cast<int64_t>(b) * (a.keep + 1);
  int32_t* before = a.before + static_cast<int64_t>(b) * (a.tiles + 1);
  int32_t* kept = a.kept != nullptr ? a.kept + static_cast<int64_t>(b) * a.keep : nullptr;
  const int gtid = rank * kEvThreads + tid, gthreads = C * kEvThreads;
  for (int i = gtid; i < a.tiles; i += gthreads) a.loaded[static_cast<int64_t>(b) * a.tiles + i] = 0;
  // (a sequence that ends below the tiles' end: no block of it writes the last entry)
  if (gtid == 0 && nb < a.tiles * kMvPlaces) before[a.tiles] = a.keep + 1;
  if (b == 0 && gtid == 0) *a.ticket = 0;
  const bool bad = len < 0 || len > a.cap_blocks * kBlock;
  if (bad || nb <= a.keep) {   // nothing to cut (or a length out of range)
    if (gtid == 0) {
      if (bad) report_error(a.st, kErrDevice, 310);
      a.meta[b] = EvictMeta{0, 0, 0, 0};
    }
    if (kept != nullptr)
      for (int j = gtid; j < a.keep; j += gthreads) kept[j] = j < nb ? j : -1;
    return;   // the whole cluster
  }
  const int lo = a.sinks, hi = nb - a.recent;            // candidates lo .. hi-1
  const uint32_t want = static_cast<uint32_t>(a.keep - a.sinks - a.recent);
  const int per = (hi - lo + C - 1) / C;
  const int i0 = min(hi, lo + rank * per), i1 = min(hi, i0 + per);   // this CTA's
  uint32_t held[kEvBatch];
  ev_hold(mass, i0, i1, held);
  // key of the last candidate that stays (prefix) and how many of that key stay (need)
  if (tid == 0) {
    sh_prefix = 0u;
    sh_need = want;
    sh_first = 0x7fffffff;   // becomes the first block that goes
  }
  const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
  for (int d = 0; d < 3 && want > 0; ++d) {
    for (int i = tid; i < kEvBins; i += kEvThreads) hist[i] = 0u;
    __syncthreads();
    const uint32_t prefix = sh_prefix, need = sh_need;
    const uint32_t bins = 1u << bits[d];
    uint32_t zeros = 0;   // blocks that were never attended to: counted apart, not one by one
    const uint32_t zero_key = weight_key(0.f);
    ev_scan(mass, i0, i1, held, [&](int, const uint32_t* key, int n) {
#pragma unroll
      for (int j = 0; j < kEvBatch; ++j) {
        const bool on = j < n && (d == 0 || (key[j] >> (shift[d] + bits[d])) == prefix);
        const uint32_t bin = (key[j] >> shift[d]) & (bins - 1);
        // a warp of one bin would queue up: one lane adds for all
        const uint32_t first_bin = __shfl_sync(0xffffffffu, bin, 0);
        const bool alone = __all_sync(0xffffffffu, on && bin == first_bin);
        if (alone) {
          if (lane == 0) atomicAdd(&hist[bin], 32u);
        } else if (on) {
          if (key[j] == zero_key) ++zeros;
          else atomicAdd(&hist[bin], 1u);
        }
      }
    });
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0 && zeros > 0) atomicAdd(&hist[(zero_key >> shift[d]) & (bins - 1)], zeros);
    const uint32_t* counts = hist;
    if (C > 1) {
      counts = all;
      cl.sync();
      // a slice of the bins: the cluster's sum, to every CTA
      const int slice = kEvBins / C;
      if (tid < slice) {
        const int bin = rank * slice + tid;
        uint32_t x = 0;
        for (int c = 0; c < C; ++c) x += *cl.map_shared_rank(&hist[bin], c);
        for (int c = 0; c < C; ++c) *cl.map_shared_rank(&all[bin], c) = x;
      }
      cl.sync();
    } else {
      __syncthreads();
    }
    // suffix counts, two bins a thread from the top: thread t has bins bins-1-2t, bins-2-2t
    const int b1 = static_cast<int>(bins) - 1 - 2 * tid, b0 = b1 - 1;
    const uint32_t h1 = b1 >= 0 ? counts[b1] : 0u, h0 = b0 >= 0 ? counts[b0] : 0u;
    uint32_t incl = h1 + h0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t total;
    const uint32_t base = ev_warps_before(warp_sum, warp, lane, &total);
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
  // larger and equal candidates in the parts before this one
  uint32_t done_gt = 0, done_eq = 0;
  if (want > 0) {
    if (C > 1) {
      uint32_t gt = 0, eq = 0;
      ev_scan(mass, i0, i1, held, [&](int, const uint32_t* key, int n) {
#pragma unroll
        for (int j = 0; j < kEvBatch; ++j) {
          gt += j < n && key[j] > last;
          eq += j < n && key[j] == last;
        }
      });
      if (tid == 0) sh_gt = sh_eq = 0u;
      __syncthreads();
      gt = __reduce_add_sync(0xffffffffu, gt);
      eq = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) {
        atomicAdd(&sh_gt, gt);
        atomicAdd(&sh_eq, eq);
      }
      cl.sync();
      for (int c = 0; c < rank; ++c) {
        done_gt += *cl.map_shared_rank(&sh_gt, c);
        done_eq += *cl.map_shared_rank(&sh_eq, c);
      }
    }
    // ordered pass: a block before which m larger and e equal candidates stand takes place
    // sinks + m + min(e, ties)
    ev_scan(mass, i0, i1, held, [&](int i, const uint32_t* key, int n) {
      // counts of both in one 32-bit scan (at most 4,096 of each)
      uint32_t own = 0;
#pragma unroll
      for (int j = 0; j < kEvBatch; ++j)
        if (j < n) own += key[j] > last ? 0x10000u : key[j] == last ? 1u : 0u;
      uint32_t incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      uint32_t total;
      const uint32_t ex = ev_warps_before(warp_sum, warp, lane, &total) + incl - own;
      uint32_t m = done_gt + (ex >> 16), e = done_eq + (ex & 0xffffu);
#pragma unroll
      for (int j = 0; j < kEvBatch; ++j) {
        if (j >= n) break;
        const int at = i + j;
        const uint32_t below = m + min(e, ties);   // kept candidates before this one
        if (at % kMvPlaces == 0 && at / kMvPlaces <= a.tiles)
          before[at / kMvPlaces] = lo + static_cast<int>(below);
        const bool gt = key[j] > last, eq = key[j] == last;
        if (gt || (eq && e < ties)) {
          const int place = lo + static_cast<int>(below);
          src[place] = at;
          if (kept != nullptr) kept[place] = at;
        } else if (below == static_cast<uint32_t>(at - lo)) {
          sh_first = at;   // all before it stay: at most one block finds that
        }
        m += gt;
        e += eq;
      }
      done_gt += total >> 16;
      done_eq += total & 0xffffu;
      __syncthreads();
    });
  } else {
    if (gtid == 0) sh_first = lo;
    for (int i = i0 + tid; i < i1; i += kEvThreads)
      if (i % kMvPlaces == 0 && i / kMvPlaces <= a.tiles) before[i / kMvPlaces] = lo;
  }
  for (int j = gtid; j < a.sinks; j += gthreads) {
    src[j] = j;
    if (j % kMvPlaces == 0) before[j / kMvPlaces] = j;
    if (kept != nullptr) kept[j] = j;
  }
  // (the last blocks, and the incomplete one behind them)
  for (int j = gtid; j <= a.recent; j += gthreads)
    if ((hi + j) % kMvPlaces == 0 && (hi + j) / kMvPlaces <= a.tiles)
      before[(hi + j) / kMvPlaces] = a.keep - a.recent + j;
  for (int j = gtid; j < a.recent; j += gthreads) {
    const int place = a.keep - a.recent + j;
    src[place] = hi + j;
    if (kept != nullptr) kept[place] = hi + j;
  }
  cl.sync();
  if (gtid == 0) {
    int first = sh_first;
    for (int c = 1; c < C; ++c) first = min(first, *cl.map_shared_rank(&sh_first, c));
    src[a.keep] = nb;
    a.meta[b] = EvictMeta{a.keep + (tail > 0), min(first, hi), a.keep, nb + (tail > 0)};
    a.len[b] = kBlock * a.keep + tail;
  }
  cl.sync();   // no CTA exits while another reads its shared memory
}

// Moves the kept blocks together, in place: place j takes block src[j] >= j, and src ascends.  A
// CTA takes a tile of places in ticket order, reads its blocks into registers and says so; it
// writes once the tiles whose blocks lie in its places have been read.  Those are lower ones (or
// itself), whose CTAs are running already, so the waits end; they are bounded all the same, and a
// CTA that gave up writes nothing.  Bound by the moved bytes (4 KB of K and V, 132 of compressed
// key and weight, each read and written once): any tile may be on its way.  16 x 64K tokens cut to
// half: 224 us, 4.9 TB/s (75% of the copy rate, in blocks of 1 KB); 1M paged tokens cut to a
// quarter: 120 us.
constexpr int kMvThreads = 512;
constexpr int kMvUnits = kMvPlaces * 4 * 64 / kMvThreads;       // 16-byte units a thread holds

// grid (tiles * batch)
__global__ void __launch_bounds__(kMvThreads, 2) k_evict_move(EvictArgs a) {
  __shared__ int sh_ticket, sh_ok;
  __shared__ int64_t sh_from[kMvPlaces], sh_to[kMvPlaces];   // pool blocks of KV head 0, or -1
  __shared__ int64_t sh_kfrom[kMvPlaces], sh_kto[kMvPlaces];
  const int tid = threadIdx.x;
  pdl_wait();
  if (tid == 0) sh_ticket = atomicAdd(a.ticket, 1);
  __syncthreads();
  // a sequence's tiles in order, the sequences side by side
  const int b = sh_ticket % a.batch, tile = sh_ticket / a.batch;
  const EvictMeta m = a.meta[b];
  if (m.count == 0) return;
  const int32_t* src = a.src + static_cast<int64_t>(b) * (a.keep + 1);
  int32_t* loaded = a.loaded + static_cast<int64_t>(b) * a.tiles;
  float* mass = a.mass + static_cast<int64_t>(b) * a.cap_blocks;
  const int j0 = tile * kMvPlaces, j1 = min(j0 + kMvPlaces, m.count);
  const bool moves = j1 > m.first;
  // the kept blocks that lie in this tile's places, as the tiles that read them: [dep0, dep1)
  const int32_t* before = a.before + static_cast<int64_t>(b) * (a.tiles + 1);
  const int dep0 = moves ? before[tile] / kMvPlaces : 0;
  const int dep1 = moves ? min((before[tile + 1] + kMvPlaces - 1) / kMvPlaces, tile) : 0;
  const int64_t kv = static_cast<int64_t>(a.pg.page_blocks);    // blocks from a head to the next
  if (moves) {
    if (tid < kMvPlaces) {
      const int j = j0 + tid;
      int64_t from = -1, to = -1, kfrom = -1, kto = -1;
      if (j >= m.first && j < j1) {
        from = pool_kv_row(a.pg, b, 0, src[j]);
        to = pool_kv_row(a.pg, b, 0, j);
        kfrom = pool_block(a.pg, b, src[j]);
        kto = pool_block(a.pg, b, j);
        if (from < 0) report_error(a.st, kErrDevice, 311);
        if (to < 0) report_error(a.st, kErrDevice, 312);
      } else {
        to = -2;   // stays where it is
      }
      sh_from[tid] = from;
      sh_to[tid] = to;
      sh_kfrom[tid] = kfrom;
      sh_kto[tid] = j < m.whole ? kto : -1;
    }
    __syncthreads();
  }
  uint4 x[kMvUnits], xk = make_uint4(0u, 0u, 0u, 0u);
  float xm = 0.f;
  // unit i of a thread: place i / 2 (of 16), K (i even) or V, both KV heads: 2 x 64 units of 16
  // bytes by 512 threads is four places at a time
  const int sub = tid >> 7, head = (tid >> 6) & 1, unit = tid & 63;
  if (moves) {
#pragma unroll
    for (int i = 0; i < kMvUnits; ++i) {
      const int p = 4 * (i >> 1) + sub;
      const int64_t from = sh_from[p];
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (from >= 0)
        x[i] = __ldcs(((i & 1) ? a.v_blocks : a.k_blocks) + (from + head * kv * kBlock) * 16 + unit);
    }
    if (tid < kMvPlaces * 8 && sh_kfrom[tid >> 3] >= 0)
      xk = __ldcs(a.kbar + sh_kfrom[tid >> 3] * 8 + (tid & 7));
    if (tid < kMvPlaces && j0 + tid >= m.first && j0 + tid < j1) xm = __ldcg(mass + src[j0 + tid]);
  }
  // Every thread's loads are done behind this barrier, since it takes their values (one release
  // by one thread then does for all: a fence in each warp cost 4 times the move's time).
  uint32_t fold = __float_as_uint(xm) ^ xk.x;
#pragma unroll
  for (int i = 0; i < kMvUnits; ++i) fold ^= moves ? x[i].x : 0u;
  __syncthreads_or(fold == 0x5a5a5a5au);
  if (tid == 0) {
    sh_ok = 1;
    if (a.fault == 0 || b + tile > 0)
      asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(loaded + tile) : "memory");
    if (moves) {
      const uint64_t t0 = globaltimer();
      for (int t = dep0; t < dep1 && sh_ok; ++t) {
        int seen = 0;
        while (true) {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(loaded + t) : "memory");
          if (seen) break;
          if (globaltimer() - t0 > a.wait_ns) {
            sh_ok = 0;
            report_error(a.st, kErrTimeout, 313);
            break;
          }
        }
      }
    }
  }
  if (j0 < j1) {
    // Weights behind the places become zero, each by the tile that holds the next kept block:
    // no other tile reads or writes them.
    const int from = j0 > 0 ? src[j0 - 1] + 1 : 0;
    const int to = j1 == m.count ? m.old : src[j1 - 1] + 1;
    for (int i = max(from, m.count) + tid; i < to; i += kMvThreads) mass[i] = 0.f;
  }
  __syncthreads();
  if (moves && sh_ok) {
#pragma unroll
    for (int i = 0; i < kMvUnits; ++i) {
      const int p = 4 * (i >> 1) + sub;
      const int64_t to = sh_to[p];
      if (to >= 0)
        __stcs(((i & 1) ? a.v_blocks : a.k_blocks) + (to + head * kv * kBlock) * 16 + unit, x[i]);
    }
    if (tid < kMvPlaces * 8 && sh_kto[tid >> 3] >= 0)
      __stcs(a.kbar + sh_kto[tid >> 3] * 8 + (tid & 7), xk);
    if (tid < kMvPlaces && j0 + tid >= m.first && j0 + tid < j1) __stcg(mass + j0 + tid, xm);
  }
}

}  // namespace qsa
