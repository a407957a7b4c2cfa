// qsa_state.cuh -- C ABI of the two memories of a decoding hybrid stack: the gated delta rule from
// and to a pool of states (extend, step), and eviction from a decode cache by accumulated attention
// weight.  Included behind qsa_api.cu, whose helpers (workspace carving, cache views, launches)
// it uses.

#pragma once

#include <atomic>
#include <cmath>
#include <new>
#include <utility>
#include <vector>

#include "qsa_delta.cuh"
#include "qsa_evict.cuh"

namespace {
// The fault that this thread's next calls make (qsa_set_debug_fault), and the limit of their waits.
thread_local int32_t debug_fault = 0;
constexpr int32_t kFaultMove = 3;
constexpr uint32_t kFaultWaitNs = 1000000;   // 1 ms
uint32_t wait_limit(bool fault) { return fault ? kFaultWaitNs : static_cast<uint32_t>(kWaitLimitNs); }
static_assert(kWaitLimitNs < 0xffffffffu, "32-bit limits");

// Launches a kernel in clusters of c CTAs along x, as a programmatic dependent (launch_pdl).
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int c,
                           cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// How many clusters of c CTAs of a kernel run at a time, for kernels whose CTAs fill an SM (a GPC's
// SMs hold whole clusters only: 16 clusters of 8 do not fit into 148 SMs).  Asked once a size, since
// the GPUs of a process are alike; `memo` has an entry a size.
template <typename... KArgs>
int active_clusters(void (*kernel)(KArgs...), int threads, size_t smem, int c, std::atomic<int>* memo) {
  int n = memo[c].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();   // a size that cannot run here
    return 0;
  }
  memo[c].store(n, std::memory_order_relaxed);
  return n;
}
}  // namespace

// ---- the gated delta rule from and to a pool of states ---------------------------------------
namespace {
// Arguments that extend and step share.
qsa_status delta_args(const void* q, const void* k, const void* v, const float* log_alpha,
                      const float* beta, int32_t rows, int32_t key_heads, int32_t heads,
                      float* states, int32_t num_slots, const int32_t* slots, void* out,
                      DeltaArgs* a) {
  for (const void* p : {q, k, v, static_cast<const void*>(states), static_cast<const void*>(out)}) {
    if (!p) return QSA_ERR_INVALID_ARG;
    if (!aligned16(p)) return QSA_ERR_ALIGNMENT;
  }
  if (!log_alpha || !beta) return QSA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(log_alpha), static_cast<const void*>(beta),
                        static_cast<const void*>(slots)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return QSA_ERR_ALIGNMENT;
  if (rows < 1 || rows > 65535 || heads < 1 || heads > 256 || key_heads < 1 ||
      heads % key_heads != 0 || num_slots < 1)
    return QSA_ERR_INVALID_ARG;
  if (!slots && num_slots < rows) return QSA_ERR_INVALID_ARG;
  a->q = static_cast<const __nv_bfloat16*>(q);
  a->k = static_cast<const __nv_bfloat16*>(k);
  a->v = static_cast<const __nv_bfloat16*>(v);
  a->log_alpha = log_alpha;
  a->beta = beta;
  a->slots = slots;
  a->num_slots = num_slots;
  a->rows = rows;
  a->heads = heads;
  a->key_heads = key_heads;
  a->states = states;
  a->out = static_cast<__nv_bfloat16*>(out);
  return QSA_OK;
}

// What a call writes (out, the pool) and what it reads must not overlap: CTAs write outputs and
// states while others still read.  out may be v itself: every value is read by the CTA that
// replaces it, or in a launch before.
bool delta_overlaps(const DeltaArgs& a) {
  struct Range {
    uintptr_t p, n;
  };
  auto range = [](const void* p, int64_t n) { return Range{reinterpret_cast<uintptr_t>(p), static_cast<uintptr_t>(n)}; };
  auto meet = [](Range x, Range y) { return x.p < y.p + y.n && y.p < x.p + x.n; };
  const int64_t keys = a.tokens * a.key_heads * kGdnDim * 2, vals = a.tokens * a.heads * kGdnDim * 2;
  const Range out = range(a.out, vals);
  const Range pool = range(a.states, int64_t(a.num_slots) * a.heads * kGdnDim * kGdnDim * 4);
  if (meet(out, pool) || (a.out != a.v && meet(out, range(a.v, vals)))) return true;
  const Range in[] = {range(a.q, keys), range(a.k, keys), range(a.log_alpha, a.tokens * a.heads * 4),
                      range(a.beta, a.tokens * a.heads * 4)};
  for (const Range& r : in)
    if (meet(out, r) || meet(pool, r)) return true;
  return meet(pool, range(a.v, vals));
}

qsa_status launch_delta_step(const DeltaArgs& a, cudaStream_t s) {
  QSA_CHECK_PDL(launch_pdl(k_delta_step, dim3(a.heads, a.rows, kGdnDim / (16 * kStepRows)), dim3(kStepThreads), 0, s, a));
  return QSA_OK;
}

qsa_status extend_check_cu(const int32_t* h_cu, int32_t num_seqs) {
  if (!h_cu || num_seqs < 1 || num_seqs > 65535 || h_cu[0] != 0) return QSA_ERR_INVALID_ARG;
  for (int32_t i = 0; i < num_seqs; ++i)
    if (h_cu[i + 1] < h_cu[i]) return QSA_ERR_INVALID_ARG;
  return QSA_OK;
}

// How a call of extend runs: heads in passes that keep records and segments within a budget, and
// long sequences cut into segments of seg_chunks chunks where that fills the SMs better.
struct ExtendPlan {
  int64_t records = 0, max_chunks = 0, seg_slots = 0;
  int32_t pass_heads = 1, seg_chunks = 1, seg_first = 1, segs = 1;
  int32_t short_len = 0;   // pieces of at most this many tokens go token by token
  int32_t listed = 0;      // the others: sequences that go in chunks
  bool index = false;      // not all do: they are listed on the device
  size_t o_list = 0, o_rec = 0, o_state = 0, o_trans = 0, total = 0;
};

// Where a call has no longer pieces than 32 tokens, all go token by token (a piece of 30 tokens x 4
// heads: 11.4 us against 24.6 by chunks).  Beside longer pieces, those of at most 16 do where
// they would fill the SMs by themselves, since a walk by chunks holds an SM for 10 us (48 pieces of
// 1 to 64 tokens x 16 heads: 107 us against 128); fewer ride along (7 pieces, one of 1 token, x 4
// heads: 71.1 us against 72.3 with their launch and the list's).
constexpr int32_t kShortAll = 32, kShortMany = 16;
constexpr int64_t kExtendBudget = int64_t(1) << 32;   // bytes of scratch, above which heads run in passes

// Rows of a state that a CTA of the join takes: as few as leave the grid in one wave.
int join_rows(int64_t heads_seqs) {
  int rows = 4;
  while (rows < 16 && heads_seqs * (kGdnDim / rows) > num_sms()) rows *= 2;
  return rows;
}

// Into how long segments sequences are cut, hp heads at a time.  chunks: the lengths of those that
// a cut may split, and how many there are of each; flat: chunks of the others together.
void extend_cuts(const std::vector<std::pair<int64_t, int64_t>>& chunks, int64_t flat, int64_t cuts,
                 int64_t total, int64_t hp, ExtendPlan* p) {
  // Microseconds of the scan, uncut and cut into about k segments: the longest walk, or all walks
  // in waves over the SMs, at what a chunk was measured to take (2.87 with outputs, 2.45 without),
  // and what a launch and a step of the join were.  Cut, first segments run whole beside the inner
  // ones' walks from zero and transitions, then all segments behind the first with outputs.  First
  // ones an eighth shorter, as they write outputs beside walks that do not, or as long as the
  // others, where that saves a shorter sequence a segment.
  constexpr double kOut = 2.87, kWalk = 2.45;
  const double sms = num_sms();
  // (a CTA takes 8 until its first chunk)
  auto waves_of = [&](double l, double all, double chunk) {
    return std::ceil(std::max(1.0, all / sms / l)) * (8 + chunk * l);
  };
  double best = 10 + kOut * std::max(double(p->max_chunks), double(total) * hp / sms);
  int64_t L = std::max<int64_t>(1, p->max_chunks), F = L;
  const int rows = join_rows(int64_t(p->listed) * hp);
  const double waves = std::ceil(double(p->listed) * hp * (kGdnDim / rows) / sms);
  auto consider = [&](int64_t l, int64_t f, int64_t k) {
    double first = double(flat), rest = 0;   // chunks walked by the two passes
    for (const auto& c : chunks) {
      const int64_t segs = delta_segments(c.first, f, l);
      first += double(c.second) * (segs > 1 ? double((2 * segs - 3) * l) : double(c.first));
      rest += double(c.second) * double((segs - 1) * l);
    }
    const double t = waves_of(double(l), first * hp, kWalk) +
                     (f == l ? (kOut - kWalk) * double(l) : 0) +
                     waves * (6 + double(k) * 0.9) + 8 + waves_of(double(l), rest * hp, kOut);
    if (t < best) {
      best = t;
      L = l;
      F = f;
    }
  };
  // where all walks together bound the uncut call, a cut only adds to them
  if (double(total) * hp < double(p->max_chunks) * sms)
    for (int64_t k = 3; k <= cuts; k += 1 + k / 16) {
      const int64_t even = (p->max_chunks + k - 1) / k;
      const int64_t l = (8 * p->max_chunks + 8 * k - 2) / (8 * k - 1);
      consider(l, l - l / 8, k);
      consider(even, even, k);
    }
  p->seg_chunks = static_cast<int32_t>(L);
  p->seg_first = static_cast<int32_t>(F);
  p->segs = static_cast<int32_t>(delta_segments(p->max_chunks, F, L));
}

// False where the host has no memory for it.
bool extend_plan(const int32_t* h_cu, int32_t num_seqs, int32_t heads, ExtendPlan* p) try {
  int64_t short_rows = 0, longest = 0;
  for (int32_t i = 0; i < num_seqs; ++i) {
    const int64_t len = int64_t(h_cu[i + 1]) - h_cu[i];
    longest = std::max(longest, len);
    short_rows += len > 0 && len <= kShortMany;
  }
  p->short_len = longest <= kShortAll ? kShortAll
                 : short_rows * heads >= num_sms() ? kShortMany : 0;
  p->max_chunks = longest > p->short_len ? (longest + kGdnChunk - 1) / kGdnChunk : 0;
  Carver cv;
  p->total = cv.off;
  if (p->max_chunks == 0) return true;
  // the most cuts that are considered, and the longest sequence that no cut splits
  const int64_t cuts = std::min<int64_t>(512, p->max_chunks / 2);
  const int64_t shortest = cuts < 3 ? p->max_chunks : (p->max_chunks + cuts - 1) / cuts * 7 / 8;
  std::vector<std::pair<int64_t, int64_t>> chunks;
  int64_t total = 0, flat = 0;
  for (int32_t i = 0; i < num_seqs; ++i) {
    const int64_t len = int64_t(h_cu[i + 1]) - h_cu[i];
    if (len <= p->short_len) continue;
    const int64_t nc = (len + kGdnChunk - 1) / kGdnChunk;
    ++p->listed;
    total += nc;
    if (nc > shortest) chunks.emplace_back(nc, 1);
    else flat += nc;
  }
  std::sort(chunks.begin(), chunks.end());
  size_t n = 0;   // one entry a length
  for (size_t i = 1; i < chunks.size(); ++i) {
    if (chunks[i].first == chunks[n].first) ++chunks[n].second;
    else chunks[++n] = chunks[i];
  }
  if (!chunks.empty()) chunks.resize(n + 1);
  p->index = p->listed < num_seqs;
  p->records = p->index ? total : h_cu[num_seqs] / kGdnChunk + num_seqs;
  const int64_t tile = int64_t(kGdnDim) * kGdnDim * 4;
  // heads in passes of equal size, the first that fits
  for (int64_t passes = 1;; ) {
    const int64_t hp = (heads + passes - 1) / passes;
    p->pass_heads = static_cast<int32_t>(hp);
    extend_cuts(chunks, flat, cuts, total, hp, p);
    p->seg_slots = 0;
    if (p->segs > 1 && !p->index) p->seg_slots = p->records / p->seg_chunks + num_seqs;
    if (p->segs > 1 && p->index)   // (a sequence that no cut splits is one segment)
      for (const auto& c : chunks)
        p->seg_slots += c.second * (delta_segments(c.first, p->seg_first, p->seg_chunks) - 1);
    const int64_t per_head = p->records * kRecBytes + 2 * p->seg_slots * tile;
    if (hp == 1 || per_head * hp <= kExtendBudget) break;
    const int64_t fit = std::max<int64_t>(1, std::min(hp - 1, kExtendBudget / per_head));
    passes = std::max(passes + 1, (heads + fit - 1) / fit);
  }
  if (p->index) p->o_list = cv.take(static_cast<size_t>(p->listed) * sizeof(int4));
  p->o_rec = cv.take(static_cast<size_t>(p->records * kRecBytes * p->pass_heads));
  if (p->segs > 1) {
    const size_t bytes = static_cast<size_t>(p->seg_slots * p->pass_heads * tile);
    p->o_state = cv.take(bytes);
    p->o_trans = cv.take(bytes);
  }
  p->total = cv.off;
  return true;
} catch (const std::bad_alloc&) {
  return false;
}
}  // namespace

extern "C" size_t qsa_gated_deltanet_extend_workspace_size(const int32_t* h_cu_seqlens,
                                                           int32_t num_seqs, int32_t key_heads,
                                                           int32_t heads) {
  if (extend_check_cu(h_cu_seqlens, num_seqs) != QSA_OK || heads < 1 || heads > 256 ||
      key_heads < 1 || heads % key_heads != 0)
    return 0;
  ExtendPlan p;
  return extend_plan(h_cu_seqlens, num_seqs, heads, &p) ? p.total : 0;
}

namespace {
qsa_status extend_impl(const void* q, const void* k, const void* v, const float* log_alpha,
                       const float* beta, const int32_t* d_cu_seqlens, const int32_t* h_cu_seqlens,
                       int32_t num_seqs, int32_t key_heads, int32_t heads, float* states,
                       int32_t num_slots, const int32_t* slots, void* out, bool zero_skipped,
                       void* workspace, size_t ws_bytes, qsa_stream_t stream) {
  DeltaChunkArgs a{};
  a.d.zero_skipped = zero_skipped;
  qsa_status st = extend_check_cu(h_cu_seqlens, num_seqs);
  if (st == QSA_OK)
    st = delta_args(q, k, v, log_alpha, beta, num_seqs, key_heads, heads, states, num_slots, slots,
                    out, &a.d);
  if (st != QSA_OK) return st;
  if (!d_cu_seqlens || !workspace) return QSA_ERR_INVALID_ARG;
  if (!aligned16(workspace) || reinterpret_cast<uintptr_t>(d_cu_seqlens) % 4 != 0)
    return QSA_ERR_ALIGNMENT;
  ExtendPlan p;
  if (!extend_plan(h_cu_seqlens, num_seqs, heads, &p)) return QSA_ERR_CUDA;
  if (ws_bytes < p.total) return QSA_ERR_WORKSPACE;
  a.d.cu = d_cu_seqlens;
  a.d.tokens = h_cu_seqlens[num_seqs];
  a.d.short_len = p.short_len;
  if (a.d.tokens == 0) return QSA_OK;
  if (delta_overlaps(a.d)) return QSA_ERR_INVALID_ARG;
  if (p.short_len > 0) {
    st = launch_delta_step(a.d, reinterpret_cast<cudaStream_t>(stream));
    if (st != QSA_OK) return st;
  }
  if (p.max_chunks == 0) return QSA_OK;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.rec = ws + p.o_rec;
  a.records = p.records;
  a.listed = p.listed;
  if (p.index) a.list = reinterpret_cast<int4*>(ws + p.o_list);
  a.seg_chunks = p.seg_chunks;
  a.seg_first = p.seg_first;
  a.seg_slots = p.seg_slots;
  if (p.segs > 1) {
    a.seg_state = reinterpret_cast<float*>(ws + p.o_state);
    a.seg_trans = reinterpret_cast<float*>(ws + p.o_trans);
  }
  a.st = dev_status(workspace);
  a.fault = debug_fault;
  a.wait_ns = wait_limit(a.fault == kFaultScan || a.fault == kFaultJoin);
  ScanMaps maps;
  {
    const uint32_t box[3] = {64, 1, kGdnChunk};
    const uint64_t tok = static_cast<uint64_t>(a.d.tokens);
    const uint64_t kd[3] = {kGdnDim, static_cast<uint64_t>(key_heads), tok};
    const uint64_t ks[2] = {kGdnDim * 2, static_cast<uint64_t>(key_heads) * kGdnDim * 2};
    if (!make_tmap(&maps.k, k, 3, kd, ks, box)) return QSA_ERR_CUDA;
  }
  const int prep_smem = static_cast<int>(sizeof(PrepSmem));
  if (!set_smem(k_delta_prep, prep_smem) || !set_smem(k_delta_scan, kScanSmemBytes)) return QSA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned listed = static_cast<unsigned>(p.listed);
  if (p.index)
    QSA_CHECK_PDL(launch_pdl(k_delta_index, dim3(1), dim3(kIndexThreads), 0, s, a, p.short_len > 0));
  for (int32_t h0 = 0; h0 < heads; h0 += p.pass_heads) {
    a.head0 = h0;
    a.nheads = std::min(p.pass_heads, heads - h0);
    // each launch sets up while the one before it finishes
    QSA_CHECK_PDL(launch_pdl(k_delta_prep, dim3(static_cast<unsigned>(p.records), a.nheads),
                             dim3(kPrepThreads), prep_smem, s, a));
    if (p.segs > 1) {
      QSA_CHECK_PDL(launch_pdl(k_delta_scan, dim3(a.nheads, listed, 2 * (p.segs - 1)),
                               dim3(kScanThreads), kScanSmemBytes, s, maps, a, kScanEnds));
      if (p.segs > 2) {
        const int rows = join_rows(int64_t(a.nheads) * p.listed);
        const auto join = rows == 4 ? k_delta_join<4> : rows == 8 ? k_delta_join<8> : k_delta_join<16>;
        if (!set_smem(join, join_smem_bytes(rows))) return QSA_ERR_CUDA;
        QSA_CHECK_PDL(launch_pdl(join, dim3(a.nheads, listed, kGdnDim / rows), dim3(kJoinThreads),
                                 join_smem_bytes(rows), s, a));
      }
    }
    QSA_CHECK_PDL(launch_pdl(k_delta_scan, dim3(a.nheads, listed, std::max(1, p.segs - 1)),
                             dim3(kScanThreads), kScanSmemBytes, s, maps, a,
                             p.segs > 1 ? kScanOutputs : kScanWhole));
  }
  return QSA_OK;
}
}  // namespace

extern "C" qsa_status qsa_gated_deltanet_extend(
    const void* q, const void* k, const void* v, const float* log_alpha, const float* beta,
    const int32_t* d_cu_seqlens, const int32_t* h_cu_seqlens, int32_t num_seqs, int32_t key_heads,
    int32_t heads, float* states, int32_t num_slots, const int32_t* slots, void* out,
    void* workspace, size_t ws_bytes, qsa_stream_t stream) {
  return extend_impl(q, k, v, log_alpha, beta, d_cu_seqlens, h_cu_seqlens, num_seqs, key_heads, heads,
                     states, num_slots, slots, out, false, workspace, ws_bytes, stream);
}

extern "C" qsa_status qsa_gated_deltanet_extend_zeroed(
    const void* q, const void* k, const void* v, const float* log_alpha, const float* beta,
    const int32_t* d_cu_seqlens, const int32_t* h_cu_seqlens, int32_t num_seqs, int32_t key_heads,
    int32_t heads, float* states, int32_t num_slots, const int32_t* slots, void* out,
    void* workspace, size_t ws_bytes, qsa_stream_t stream) {
  return extend_impl(q, k, v, log_alpha, beta, d_cu_seqlens, h_cu_seqlens, num_seqs, key_heads, heads,
                     states, num_slots, slots, out, true, workspace, ws_bytes, stream);
}

extern "C" qsa_status qsa_gated_deltanet_step(const void* q, const void* k, const void* v,
                                              const float* log_alpha, const float* beta,
                                              int32_t batch, int32_t n_new, const int32_t* counts,
                                              int32_t key_heads, int32_t heads, float* states,
                                              int32_t num_slots, const int32_t* slots, void* out,
                                              qsa_stream_t stream) {
  DeltaArgs a{};
  const qsa_status st = delta_args(q, k, v, log_alpha, beta, batch, key_heads, heads, states,
                                   num_slots, slots, out, &a);
  if (st != QSA_OK) return st;
  if (n_new < 0) return QSA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(counts) % 4 != 0) return QSA_ERR_ALIGNMENT;
  if (n_new == 0) return QSA_OK;
  a.n_new = n_new;
  a.counts = counts;
  a.tokens = static_cast<int64_t>(batch) * n_new;
  if (delta_overlaps(a)) return QSA_ERR_INVALID_ARG;
  return launch_delta_step(a, reinterpret_cast<cudaStream_t>(stream));
}

// ---- eviction by accumulated attention weight --------------------------------------------------
namespace {
qsa_status check_cache_geom(const qsa_cache* c) {
  if (!c || c->batch <= 0 || c->batch > 65535 || c->capacity <= 0 || c->capacity % 4 != 0 ||
      c->capacity > QSA_MAX_SEQ_LEN)
    return QSA_ERR_INVALID_ARG;
  return QSA_OK;
}

qsa_status weights_impl(const void* q, const CacheView& view, const int32_t* sel_idx,
                        const int32_t* sel_cnt, int32_t topk, float* mass, void* workspace,
                        size_t ws_bytes, qsa_stream_t stream) {
  const qsa_cache* c = view.c;
  qsa_status st = check_cache_geom(c);
  if (st != QSA_OK) return st;
  st = check_prefill_ptrs({q, c->k_blocks, c->len, sel_idx, sel_cnt, mass, workspace});
  if (st != QSA_OK) return st;
  if (topk < 1 || topk > QSA_MAX_TOPK) return QSA_ERR_INVALID_ARG;
  if (ws_bytes < QSA_WS_HEADER_BYTES) return QSA_ERR_WORKSPACE;
  WeightArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_blocks = static_cast<const __nv_bfloat16*>(c->k_blocks);
  a.len = c->len;
  a.idx = sel_idx;
  a.cnt = sel_cnt;
  a.topk = topk;
  a.cap_blocks = c->capacity / kBlock;
  a.mass = mass;
  a.pg = view.pg;
  a.st = dev_status(workspace);
  // CTAs of 512 threads, one to an SM, in the largest clusters that all run at once: 16 sequences of
  // 60K tokens in clusters of 6 take 10.2 us, 11.9 of 4 and 18.0 of 8 (in turns), 32 of 4 12.2, 64 of
  // 2 17.8.  Sequences beyond clusters of two: CTAs of 256 threads, two to an SM, in as large clusters
  // as keep to that (64 so, of 4: 18.7, and one wide CTA a sequence 28.3).
  static std::atomic<int> memo[kWtMaxCluster + 1];
  const int most = wt_smem_bytes(QSA_MAX_TOPK, 1);
  if (!set_smem(k_block_weights<512>, most) || !set_smem(k_block_weights<256>, most)) return QSA_ERR_CUDA;
  int cluster = kWtMaxCluster;
  while (cluster > 1 && (wt_tiles_per_cta(topk, cluster) < 4 ||
                         active_clusters(k_block_weights<512>, 512, wt_smem_bytes(QSA_MAX_TOPK, cluster),
                                         cluster, memo) < c->batch))
    --cluster;
  const bool wide = cluster > 1;
  if (!wide) {
    cluster = kWtMaxCluster;
    while (cluster > 1 && (int64_t(cluster) * c->batch > 2 * num_sms() || wt_tiles_per_cta(topk, cluster) < 4))
      cluster /= 2;
  }
  const auto kernel = wide ? k_block_weights<512> : k_block_weights<256>;
  const int smem = wt_smem_bytes(topk, cluster);
  QSA_CHECK_PDL(launch_cluster(kernel, dim3(cluster, c->batch), dim3(wide ? 512 : 256), smem, cluster,
                               reinterpret_cast<cudaStream_t>(stream), a));
  return QSA_OK;
}

struct EvictGeom {
  size_t o_meta = 0, o_src = 0, o_loaded = 0, o_before = 0, o_ticket = 0, total = 0;
  int32_t tiles = 0;
};

qsa_status evict_geom(const qsa_cache* c, int32_t keep, int32_t sinks, int32_t recent,
                      EvictGeom* g) {
  const qsa_status st = check_cache_geom(c);
  if (st != QSA_OK) return st;
  if (keep < 1 || keep > QSA_MAX_SEQ_LEN / 4 || sinks < 0 || recent < 0 || sinks > keep ||
      recent > keep - sinks)
    return QSA_ERR_INVALID_ARG;
  Carver cv;
  g->o_meta = cv.take(static_cast<size_t>(c->batch) * sizeof(EvictMeta));
  g->o_src = cv.take(static_cast<size_t>(c->batch) * (static_cast<size_t>(keep) + 1) * 4);
  // a cache that cannot hold more than keep complete blocks has nothing to move
  g->tiles = c->capacity / kBlock > keep ? keep / kMvPlaces + 1 : 0;
  g->o_loaded = cv.take(static_cast<size_t>(c->batch) * g->tiles * 4);
  g->o_before = cv.take(static_cast<size_t>(c->batch) * (g->tiles + 1) * 4);
  g->o_ticket = cv.take(4);
  g->total = cv.off;
  return QSA_OK;
}

qsa_status evict_impl(const CacheView& view, float* mass, int32_t keep, int32_t sinks,
                      int32_t recent, int32_t* kept, void* workspace, size_t ws_bytes,
                      qsa_stream_t stream) {
  const qsa_cache* c = view.c;
  EvictGeom g;
  qsa_status st = evict_geom(c, keep, sinks, recent, &g);
  if (st != QSA_OK) return st;
  st = check_prefill_ptrs({c->k_blocks, c->v_blocks, c->kbar, c->len, mass, workspace});
  if (st != QSA_OK) return st;
  if (kept && !aligned16(kept)) return QSA_ERR_ALIGNMENT;
  if (ws_bytes < g.total) return QSA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  EvictArgs a{};
  a.len = c->len;
  a.mass = mass;
  a.cap_blocks = c->capacity / kBlock;
  a.batch = c->batch;
  a.keep = keep;
  a.sinks = sinks;
  a.recent = recent;
  a.kept = kept;
  a.src = reinterpret_cast<int32_t*>(ws + g.o_src);
  a.meta = reinterpret_cast<EvictMeta*>(ws + g.o_meta);
  a.k_blocks = static_cast<uint4*>(c->k_blocks);
  a.v_blocks = static_cast<uint4*>(c->v_blocks);
  a.kbar = static_cast<uint4*>(c->kbar);
  a.pg = view.pg;
  a.st = dev_status(workspace);
  a.fault = debug_fault == kFaultMove;
  a.wait_ns = wait_limit(a.fault);
  a.tiles = g.tiles;
  a.loaded = reinterpret_cast<int32_t*>(ws + g.o_loaded);
  a.before = reinterpret_cast<int32_t*>(ws + g.o_before);
  a.ticket = reinterpret_cast<int32_t*>(ws + g.o_ticket);
  // The largest clusters that all run at once (a CTA fills an SM), with at least 4,096 weights a CTA
  // (four a thread): below that the cluster's barriers cost more than its reads.  Four sequences of
  // 262,140 tokens cut to almost all: 112 us in clusters of 16, 117 of 8; 16 of 65,535 cut to 64
  // blocks: 26.7 of 4, 40.8 of 8 (in turns).
  static std::atomic<int> memo[kEvMaxCluster + 1];
  int cluster = kEvMaxCluster;
  while (cluster > 1 && a.cap_blocks / cluster < kEvThreads * kEvBatch) cluster /= 2;
  if (cluster > 8 &&
      cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return QSA_ERR_CUDA;
  while (cluster > 1 && active_clusters(k_evict_select, kEvThreads, 0, cluster, memo) < c->batch)
    cluster /= 2;
  QSA_CHECK_PDL(launch_cluster(k_evict_select, dim3(cluster, c->batch), dim3(kEvThreads), 0, cluster, s, a));
  if (g.tiles > 0)
    QSA_CHECK_PDL(launch_pdl(k_evict_move, dim3(static_cast<unsigned>(g.tiles) * c->batch),
                             dim3(kMvThreads), 0, s, a));
  return QSA_OK;
}
}  // namespace

extern "C" {

qsa_status qsa_set_debug_fault(int32_t fault) {
  if (fault < 0 || fault > kFaultMove) return QSA_ERR_INVALID_ARG;
  debug_fault = fault;
  return QSA_OK;
}

qsa_status qsa_accumulate_weights(const void* q, const qsa_cache* cache, const int32_t* sel_idx,
                                  const int32_t* sel_cnt, int32_t topk, float* mass,
                                  void* workspace, size_t ws_bytes, qsa_stream_t stream) {
  if (!cache) return QSA_ERR_INVALID_ARG;
  return weights_impl(q, contiguous_view(cache), sel_idx, sel_cnt, topk, mass, workspace, ws_bytes,
                      stream);
}

qsa_status qsa_accumulate_weights_paged(const void* q, const qsa_paged_cache* cache,
                                        const int32_t* sel_idx, const int32_t* sel_cnt,
                                        int32_t topk, float* mass, void* workspace,
                                        size_t ws_bytes, qsa_stream_t stream) {
  CacheView view;
  const qsa_status st = paged_view(cache, &view);
  if (st != QSA_OK) return st;
  return weights_impl(q, view, sel_idx, sel_cnt, topk, mass, workspace, ws_bytes, stream);
}

size_t qsa_evict_workspace_size(const qsa_cache* cache, int32_t keep_blocks, int32_t sink_blocks,
                                int32_t recent_blocks) {
  EvictGeom g;
  return evict_geom(cache, keep_blocks, sink_blocks, recent_blocks, &g) == QSA_OK ? g.total : 0;
}

qsa_status qsa_evict(const qsa_cache* cache, float* mass, int32_t keep_blocks, int32_t sink_blocks,
                     int32_t recent_blocks, int32_t* kept, void* workspace, size_t ws_bytes,
                     qsa_stream_t stream) {
  if (!cache) return QSA_ERR_INVALID_ARG;
  return evict_impl(contiguous_view(cache), mass, keep_blocks, sink_blocks, recent_blocks, kept,
                    workspace, ws_bytes, stream);
}

qsa_status qsa_evict_paged(const qsa_paged_cache* cache, float* mass, int32_t keep_blocks,
                           int32_t sink_blocks, int32_t recent_blocks, int32_t* kept,
                           void* workspace, size_t ws_bytes, qsa_stream_t stream) {
  CacheView view;
  const qsa_status st = paged_view(cache, &view);
  if (st != QSA_OK) return st;
  return evict_impl(view, mass, keep_blocks, sink_blocks, recent_blocks, kept, workspace, ws_bytes,
                    stream);
}

}  // extern "C"
