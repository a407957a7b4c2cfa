// qsa_delta.cuh -- the gated delta rule from and to a pool of states: token by token for
// decoding rows, in chunks for pieces of prompts.  (The layer over whole sequences from a zero
// state is in qsa_gdn.cuh.)
//
// Per row (sequence) and value head, with the state S (d_v x d_k, fp32) kept in a slot of a
// caller-owned pool [slots][heads][128 (v)][128 (k)]:
//     S <- a S + beta (v - a S k) k^T,   o = S q,      a = exp(max(log_alpha, -87)).
// heads / key_heads value heads in a row share one key (and query) head.
//
// A row is skipped (state and outputs untouched, or outputs zeroed where zero_skipped says so) when
// its slot lies outside the pool, which is how rows of a padded batch are marked, or when an earlier
// row of the call names the same slot: the first row owns it.

#pragma once

#include <cuda_fp16.h>

#include "qsa_common.cuh"
#include "qsa_gdn.cuh"

namespace qsa {

struct DeltaArgs {
  const __nv_bfloat16* q;   // [tokens][key_heads][128]
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;   // [tokens][heads][128]
  const float* log_alpha;   // [tokens][heads]
  const float* beta;
  const int32_t* cu;        // [rows+1]: row r's tokens are cu[r] .. cu[r+1]-1; or null:
  int32_t n_new;            //   row r's tokens are r*n_new .. r*n_new + count - 1
  const int32_t* counts;    // [rows] (clamped to 0..n_new) or null for n_new each
  const int32_t* slots;     // [rows] or null: row r has slot r
  int32_t num_slots;
  int32_t rows;
  int64_t tokens;           // rows of q, k, v and out
  int32_t short_len;        // with cu: rows of at most this many tokens are taken token by token
  int32_t heads, key_heads;
  float* states;            // [num_slots][heads][128][128]
  __nv_bfloat16* out;       // [tokens][heads][128]
  bool zero_skipped;        // rows of skipped sequences become zero in out
};

// Row r's first token and number of tokens.
__device__ __forceinline__ int64_t delta_row_tokens(const DeltaArgs& a, int r, int64_t* n) {
  int64_t begin, end;
  if (a.cu != nullptr) {
    begin = a.cu[r];
    end = a.cu[r + 1];
  } else {
    int c = a.counts != nullptr ? a.counts[r] : a.n_new;
    c = c < 0 ? 0 : (c > a.n_new ? a.n_new : c);
    begin = static_cast<int64_t>(r) * a.n_new;
    end = begin + c;
  }
  if (begin < 0 || end > a.tokens) end = begin = 0;   // lengths that disagree with the host's
  *n = end - begin;
  return begin;
}

// Whether an earlier row names row r's slot.  All threads of the block call
// it, and all get the answer.
__device__ __forceinline__ bool delta_slot_taken(const DeltaArgs& a, int r, int slot) {
  if (a.slots == nullptr) return false;
  int hit = 0;
  for (int i = threadIdx.x; i < r; i += blockDim.x) hit |= a.slots[i] == slot;
  return __syncthreads_or(hit) != 0;
}

// A log gate, no smaller than the reset's; NaN stays (fmaxf would make a reset of it).
__device__ __forceinline__ float delta_gate(float la) {
  return la < kGdnMinLogAlpha ? kGdnMinLogAlpha : la;
}

__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float* f) {
  f[0] = __uint_as_float(w << 16);
  f[1] = __uint_as_float(w & 0xffff0000u);
}

// ---------------------------------------------------------------------------------------
// Token by token.  Eight lanes hold one value row of S (16 key columns each, in four groups of
// four so that a row's loads are 128-byte segments), two rows a thread, so a block of 128 threads
// holds 32 rows and the grid (heads, rows, 4) covers S.  The state
// stays in registers over a row's tokens: it is read once and written once.  With
// o = a S q + u (k.q), u = beta (v - a S k), both dots of a token come from the old state in one
// pass, and the reductions are three shuffles.  A token's inputs are fetched while the one before
// it is taken.  Bound by the state's bytes: 128 KB per (row, head) against about 4.5 KB of
// everything else at one token.  64 rows x 32 heads x 1 token: 45 us, 6.0 TB/s, 92% of the measured
// copy rate; 24 rows of up to 5 tokens x 16 heads: 10 us a call (its states' bytes take 6.9).
constexpr int kStepThreads = 128;
constexpr int kStepRows = 2;

__global__ void __launch_bounds__(kStepThreads) k_delta_step(DeltaArgs a) {
  const int tid = threadIdx.x, l8 = tid & 7, grp = tid >> 3;   // 16 groups of 8 lanes
  const int h = blockIdx.x, r = blockIdx.y;
  const int v0 = (blockIdx.z * 16 + grp) * kStepRows;
  pdl_wait();      // launched as a programmatic dependent of the caller's last kernel, which is done
  pdl_trigger();   // before any kernel behind this one starts
  int64_t n;
  const int64_t t0 = delta_row_tokens(a, r, &n);
  const int slot = a.slots != nullptr ? a.slots[r] : r;
  if (n <= 0 || (a.cu != nullptr && n > a.short_len)) return;
  auto skip = [&]() {
    if (a.zero_skipped && l8 == 0)
      for (int64_t t = t0; t < t0 + n; ++t)
        for (int i = 0; i < kStepRows; ++i)
          a.out[(t * a.heads + h) * kGdnDim + v0 + i] = __float2bfloat16(0.f);
  };
  if (slot < 0 || slot >= a.num_slots) {
    skip();
    return;
  }
  const int kh = h / (a.heads / a.key_heads);
  float* st = a.states +
              ((static_cast<int64_t>(slot) * a.heads + h) * kGdnDim + v0) * kGdnDim + 4 * l8;
  float4 S[kStepRows][4];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      S[i][j] = __ldcs(reinterpret_cast<const float4*>(st + i * kGdnDim + 32 * j));
  // a token's inputs, on their way while the one before it is taken
  uint2 wq[4], wk[4];
  float la, beta;
  __nv_bfloat16 wv[kStepRows];
  auto fetch = [&](int64_t t) {
    const uint2* qp = reinterpret_cast<const uint2*>(a.q + (t * a.key_heads + kh) * kGdnDim) + l8;
    const uint2* kp = reinterpret_cast<const uint2*>(a.k + (t * a.key_heads + kh) * kGdnDim) + l8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wq[j] = qp[8 * j];
      wk[j] = kp[8 * j];
    }
    la = a.log_alpha[t * a.heads + h];
    beta = a.beta[t * a.heads + h];
    const __nv_bfloat16* vp = a.v + (t * a.heads + h) * kGdnDim + v0;
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) wv[i] = vp[i];
  };
  fetch(t0);
  if (delta_slot_taken(a, r, slot)) {
    skip();
    return;
  }
  for (int64_t t = t0; t < t0 + n; ++t) {
    const float al = expf(delta_gate(la));
    const float bt = beta;
    float q[16], k[16], x[kStepRows];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      unpack_bf16x2(wq[j].x, q + 4 * j);
      unpack_bf16x2(wq[j].y, q + 4 * j + 2);
      unpack_bf16x2(wk[j].x, k + 4 * j);
      unpack_bf16x2(wk[j].y, k + 4 * j + 2);
    }
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) x[i] = __bfloat162float(wv[i]);
    if (t + 1 < t0 + n) fetch(t + 1);
    float kq = 0.f, sk[kStepRows], sq[kStepRows];
#pragma unroll
    for (int e = 0; e < 16; ++e) kq = fmaf(k[e], q[e], kq);
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      const float* s = reinterpret_cast<const float*>(S[i]);
      sk[i] = sq[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        sk[i] = fmaf(s[e], k[e], sk[i]);
        sq[i] = fmaf(s[e], q[e], sq[i]);
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      kq += __shfl_xor_sync(0xffffffffu, kq, o);
#pragma unroll
      for (int i = 0; i < kStepRows; ++i) {
        sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], o);
        sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
      }
    }
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      const float u = bt * (x[i] - al * sk[i]);
      float* s = reinterpret_cast<float*>(S[i]);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = fmaf(u, k[e], al * s[e]);
      if (l8 == 0)
        a.out[(t * a.heads + h) * kGdnDim + v0 + i] = __float2bfloat16(fmaf(u, kq, al * sq[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __stcs(reinterpret_cast<float4*>(st + i * kGdnDim + 32 * j), S[i][j]);
}

// ---------------------------------------------------------------------------------------
// In chunks.  With S0 the state that a chunk of C = 64 tokens is entered with, g_t the running
// sum of its log gates, L the strictly lower part of diag(beta) (e^(g_t - g_j) k_t.k_j) and
// Tu = (I + L)^-1,
//     T = Tu diag(beta),   W = T diag(e^g) K,   U = T V - W S0^T      (what the tokens write)
//     O = diag(e^g) Q S0^T + M U,   M_tj = e^(g_t - g_j) q_t.k_j  for j <= t
//     S = e^(g_C) S0 + (diag(e^(g_C - g)) U)^T K.
// T V, W and M do not depend on the state: k_delta_prep forms them for every chunk and head at
// once and leaves them in a record; k_delta_scan walks the chunks in order with two dependent
// products a chunk (W S0^T, then U^T K) on the tcgen05 tensor cores.  Where the walks do not fill
// the SMs, sequences are cut into segments: a segment is affine in the state it is entered with,
// E -> E P + S, so a first pass of the scan finds S (from zero) and P (from the identity, without
// writes) of the inner segments while the first ones run whole, k_delta_join takes the states
// through, and a second pass writes the other segments' outputs.
//
// q, k and v are bf16 and exact as operands; the fp32 operands go in as parts.  T, U and M: three
// bf16 parts each, x = hi + mid + lo to 2^-24 of x (of M U, the products of at least 2^-16).  W and
// S: two fp16 parts each (hi + lo to 2^-22 of x), scaled by powers of two (a row of S, a row of W) so
// that fp16 holds them; the product lo lo (2^-24) of W S is left out.  So an output is rounded to
// fewer than 22 bits once, to bf16 at its end.  Sums are fp32 throughout, running log gates fp64 (a
// reset adds -87, after which fp32 differences would be off by 2^-11).

// A record: operand tiles in the layout that the tensor core reads (rows of 128 bytes, 16-byte
// words exchanged within 8 rows), then the gates.
constexpr int kRecW = 0;                    // -W [64 t][128 d] fp16, rows scaled, two 64-column panels: hi, lo each
constexpr int kRecU = 32768;                // T V [64 t][128 v] fp32
constexpr int kRecM = 65536;                // M bf16, hi, mid, lo: its lower triangle by 16 columns j
constexpr int kRecQ = 80896;                // Q [64 t][128 d] fp16, rows scaled (two panels)
constexpr int kRecGate = 97280;             // fp32 [256], as follows
constexpr int kRecBytes = 98304;
constexpr int kGateQ = 0;                   // [64] e^g over the scale of the Q row
constexpr int kGateU = 64;                  // [64] e^(g_C - g)
constexpr int kGateW = 128;                 // [64] 1 over the scale of the W row
constexpr int kGateC = 192;                 // e^(g_C)
constexpr int kGateK = 193;                 // the largest |K|

// Byte of element (r, c) of a [rows][64] bf16 tile.
__host__ __device__ constexpr uint32_t tile_byte(uint32_t r, uint32_t c) {
  return r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2;
}

// Columns 16 k .. of M, rows t >= 16 k: rows of 32 bytes whose two 16-byte words change places every
// 4 rows, the four panels one behind the other.
constexpr int kMPart = 5120;
__host__ __device__ constexpr uint32_t m_panel(uint32_t k) { return 2048 * k - 256 * k * (k - 1); }
__host__ __device__ constexpr uint32_t m_byte(uint32_t t, uint32_t j) {
  const uint32_t r = t - (j & ~15u);
  return m_panel(j >> 4) + r * 32 + ((((j >> 3) ^ (r >> 2)) & 1) << 4) + (j & 7) * 2;
}
static_assert(m_panel(4) == kMPart && 3 * kMPart <= kRecQ - kRecM, "M's parts");

// First record of sequence s whose tokens start at `begin`: sequences never overlap, since
// floor(end / 64) - floor(begin / 64) + 1 >= ceil((end - begin) / 64).
__host__ __device__ constexpr int64_t delta_first_record(int64_t begin, int s) {
  return begin / kGdnChunk + s;
}

// Segments of a sequence of nc chunks.
__host__ __device__ constexpr int64_t delta_segments(int64_t nc, int64_t seg_first, int64_t seg_chunks) {
  return nc <= seg_first ? 1 : 1 + (nc - seg_first + seg_chunks - 1) / seg_chunks;
}

struct DeltaChunkArgs {
  DeltaArgs d;
  int32_t head0, nheads;     // the heads of this pass
  // The sequences that go in chunks: {row, first record, first segment slot, 0}, row -1 for none; or
  // null where all do.
  int4* list;
  int32_t listed;            // as the host counts them
  int64_t records;
  unsigned char* rec;        // [records][nheads][kRecBytes]
  int32_t seg_chunks;        // chunks of a segment (a sequence is walked by one CTA a segment)
  int32_t seg_first;         // and of a sequence's first segment, at most as many
  int64_t seg_slots;
  float* seg_state;          // [segment slots][nheads][128][128]: state at the segment's end
  float* seg_trans;          // the same shape: the segment's transition (P of S0 P + S)
  DevStatus st;
  uint32_t wait_ns;          // limit of every wait
  int32_t fault;             // testing: a copy that block (0, 0, 0) does not issue (kFault..)
};
constexpr int32_t kFaultScan = 1, kFaultJoin = 2;

// The i-th sequence that goes in chunks.
struct DeltaPiece {
  int row;            // -1: none
  int64_t begin, len;
  int64_t record, segment;   // its first record and segment slot
};
__device__ __forceinline__ DeltaPiece delta_piece(const DeltaChunkArgs& ca, int i) {
  DeltaPiece p;
  p.row = i;
  p.begin = p.len = p.record = p.segment = 0;
  if (ca.list != nullptr) {
    const int4 x = __ldcg(ca.list + i);
    p.row = x.x;
    p.record = x.y;
    p.segment = x.z;
    if (p.row < 0) return p;
  }
  p.begin = delta_row_tokens(ca.d, p.row, &p.len);
  if (ca.list == nullptr) {
    p.record = delta_first_record(p.begin, p.row);
    p.segment = p.record / ca.seg_chunks + p.row;     // as records: segments never overlap
  }
  return p;
}

// ---- k_delta_index: one CTA that lists the sequences in chunks --------------------------------
// Where a call has sequences that go token by token, or empty ones: without the list each would
// hold a record a head (96 KB) and a CTA in every launch.  It runs beside the former (`beside`: the
// launch before is theirs, and has itself waited for all before it).
constexpr int kIndexThreads = 1024;

__global__ void __launch_bounds__(kIndexThreads) k_delta_index(DeltaChunkArgs ca, bool beside) {
  __shared__ int3 part[32];
  const DeltaArgs& a = ca.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!beside) pdl_wait();
  int3 done = make_int3(0, 0, 0);   // sequences, records and segment slots before this turn's
  for (int r0 = 0; r0 < a.rows; r0 += kIndexThreads) {
    const int r = r0 + tid;
    int64_t len = 0;
    if (r < a.rows) delta_row_tokens(a, r, &len);
    int3 own = make_int3(0, 0, 0);
    if (len > a.short_len) {
      const int64_t nc = (len + kGdnChunk - 1) / kGdnChunk;
      own = make_int3(1, static_cast<int>(nc),
                      static_cast<int>(delta_segments(nc, ca.seg_first, ca.seg_chunks) - 1));
    }
    int3 x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int3 y = make_int3(__shfl_up_sync(0xffffffffu, x.x, o), __shfl_up_sync(0xffffffffu, x.y, o),
                               __shfl_up_sync(0xffffffffu, x.z, o));
      if (lane >= o) x = make_int3(x.x + y.x, x.y + y.y, x.z + y.z);
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int3 at = make_int3(done.x + x.x - own.x, done.y + x.y - own.y, done.z + x.z - own.z);
    for (int w = 0; w < 32; ++w) {
      const int3 y = part[w];
      done = make_int3(done.x + y.x, done.y + y.y, done.z + y.z);
      if (w < warp) at = make_int3(at.x + y.x, at.y + y.y, at.z + y.z);
    }
    if (own.x) {   // (lengths that disagree with the host's: what has no space is left out)
      const bool fits = at.x < ca.listed && at.y + own.y <= ca.records && at.z + own.z <= ca.seg_slots;
      if (!fits) report_error(ca.st, kErrDevice, 321);
      if (at.x < ca.listed) ca.list[at.x] = make_int4(fits ? r : -1, fits ? at.y : 0x7fffffff, at.z, 0);
    }
    __syncthreads();
  }
  for (int i = done.x + tid; i < ca.listed; i += kIndexThreads)
    ca.list[i] = make_int4(-1, 0x7fffffff, 0, 0);
  if (beside) pdl_wait();   // the launches after this one count on all before it
}

// Instruction descriptor: kind::f16 with f16 A/B, fp32 D, dense.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn_major, int b_mn_major) {
  return idesc_bf16_f32(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}

// Shared-memory descriptor of a K-major tile with rows of 32 bytes, 8-row atoms `sbo_bytes` apart,
// words exchanged as m_byte has them (the 32-byte swizzle).
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t saddr, uint32_t sbo_bytes) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32 | 1ull << 46 | 6ull << 61;
}

// x -= lo(h), y -= hi(h): one mixed-precision instruction each
__device__ __forceinline__ void take_bf16x2(uint32_t h, float* x, float* y) {
  asm("{\n\t.reg .b16 l, h, m;\n\tmov.b32 {l, h}, %2;\n\tmov.b16 m, 0xBF80;\n\t"
      "fma.rn.f32.bf16 %0, l, m, %0;\n\tfma.rn.f32.bf16 %1, h, m, %1;\n\t}"
      : "+f"(*x), "+f"(*y)
      : "r"(h));
}
__device__ __forceinline__ void take_f16x2(uint32_t h, float* x, float* y) {
  asm("{\n\t.reg .b16 l, h, m;\n\tmov.b32 {l, h}, %2;\n\tmov.b16 m, 0xBC00;\n\t"
      "fma.rn.f32.f16 %0, l, m, %0;\n\tfma.rn.f32.f16 %1, h, m, %1;\n\t}"
      : "+f"(*x), "+f"(*y)
      : "r"(h));
}
__device__ __forceinline__ uint32_t pack_f16x2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x = hi + mid + lo, 8 bits each, the upper ones cut off: exact, in fewer cycles than rounded parts
__device__ __forceinline__ void split3_bf16x2(float x, float y, uint32_t* hi, uint32_t* mid,
                                              uint32_t* lo) {
  *hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  take_bf16x2(*hi, &x, &y);
  *mid = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  take_bf16x2(*mid, &x, &y);
  *lo = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}
__device__ __forceinline__ void split_f16x2(float x, float y, uint32_t* hi, uint32_t* lo) {
  *hi = pack_f16x2(x, y);
  take_f16x2(*hi, &x, &y);
  *lo = pack_f16x2(x, y);
}
// The power of two that brings a largest magnitude m into [2^7, 2^8), and its inverse (rows of
// zeros, or below 2^-119, take that of 2^-119).
__device__ __forceinline__ float row_scale(float m, float* inverse) {
  const uint32_t e = max(__float_as_uint(m) >> 23, 8u);
  *inverse = __uint_as_float((e - 7u) << 23);
  return __uint_as_float((261u - e) << 23);
}

// the larger magnitudes of two pairs of bf16
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t x) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
  return r;
}
// a pair of bf16 times a power of two (as bf16), in fp16
__device__ __forceinline__ uint32_t scale_to_f16x2(uint32_t x, uint16_t s) {
  float lo = 0.f, hi = 0.f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tfma.rn.f32.bf16 %0, l, %3, %0;\n\t"
      "fma.rn.f32.bf16 %1, h, %3, %1;\n\t}"
      : "+f"(lo), "+f"(hi)
      : "r"(x), "h"(s));
  return pack_f16x2(lo, hi);
}

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a b, 16 x 8 x 16, bf16 operands, fp32 accumulation
__device__ __forceinline__ void delta_mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes global -> shared, or 16 zero bytes
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
// until the shared memory of this thread's stores has been read
__device__ __forceinline__ void bulk_store_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}

// ---- k_delta_prep: one CTA of 256 threads per (record, head) ---------------------------------
// Warp MMAs, since the parts between the products (decays, the inverse by 16 x 16 blocks, the
// splits into parts) outweigh them and take registers, and since with four CTAs an SM the phases
// of one fill the gaps of another.  The record leaves in pieces, out of the space of an operand
// that is done with: Q becomes the scaled fp16 Q in place, then holds M, then V; K and Tu become W.
// 16,384 chunks (8 x 8,192 tokens x 16 heads): 570 us, 5.2 us of an SM a chunk, bound by shared
// memory (68% of its cycles; instructions issue in 56%; three CTAs an SM take as long); the bytes
// (48 KB in, 96 KB out) would take 360 us.
constexpr int kPrepThreads = 256;
constexpr int kPrepLdA = kGdnChunk + 8;   // fp32 row stride of L / Tu: 8 rows x 4 pairs without conflicts
struct PrepSmem {
  unsigned char k[16384];                 // [64 t][128 d] bf16 as two tiles of 64 columns
  float a[kGdnChunk * kPrepLdA];          // L, then Tu
  unsigned char q[16384];
  float gate[256];
  float g_hi[kGdnChunk], g_lo[kGdnChunk]; // running log gate in base 2, as a sum
  float beta[kGdnChunk], eg[kGdnChunk], beg[kGdnChunk];   // beta, e^g, their product
  float wmax[2][kGdnChunk], kmax[4];
};
static_assert(16384 + 4 * kGdnChunk * kPrepLdA >= 32768, "W fits");
static_assert(sizeof(PrepSmem) <= 55 * 1024, "four CTAs an SM");

__device__ __forceinline__ float exp2_approx(float x) {   // 2 ulp; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// z += left (16 x 16) right (16 x 8) of S.a, operands in three bf16 parts
__device__ __forceinline__ void prep_mma3(float* z, const float* left, const float* right, int gq,
                                          int tq) {
  uint32_t x[3][4], y[3][2];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = *reinterpret_cast<const float2*>(left + (gq + 8 * (e & 1)) * kPrepLdA + 2 * tq +
                                                      8 * (e >> 1));
    split3_bf16x2(v.x, v.y, &x[0][e], &x[1][e], &x[2][e]);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float* p = right + (2 * tq + 8 * e) * kPrepLdA + gq;
    split3_bf16x2(p[0], p[kPrepLdA], &y[0][e], &y[1][e], &y[2][e]);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int j = 0; i + j < 3; ++j) delta_mma(z, x[i], y[j][0], y[j][1]);
}
__device__ __forceinline__ void prep_put(float* to, const float* z, float sign, int gq, int tq) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<float2*>(to + (gq + 8 * i) * kPrepLdA + 2 * tq) =
        make_float2(sign * z[2 * i], sign * z[2 * i + 1]);
}

__global__ void __launch_bounds__(kPrepThreads, 4) k_delta_prep(DeltaChunkArgs ca) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  PrepSmem& S = *reinterpret_cast<PrepSmem*>(smem_raw);
  const DeltaArgs& a = ca.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int64_t r = blockIdx.x;
  pdl_wait();      // the caller's last kernel
  pdl_trigger();   // the scan sets up while the last of these run
  // the last sequence whose first record is not past r, 256 candidates at a time
  int seq = 0;
  for (int step = ca.listed > kPrepThreads ? kPrepThreads : 1; step > 0; step = step > 1 ? 1 : 0) {
    const int64_t s = seq + static_cast<int64_t>(tid) * step;
    const bool in = s < ca.listed &&
                    (ca.list != nullptr ? __ldcg(&ca.list[s].y) : delta_first_record(a.cu[s], static_cast<int>(s))) <= r;
    const int m = __syncthreads_count(in);
    seq += (m > 0 ? m - 1 : 0) * step;
  }
  const DeltaPiece piece = delta_piece(ca, seq);
  const int64_t begin = piece.begin, len = piece.len, c = r - piece.record;
  if (c < 0 || c * kGdnChunk >= len || len <= a.short_len) return;
  const int64_t t0 = begin + c * kGdnChunk;
  const int n = static_cast<int>(len - c * kGdnChunk < kGdnChunk ? len - c * kGdnChunk : kGdnChunk);
  const int h = ca.head0 + blockIdx.y, kh = h / (a.heads / a.key_heads);
  unsigned char* rec = ca.rec + (r * ca.nheads + blockIdx.y) * static_cast<int64_t>(kRecBytes);
  asm volatile("" : "+l"(rec));   // one register pair, not what it is computed from (spills cost 50 us)
  float la[2] = {0.f, 0.f}, bt[2] = {0.f, 0.f};
  if (warp == 0) {   // two tokens a lane
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      if (t < n) {
        la[i] = delta_gate(a.log_alpha[(t0 + t) * a.heads + h]);
        bt[i] = a.beta[(t0 + t) * a.heads + h];
      }
    }
  }
  const uint32_t sk = smem_u32(S.k), sq = smem_u32(S.q);
  for (int e = tid; e < kGdnChunk * 16; e += kPrepThreads) {
    const int t = e >> 4, w = e & 15;
    const int64_t off = ((t0 + (t < n ? t : 0)) * a.key_heads + kh) * kGdnDim + 8 * w;
    const uint32_t at = 8192 * (w >> 3) + tile_byte(t, 8 * (w & 7));
    cp_async16(sk + at, a.k + off, t < n);
    cp_async16(sq + at, a.q + off, t < n);
  }
  float* gate = S.gate;
  if (warp == 0) {
    // an inclusive scan of the clamped log gates, in base 2
    const double l2e = 1.4426950408889634;
    const double l0 = l2e * la[0], pair = l0 + l2e * la[1];
    double incl = pair;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const double g2[2] = {incl - pair + l0, incl}, gc = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      S.g_hi[t] = static_cast<float>(g2[i]);
      S.g_lo[t] = static_cast<float>(g2[i] - static_cast<double>(S.g_hi[t]));
      S.beta[t] = bt[i];
      S.eg[t] = exp2f(static_cast<float>(g2[i]));
      S.beg[t] = bt[i] * S.eg[t];
      gate[kGateU + t] = exp2f(static_cast<float>(gc - g2[i]));
    }
    if (lane == 0) gate[kGateC] = exp2f(static_cast<float>(gc));
  }
  cp_async_wait_all();
  __syncthreads();
  const bool isq = warp >= 4;
  // 16 rows; the causal mask leaves rb + 1 parts of four, so that the two warps of a scheduler
  // take rb and 3 - rb
  int rb = isq ? 3 - (warp & 3) : warp & 3;
  int ta = 16 * rb + gq, tb = ta + 8;
  float acc[8][4];
  {
    // K K^T (warps 0..3) and Q K^T (4..7), the columns that the causal mask keeps
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    const uint32_t ap = isq ? sq : sk;
    const int ar = 16 * rb + (lane & 15), ac = 8 * (lane >> 4), br = lane & 7, bc = 8 * (lane >> 3);
#pragma unroll 1
    for (int k0 = 0; k0 < kGdnDim; k0 += 32) {
      const uint32_t panel = 8192 * (k0 >> 6);
      uint32_t fa[2][4];
      ldsm4(fa[0], ap + panel + tile_byte(ar, (k0 & 63) + ac));
      ldsm4(fa[1], ap + panel + tile_byte(ar, (k0 & 63) + 16 + ac));
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        if (nt < 2 * (rb + 1)) {
          uint32_t fb[4];
          ldsm4(fb, sk + panel + tile_byte(8 * nt + br, (k0 & 63) + bc));
          delta_mma(acc[nt], fa[0], fb[0], fb[1]);
          delta_mma(acc[nt], fa[1], fb[2], fb[3]);
        }
      }
    }
    const float ha = S.g_hi[ta], hb = S.g_hi[tb], la2 = S.g_lo[ta], lb2 = S.g_lo[tb];
    const float ba = isq ? 1.f : S.beta[ta], bb = isq ? 1.f : S.beta[tb];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt < 2 * (rb + 1)) {
        const float2 jh = *reinterpret_cast<const float2*>(&S.g_hi[8 * nt + 2 * tq]);
        const float2 jl = *reinterpret_cast<const float2*>(&S.g_lo[8 * nt + 2 * tq]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = e < 2 ? ta : tb, j = 8 * nt + 2 * tq + (e & 1);
          const float d = ((e < 2 ? ha : hb) - ((e & 1) ? jh.y : jh.x)) +
                          ((e < 2 ? la2 : lb2) - ((e & 1) ? jl.y : jl.x));
          const bool in = isq ? j <= t : j < t;
          acc[nt][e] = in ? exp2_approx(d) * ((e < 2 ? ba : bb) * acc[nt][e]) : 0.f;
        }
      }
    }
    if (!isq) {
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const int j = 8 * nt + 2 * tq;
        *reinterpret_cast<float2*>(&S.a[ta * kPrepLdA + j]) = make_float2(acc[nt][0], acc[nt][1]);
        *reinterpret_cast<float2*>(&S.a[tb * kPrepLdA + j]) = make_float2(acc[nt][2], acc[nt][3]);
      }
    }
  }
  __syncthreads();
  if (isq) {
    // Q as fp16 with scaled rows, in place (half a row a thread); then M in its space
    const int t = (tid - 128) >> 1, half = tid & 1;
    unsigned char* p = S.q + 8192 * half;
    uint32_t m2 = 0u;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      // the two panels' words of a row lie in the same banks: the halves take them in turn
      const uint4 x = *reinterpret_cast<const uint4*>(p + tile_byte(t, 8 * (i ^ (4 * half))));
      m2 = max_abs_bf16x2(max_abs_bf16x2(m2, x.x), x.y);
      m2 = max_abs_bf16x2(max_abs_bf16x2(m2, x.z), x.w);
    }
    float m = fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    float inv;
    const uint16_t sc = static_cast<uint16_t>(__float_as_uint(row_scale(m, &inv)) >> 16);
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      uint4* at = reinterpret_cast<uint4*>(p + tile_byte(t, 8 * (i ^ (4 * half))));
      const uint4 x = *at;
      *at = make_uint4(scale_to_f16x2(x.x, sc), scale_to_f16x2(x.y, sc), scale_to_f16x2(x.z, sc),
                       scale_to_f16x2(x.w, sc));
    }
    if (half == 0) gate[kGateQ + t] = S.eg[t] * inv;
    fence_proxy_async_smem();
    named_barrier_sync(1, 128);
    if (tid == 128) {
      bulk_store(rec + kRecQ, S.q, 16384);
      bulk_store_wait();
    }
    named_barrier_sync(1, 128);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt < 2 * (rb + 1)) {
        const int j = 8 * nt + 2 * tq;
        const float* x = acc[nt];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t part[3];
          split3_bf16x2(x[2 * i], x[2 * i + 1], &part[0], &part[1], &part[2]);
          unsigned char* at = S.q + m_byte(i ? tb : ta, j);
#pragma unroll
          for (int e = 0; e < 3; ++e) *reinterpret_cast<uint32_t*>(at + e * kMPart) = part[e];
        }
      }
    }
    fence_proxy_async_smem();
    named_barrier_sync(1, 128);
    if (tid == 128) {
      bulk_store(rec + kRecM, S.q, 3 * kMPart);
      bulk_store_wait();
    }
    __syncwarp();
  } else {
    // Tu = (I + L)^-1 in place.  The four 16 x 16 diagonal blocks by forward substitution, a block
    // a warp, a column a lane (both halves of the warp alike); then twice by halves, the block
    // below the diagonal being -T22 (L21 T11).  Upper blocks hold what was in the way: they are
    // zero in Tu, and nothing reads them as Tu.
    const int o = 16 * warp;
    float u[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      float x[2] = {t == (lane & 15) ? 1.f : 0.f, 0.f};
      const float* row = &S.a[(o + t) * kPrepLdA + o];
#pragma unroll
      for (int j = 0; j + 4 <= t; j += 4) {
        const float4 l = *reinterpret_cast<const float4*>(row + j);
        x[0] = fmaf(-l.x, u[j], x[0]);
        x[1] = fmaf(-l.y, u[j + 1], x[1]);
        x[0] = fmaf(-l.z, u[j + 2], x[0]);
        x[1] = fmaf(-l.w, u[j + 3], x[1]);
      }
#pragma unroll
      for (int j = t & ~3; j < t; ++j) x[j & 1] = fmaf(-row[j], u[j], x[j & 1]);
      u[t] = x[0] + x[1];
    }
    __syncwarp();
    if (lane < 16)
#pragma unroll
      for (int t = 0; t < 16; ++t) S.a[(o + t) * kPrepLdA + o + lane] = u[t];
    // the largest |K|: half a row a lane
    {
      uint32_t m2 = 0u;
      const unsigned char* p = S.k + 8192 * (lane & 1);
      const int t = o + (lane >> 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + tile_byte(t, 8 * (i ^ (4 * (lane & 1)))));
        m2 = max_abs_bf16x2(max_abs_bf16x2(m2, x.x), x.y);
        m2 = max_abs_bf16x2(max_abs_bf16x2(m2, x.z), x.w);
      }
      float m = fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u));
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
      if (lane == 0) S.kmax[warp] = m;
    }
    named_barrier_sync(2, 128);
    // 16 -> 32: two blocks, two tiles of 8 columns each
    const int d = 32 * (warp >> 1), c8 = 8 * (warp & 1);
    float z[4] = {0.f, 0.f, 0.f, 0.f};
    prep_mma3(z, &S.a[(d + 16) * kPrepLdA + d], &S.a[d * kPrepLdA + d + c8], gq, tq);
    prep_put(&S.a[d * kPrepLdA + d + 16 + c8], z, 1.f, gq, tq);
    named_barrier_sync(2, 128);
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = 0.f;
    prep_mma3(z, &S.a[(d + 16) * kPrepLdA + d + 16], &S.a[d * kPrepLdA + d + 16 + c8], gq, tq);
    prep_put(&S.a[(d + 16) * kPrepLdA + d + c8], z, -1.f, gq, tq);
  }
  __syncthreads();
  // V in Q's and M's space (M has been read: the barrier)
  for (int e = tid; e < kGdnChunk * 16; e += kPrepThreads) {
    const int t = e >> 4, w = e & 15;
    cp_async16(sq + 8192 * (w >> 3) + tile_byte(t, 8 * (w & 7)),
               a.v + ((t0 + (t < n ? t : 0)) * a.heads + h) * kGdnDim + 8 * w, t < n);
  }
  {
    // 32 -> 64: T21 = -T22 (L21 T11), a 16 x 8 tile a warp; T11 and T22 are zero above their
    // diagonal
    const int r0 = 16 * (warp & 1), c0 = 8 * (warp >> 1);
    float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int k0 = c0 & 16; k0 < 32; k0 += 16)
      prep_mma3(z, &S.a[(32 + r0) * kPrepLdA + k0], &S.a[k0 * kPrepLdA + c0], gq, tq);
    prep_put(&S.a[r0 * kPrepLdA + 32 + c0], z, 1.f, gq, tq);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 <= r0; k0 += 16)
      prep_mma3(z, &S.a[(32 + r0) * kPrepLdA + 32 + k0], &S.a[k0 * kPrepLdA + 32 + c0], gq, tq);
    prep_put(&S.a[(32 + r0) * kPrepLdA + c0], z, -1.f, gq, tq);
  }
  cp_async_wait_all();
  __syncthreads();
  // T V, T = Tu diag(beta), and then W = T diag(e^g) K: warp = 16 rows x 64 columns
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    rb = pass ? 3 - (warp & 3) : warp & 3;
    ta = 16 * rb + gq;
    tb = ta + 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    const uint32_t src = (pass ? sk : sq) + 8192 * (warp >> 2);
    const float* scale = pass ? S.beg : S.beta;
#pragma unroll 1
    for (int ks = 0; ks <= rb; ++ks) {
      uint32_t fh[4], fm[4], fl[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = (e & 1) ? tb : ta, j = 16 * ks + 2 * tq + 8 * (e >> 1);
        const float2 x = *reinterpret_cast<const float2*>(&S.a[t * kPrepLdA + j]);
        const float2 y = *reinterpret_cast<const float2*>(&scale[j]);
        split3_bf16x2(x.x * y.x, x.y * y.y, &fh[e], &fm[e], &fl[e]);
      }
      // ks <= rb: never a block above the diagonal
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t fb[4];
        ldsm4_t(fb, src + tile_byte(16 * ks + (lane & 15), 16 * np + 8 * (lane >> 4)));
        delta_mma(acc[2 * np], fh, fb[0], fb[1]);
        delta_mma(acc[2 * np + 1], fh, fb[2], fb[3]);
        delta_mma(acc[2 * np], fm, fb[0], fb[1]);
        delta_mma(acc[2 * np + 1], fm, fb[2], fb[3]);
        delta_mma(acc[2 * np], fl, fb[0], fb[1]);
        delta_mma(acc[2 * np + 1], fl, fb[2], fb[3]);
      }
    }
    if (pass == 0) {
      float* tv = reinterpret_cast<float*>(rec + kRecU) + 64 * (warp >> 2) + 2 * tq;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        *reinterpret_cast<float2*>(tv + ta * kGdnDim + 8 * nt) = make_float2(acc[nt][0], acc[nt][1]);
        *reinterpret_cast<float2*>(tv + tb * kGdnDim + 8 * nt) = make_float2(acc[nt][2], acc[nt][3]);
      }
    }
  }
  // a row's largest |W|, each half of the columns by another warp
  float ma = 0.f, mb = 0.f;
#pragma unroll
  for (int nt = 0; nt < 8; ++nt) {
    ma = fmaxf(ma, fmaxf(fabsf(acc[nt][0]), fabsf(acc[nt][1])));
    mb = fmaxf(mb, fmaxf(fabsf(acc[nt][2]), fabsf(acc[nt][3])));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
    mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
  }
  if (tq == 0) {
    S.wmax[warp >> 2][ta] = ma;
    S.wmax[warp >> 2][tb] = mb;
  }
  __syncthreads();   // also: K and Tu have been read
  float ia, ib;
  const float sa = -row_scale(fmaxf(S.wmax[0][ta], S.wmax[1][ta]), &ia);
  const float sb = -row_scale(fmaxf(S.wmax[0][tb], S.wmax[1][tb]), &ib);
  if (warp < 4 && tq == 0) {
    gate[kGateW + ta] = ia;
    gate[kGateW + tb] = ib;
  }
  if (tid == 0) gate[kGateK] = fmaxf(fmaxf(S.kmax[0], S.kmax[1]), fmaxf(S.kmax[2], S.kmax[3]));
  unsigned char* w = S.k + 16384 * (warp >> 2);   // on into Tu's space
#pragma unroll
  for (int nt = 0; nt < 8; ++nt) {
    uint32_t vh, vl;
    const int d = 8 * nt + 2 * tq;
    split_f16x2(sa * acc[nt][0], sa * acc[nt][1], &vh, &vl);
    *reinterpret_cast<uint32_t*>(w + tile_byte(ta, d)) = vh;
    *reinterpret_cast<uint32_t*>(w + 8192 + tile_byte(ta, d)) = vl;
    split_f16x2(sb * acc[nt][2], sb * acc[nt][3], &vh, &vl);
    *reinterpret_cast<uint32_t*>(w + tile_byte(tb, d)) = vh;
    *reinterpret_cast<uint32_t*>(w + 8192 + tile_byte(tb, d)) = vl;
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    bulk_store(rec + kRecW, S.k, 32768);
    bulk_store(rec + kRecGate, S.gate, kRecBytes - kRecGate);
    bulk_store_wait();
  }
}

// ---- k_delta_scan: one CTA per (head, sequence, segment) --------------------------------------
// With v along the 128 lanes of tensor memory, every operand that depends on the state is an A
// operand in tensor memory, written there by the threads that computed it, and no result goes
// back to shared memory:
//     D_W [v][t] = -S0 W^T          A = S0 (fp16 parts); S0 hi W hi^T and S0 hi W lo^T side by side
//     D_Q [v][t] = S0 Q^T, then U^T M^T (by 16 columns j of M, whose rows t >= j count)
//     D_S [v][d] = U'^T K,  U' = diag(e^(g_C - g)) U,  U = (T V)^T + D_W
// Four warpgroups hold the fp32 state in registers (a lane has one v, 32 of its d's), form U and
// U' and then S; two write the outputs; one warp issues the products and three load, each its own
// operands, whose space is free again as soon as their last product is done.
//
// Bound by the chain of a chunk, S -> D_W -> U' -> D_S -> S, 2.87 us (2.45 where no outputs are
// written): about 1,000 cycles for D_W (16 products of 128 x 64 or 128 x 128 x 16), 1,250 for U',
// 1,000 for D_S (12 of 128 x 128 x 16), 1,600 for S, most of whose conversion is instruction issue
// (two products' parts, 5 to 9 instructions an element).  S goes over in two parts, so that the
// products of one run while the other is converted; S is scaled before it is known, by a bound on
// its rows, |S| <= e^(g_C) max|S0| + 64 max|U'| max|K|; what only the outputs need (D_Q) runs in the
// gaps, but for 0.1 us that the next D_W waits for the 24 products of U^T M^T (12, of parts to 2^-17,
// measured that much less).  A form without W (X = V - e^g K S0^T, U = T X) would read 32 KB less a
// chunk and have one more product and conversion in the chain.  8 x 8,192 tokens x 16 heads: 432 us on
// 128 SMs (129 KB a chunk: 4.9 TB/s); the same walk with fp32 state in shared memory and warp MMAs
// (k_gated_deltanet, preparation included) takes 2.6 ms.
constexpr int kScanThreads = 896;
constexpr int kScanW = 0;                               // [2] W, K, gates
constexpr int kScanWBytes = 32768 + 16384 + 1024;
constexpr int kScanQ = kScanW + 2 * kScanWBytes;        // [2] Q, the gates again (the outputs' warps read them late)
constexpr int kScanQBytes = 16384 + 1024;
constexpr int kScanM = kScanQ + 2 * kScanQBytes;        // M, once: asked for a chunk ahead of its product
constexpr int kScanMBytes = 3 * kMPart;
constexpr int kScanU = kScanM + kScanMBytes;            // [2] T V
constexpr int kScanUBytes = 32768;
constexpr int kScanBars = kScanU + 2 * kScanUBytes;
constexpr int kScanSmemBytes = kScanBars + 6144;
static_assert(kScanSmemBytes <= 232448, "shared memory per CTA");
static_assert(kScanWBytes % 1024 == 0 && kScanQBytes % 1024 == 0 && kScanMBytes % 1024 == 0, "tiles on 1 KB boundaries");

// what a launch does: the whole walk; or, where sequences are cut into segments, the first segments
// whole and the inner ones' states from zero and transitions, then the outputs of all segments
// behind the first from the joined states
constexpr int kScanWhole = 0, kScanEnds = 1, kScanOutputs = 2;

struct ScanBars {
  uint64_t full_w[2], empty_w[2], full_u[2], empty_u[2], full_q[2], empty_q[2], full_m, empty_m;
  uint64_t s_part[2];           // 16 columns of S of every quarter
  uint64_t d1, uw_full, u_full, ds, qs, q_free, o, o_free, mma_done;
  uint64_t rows[4];             // the four warps of 32 rows have their maxima in place
  uint32_t tmem;
  int abort;
  // by row: 1 over the scale of S (by the parity of the chunk); the quarters' largest |S|, |U'|
  float scale[2][kGdnDim];
  float smax[4][kGdnDim], umax[4][kGdnDim];
};
static_assert(sizeof(ScanBars) <= 6144, "barriers");

// 32 lanes x 32 bit, 8 (4) consecutive columns per thread
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void reg_fence8(uint32_t* r) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
               "+r"(r[6]), "+r"(r[7]));
}
// Keeps the reads of a tcgen05.ld's 16 registers behind tcgen05.wait::ld.
__device__ __forceinline__ void reg_fence16(uint32_t* r) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
               "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
               "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void tmem_ld16_at(uint32_t taddr, float* f) {
  uint32_t r[16];
  tmem_ld16(taddr, r);
  tmem_wait_ld();
  reg_fence16(r);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
}

// Bounded wait for the phase of the given parity.  Past the limit (on the global timer's low word,
// which wraps after 4.3 s) the site is noted for the CTA's other waits, which then give up too, and
// for the status that the kernel reports at its end.  Small, since the kernel's loop has to stay in
// the instruction cache.
__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool scan_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t limit_ns, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = globaltimer_lo();
#pragma unroll 1
  while (*abort == 0) {
    if (mbar_try_wait(bar, parity)) return true;
    if (globaltimer_lo() - t0 > limit_ns) *abort = site;
  }
  return false;
}

// K as [tokens][key heads][128], boxes of 64 tokens x 64 columns of one head
struct ScanMaps {
  CUtensorMap k;
};

__global__ void __launch_bounds__(kScanThreads, 1)
    k_delta_scan(const __grid_constant__ ScanMaps maps, DeltaChunkArgs ca, int mode) {
  extern __shared__ __align__(1024) unsigned char smem[];
  ScanBars& B = *reinterpret_cast<ScanBars*>(smem + kScanBars);
  const DeltaArgs& a = ca.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hl = blockIdx.x, h = ca.head0 + hl;
  pdl_trigger();
  // the first pass has two CTAs a segment: states, and transitions
  const bool trans = mode == kScanEnds && (blockIdx.z & 1);
  const int seg = mode == kScanEnds ? blockIdx.z >> 1 : blockIdx.z + (mode == kScanOutputs);
  const DeltaPiece piece = delta_piece(ca, blockIdx.y);
  const int row = piece.row;
  const int64_t begin = piece.begin, len = piece.len, chunks = (len + kGdnChunk - 1) / kGdnChunk;
  const int64_t c0 = seg == 0 ? 0 : ca.seg_first + static_cast<int64_t>(seg - 1) * ca.seg_chunks;
  const int64_t len_c = seg == 0 ? ca.seg_first : ca.seg_chunks;
  const int64_t c1 = c0 + len_c < chunks ? c0 + len_c : chunks;
  const int nc = static_cast<int>(c1 - c0);
  const bool last = c1 == chunks;
  const int slot = a.slots != nullptr && row >= 0 ? a.slots[row] : row;
  const bool outputs = mode != kScanEnds || seg == 0;
  const int64_t t0 = begin + c0 * kGdnChunk;
  const int ntok = static_cast<int>((last ? len : c1 * kGdnChunk) - c0 * kGdnChunk);
  bool idle = nc <= 0 || len <= a.short_len || (mode == kScanEnds && (seg == 0 ? trans : last));
  if (!idle && (slot < 0 || slot >= a.num_slots || delta_slot_taken(a, row, slot))) {
    idle = true;
    if (a.zero_skipped && outputs) {
      pdl_wait();
      for (int i = tid; i < ntok * 16; i += kScanThreads)
        reinterpret_cast<uint4*>(a.out)[((t0 + (i >> 4)) * a.heads + h) * 16 + (i & 15)] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (!idle && (smem_u32(smem) & 1023u) != 0) {   // the tiles need it; the runtime places them so
    if (tid == 0) report_error(ca.st, kErrDevice, 320);
    idle = true;
  }
  if (idle) {
    pdl_wait();   // every CTA waits: the kernels after this one count on all before it
    return;
  }
  const int64_t rec0 = piece.record, seg0 = piece.segment;
  const int64_t tile = static_cast<int64_t>(kGdnDim) * kGdnDim;
  float* state = a.states + (static_cast<int64_t>(slot) * a.heads + h) * tile;
  const int64_t seg_stride = static_cast<int64_t>(ca.nheads) * tile;
  float* ends = ca.seg_state + (seg0 + seg) * seg_stride + hl * tile;
  const float* src = seg > 0 ? ends - seg_stride : state;
  float* dst = last ? state : trans ? ca.seg_trans + (ends - ca.seg_state) : ends;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.full_w[i], 2);
      mbar_init(&B.empty_w[i], 1 + 16);
      mbar_init(&B.full_u[i], 1);
      mbar_init(&B.empty_u[i], 16);
      mbar_init(&B.full_q[i], 1);
      mbar_init(&B.empty_q[i], 1 + 8);
    }
    mbar_init(&B.full_m, 1);
    mbar_init(&B.empty_m, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&B.s_part[i], 16);
    mbar_init(&B.uw_full, 16);
    mbar_init(&B.d1, 1);
    mbar_init(&B.u_full, 16);
    mbar_init(&B.ds, 1);
    mbar_init(&B.qs, 1);
    mbar_init(&B.q_free, 8);
    mbar_init(&B.o, 1);
    mbar_init(&B.o_free, 8);
    mbar_init(&B.mma_done, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&B.rows[i], 4);
    B.abort = 0;
    fence_mbar_init();
  }
  if (warp == 24) {
    tmem_alloc(&B.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  // all 512 columns are this CTA's, so they start at 0: addresses are known to the compiler
  constexpr uint32_t tm = 0;
  // columns: S hi 64, S lo 64, D_S 128, D_W 64, its (hi, lo) part 64 (then, each quarter of the
  // threads in the 16 columns that it has read, U' mid and lo, 8 each, and U mid and lo behind
  // them), D_Q 64, U' hi 32, U hi 32
  constexpr uint32_t tS = tm, tDS = tm + 128, tDW = tm + 256, tDQ = tm + 384, tUw = tm + 448,
                     tU = tm + 480;
  volatile int* abort = &B.abort;

  if (warp < 16) {
    regs_raise<80>();
    // ---- the state: lane = value row v, 32 columns d of it -----------------------------------
    const int quarter = warp >> 2, v = 32 * (warp & 3) + lane;
    const uint32_t lb = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    float s[32];
    if (trans) {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = 32 * quarter + i == v ? 1.f : 0.f;
    } else if (mode == kScanEnds && seg > 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = 0.f;
    } else {
      const float4* p = reinterpret_cast<const float4*>(src + v * kGdnDim + 32 * quarter);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = p[i];
        s[4 * i] = x.x;
        s[4 * i + 1] = x.y;
        s[4 * i + 2] = x.z;
        s[4 * i + 3] = x.w;
      }
    }
    auto signal = [&](uint64_t* bar) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto joined = [&](int phase) -> bool {   // the maxima of all quarters of the rows are in place
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.rows[warp & 3]);
      return __all_sync(0xffffffffu, scan_wait(&B.rows[warp & 3], phase & 1, abort, ca.wait_ns, 337));
    };
    auto row_max = [&](const float (*m)[kGdnDim]) -> float {
      return fmaxf(fmaxf(m[0][v], m[1][v]), fmaxf(m[2][v], m[3][v]));
    };
    bool ok = true;
    float inv = 1.f, smax = 0.f;   // 1 over the scale of this row of S; its largest entry (quarter)
    // turn c: S0 of chunk c into U, then into S, which goes over as the S0 of chunk c + 1; turn -1
    // only hands the first one over
#pragma unroll 1
    for (int c = -1; c < nc; ++c) {
      const int sg = c & 1;
      const bool first = c < 0, more = c + 1 < nc;
      {
        float m[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) m[i & 1] = fmaxf(m[i & 1], fabsf(s[i]));
        smax = fmaxf(m[0], m[1]);
      }
      float gc = 1.f, sc = 1.f;
      if (!first) {
        const float* gate = reinterpret_cast<const float*>(smem + kScanW + sg * kScanWBytes + 49152);
        float u[16];
        if (trans) {
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = 0.f;
        } else {
          ok = scan_wait(&B.full_u[sg], (c >> 1) & 1, abort, ca.wait_ns, 338);
          const float* tv = reinterpret_cast<const float*>(smem + kScanU + sg * kScanUBytes) + 16 * quarter * kGdnDim + v;
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = tv[i * kGdnDim];
        }
        ok = ok && scan_wait(&B.full_w[sg], (c >> 1) & 1, abort, ca.wait_ns, 330) &&
             scan_wait(&B.d1, c & 1, abort, ca.wait_ns, 331);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const float4* wk = reinterpret_cast<const float4*>(gate + kGateU + 16 * quarter);
        const float4* wi = reinterpret_cast<const float4*>(gate + kGateW + 16 * quarter);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t x[8], y[8], vh[4], vm[4], vl[4];
          tmem_ld8(tDW + lb + 16 * quarter + 8 * b, y);
          tmem_ld8(tDW + 64 + lb + 16 * quarter + 8 * b, x);
          tmem_wait_ld();
          reg_fence8(x);
          reg_fence8(y);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 w = wk[2 * b + i], z = wi[2 * b + i];
            const float r[4] = {inv * z.x, inv * z.y, inv * z.z, inv * z.w};
            float* p = u + 8 * b + 4 * i;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = fmaf(r[e], __uint_as_float(y[4 * i + e]) + __uint_as_float(x[4 * i + e]), p[e]);
            split3_bf16x2(w.x * p[0], w.y * p[1], &vh[2 * i], &vm[2 * i], &vl[2 * i]);
            split3_bf16x2(w.z * p[2], w.w * p[3], &vh[2 * i + 1], &vm[2 * i + 1], &vl[2 * i + 1]);
          }
          // mid and lo take columns of D_W that were just read
          tmem_st4(tUw + lb + 8 * quarter + 4 * b, vh);
          tmem_st4(tDW + lb + 16 * quarter + 4 * b, vm);
          tmem_st4(tDW + 64 + lb + 16 * quarter + 4 * b, vl);
        }
        signal(&B.uw_full);
        float umax = 0.f;   // of U', not of U: what a later gate takes back does not count
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 w = wk[i];
          umax = fmaxf(fmaxf(umax, fabsf(w.x * u[4 * i])), fabsf(w.y * u[4 * i + 1]));
          umax = fmaxf(fmaxf(umax, fabsf(w.z * u[4 * i + 2])), fabsf(w.w * u[4 * i + 3]));
        }
        B.smax[quarter][v] = smax;
        B.umax[quarter][v] = umax;
        gc = gate[kGateC];
        const float kmax = gate[kGateK];
        ok = joined(c + 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive(&B.empty_w[sg]);
          if (!trans) mbar_arrive(&B.empty_u[sg]);
        }
        umax = row_max(B.umax);
        sc = row_scale(fmaf(gc, row_max(B.smax), 64.f * kmax * umax), &inv);
        if (outputs) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t vh[4], vm[4], vl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              split3_bf16x2(u[8 * b + 2 * i], u[8 * b + 2 * i + 1], &vh[i], &vm[i], &vl[i]);
            tmem_st4(tU + lb + 8 * quarter + 4 * b, vh);
            tmem_st4(tDW + 8 + lb + 16 * quarter + 4 * b, vm);
            tmem_st4(tDW + 72 + lb + 16 * quarter + 4 * b, vl);
          }
          signal(&B.u_full);
        }
        ok = scan_wait(&B.ds, c & 1, abort, ca.wait_ns, 332);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
      } else {
        B.smax[quarter][v] = smax;
        ok = joined(0);
        if (!ok) break;
        sc = row_scale(row_max(B.smax), &inv);
      }
      if (more && quarter == 0) B.scale[(c + 1) & 1][v] = inv;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!first) {
          uint32_t x[16];
          tmem_ld16(tDS + lb + 32 * quarter + 16 * g, x);
          tmem_wait_ld();
          reg_fence16(x);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[16 * g + i] = fmaf(gc, s[16 * g + i], __uint_as_float(x[i]));
        }
        if (more) {   // columns 16 g .. of this quarter, as fp16 parts
          uint32_t vh[8], vl[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            split_f16x2(sc * s[16 * g + 2 * i], sc * s[16 * g + 2 * i + 1], &vh[i], &vl[i]);
          tmem_st8(tS + lb + 16 * quarter + 8 * g, vh);
          tmem_st8(tS + lb + 64 + 16 * quarter + 8 * g, vl);
          signal(&B.s_part[g]);
        }
      }
    }
    // in the outputs pass the joined states hold what the inner segments would write
    if (__all_sync(0xffffffffu, ok) && (mode == kScanEnds || last)) {
      float4* p = reinterpret_cast<float4*>(dst + v * kGdnDim + 32 * quarter);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        p[i] = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    }
  } else if (warp < 24) {
    regs_lower<72>();
    // ---- outputs: lane = value v, 32 tokens --------------------------------------------------
    if (outputs) {
      const int half = (warp - 16) >> 2, v = 32 * (warp & 3) + lane;
      const uint32_t lb = static_cast<uint32_t>(32 * (warp & 3)) << 16;
      const int64_t step = static_cast<int64_t>(a.heads) * kGdnDim;
      const uint32_t sel = (lane & 1) ? 0x3276 : 0x5410;
#pragma unroll 1
      for (int c = 0; c < nc; ++c) {
        const int sg = c & 1;
        const float* gate = reinterpret_cast<const float*>(smem + kScanQ + sg * kScanQBytes + 16384);
        const float4* eg = reinterpret_cast<const float4*>(gate + kGateQ + 32 * half);
        bool ok = scan_wait(&B.full_q[sg], (c >> 1) & 1, abort, ca.wait_ns, 333) &&
                  scan_wait(&B.qs, c & 1, abort, ca.wait_ns, 334);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const float inv = B.scale[sg][v];
        float y[32];
#pragma unroll
        for (int i0 = 0; i0 < 32; i0 += 16) {
          tmem_ld16_at(tDQ + lb + 32 * half + i0, y + i0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 e = eg[i0 / 4 + i];
            y[i0 + 4 * i] *= inv * e.x;
            y[i0 + 4 * i + 1] *= inv * e.y;
            y[i0 + 4 * i + 2] *= inv * e.z;
            y[i0 + 4 * i + 3] *= inv * e.w;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&B.q_free);
          mbar_arrive(&B.empty_q[sg]);   // the gates have been read
        }
        ok = scan_wait(&B.o, c & 1, abort, ca.wait_ns, 335);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const int left = ntok - c * kGdnChunk - 32 * half - (lane & 1);
        const int n = left < kGdnChunk ? left : kGdnChunk;   // mine: tokens i < n
        // lanes in pairs: the even one stores both its own and its neighbour's value of token t,
        // the odd one of token t + 1
        __nv_bfloat16* op = a.out + ((t0 + static_cast<int64_t>(c) * kGdnChunk + 32 * half + (lane & 1)) * a.heads + h) * kGdnDim +
                            (v & ~1);
#pragma unroll
        for (int i0 = 0; i0 < 32; i0 += 16) {
          float x[16];
          tmem_ld16_at(tDQ + lb + 32 * half + i0, x);
          if (i0 == 16) {   // D_Q has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.o_free);
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const uint32_t w = pack_bf16x2(x[i] + y[i0 + i], x[i + 1] + y[i0 + i + 1]);
            const uint32_t z = __shfl_xor_sync(0xffffffffu, w, 1);
            const uint32_t both = __byte_perm(w, z, sel);
            if (i0 + i < n) *reinterpret_cast<uint32_t*>(op) = both;
            op += 2 * step;
          }
        }
      }
    }
  } else {
    regs_lower<40>();
    if (warp == 24) {
    // ---- products: the whole warp walks the loop, one elected lane issues ----------------------
    constexpr uint32_t kIdF16 = idesc_f16_f32(128, 64, 0, 0);
    constexpr uint32_t kIdF16x2 = idesc_f16_f32(128, 128, 0, 0);   // W's hi and lo rows at once
    constexpr uint32_t kIdDS = idesc_bf16_f32(128, 128, 0, 1);  // B = K, tokens along its rows
    // Descriptors; a step along a tile adds its bytes / 16.  The loops stay loops: unrolled, this
    // warp alone would fill the instruction cache.
    const uint64_t dk = smem_desc_sw128(smem_u32(smem), 0, 1024);        // rows of 128 bytes
    const uint64_t dm = smem_desc_sw128(smem_u32(smem), 8192, 1024);     // two column panels
    const uint64_t dmm = smem_desc_sw32(smem_u32(smem) + kScanM, 256);   // M: rows of 32 bytes
    // (the lanes stay together, whatever each has seen)
    auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
      return __all_sync(0xffffffffu, scan_wait(bar, parity, abort, ca.wait_ns, site)) != 0;
    };
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
      const int sg = c & 1;
      const uint32_t ph = (c >> 1) & 1;
      const uint64_t sw = (kScanW + sg * kScanWBytes) >> 4, sq = (kScanQ + sg * kScanQBytes) >> 4;
      {
        if (!wait(&B.full_w[sg], ph, 342)) break;
        // D_W = -S0 W^T: (hi, hi and lo), (lo, hi) of 16 columns of each quarter at a time
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          ok = wait(&B.s_part[g], c & 1, 341);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll 1
            for (int kh = 0; kh < 2; ++kh) {
              const uint64_t dw = dk + sw + 1024 * kh + 2 * g;
              const uint32_t ts = tS + 32 * kh + 8 * g;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                umma_ts(tDW, ts + 16 * q, dw + 4 * q, kIdF16x2, g + kh + q > 0 ? 1u : 0u);
                umma_ts(tDW, ts + 64 + 16 * q, dw + 4 * q, kIdF16, 1u);
              }
            }
            if (g == 1) umma_commit(&B.d1);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (outputs) {
          if (!wait(&B.full_q[sg], ph, 343)) break;
          if (c > 0 && !wait(&B.o_free, (c - 1) & 1, 344)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll 1
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int kh = 0; kh < 2; ++kh) {
                const uint64_t dq = dk + sq + 512 * kh + 2 * k;
                umma_ts(tDQ, tS + 32 * kh + 8 * k, dq, kIdF16, k + kh > 0 ? 1u : 0u);
                umma_ts(tDQ, tS + 64 + 32 * kh + 8 * k, dq, kIdF16, 1u);
              }
            umma_commit(&B.qs);
            umma_commit(&B.empty_q[sg]);
          }
          __syncwarp();
        }
      }
      if (!wait(&B.uw_full, c & 1, 345)) break;
      tc_fence_after();
      if (elect_one()) {
        // D_S = U'^T K: hi, mid, lo
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const uint64_t d = dm + sw + 2048 + 128 * k;
          umma_ts(tDS, tUw + 8 * k, d, kIdDS, k > 0 ? 1u : 0u);
          umma_ts(tDS, tDW + 16 * k, d, kIdDS, 1u);
          umma_ts(tDS, tDW + 64 + 16 * k, d, kIdDS, 1u);
        }
        umma_commit(&B.ds);
        umma_commit(&B.empty_w[sg]);
      }
      __syncwarp();
      if (outputs) {
        if (!wait(&B.q_free, c & 1, 346)) break;
        if (!wait(&B.full_m, c & 1, 349)) break;
        if (!wait(&B.u_full, c & 1, 348)) break;
        tc_fence_after();
        if (elect_one()) {
          // D_Q = U^T M^T: hi (hi, mid, lo), mid (hi, mid), lo hi; M is zero above its diagonal, so
          // that columns j = 16 k .. take part in tokens t >= 16 k only
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            const uint64_t d = dmm + (m_panel(k) >> 4);
            const uint32_t to = tDQ + 16 * k, id = idesc_bf16_f32(128, 64 - 16 * k, 0, 0);
            umma_ts(to, tU + 8 * k, d, id, k > 0 ? 1u : 0u);
            umma_ts(to, tU + 8 * k, d + (kMPart >> 4), id, 1u);
            umma_ts(to, tU + 8 * k, d + 2 * (kMPart >> 4), id, 1u);
            umma_ts(to, tDW + 8 + 16 * k, d, id, 1u);
            umma_ts(to, tDW + 8 + 16 * k, d + (kMPart >> 4), id, 1u);
            umma_ts(to, tDW + 72 + 16 * k, d, id, 1u);
          }
          umma_commit(&B.o);
          umma_commit(&B.empty_m);
        }
        __syncwarp();
      }
    }
    __syncwarp();
    if (elect_one()) umma_commit(&B.mma_done);
    mbar_drain(&B.mma_done, 0);
    __syncwarp();
  } else {
    // ---- loads: warp 25: W, K and the gates; 26: T V; 27: Q and the gates, M -------------------
    const int who = warp - 25;
    uint64_t* full = who == 0 ? B.full_w : who == 1 ? B.full_u : B.full_q;
    uint64_t* empty = who == 0 ? B.empty_w : who == 1 ? B.empty_u : B.empty_q;
    const bool on = who == 0 || (who == 1 ? !trans && !(ca.fault == kFaultScan && hl + blockIdx.y + blockIdx.z == 0)
                                          : outputs);
    const int kh = h / (a.heads / a.key_heads);
    int issued = 0, issued_m = 0;
    const unsigned char* rec = ca.rec + ((rec0 + c0) * ca.nheads + hl) * static_cast<int64_t>(kRecBytes);
#pragma unroll 1
    for (int c = 0; on && c < nc; ++c, rec += ca.nheads * static_cast<int64_t>(kRecBytes)) {
      const int sg = c & 1;
      const bool ok = c < 2 || scan_wait(&empty[sg], ((c >> 1) & 1) ^ 1, abort, ca.wait_ns, 347);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int at = static_cast<int>(t0) + c * kGdnChunk;
      const int left = ntok - c * kGdnChunk;
      const int n = left < kGdnChunk ? left : kGdnChunk;
      const bool whole = n == kGdnChunk;
      unsigned char* stage = smem + (who == 0 ? kScanW + sg * kScanWBytes : who == 1 ? kScanU + sg * kScanUBytes : kScanQ + sg * kScanQBytes);
      if (lane == 0) {
        if (who == 0) {
          mbar_arrive_expect_tx(&full[sg], 32768 + 1024 + (whole ? 16384 : 0));
          bulk_load(stage, rec + kRecW, 32768, &full[sg]);
          bulk_load(stage + 49152, rec + kRecGate, 1024, &full[sg]);
          if (whole) {
            tma_load_3d(stage + 32768, &maps.k, 0, kh, at, &full[sg]);
            tma_load_3d(stage + 32768 + 8192, &maps.k, 64, kh, at, &full[sg]);
          }
        } else if (who == 1) {
          mbar_arrive_expect_tx(&full[sg], kScanUBytes);
          bulk_load(stage, rec + kRecU, kScanUBytes, &full[sg]);
        } else {
          mbar_arrive_expect_tx(&full[sg], kScanQBytes);
          bulk_load(stage, rec + kRecQ, 16384, &full[sg]);
          bulk_load(stage + 16384, rec + kRecGate, 1024, &full[sg]);
        }
      }
      __syncwarp();
      ++issued;
      if (who == 0) {
        if (!whole) {   // the rows behind the sequence's last token must be zero
          const uint32_t to = smem_u32(stage + 32768);
          const __nv_bfloat16* from = a.k + (static_cast<int64_t>(at) * a.key_heads + kh) * kGdnDim;
          const int64_t step = static_cast<int64_t>(a.key_heads) * kGdnDim;
#pragma unroll 1
          for (int e = lane; e < kGdnChunk * 16; e += 32) {
            const int t = e >> 4, w = e & 15;
            cp_async16(to + 8192 * (w >> 3) + tile_byte(t, 8 * (w & 7)),
                       from + (t < n ? t : 0) * step + 8 * w, t < n);
          }
          cp_async_wait_all();
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&full[sg]);
      } else if (who == 2) {
        const bool free = c == 0 || scan_wait(&B.empty_m, (c - 1) & 1, abort, ca.wait_ns, 336);
        if (!__all_sync(0xffffffffu, free)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&B.full_m, kScanMBytes);
          bulk_load(smem + kScanM, rec + kRecM, kScanMBytes, &B.full_m);
        }
        __syncwarp();
        ++issued_m;
      }
    }
    if (lane == 0 && *abort) {   // no copy may land after the CTA is gone
      for (int c = issued > 2 ? issued - 2 : 0; c < issued; ++c) mbar_drain(&full[c & 1], (c >> 1) & 1);
      if (issued_m > 0) mbar_drain(&B.full_m, (issued_m - 1) & 1);
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort != 0) report_error(ca.st, kErrTimeout, *abort);
  if (warp == 24) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

// Joins the segments of a sequence: entered with E (the state at its start), a segment ends with
// E P + S.  Rows of the state are independent: a CTA takes kRows of them through the segments in
// order.  A warp takes 32 of the 128 terms of every product and a lane four columns, so that P
// leaves shared memory once (64 KB, 512 cycles, which is what a step of four or eight rows is
// bound by); the warps' parts are added in order.  The P of the next segments are on their way: at
// one head its 64 KB a step (1.0 us measured) are what an SM takes in from L2.
constexpr int kJoinThreads = 128;
constexpr int join_stages(int rows) { return rows > 8 ? 2 : 3; }
constexpr int join_smem_bytes(int rows) {
  return join_stages(rows) * kGdnDim * kGdnDim * 4 + 5 * rows * kGdnDim * 4;
}

// grid (heads of the pass, sequences, 128 / kRows)
template <int kRows>
__global__ void __launch_bounds__(kJoinThreads) k_delta_join(DeltaChunkArgs ca) {
  constexpr int kStages = join_stages(kRows), kTile = kGdnDim * kGdnDim;
  extern __shared__ __align__(128) float join_sh[];   // P [stages][128][128], E, the warps' parts
  __shared__ uint64_t full[kStages];
  __shared__ int abort_flag;
  float* e = join_sh + kStages * kTile;               // [rows][128]
  float* part = e + kRows * kGdnDim;                  // [4][rows][128]
  const int hl = blockIdx.x, d = threadIdx.x, v0 = blockIdx.z * kRows;
  const int warp = d >> 5, lane = d & 31;
  pdl_trigger();
  const DeltaPiece piece = delta_piece(ca, blockIdx.y);
  const int64_t segs = delta_segments((piece.len + kGdnChunk - 1) / kGdnChunk, ca.seg_first, ca.seg_chunks);
  if (d == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  if (segs < 3) return;
  volatile int* abort = &abort_flag;
  const int64_t stride = static_cast<int64_t>(ca.nheads) * kTile;
  const int64_t at = (piece.segment * ca.nheads + hl) * kTile;
  float* s = ca.seg_state + at + v0 * kGdnDim + d;
  const float* p = ca.seg_trans + at;
  const int64_t absent = ca.fault == kFaultJoin && hl + blockIdx.y + blockIdx.z == 0 ? 1 : 0;
  auto fetch = [&](int64_t g) {   // segment g's transition
    if (d == 0 && g + 1 < segs && g != absent) {
      uint64_t* bar = &full[(g - 1) % kStages];
      mbar_arrive_expect_tx(bar, kTile * 4);
      bulk_load(join_sh + ((g - 1) % kStages) * kTile, p + g * stride, kTile * 4, bar);
    }
  };
  int64_t fetched = 0;   // segments 1 .. fetched are on their way or here
  for (int g = 1; g <= kStages; ++g) fetch(fetched = g);
  float next[kRows];   // the next segment's S
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    e[i * kGdnDim + d] = s[i * kGdnDim];
    next[i] = s[stride + i * kGdnDim];
  }
  __syncthreads();
  bool ok = true;
  for (int64_t g = 1; g + 1 < segs; ++g) {
    s += stride;
    float own[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      own[i] = next[i];
      if (g + 2 < segs) next[i] = s[stride + i * kGdnDim];
    }
    ok = scan_wait(&full[(g - 1) % kStages], ((g - 1) / kStages) & 1, abort, ca.wait_ns, 350);
    if (__syncthreads_or(!ok)) break;
    const float* pg = join_sh + ((g - 1) % kStages) * kTile + 32 * warp * kGdnDim + 4 * lane;
    float4 acc[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = 0; k < 32; k += 4) {
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const float4*>(pg + (k + j) * kGdnDim);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float4 y = *reinterpret_cast<const float4*>(e + i * kGdnDim + 32 * warp + k);
        acc[i].x = fmaf(y.x, x[0].x, fmaf(y.y, x[1].x, fmaf(y.z, x[2].x, fmaf(y.w, x[3].x, acc[i].x))));
        acc[i].y = fmaf(y.x, x[0].y, fmaf(y.y, x[1].y, fmaf(y.z, x[2].y, fmaf(y.w, x[3].y, acc[i].y))));
        acc[i].z = fmaf(y.x, x[0].z, fmaf(y.y, x[1].z, fmaf(y.z, x[2].z, fmaf(y.w, x[3].z, acc[i].z))));
        acc[i].w = fmaf(y.x, x[0].w, fmaf(y.y, x[1].w, fmaf(y.z, x[2].w, fmaf(y.w, x[3].w, acc[i].w))));
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      *reinterpret_cast<float4*>(part + (warp * kRows + i) * kGdnDim + 4 * lane) = acc[i];
    __syncthreads();   // P and E are done with, the parts are in place
    fetch(fetched = g + kStages);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float* q = part + i * kGdnDim + d;
      const float x = own[i] + ((q[0] + q[kRows * kGdnDim]) + (q[2 * kRows * kGdnDim] + q[3 * kRows * kGdnDim]));
      e[i * kGdnDim + d] = x;
      s[i * kGdnDim] = x;
    }
    // (the next turn's barrier puts E in place before it is read)
  }
  if (d == 0 && *abort) {   // no copy may land after the CTA is gone
    report_error(ca.st, kErrTimeout, 350);
    for (int64_t g = fetched > kStages ? fetched - kStages + 1 : 1; g <= fetched && g + 1 < segs; ++g)
      if (g != absent) mbar_drain(&full[(g - 1) % kStages], ((g - 1) / kStages) & 1);
  }
}

}  // namespace qsa
