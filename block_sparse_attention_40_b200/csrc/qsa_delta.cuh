// qsa_delta.cuh -- the gated delta rule from and to a pool of states: token by token for
// decoding rows.  (The layer over whole sequences from a zero state is in qsa_gdn.cuh.)
//
// Per row (sequence) and value head, with the state S (d_v x d_k, fp32) kept in a slot of a
// caller-owned pool [slots][heads][128 (v)][128 (k)]:
//     S <- a S + beta (v - a S k) k^T,   o = S q,      a = exp(max(log_alpha, -87)).
// heads / key_heads value heads in a row share one key (and query) head.
//
// A row's slot is skipped (state and outputs untouched) when it lies outside the pool, which
// is how rows of a padded batch are marked, or when an earlier row of the call names the same
// slot: the first row owns it.

#pragma once

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
  int32_t heads, key_heads;
  float* states;            // [num_slots][heads][128][128]
  __nv_bfloat16* out;       // [tokens][heads][128]
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

// Whether an earlier row with tokens to take names row r's slot.  All threads of the block call
// it, and all get the answer.
__device__ __forceinline__ bool delta_slot_taken(const DeltaArgs& a, int r, int slot) {
  if (a.slots == nullptr) return false;
  int hit = 0;
  for (int i = threadIdx.x; i < r; i += blockDim.x) hit |= a.slots[i] == slot;
  return __syncthreads_or(hit) != 0;
}

__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float* f) {
  f[0] = __uint_as_float(w << 16);
  f[1] = __uint_as_float(w & 0xffff0000u);
}

// ---------------------------------------------------------------------------------------
// Token by token.  Eight lanes hold one value row of S (16 key columns each, in four groups of
// four so that a row's loads are 128-byte segments), RV rows a thread, so a block of 128
// threads holds 16 * RV rows and the grid (heads, rows, 128 / (16 RV)) covers S.  The state
// stays in registers over a row's tokens: it is read once and written once.  With
// o = a S q + u (k.q), u = beta (v - a S k), both dots of a token come from the old state in one
// pass, and the reductions are three shuffles.  Bound by the state's bytes: 128 KB per (row,
// head) against about 4.5 KB of everything else at one token.
constexpr int kStepThreads = 128;

template <int RV>
__global__ void __launch_bounds__(kStepThreads) k_delta_step(DeltaArgs a) {
  const int tid = threadIdx.x, l8 = tid & 7, grp = tid >> 3;   // 16 groups of 8 lanes
  const int h = blockIdx.x, r = blockIdx.y;
  const int v0 = (blockIdx.z * 16 + grp) * RV;
  int64_t n;
  const int64_t t0 = delta_row_tokens(a, r, &n);
  const int slot = a.slots != nullptr ? a.slots[r] : r;
  if (n <= 0 || slot < 0 || slot >= a.num_slots) return;
  const int kh = h / (a.heads / a.key_heads);
  float* st = a.states +
              ((static_cast<int64_t>(slot) * a.heads + h) * kGdnDim + v0) * kGdnDim + 4 * l8;
  float4 S[RV][4];
#pragma unroll
  for (int i = 0; i < RV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      S[i][j] = __ldcs(reinterpret_cast<const float4*>(st + i * kGdnDim + 32 * j));
  if (delta_slot_taken(a, r, slot)) return;
  for (int64_t t = t0; t < t0 + n; ++t) {
    const uint2* qp = reinterpret_cast<const uint2*>(a.q + (t * a.key_heads + kh) * kGdnDim) + l8;
    const uint2* kp = reinterpret_cast<const uint2*>(a.k + (t * a.key_heads + kh) * kGdnDim) + l8;
    const float al = expf(fmaxf(a.log_alpha[t * a.heads + h], kGdnMinLogAlpha));
    const float bt = a.beta[t * a.heads + h];
    const __nv_bfloat16* vp = a.v + (t * a.heads + h) * kGdnDim + v0;
    float q[16], k[16], x[RV];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint2 wq = qp[8 * j], wk = kp[8 * j];
      unpack_bf16x2(wq.x, q + 4 * j);
      unpack_bf16x2(wq.y, q + 4 * j + 2);
      unpack_bf16x2(wk.x, k + 4 * j);
      unpack_bf16x2(wk.y, k + 4 * j + 2);
    }
#pragma unroll
    for (int i = 0; i < RV; ++i) x[i] = __bfloat162float(vp[i]);
    float kq = 0.f, sk[RV], sq[RV];
#pragma unroll
    for (int e = 0; e < 16; ++e) kq = fmaf(k[e], q[e], kq);
#pragma unroll
    for (int i = 0; i < RV; ++i) {
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
      for (int i = 0; i < RV; ++i) {
        sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], o);
        sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
      }
    }
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      const float u = bt * (x[i] - al * sk[i]);
      float* s = reinterpret_cast<float*>(S[i]);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = fmaf(u, k[e], al * s[e]);
      if (l8 == 0)
        a.out[(t * a.heads + h) * kGdnDim + v0 + i] = __float2bfloat16(fmaf(u, kq, al * sq[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < RV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __stcs(reinterpret_cast<float4*>(st + i * kGdnDim + 32 * j), S[i][j]);
}

}  // namespace qsa
