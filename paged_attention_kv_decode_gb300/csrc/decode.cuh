// What the decode kernels share (decode.cu, decode_fp8.cu): their parameters, the token
// range of a work item, the longest-first order, and the merge of the warps' softmax
// states into the item's result.
#pragma once

#include <math.h>

#include "common.cuh"

namespace metis {

struct DecodeParams {
  const void* q;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  float* lse_out;
  float* part_out;  // split-KV partials [S, H, max_parts, D] (NULL: no split)
  float* part_lse;  // [S, H, max_parts]
  int S, H, G, D, bs, max_blocks, num_blocks, r;
  float scale_log2;  // softmax scale * log2(e)
  int partition_size;
  int max_parts;
  int cap;  // tokens readable per sequence: min(max_blocks * bs, max_seq_len)
  // Decodes of a chunked-prefill batch (NULL otherwise): the batch's cu_q_lens.
  // Sequence s is handled only if rows[s + 1] - rows[s] == 1 and that row exists; its
  // query, output and lse row is rows[s] of the packed [T, H, D] tensors.
  const int32_t* rows;
  int T;
};

// The sequence's single query row in a mixed batch of T packed rows; -1: it has several,
// none, or one outside them.
__device__ __forceinline__ int single_row(const int32_t* rows, int T, int s) {
  const int r0 = rows[s];
  return r0 >= 0 && r0 < T && rows[s + 1] == r0 + 1 ? r0 : -1;
}

// Output (and query) row of sequence s; -1 when the call skips it (single_row).
__device__ __forceinline__ int decode_row(const DecodeParams& p, int s) {
  return p.rows ? single_row(p.rows, p.T, s) : s;
}

// Tokens [t0, t1) of partition `part` (of P tokens each) of a sequence of L; t1 <= t0: none.
// (t0 + P may pass 2^31.)
__host__ __device__ __forceinline__ void partition_tokens(int L, int P, int part, int& t0, int& t1) {
  t0 = part * P;
  t1 = L - t0 > P ? t0 + P : L;
}

// Token range of this CTA, after clamping the sequence length.  Returns
// false when the CTA has nothing to do (after writing what an empty
// partition or sequence must leave behind).
// tid / nthr: this thread's index among the threads that share the item.
// status: the calling file's device status word.
template <typename OutT>
__device__ __forceinline__ bool decode_range(const DecodeParams& p, int part, int g, int s, int orow, int& t0,
                                             int& t1, int tid, int nthr, unsigned int* status) {
  int L_raw = p.seq_lens[s];
  int L = L_raw;
  if (L > p.cap) {
    if (tid == 0) atomicOr(status, METIS_STATUS_SEQ_TOO_LONG);
    L = p.cap;
  }
  if (L < 0) L = 0;
  if (p.partition_size > 0) {
    partition_tokens(L, p.partition_size, part, t0, t1);
  } else {
    t0 = 0;
    t1 = L;
  }
  if (t1 > t0) return true;
  if (p.partition_size > 0) {
    // A partition the merge will look at but that holds no readable token.
    if (L_raw > 0 && t0 < L_raw && tid < p.r)
      p.part_lse[((size_t)s * p.H + g * p.r + tid) * p.max_parts + part] = -INFINITY;
  } else {
    OutT* o = reinterpret_cast<OutT*>(p.out) + ((size_t)orow * p.H + (size_t)g * p.r) * p.D;
    for (int i = tid; i < p.r * p.D; i += nthr) o[i] = OutT(0.0f);
    if (p.lse_out && tid < p.r) p.lse_out[(size_t)orow * p.H + g * p.r + tid] = -INFINITY;
  }
  return false;
}

template <typename OutT>
__device__ __forceinline__ void store4(OutT* dst, float a, float b, float c, float d);

template <>
__device__ __forceinline__ void store4<float>(float* dst, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
}

template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* dst, float a, float b, float c, float d) {
  uint2 v;
  v.x = pack_bf16x2(a, b);
  v.y = pack_bf16x2(c, d);
  *reinterpret_cast<uint2*>(dst) = v;
}

// Merge the per-warp online-softmax states held in shared memory (cm, cl:
// [NW][8] running max in log2 units and running sum; co: [NW][D][8] unnormalised
// accumulators) and write the CTA's result: the final output row or a
// split-KV partial.  NAN_LSE_AS_INF: a partial whose lse is NaN says +inf, which the
// merge turns into NaN (it passes a NaN over).
template <typename OutT, int NW, bool NAN_LSE_AS_INF = false>
__device__ __forceinline__ void combine_and_store(const DecodeParams& p, const float* cm, const float* cl,
                                                  const float* co, int part, int g, int s, int orow, int tid) {
  const int D = p.D;
  const int nq = D / 4;
  for (int idx = tid; idx < p.r * nq; idx += NW * 32) {
    const int h = idx / nq;
    const int d = (idx - h * nq) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, cm[w * 8 + h]);
    float Lsum = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = cm[w * 8 + h];
      if (mw == -INFINITY) continue;
      const float f = exp2_approx(mw - M);
      Lsum += cl[w * 8 + h] * f;
      const float* c = co + ((size_t)w * D + d) * 8 + h;
      a0 += c[0] * f;
      a1 += c[8] * f;
      a2 += c[16] * f;
      a3 += c[24] * f;
    }
    const float inv = 1.0f / Lsum;
    const int head = g * p.r + h;
    const float lse = (M + log2f(Lsum)) * kLn2;
    if (p.partition_size > 0) {
      float* dst = p.part_out + (((size_t)s * p.H + head) * p.max_parts + part) * D + d;
      *reinterpret_cast<float4*>(dst) = make_float4(a0 * inv, a1 * inv, a2 * inv, a3 * inv);
      if (d == 0)
        p.part_lse[((size_t)s * p.H + head) * p.max_parts + part] = NAN_LSE_AS_INF && lse != lse ? INFINITY : lse;
    } else {
      OutT* dst = reinterpret_cast<OutT*>(p.out) + ((size_t)orow * p.H + head) * D + d;
      store4<OutT>(dst, a0 * inv, a1 * inv, a2 * inv, a3 * inv);
      if (d == 0 && p.lse_out) p.lse_out[(size_t)orow * p.H + head] = lse;
    }
  }
}

// Longest-first order for the unsplit path: CTAs launch in grid order, so the
// CTA with z-index k takes the sequence of rank k by length (ties: lower index
// first).  Every CTA ranks the whole batch itself -- S^2 / blockDim comparisons in
// shared memory, small for the batches it is used on (kMaxRankSeqs) -- which
// needs no schedule kernel and no workspace.  The heaviest sequences start first
// and the short ones fill the SMs that free up, instead of a ragged last wave.
constexpr int kMaxRankSeqs = 128;

__device__ __forceinline__ int seq_of_rank(const DecodeParams& p, int rank, int* lens, int* found) {
  // sequences the call skips rank last
  for (int i = threadIdx.x; i < p.S; i += blockDim.x)
    lens[i] = decode_row(p, i) < 0 ? -1 : min(max(p.seq_lens[i], 0), p.cap);
  if (threadIdx.x == 0) *found = rank;
  __syncthreads();
  for (int c = threadIdx.x; c < p.S; c += blockDim.x) {
    const int Lc = lens[c];
    int r = 0;
    for (int k = 0; k < p.S; ++k) r += (lens[k] > Lc) || (lens[k] == Lc && k < c);
    if (r == rank) *found = c;
  }
  __syncthreads();
  return *found;
}

}  // namespace metis
