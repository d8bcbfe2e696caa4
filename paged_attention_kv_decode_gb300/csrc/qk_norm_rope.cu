// Between a layer's projection and its attention: queries and keys normalised per head, rotated
// by their positions, keys and values into their pages -- one pass over the step's new rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w          over the head's dims (no weight: y = x)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)      for the pairs (a, b) of the first
//                 rotary_dim dims: (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when interleaved
//
// with cos and sin from a table's row for the token's position (the pages: "paged attention ...
// kernels fed by the scheduler's block table", vllm-metal article, sections 3 and 4; the write is
// the one of cache_write.cu).  Everything between load and store is fp32: one rounding.
//
// Bound by HBM: each row is read once and written once.  One CTA per token, its warps share the
// token's heads: a row of head_dim elements is 8 to 32 lanes with 16 bytes each, so a warp's
// angles and weights stay in registers over all of its rows, up to kRows of which are in flight.
// The partner of a pair is in the same lane (interleaved) or half of rotary_dim away: a shuffle.
#include <algorithm>

#include "../../include/metis_attn.h"
#include "common.cuh"
#include "host.h"

namespace metis {

__device__ unsigned int g_status_rope = 0;

constexpr int kRopeThreads = 256;
constexpr int kRows = 3;  // rows a thread has in flight

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;          // NULL: rows of q and k only
  const void* q_weight;   // NULL: not normalised
  const void* k_weight;
  const float* cos_sin;   // [max_position, R]: R / 2 cosines, then as many sines
  const int32_t* positions;
  const int64_t* slots;   // NULL: k_out is [T, G, D]
  void* q_out;
  void* k_out;            // rows or pages
  void* v_out;
  long long q_stride, k_stride, v_stride;  // elements from token to token
  long long total_slots;
  float eps;
  int H, G, R, max_position;
};

template <typename T>
struct RopeVec;
template <>
struct RopeVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct RopeVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

// Sum over the LANES neighbouring lanes of a row
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// x[] of the row's lane -> x / sqrt(mean(x^2) + eps) * w.  Squares that leave fp32's range are taken
// of x times a power of two, which also goes to eps: exact, and rare.
template <int D, int N, int LANES>
__device__ __forceinline__ void normalise(float* x, const float* w, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
  ss = row_sum<LANES>(ss);
  const float up = !(ss < 1.3e36f) ? 8.271806e-25f /* 2^-80 */ : ss + eps < 1e-30f ? 1.2089258e24f /* 2^80 */ : 1.f;
  if (__any_sync(0xffffffffu, up != 1.f)) {
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] *= up;
      ss = fmaf(x[i], x[i], ss);
    }
    ss = row_sum<LANES>(ss);
    eps = eps * up * up;
  }
  const float f = 1.0f / sqrtf(fmaf(ss, 1.0f / D, eps));
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = x[i] * f * w[i];
}

// The rows of one token: rows 0 .. H - 1 are queries, then G keys, then (v given) G values.
template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p, const int interleaved) {
  using Vec = RopeVec<T>;
  constexpr int N = Vec::kN, LANES = D / N, PER_WARP = 32 / LANES;
  constexpr int STEP = kRopeThreads / LANES;  // rows of the CTA at a time
  pdl_launch_dependents();
  pdl_wait();  // rows, positions and slots may be what the kernel in front writes
  const long long n = blockIdx.x;
  const int lane = threadIdx.x & 31, at = lane % LANES;  // this thread's elements: at * N ..
  const int first = (threadIdx.x >> 5) * PER_WARP + lane / LANES;
  const int rows = p.H + (p.v ? 2 : 1) * p.G;

  auto source = [&](int row) -> const uint4* {
    const T* base;
    if (row < p.H)
      base = reinterpret_cast<const T*>(p.q) + n * p.q_stride + (long long)row * D;
    else if (row < p.H + p.G)
      base = reinterpret_cast<const T*>(p.k) + n * p.k_stride + (long long)(row - p.H) * D;
    else
      base = reinterpret_cast<const T*>(p.v) + n * p.v_stride + (long long)(row - p.H - p.G) * D;
    return reinterpret_cast<const uint4*>(base) + at;
  };
  uint4 raw[kRows];
  auto load = [&](int row0) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      raw[j] = make_uint4(0u, 0u, 0u, 0u);
      if (row0 + j * STEP < rows) raw[j] = *source(row0 + j * STEP);
    }
  };
  load(first);

  // angles of this lane's elements: element e belongs to pair e / 2 (interleaved) or e mod R / 2
  float c[N], s[N];
  long long slot = n;
  {
    const int half = p.R / 2;
    int pos = 0;
    if (p.R > 0) pos = p.positions[n];
    if (p.slots) slot = p.slots[n];
    const bool known = pos >= 0 && pos < p.max_position;
    if (p.R > 0 && !known && threadIdx.x == 0) atomicOr(&g_status_rope, METIS_STATUS_BAD_POSITION);
    const float* turn = p.cos_sin + (long long)pos * p.R;
    const int e0 = at * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
    if (e0 < p.R) {
      if (!known) {  // reads as zeros
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = s[i] = 0.f;
      } else if (interleaved) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          c[i] = turn[(e0 + i) / 2];
          s[i] = turn[half + (e0 + i) / 2];
          if (!(i & 1)) s[i] = -s[i];
        }
      } else {
        const bool low = e0 < half;
        const float4* t4 = reinterpret_cast<const float4*>(turn + (low ? e0 : e0 - half));
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 a = t4[i / 4], b = t4[half / 4 + i / 4];
          const float sign = low ? -1.f : 1.f;
          c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
          s[i] = sign * b.x, s[i + 1] = sign * b.y, s[i + 2] = sign * b.z, s[i + 3] = sign * b.w;
        }
      }
    }
  }
  const int half_lanes = p.R / (2 * N);
  // the lane that holds this lane's partners (interleaved, or not rotated: itself)
  const int mate = interleaved || at * N >= p.R ? lane : at < half_lanes ? lane + half_lanes : lane - half_lanes;
  uint4 qw = make_uint4(0u, 0u, 0u, 0u), kw = qw;
  if (p.q_weight) qw = reinterpret_cast<const uint4*>(p.q_weight)[at];
  if (p.k_weight) kw = reinterpret_cast<const uint4*>(p.k_weight)[at];
  if (p.slots && slot >= p.total_slots) {
    if (threadIdx.x == 0) atomicOr(&g_status_rope, METIS_STATUS_BAD_BLOCK_ID);
    slot = -1;
  }

  const int warp_first = (threadIdx.x >> 5) * PER_WARP;
  for (int row0 = first, w0 = warp_first; w0 < rows; row0 += kRows * STEP, w0 += kRows * STEP) {
    if (w0 != warp_first) load(row0);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (w0 + j * STEP >= rows) break;  // (uniform over the warp)
      const int row = row0 + j * STEP;
      uint4 out = raw[j];
      const bool is_q = row < p.H, is_v = row >= p.H + p.G;
      if (w0 + j * STEP < p.H + p.G) {  // a warp with a query or a key: all lanes take part in the shuffles
        float x[N];
        Vec::unpack(raw[j], x);
        const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
        if (norm_q || norm_k) {
          float y[N], w[N];
#pragma unroll
          for (int i = 0; i < N; ++i) y[i] = x[i];
          Vec::unpack(is_q ? qw : kw, w);
          normalise<D, N, LANES>(y, w, p.eps);
          if (is_q ? norm_q : norm_k) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = y[i];
          }
        }
        if (p.R > 0) {
          float z[N];
          if (interleaved) {
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = x[i ^ 1];
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = __shfl_sync(0xffffffffu, x[i], mate);
          }
          if (at * N < p.R) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = fmaf(x[i], c[i], z[i] * s[i]);
          }
        }
        if (!is_v) out = Vec::pack(x);
      }
      if (row >= rows) continue;
      if (is_q) {
        reinterpret_cast<uint4*>(p.q_out)[(n * p.H + row) * LANES + at] = out;
      } else if (slot >= 0) {
        uint4* to = reinterpret_cast<uint4*>(is_v ? p.v_out : p.k_out);
        to[(slot * p.G + (row - p.H - (is_v ? p.G : 0))) * LANES + at] = out;
      }
    }
  }
}

int rope_status(uint32_t* bits, int clear) {
  unsigned int v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_status_rope, sizeof(v));
  if (e == cudaSuccess && clear) {
    unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_status_rope, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  *bits |= v;
  return METIS_OK;
}

// Both entry points; slots NULL: rows of q and k only.
static int norm_rope(const RopeParams& p, int num_tokens, int head_dim, int interleaved, int dtype, bool pages,
                     cudaStream_t st) {
  if (num_tokens < 0) return fail(METIS_E_SHAPE, "num_tokens < 0");
  if (num_tokens == 0) return METIS_OK;
  if (!p.q || !p.k || !p.q_out || !p.k_out || (pages && (!p.v || !p.v_out || !p.slots)) ||
      (p.R > 0 && (!p.cos_sin || !p.positions)))
    return fail(METIS_E_NULL, "q, k, their outputs, cos_sin and positions (and v, the caches and slot_mapping) are required");
  if (p.H <= 0 || p.G <= 0 || p.R < 0 || (p.R > 0 && p.max_position <= 0) || (pages && p.total_slots <= 0))
    return fail(METIS_E_SHAPE, "sizes must be positive");
  if (dtype != METIS_F32 && dtype != METIS_BF16) return fail(METIS_E_UNSUPPORTED, "dtype must be METIS_F32 or METIS_BF16");
  if (head_dim != 64 && head_dim != 128) return fail(METIS_E_UNSUPPORTED, "head_dim must be 64 or 128");
  if (p.R % 16 || p.R > head_dim) return fail(METIS_E_UNSUPPORTED, "rotary_dim must be a multiple of 16 up to head_dim");
  if (!(p.eps >= 0.f)) return fail(METIS_E_SHAPE, "eps must be >= 0");
  const long long vec = dtype == METIS_F32 ? 4 : 8;
  const long long q_row = (long long)p.H * head_dim, k_row = (long long)p.G * head_dim;
  if (p.q_stride < q_row || p.k_stride < k_row || (pages && p.v_stride < k_row))
    return fail(METIS_E_SHAPE, "a token stride is shorter than the token's heads");
  if (p.q_stride % vec || p.k_stride % vec || (pages && p.v_stride % vec))
    return fail(METIS_E_ALIGN, "token strides must be multiples of 16 bytes");
  if ((p.q_out == p.q && p.q_stride != q_row) || (!pages && p.k_out == p.k && p.k_stride != k_row))
    return fail(METIS_E_SHAPE, "in place needs dense rows");
  if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.q_weight, 16) ||
      !aligned(p.k_weight, 16) || !aligned(p.cos_sin, 16) || !aligned(p.q_out, 16) || !aligned(p.k_out, 16) ||
      !aligned(p.v_out, 16) || !aligned(p.positions, 4) || !aligned(p.slots, 8))
    return fail(METIS_E_ALIGN, "tensors must be 16-byte aligned (positions: 4-byte, slot_mapping: 8-byte)");
  const dim3 grid((unsigned)num_tokens), block(kRopeThreads);
  auto launch = [&](auto kern) {
    return launch_dependent(kern, grid, block, 0, st, "qk_norm_rope_kernel launch", p, interleaved ? 1 : 0);
  };
  if (dtype == METIS_F32)
    return head_dim == 64 ? launch(qk_norm_rope_kernel<float, 64>) : launch(qk_norm_rope_kernel<float, 128>);
  return head_dim == 64 ? launch(qk_norm_rope_kernel<__nv_bfloat16, 64>) : launch(qk_norm_rope_kernel<__nv_bfloat16, 128>);
}

}  // namespace metis

using namespace metis;

extern "C" int metis_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight,
                                  const float* cos_sin, const int32_t* positions, void* q_out, void* k_out,
                                  int num_tokens, int num_heads, int num_kv_heads, int head_dim, int64_t q_stride,
                                  int64_t k_stride, int rotary_dim, int max_position, int interleaved, float eps,
                                  int dtype, void* stream) {
  clear_error();
  RopeParams p{};
  p.q = q;
  p.k = k;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.eps = eps;
  p.H = num_heads;
  p.G = num_kv_heads;
  p.R = rotary_dim;
  p.max_position = max_position;
  return norm_rope(p, num_tokens, head_dim, interleaved, dtype, false, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int metis_qk_norm_rope_and_cache(const void* q, const void* k, const void* v, const void* q_weight,
                                            const void* k_weight, const float* cos_sin, const int32_t* positions,
                                            void* q_out, void* k_cache, void* v_cache, const int64_t* slot_mapping,
                                            int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                            int64_t q_stride, int64_t k_stride, int64_t v_stride, int rotary_dim,
                                            int max_position, int interleaved, float eps, int block_size,
                                            int num_blocks, int dtype, void* stream) {
  clear_error();
  if (num_tokens > 0 && (block_size <= 0 || num_blocks <= 0)) return fail(METIS_E_SHAPE, "sizes must be positive");
  RopeParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.slots = slot_mapping;
  p.q_out = q_out;
  p.k_out = k_cache;
  p.v_out = v_cache;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.total_slots = (long long)block_size * num_blocks;
  p.eps = eps;
  p.H = num_heads;
  p.G = num_kv_heads;
  p.R = rotary_dim;
  p.max_position = max_position;
  return norm_rope(p, num_tokens, head_dim, interleaved, dtype, true, reinterpret_cast<cudaStream_t>(stream));
}
