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
// Each row is read once and written once.  A warp takes a token, or where there are few
// tokens a share of a token's heads: a row of head_dim elements is 8 to 32 lanes with 16 bytes each, so the
// token's angles and the weights stay in registers over all of the warp's rows, kRows loads of which are in
// flight per lane.  The partner of a pair is in the same lane (interleaved) or half of rotary_dim away: a
// shuffle.  With a = weight cos and b = +- weight sin formed once for a warp's token, an element costs two packed
// fp32 operations and its conversions.
//
// Measured, 8,240 rows of 32 + 8 + 8 heads x 128 (207 MB): 42.6 us, 4.8 TB/s, 73 % of a copy (a CTA per token
// with the factors per row took 72); without the pages 37.5 (169 MB), fp32 60.2; 64 rows 2.8 us.  Neither HBM (47 % of
// its nominal rate) nor the SMs (48 %) are busy then: it is the latency of a warp's start, its token's position and slot,
// then angles and rows, one token and exit, with 28 warps an SM to cover it.  (The write alone: 81 % of a copy.)
#include <algorithm>

#include "../../include/metis_attn.h"
#include "common.cuh"
#include "host.h"

namespace metis {

__device__ unsigned int g_status_rope = 0;

constexpr int kRopeWarps = 4;
// (8,240 rows: 2 to 8 rows in flight on 5 to 16 CTAs are within 5 %; 2 x 8 took 45.1 us)
constexpr int kRows = 3;  // rows a lane has in flight
constexpr int kRopeCtas = 7;   // CTAs of an SM
constexpr int kRopeFill = 28;  // warps for each SM, below which tokens are shared by several

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

// 16 bytes of a row as pairs of fp32, and back
template <typename T>
struct RopeVec;
template <>
struct RopeVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, uint64_t* x) {
    x[0] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct RopeVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, uint64_t* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
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

// How a warp's rows are worked on: lane `at` of a row of LANES lanes holds its elements at * N .. + N - 1.
struct RopeLane {
  int at, sub, mate;   // sub: the lane's row among the warp's; mate: the lane that holds the partners
  bool turned, inter;  // the lane's elements are rotated; their partners are in the lane itself
  bool known;          // the position has a row in the table (else: reads as zeros)
};

// The rows [lo, hi) of one kind (queries or keys) of a token: out = f (x a + x' b), x' the partner of x, with
// a = weight cos and b = +-weight' sin (weight' the partner's), f = 1 / sqrt(mean(x^2) + eps) or 1.
template <typename T, int D, typename Source, typename Target>
__device__ __forceinline__ void turn_rows(const RopeParams& p, const RopeLane& me, const float* turn,
                                          const void* weight, int lo, int hi, Source source, Target target) {
  using Vec = RopeVec<T>;
  constexpr int N = Vec::kN, LANES = D / N, STEP = 32 / LANES;
  uint4 raw[kRows];
  auto load = [&](int row0) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      raw[j] = make_uint4(0u, 0u, 0u, 0u);
      const int row = row0 + j * STEP + me.sub;
      if (row < hi) raw[j] = *source(row);
    }
  };
  load(lo);
  // the factors of this lane's elements: element e belongs to pair e / 2 (interleaved) or e mod R / 2
  float a[N], b[N];
  {
    const int e0 = me.at * N, half = p.R / 2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = 1.f;
      b[i] = 0.f;
    }
    if (me.turned) {
      if (me.inter) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          a[i] = turn[(e0 + i) / 2];
          b[i] = (i & 1) ? turn[half + (e0 + i) / 2] : -turn[half + (e0 + i) / 2];
        }
      } else {
        const bool low = e0 < half;
        const float4* t4 = reinterpret_cast<const float4*>(turn + (low ? e0 : e0 - half));
        const float sign = low ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 c = t4[i / 4], s = t4[half / 4 + i / 4];
          a[i] = c.x, a[i + 1] = c.y, a[i + 2] = c.z, a[i + 3] = c.w;
          b[i] = sign * s.x, b[i + 1] = sign * s.y, b[i + 2] = sign * s.z, b[i + 3] = sign * s.w;
        }
      }
    }
    if (!me.known && me.turned) {
#pragma unroll
      for (int i = 0; i < N; ++i) a[i] = b[i] = 0.f;
    }
    if (weight != nullptr) {
      const uint4* w4 = reinterpret_cast<const uint4*>(weight);
      uint64_t w2[N / 2], m2[N / 2];
      Vec::unpack(w4[me.at], w2);
      Vec::unpack(w4[me.mate % LANES], m2);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        float w0, w1, m0, m1;
        f2_unpack(w2[i], w0, w1);
        f2_unpack(m2[i], m0, m1);
        a[2 * i] *= w0;
        a[2 * i + 1] *= w1;
        b[2 * i] *= me.inter ? m1 : m0;
        b[2 * i + 1] *= me.inter ? m0 : m1;
      }
    }
  }
  uint64_t a2[N / 2], b2[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    a2[i] = f2_pack(a[2 * i], a[2 * i + 1]);
    b2[i] = f2_pack(b[2 * i], b[2 * i + 1]);
  }
  for (int row0 = lo; row0 < hi; row0 += kRows * STEP) {
    if (row0 != lo) load(row0);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (row0 + j * STEP >= hi) break;  // (uniform over the warp)
      uint64_t x[N / 2], m[N / 2];
      Vec::unpack(raw[j], x);
      uint4 other = make_uint4(0u, 0u, 0u, 0u);  // (not rotated: b is zero, and 0 * infinity is not)
      if (p.R > 0) {
        uint4 got = raw[j];
        if (!me.inter) {  // (uniform)
          got.x = __shfl_sync(0xffffffffu, raw[j].x, me.mate);
          got.y = __shfl_sync(0xffffffffu, raw[j].y, me.mate);
          got.z = __shfl_sync(0xffffffffu, raw[j].z, me.mate);
          got.w = __shfl_sync(0xffffffffu, raw[j].w, me.mate);
        }
        if (me.turned) other = got;
      }
      Vec::unpack(other, m);
      if (me.inter) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          float m0, m1;
          f2_unpack(m[i], m0, m1);
          m[i] = f2_pack(m1, m0);
        }
      }
      float f = 1.f;
      if (weight != nullptr) {
        auto squares = [&]() {
          uint64_t s2 = f2_mul(x[0], x[0]);
#pragma unroll
          for (int i = 1; i < N / 2; ++i) s2 = f2_fma(x[i], x[i], s2);
          float s0, s1;
          f2_unpack(s2, s0, s1);
          return row_sum<LANES>(s0 + s1);
        };
        float ss = squares(), eps = p.eps;
        // Squares that leave fp32's range are taken of x times a power of two, which eps takes along: exact, and rare.
        const float up = !(ss < 1.3e36f) ? 8.271806e-25f /* 2^-80 */ : ss + eps < 1e-30f ? 1.2089258e24f /* 2^80 */ : 1.f;
        if (__any_sync(0xffffffffu, up != 1.f)) {
          const uint64_t up2 = f2_pack(up, up);
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            x[i] = f2_mul(x[i], up2);
            m[i] = f2_mul(m[i], up2);
          }
          ss = squares();
          eps = eps * up * up;
        }
        f = rsqrtf(fmaf(ss, 1.0f / D, eps));
      }
      const uint64_t f2 = f2_pack(f, f);
      float y[N];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const uint64_t v = f2_mul(f2_fma(m[i], b2[i], f2_mul(x[i], a2[i])), f2);
        f2_unpack(v, y[2 * i], y[2 * i + 1]);
      }
      const int row = row0 + j * STEP + me.sub;
      if (row < hi) target(row, Vec::pack(y));
    }
  }
}

// The rows of a token: 0 .. H - 1 are queries, then G keys, then (v given) G values.  `share` warps take
// `chunk` of them each.
template <typename T, int D>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeCtas) qk_norm_rope_kernel(const RopeParams p, const int interleaved,
                                                                       const int num_tokens, const int share,
                                                                       const int chunk) {
  constexpr int N = RopeVec<T>::kN, LANES = D / N, STEP = 32 / LANES;  // STEP: rows of the warp at a time
  pdl_launch_dependents();
  pdl_wait();  // rows, positions and slots may be what the kernel in front writes
  const long long item = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const long long n = item / share;
  if (n >= num_tokens) return;
  const int lane = threadIdx.x & 31;
  const int lo = (int)(item - n * share) * chunk, hi = min(p.H + (p.v ? 2 : 1) * p.G, lo + chunk);

  // (No branch on either before the first rows are on their way.)
  long long slot = n;
  if (p.slots) slot = p.slots[n];
  int pos = 0;
  if (p.R > 0) pos = p.positions[n];
  RopeLane me;
  me.known = p.R == 0 || (pos >= 0 && pos < p.max_position);
  const float* turn = p.cos_sin + (long long)(me.known ? pos : 0) * p.R;
  me.at = lane % LANES;
  me.sub = lane / LANES;
  me.turned = me.at * N < p.R;
  me.inter = interleaved != 0;
  const int half_lanes = p.R / (2 * N);
  me.mate = interleaved || !me.turned ? lane : me.at < half_lanes ? lane + half_lanes : lane - half_lanes;

  if (lo < p.H) {
    const T* from = reinterpret_cast<const T*>(p.q) + n * p.q_stride;
    uint4* to = reinterpret_cast<uint4*>(p.q_out) + n * p.H * LANES + me.at;
    turn_rows<T, D>(p, me, turn, p.q_weight, lo, min(hi, p.H),
                    [&](int row) { return reinterpret_cast<const uint4*>(from + row * D) + me.at; },
                    [&](int row, const uint4& v) { to[row * LANES] = v; });
  }
  if (!me.known && lane == 0 && lo < p.H + p.G) atomicOr(&g_status_rope, METIS_STATUS_BAD_POSITION);
  if (hi <= p.H) return;
  if (p.slots && slot >= p.total_slots) {
    if (lane == 0) atomicOr(&g_status_rope, METIS_STATUS_BAD_BLOCK_ID);
    return;
  }
  if (slot < 0) return;  // a padding row: neither its key nor its value is written
  if (lo < p.H + p.G) {
    const T* from = reinterpret_cast<const T*>(p.k) + n * p.k_stride;
    uint4* to = reinterpret_cast<uint4*>(p.k_out) + slot * p.G * LANES + me.at;
    turn_rows<T, D>(p, me, turn, p.k_weight, max(lo - p.H, 0), min(hi - p.H, p.G),
                    [&](int row) { return reinterpret_cast<const uint4*>(from + row * D) + me.at; },
                    [&](int row, const uint4& v) { to[row * LANES] = v; });
  }
  if (hi > p.H + p.G) {
    const T* from = reinterpret_cast<const T*>(p.v) + n * p.v_stride;
    uint4* to = reinterpret_cast<uint4*>(p.v_out) + slot * p.G * LANES + me.at;
    const int last = hi - p.H - p.G;
    for (int row0 = max(lo - p.H - p.G, 0); row0 < last; row0 += kRows * STEP) {
      uint4 raw[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (row0 + j * STEP + me.sub < last)
          raw[j] = reinterpret_cast<const uint4*>(from + (row0 + j * STEP + me.sub) * D)[me.at];
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (row0 + j * STEP + me.sub < last) to[(row0 + j * STEP + me.sub) * LANES] = raw[j];
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
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "querying the SM count: %s", cudaGetErrorString(e));
  // a token's rows, as often as a warp holds some at a time; few tokens: shared by as many warps as fill the GPU
  const int step = 32 / (int)(head_dim / vec);
  const long long rows = (long long)p.H + (pages ? 2 : 1) * (long long)p.G, steps = (rows + step - 1) / step;
  const long long want = std::max<long long>(1, std::min<long long>(steps, (long long)kRopeFill * sms / num_tokens));
  const long long chunk = (steps + want - 1) / want * step, share = (rows + chunk - 1) / chunk;
  if (rows * head_dim > 0x7fffffffLL) return fail(METIS_E_SHAPE, "too many heads");
  const long long ctas = (share * num_tokens + kRopeWarps - 1) / kRopeWarps;
  if (ctas > 0x7fffffffLL) return fail(METIS_E_SHAPE, "too many rows");
  auto launch = [&](auto kern) {
    return launch_dependent(kern, dim3((unsigned)ctas), dim3(kRopeWarps * 32), 0, st, "qk_norm_rope_kernel launch", p,
                            interleaved ? 1 : 0, num_tokens, (int)share, (int)chunk);
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
