// The 8-bit paged cache: quantising a step's K/V rows into their pages, and reading
// cached tokens back as bf16 or fp32 rows.
//
// An element of the cache is value(code) * 2^(b - 127): an e4m3 code and the scale byte
// b of its page and KV head (one byte each for K and V).  A power of two keeps the
// rounding of a code to three mantissa bits the only loss: x * 2^-k is exact, and so is
// reading back.
//
// Write.  For a page's new rows and one head, k is the smallest exponent with
// amax <= 448 * 2^k.  A page that already holds earlier tokens of its sequence keeps the
// larger of its byte and the new one; when it grows, the earlier codes are rounded again
// at the larger scale (an exact shift for all but the codes that become subnormal).
// Work is dealt by page, not by token, since a page's scale needs all of its new rows:
// item i of the grid finds its (sequence, page) by searching the monotone bound
//   off(s) = floor(cu_q_lens[s] / bs) + 2 s,
// which leaves each sequence at least as many items as pages its q rows can touch
// (floor((q + bs - 2) / bs) + 1 <= floor(q / bs) + 2, and
// floor(a + b) >= floor(a) + floor(b)); surplus items exit.  No schedule kernel, no
// workspace, no atomics on data: one launch.
#include <math.h>

#include <algorithm>

#include "../../include/metis_attn.h"
#include "common.cuh"
#include "fp8.cuh"
#include "host.h"

namespace metis {

__device__ unsigned int g_status_fp8 = 0;

// ---------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------
struct WriteFp8Params {
  const void* src[2];  // key, value [T, G, D]
  uint8_t* cache[2];   // codes [num_blocks, bs, G, D]
  uint8_t* scale[2];   // bytes [num_blocks, G]
  const int32_t* cu_q_lens;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int S, T, G, bs, max_blocks, num_blocks;
};

constexpr int kWriteWarps = 8;

// Index of the sequence that item i belongs to: the largest s with off(s) <= i, by a
// 32-way search of the warp.  All lanes return it.
__device__ __forceinline__ int seq_of_item(const WriteFp8Params& p, int i, int lane) {
  int lo = 0, n = p.S;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int s = lo + lane * step;
    const bool le = lane * step < n && max(__ldg(p.cu_q_lens + s), 0) / p.bs + 2ll * s <= i;
    const int c = max(__popc(__ballot_sync(0xffffffffu, le)), 1);
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
  }
  return lo;
}

// One warp: 16 slots of a page x one head of K or V.  Lanes hold 16-byte pieces of the
// new rows (8 bf16 or 4 fp32), several rows per load, all loads issued before the first
// use; the rows stay in registers between the maximum and the rounding, so each input is
// read once.  Pages of 32 or 64 slots take 2 or 4 warps that share their maximum.
template <typename T, int D>
__global__ void __launch_bounds__(kWriteWarps * 32) write_fp8_kernel(const WriteFp8Params p) {
  constexpr int VEC = 16 / (int)sizeof(T);  // elements per lane and load
  constexpr int LPR = D / VEC;              // lanes per row
  constexpr int RPL = 32 / LPR;             // rows per load
  constexpr int NL = 16 / RPL;              // loads for 16 slots
  __shared__ float part_max[kWriteWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int subs = p.bs / 16;                                         // warps per page, head and cache
  const int combo = (blockIdx.y * (blockDim.x >> 5) + warp) / subs;   // head * 2 + cache
  const int sub = warp & (subs - 1);                                  // (a block holds whole combos)

  const int i = blockIdx.x;
  const int s = seq_of_item(p, i, lane);
  const int r0 = p.cu_q_lens[s], q = p.cu_q_lens[s + 1] - r0, L = p.seq_lens[s];
  if (q == 0) return;
  if (q < 0 || r0 < 0 || r0 > p.T - q || q > L || L > p.max_blocks * p.bs) {
    if (threadIdx.x == 0)
      atomicOr(&g_status_fp8, (q < 0 || q > L) ? METIS_STATUS_BAD_Q_LEN
                              : (r0 < 0 || r0 > p.T - q) ? METIS_STATUS_BAD_OFFSETS : METIS_STATUS_SEQ_TOO_LONG);
    return;
  }
  const int first = L - q;                         // earlier tokens of the sequence
  const int j = i - (r0 / p.bs + 2 * s);           // page of this sequence's new rows
  if (j < 0 || ((long long)(first / p.bs) + j) * p.bs >= L) return;
  const int page = first / p.bs + j;
  const int base = page * p.bs;
  const int b = checked_block(p.block_table + (size_t)s * p.max_blocks, page, p.num_blocks, &g_status_fp8);
  if (b < 0) return;
  const int kept = max(first - base, 0);           // slots [0, kept): earlier tokens
  const int end = min(L - base, p.bs);             // slots [kept, end): new rows
  const bool live = combo < 2 * p.G;
  const int g = combo >> 1, which = combo & 1;
  uint8_t* const byte_at = (which ? p.scale[1] : p.scale[0]) + (size_t)b * p.G + g;
  const uint32_t before = live && kept > 0 ? min((uint32_t)*byte_at, 254u) : 0u;

  const int col = (lane % LPR) * VEC;
  const int slot0 = sub * 16 + lane / LPR;
  const T* src = reinterpret_cast<const T*>(which ? p.src[1] : p.src[0]) + ((size_t)(r0 + base - first) * p.G + g) * D + col;
  uint4 raw[NL];
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    const int slot = slot0 + k * RPL;
    raw[k] = live && slot >= kept && slot < end
                 ? __ldg(reinterpret_cast<const uint4*>(src + (long long)slot * p.G * D))
                 : make_uint4(0u, 0u, 0u, 0u);
  }
  auto value = [&](int k, int e) -> float {  // element e of piece k
    const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    if (sizeof(T) == 4) return __uint_as_float(w[e & 3]);
    return __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  };
  float amax = 0.f;  // fmaxf drops NaN
#pragma unroll
  for (int k = 0; k < NL; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fabsf(value(k, e)));
  const bool odd = amax == INFINITY;  // this lane holds an infinity: it counts as NaN
  if (odd) {
    amax = 0.f;
#pragma unroll
    for (int k = 0; k < NL; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float a = fabsf(value(k, e));
        if (a < INFINITY) amax = fmaxf(amax, a);
      }
  }
  amax = warp_max_xor(amax, 1);
  if (subs > 1) {
    if (lane == 0) part_max[warp] = amax;
    __syncthreads();  // also: every warp of the page has read the old byte
    for (int w = 0; w < subs; ++w) amax = fmaxf(amax, part_max[(warp & ~(subs - 1)) + w]);
  }
  if (!live) return;
  const uint32_t byte = max(byte_of_amax(amax), before);
  if (sub == 0 && lane == 0) *byte_at = (uint8_t)byte;

  uint8_t* const codes = (which ? p.cache[1] : p.cache[0]) + ((size_t)b * p.bs * p.G + g) * D;
  const float inv = scale_of_byte(254u - byte);  // 2^(127 - byte)
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    const int slot = slot0 + k * RPL;
    if (slot < kept || slot >= end) continue;
    uint32_t out[VEC / 4];
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      float y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        y[u] = value(k, e + u) * inv;
        if (odd) y[u] = fmaf(y[u], 0.f, y[u]);  // infinity -> NaN, anything else stays
      }
      out[e / 4] = pack_e4m3x4(y[0], y[1], y[2], y[3]);
    }
    uint8_t* dst = codes + (size_t)slot * p.G * D + col;
    if (VEC == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[VEC / 8]);
    else
      *reinterpret_cast<uint32_t*>(dst) = out[0];
  }

  // the scale grew: round the earlier codes at the new one
  if (kept > 0 && byte > before) {
    // 2^(before - byte); below 2^-126 every code becomes zero either way
    const float shrink = __uint_as_float((uint32_t)max(127 + (int)before - (int)byte, 1) << 23);
    constexpr int CPR = D / 16;  // 16-byte pieces per row
    const int top = min(kept, sub * 16 + 16);
    for (int slot = sub * 16 + lane / CPR; slot < top; slot += 32 / CPR) {
      uint4* at = reinterpret_cast<uint4*>(codes + (size_t)slot * p.G * D) + lane % CPR;
      const uint4 c = *at;
      uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float v[4];
        unpack_e4m3x4_f32(w[u], v);
        w[u] = pack_e4m3x4(v[0] * shrink, v[1] * shrink, v[2] * shrink, v[3] * shrink);
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// read back
// ---------------------------------------------------------------------------
struct GatherFp8Params {
  const uint8_t* cache[2];
  const uint8_t* scale[2];
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* row_offsets;
  void* out[2];
  int S, G, D, bs, max_blocks, num_blocks, cap;
  long long num_rows;
};

constexpr int kGatherThreads = 256;
constexpr int kGatherTile = 16;  // tokens per CTA: one page's worth, so one block id

template <typename T>
__device__ __forceinline__ void store16(T* dst, const uint4& c, float scale);

template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* dst, const uint4& c, float scale) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float v[4];
    unpack_e4m3x4_f32(w[u], v);
    o[2 * u] = pack_bf16x2(v[0] * scale, v[1] * scale);
    o[2 * u + 1] = pack_bf16x2(v[2] * scale, v[3] * scale);
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

template <>
__device__ __forceinline__ void store16<float>(float* dst, const uint4& c, float scale) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float v[4];
    unpack_e4m3x4_f32(w[u], v);
    reinterpret_cast<float4*>(dst)[u] = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
  }
}

// One CTA: 16 tokens of one sequence (inside one page), every head of K and V.  A thread
// takes 16-byte pieces of codes and writes 16 values.
template <typename T>
__global__ void __launch_bounds__(kGatherThreads) gather_fp8_kernel(const GatherFp8Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int s = blockIdx.y;
  const int tok0 = blockIdx.x * kGatherTile;
  int L = p.seq_lens[s];
  if (L > p.cap) {
    if (threadIdx.x == 0 && tok0 == 0) atomicOr(&g_status_fp8, METIS_STATUS_SEQ_TOO_LONG);
    L = p.cap;
  }
  if (tok0 >= L) return;
  const int n = min(L - tok0, kGatherTile);
  const long long row0 = (long long)p.row_offsets[s] + tok0;
  if (row0 < 0 || row0 + n > p.num_rows) {
    if (threadIdx.x == 0) atomicOr(&g_status_fp8, METIS_STATUS_BAD_OFFSETS);
    return;
  }
  const int page = tok0 / p.bs;
  const int b = checked_block(p.block_table + (size_t)s * p.max_blocks, page, p.num_blocks, &g_status_fp8);
  const int pieces = p.G * p.D / 16;  // per token row
  const size_t src0 = b < 0 ? 0 : ((size_t)b * p.bs + (tok0 - page * p.bs)) * p.G * p.D;
  for (int c = threadIdx.x; c < n * pieces; c += kGatherThreads) {
    const int g = (c % pieces) * 16 / p.D;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      float scale = 0.f;
      if (b >= 0) {
        v = __ldg(reinterpret_cast<const uint4*>(p.cache[w] + src0) + c);
        scale = scale_of_byte(__ldg(p.scale[w] + (size_t)b * p.G + g));
      }
      store16<T>(reinterpret_cast<T*>(p.out[w]) + (size_t)row0 * p.G * p.D + (size_t)c * 16, v, scale);
    }
  }
}

int fp8_status(uint32_t* bits, int clear) {
  unsigned int v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_status_fp8, sizeof(v));
  if (e == cudaSuccess && clear) {
    unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_status_fp8, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  *bits |= v;
  return METIS_OK;
}

}  // namespace metis

using namespace metis;

extern "C" int metis_reshape_and_cache_fp8(const void* key, const void* value, void* k_cache, void* v_cache,
                                           uint8_t* k_scale, uint8_t* v_scale, const int32_t* cu_q_lens,
                                           const int32_t* block_table, const int32_t* seq_lens, int num_seqs,
                                           int num_tokens, int num_kv_heads, int head_dim, int block_size,
                                           int max_blocks, int num_blocks, int dtype, void* stream) {
  clear_error();
  if (num_seqs < 0 || num_tokens < 0) return fail(METIS_E_SHAPE, "num_seqs and num_tokens must be >= 0");
  if (num_seqs == 0 || num_tokens == 0) return METIS_OK;
  if (!key || !value || !k_cache || !v_cache || !k_scale || !v_scale || !cu_q_lens || !block_table || !seq_lens)
    return fail(METIS_E_NULL,
                "key, value, k_cache, v_cache, k_scale, v_scale, cu_q_lens, block_table and seq_lens are required");
  if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks <= 0 || num_blocks <= 0)
    return fail(METIS_E_SHAPE, "sizes must be positive");
  if (head_dim != 64 && head_dim != 128) return fail(METIS_E_UNSUPPORTED, "head_dim must be 64 or 128");
  if (block_size != 16 && block_size != 32 && block_size != 64)
    return fail(METIS_E_UNSUPPORTED, "block_size must be 16, 32 or 64");
  if (dtype != METIS_F32 && dtype != METIS_BF16) return fail(METIS_E_UNSUPPORTED, "dtype must be METIS_F32 or METIS_BF16");
  if ((long long)max_blocks * block_size > 0x7fffffffLL || (long long)num_blocks * block_size > 0x7fffffffLL)
    return fail(METIS_E_SHAPE, "max_blocks * block_size and num_blocks * block_size must fit in int32");
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(cu_q_lens, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(METIS_E_ALIGN, "tensors must be 16-byte aligned (index arrays: 4-byte; scales: any)");
  const long long items = (long long)num_tokens / block_size + 2ll * num_seqs;
  const int subs = block_size / 16;
  const long long combos = 2ll * num_kv_heads;
  const int warps = (int)std::min<long long>(kWriteWarps, combos * subs);  // a multiple of subs
  const long long rows = (combos * subs + warps - 1) / warps;
  if (items > 0x7fffffffLL || rows > 65535) return fail(METIS_E_SHAPE, "too many pages or KV heads");
  WriteFp8Params p{};
  p.src[0] = key;
  p.src[1] = value;
  p.cache[0] = reinterpret_cast<uint8_t*>(k_cache);
  p.cache[1] = reinterpret_cast<uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.cu_q_lens = cu_q_lens;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.S = num_seqs;
  p.T = num_tokens;
  p.G = num_kv_heads;
  p.bs = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  auto kern = dtype == METIS_F32 ? (head_dim == 64 ? write_fp8_kernel<float, 64> : write_fp8_kernel<float, 128>)
                                 : (head_dim == 64 ? write_fp8_kernel<__nv_bfloat16, 64>
                                                   : write_fp8_kernel<__nv_bfloat16, 128>);
  return launch_dependent(kern, dim3((unsigned)items, (unsigned)rows), dim3(warps * 32), 0,
                          reinterpret_cast<cudaStream_t>(stream), "write_fp8_kernel launch", p);
}

extern "C" int metis_gather_cache_fp8(const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                                      const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens,
                                      const int32_t* row_offsets, void* k_out, void* v_out, int num_seqs, int num_rows,
                                      int num_kv_heads, int head_dim, int block_size, int max_blocks, int num_blocks,
                                      int out_dtype, int max_seq_len, void* stream) {
  clear_error();
  if (num_seqs < 0 || num_rows < 0) return fail(METIS_E_SHAPE, "num_seqs and num_rows must be >= 0");
  if (num_seqs == 0 || num_rows == 0) return METIS_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !row_offsets || !k_out || !v_out)
    return fail(METIS_E_NULL,
                "k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, row_offsets, k_out and v_out are required");
  if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks <= 0 || num_blocks <= 0 || max_seq_len <= 0)
    return fail(METIS_E_SHAPE, "sizes must be positive");
  if (head_dim != 64 && head_dim != 128) return fail(METIS_E_UNSUPPORTED, "head_dim must be 64 or 128");
  if (block_size != 16 && block_size != 32 && block_size != 64)
    return fail(METIS_E_UNSUPPORTED, "block_size must be 16, 32 or 64");
  if (out_dtype != METIS_F32 && out_dtype != METIS_BF16)
    return fail(METIS_E_UNSUPPORTED, "out_dtype must be METIS_F32 or METIS_BF16");
  if ((long long)max_blocks * block_size > 0x7fffffffLL || (long long)num_blocks * block_size > 0x7fffffffLL)
    return fail(METIS_E_SHAPE, "max_blocks * block_size and num_blocks * block_size must fit in int32");
  if ((long long)num_kv_heads * head_dim > (1 << 24)) return fail(METIS_E_SHAPE, "token row too large");
  if (num_seqs > 65535) return fail(METIS_E_SHAPE, "num_seqs must be <= 65535");
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(row_offsets, 4))
    return fail(METIS_E_ALIGN, "tensors must be 16-byte aligned (index arrays: 4-byte; scales: any)");
  GatherFp8Params p{};
  p.cache[0] = reinterpret_cast<const uint8_t*>(k_cache);
  p.cache[1] = reinterpret_cast<const uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.row_offsets = row_offsets;
  p.out[0] = k_out;
  p.out[1] = v_out;
  p.S = num_seqs;
  p.G = num_kv_heads;
  p.D = head_dim;
  p.bs = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.cap = (int)std::min<long long>((long long)max_blocks * block_size, (long long)max_seq_len);
  p.num_rows = num_rows;
  const dim3 grid((unsigned)((p.cap - 1) / kGatherTile + 1), (unsigned)num_seqs);
  return launch_dependent(out_dtype == METIS_BF16 ? gather_fp8_kernel<__nv_bfloat16> : gather_fp8_kernel<float>, grid,
                          dim3(kGatherThreads), 0, reinterpret_cast<cudaStream_t>(stream), "gather_fp8_kernel launch",
                          p);
}
