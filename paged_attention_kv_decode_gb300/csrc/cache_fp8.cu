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
#include <type_traits>

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
  int S, T, G, bs, bs_log, max_blocks, num_blocks;
};

constexpr int kWriteWarps = 8;

// The sequence that item i belongs to, the largest s with off(s) <= i, with its row range
// and length; every lane returns them.  A 128-way search of the warp, four probes per lane
// in flight; up to 127 sequences take one round of loads, which brings the lengths along.
struct ItemSeq {
  int s, r0, r1, L;
};

__device__ __forceinline__ ItemSeq seq_of_item(const WriteFp8Params& p, int i, int lane) {
  ItemSeq it;
  int cu[4];
  int lo = 0, n = p.S;
  if (n < 128) {
    int len[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = k * 32 + lane;
      cu[k] = at <= n ? p.cu_q_lens[at] : 0;
      len[k] = at < n ? p.seq_lens[at] : 0;
    }
    int c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = k * 32 + lane;
      c += __popc(__ballot_sync(0xffffffffu, at < n && (max(cu[k], 0) >> p.bs_log) + 2ll * at <= i));
    }
    it.s = max(c, 1) - 1;
    const int k0 = it.s >> 5, k1 = (it.s + 1) >> 5;  // uniform over the warp
    it.r0 = __shfl_sync(0xffffffffu, k0 == 0 ? cu[0] : k0 == 1 ? cu[1] : k0 == 2 ? cu[2] : cu[3], it.s & 31);
    it.r1 = __shfl_sync(0xffffffffu, k1 == 0 ? cu[0] : k1 == 1 ? cu[1] : k1 == 2 ? cu[2] : cu[3], (it.s + 1) & 31);
    it.L = __shfl_sync(0xffffffffu, k0 == 0 ? len[0] : k0 == 1 ? len[1] : k0 == 2 ? len[2] : len[3], it.s & 31);
    return it;
  }
  while (n > 1) {
    const int step = (n + 127) / 128;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = (k * 32 + lane) * step;
      cu[k] = at < n ? p.cu_q_lens[lo + at] : 0;
    }
    int c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = (k * 32 + lane) * step;
      c += __popc(__ballot_sync(0xffffffffu, at < n && (max(cu[k], 0) >> p.bs_log) + 2ll * (lo + at) <= i));
    }
    c = max(c, 1);
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
  }
  it.s = lo;
  it.r0 = p.cu_q_lens[lo];
  it.r1 = p.cu_q_lens[lo + 1];
  it.L = p.seq_lens[lo];
  return it;
}

// Magnitudes of a lane's values: they order like their bits, for bf16 two to a word.
template <typename T>
struct WriteVals;

template <>
struct WriteVals<__nv_bfloat16> {
  __device__ static __forceinline__ uint32_t larger(uint32_t m, const uint4& v) {
    m = max_u16x2(max_u16x2(m, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
    return max_u16x2(max_u16x2(m, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
  }
  __device__ static __forceinline__ uint32_t bits(uint32_t m) { return max(m & 0xffffu, m >> 16) << 16; }
  static constexpr int N = 8;
  __device__ static __forceinline__ void get(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

template <>
struct WriteVals<float> {
  __device__ static __forceinline__ uint32_t larger(uint32_t m, const uint4& v) {
    return max(max(max(m, v.x & 0x7fffffffu), v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
  }
  __device__ static __forceinline__ uint32_t bits(uint32_t m) { return m; }
  static constexpr int N = 4;
  __device__ static __forceinline__ void get(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
};

// Four values times the pair inv2 as codes
__device__ __forceinline__ uint32_t quantize4(const float* x, uint64_t inv2) {
  float y0, y1, y2, y3;
  f2_unpack(f2_mul(f2_pack(x[0], x[1]), inv2), y0, y1);
  f2_unpack(f2_mul(f2_pack(x[2], x[3]), inv2), y2, y3);
  return pack_e4m3x4(y0, y1, y2, y3);
}

// One warp: 16 slots of a page x one head of K or V.  Lanes hold 16-byte pieces of the
// new rows (8 bf16 or 4 fp32), several rows per load, all loads issued before the first
// use; the rows stay in registers between the maximum and the rounding, so each input is
// read once.  Pages of 32 or 64 slots take 2 or 4 warps that share their maximum.
// The grid is a few waves of short CTAs, so CTAs per SM (registers) decide: 8,240 rows of
// 8 x 128 bf16 take 11.0 us with five or four on an SM, 11.3 us with three, 11.4 us with six;
// fp32 rows of 8 x 128, twice the registers, 15.4 us with three, 16.0 us with two, 23.9 us
// with five.  Eight slots per warp instead of 16 were 8 % slower.
template <typename T, int D>
__global__ void __launch_bounds__(kWriteWarps * 32, sizeof(T) * D == 512 ? 3 : 5) write_fp8_kernel(const WriteFp8Params p) {
  constexpr int VEC = 16 / (int)sizeof(T);  // elements per lane and load
  constexpr int LPR = D / VEC;              // lanes per row
  constexpr int RPL = 32 / LPR;             // rows per load
  constexpr int NL = 16 / RPL;              // loads for 16 slots
  __shared__ float part_max[kWriteWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int subs = p.bs >> 4;                                                       // warps per page, head and cache
  const int combo = (int)((blockIdx.y * (blockDim.x >> 5) + warp) >> (p.bs_log - 4));  // head * 2 + cache
  const int sub = warp & (subs - 1);                                                // (a block holds whole combos)

  const int i = blockIdx.x;
  const ItemSeq it = seq_of_item(p, i, lane);
  const int s = it.s, r0 = it.r0, q = it.r1 - r0, L = it.L;
  if (q == 0) return;
  if (q < 0 || r0 < 0 || r0 > p.T - q || q > L || L > p.max_blocks * p.bs) {
    if (threadIdx.x == 0)
      atomicOr(&g_status_fp8, (q < 0 || q > L) ? METIS_STATUS_BAD_Q_LEN
                              : (r0 < 0 || r0 > p.T - q) ? METIS_STATUS_BAD_OFFSETS : METIS_STATUS_SEQ_TOO_LONG);
    return;
  }
  const int first = L - q;                         // earlier tokens of the sequence
  const int page0 = first >> p.bs_log;
  const int j = i - ((r0 >> p.bs_log) + 2 * s);    // page of this sequence's new rows
  if (j < 0 || ((long long)page0 + j) * p.bs >= L) return;
  const int page = page0 + j;
  const int base = page * p.bs;
  const int kept = max(first - base, 0);           // slots [0, kept): earlier tokens
  const int end = min(L - base, p.bs);             // slots [kept, end): new rows
  const bool live = combo < 2 * p.G;
  const int g = combo >> 1, which = combo & 1;

  // the rows are on their way before the page's block id is known
  const int col = (lane % LPR) * VEC;
  const int slot0 = sub * 16 + lane / LPR;
  const size_t row_len = (size_t)p.G * D;
  const T* src = reinterpret_cast<const T*>(which ? p.src[1] : p.src[0]) +
                 ((long long)(r0 + base - first + slot0) * p.G + g) * D + col;
  uint4 raw[NL];
  const unsigned rows = live ? (unsigned)max(end - kept, 0) : 0u;
#pragma unroll
  for (int k = 0; k < NL; ++k, src += RPL * row_len)
    raw[k] = (unsigned)(slot0 + k * RPL - kept) < rows ? ld_codes(reinterpret_cast<const uint4*>(src))
                                                       : make_uint4(0u, 0u, 0u, 0u);
  const int b = checked_block(p.block_table + (size_t)s * p.max_blocks, page, p.num_blocks, &g_status_fp8);
  if (b < 0) return;
  uint8_t* const byte_at = (which ? p.scale[1] : p.scale[0]) + (size_t)b * p.G + g;
  uint32_t before = 0;  // the scale byte of the earlier tokens, if any
  if (live && kept > 0) before = ld_byte(byte_at);
  // the largest finite magnitude; infinities and NaN (rare) are stored as NaN and do not count
  using Vals = WriteVals<T>;
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < NL; ++k) top = Vals::larger(top, raw[k]);
  float amax = __uint_as_float(Vals::bits(top));
  const bool odd = __any_sync(0xffffffffu, !(amax < INFINITY));
  if (odd) {
    amax = 0.f;
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      float x[VEC];
      Vals::get(raw[k], x);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (fabsf(x[e]) < INFINITY) amax = fmaxf(amax, fabsf(x[e]));
    }
  }
  amax = warp_max_xor(amax, 1);
  if (subs > 1) {
    if (lane == 0) part_max[warp] = amax;
    __syncthreads();  // also: every warp of the page has read the old byte
    for (int w = 0; w < subs; ++w) amax = fmaxf(amax, part_max[(warp & ~(subs - 1)) + w]);
  }
  if (!live) return;
  before = min(before, 254u);
  const uint32_t byte = max(byte_of_amax(amax), before);
  if (sub == 0 && lane == 0) *byte_at = (uint8_t)byte;

  uint8_t* const codes = (which ? p.cache[1] : p.cache[0]) + ((size_t)b * p.bs * p.G + g) * D;
  const float inv = scale_of_byte(254u - byte);  // 2^(127 - byte)
  const uint64_t inv2 = f2_pack(inv, inv);
  uint8_t* dst = codes + slot0 * row_len + col;
  auto put = [&](auto with_odd) {
#pragma unroll
    for (int k = 0; k < NL; ++k, dst += RPL * row_len) {
      float x[VEC];
      Vals::get(raw[k], x);
      if (decltype(with_odd)::value) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = fmaf(x[e], 0.f, x[e]);  // infinity -> NaN, anything else stays
      }
      if ((unsigned)(slot0 + k * RPL - kept) < (unsigned)(end - kept)) {
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(dst) = make_uint2(quantize4(x, inv2), quantize4(x + 4, inv2));
        else
          *reinterpret_cast<uint32_t*>(dst) = quantize4(x, inv2);
      }
    }
  };
  if (!odd)
    put(std::false_type{});
  else
    put(std::true_type{});

  // the scale grew: round the earlier codes at the new one
  if (kept > 0 && byte > before) {
    // 2^(before - byte); below 2^-126 every code becomes zero either way
    const float shrink = __uint_as_float((uint32_t)max(127 + (int)before - (int)byte, 1) << 23);
    constexpr int CPR = D / 16;  // 16-byte pieces per row
    const int top = min(kept, sub * 16 + 16);
    for (int slot = sub * 16 + lane / CPR; slot < top; slot += 32 / CPR) {
      uint4* at = reinterpret_cast<uint4*>(codes + (size_t)slot * p.G * D) + lane % CPR;
      const uint4 c = ld_codes(at);
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
  int S, G, D, bs, bs_log, max_blocks, num_blocks, cap;
  int tile;  // tokens per CTA
  long long num_rows;
};

constexpr int kGatherThreads = 256;
constexpr int kGatherBatch = 4;        // rows of K and of V that a thread has in flight
constexpr int kGatherTileBatches = 2;  // such batches per CTA (one or two are alike, four leave small batches few CTAs)

// One store of values: eight codes to bf16, four to fp32 (16 bytes either way)
template <typename T>
struct GatherVec;

template <>
struct GatherVec<__nv_bfloat16> {
  using Codes = uint2;
  static constexpr int N = 8;
  __device__ static __forceinline__ Codes zero() { return make_uint2(0u, 0u); }
  __device__ static __forceinline__ uint4 values(const Codes& c, float scale) {
    float a[4], b[4];
    unpack_e4m3x4_f32(c.x, a);
    unpack_e4m3x4_f32(c.y, b);
    return make_uint4(pack_bf16x2(a[0] * scale, a[1] * scale), pack_bf16x2(a[2] * scale, a[3] * scale),
                      pack_bf16x2(b[0] * scale, b[1] * scale), pack_bf16x2(b[2] * scale, b[3] * scale));
  }
};

template <>
struct GatherVec<float> {
  using Codes = uint32_t;
  static constexpr int N = 4;
  __device__ static __forceinline__ Codes zero() { return 0u; }
  __device__ static __forceinline__ uint4 values(const Codes& c, float scale) {
    float a[4];
    unpack_e4m3x4_f32(c, a);
    return make_uint4(__float_as_uint(a[0] * scale), __float_as_uint(a[1] * scale), __float_as_uint(a[2] * scale),
                      __float_as_uint(a[3] * scale));
  }
};

// One CTA: `tile` tokens of one sequence, every head of K and V.  A thread keeps one column
// of 16 bytes of output and walks the rows, kGatherBatch of K and of V in flight, so that
// loads and stores of a warp are whole runs of a row.  HBM-bound: 64 sequences of 512..4096
// tokens of 8 x 128 to bf16 in 137 us (6,650 GB/s, the measured copy rate), to fp32 in 233 us;
// with 16 codes per thread and two 16-byte stores side by side the bf16 case took 151 us.
template <typename T>
__global__ void __launch_bounds__(kGatherThreads) gather_fp8_kernel(const GatherFp8Params p) {
  using Vec = GatherVec<T>;
  using Codes = typename Vec::Codes;
  pdl_wait();
  pdl_launch_dependents();
  const int s = blockIdx.y;
  const long long tile0 = (long long)blockIdx.x * p.tile;
  int L = p.seq_lens[s];
  if (L > p.cap) {
    if (threadIdx.x == 0 && tile0 == 0) atomicOr(&g_status_fp8, METIS_STATUS_SEQ_TOO_LONG);
    L = p.cap;
  }
  if (tile0 >= L) return;
  const int tok0 = (int)tile0;
  const int n = min(L - tok0, p.tile);
  const long long first_row = (long long)p.row_offsets[s] + tok0;
  const int32_t* bt_row = p.block_table + (size_t)s * p.max_blocks;
  const int cols = p.G * p.D / Vec::N;                  // stores per row
  const int lanes = min(cols, kGatherThreads);          // threads across a row
  const int rows = kGatherThreads / lanes;              // rows at a time
  const int ty = threadIdx.x / lanes;
  if (ty >= rows) return;
  for (int col = threadIdx.x - ty * lanes; col < cols; col += lanes) {
    const int g = col * Vec::N / p.D;
    for (int r0 = ty; r0 < n; r0 += rows * kGatherBatch) {
      Codes c[2][kGatherBatch];
      uint32_t byte[2][kGatherBatch];
#pragma unroll
      for (int u = 0; u < kGatherBatch; ++u) {
        const int r = r0 + u * rows;
        c[0][u] = c[1][u] = Vec::zero();                // a page with a bad id reads as zeros
        byte[0][u] = byte[1][u] = 127;
        if (r < n) {
          const int tok = tok0 + r, page = tok >> p.bs_log;
          const int b = checked_block(bt_row, page, p.num_blocks, &g_status_fp8);
          if (b >= 0) {
            const size_t row = ((size_t)b << p.bs_log) + (tok & (p.bs - 1));
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              c[w][u] = ld_codes(reinterpret_cast<const Codes*>(p.cache[w] + row * p.G * p.D) + col);
              byte[w][u] = ld_byte(p.scale[w] + (size_t)b * p.G + g);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kGatherBatch; ++u) {
        const int r = r0 + u * rows;
        if (r >= n) break;
        const long long row = first_row + r;
        if (row < 0 || row >= p.num_rows) {             // rows outside the outputs are not written
          if (col == 0) atomicOr(&g_status_fp8, METIS_STATUS_BAD_OFFSETS);
          continue;
        }
#pragma unroll
        for (int w = 0; w < 2; ++w)
          reinterpret_cast<uint4*>(p.out[w])[(size_t)row * cols + col] = Vec::values(c[w][u], scale_of_byte(byte[w][u]));
      }
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
  p.bs_log = block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
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
  p.bs_log = block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
  // two batches per thread: fewer tokens for wide rows, at least 16
  const int cols = num_kv_heads * head_dim / (out_dtype == METIS_BF16 ? 8 : 4);
  p.tile = std::max(16, kGatherTileBatches * kGatherBatch * (kGatherThreads / std::min(cols, kGatherThreads)));
  const dim3 grid((unsigned)((p.cap - 1) / p.tile + 1), (unsigned)num_seqs);
  return launch_dependent(out_dtype == METIS_BF16 ? gather_fp8_kernel<__nv_bfloat16> : gather_fp8_kernel<float>, grid,
                          dim3(kGatherThreads), 0, reinterpret_cast<cudaStream_t>(stream), "gather_fp8_kernel launch",
                          p);
}
