// Decode attention with a sliding window: the query of a sequence of L cached tokens sees the last
// `window` of them (its own among them) and the first `sinks`, which stay visible however far the
// window has moved on (attention spends weight on a sequence's first tokens whatever they hold; a
// window that drops them loses it).  The paged-attention kernel of the vllm-metal article, section 3,
// over fewer tokens: z_t = scale q . k_t for t >= L - window or t < sinks, softmax, weighted sum of v.
//
// Bound by HBM, as the decode of all tokens is (decode.cu), but a sequence's bytes no longer grow with
// its length: min(L, window + sinks) tokens.  So the items are about equal and, with a short window, small:
// 16-token units hold the visible tokens (decode_items.cuh), those in between are never visited -- their
// pages may have been given back -- and tokens of a unit's other part are masked as those behind the
// sequence's end are.  Where (sequence, KV head) items leave SMs idle, an item is shared by the CTAs of a
// cluster, whose results join in shared memory: no workspace, one launch.  Where there are many items of few
// tokens, warps walk them one after another with their loads running on.
//
// Measured (8 KV heads x 128, bf16): 64 sequences with windows of 4,096 (1.02 GB) 152 us, 6.7 TB/s; 8 with
// windows of 1,024 (34 MB) 11.3 us, most of it a CTA's start: lengths, ids, first loads, join; 2,048 with windows
// of 64 (537 MB) 120 us.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "../../include/metis_attn.h"
#include "decode_items.cuh"
#include "decode_stream.cuh"

namespace metis {

__device__ unsigned int g_status_window = 0;

struct WindowParams {
  DecodeParams d;
  int window, sinks;
};

// parts: CTAs that share an item.  One: a grid of items, longest first, each CTA writing its rows.
template <int D, bool JOIN>
__global__ void __launch_bounds__(kBf16Warps * 32) decode_window_bf16_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                             const __grid_constant__ CUtensorMap tmV,
                                                                             const WindowParams wp) {
  constexpr int NW = kBf16Warps, STAGES = kBf16Stages, STAGE_BYTES = Bf16DecodeShape<D>::kStageBytes;
  static_assert(NW * (64 + D * 32) <= NW * STAGES * STAGE_BYTES, "combine area must fit in the ring");
  const DecodeParams& p = wp.d;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // 1024-aligned for the swizzle
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + NW * STAGES * STAGE_BYTES);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < NW * STAGES; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  pdl_wait();  // inputs are read after the previous grid in the stream has completed
  pdl_launch_dependents();
  if constexpr (JOIN) {
    const int g = blockIdx.x, part = blockIdx.y, s = blockIdx.z;
    int L = p.seq_lens[s];
    if (L > p.cap) {
      if (threadIdx.x == 0 && part == 0) atomicOr(&g_status_window, METIS_STATUS_SEQ_TOO_LONG);
      L = p.cap;
    }
    __syncthreads();  // the barriers are initialised
    decode_joined_item<D, NW, STAGES>(tmK, tmV, p, smem, bars, g, s, part, gridDim.y, L > 0,
                                      window_span(L, wp.window, wp.sinks), &g_status_window);
  } else {
    __shared__ int rank_lens[kMaxRankSeqs];
    __shared__ int rank_found;
    const int g = blockIdx.x;
    const int s = p.S <= kMaxRankSeqs ? seq_of_rank(p, blockIdx.y, rank_lens, &rank_found) : (int)blockIdx.y;
    int t0, t1;
    if (!decode_range<__nv_bfloat16>(p, 0, g, s, s, t0, t1, threadIdx.x, blockDim.x, &g_status_window)) return;
    __syncthreads();  // the barriers are initialised
    int kb = 0;
    decode_bf16_item<D, NW, STAGES>(tmK, tmV, p, smem, bars, g, s, s, window_span(t1, wp.window, wp.sinks),
                                    threadIdx.x >> 5, threadIdx.x & 31, kb, &g_status_window, [] { __syncthreads(); },
                                    [&](const float* cm, const float* cl, const float* co) {
                                      combine_and_store<__nv_bfloat16, NW>(p, cm, cl, co, 0, g, s, s, threadIdx.x);
                                    });
  }
}

// Many items of few tokens: a warp walks items (decode_stream.cuh), every `warps`-th of the grid's.
template <int D>
__global__ void __launch_bounds__(kStreamWarps * 32, 1) decode_window_stream_kernel(
    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const WindowParams wp) {
  constexpr int STAGES = stream_stages<D>(), STAGE_BYTES = Bf16DecodeShape<D>::kStageBytes;
  constexpr int KS = Bf16DecodeShape<D>::kSteps;
  const DecodeParams& p = wp.d;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // 1024-aligned for the swizzle
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStreamWarps * STAGES * STAGE_BYTES);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < kStreamWarps * STAGES; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  pdl_wait();  // inputs are read after the previous grid in the stream has completed
  pdl_launch_dependents();
  __syncthreads();  // the barriers are initialised
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long items = (long long)p.S * p.G, warps = (long long)gridDim.x * kStreamWarps;
  long long item = (long long)blockIdx.x * kStreamWarps + warp;  // KV heads side by side, as their rows are
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out);
  auto next = [&](StreamItem& it) -> bool {
    for (; item < items; item += warps) {
      it.s = (int)(item / p.G);
      it.g = (int)(item - (long long)it.s * p.G);
      int L = p.seq_lens[it.s];
      if (L > p.cap) {
        if (lane == 0) atomicOr(&g_status_window, METIS_STATUS_SEQ_TOO_LONG);
        L = p.cap;
      }
      if (L > 0) {
        it.span = window_span(L, wp.window, wp.sinks);
        item += warps;
        return true;
      }
      const size_t row = (size_t)it.s * p.H + it.g * p.r;  // an empty sequence
      for (int i = lane; i < p.r * D; i += 32) out[row * D + i] = __nv_bfloat16(0.0f);
      if (p.lse_out && lane < p.r) p.lse_out[row + lane] = -INFINITY;
    }
    return false;
  };
  auto store = [&](const StreamItem& it, const DecodeWarp<D>& state) {
    const int q4 = lane & 3, rA = lane >> 2, h = 2 * q4;
    const float l0 = warp_sum_xor(state.l0, 4), l1 = warp_sum_xor(state.l1, 4);
    const float i0 = 1.f / l0, i1 = 1.f / l1;
    const size_t row = (size_t)it.s * p.H + it.g * p.r + h;
    // lanes rA and rA ^ 1 hold neighbouring dims: the even one writes both for head h, the odd one for h + 1
    const bool odd = rA & 1;
    __nv_bfloat16* to = out + (row + odd) * D + (rA & ~1);
    const bool live = h + odd < p.r;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float a = state.o[mt][2 * half] * i0, b = state.o[mt][2 * half + 1] * i1;
        const float other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 4);  // (lane ^ 4: rA ^ 1)
        const uint32_t v = odd ? pack_bf16x2(other, b) : pack_bf16x2(a, other);
        if (live) *reinterpret_cast<uint32_t*>(to + mt * 16 + half * 8) = v;
      }
    if (p.lse_out && rA == 0) {
      if (h < p.r) p.lse_out[row] = (state.m0 + log2f(l0)) * kLn2;
      if (h + 1 < p.r) p.lse_out[row + 1] = (state.m1 + log2f(l1)) * kLn2;
    }
  };
  decode_stream<D>(tmK, tmV, p, smem + warp * STAGES * STAGE_BYTES, bars + warp * STAGES, lane, &g_status_window, next,
                   store);
}

template <int D>
__global__ void __launch_bounds__(kF32Warps * 32) decode_window_f32_kernel(const float* k_cache, const float* v_cache,
                                                                           const WindowParams wp) {
  const DecodeParams& p = wp.d;
  pdl_launch_dependents();
  pdl_wait();  // inputs are read after the previous grid in the stream has completed
  const int g = blockIdx.x, s = blockIdx.y;
  int t0, t1;
  if (!decode_range<float>(p, 0, g, s, s, t0, t1, threadIdx.x, blockDim.x, &g_status_window)) return;
  decode_f32_item<D>(k_cache, v_cache, p, 0, g, s, window_span(t1, wp.window, wp.sinks), &g_status_window);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int window_status(uint32_t* bits, int clear) {
  unsigned int v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_status_window, sizeof(v));
  if (e == cudaSuccess && clear) {
    unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_status_window, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  *bits |= v;
  return METIS_OK;
}

template <int D, bool JOIN>
static int launch_window(const WindowParams& wp, const void* k_cache, const void* v_cache, int parts, cudaStream_t st) {
  CUtensorMap tmK, tmV;
  int rc = encode_kv_maps<D>(wp.d, k_cache, v_cache, &tmK, &tmV);
  if (rc) return rc;
  constexpr int smem = bf16_decode_smem_bytes<D, kBf16Warps, kBf16Stages>();
  static int done = 0;
  auto kern = decode_window_bf16_kernel<D, JOIN>;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem, &done);
  if (rc) return rc;
  const unsigned G = (unsigned)wp.d.G, S = (unsigned)wp.d.S;
  if (JOIN)
    return launch_dependent_cluster(kern, dim3(G, (unsigned)parts, S), dim3(1, (unsigned)parts, 1),
                                    dim3(kBf16Warps * 32), (size_t)smem, st, "decode_window_bf16_kernel launch", tmK,
                                    tmV, wp);
  return launch_dependent(kern, dim3(G, S), dim3(kBf16Warps * 32), (size_t)smem, st, "decode_window_bf16_kernel launch",
                          tmK, tmV, wp);
}

template <int D>
static int launch_window_stream(const WindowParams& wp, const void* k_cache, const void* v_cache, int sms,
                                cudaStream_t st) {
  CUtensorMap tmK, tmV;
  int rc = encode_kv_maps<D>(wp.d, k_cache, v_cache, &tmK, &tmV);
  if (rc) return rc;
  constexpr int smem = stream_smem_bytes<D>();
  static int done = 0;
  auto kern = decode_window_stream_kernel<D>;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem, &done);
  if (rc) return rc;
  return launch_dependent(kern, dim3((unsigned)sms), dim3(kStreamWarps * 32), (size_t)smem, st,
                          "decode_window_stream_kernel launch", tmK, tmV, wp);
}

// Items of at most this many tokens, at least kStreamItems for each of the stream's warps, are walked by those.
// (Walked and a CTA per item, us: 512 sequences of 8 KV heads with windows of 128 54 and 81, 2,048 with 64 120 and
// 263, 304 with 500 99.5 and 107.7, 512 with 500 168.5 and 170.4: the longer an item, the less its start weighs.)
constexpr int kStreamTokens = 512;
constexpr int kStreamItems = 2;

}  // namespace metis

using namespace metis;

extern "C" int metis_paged_attn_decode_window(const void* q, const void* k_cache, const void* v_cache,
                                              const int32_t* block_table, const int32_t* seq_lens, void* out,
                                              float* lse_out, int num_seqs, int num_heads, int num_kv_heads,
                                              int head_dim, int block_size, int max_blocks, int num_blocks, int dtype,
                                              float scale, int window, int sinks, int max_seq_len, void* stream) {
  clear_error();
  if (num_seqs < 0) return fail(METIS_E_SHAPE, "num_seqs < 0");
  if (num_seqs == 0) return METIS_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return fail(METIS_E_NULL, "q, k_cache, v_cache, block_table, seq_lens and out are required");
  const int rc = check_decode_sizes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks,
                                    max_seq_len, scale);
  if (rc) return rc;
  if (dtype != METIS_F32 && dtype != METIS_BF16) return fail(METIS_E_UNSUPPORTED, "dtype must be METIS_F32 or METIS_BF16");
  if (window <= 0 || sinks < 0) return fail(METIS_E_SHAPE, "window must be positive and sinks >= 0");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse_out, 4))
    return fail(METIS_E_ALIGN, "tensors must be 16-byte aligned (block_table, seq_lens, lse_out: 4-byte)");
  WindowParams wp{};
  wp.window = window;
  wp.sinks = sinks;
  DecodeParams& p = wp.d;
  p.q = q;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.lse_out = lse_out;
  p.S = num_seqs;
  p.H = num_heads;
  p.G = num_kv_heads;
  p.D = head_dim;
  p.bs = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.r = num_heads / num_kv_heads;
  p.scale_log2 = scale * kLog2e;
  p.max_parts = 1;
  p.cap = effective_max_len(max_seq_len, max_blocks, block_size);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == METIS_F32) {
    const float* kc = reinterpret_cast<const float*>(k_cache);
    const float* vc = reinterpret_cast<const float*>(v_cache);
    const dim3 grid((unsigned)num_kv_heads, (unsigned)num_seqs), block(kF32Warps * 32);
    return head_dim == 64 ? launch_dependent(decode_window_f32_kernel<64>, grid, block, 0, st,
                                             "decode_window_f32_kernel launch", kc, vc, wp)
                          : launch_dependent(decode_window_f32_kernel<128>, grid, block, 0, st,
                                             "decode_window_f32_kernel launch", kc, vc, wp);
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "querying the SM count: %s", cudaGetErrorString(e));
  const int seen = (int)std::min<long long>((long long)window + sinks, p.cap);
  const long long items = (long long)num_kv_heads * num_seqs;
  if (seen <= kStreamTokens && items >= (long long)kStreamItems * kStreamWarps * sms)
    return head_dim == 64 ? launch_window_stream<64>(wp, k_cache, v_cache, sms, st)
                          : launch_window_stream<128>(wp, k_cache, v_cache, sms, st);
  const int parts = item_parts(items, seen, sms);
  auto launch = [&](auto dim, auto join) {
    return launch_window<decltype(dim)::value, decltype(join)::value>(wp, k_cache, v_cache, parts, st);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (parts > 1) return head_dim == 64 ? launch(D64{}, std::true_type{}) : launch(D128{}, std::true_type{});
  return head_dim == 64 ? launch(D64{}, std::false_type{}) : launch(D128{}, std::false_type{});
}
