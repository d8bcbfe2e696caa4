// Decode attention of a batch whose sequences share their first tokens in groups (a system prompt, a
// document that many requests ask about): the paged-attention kernel of the vllm-metal article,
// section 3, over the pages that prefix caching lets sequences share (vllm-metis 0.1.0 page, "Caches").
//
// Softmax attention over a sequence's tokens is the log-sum-exp join of its attention over the shared
// ones and over its own.  Decoding each sequence by itself reads the shared pages once per sequence; here
//
//   1 the members' queries of a group become the rows of query tiles, and the chunk kernel (prefill.cu,
//     SHARED) runs them over the prefix on the tensor cores: its K and V are read once per 256 rows.  All
//     tiles of all groups are cut into equal shares, one per SM, so a unit may be several CTAs' parts.
//   2 one CTA (or a cluster) per sequence and KV head decodes the sequence's own tokens (decode_items.cuh)
//     and joins the prefix's parts in its epilogue.  It is a programmatic dependent of 1 that waits for it
//     only there: its CTAs start on SMs that 1 has left, and its K/V stream under 1's tail.
//
// Bound by HBM for the own tokens, by the chunk kernel's tile loop (or HBM, few members) for the prefix.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "../../include/metis_attn.h"
#include "decode_items.cuh"

namespace metis {

__device__ unsigned int g_status_shared = 0;

constexpr int kSharedRows = 128;  // rows of a query tile

struct SharedParams {
  DecodeParams d;
  const int32_t* cu_group_seqs;
  const int32_t* prefix_lens;
  const SharedPlan* plan;
  const float* part_lse;
  const float* part_out;
  int num_groups, Tq;
};

// The group of sequence s, the last that begins at or before it (-1: none), by a whole warp.
__device__ __forceinline__ int group_of(const SharedParams& sp, int s, int lane) {
  int lo = 0, n = sp.num_groups;
  while (n > 0) {
    const int step = (n + 31) / 32, at = lane * step;
    const int before = __popc(__ballot_sync(0xffffffffu, at < n && sp.cu_group_seqs[lo + min(at, n - 1)] <= s));
    if (before == 0) return -1;
    lo += (before - 1) * step;
    n = min(step, n - (before - 1) * step);
    if (n == 1) return lo;
  }
  return -1;
}

// The prefix's parts of the rows of one (sequence, KV head): row h * Tq + qi of query tile `tile` of the
// parts first .. first + count - 1.  grp < 0: the sequence shares nothing.
struct PrefixParts {
  const SharedParams& sp;
  int grp, s, g;
  const float *lse, *out;
  int first, count, tile, qi, Tq, D;

  __device__ __forceinline__ PrefixParts(const SharedParams& sp_, int grp_, int s_, int g_)
      : sp(sp_), grp(grp_), s(s_), g(g_), lse(sp_.part_lse), out(sp_.part_out), first(0), count(0), tile(0), qi(0),
        Tq(sp_.Tq), D(sp_.d.D) {}

  // Waits for the kernel over the prefixes (every CTA does, so that this grid completes after it).
  __device__ __forceinline__ void prepare() {
    pdl_wait();
    if (grp < 0) return;
    const int4 v = __ldcg(sp.plan->group + grp);  // tiles before, tiles of a unit, units before, units per KV head
    const int2 all = __ldcg(&sp.plan->total);
    if (v.y <= 0 || all.x <= 0) return;
    const int member = s - sp.cu_group_seqs[grp], pair = member / (2 * Tq), in = member - pair * 2 * Tq;
    const int unit = g * v.w + pair;
    // the CTAs whose shares hold the unit's first and last tile
    const long long x0 = v.x + (long long)unit * v.y, x1 = x0 + v.y - 1;
    const int c0 = (int)(((x0 + 1) * all.y - 1) / all.x), c1 = (int)(((x1 + 1) * all.y - 1) / all.x);
    first = v.z + unit + c0;
    count = c1 - c0 + 1;
    tile = in / Tq;
    qi = in - tile * Tq;
  }

  __device__ __forceinline__ void add(JoinedRow& row, int h, int d) const {
    constexpr int kBatch = 8;  // loads in flight
    for (int k = 0; k < count; k += kBatch) {
      float x[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        x[j] = -INFINITY;
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k + j < count) {
          const size_t at = ((size_t)(first + k + j) * 2 + tile) * kSharedRows + h * Tq + qi;
          x[j] = __ldcg(lse + at);
          v[j] = __ldcg(reinterpret_cast<const float4*>(out + at * D + d));
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) row.add(x[j], v[j]);
    }
  }
};

template <int D, int NW>
__global__ void __launch_bounds__(NW * 32) decode_shared_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                        const __grid_constant__ CUtensorMap tmV,
                                                                        const SharedParams sp) {
  constexpr int STAGES = kBf16Stages, STAGE_BYTES = Bf16DecodeShape<D>::kStageBytes;
  const DecodeParams& p = sp.d;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // 1024-aligned for the swizzle
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + NW * STAGES * STAGE_BYTES);
  // The kernel over the prefixes, in front of this one, let it start once all its CTAs had waited for
  // the kernels before: their outputs are there (lines that they left in this SM's L1 are dropped).
  __threadfence();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < NW * STAGES; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  __shared__ int rank_lens[kMaxRankSeqs];
  __shared__ int rank_found;
  const int g = blockIdx.x, part = blockIdx.y, parts = gridDim.y;
  const int s = p.S <= kMaxRankSeqs && parts == 1 ? seq_of_rank(p, blockIdx.z, rank_lens, &rank_found) : (int)blockIdx.z;
  int L = p.seq_lens[s];
  if (L > p.cap) {
    if (threadIdx.x == 0) atomicOr(&g_status_shared, METIS_STATUS_SEQ_TOO_LONG);
    L = p.cap;
  }
  L = max(L, 0);
  int grp = group_of(sp, s, threadIdx.x & 31), shared = 0;
  if (grp >= 0) {
    const int a = sp.cu_group_seqs[grp], b = sp.cu_group_seqs[grp + 1], tokens = sp.prefix_lens[grp];
    if (a >= 0 && a <= s && s < b && b <= p.S && tokens > 0 && L >= tokens) shared = tokens;
  }
  if (shared == 0) grp = -1;  // every token is the sequence's own
  __syncthreads();            // the barriers are initialised
  decode_joined_item<D, NW, STAGES>(tmK, tmV, p, smem, bars, g, s, part, parts, L > shared,
                                    window_span(L, L - shared, 0), &g_status_shared, PrefixParts(sp, grp, s, g));
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int shared_status(uint32_t* bits, int clear) {
  unsigned int v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_status_shared, sizeof(v));
  if (e == cudaSuccess && clear) {
    unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_status_shared, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  *bits |= v;
  return METIS_OK;
}

// Units of a call at most: a pair of query tiles for each 2 Tq members of a group, for each KV head
static long long shared_units(int num_seqs, int num_groups, int r, int G) {
  const int members = 2 * (kSharedRows / r);
  return ((long long)(num_seqs + members - 1) / members + std::min(num_groups, num_seqs)) * G;
}

// Workspace: the plan, the parts' lse, their rows
static size_t shared_plan_bytes(int num_groups) { return align_up(sizeof(SharedPlan) + (size_t)num_groups * sizeof(int4), 256); }
static size_t shared_lse_bytes(size_t parts) { return parts * 2 * kSharedRows * sizeof(float); }

static int current_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(METIS_E_CUDA, "querying the SM count: %s", cudaGetErrorString(e));
  }
  *sms = std::max(*sms, 1);
  return METIS_OK;
}

static size_t shared_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int num_groups, int sms) {
  const size_t parts = (size_t)shared_units(num_seqs, num_groups, num_heads / num_kv_heads, num_kv_heads) + sms;
  return shared_plan_bytes(num_groups) + shared_lse_bytes(parts) * (1 + (size_t)head_dim);
}

template <int D, int NW>
static int launch_shared(const SharedParams& sp, const SharedArgs& a, int parts, cudaStream_t st) {
  CUtensorMap tmK, tmV;
  int rc = encode_kv_maps<D>(sp.d, a.k_cache, a.v_cache, &tmK, &tmV);
  if (rc) return rc;
  constexpr int smem = bf16_decode_smem_bytes<D, NW, kBf16Stages>();
  static int done = 0;
  auto kern = decode_shared_kernel<D, NW>;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem, &done);
  if (rc) return rc;
  return launch_dependent_cluster(kern, dim3((unsigned)a.G, (unsigned)parts, (unsigned)a.S),
                                  dim3(1, (unsigned)parts, 1), dim3(NW * 32), (size_t)smem, st,
                                  "decode_shared_kernel launch", tmK, tmV, sp);
}

}  // namespace metis

using namespace metis;

extern "C" size_t metis_shared_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                               int num_groups) {
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_groups < 0 ||
      num_heads % num_kv_heads || num_heads / num_kv_heads > kSharedRows)
    return 0;
  int sms = 0;
  if (current_sms(&sms)) return 0;
  return shared_bytes(num_seqs, num_heads, num_kv_heads, head_dim, num_groups, sms);
}

extern "C" int metis_paged_attn_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                                              const int32_t* block_table, const int32_t* seq_lens,
                                              const int32_t* cu_group_seqs, const int32_t* prefix_lens, void* out,
                                              float* lse_out, int num_seqs, int num_groups, int num_heads,
                                              int num_kv_heads, int head_dim, int block_size, int max_blocks,
                                              int num_blocks, int dtype, float scale, int max_seq_len,
                                              void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  if (num_seqs < 0 || num_groups < 0) return fail(METIS_E_SHAPE, "num_seqs and num_groups must be >= 0");
  if (num_seqs == 0) return METIS_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || (num_groups > 0 && (!cu_group_seqs || !prefix_lens)))
    return fail(METIS_E_NULL, "q, k_cache, v_cache, block_table, seq_lens, cu_group_seqs, prefix_lens and out are required");
  int rc = check_decode_sizes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks,
                              max_seq_len, scale);
  if (rc) return rc;
  if (dtype != METIS_BF16) return fail(METIS_E_UNSUPPORTED, "shared prefixes are built for bf16");
  const int r = num_heads / num_kv_heads;
  if (r & (r - 1)) return fail(METIS_E_UNSUPPORTED, "num_heads / num_kv_heads must be 1, 2, 4 or 8");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_group_seqs, 4) || !aligned(prefix_lens, 4) ||
      !aligned(lse_out, 4))
    return fail(METIS_E_ALIGN, "tensors must be 16-byte aligned (index arrays and lse_out: 4-byte)");
  SharedArgs a;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.cu_group_seqs = cu_group_seqs;
  a.prefix_lens = prefix_lens;
  a.out = out;
  a.lse_out = lse_out;
  a.S = num_seqs;
  a.num_groups = num_groups;
  a.H = num_heads;
  a.G = num_kv_heads;
  a.D = head_dim;
  a.bs = block_size;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.cap = effective_max_len(max_seq_len, max_blocks, block_size);
  a.scale = scale;
  const long long units = shared_units(num_seqs, num_groups, r, num_kv_heads);
  if (units * ((a.cap - 1) / kSharedRows + 1) > 0x7fffffffLL) return fail(METIS_E_SHAPE, "too many tiles of shared tokens");
  int sms = 0;
  rc = current_sms(&sms);
  if (rc) return rc;
  const size_t need = shared_bytes(num_seqs, num_heads, num_kv_heads, head_dim, num_groups, sms);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
    return fail(METIS_E_WORKSPACE, "workspace must hold %zu bytes (256-byte aligned)", need);
  SharedPlan* plan = reinterpret_cast<SharedPlan*>(workspace);
  float* part_lse = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + shared_plan_bytes(num_groups));
  float* part_out = part_lse + (size_t)(units + sms) * 2 * kSharedRows;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = launch_shared_prefix(a, plan, part_lse, part_out, sms, st);
  if (rc) return rc;
  SharedParams sp{};
  DecodeParams& p = sp.d;
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
  p.r = r;
  p.scale_log2 = scale * kLog2e;
  p.max_parts = 1;
  p.cap = a.cap;
  sp.cu_group_seqs = cu_group_seqs;
  sp.prefix_lens = prefix_lens;
  sp.plan = plan;
  sp.part_lse = part_lse;
  sp.part_out = part_out;
  sp.num_groups = num_groups;
  sp.Tq = kSharedRows / r;
  const long long items = (long long)num_kv_heads * num_seqs;
  const int parts = item_parts(items, a.cap, sms);
  if (one_warp_items(items, sms))
    return head_dim == 64 ? launch_shared<64, 1>(sp, a, 1, st) : launch_shared<128, 1>(sp, a, 1, st);
  return head_dim == 64 ? launch_shared<64, kBf16Warps>(sp, a, parts, st)
                        : launch_shared<128, kBf16Warps>(sp, a, parts, st);
}
