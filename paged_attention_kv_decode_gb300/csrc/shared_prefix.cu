// Decode attention of a batch whose sequences share their first tokens in groups (a system prompt, a
// document that many requests ask about): the paged-attention kernel of the vllm-metal article,
// section 3, over the pages that prefix caching lets sequences share (vllm-metis 0.1.0 page, "Caches").
//
// Softmax attention over a sequence's tokens is the log-sum-exp join of its attention over the shared
// ones and over its own.  Decoding each sequence by itself reads the shared pages once per sequence; here
//
//   1 the members' queries of a group become the rows of query tiles, and the chunk kernel (prefill.cu,
//     SHARED) runs them over the prefix on the tensor cores: its K and V are read once per 256 rows.  All
//     tiles of all groups are cut into equal shares, so a unit may be several CTAs' parts.
//   2 the sequences' own tokens are decoded by warps that walk shares of them (decode_stream.cuh): the 16-token
//     units of all sequences in a row, cut into equal shares that the warps claim for a KV head each.
//   3 a kernel over the rows joins their parts.
//
// 1 is bound by the tensor cores and the start and end of its units, 2 by HBM: they run side by side.  1
// takes as many SMs as make the two end together (shared_split.cuh), 2 the others.  2 is a
// programmatic dependent of 1 that does not wait for it but at its very end; what 2 needs of 1 (the number of
// SMs, where each sequence's own tokens begin) is written before 1 lets it start.
//
// Measured (32 / 8 heads x 128): 64 sequences behind a document of 16,384 tokens 52.3 us, of which 1 and 2 run until
// 44 and 3 ends 5 later (2 behind 1, a CTA per item: 64); 1,024 sequences behind 16 system prompts 110 us, 2 on 126
// SMs until 95, an SM taking in 40 GB/s, and 3 (50 MB of parts) 14 (2 behind 1: 132).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "../../include/metis_attn.h"
#include "decode_stream.cuh"

namespace metis {

__device__ unsigned int g_status_shared = 0;

constexpr int kSharedRows = 128;  // rows of a query tile
constexpr int kMinUnits = 4;      // units (16 tokens of a KV head) of a share at least
constexpr int kLargeShares = 2;   // shares for each warp: large ones of the first three quarters of the units,
constexpr int kSmallShares = 4;   // small ones of the others, so that the warps end together (shares of one size: the
                                  // document's 56.7 us for 51.7, the prompts' 112 for 110)
constexpr int kRuns = 2048;       // (65,535 sequences: runs of 32)

struct SharedParams {
  DecodeParams d;
  const int32_t* cu_group_seqs;
  SharedPlan* plan;
  const SharedOwn* own;     // [S]
  const float* prefix_lse;  // [part][query tile][row], log2 units
  const float* prefix_out;  // ... [head_dim], normalised
  const int2* unit_parts;   // [unit]: its first and last part
  int2* own_parts;          // [S]: the first and last share with units of the sequence
  float* own_lse;           // [part][r], log2 units; part: (number of the sequence + of the share) * G + KV head
  float* own_out;           // ... [head_dim], normalised
  int Tq, prefix_slots, own_slots;  // slots: parts that there is memory for (own: for each KV head)
};

// The shares of a KV head's units: the first `large` of them cut [0, first) evenly, the `small` others the rest.
struct OwnShares {
  long long units, first;
  int large, small;
  __device__ __forceinline__ OwnShares(long long units_, long long warps)  // warps: for each KV head, at least one
      : units(units_), first(units_ - units_ / 4) {
    large = (int)max(min(warps * kLargeShares, first / kMinUnits), first > 0 ? 1ll : 0ll);
    small = (int)max(min(warps * kSmallShares, (units - first) / kMinUnits), units > first ? 1ll : 0ll);
  }
  __device__ __forceinline__ int count() const { return large + small; }
  __device__ __forceinline__ long long edge(int i) const {
    return i < large ? i * first / large : small ? first + (i - large) * (units - first) / small : units;
  }
};

// Exclusive prefix over the kStreamWarps * 32 threads of a block; *total: of all.
__device__ __forceinline__ long long stream_scan(long long v, long long* sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the last round's sums were read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long front = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kStreamWarps; ++w) {
    if (w < warp) front += sums[w];
    all += sums[w];
  }
  *total = all;
  return front + x - v;
}

template <int D>
__global__ void __launch_bounds__(kStreamWarps * 32, 1) decode_own_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                          const __grid_constant__ CUtensorMap tmV,
                                                                          const SharedParams sp) {
  constexpr int STAGES = stream_stages<D>(), STAGE_BYTES = Bf16DecodeShape<D>::kStageBytes;
  constexpr int KS = Bf16DecodeShape<D>::kSteps;
  const DecodeParams& p = sp.d;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // 1024-aligned for the swizzle
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStreamWarps * STAGES * STAGE_BYTES);
  // The kernel over the prefixes, in front of this one, let it start once all its CTAs had waited for
  // the kernels before: their outputs are there (lines that they left in this SM's L1 are dropped).
  __threadfence();
  pdl_launch_dependents();
  // A CTA that starts behind the other kernel's, with nothing left to do.  One thread looks: others claim
  // meanwhile, and a CTA whose threads saw different counts would run without its barriers.
  bool late = false;
  if (threadIdx.x == 0) {
    const long long planned = __ldcg(&sp.plan->own_shares);  // (0: not counted yet)
    late = planned > 0 && __ldcg(&sp.plan->next_share) >= planned * p.G;
  }
  if (__syncthreads_or(late)) {
    pdl_wait();
    return;
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < kStreamWarps * STAGES; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // Sequence s's units of one KV head
  auto units_of = [&](int s, WindowSpan* span) {
    const int L = min(max(p.seq_lens[s], 0), p.cap), begin = __ldcg(&sp.own[s].begin);
    *span = window_span(L, L - begin, 0);
    return L > begin ? span->n : 0;
  };
  // Every CTA adds them up, kPer sequences per thread and round, and keeps the sums in front of each run of
  // `run` sequences.
  constexpr int kPer = 4, kRound = kStreamWarps * 32 * kPer;
  __shared__ long long sums[kStreamWarps];
  __shared__ long long front[kRuns + 1];
  const int run = (p.S + kRuns - 1) / kRuns;
  long long total = 0;
  for (int s0 = 0; s0 < p.S; s0 += kRound) {
    int n[kPer];
    long long sum = 0, all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = s0 + tid * kPer + i;
      WindowSpan span;
      n[i] = s < p.S ? units_of(s, &span) : 0;
      sum += n[i];
    }
    long long at = total + stream_scan(sum, sums, &all);
    total += all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = s0 + tid * kPer + i;
      if (s < p.S && s % run == 0) front[s / run] = at;
      at += n[i];
    }
  }
  const int runs = (p.S + run - 1) / run;
  // shares for the warps of the SMs that the other kernel leaves; what one has not claimed when another is done
  // (on those that it leaves later, too) goes to that
  const int warps = max(((int)gridDim.x - __ldcg(&sp.plan->total.y)) * kStreamWarps / p.G, 1);
  const OwnShares shares(total, warps);
  if (blockIdx.x == 0 && tid == 0) sp.plan->own_shares = max(shares.count(), 1);
  __syncthreads();  // (the barriers are initialised, too)

  // The walk over this warp's shares: the next unit `at` of the share, which ends at `end`, is unit u of `units` of
  // sequence s, KV head g.  The KV heads of a share are claimed one after another, so that they run at about the same
  // time: the rows of a token's heads lie side by side in memory.
  long long at = 0, end = 0;
  int s = 0, g = 0, u = 0, units = 0, share = 0;
  WindowSpan span{};
  auto next = [&](StreamItem& it) -> bool {
    if (at >= end) {
      unsigned id = 0;
      if (lane == 0) id = atomicAdd(&sp.plan->next_share, 1u);
      id = __shfl_sync(0xffffffffu, id, 0);
      share = (int)(id / (unsigned)p.G);
      g = (int)(id - (unsigned)share * p.G);
      if (share >= shares.count()) return false;
      at = shares.edge(share);
      end = shares.edge(share + 1);
      int lo = 0, hi = runs - 1;  // the last run that begins at or before the share
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (front[mid] <= at)
          lo = mid;
        else
          hi = mid - 1;
      }
      // its sequences, one per lane
      const int mine = lo * run + lane;
      WindowSpan ignored;
      const long long n = lane < run && mine < p.S ? units_of(mine, &ignored) : 0;
      long long x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      x += front[lo];  // units up to the lane's sequence's end
      const uint32_t behind = __ballot_sync(0xffffffffu, x > at);
      const int k = behind ? __ffs(behind) - 1 : 0;
      u = (int)(at - __shfl_sync(0xffffffffu, x - n, k));
      s = lo * run + k;
      units = units_of(s, &span);
    }
    while (u >= units) {
      if (s + 1 >= p.S) return false;  // (not met: a share ends within the sequences' units)
      units = units_of(++s, &span);
      u = 0;
    }
    it.s = s;
    it.g = g;
    it.part = (s + share) * p.G + g;
    it.span = span;
    it.span.first = u;
    it.span.n = (int)min((long long)(units - u), end - at);
    if (g == 0 && lane == 0) {
      if (u == 0) sp.own_parts[s].x = share;
      if (u + it.span.n == units) sp.own_parts[s].y = share;
    }
    at += it.span.n;
    u += it.span.n;
    return true;
  };
  auto store = [&](const StreamItem& it, const DecodeWarp<D>& state) {
    const int q4 = lane & 3, rA = lane >> 2, h = 2 * q4;
    const float l0 = warp_sum_xor(state.l0, 4), l1 = warp_sum_xor(state.l1, 4);
    const float i0 = 1.f / l0, i1 = 1.f / l1;
    const size_t row = (size_t)it.part * p.r + h;
    float* to = sp.own_out + row * D + rA;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      if (h < p.r) {
        to[mt * 16] = state.o[mt][0] * i0;
        to[mt * 16 + 8] = state.o[mt][2] * i0;
      }
      if (h + 1 < p.r) {
        to[D + mt * 16] = state.o[mt][1] * i1;
        to[D + mt * 16 + 8] = state.o[mt][3] * i1;
      }
    }
    if (rA == 0 && h < p.r) sp.own_lse[row] = state.m0 + log2f(l0);
    if (rA == 0 && h + 1 < p.r) sp.own_lse[row + 1] = state.m1 + log2f(l1);
  };
  decode_stream<D>(tmK, tmV, p, smem + warp * STAGES * STAGE_BYTES, bars + warp * STAGES, lane, &g_status_shared, next,
                   store);
  pdl_wait();  // this grid completes after the one over the prefixes
}

// A float4 column per lane (head_dim 64: two query heads at a time): the chunks of the sequence's own tokens,
// then the parts of its prefix, kBatch of them for kHeads heads in flight.  A row's few parts: a warp per
// (sequence, KV head), four heads at a time; many (MANY: units with a good share of the SMs each): one.
constexpr int kJoinWarps = 4;
template <int D>
constexpr int join_heads(bool many) {  // query heads of a warp at a time
  return many ? 128 / D : 4;
}
template <int D, bool MANY>
__global__ void __launch_bounds__(kJoinWarps * 32) join_shared_kernel(const SharedParams sp) {
  constexpr int LANES = D / 4, ROWS = 32 / LANES, kBatch = MANY ? 8 : 2, kHeads = join_heads<D>(MANY) / ROWS;
  const DecodeParams& p = sp.d;
  // What the kernel over the prefixes wrote before it let the one in front of this start, and the call's inputs,
  // are there (lines left in this SM's L1 are dropped); the rest behind the wait.
  __threadfence();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int blocks = (p.r + kHeads * ROWS - 1) / (kHeads * ROWS);  // of a KV head's query heads
  if (item >= (long long)p.S * p.G * blocks) return;  // (the others' waits hold this grid back)
  const int sg = (int)(item / blocks), h0 = (int)(item - (long long)sg * blocks) * kHeads * ROWS;
  const int s = sg / p.G, g = sg - s * p.G, d = (lane % LANES) * 4;
  const SharedOwn own{__ldcg(&sp.own[s].begin), __ldcg(&sp.own[s].group)};
  int unit = -1;  // of the prefix
  size_t at = 0;  // the first head's row in each of its parts
  if (own.group >= 0) {
    const int2 v = __ldcg(sp.plan->group + own.group);
    if (v.y > 0 && __ldcg(&sp.plan->total.x) > 0) {
      const int member = s - sp.cu_group_seqs[own.group], pair = member / (2 * sp.Tq), in = member - pair * 2 * sp.Tq;
      unit = v.x + g * v.y + pair;
      at = (size_t)(in / sp.Tq) * kSharedRows + in % sp.Tq;
    }
  }
  const int L = min(max(p.seq_lens[s], 0), p.cap);
  const int units = L > own.begin ? window_span(L, L - own.begin, 0).n : 0;
  pdl_wait();  // the kernels over the own tokens and, before it, over the prefixes are complete
  // parts: first, first + 1, ..., and chunks of the own tokens
  int first = 0, count = 0, chunks = 0;
  size_t own_row = 0;
  // (held to the workspace's, should a wait of the kernels in front have given up)
  if (units > 0) {
    const int2 v = __ldcg(sp.own_parts + s);
    const int x = min(max(v.x, 0), sp.own_slots - 1 - s);
    chunks = min(max(v.y - x + 1, 0), sp.own_slots - s - x);
    own_row = ((size_t)(s + x) * p.G + g) * p.r;
  }
  if (unit >= 0) {
    const int2 v = __ldcg(sp.unit_parts + unit);
    first = min(max(v.x, 0), sp.prefix_slots - 1);
    count = min(max(v.y - first + 1, 0), sp.prefix_slots - first);
  }
  {
    JoinedRow sum[kHeads];
    for (int k0 = 0; k0 < chunks + count; k0 += kBatch) {
      float x[kHeads][kBatch];
      float4 v[kHeads][kBatch];
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int k = k0 + j, h = h0 + i * ROWS + lane / LANES;
          x[i][j] = -INFINITY;
          v[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (h >= p.r) continue;
          if (k < chunks) {
            const size_t r = own_row + (size_t)k * p.H + h;
            x[i][j] = __ldcg(sp.own_lse + r);
            v[i][j] = __ldcg(reinterpret_cast<const float4*>(sp.own_out + r * D + d));
          } else if (k < chunks + count) {
            const size_t r = (size_t)(first + k - chunks) * 2 * kSharedRows + at + h * sp.Tq;
            x[i][j] = __ldcg(sp.prefix_lse + r);
            v[i][j] = __ldcg(reinterpret_cast<const float4*>(sp.prefix_out + r * D + d));
          }
        }
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
#pragma unroll
        for (int j = 0; j < kBatch; ++j) sum[i].add(x[i][j], v[i][j]);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i * ROWS + lane / LANES;
      if (h >= p.r) continue;
      const bool empty = sum[i].W == 0.f;  // no token
      const float inv = empty ? 0.f : 1.f / sum[i].W;
      const size_t row = (size_t)s * p.H + g * p.r + h;
      store4<__nv_bfloat16>(reinterpret_cast<__nv_bfloat16*>(p.out) + row * D + d, sum[i].a0 * inv, sum[i].a1 * inv,
                            sum[i].a2 * inv, sum[i].a3 * inv);
      if (d == 0 && p.lse_out) p.lse_out[row] = empty ? -INFINITY : (sum[i].M + log2f(sum[i].W)) * kLn2;
    }
  }
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

// The workspace, in this order
struct SharedSpace {
  size_t own, unit_parts, own_parts, prefix_lse, prefix_out, own_lse, own_out, bytes;  // offsets behind the plan
  int prefix_slots, own_slots;
};
static SharedSpace shared_space(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int num_groups, int sms) {
  SharedSpace w;
  const size_t r = num_heads / num_kv_heads, items = (size_t)num_seqs * num_kv_heads;
  const size_t units = (size_t)shared_units(num_seqs, num_groups, (int)r, num_kv_heads), parts = units + sms;
  const size_t rows = (items + ((size_t)sms * kStreamWarps + num_kv_heads) * (kLargeShares + kSmallShares)) * r;
  w.prefix_slots = (int)parts;
  w.own_slots = (int)(rows / r / num_kv_heads);
  w.own = align_up(sizeof(SharedPlan) + (size_t)num_groups * sizeof(int2), 256);
  w.unit_parts = align_up(w.own + (size_t)num_seqs * sizeof(SharedOwn), 256);
  w.own_parts = align_up(w.unit_parts + units * sizeof(int2), 256);
  w.prefix_lse = align_up(w.own_parts + (size_t)num_seqs * sizeof(int2), 256);
  w.prefix_out = align_up(w.prefix_lse + parts * 2 * kSharedRows * sizeof(float), 256);
  w.own_lse = align_up(w.prefix_out + parts * 2 * kSharedRows * head_dim * sizeof(float), 256);
  w.own_out = align_up(w.own_lse + rows * sizeof(float), 256);
  w.bytes = align_up(w.own_out + rows * head_dim * sizeof(float), 256);
  return w;
}

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

template <int D>
static int launch_own(const SharedParams& sp, const SharedArgs& a, long long units, int sms, cudaStream_t st) {
  CUtensorMap tmK, tmV;
  int rc = encode_kv_maps<D>(sp.d, a.k_cache, a.v_cache, &tmK, &tmV);
  if (rc) return rc;
  constexpr int smem = stream_smem_bytes<D>();
  static int done = 0;
  auto kern = decode_own_kernel<D>;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem, &done);
  if (rc) return rc;
  rc = launch_dependent(kern, dim3((unsigned)sms), dim3(kStreamWarps * 32), (size_t)smem, st,
                        "decode_own_kernel launch", tmK, tmV, sp);
  if (rc) return rc;
  // a unit in four parts and more (document, 8 units: 51.7 us, four heads at a time 59.6; prompts, 256 units: 120.1
  // and 109.4)
  const bool many = 4 * units <= sms;
  const int heads = join_heads<D>(many);
  const long long warps = (long long)a.S * a.G * ((sp.d.r + heads - 1) / heads);
  const dim3 grid((unsigned)((warps + kJoinWarps - 1) / kJoinWarps)), block(kJoinWarps * 32);
  return many ? launch_dependent(join_shared_kernel<D, true>, grid, block, 0, st, "join_shared_kernel launch", sp)
              : launch_dependent(join_shared_kernel<D, false>, grid, block, 0, st, "join_shared_kernel launch", sp);
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
  return shared_space(num_seqs, num_heads, num_kv_heads, head_dim, num_groups, sms).bytes;
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
  const SharedSpace w = shared_space(num_seqs, num_heads, num_kv_heads, head_dim, num_groups, sms);
  if (!workspace || workspace_bytes < w.bytes || !aligned(workspace, 256))
    return fail(METIS_E_WORKSPACE, "workspace must hold %zu bytes (256-byte aligned)", w.bytes);
  if ((long long)num_seqs * num_kv_heads > 0x70000000LL) return fail(METIS_E_SHAPE, "too many items");
  char* base = reinterpret_cast<char*>(workspace);
  SharedPlan* plan = reinterpret_cast<SharedPlan*>(base);
  SharedOwn* own = reinterpret_cast<SharedOwn*>(base + w.own);
  float* prefix_lse = reinterpret_cast<float*>(base + w.prefix_lse);
  float* prefix_out = reinterpret_cast<float*>(base + w.prefix_out);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = launch_shared_prefix(a, plan, own, reinterpret_cast<int2*>(base + w.unit_parts), prefix_lse, prefix_out, sms, st);
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
  sp.plan = plan;
  sp.own = own;
  sp.prefix_lse = prefix_lse;
  sp.prefix_out = prefix_out;
  sp.own_lse = reinterpret_cast<float*>(base + w.own_lse);
  sp.own_out = reinterpret_cast<float*>(base + w.own_out);
  sp.unit_parts = reinterpret_cast<int2*>(base + w.unit_parts);
  sp.own_parts = reinterpret_cast<int2*>(base + w.own_parts);
  sp.Tq = kSharedRows / r;
  sp.prefix_slots = w.prefix_slots;
  sp.own_slots = w.own_slots;
  return head_dim == 64 ? launch_own<64>(sp, a, units, sms, st) : launch_own<128>(sp, a, units, sms, st);
}
