// The index arrays of a serving step, built on the GPU from the requests' lengths.
//
// The scheduler's block table and sequence lengths drive every attention call (vllm-metal
// article, section 4), and vLLM's cache manager deals out the pages (vllm-metis 0.1.0 page,
// "How the model maps onto vLLM", "Caches").  Here one launch does for a batch what a host
// loop would: sequence s has L0 cached tokens and gets n new ones;
//
//   pages     ceil((L0 + n) / block_size) of them, those missing from its table row taken from the
//             top of the free stack, sequence by sequence and page by page
//   row i     of its n rows: position L0 + i, slot page * block_size + position % block_size
//   offsets   cu[s] = n_0 + ... + n_(s-1)
//
// so that a captured decode loop advances without the host (lengths, page counts and the stack's
// depth may be updated in place).
//
// Bound by latency: a step of 64 tokens moves 2 KB, 400,000 rows 5 MB.  Every CTA of a cluster scans all
// lengths itself (a few sequences per thread and round; two scans, tokens and then pages), the cluster's
// barrier separates the reads of those lengths from their update, and the CTAs share the pages and rows.  A
// small step is one CTA of 256 threads: its barriers are the time.  Many rows would keep the cluster's eight
// SMs busy with finding each row's sequence: a second kernel fills them, on every SM, from the offsets,
// lengths and table that the first one wrote.
//
// Measured: 64 sequences of one token 3.9 us, 1,024 of them 7.3 (by the cluster 7.0 and 8.4; around 2,048 rows, of 256
// sequences 8.8 and 8.9, of 1,024 sequences 11.6 and 9.6); 4,096 prompts with 393 K rows 16.9 us, 11 of them the first
// kernel.
#include <algorithm>

#include "../../include/metis_attn.h"
#include "cluster.cuh"
#include "common.cuh"
#include "host.h"

namespace metis {

__device__ unsigned int g_status_plan = 0;

constexpr int kPlanTile = 128;       // rows a warp takes at a time
constexpr int kMaxCluster = 8;
constexpr int kPlanSmall = 256;      // threads of a small step's one CTA, 4 sequences each in a round: one round,
constexpr int kPlanSmallRows = 2048; // and up to so many rows
constexpr int kPlanWide = 1024;      // otherwise: 8 sequences each
template <int NT>
constexpr int plan_per() {
  return NT == kPlanSmall ? 4 : 8;
}
// More rows are left to the second kernel.  (7.7 K rows 8.5 us in the first, 10.7 in the second, 24 K even at 11.0,
// 393 K 65.6 and 16.9.)
constexpr int kPlanOwnRows = 8192;
constexpr int kRowWarps = 4;

struct PlanParams {
  const int32_t* q_lens;
  const int32_t* cached_lens;
  const int32_t* held_blocks;  // NULL: ceil(cached / block_size)
  const int32_t* free_stack;
  const int32_t* free_count;
  int32_t* block_table;
  int32_t* refcount;           // NULL: not kept
  int32_t* seq_lens;
  int32_t* held_out;           // NULL: not wanted
  int32_t* free_count_out;
  int32_t* cu_q_lens;
  int64_t* slot_mapping;
  int32_t* positions;
  int S, T, bs, max_blocks, num_blocks, free_capacity;
};

// What a CTA keeps of the sequences of the current round
template <int NT>
struct PlanSeqs {
  static constexpr int N = NT * plan_per<NT>();
  int cu[N + 1];  // first row
  int before[N];  // cached tokens
  int held[N];    // pages in its table row
  int page[N];    // its first new page, in the order of taking
};

// Exclusive prefix of one value per thread, sums held at `top` (the sums of a batch may pass it:
// min(a + b, top) adds up in any order); *total: of all.
template <int NT>
__device__ __forceinline__ int plan_scan(int v, int top, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto add = [top](int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)top); };
  auto inclusive = [&](int x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = add(x, y);
    }
    return x;
  };
  const int x = inclusive(v);
  int left = __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == 0) left = 0;
  __syncthreads();  // the last scan's sums were read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  // every warp sums the warps for itself: one barrier less
  const int sums = inclusive(lane < NT / 32 ? warp_sums[lane] : 0);
  *total = __shfl_sync(0xffffffffu, sums, NT / 32 - 1);
  const int front = __shfl_sync(0xffffffffu, sums, max(warp - 1, 0));
  return warp > 0 ? add(left, front) : left;
}

// The last of v[lo .. hi] at or below x (v[lo] is)
__device__ __forceinline__ int plan_find(const int* v, int lo, int hi, int x) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <int NT, bool ROWS>
__global__ void __launch_bounds__(NT, 1) plan_step_kernel(const PlanParams p) {
  constexpr int PER = plan_per<NT>(), SEQS = NT * PER;
  extern __shared__ uint8_t plan_smem[];
  PlanSeqs<NT>& seqs = *reinterpret_cast<PlanSeqs<NT>*>(plan_smem);
  __shared__ int warp_sums[NT / 32];
  pdl_launch_dependents();
  pdl_wait();  // lengths, table and stack may be what the kernel in front writes
  const int tid = threadIdx.x, ctas = gridDim.x, cta = blockIdx.x;  // the grid is one cluster
  const int depth = min(max(*p.free_count, 0), p.free_capacity);

  int rows = 0, taken = 0;  // by the rounds before this one
  for (int base = 0; base < p.S; base += SEQS) {
    const int n_seqs = min(p.S - base, SEQS);
    int n[PER], before[PER], held[PER];
    int sum = 0;
    unsigned bad = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = tid * PER + i;
      n[i] = before[i] = held[i] = 0;
      if (s < n_seqs) {
        n[i] = p.q_lens[base + s];
        before[i] = p.cached_lens[base + s];
        if (p.held_blocks) held[i] = p.held_blocks[base + s];
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (n[i] < 0 || before[i] < 0) bad |= METIS_STATUS_BAD_Q_LEN;
      n[i] = max(n[i], 0);
      before[i] = max(before[i], 0);
      sum = (int)min((unsigned)sum + (unsigned)n[i], (unsigned)p.T);
    }
    int total;
    const int left = p.T - rows;  // rows that the call still has
    int at = plan_scan<NT>(min(sum, left), left, warp_sums, &total), pages = 0, take[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = tid * PER + i;
      if (n[i] > left - at) {  // rows past the call's: those tokens are not planned
        n[i] = left - at;
        bad |= METIS_STATUS_BAD_OFFSETS;
      }
      const int have = (int)(((unsigned)before[i] + p.bs - 1) / (unsigned)p.bs);
      held[i] = min(max(held[i], have), p.max_blocks);
      const unsigned after = (unsigned)before[i] + (unsigned)n[i];
      const int want = (int)min((after + p.bs - 1) / (unsigned)p.bs, (unsigned)p.max_blocks);
      if (n[i] > 0 && (after - 1) / (unsigned)p.bs >= (unsigned)p.max_blocks) bad |= METIS_STATUS_SEQ_TOO_LONG;
      take[i] = n[i] > 0 ? max(want - held[i], 0) : 0;
      pages += take[i];
      if (s < n_seqs) {
        seqs.cu[s] = rows + at;
        seqs.before[s] = before[i];
        seqs.held[s] = held[i];
      }
      at += n[i];
    }
    int total_pages;
    int first = taken + plan_scan<NT>(pages, 0x7fffffff, warp_sums, &total_pages);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = tid * PER + i;
      if (s < n_seqs) seqs.page[s] = first;
      first += take[i];
    }
    if (tid == 0) seqs.cu[n_seqs] = rows + total;
    if (tid == 0 && taken + total_pages > depth) bad |= METIS_STATUS_OUT_OF_PAGES;
    if (bad) atomicOr(&g_status_plan, bad);
    if (ctas > 1)
      cluster_sync_all();  // every CTA has read the lengths: they may be updated in place
    else
      __syncthreads();

    // per sequence
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = tid * PER + i;
      if (s < n_seqs && s % ctas == cta) {
        p.seq_lens[base + s] = (int)min((unsigned)before[i] + (unsigned)n[i], 0x7fffffffu);
        if (p.held_out) p.held_out[base + s] = held[i] + take[i];
        p.cu_q_lens[base + s] = seqs.cu[s];
        if (!ROWS && n[i] > 0) {  // entries that the row names already and its new tokens use
          const int last = min((before[i] + n[i] - 1) / p.bs, held[i] - 1);
          for (int page = before[i] / p.bs; page <= last; ++page)
            checked_block(p.block_table + (size_t)(base + s) * p.max_blocks, page, p.num_blocks, &g_status_plan);
        }
      }
    }
    // per new page
    for (long long next = (long long)taken + cta * NT + tid; next < (long long)taken + total_pages; next += ctas * NT) {
      const int k = (int)next, s = plan_find(seqs.page, 0, n_seqs - 1, k);
      int block = -1;
      if (k < depth) block = checked_block(p.free_stack, depth - 1 - k, p.num_blocks, &g_status_plan);
      p.block_table[(size_t)(base + s) * p.max_blocks + seqs.held[s] + (k - seqs.page[s])] = block;
      if (p.refcount && block >= 0) p.refcount[block] = 1;
    }
    // per row
    const int end = rows + total;
    if constexpr (ROWS) {
      for (long long next = (long long)rows + cta * NT + tid; next < end; next += ctas * NT) {
        const int row = (int)next, s = plan_find(seqs.cu, 0, n_seqs - 1, row);
        const unsigned pos = (unsigned)seqs.before[s] + (unsigned)(row - seqs.cu[s]);
        const unsigned page = pos / (unsigned)p.bs, off = pos - page * (unsigned)p.bs;
        int block = -1;
        if ((int)page < seqs.held[s]) {
          block = checked_block(p.block_table + (size_t)(base + s) * p.max_blocks, (int)page, p.num_blocks, &g_status_plan);
        } else if (page < (unsigned)p.max_blocks) {
          const int k = seqs.page[s] + (int)page - seqs.held[s];
          if (k < depth) block = checked_block(p.free_stack, depth - 1 - k, p.num_blocks, &g_status_plan);
        }
        p.slot_mapping[row] = block < 0 ? -1 : (int64_t)block * p.bs + off;
        p.positions[row] = (int)min(pos, 0x7fffffffu);
      }
    }
    rows += total;
    taken += total_pages;
    __syncthreads();  // the next round overwrites the sequences
  }
  if constexpr (ROWS) {  // rows behind the last sequence's: padding
    for (long long row = (long long)rows + cta * NT + tid; row < p.T; row += ctas * NT) {
      p.slot_mapping[row] = -1;
      p.positions[row] = 0;
    }
  }
  if (cta == 0 && tid == 0) {
    p.cu_q_lens[p.S] = rows;
    *p.free_count_out = max(depth - taken, 0);  // every CTA read the depth before the first barrier
  }
}

// The rows of a step from its offsets, lengths and table.  A warp finds the sequence of its tile's first
// row by thirty-two probes at a time; the offsets of the 32 sequences from there on, one per lane, then
// place every row by shuffles.  (Shorter sequences: by halves, in memory.)
__global__ void __launch_bounds__(kRowWarps * 32) plan_rows_kernel(const PlanParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long tile = ((long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5)) * kPlanTile;
  if (tile >= p.T) return;
  const int* cu = p.cu_q_lens;
  int lo = 0, n = p.S;  // the last of cu[0 .. S - 1] at or below the tile's first row
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = min(lane * step, n - 1);
    const int before = __popc(__ballot_sync(0xffffffffu, lane * step < n && cu[lo + at] <= (int)tile));
    lo += (before - 1) * step;  // (cu[0] = 0: the first probe counts)
    n = min(step, n - (before - 1) * step);
  }
  const int rows = cu[p.S];
  const int edge = cu[min(lo + 1 + lane, p.S)];  // where the sequences from lo + 1 on begin
  const bool near = __shfl_sync(0xffffffffu, edge, 31) > min((int)tile + kPlanTile, rows) - 1;
  constexpr int J = kPlanTile / 32;
  int s[J], from[J], pos[J], block[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int row = (int)min(tile + j * 32 + lane, (long long)p.T - 1);
    int k = 0;  // sequences from lo + 1 on that begin at or before the row
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (__shfl_sync(0xffffffffu, edge, k + o - 1) <= row) k += o;
    s[j] = min(lo + k, p.S - 1);
    if (!near) s[j] = plan_find(cu, lo, p.S - 1, row);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    from[j] = cu[s[j] + 1];
    pos[j] = p.seq_lens[s[j]];
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const long long row = tile + j * 32 + lane;
    pos[j] -= from[j] - (int)row;
    const int page = pos[j] / p.bs;
    block[j] = -1;
    if (row < rows && page >= 0 && page < p.max_blocks) block[j] = p.block_table[(size_t)s[j] * p.max_blocks + page];
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const long long row = tile + j * 32 + lane;
    if (row >= p.T) continue;
    const bool fine = block[j] >= 0 && block[j] < p.num_blocks;  // (else flagged by the kernel in front)
    p.slot_mapping[row] = fine ? (int64_t)block[j] * p.bs + pos[j] % p.bs : -1;
    p.positions[row] = row < rows ? pos[j] : 0;
  }
}

int plan_status(uint32_t* bits, int clear) {
  unsigned int v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_status_plan, sizeof(v));
  if (e == cudaSuccess && clear) {
    unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_status_plan, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  *bits |= v;
  return METIS_OK;
}

}  // namespace metis

using namespace metis;

extern "C" int metis_plan_step(const int32_t* q_lens, const int32_t* cached_lens, const int32_t* held_blocks,
                               int32_t* block_table, const int32_t* free_stack, int free_capacity,
                               const int32_t* free_count, int32_t* refcount, int32_t* seq_lens, int32_t* held_blocks_out,
                               int32_t* free_count_out, int32_t* cu_q_lens, int64_t* slot_mapping, int32_t* positions,
                               int num_seqs, int num_tokens, int block_size, int max_blocks, int num_blocks,
                               void* stream) {
  clear_error();
  if (num_seqs < 0 || num_tokens < 0) return fail(METIS_E_SHAPE, "num_seqs and num_tokens must be >= 0");
  if (num_seqs == 0) return METIS_OK;
  if (!q_lens || !cached_lens || !block_table || !free_count || !seq_lens || !free_count_out || !cu_q_lens ||
      (num_tokens > 0 && (!slot_mapping || !positions)) || (free_capacity > 0 && !free_stack))
    return fail(METIS_E_NULL, "q_lens, cached_lens, block_table, free_stack, free_count, seq_lens, free_count_out, "
                              "cu_q_lens, slot_mapping and positions are required");
  if (block_size <= 0 || max_blocks <= 0 || num_blocks <= 0 || free_capacity < 0)
    return fail(METIS_E_SHAPE, "sizes must be positive");
  if ((long long)max_blocks * block_size > 0x7fffffffLL)
    return fail(METIS_E_SHAPE, "max_blocks * block_size must fit in int32");
  if (!aligned(q_lens, 4) || !aligned(cached_lens, 4) || !aligned(held_blocks, 4) || !aligned(block_table, 4) ||
      !aligned(free_stack, 4) || !aligned(free_count, 4) || !aligned(refcount, 4) || !aligned(seq_lens, 4) ||
      !aligned(held_blocks_out, 4) || !aligned(free_count_out, 4) || !aligned(cu_q_lens, 4) ||
      !aligned(slot_mapping, 8) || !aligned(positions, 4))
    return fail(METIS_E_ALIGN, "index arrays must be 4-byte aligned (slot_mapping: 8-byte)");
  PlanParams p;
  p.q_lens = q_lens;
  p.cached_lens = cached_lens;
  p.held_blocks = held_blocks;
  p.free_stack = free_stack;
  p.free_count = free_count;
  p.block_table = block_table;
  p.refcount = refcount;
  p.seq_lens = seq_lens;
  p.held_out = held_blocks_out;
  p.free_count_out = free_count_out;
  p.cu_q_lens = cu_q_lens;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.S = num_seqs;
  p.T = num_tokens;
  p.bs = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.free_capacity = free_capacity;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (num_seqs <= PlanSeqs<kPlanSmall>::N && num_tokens <= kPlanSmallRows)
    return launch_dependent(plan_step_kernel<kPlanSmall, true>, dim3(1), dim3(kPlanSmall), sizeof(PlanSeqs<kPlanSmall>), st,
                            "plan_step_kernel launch", p);
  // (positions within int32: the second kernel counts them back from the lengths)
  const bool own_rows = num_tokens <= kPlanOwnRows || (long long)max_blocks * block_size > 0x7fffffffLL - num_tokens;
  auto launch = [&](auto kern, int ctas, int* done) {
    const int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), (int)sizeof(PlanSeqs<kPlanWide>), done);
    if (rc) return rc;
    return launch_dependent_cluster(kern, dim3((unsigned)ctas), dim3((unsigned)ctas), dim3(kPlanWide),
                                    sizeof(PlanSeqs<kPlanWide>), st, "plan_step_kernel launch", p);
  };
  static int done_rows = 0, done = 0;
  if (own_rows)
    return launch(plan_step_kernel<kPlanWide, true>,
                  (int)std::min<long long>(kMaxCluster, 1 + num_tokens / (2 * kPlanWide)), &done_rows);
  const int rc = launch(plan_step_kernel<kPlanWide, false>, kMaxCluster, &done);
  if (rc) return rc;
  const unsigned ctas = (unsigned)((num_tokens - 1) / (kRowWarps * kPlanTile) + 1);
  return launch_dependent(plan_rows_kernel, dim3(ctas), dim3(kRowWarps * 32), 0, st, "plan_rows_kernel launch", p);
}
