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
// Bound by latency: a step of 64 tokens moves 2 KB, 400,000 rows 5 MB.  One cluster of up to
// kMaxCluster CTAs: every CTA scans all lengths itself (4,096 sequences at a time, four per thread; two
// scans, tokens and then pages), the cluster's barrier separates the reads of those lengths from
// their update, and the CTAs share the rows.  Every page's first row also writes its table entry
// and reference count, so pages need no pass of their own.
#include <algorithm>

#include "../../include/metis_attn.h"
#include "cluster.cuh"
#include "common.cuh"
#include "host.h"

namespace metis {

__device__ unsigned int g_status_plan = 0;

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 4;                            // sequences per thread and scan
constexpr int kPlanSeqs = kPlanThreads * kPlanPer;     // sequences per scan
constexpr int kPlanTile = 128;                         // rows a warp takes at a time
constexpr int kMaxCluster = 8;

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

// What a CTA keeps of each sequence of the current scan
struct PlanSeqs {
  int cu[kPlanSeqs + 1];  // first row
  int before[kPlanSeqs];  // cached tokens
  int held[kPlanSeqs];    // pages in its table row
  int rank[kPlanSeqs];    // (first new page's place in the order of taking) - held
};

// Exclusive prefix of one value per thread, sums held at `top` (the sums of a batch may pass it:
// min(a + b, top) adds up in any order); *total: of all.
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
  if (warp == 0) warp_sums[lane] = inclusive(warp_sums[lane]);
  __syncthreads();
  *total = warp_sums[kPlanThreads / 32 - 1];
  return warp > 0 ? add(left, warp_sums[warp - 1]) : left;
}

__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(const PlanParams p) {
  extern __shared__ uint8_t plan_smem[];
  PlanSeqs& seqs = *reinterpret_cast<PlanSeqs*>(plan_smem);
  __shared__ int warp_sums[kPlanThreads / 32];
  static_assert(kPlanThreads == 32 * 32, "one warp scans the warp sums");
  pdl_launch_dependents();
  pdl_wait();  // lengths, table and stack may be what the kernel in front writes
  const int tid = threadIdx.x, lane = tid & 31;
  const int ctas = gridDim.x, cta = blockIdx.x;  // the grid is one cluster
  const int depth = min(max(*p.free_count, 0), p.free_capacity);
  const int all_warps = ctas * (kPlanThreads / 32), my_warp = cta * (kPlanThreads / 32) + (tid >> 5);

  int rows = 0, taken = 0;  // by the scans before this one
  for (int base = 0; base < p.S; base += kPlanSeqs) {
    const int n_seqs = min(p.S - base, kPlanSeqs);
    int n[kPlanPer], before[kPlanPer], held[kPlanPer];
    int sum = 0;
    unsigned bad = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int s = tid * kPlanPer + i;
      n[i] = before[i] = held[i] = 0;
      if (s < n_seqs) {
        n[i] = p.q_lens[base + s];
        before[i] = p.cached_lens[base + s];
        if (p.held_blocks) held[i] = p.held_blocks[base + s];
        if (n[i] < 0 || before[i] < 0) bad |= METIS_STATUS_BAD_Q_LEN;
        n[i] = max(n[i], 0);
        before[i] = max(before[i], 0);
      }
      sum = (int)min((unsigned)sum + (unsigned)n[i], (unsigned)p.T);
    }
    int total;
    const int left = p.T - rows;  // rows that the call still has
    const int first = plan_scan(min(sum, left), left, warp_sums, &total);
    int at = first, pages = 0, take[kPlanPer];
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int s = tid * kPlanPer + i;
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
    int rank = taken + plan_scan(pages, 0x7fffffff, warp_sums, &total_pages);
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int s = tid * kPlanPer + i;
      if (s < n_seqs) seqs.rank[s] = rank - held[i];
      rank += take[i];
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
    for (int i = 0; i < kPlanPer; ++i) {
      const int s = tid * kPlanPer + i;
      if (s < n_seqs && s % ctas == cta) {
        p.seq_lens[base + s] = (int)min((unsigned)before[i] + (unsigned)n[i], 0x7fffffffu);
        if (p.held_out) p.held_out[base + s] = held[i] + take[i];
        p.cu_q_lens[base + s] = seqs.cu[s];
      }
    }
    // per row
    const int end = rows + total;
    for (long long tile = (long long)rows + (long long)my_warp * kPlanTile; tile < end;
         tile += (long long)all_warps * kPlanTile) {
      int s = -1;
#pragma unroll 1
      for (int j = 0; j < kPlanTile; j += 32) {
        const long long row_ll = tile + j + lane;
        if (row_ll >= end) break;
        const int row = (int)row_ll;
        // the last sequence that begins at or before the row: a few steps on, else by halves
        int lo = max(s, 0), hi = n_seqs - 1;
        if (s >= 0)
          for (int step = 0; step < 4 && lo < hi; ++step) {
            if (seqs.cu[lo + 1] > row) hi = lo;
            else ++lo;
          }
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (seqs.cu[mid] <= row) lo = mid;
          else hi = mid - 1;
        }
        s = lo;
        const unsigned pos = (unsigned)seqs.before[s] + (unsigned)(row - seqs.cu[s]);
        const unsigned page = pos / (unsigned)p.bs, off = pos - page * (unsigned)p.bs;
        int block = -1;
        if (page < (unsigned)p.max_blocks) {
          int32_t* entry = p.block_table + (size_t)(base + s) * p.max_blocks + page;
          if ((int)page < seqs.held[s]) {
            block = checked_block(entry, 0, p.num_blocks, &g_status_plan);
          } else {
            const int k = seqs.rank[s] + (int)page;  // in the order of taking
            if (k < depth) block = checked_block(p.free_stack, depth - 1 - k, p.num_blocks, &g_status_plan);
            if (off == 0) {  // the page's first row
              *entry = block;
              if (p.refcount && block >= 0) p.refcount[block] = 1;
            }
          }
        }
        p.slot_mapping[row] = block < 0 ? -1 : (int64_t)block * p.bs + off;
        p.positions[row] = (int)min(pos, 0x7fffffffu);
      }
    }
    rows += total;
    taken += total_pages;
    __syncthreads();  // the next scan overwrites the sequences
  }
  // rows behind the last sequence's: padding
  for (long long row = (long long)rows + cta * kPlanThreads + tid; row < p.T; row += (long long)ctas * kPlanThreads) {
    p.slot_mapping[row] = -1;
    p.positions[row] = 0;
  }
  if (cta == 0 && tid == 0) {
    p.cu_q_lens[p.S] = rows;
    *p.free_count_out = max(depth - taken, 0);  // every CTA read the depth before the first barrier
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
  static int done = 0;
  const int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(plan_step_kernel), (int)sizeof(PlanSeqs), &done);
  if (rc) return rc;
  // a CTA for every two tiles of its warps' rows
  const int ctas = std::min(kMaxCluster, 1 + (num_tokens - 1) / (2 * kPlanThreads / 32 * kPlanTile));
  return launch_dependent_cluster(plan_step_kernel, dim3(std::max(ctas, 1)), dim3(std::max(ctas, 1)), dim3(kPlanThreads),
                                  sizeof(PlanSeqs), reinterpret_cast<cudaStream_t>(stream), "plan_step_kernel launch", p);
}
