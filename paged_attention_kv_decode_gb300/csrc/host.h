// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/metis_attn.h"

namespace metis {

// Record a message for metis_last_error() and return `code`.
int fail(int code, const char* fmt, ...);
void clear_error();

// cudaGetLastError() after a launch: METIS_OK, or METIS_E_CUDA with a message.
int check_launch(const char* what);

// Encode a tiled TMA descriptor (cuTensorMapEncodeTiled, fetched from the
// driver at run time).  dims / box are innermost first; strides are the byte
// strides of dims 1..rank-1.  Returns METIS_OK or an error code.
int encode_tiled(CUtensorMap* map, CUtensorMapDataType dtype, int rank, const void* base,
                 const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                 CUtensorMapSwizzle swizzle,
                 CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B);

// Launch `kernel` as a programmatic dependent of the previous kernel in the
// stream: it may start launching while that kernel still runs, so it must
// execute pdl_wait() (common.cuh) before touching anything the previous kernel
// writes.  Returns METIS_OK or METIS_E_CUDA.
// The _cluster form launches clusters of the given shape.
template <typename... KArgs, typename... Args>
int launch_dependent_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 cluster, dim3 block, size_t smem,
                             cudaStream_t st, const char* what, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster.x;
  attr[1].val.clusterDim.y = cluster.y;
  attr[1].val.clusterDim.z = cluster.z;
  cfg.attrs = attr;
  cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return METIS_OK;
}

template <typename... KArgs, typename... Args>
int launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const char* what,
                     Args... args) {
  return launch_dependent_cluster(kernel, grid, dim3(1, 1, 1), block, smem, st, what, args...);
}

// Raise a kernel's dynamic shared memory limit once per device.
int set_max_dynamic_smem(const void* func, int bytes, int* done_mask);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Partitions a split call launches: ceil(max_seq_len / partition_size), in 64
// bits (max_seq_len near INT_MAX must not overflow); 0 when unsplit.
inline size_t split_parts(int max_seq_len, int partition_size) {
  if (partition_size <= 0 || max_seq_len <= 0) return 0;
  return (size_t)(((long long)max_seq_len + partition_size - 1) / partition_size);
}

// The longest sequence a call can read: max_seq_len, clamped to what a
// block-table row addresses (max_blocks * block_size).  Partitions past it
// would only ever be empty, so they are neither launched nor given scratch.
inline int effective_max_len(int max_seq_len, int max_blocks, int block_size) {
  return (int)std::min<long long>((long long)max_blocks * block_size, (long long)max_seq_len);
}

// Log-sum-exp merge of split partials [S, H, max_parts, D] (decode.cu); with
// skip_single, sequences with at most one partition are left untouched.
int launch_merge_ex(const float* part_out, const float* part_lse, const int32_t* seq_lens, int P, void* out,
                    float* lse_out, int S, int H, int D, int max_parts, int out_dtype, int skip_single,
                    cudaStream_t st);
// The merge of the sequences with two or more partitions only (the others were
// written directly): one CTA per SM lists them and takes their rows in turn.
// Falls back to launch_merge_ex(..., skip_single = 1) outside its reach.
int launch_merge_split_rows(const float* part_out, const float* part_lse, const int32_t* seq_lens, int P, void* out,
                            float* lse_out, int S, int H, int D, int max_parts, int out_dtype, int sms,
                            cudaStream_t st);

// The single-token sequences of a chunked-prefill batch of T packed rows, persistent,
// beside the chunk kernel (decode.cu); rows = the batch's cu_q_lens.  One CTA per SM in a
// grid of `grid` CTAs, of which the first *n_ctas (device value, written by the prefill
// schedule kernel before this grid reads it) take (sequence, KV head) items from the counter
// *next_item (zeroed by that kernel); the others exit at once.  Every CTA lets the next grid
// launch only after waiting for the previous one.  window > 0: a query sees the last `window` and the
// first `sinks` tokens of its sequence.
int launch_decode_rows_beside(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                              const int32_t* seq_lens, const int32_t* rows, int T, void* out, float* lse_out, int S,
                              int H, int G, int D, int bs, int max_blocks, int num_blocks, float scale, int cap,
                              int window, int sinks, const int* n_ctas, int* next_item, int grid, cudaStream_t st);

// The same for an 8-bit cache (decode_fp8.cu).
struct Fp8Cache {
  const void* k_cache;  // e4m3 codes [num_blocks, bs, G, D]
  const void* v_cache;
  const uint8_t* k_scale;  // scale bytes [num_blocks, G]
  const uint8_t* v_scale;
};
int launch_decode_fp8_rows_beside(const void* q, const Fp8Cache& cache, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* rows, int T, void* out, float* lse_out, int S,
                                  int H, int G, int D, int bs, int max_blocks, int num_blocks, float scale, int cap,
                                  const int* n_ctas, int* next_item, int grid, cudaStream_t st);

// The sizes that a bf16 or fp32 decode takes (head ratios up to 8).  Returns METIS_OK or an error code.
inline int check_decode_sizes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                              int max_blocks, int num_blocks, int max_seq_len, float scale) {
  if (num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks <= 0 || num_blocks <= 0 ||
      max_seq_len <= 0)
    return fail(METIS_E_SHAPE, "sizes must be positive");
  if (num_heads % num_kv_heads) return fail(METIS_E_SHAPE, "num_heads %% num_kv_heads != 0");
  if (num_seqs > 65535 || num_kv_heads > 65535) return fail(METIS_E_SHAPE, "num_seqs and num_kv_heads must be <= 65535");
  if ((long long)max_blocks * block_size > 0x7fffffffLL || (long long)num_blocks * block_size > 0x7fffffffLL)
    return fail(METIS_E_SHAPE, "max_blocks * block_size and num_blocks * block_size must fit in int32");
  if (head_dim != 64 && head_dim != 128) return fail(METIS_E_UNSUPPORTED, "head_dim must be 64 or 128");
  if (block_size != 16 && block_size != 32 && block_size != 64)
    return fail(METIS_E_UNSUPPORTED, "block_size must be 16, 32 or 64");
  if (num_heads / num_kv_heads > 8) return fail(METIS_E_UNSUPPORTED, "num_heads / num_kv_heads must be <= 8");
  if (!(scale == scale)) return fail(METIS_E_SHAPE, "scale is NaN");
  return METIS_OK;
}

// Decodes whose sequences share their first tokens in groups (shared_prefix.cu): the call's arguments,
struct SharedArgs {
  const void *q, *k_cache, *v_cache;
  const int32_t *block_table, *seq_lens, *cu_group_seqs, *prefix_lens;
  void* out;
  float* lse_out;
  int S, num_groups, H, G, D, bs, max_blocks, num_blocks, cap;
  float scale;
};
// what the kernel over the shared prefixes leaves for those behind it -- of the groups,
struct SharedPlan {
  int2 total;           // K/V tiles of all units, CTAs that share them (0: none)
  int own_shares;           // of the sequences' own tokens: shares, at least 1 (0: not counted yet),
  unsigned int next_share;  // the next (share, KV head) to hand out
  int2 group[1];            // [num_groups]: units before the group, units per KV head
};
// of each sequence,
struct SharedOwn {
  int begin, group;  // its first token that is its own; its group (-1: every token is)
};
// and the launch of the first (prefill.cu), `sms` CTAs: a part is [2][128] rows; unit_parts: a unit's first and last.
int launch_shared_prefix(const SharedArgs& a, SharedPlan* plan, SharedOwn* own, int2* unit_parts, float* part_lse,
                         float* part_out, int sms, cudaStream_t st);

// Per-translation-unit device status words.
int decode_status(uint32_t* bits, int clear);
int prefill_status(uint32_t* bits, int clear);
int mla_status(uint32_t* bits, int clear);
int cache_status(uint32_t* bits, int clear);
int prefix_status(uint32_t* bits, int clear);
int fp8_status(uint32_t* bits, int clear);
int decode_fp8_status(uint32_t* bits, int clear);
int plan_status(uint32_t* bits, int clear);
int rope_status(uint32_t* bits, int clear);
int window_status(uint32_t* bits, int clear);
int shared_status(uint32_t* bits, int clear);

}  // namespace metis
