// Chunked prefill over a paged KV cache (prefix cache + causal chunk), on the
// 5th-generation tensor cores.
//
// The operation: vllm-metis 0.1.0 page, introduction and "How the model maps
// onto vLLM -> Caches" (prefix caching and chunked prefill on vLLM's attention
// kernels), with the chunk sizes of the vllm-mblt 0.8.0 page ("Chunked Prefill
// Auto-Tuning").  Sequence s holds seq_lens[s] cached tokens, the last
// q_len = cu_q_lens[s+1] - cu_q_lens[s] of which are queried; query i sits at
// position L - q_len + i and sees every key t <= L - q_len + i (the cached
// prefix plus a causal mask inside the chunk).  Single-token decodes are the
// q_len = 1 case: with a head ratio up to 8 the entry point hands them to the
// decode kernel (memory-bound, 16-token page units per warp) and lists no tiles
// for them here; above 8 they run through the same tiles.
//
// Tiling.  A query tile is 128 rows of one KV head's group: the r = H/G query
// heads times 128/r consecutive query tokens (GQA packing).  One CTA per SM
// computes TWO consecutive query tiles of the same sequence and group against
// each 128-token K/V tile, so every K/V byte gathered (page by page, with TMA,
// 128-byte swizzle) feeds 256 query rows.
//
//   warps 0..3   softmax of query tile 0, one row (TMEM lane) per thread
//   warps 4..7   softmax of query tile 1
//   warps 8..11  TMA producers: K tiles (warps 8, 9) and V tiles (warps 10, 11)
//                into 3- and 2-stage rings, each tile's pages
//                split between two warps (16-token pages make many small boxes,
//                and one warp alone cannot issue them fast enough)
//   warp 13      query loader; warp 14 hands out the units; warp 15 idle but with
//                windows (the last warpgroup gives up registers to the softmax groups)
//   warp 12      allocates TMEM (S0 | S1 | O0 | O1, 512 columns); one lane
//                issues the UMMAs in the order
//                  PV0_j, QK0_{j+1}, PV1_j, QK1_{j+1}
//                so that while one softmax group works the tensor pipe runs the
//                other group's products (ping-pong).
//                  S_w = Q_w K_j^T  (M 128, N 128, K = head_dim)
//                  O_w += P_w V_j   (M 128, N head_dim, K 128; P_w read from TMEM)
// Registers: the producer and UMMA warpgroups drop to kRegsProd / kRegsMma so that each
// softmax thread holds its row's 128 scores at once (one TMEM read per tile).
// Softmax: running max in log2 units, P = exp2(S - m) written back as bf16
// pairs over its own S columns; O is rescaled in TMEM only when the max grows
// by more than 2^8.  Because QK_w_{j+1} is issued after PV_w_j, "S_w_j landed"
// already implies "PV_w_{j-1} finished", so the rescale never waits.
//
// Persistent mixed batch: a small schedule kernel lists the (sequence,
// query-tile pair) items heaviest first -- the chunks of every length in one
// list -- and one CTA per SM takes units (item, KV head) from that list as it
// goes (warp 14 claims the next one with an atomic once every warp has taken the
// current one, and publishes it with its derived fields to the other warps through
// a two-slot ring).  Every role keeps its ring and barrier counters
// running across units, so the next unit's queries (warp 13, once the current
// unit's last QK has completed) and K/V tiles stream in while the current unit's
// last softmax, PV and epilogue drain.
//
// 8-bit cache (e4m3 codes with a power-of-two scale per page and KV head; the KV8 variant).
// K codes feed the tensor cores as they are (kind::f8f6f4, twice the bf16 rate): the
// softmax threads split their query row, scaled by a power of two, into two e4m3 parts,
// S = (hi + lo) codes^T, so that QK costs what it costs in bf16 at half of K's bytes.  A K
// page's scale joins the softmax factor of its 16 tokens.  V's codes are staged by TMA and
// become bf16 rows, scale included (exact), by four warps.  P is bf16 with it: the operands of
// one UMMA are of one type, and V times its scale needs bf16's range.  Its 2^-8 per weight
// puts the rows' error against float64 at 2.3e-3, 1.7e-3 with weights of fp32.  2,048 queries over
// 16,384 tokens, 32/8 heads of 128, take 420-435 us = 1,185-1,230 TFLOP/s (bf16 kernel 460 us);
// 16 chunks of 512 behind up to 4,096 tokens 258 us (247).  What bounds it: a K/V-tile pair
// takes 2,930 cycles, of which the tensor work is 2,054, and shared memory's port is busy for
// 2,176 (QK's and PV's operands, V's conversion, the TMA writes); the rest are the hand-offs
// between softmax, converters and issuer (without V's conversion 3 % less).  On the way
// there: K converted to bf16 as well 2,154 us for the first; codes into the UMMAs and V
// converted by three warps 528 us; the issuer's operands uniform over its warp, queries
// split by the softmax threads and a fourth converter 431 us.  Few chunks: units are split
// over their keys (SPLIT, at kMaxSplits).
//
// Windows (WINDOW).  A unit's keys are a row of whole pages, those of the first tokens and then those
// from its first query's oldest key on (PfSpan); tiles, positions and masks count along it, so first tokens
// cost a page and not a tile (16 chunks of 512 and 48 decodes, window of 1,024: 255 us, 224 so).  A hidden key's weight is
// 0, but 0 times an infinity or NaN is not: warp 15 looks at the V rows that some query of the unit does
// not see, once they have landed.  Hidden keys are masked in pieces of 32 columns, and only in those that the
// edges cross; rows are written in 32-byte stores; the issuer is the uniform one of the 8-bit cache.  Measured there:
// 224 us, uniform issuer 192, masks, V rows in batches and stores 165 (779 TFLOP/s of the visible keys: units of nine
// tiles, whose queries, first products and epilogue cost as much as three); 2,048 queries, window of 4,096,
// 175, 126, 120 us (1,162 TFLOP/s: 256 units on 152 SMs); 8,192 queries 556, 412, 380 us (1,450 TFLOP/s).
//
// Shared prefixes (SHARED): at PfGroup and in shared_split.cuh.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "../../include/metis_attn.h"
#include "common.cuh"
#include "decode.cuh"
#include "fp8.cuh"
#include "host.h"
#include "shared_split.cuh"
#include "tcgen05.cuh"

namespace metis {

__device__ unsigned int g_status_prefill = 0;

constexpr int kPfThreads = 512;   // 2 softmax groups + 4 TMA warps + MMA warp + 3 idle warps
constexpr int kMmaWarp = 12;
constexpr int kUnitReaders = 14;  // warps 0..13 read every unit from the unit ring (8-bit cache: and warp 15)
constexpr int kRegsLaunch = 65536 / kPfThreads;  // 128: the block takes the whole register file
#ifndef PF_REGS_SOFTMAX
#define PF_REGS_SOFTMAX 216
#define PF_REGS_PROD 40
#define PF_REGS_MMA 40
#endif
constexpr int kRegsSoftmax = PF_REGS_SOFTMAX;  // warpgroups 0, 1: softmax
constexpr int kRegsProd = PF_REGS_PROD;        // warpgroup 2: K/V producers
constexpr int kRegsMma = PF_REGS_MMA;          // warpgroup 3: UMMA issuer, query loader, idle warps
static_assert(128 * (2 * kRegsSoftmax + kRegsProd + kRegsMma) <= kPfThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
// windows, shared prefixes: the issuer's uniform loop needs a few more
constexpr int kRegsSoftmaxU = 208;
constexpr int kRegsMmaU = 56;
static_assert(128 * (2 * kRegsSoftmaxU + kRegsProd + kRegsMmaU) <= kPfThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
// 8-bit cache: the converters in the last two warpgroups need more
constexpr int kRegsSoftmax8 = 200;
constexpr int kRegsOther8 = 56;
static_assert(128 * (2 * kRegsSoftmax8 + 2 * kRegsOther8) <= kPfThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
#ifndef METIS_PF_K_STAGES
#define METIS_PF_K_STAGES 3
#define METIS_PF_V_STAGES 2
#endif
constexpr int kKStages = METIS_PF_K_STAGES;  // K ring depth
constexpr int kVStages = METIS_PF_V_STAGES;  // V ring depth
constexpr int kV8Stages = 3;      // 8-bit cache: staged e4m3 V tiles
constexpr int kKvTile = 128;      // tokens per K/V tile
constexpr int kRows = 128;        // query rows per tile
constexpr int kTmemCols = 512;    // S0 | S1 | O0 | O1
constexpr int kSortMax = 2048;    // schedule: heaviest-first sort up to this many items
// 8-bit cache, few chunks: parts of a unit at most, K/V tiles of each at least, and of the whole
// unit (a tile takes 1.5 us).  64 units, 512 queries at 32/8 heads: behind 1,024 tokens (9 tiles
// and more) 37 us in parts and 34 whole, behind 2,048 43.7 and 47.7, behind 8,192 84.6 and 126.9,
// behind 32,768 264 and 476.  32 units behind 16,384: 85 and 232.  192, 40 of them behind a whole
// round, behind 8,192: 196 and 257.
constexpr int kMaxSplits = 8;
constexpr int kMinPartTiles = 4;
constexpr int kMinSplitTiles = 13;

struct PrefillParams {
  const int32_t* cu_q_lens;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  float* lse_out;
  const int4* items;
  const int* item_count;
  int* unit_head;   // next unit to hand out (the schedule kernel zeroes it)
  int S, T, H, G, r, Tq, bs, max_blocks, num_blocks, cap;
  float scale_log2;
  int skip_decodes;  // single-token sequences are served by the decode kernel: list no tiles for them
  // Decodes beside the chunk kernel (dec_ctas != NULL): the schedule kernel writes the
  // number of SMs the decode kernel keeps (*dec_ctas) and zeroes its item counter
  // (*dec_next); this kernel then launches behind that decode kernel, which lets it
  // launch only once its CTAs have waited for the schedule, so the list is ready at
  // launch: no wait at the start, the wait for the decode grid just before exiting.
  int* dec_ctas;
  int* dec_next;
  int num_sms, D;
  int kv_token_bytes;  // K and V of one cached token, every KV head
  int wait_at_exit;
  // window > 0: a query at position p sees the keys t <= p with t > p - window or t < sinks
  int window, sinks;
  const void *q, *k_cache, *v_cache;  // (window only: the rows behind the tensor maps)
  Fp8Cache fp8;  // an 8-bit cache (k_cache NULL: bf16)
  // 8-bit cache, splits != NULL: the units of a last round that leaves SMs idle are split
  // over their keys.  The schedule kernel writes {how often, how many units stay whole} and
  // zeroes the counters of finished parts.
  int2* splits;
  int max_parts;    // memory for this many parts
  int* parts_done;  // [split unit][query tile][warp]
  float* part_lse;  // [part][query tile][row], log2 units
  float* part_out;  // [part][query tile][head_dim / 4][row][4], normalised (shared prefixes: [head_dim])
  // Shared prefixes: the groups (cu_q_lens: their first sequences), their shared tokens, and what the
  // kernel behind this one needs to find a row's parts.
  const int32_t* prefix_lens;
  SharedPlan* plan;
  SharedOwn* own;
  int2* unit_parts;
  int num_groups;
};

// Shared-memory layout (all tiles 128-byte swizzled, [64-column half][row][128 B]).
template <int D, bool KV8>
struct PfShape {
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = kRows * 128;                   // 128 query rows x 64 bf16
  static constexpr int kQBytes = kHalves * kQHalf;             // one query tile
  static constexpr int kKvHalf = kKvTile * 128;                // 128 tokens x 64 bf16
  static constexpr int kKvBytes = kHalves * kKvHalf;
  // 8-bit cache: K tiles stay e4m3 (rows of D bytes), a query tile is its two e4m3 parts
  // (the same bytes as bf16), V tiles are converted from staged e4m3 tiles
  static constexpr int kQPart = kRows * D;
  static constexpr int kKBytes = KV8 ? kKvTile * D : kKvBytes;
  static constexpr int kQ = 0;                                 // 2 query tiles
  static constexpr int kK = kQ + 2 * kQBytes;                  // kKStages stages
  static constexpr int kV = kK + kKStages * kKBytes;           // kVStages stages
  static constexpr int kStage = kV + kVStages * kKvBytes;      // kV8Stages staged e4m3 tiles of V
  static constexpr int kTiles = kStage + (KV8 ? kV8Stages * kKvTile * D : 0);  // bf16: 224 KB at head_dim 128
  // + 1 KB: the barriers live in the alignment slack (below the aligned base when it
  // is at least 256 B, else just past the tiles).  At least 120 KB so that one CTA
  // (all 512 TMEM columns) is resident per SM.
  static constexpr int kSmem = (kTiles + 1024) > 120 * 1024 ? (kTiles + 1024) : 120 * 1024;
};

// 8-bit cache, roles of the warps that differ: warp 8 loads K tiles and stages V tiles
// (TMA), warps 9..11 and 15 convert staged V tiles to bf16 (none on the UMMA issuer's
// scheduler: one there cost 4 %), warp 13 loads the bf16 query rows and the softmax groups
// split them.
constexpr int kV8Converters = 4;
constexpr int kKScaleSlots = 4;  // tiles whose K factors are kept
// Units whose NaN notes are kept.  Unit k is published once every warp has taken unit k - 1,
// which a softmax group does after it has written out unit k - 3: its notes may be cleared.
constexpr int kNanUnits = 3;

struct PfFp8Shared {
  uint64_t stage_full[kV8Stages];   // staged V tile landed
  uint64_t stage_empty[kV8Stages];  // every converter has read it
  uint64_t q_raw[2];                // bf16 rows of a query tile landed
  uint64_t q_full[2];               // ... split into their two e4m3 parts (4 warps)
  float4 ks[kKScaleSlots][2];       // per 16 tokens of a K tile: its page's scale
  float vs[kV8Stages][8];           // ... of a staged V tile
  // NaN in V rows that only some of a unit's query rows see: kept out of the V tile, where
  // 0 * NaN would reach every row, and put into the output columns of the rows that see them
  int nan_any[kNanUnits];
  uint16_t nan_first[kNanUnits][128];  // per column: the first such token behind the unit's first query
  int tag[kNanUnits];                  // the unit's PfUnit8::tag
};

// The converters' rare case: one row's 16 codes from column `col` on, or their scale, hold
// NaN; the codes become zeros (returned) and their columns are noted.
__device__ __forceinline__ uint4 note_nan_codes(uint4 c, bool scale_nan, uint16_t* first, int* any, uint16_t rel) {
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll 1
    for (int b = 0; b < 4; ++b)
      if (scale_nan || ((w[i] >> (8 * b)) & 0x7fu) == 0x7fu) {
        w[i] &= ~(0xffu << (8 * b));
        uint16_t* at = first + 4 * i + b;
        uint16_t seen = *reinterpret_cast<volatile uint16_t*>(at);
        while (rel < seen) {  // each turn that another lane wins lowers `seen`
          const uint16_t was = atomicCAS(at, seen, rel);
          if (was == seen) break;
          seen = was;
        }
      }
  }
  *reinterpret_cast<volatile int*>(any) = 1;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Any NaN (0x7f, 0xff) among 16 codes
__device__ __forceinline__ bool any_nan_code(const uint4& c) {
  return ((((c.x & 0x7f7f7f7fu) + 0x01010101u) | ((c.y & 0x7f7f7f7fu) + 0x01010101u) |
           ((c.z & 0x7f7f7f7fu) + 0x01010101u) | ((c.w & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u) != 0;
}

// Windows: V rows that hold an infinity or NaN and that only some of a unit's query rows see.  They
// are kept out of the V tile, where 0 * NaN would reach every row; the rows that see them add them
// in the epilogue.  A bit for each of the 2 x `span` tokens that may be such (span: the unit's query
// tokens): first those that leave the window of some of them, then those behind the first query.
constexpr int kOddWords = 4 * kRows / 32;  // span <= 2 x 128
struct PfWindowShared {
  uint64_t v_ready[kVStages];  // the tile's rows that not every query sees have been looked at
  uint32_t odd[2][kOddWords];  // of the unit in hand and the one before
  int any_odd[2];
};

// mbarrier layout (indices into the barrier area) and arrival counts
struct PfBar {
  static constexpr int kQFull = 0, kKFull = 1, kKEmpty = kKFull + kKStages, kVFull = kKEmpty + kKStages,
                       kVEmpty = kVFull + kVStages, kSFull = kVEmpty + kVStages, kPFull = kSFull + 2,
                       kPvDone = kPFull + 2, kDrain = kPvDone + 2, kQFree = kDrain + 1, kUnitFull = kQFree + 1,
                       kUnitEmpty = kUnitFull + 2, kCount = kUnitEmpty + 2;
  // full barriers: one arrival per producer warp of the ring; p_full: 128 softmax threads
  __host__ __device__ static constexpr int arrivals(int i, bool kv8, bool window) {
    return (i >= kPFull && i < kPFull + 2) ? 128
           : (i >= kKFull && i < kKFull + kKStages) ? (kv8 ? 1 : 2)
           : (i >= kVFull && i < kVFull + kVStages) ? (kv8 ? kV8Converters : 2)
           : (i >= kVEmpty && i < kVEmpty + kVStages) ? (window ? 2 : 1)
           : (i >= kUnitEmpty && i < kUnitEmpty + 2) ? kUnitReaders + (kv8 || window ? 1 : 0)
                                                      : 1;
  }
};
static_assert((PfBar::kCount + 4) * 8 <= 256, "prefill barrier area");

// Shared prefixes.  A group's members are the query rows of its prefix: q_len members, L shared tokens, no
// causal mask, the pages those of the first member that is at least as long.  A unit is (group, KV head,
// pair of query tiles); all units' K/V tiles in a row are cut into equal shares, one per CTA, and
// what a CTA computes of a unit is a part, number (index of the unit) + (index of the CTA): both
// grow along the row, and one of them from each part to the next.
struct PfGroup {
  int q0, n;           // first member, members
  int leader, tokens;  // the sequence whose pages are read (~s: not among those in front of s), shared tokens
  int tiles, units;    // K/V tiles of a unit, units (0: nothing shared)
};

// A group's first members that are shorter than its prefix (a padded batch's rows): a thread looks at this many
// itself, the warp at the others, so that many of them do not cost a load in series each.  (20,000 empty rows in front of
// 64 members: 1,480 us by threads alone, 221 so, 88 with none in front.)
constexpr int kLeaderLook = 8;

// *bad: status bits; *decreases: the group's offsets do.  The leader may be left open (pf_lead, pf_lead_all).
__device__ __forceinline__ PfGroup pf_group(const PrefillParams& p, int g, unsigned* bad, bool* decreases) {
  PfGroup v{};
  const int a = p.cu_q_lens[g], b = p.cu_q_lens[g + 1], tokens = p.prefix_lens[g];
  *decreases = a > b;
  if (a < 0 || b > p.S || a > b) {
    *bad |= METIS_STATUS_BAD_OFFSETS;
    return v;
  }
  if (tokens < 0) *bad |= METIS_STATUS_BAD_Q_LEN;
  if (tokens <= 0 || tokens > p.cap) {
    if (tokens > p.cap && b > a) *bad |= METIS_STATUS_SEQ_TOO_LONG;
    return v;
  }
  const int near = b - a > kLeaderLook ? a + kLeaderLook : b;
  int s = a;
  while (s < near && p.seq_lens[s] < tokens) ++s;
  if (s == b) return v;
  v.q0 = a;
  v.n = b - a;
  v.leader = s < near ? s : ~s;
  v.tokens = tokens;
  v.tiles = (tokens - 1) / kKvTile + 1;
  v.units = ((v.n - 1) / (2 * p.Tq) + 1) * p.G;
  return v;
}

// The first of the sequences [from, end) with at least `tokens` tokens (-1: none), by a warp.
__device__ __forceinline__ int pf_first_member(const int32_t* seq_lens, int from, int end, int tokens) {
#pragma unroll 1
  for (int s0 = from; s0 < end; s0 += 32) {
    const int s = s0 + (threadIdx.x & 31);
    const uint32_t votes = __ballot_sync(0xffffffffu, s < end && seq_lens[s] >= tokens);
    if (votes) return s0 + __ffs(votes) - 1;
  }
  return -1;
}

// The group's leader, if it is open still; without one nothing is shared.  By a warp, all of it with the same group.
__device__ __forceinline__ void pf_lead(const PrefillParams& p, PfGroup& v) {
  if (v.units == 0 || v.leader >= 0) return;
  v.leader = pf_first_member(p.seq_lens, ~v.leader, v.q0 + v.n, v.tokens);
  if (v.leader < 0) v = PfGroup{};
}

// The leaders of the lanes' groups, by the warp.
__device__ __forceinline__ void pf_lead_all(const PrefillParams& p, PfGroup& v) {
#pragma unroll 1
  for (uint32_t open = __ballot_sync(0xffffffffu, v.units > 0 && v.leader < 0); open; open &= open - 1) {
    const int src = __ffs(open) - 1;
    const int s = pf_first_member(p.seq_lens, ~__shfl_sync(0xffffffffu, v.leader, src),
                                  __shfl_sync(0xffffffffu, v.q0 + v.n, src), __shfl_sync(0xffffffffu, v.tokens, src));
    if ((int)(threadIdx.x & 31) == src) {
      v.leader = s;
      if (s < 0) v = PfGroup{};
    }
  }
}

// Effective (sequence length, query count) after clamping to what can be read.  `flag`: report
// what had to be clamped (the schedule kernel, which sees every sequence once).
__device__ __forceinline__ void pf_lengths(const PrefillParams& p, int s, int& L, int& q_len, bool flag) {
  L = p.seq_lens[s];
  const int r0 = p.cu_q_lens[s], r1 = p.cu_q_lens[s + 1];
  if (r0 < 0 || r1 < 0 || r0 > p.T || r1 > p.T) {  // rows outside the batch's: the sequence is left out
    if (flag) atomicOr(&g_status_prefill, METIS_STATUS_BAD_OFFSETS);
    L = q_len = 0;
    return;
  }
  q_len = r1 - r0;
  if (L > p.cap) {
    if (flag && q_len != 0) atomicOr(&g_status_prefill, METIS_STATUS_SEQ_TOO_LONG);
    L = p.cap;
  }
  if (L < 0) L = 0;
  if (q_len > L || q_len < 0) {
    if (flag) atomicOr(&g_status_prefill, METIS_STATUS_BAD_Q_LEN);
    q_len = q_len < 0 ? 0 : L;
  }
}

// K/V tiles a query tile needs: keys up to the position of its last valid query.
__device__ __forceinline__ int pf_kv_tiles(int L, int q_len, int tile, int Tq) {
  const int qi0 = tile * Tq;
  if (qi0 >= q_len) return 0;
  const int p_max = L - q_len + min(q_len - 1, qi0 + Tq - 1);
  return (p_max + kKvTile) / kKvTile;
}

// Windows: what the queries of a query-tile pair see of a sequence, in whole pages: the pages of the first
// tokens, then those from the first query's oldest key on.  Their tokens in a row are the unit's keys; its
// K/V tiles, lengths and positions count along that row, in which the pages in between do not exist.
struct PfSpan {
  int low, skip;  // pages of first tokens, pages left out behind them (none left out: low = skip = 0)
  int sinks;      // the row's first tokens that every query sees
};
__device__ __forceinline__ PfSpan pf_span(const PrefillParams& p, int L, int q_len, int pair) {
  const int oldest = max(L - q_len + 2 * pair * p.Tq - p.window + 1, 0);
  const int ns = min(p.sinks, oldest), low = ns / p.bs + (ns % p.bs != 0), recent = oldest / p.bs;
  PfSpan w{0, 0, p.sinks};
  if (low < recent) w = PfSpan{low, recent - low, ns};
  return w;
}

// Keys seen by the q_len last queries of L tokens, summed, when each sees `most` at most.
__device__ __forceinline__ long long pf_pairs(int L, int q_len, long long most) {
  const long long free = min(max(most - (L - q_len), 0ll), (long long)q_len);  // queries that see all before them
  return free * (L - q_len) + free * (free + 1) / 2 + (q_len - free) * most;
}

// ---------------------------------------------------------------------------
// schedule: the (sequence, query-tile pair) work list, heaviest first
// ---------------------------------------------------------------------------
constexpr int kSchedThreads = 1024;
// One SM's rates, for sizing the decodes' share of SMs beside the chunks: decode
// K/V bytes per second while the chunks run (a CTA of two 4-warp groups, each warp
// a 3-stage ring: ~192 KB in flight; timestamps on a GB300 show 453 MB of decodes
// taking ~253 us on 24 SMs beside 16 chunks of 512, i.e. ~75 GB/s per SM.  Too few
// decode SMs, so that the decodes finish last, costs far more than a few too many),
// and the chunk kernel's FLOP/s (the chunks alone reach ~1.07-1.13 PFLOP/s on 152 SMs;
// with 7 TFLOP/s per SM the mixed batch above ends its decodes and chunks together).
constexpr float kDecSmBytesPerS = 75e9f;
constexpr float kChunkSmFlopsPerS = 7.0e12f;
// The same two over an 8-bit cache (rates between 40 and 46 GB/s change the mixed batch above by
// 1 %; 58 GB/s, which leaves the decodes too few SMs, costs 15 %)
constexpr float kDec8SmBytesPerS = 43e9f;
constexpr float kChunk8SmFlopsPerS = 7.0e12f;

// How often to split each unit of the last round, units % sms of them on `sms` SMs with up to
// `tiles` K/V tiles each: the least time, in tiles.  Parts cost two on top in a round of their
// own and nine for each round that begins behind another (the next unit is claimed, and its
// queries fetched, when the last one's QK is done).
__host__ __device__ inline int pf_splits(long long units, int sms, int tiles, int max_parts) {
  const int rest = (int)(units % sms);
  if (tiles < kMinSplitTiles || rest == 0) return 1;
  int best = 1, cost = tiles;
  for (int n = 2; n <= kMaxSplits && rest * n <= max_parts; ++n) {
    const int len = (tiles + n - 1) / n, rounds = (rest * n + sms - 1) / sms;
    if (len < kMinPartTiles) break;
    const int c = rounds * len + 2 + 9 * (rounds - 1) + (units > rest ? 9 : 0);
    if (c < cost) {
      cost = c;
      best = n;
    }
  }
  return best;
}

__global__ void __launch_bounds__(kSchedThreads) prefill_schedule_kernel(const PrefillParams p, int4* items,
                                                                          int* count, int max_items) {
  __shared__ int warp_sums[32];
  __shared__ int4 buf[kSortMax];
  pdl_launch_dependents();  // the attention kernel may start launching (it waits for the items)
  pdl_wait();  // a programmatic dependent itself: inputs are read once the previous grid completed
  const int tid = threadIdx.x;
  const int per = (p.S + kSchedThreads - 1) / kSchedThreads;
  const int s0 = min(p.S, tid * per), s1 = min(p.S, s0 + per);
  const int pair_tokens = 2 * p.Tq;
  int local = 0;
  // decode tokens read; (query, key) pairs of the chunks.  Integers and a float ratio:
  // this GPU's fp64 rate is a small fraction of its fp32 rate.
  long long dec_tok = 0, chunk_qk = 0;
  int L_first = 0, q_first = 0;  // this thread's first sequence, kept for the listing pass
  bool routed_first = false;
  for (int s = s0; s < s1; ++s) {
    int L, q_len;
    const bool routed = p.skip_decodes && single_row(p.cu_q_lens, p.T, s) >= 0;
    pf_lengths(p, s, L, q_len, true);
    if (s == s0) {
      L_first = L;
      q_first = q_len;
      routed_first = routed;
    }
    if (!routed) {
      local += (q_len + pair_tokens - 1) / pair_tokens;
      chunk_qk += p.window ? pf_pairs(L, q_len, (long long)p.window + p.sinks)
                           : (long long)q_len * (L - q_len) + (long long)q_len * (q_len + 1) / 2;
    } else {
      dec_tok += p.window ? min((long long)L, (long long)p.window + p.sinks) : L;
    }
  }
  // The decodes' share of SMs, from warp sums published before the scan's barriers
  // and combined by the last warp (no sequences there unless S > 992): off the path
  // of the listing and the sort.
  __shared__ long long red[2][kSchedThreads / 32];
  __shared__ int dec_share, longest;
  static_assert(kSchedThreads == 32 * 32, "one warp combines the warp sums");
  const int lane = tid & 31, warp = tid >> 5;
  if (p.dec_ctas) {
    for (int o = 16; o > 0; o >>= 1) {
      dec_tok += __shfl_xor_sync(0xffffffffu, dec_tok, o);
      chunk_qk += __shfl_xor_sync(0xffffffffu, chunk_qk, o);
    }
    if (lane == 0) {
      red[0][warp] = dec_tok;
      red[1][warp] = chunk_qk;
    }
  }
  int all;
  int pos = block_exclusive_scan<kSchedThreads>(local, warp_sums, &all);
  if (p.dec_ctas && warp == kSchedThreads / 32 - 1) {
    // SMs for the decodes beside the chunks: decodes on k SMs and chunks on the
    // other N - k finish together when k / N = d / (d + c), with d and c the SM time
    // each kind needs alone (rates of one SM: kDecSmBytesPerS, kChunkSmFlopsPerS): K and V
    // rows of every decode, QK^T and PV of every chunk query
    long long dt = red[0][lane], cq = red[1][lane];
    for (int o = 16; o > 0; o >>= 1) {
      dt += __shfl_xor_sync(0xffffffffu, dt, o);
      cq += __shfl_xor_sync(0xffffffffu, cq, o);
    }
    if (lane == 0) {
      const bool kv8 = p.fp8.k_cache != nullptr;
      const float d = (float)dt * ((float)p.kv_token_bytes / (kv8 ? kDec8SmBytesPerS : kDecSmBytesPerS));  // K, V rows
      const float c = (float)cq * ((float)p.H * p.D * 4.0f / (kv8 ? kChunk8SmFlopsPerS : kChunkSmFlopsPerS));
      int k = 0;
      if (dt > 0) k = cq > 0 ? (int)ceilf(p.num_sms * (d / (d + c))) : p.num_sms;
      *p.dec_ctas = dec_share = min(max(k, dt > 0 ? 1 : 0), p.num_sms);
      *p.dec_next = 0;
    }
  }
  const int total = min(max(all, 0), max_items);
  const bool sort = total <= kSortMax;
  if (p.splits) {
    if (tid == 0) longest = 0;
    __syncthreads();
  }
  for (int s = s0; s < s1; ++s) {
    int L = L_first, q_len = q_first;
    bool routed = routed_first;
    if (s != s0) {
      pf_lengths(p, s, L, q_len, false);
      routed = p.skip_decodes && single_row(p.cu_q_lens, p.T, s) >= 0;
    }
    const int np = routed ? 0 : (q_len + pair_tokens - 1) / pair_tokens;
    for (int t = 0; t < np; ++t, ++pos) {
      if ((unsigned)pos >= (unsigned)total) break;  // (offsets that decrease may list more than fits)
      int work = pf_kv_tiles(L, q_len, 2 * t, p.Tq) + pf_kv_tiles(L, q_len, 2 * t + 1, p.Tq);
      if (p.window) {
        const int row = L - pf_span(p, L, q_len, t).skip * p.bs;
        work = pf_kv_tiles(row, q_len, 2 * t, p.Tq) + pf_kv_tiles(row, q_len, 2 * t + 1, p.Tq);
      }
      const int4 it = make_int4(s, t, work, 0);
      if (p.splits) atomicMax(&longest, pf_kv_tiles(L, q_len, 2 * t, p.Tq));
      if (sort)
        buf[pos] = it;
      else
        items[pos] = it;
    }
  }
  if (sort) {
    // rank = number of items heavier than this one (ties: earlier in the list first);
    // `ways` threads (a power of two, within a warp) count a share of the list each
    __syncthreads();
    int ways = 1;
    while (ways < 32 && total * ways * 2 <= kSchedThreads) ways *= 2;
    const int sub = tid & (ways - 1);
    for (int base = 0; base < total; base += kSchedThreads / ways) {  // the same trip count in every thread
      const int i = base + tid / ways;
      const bool live = i < total;
      int4 me = make_int4(0, 0, 0, 0);
      int rank = 0;
      if (live) {
        me = buf[i];
        for (int k = sub; k < total; k += ways) {
          const int w = buf[k].z;
          rank += (w > me.z) || (w == me.z && k < i);
        }
      }
      for (int o = ways >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (live && sub == 0) items[rank] = me;
    }
  }
  if (p.splits) {
    __syncthreads();  // the decodes' share and the longest unit are known
    const int units = total * p.G, sms = max(p.num_sms - (p.dec_ctas ? dec_share : 0), 1);
    const int rest = units % sms, n = pf_splits(units, sms, longest, p.max_parts);
    if (tid == 0) *p.splits = make_int2(n, n > 1 ? units - rest : units);
    if (n > 1)
      for (int i = tid; i < rest * 2 * (kRows / 32); i += kSchedThreads) p.parts_done[i] = 0;
  }
  if (tid == 0) {
    *count = total;
    *p.unit_head = 0;
  }
}

// ---------------------------------------------------------------------------
// main kernel (persistent: one CTA per SM walks the work list)
// ---------------------------------------------------------------------------
// One unit of work as every role sees it: query-tile pair `pair` of sequence s,
// KV head g.  Each role derives it from the schedule's list on its own.
struct PfUnit {
  int s, pair, g, L, q_len, n0, n1, n_kv, q0, n_pages;
};

// 8-bit cache: a unit may be one of `parts` parts of the pair's K/V tiles, [j0, j0 + n_kv).
struct PfUnit8 : PfUnit {
  int j0;
  int tag;  // 0: all of them, else index among the split units << 8 | parts << 4 | part
};

// Windows: L, n_pages and the tiles are those of the unit's row of keys.
struct PfUnitW : PfUnit {
  PfSpan w;
  int a0, a1, b0;  // tiles [a0, a1) and from b0 on hold keys that some query of the unit does not see
};

// Shared prefixes: tiles [j0, j0 + n_kv) of the unit, part number `part`.
struct PfUnitS : PfUnit {
  int j0, part;
};

// The K/V tile that the unit visits j-th
__device__ __forceinline__ int pf_tile(const PfUnit&, int j) { return j; }

__device__ __forceinline__ int pf_tile(const PfUnitS& it, int j) { return it.j0 + j; }

// The unit's first K/V tile
__device__ __forceinline__ int pf_first(const PfUnit&) { return 0; }
__device__ __forceinline__ int pf_first(const PfUnit8& it) { return it.j0; }

__device__ __forceinline__ bool pf_unit(const PrefillParams& p, int u, PfUnit& it) {
  const int item_idx = u / p.G;
  it.g = u - item_idx * p.G;
  const int4 v = __ldcg(p.items + item_idx);  // written by this call's schedule kernel: read from L2
  it.s = v.x;
  it.pair = v.y;
  pf_lengths(p, it.s, it.L, it.q_len, false);
  it.n0 = pf_kv_tiles(it.L, it.q_len, 2 * it.pair, p.Tq);      // K/V tiles of query tile 0
  it.n1 = pf_kv_tiles(it.L, it.q_len, 2 * it.pair + 1, p.Tq);  // ... of query tile 1 (0: no second tile)
  it.n_kv = max(it.n0, it.n1);
  it.q0 = p.cu_q_lens[it.s];
  it.n_pages = (it.L + p.bs - 1) / p.bs;
  return it.n0 > 0;
}

__device__ __forceinline__ bool pf_unit(const PrefillParams& p, int u, PfUnitW& it) {
  PfUnit& plain = it;
  if (!pf_unit(p, u, plain)) return false;
  it.w = pf_span(p, it.L, it.q_len, it.pair);
  it.L -= it.w.skip * p.bs;
  it.n_pages -= it.w.skip;
  it.n0 = pf_kv_tiles(it.L, it.q_len, 2 * it.pair, p.Tq);
  it.n1 = pf_kv_tiles(it.L, it.q_len, 2 * it.pair + 1, p.Tq);
  it.n_kv = max(it.n0, it.n1);
  const int first = it.L - it.q_len + 2 * it.pair * p.Tq;
  const int last = it.L - it.q_len + min(it.q_len, (2 * it.pair + 2) * p.Tq) - 1;
  it.a0 = it.w.sinks / kKvTile;
  it.a1 = last >= p.window ? (last - p.window) / kKvTile + 1 : 0;
  it.b0 = (first + 1) / kKvTile;
  return true;
}

// Positions of a unit's first and last query
__device__ __forceinline__ int pf_first_query(const PrefillParams& p, const PfUnit& it) {
  return it.L - it.q_len + 2 * it.pair * p.Tq;
}
__device__ __forceinline__ int pf_last_query(const PrefillParams& p, const PfUnit& it) {
  return it.L - it.q_len + min(it.q_len, (2 * it.pair + 2) * p.Tq) - 1;
}

// Windows: does the unit's K/V tile j hold keys that some of its queries do not see?
__device__ __forceinline__ bool pf_partial(const PfUnitW& it, int j) { return (j >= it.a0 && j < it.a1) || j >= it.b0; }

// Any infinity or NaN among eight bf16
__device__ __forceinline__ bool any_nonfinite_bf16(const uint4& v) {
  return ((((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
           ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u)) & 0x80008000u) != 0;
}

// Windows: rows [r0, r1) of a V tile become zeros, by one warp.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int r1, int lane) {
  constexpr int CPR = D / 8;  // 16-byte pieces of a row
  for (int i = r0 * CPR + lane; i < r1 * CPR; i += 32) {
    const int row = i / CPR, piece = i % CPR;
    *reinterpret_cast<uint4*>(tile + (piece / 8) * (kKvTile * 128) + row * 128 + (piece % 8) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

// ... and of rows [r0, r1) those that hold an infinity or NaN do; note(row) for each.
template <int D, typename Note>
__device__ __forceinline__ void look_at_rows(uint8_t* tile, int r0, int r1, int lane, Note note) {
  constexpr int CPR = D / 8, RPS = 32 / CPR;  // rows per step
  constexpr int kSteps = 8;                   // loads in flight
  const int piece = lane % CPR;
  uint8_t* at = tile + (piece / 8) * (kKvTile * 128) + (piece % 8) * 16;
#pragma unroll 1
  for (int row0 = r0 + lane / CPR; row0 - lane / CPR < r1; row0 += kSteps * RPS) {
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (row0 + i * RPS < r1 && any_nonfinite_bf16(*reinterpret_cast<const uint4*>(at + (row0 + i * RPS) * 128))) odd |= 1u << i;
    if (!__any_sync(0xffffffffu, odd != 0)) continue;
#pragma unroll 1
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t votes = __ballot_sync(0xffffffffu, (odd >> i) & 1u);
      if (!((votes >> (lane - piece)) & ((1u << CPR) - 1u))) continue;  // (CPR is 8 or 16)
      *reinterpret_cast<uint4*>(at + (row0 + i * RPS) * 128) = make_uint4(0u, 0u, 0u, 0u);
      if (piece == 0) note(row0 + i * RPS);
    }
  }
}

// Windows, the rare case: V rows with an infinity or NaN that were kept out of the unit's V tiles.
// Every row of the warp that sees such a token adds weight * V to its O in TMEM (its sum of weights
// has the weight already).  q: the thread's query row (NULL: none).
template <int D>
__device__ __forceinline__ void add_odd_tokens(const PrefillParams& p, const PfUnitW& it, const uint32_t* odd,
                                            uint32_t o_tmem, const __nv_bfloat16* q, int p_row, float m_run) {
  const int p_first = pf_first_query(p, it), span = 2 * p.Tq;
  __threadfence();  // beside decodes nothing has waited: lines that an earlier kernel left in this SM's L1 are dropped
#pragma unroll 1
  for (int i = 0; i < 2 * span; ++i) {
    if (!((*reinterpret_cast<const volatile uint32_t*>(odd + i / 32) >> (i % 32)) & 1u)) continue;
    const int t = i < span ? i + p_first - p.window + 1 : i - span + p_first + 1;
    const bool sees = q && t <= p_row && (t > p_row - p.window || t < it.w.sinks);
    const int page = t / p.bs;
    const int b = checked_block(p.block_table + (size_t)it.s * p.max_blocks, page < it.w.low ? page : page + it.w.skip,
                                p.num_blocks, &g_status_prefill);
    const size_t row = (((size_t)max(b, 0) * p.bs + (t - page * p.bs)) * p.G + it.g) * D;
    float weight = 0.f;
    if (sees) {
      const uint4* a = reinterpret_cast<const uint4*>(q);
      const uint4* k = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.k_cache) + row);
      float s = 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = a[c], y = k[c];
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), s);
          s = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), s);
        }
      }
      weight = exp2_approx(s * p.scale_log2 - m_run);
    }
    const uint32_t* v = reinterpret_cast<const uint32_t*>(reinterpret_cast<const __nv_bfloat16*>(p.v_cache) + row);
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      uint32_t ov[16];
      tmem_ld16(o_tmem + c * 16, ov);
      tmem_ld_wait();
      if (sees) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = v[c * 8 + e];
          ov[2 * e] = __float_as_uint(fmaf(weight, __uint_as_float(w << 16), __uint_as_float(ov[2 * e])));
          ov[2 * e + 1] = __float_as_uint(fmaf(weight, __uint_as_float(w & 0xffff0000u), __uint_as_float(ov[2 * e + 1])));
        }
      }
      tmem_st16(o_tmem + c * 16, ov);
      tmem_st_wait();
    }
  }
}

// Unit u: `whole` units in one piece, then the parts of `rest` others.  A part begins where
// every query row of the pair sees keys: its running maximum is finite from its first tile on.
__device__ __forceinline__ bool pf_unit(const PrefillParams& p, int u, int whole, int rest, int splits, PfUnit8& it) {
  int part = 0;
  if (u >= whole) {
    part = (u - whole) / rest;
    u -= part * rest;
  }
  it.j0 = it.tag = 0;
  if (!pf_unit(p, u, it)) return false;
  if (u >= whole && it.n_kv < kMinSplitTiles) return part == 0;
  if (u >= whole) {
    const int len = max((it.n_kv + splits - 1) / splits, kMinPartTiles);
    const int last = (it.L - it.q_len + 2 * it.pair * p.Tq) / kKvTile;  // the latest first tile
    const int parts = min(splits, last / len + 1);
    if (part >= parts) return false;
    if (parts > 1) it.tag = (u - whole) << 8 | parts << 4 | part;
    it.j0 = part * len;
    const int end = part == parts - 1 ? it.n_kv : it.j0 + len;
    it.n0 = min(it.n0, end) - it.j0;
    if (it.n1 > 0) it.n1 = min(it.n1, end) - it.j0;
    it.n_kv = max(it.n0, it.n1);
  }
  return true;
}

// Eight e4m3 codes of one row times their page's scale, as bf16 (exact: four significant
// bits and a power of two).  Values past bf16's range become its largest: an infinity of a
// token that a row must not see would reach it as 0 * infinity.
__device__ __forceinline__ uint4 codes_to_bf16x8(uint32_t w0, uint32_t w1, float scale) {
  float a[4], b[4];
  unpack_e4m3x4_f32(w0, a);
  unpack_e4m3x4_f32(w1, b);
  return make_uint4(pack_bf16x2_sat(a[0] * scale, a[1] * scale), pack_bf16x2_sat(a[2] * scale, a[3] * scale),
                    pack_bf16x2_sat(b[0] * scale, b[1] * scale), pack_bf16x2_sat(b[2] * scale, b[3] * scale));
}

// 8-bit cache: the query row `row` of a 128-row bf16 tile as two e4m3 parts, q up = hi + lo, so
// that S = (hi + lo) codes^T runs on the codes themselves at twice the bf16 rate, twice.  up
// is a power of two that brings the row's largest element into [2^7, 2^8): the parts are
// exact for elements down to 2^-8 of it and off by at most 2^-10 (of 2^7) below that.
// In place, one thread per row: the row's bytes of hi go over its first 128-byte half and
// those of lo over the second (head_dim 64: both into its one 128 bytes).  Returns 1 / up,
// or NaN for a row with an infinity or NaN (its scores are NaN).
template <int D>
__device__ __forceinline__ float split_query_row(uint8_t* tile, int row) {
  constexpr int kChunks = D / 8;  // 16-byte chunks of the bf16 row
  uint8_t* at = tile + row * 128;
  uint4 v[kChunks];
  uint32_t top = 0;               // bf16 magnitudes order like their bits
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    v[c] = *reinterpret_cast<const uint4*>(at + (c >> 3) * (kRows * 128) + (((c & 7) ^ (row & 7)) << 4));
    top = max_u16x2(max_u16x2(top, v[c].x & 0x7fff7fffu), v[c].y & 0x7fff7fffu);
    top = max_u16x2(max_u16x2(top, v[c].z & 0x7fff7fffu), v[c].w & 0x7fff7fffu);
  }
  top = max(top >> 16, top & 0xffffu);
  const uint32_t field = max(top >> 7, 8u);  // exponent field of the largest element
  const float up = __uint_as_float((261u - min(field, 254u)) << 23);
#pragma unroll
  for (int c = 0; c < kChunks; c += 2) {
    uint32_t hi[4], lo[4];
    split_e4m3x4(make_uint2(v[c].x, v[c].y), up, hi[0], lo[0]);
    split_e4m3x4(make_uint2(v[c].z, v[c].w), up, hi[1], lo[1]);
    split_e4m3x4(make_uint2(v[c + 1].x, v[c + 1].y), up, hi[2], lo[2]);
    split_e4m3x4(make_uint2(v[c + 1].z, v[c + 1].w), up, hi[3], lo[3]);
    const int o = c / 2;  // output chunk of the row
    *reinterpret_cast<uint4*>(at + ((o ^ (row & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    uint8_t* lo_at = D == 128 ? at + kRows * D + ((o ^ (row & 7)) << 4) : at + (((4 + o) ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(lo_at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  return __uint_as_float(field >= 255u ? 0x7fc00000u : (field - 7u) << 23);
}

// A part's result for row `row` of query tile w, for join_parts: normalised, rows side by side.
template <int D>
__device__ __forceinline__ void write_part(const PrefillParams& p, int tag, int rest, int w, int row,
                                           uint32_t o_tmem, float inv, float lse2, bool nan_any,
                                           const uint16_t* nan_first, int rel) {
  const size_t tile = (size_t)((tag & 15) * rest + (tag >> 8)) * 2 + w;
  float4* out = reinterpret_cast<float4*>(p.part_out) + tile * (D / 4) * kRows + row;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t ov[32];
    tmem_ld32(o_tmem + c * 32, ov);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      out[(c * 8 + i / 4) * kRows] = make_float4(__uint_as_float(ov[i]) * inv, __uint_as_float(ov[i + 1]) * inv,
                                                 __uint_as_float(ov[i + 2]) * inv, __uint_as_float(ov[i + 3]) * inv);
  }
  if (nan_any) {
#pragma unroll 1
    for (int d = 0; d < D; ++d)
      if (nan_first[d] <= rel) reinterpret_cast<float*>(out + (d / 4) * kRows)[d % 4] = __uint_as_float(0x7fc00000u);
  }
  p.part_lse[tile * kRows + row] = lse2;
}

// The warp that finishes its 32 rows of a unit last merges their parts, in the order of the
// keys: out = sum of o_i 2^(x_i - M) over sum of 2^(x_i - M).
template <int D>
__device__ __forceinline__ void join_parts(const PrefillParams& p, int tag, int rest, int w, int row, int lane,
                                           __nv_bfloat16* orow, float* lse) {
  const int parts = (tag >> 4) & 15;
  __threadfence();  // the part is visible before it is counted
  __syncwarp();
  int before = 0;
  if (lane == 0) before = atomicAdd(p.parts_done + ((size_t)(tag >> 8) * 2 + w) * (kRows / 32) + row / 32, 1);
  before = __shfl_sync(0xffffffffu, before, 0);
  if (before != parts - 1) return;
  __threadfence();
  if (orow == nullptr) return;
  const size_t tile = (size_t)(tag >> 8) * 2 + w, next = (size_t)rest * 2;
  float x[kMaxSplits], M = -INFINITY, W = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits; ++i) {
    x[i] = i < parts ? __ldcg(p.part_lse + (tile + i * next) * kRows + row) : -INFINITY;
    M = fmaxf(M, x[i]);
  }
#pragma unroll
  for (int i = 0; i < kMaxSplits; ++i) {
    x[i] = i < parts ? exp2_approx(x[i] - M) : 0.f;
    W += x[i];
  }
  const float inv = 1.f / W;
  const float4* src = reinterpret_cast<const float4*>(p.part_out) + tile * (D / 4) * kRows + row;
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll
    for (int i = 0; i < kMaxSplits; ++i)
      if (i < parts) {
        const float4* at = src + i * next * (D / 4) * kRows + (size_t)(2 * c) * kRows;
        const float4 u = __ldcg(at), v = __ldcg(at + kRows);
        a = make_float4(fmaf(x[i], u.x, a.x), fmaf(x[i], u.y, a.y), fmaf(x[i], u.z, a.z), fmaf(x[i], u.w, a.w));
        b = make_float4(fmaf(x[i], v.x, b.x), fmaf(x[i], v.y, b.y), fmaf(x[i], v.z, b.z), fmaf(x[i], v.w, b.w));
      }
    *reinterpret_cast<uint4*>(orow + c * 8) =
        make_uint4(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv),
                   pack_bf16x2(b.x * inv, b.y * inv), pack_bf16x2(b.z * inv, b.w * inv));
  }
  if (lse) *lse = (M + log2f(W)) * kLn2;
}

// Shared prefixes: a CTA's share [begin, end) of all units' K/V tiles in a row, the group in which it begins, and
// the tiles and units of the groups before that one.
struct PfShare {
  int begin, end, group, x, unit;
  PfGroup now;  // the group
};

// Shared prefixes, by one warp of every CTA, 32 sequences each at a time: where the sequences' own tokens begin.
__device__ __forceinline__ void pf_own_tokens(const PrefillParams& p, int lane) {
  for (long long s0 = (long long)blockIdx.x * 32; s0 < p.S; s0 += (long long)gridDim.x * 32) {
    const int s = (int)min(s0 + lane, (long long)p.S - 1);
    int lo = -1, hi = p.num_groups - 1;  // the last group that begins at or before s (-1: none)
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.cu_q_lens[mid] <= s)
        lo = mid;
      else
        hi = mid - 1;
    }
    SharedOwn v{0, -1};
    int L = p.seq_lens[s];
    if (L > p.cap) atomicOr(&g_status_prefill, METIS_STATUS_SEQ_TOO_LONG);
    L = min(L, p.cap);
    if (lo >= 0) {
      const int a = p.cu_q_lens[lo], b = p.cu_q_lens[lo + 1], tokens = p.prefix_lens[lo];
      if (a >= 0 && a <= s && s < b && b <= p.S && tokens > 0 && L >= tokens) v = SharedOwn{tokens, lo};
    }
    if (s0 + lane < p.S) p.own[s] = v;
  }
}

// Shared prefixes: how many of the grid's CTAs share the `total` K/V tiles of `units` units (shared_split.cuh).
// shared_tokens: of the caller's groups, over all threads the members' shared tokens.
__device__ __forceinline__ int pf_shared_ctas(const PrefillParams& p, int total, int units, long long shared_tokens) {
  __shared__ long long warp_tokens[kPfThreads / 32];
  __shared__ unsigned long long warp_best[kPfThreads / 32];
  const int tid = threadIdx.x, sms = gridDim.x;
  // Whole numbers: every CTA has to come to the same count, in whichever order its threads add up.
  long long tokens = -shared_tokens;
  for (int s = tid; s < p.S; s += kPfThreads) tokens += min(max(p.seq_lens[s], 0), p.cap);
  // (a batch has at most 2^47 of either kind: in two parts that 32 bits hold)
  const unsigned low = __reduce_add_sync(0xffffffffu, (unsigned)tokens & 0x3ffffffu);
  const int high = __reduce_add_sync(0xffffffffu, (int)(tokens >> 26));
  if ((tid & 31) == 0) warp_tokens[tid >> 5] = ((long long)high << 26) + low;
  __syncthreads();
  if (total == 0) return 0;
  tokens = 0;
#pragma unroll
  for (int w = 0; w < kPfThreads / 32; ++w) tokens += warp_tokens[w];
  const float bytes = (float)max(tokens, 0ll) * p.kv_token_bytes;
  unsigned long long best = ~0ull;
  for (int n = tid + 1; n <= shared_split_most(bytes, sms); n += kPfThreads)
    best = min(best, shared_split_key(total, units, bytes, n, sms));
  const unsigned time = __reduce_min_sync(0xffffffffu, (unsigned)(best >> 32));
  const unsigned count = __reduce_min_sync(0xffffffffu, (unsigned)(best >> 32) == time ? (unsigned)best : 0xffffffffu);
  if ((tid & 31) == 0) warp_best[tid >> 5] = (unsigned long long)time << 32 | count;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPfThreads / 32; ++w) best = min(best, warp_best[w]);
  return min((int)(unsigned)best, total);
}

// Shared prefixes: this CTA's share.  Called by the whole block.  On the way the grid leaves the plan for the
// kernels behind, the first of which may then start: every CTA has waited for the kernels in front.
__device__ __forceinline__ PfShare pf_share(const PrefillParams& p) {
  __shared__ int warp_sums[kPfThreads / 32];
  __shared__ PfShare mine;
  const int tid = threadIdx.x;
  int x = 0, unit = 0;  // of the groups before this round's
  PfGroup v{};
  int my_x = 0, my_unit = 0;
  long long shared_tokens = 0;  // of this thread's groups' members
  bool disorder = false;
  if (tid >= kPfThreads - 32) pf_own_tokens(p, tid & 31);
  auto round = [&](int g0, bool first) {
    unsigned bad = 0;
    bool decreases = false;
    v = g0 + tid < p.num_groups ? pf_group(p, g0 + tid, &bad, &decreases) : PfGroup{};
    __syncwarp();
    pf_lead_all(p, v);
    disorder |= __syncthreads_or(decreases);
    int sum;
    my_unit = unit + block_exclusive_scan<kPfThreads>(v.units, warp_sums, &sum);
    unit += sum;
    __syncthreads();  // the sums were read
    my_x = x + block_exclusive_scan<kPfThreads>(v.units * v.tiles, warp_sums, &sum);
    x += sum;
    __syncthreads();
    if (first && v.units) shared_tokens += (long long)v.n * v.tokens;
    if (first && blockIdx.x == 0 && g0 + tid < p.num_groups) {
      p.plan->group[g0 + tid] = make_int2(my_unit, v.units / p.G);
      if (bad) atomicOr(&g_status_prefill, bad);
    }
  };
  for (int g0 = 0; g0 < p.num_groups; g0 += kPfThreads) round(g0, true);
  // Groups that overlap (offsets that decrease somewhere) could have more units than there is room for
  const int total = disorder ? 0 : x, ctas = pf_shared_ctas(p, total, unit, shared_tokens);
  if (tid >= kPfThreads - 32) {
    if (blockIdx.x == 0 && tid == kPfThreads - 1) {
      p.plan->total = make_int2(total, ctas);
      p.plan->own_shares = 0;
      p.plan->next_share = 0;
    }
    __threadfence();
    __syncwarp();
    if (tid == kPfThreads - 1) pdl_launch_dependents();
  }
  PfShare s{};
  if (total == 0) return s;
  s.begin = (int)((long long)min((int)blockIdx.x, ctas) * total / ctas);
  s.end = (int)((long long)min((int)blockIdx.x + 1, ctas) * total / ctas);
  if (s.begin == s.end) return s;
  auto find = [&](int g0) {  // the group with tile s.begin is this thread's
    if (my_x <= s.begin && s.begin - my_x < v.units * v.tiles) {
      mine.group = g0 + tid;
      mine.x = my_x;
      mine.unit = my_unit;
      mine.now = v;
    }
  };
  if (p.num_groups <= kPfThreads) {
    find(0);
  } else {
    x = unit = 0;
    for (int g0 = 0; g0 < p.num_groups; g0 += kPfThreads) {
      round(g0, false);
      find(g0);
    }
  }
  __syncthreads();
  s.group = mine.group;
  s.x = mine.x;
  s.unit = mine.unit;
  s.now = mine.now;
  return s;
}

// KV8: the cache holds e4m3 codes.  K tiles feed the tensor cores as they are, against the
// query rows split into two e4m3 parts; V tiles are converted to bf16 on the way; a K page's
// scale joins the softmax factor of its 16 tokens.
// SPLIT (8-bit cache): units may be parts of a pair's keys.  An instantiation of its own: the
// registers and the code of the parts cost whole units 2-3 %.
// WINDOW (bf16 cache): a query sees the last `window` and the first `sinks` keys before it.  Only tiles with
// such keys are visited.  Their hidden keys are masked per row as later ones are; the row may see nothing in its
// first tiles.  Warp 15 looks at the V rows that not every query of the unit sees (PfWindowShared).
// SHARED (bf16 cache): prefixes that groups of decodes share (PfGroup).  The units come from the groups
// directly, without a schedule kernel, and every result is a part for the kernel behind this one.
template <int D, bool KV8, bool SPLIT, bool WINDOW, bool SHARED>
__global__ void __launch_bounds__(kPfThreads, 1) prefill_bf16_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                       const __grid_constant__ CUtensorMap tmK,
                                                                       const __grid_constant__ CUtensorMap tmV,
                                                                       const PrefillParams p) {
  using Sh = PfShape<D, KV8>;
  constexpr int HALVES = Sh::kHalves;
  constexpr int kStages8 = kV8Stages;
  constexpr int kOther = KV8 ? kRegsOther8 : WINDOW || SHARED ? kRegsMmaU : kRegsMma;  // registers of the last warpgroup
  static_assert(KV8 || !SPLIT, "parts of units: 8-bit cache only");
  static_assert(!(WINDOW && KV8), "windows: bf16 cache only");
  static_assert(!(SHARED && (WINDOW || KV8)), "shared prefixes: bf16 cache only");
  using Unit = std::conditional_t<SPLIT, PfUnit8, std::conditional_t<WINDOW, PfUnitW, std::conditional_t<SHARED, PfUnitS, PfUnit>>>;
  // The schedule kernel's items, and what the kernels in front of it wrote (tables, scale bytes),
  // are complete: waited for here, or by every CTA of the decode grid in front before it let this
  // grid launch (the warps that read more than the items then fence, below).
  if (!p.wait_at_exit) pdl_wait();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t slack = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + slack;
  uint8_t* sQ = smem + Sh::kQ;
  uint8_t* sK = smem + Sh::kK;
  uint8_t* sV = smem + Sh::kV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(slack >= 256 ? smem - 256 : smem + Sh::kTiles);
  uint64_t* q_full = bars + PfBar::kQFull;
  uint64_t* k_full = bars + PfBar::kKFull;      // [kKStages]
  uint64_t* k_empty = bars + PfBar::kKEmpty;    // [kKStages]
  uint64_t* v_full = bars + PfBar::kVFull;      // [kVStages]
  uint64_t* v_empty = bars + PfBar::kVEmpty;    // [kVStages]
  uint64_t* s_full = bars + PfBar::kSFull;      // [2 groups] QK_w_j landed in S_w
  uint64_t* p_full = bars + PfBar::kPFull;      // [2 groups] P_w_j written over S_w (128 arrivals)
  uint64_t* pv_done = bars + PfBar::kPvDone;    // [2 groups] PV_w_j completed
  uint64_t* drain = bars + PfBar::kDrain;
  uint64_t* q_free = bars + PfBar::kQFree;      // every QK of a unit completed: its query tiles may be replaced
  uint64_t* unit_full = bars + PfBar::kUnitFull;    // [2] a unit index published
  uint64_t* unit_empty = bars + PfBar::kUnitEmpty;  // [2] every consuming warp has read it (kUnitReaders arrivals)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + PfBar::kCount);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + PfBar::kCount + 1);
  volatile int* unit_slot = reinterpret_cast<volatile int*>(bars + PfBar::kCount + 2);  // [2]
  __shared__ Unit unit_info[2];  // the published unit, derived once by the fetcher
  __shared__ PfFp8Shared x8;       // (8-bit cache only)
  __shared__ PfWindowShared xw;    // (windows only)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  [[maybe_unused]] PfShare share{};  // shared prefixes
  int units;
  if constexpr (SHARED) {
    share = pf_share(p);
    units = share.end > share.begin ? gridDim.x : 0;
  } else {
    units = __ldcg(p.item_count) * p.G;
  }
  [[maybe_unused]] int2 splits = make_int2(1, units);  // parts of each unit that is split, units that are not
  [[maybe_unused]] const int rest = SPLIT ? units - (splits = __ldcg(p.splits)).y : 0;
  if (SPLIT) units = splits.y + rest * splits.x;
  if ((int)blockIdx.x >= units) {
    if (p.wait_at_exit) pdl_wait();  // complete only after the decode grid in front of this one
    return;
  }

  if (threadIdx.x == 0) {
    // full barriers: one arrival per producer warp of the ring; p_full: 128 softmax threads
    for (int i = 0; i < PfBar::kCount; ++i) mbar_init(&bars[i], PfBar::arrivals(i, KV8, WINDOW));
    if constexpr (WINDOW) {
      for (int i = 0; i < kVStages; ++i) mbar_init(&xw.v_ready[i], 1);
    }
    if constexpr (KV8) {
      for (int i = 0; i < kV8Stages; ++i) {
        mbar_init(&x8.stage_full[i], 1);
        mbar_init(&x8.stage_empty[i], kV8Converters);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&x8.q_raw[i], 1);
        mbar_init(&x8.q_full[i], 4);
      }
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  } else if (warp >= 8 && p.wait_at_exit) {
    __threadfence();  // nothing here waited: lines that an earlier kernel left in this SM's L1 are dropped
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // A wait that also gives up when another role has aborted.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1; i < kMaxPolls; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((i & 255u) == 0) {
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > kMaxWaitNs) break;
      }
    }
    atomicOr(&g_status_prefill, METIS_STATUS_WAIT_TIMEOUT);
    *abort_flag = 1;
    return false;
  };
  // every role calls waits with all 32 lanes: agree on the outcome before any warp-collective op
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
  // The k-th unit of this CTA, from the unit ring: 1 = a unit, 0 = no more, -1 = aborted.
  // The fetcher publishes the unit's derived fields with it, so that no role waits on
  // global loads at a unit boundary.
  auto next_unit = [&](uint32_t& k, Unit& it) -> int {
    const int slot = k & 1;
    if (!wait_all(&unit_full[slot], (k >> 1) & 1)) return -1;
    const int u = unit_slot[slot];
    if (u >= 0) it = unit_info[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&unit_empty[slot]);  // release: the reads above are done
    ++k;
    return u < 0 ? 0 : 1;
  };

  // Ring positions run on across units: K/V tile t (counted over every unit this
  // CTA has processed) sits in K stage t % kKStages and V stage t % kVStages, and each
  // barrier's phase is the number of its earlier completions.
  if (KV8 && warp == 8) {
    // ------------------------------------------------------------ 8-bit cache: TMA producer
    regs_dec<kRegsOther8>();
    const int npg = kKvTile / p.bs;            // pages per K/V tile (2, 4 or 8)
    const int reps = p.bs >> 4;                // 16-token groups per page
    const uint64_t pol = l2_policy_evict_last();
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    uint32_t t = 0, k = 0;                     // tiles issued so far, units read
    bool ok = true;
    Unit it;
    while (ok && next_unit(k, it) > 0) {
      const int32_t* bt_row = p.block_table + (size_t)it.s * p.max_blocks;
      {
        const int slot = (k - 1) % kNanUnits;  // (the converters see it cleared by the unit's first V tile)
        uint32_t* first = reinterpret_cast<uint32_t*>(x8.nan_first[slot]);
        for (int i = lane; i < 64; i += 32) first[i] = 0xffffffffu;
        if (lane == 0) x8.nan_any[slot] = 0;
        if constexpr (SPLIT)
          if (lane == 0) x8.tag[slot] = it.tag;
        __syncwarp();
      }
      // page `lane` of tile j: its TMA row (a bad id reads a box out of bounds: zeros) and scales
      auto page_of = [&](int j, int& rowc, float& fk, float& fv) -> bool {
        const int pg = (pf_first(it) + j) * npg + lane;
        rowc = -p.bs;
        fk = fv = 1.f;
        if (lane >= npg || pg >= it.n_pages) return false;
        const int b = checked_block(bt_row, pg, p.num_blocks, &g_status_prefill);
        if (b >= 0) {
          rowc = b * p.bs;
          fk = scale_of_byte(ld_byte(p.fp8.k_scale + (size_t)b * p.G + it.g));
          fv = scale_of_byte(ld_byte(p.fp8.v_scale + (size_t)b * p.G + it.g));
        }
        return true;
      };
      int rowc = 0;
      float fk = 1.f, fv = 1.f;
      bool live = page_of(0, rowc, fk, fv);
      for (int j = 0; j < it.n_kv; ++j, ++t) {
        int next_row = 0;
        float next_k = 1.f, next_v = 1.f;
        bool next_live = false;
        if (j + 1 < it.n_kv) next_live = page_of(j + 1, next_row, next_k, next_v);  // in flight during the waits
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, live)) * p.bs * D;
        const int st = t % kKStages, sv = t % kStages8;
        // K_{t-3} consumed: also every softmax group is past tile t - 4, whose factors sit in this slot
        if (t >= (uint32_t)kKStages && !wait_all(&k_empty[st], ((t / kKStages) - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane < npg)
          for (int u = 0; u < reps; ++u)
            reinterpret_cast<float*>(x8.ks[t % kKScaleSlots])[lane * reps + u] = fk;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&k_full[st], bytes);
        __syncwarp();
        if (live) tma_load_3d(sK + st * Sh::kKBytes + lane * p.bs * D, &tmK, &k_full[st], 0, it.g, rowc, pol);
        if (t >= (uint32_t)kStages8 && !wait_all(&x8.stage_empty[sv], ((t / kStages8) - 1) & 1)) {
          ok = false;
          ++t;  // K of this tile is in flight
          break;
        }
        if (lane < npg)
          for (int u = 0; u < reps; ++u) x8.vs[sv][lane * reps + u] = fv;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&x8.stage_full[sv], bytes);
        __syncwarp();
        if (live)
          tma_load_3d(smem + Sh::kStage + sv * kKvTile * D + lane * p.bs * D, &tmV, &x8.stage_full[sv], 0, it.g, rowc,
                      pol);
        rowc = next_row;
        fk = next_k;
        fv = next_v;
        live = next_live;
      }
    }
    if (*abort_flag) {
      // let the loads still in flight land before the CTA's memory goes away (the limit of
      // each wait bounds the one on a V tile that was not issued)
      for (uint32_t i = t > (uint32_t)kKStages ? t - kKStages : 0; i < t; ++i)
        mbar_wait(&k_full[i % kKStages], (i / kKStages) & 1, &g_status_prefill);
      for (uint32_t i = t > (uint32_t)kStages8 ? t - kStages8 : 0; i < t; ++i)
        mbar_wait(&x8.stage_full[i % kStages8], (i / kStages8) & 1, &g_status_prefill);
    }
  } else if (KV8 && ((warp > 8 && warp < kMmaWarp) || warp == 15)) {
    // ------------------------------------------------------------ 8-bit cache: V converters
    regs_dec<kRegsOther8>();
    const int cw = warp == 15 ? 3 : warp - 9;
    uint32_t t = 0, k = 0;
    bool ok = true;
    Unit it;
    while (ok && next_unit(k, it) > 0) {
      constexpr int CPR = D / 16, RPC = 32 / CPR;   // V: 16-byte pieces of a row, rows per pass
      const int piece = lane % CPR;
      const int flip = D == 128 ? piece >> 2 : 0;   // the two halves' lanes write opposite chunks at a time
      const int p_min = it.L - it.q_len + 2 * it.pair * p.Tq;  // position of the unit's first query token
      const int nan_slot = (k - 1) % kNanUnits;
      for (int j = 0; j < it.n_kv; ++j, ++t) {
        const int sv = t % kStages8, st = t % kVStages;
        if (!wait_all(&x8.stage_full[sv], (t / kStages8) & 1) ||
            (t >= (uint32_t)kVStages && !wait_all(&v_empty[st], ((t / kVStages) - 1) & 1))) {
          ok = false;
          break;
        }
        const uint4* src = reinterpret_cast<const uint4*>(smem + Sh::kStage + sv * kKvTile * D) + lane;
        uint8_t* tile = sV + st * Sh::kKvBytes + (piece * 16 / 64) * Sh::kKvHalf;
        auto put = [&](int row, const uint4& c, float f) {
          const uint4 a = codes_to_bf16x8(c.x, c.y, f), b = codes_to_bf16x8(c.z, c.w, f);
          const int ch = (piece * 2 & 7) + flip;
          uint8_t* dst = tile + row * 128;
          *reinterpret_cast<uint4*>(dst + ((ch ^ (row & 7)) << 4)) = flip ? b : a;
          *reinterpret_cast<uint4*>(dst + (((ch ^ 1) ^ (row & 7)) << 4)) = flip ? a : b;
        };
        const int seen_rows = p_min + 1 - (pf_first(it) + j) * kKvTile;  // rows that every query row of the unit sees
        if (seen_rows >= kKvTile) {
#pragma unroll 1
          for (int i = cw; i < kKvTile / RPC; i += kV8Converters) {
            const int row = i * RPC + lane / CPR;
            put(row, src[i * 32], x8.vs[sv][row >> 4]);
          }
        } else {
          const int live_rows = it.L - (pf_first(it) + j) * kKvTile;  // rows past the sequence end become zeros
#pragma unroll 1
          for (int i = cw; i < kKvTile / RPC; i += kV8Converters) {
            const int row = i * RPC + lane / CPR;
            uint4 c = src[i * 32];
            float f = x8.vs[sv][row >> 4];
            if (row >= live_rows) {
              c = make_uint4(0u, 0u, 0u, 0u);
              f = 1.f;
            } else if (row >= seen_rows && (any_nan_code(c) || f != f)) {
              c = note_nan_codes(c, f != f, x8.nan_first[nan_slot] + piece * 16, &x8.nan_any[nan_slot],
                                 (uint16_t)(row - seen_rows + 1));
              f = f != f ? 1.f : f;
            }
            put(row, c, f);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&x8.stage_empty[sv]);
          mbar_arrive(&v_full[st]);
        }
      }
    }
  } else if (warp >= 8 && warp < kMmaWarp) {
    // ------------------------------------------------------------ K/V producers
    regs_dec<kRegsProd>();
    const int pw = warp - 8;
    const bool is_k = pw < 2;
    const int part = pw & 1;                   // which half of each tile's pages
    const CUtensorMap* map = is_k ? &tmK : &tmV;
    uint8_t* ring = is_k ? sK : sV;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    const int npg = kKvTile / p.bs;            // pages per K/V tile (2, 4 or 8)
    const int half_pg = npg >> 1;              // pages of this warp
    const uint64_t pol = l2_policy_evict_last();
    const int depth = is_k ? kKStages : kVStages;
    if (lane == 0) tma_prefetch_desc(map);
    uint32_t t = 0, k = 0;                     // tiles issued so far, units read
    bool ok = true;
    Unit it;
    while (ok && next_unit(k, it) > 0) {
      const int32_t* bt_row = p.block_table + (size_t)it.s * p.max_blocks;
      for (int j = 0; j < it.n_kv; ++j, ++t) {
        const int st = t % depth;
        const int lp = part * half_pg + lane;  // page index inside the tile
        int pg = pf_tile(it, j) * npg + lp;
        const bool live = lane < half_pg && pg < it.n_pages;
        if constexpr (WINDOW) pg += pg < it.w.low ? 0 : it.w.skip;
        int rowc = 0;
        if (live) {
          const int b = checked_block(bt_row, pg, p.num_blocks, &g_status_prefill);
          rowc = b < 0 ? -p.bs : b * p.bs;   // a bad id reads a box entirely out of bounds: zeros
        }
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, live)) * p.bs * 128 * HALVES;
        if (t >= (uint32_t)depth && !wait_all(&empty[st], ((t / depth) - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
        __syncwarp();
        if (live)
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(ring + st * Sh::kKvBytes + h * Sh::kKvHalf + lp * p.bs * 128, map, &full[st], h * 64, it.g,
                        rowc, pol);
      }
    }
    if (*abort_flag) {
      // let the loads still in flight land before the CTA's memory goes away
      for (uint32_t k = t > (uint32_t)depth ? t - depth : 0; k < t; ++k)
        mbar_wait(&full[k % depth], (k / depth) & 1, &g_status_prefill);
    }
  } else if ((KV8 || WINDOW || SHARED) && warp == kMmaWarp) {
    // ------------------------------------------------------------ UMMA issuer (8-bit cache, windows, shared prefixes)
    // The same order of products as below, PV0_j, QK0_{j+1}, PV1_j, QK1_{j+1}.  Everything
    // the instructions' operands come from is kept uniform over the warp (values from
    // shared memory by shuffle, outcomes of waits by vote, ring positions counted instead
    // of divided), so that descriptors are built on the uniform datapath.
    regs_dec<kOther>();
    constexpr uint32_t kIdQK = KV8 ? umma_idesc_e4m3_f32(kRows, kKvTile) : umma_idesc_bf16_f32(kRows, kKvTile, false, false);
    constexpr uint32_t kIdPV = umma_idesc_bf16_f32(kRows, D, false, true);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t q_at = __shfl_sync(0xffffffffu, smem_u32(sQ), 0);
    const uint32_t k_at = __shfl_sync(0xffffffffu, smem_u32(sK), 0);
    const uint32_t v_at = __shfl_sync(0xffffffffu, smem_u32(sV), 0);
    uint32_t k_st = 0, k_ph = 0, v_st = 0, v_ph = 0;   // next K and V tile: ring stage, phase parity
    uint32_t p_ph[2] = {0u, 0u}, u = 0, n_two = 0;     // p_full parities; units; units with two query tiles
    [[maybe_unused]] uint32_t looked = 0;              // windows: per V stage, v_ready's parity
    bool ok = true, issued = false;
    auto qk = [&](int w) {  // S_w = Q_w K^T of the K tile in stage k_st (8-bit: (hi_w + lo_w) codes^T, 32 dims per instruction)
      const uint32_t a = q_at + w * Sh::kQBytes, b = k_at + k_st * Sh::kKBytes;
      if (elect_one()) {
        if constexpr (KV8) {
#pragma unroll
          for (int kk = 0; kk < 2 * (D / 32); ++kk) {
            const uint32_t qa = a + (kk / (D / 32)) * (D == 128 ? Sh::kQPart : 64) + (kk % (D / 32)) * 32;
            const uint32_t ka = b + (kk % (D / 32)) * 32;
            umma_e4m3(tm + w * kKvTile, umma_desc_sw128(qa, 16, 1024),
                      D == 128 ? umma_desc_sw128(ka, 16, 1024) : umma_desc_sw64(ka, 512), kIdQK, kk > 0 ? 1u : 0u);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t within = (kk & 3) * 32;
            umma_bf16(tm + w * kKvTile, umma_desc_sw128(a + (kk >> 2) * Sh::kQHalf + within, 16, 1024),
                      umma_desc_sw128(b + (kk >> 2) * Sh::kKvHalf + within, 16, 1024), kIdQK, kk > 0 ? 1u : 0u);
          }
        }
        umma_commit(&s_full[w]);
      }
    };
    auto pv = [&](int w, uint32_t add) {  // O_w (+)= P_w V of the V tile in stage v_st, P_w over S_w's first columns
      const uint32_t b = v_at + v_st * Sh::kKvBytes;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kKvTile / 16; ++kk)
          umma_bf16_tmem_a(tm + 2 * kKvTile + w * D, tm + w * kKvTile + kk * 8,
                           umma_desc_sw128(b + kk * 2048, Sh::kKvHalf, 1024), kIdPV, kk > 0 ? 1u : add);
        umma_commit(&pv_done[w]);
      }
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
    };
    for (;; ++u) {
      const int slot = u & 1;
      if (!(ok = wait_all(&unit_full[slot], (u >> 1) & 1))) break;
      const int index = __shfl_sync(0xffffffffu, unit_slot[slot], 0);
      const int n0 = __shfl_sync(0xffffffffu, unit_info[slot].n0, 0);
      const int n1 = __shfl_sync(0xffffffffu, unit_info[slot].n1, 0);
      [[maybe_unused]] int a0 = 0, a1 = 0, b0 = 0, live = 0;
      if constexpr (WINDOW) {  // the tiles that pf_partial tells
        a0 = __shfl_sync(0xffffffffu, unit_info[slot].a0, 0);
        a1 = __shfl_sync(0xffffffffu, unit_info[slot].a1, 0);
        b0 = __shfl_sync(0xffffffffu, unit_info[slot].b0, 0);
      }
      if constexpr (SHARED)  // keys from the part's first tile on
        live = __shfl_sync(0xffffffffu, unit_info[slot].L - unit_info[slot].j0 * kKvTile, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_empty[slot]);  // release: the reads above are done
      if (index < 0) break;
      const int n_kv = max(n0, n1);
      if (!(ok = wait_all(KV8 ? &x8.q_full[0] : q_full, u & 1) && wait_all(&k_full[k_st], k_ph))) break;
      tc_fence_after_sync();
      issued = true;
      qk(0);
      if (n1 > 0) {
        if constexpr (KV8) {
          if (!(ok = wait_all(&x8.q_full[1], n_two & 1))) break;
          ++n_two;
          tc_fence_after_sync();
        }
        qk(1);
      }
      commit(&k_empty[k_st]);
      if (n_kv == 1) commit(q_free);  // the unit's last QK is issued
      if (++k_st == kKStages) k_st = 0, k_ph ^= 1;
      for (int j = 0; j < n_kv; ++j) {
        if (!(ok = wait_all(&v_full[v_st], v_ph))) break;
        if constexpr (WINDOW) {
          if ((j >= a0 && j < a1) || j >= b0) {
            if (!(ok = wait_all(&xw.v_ready[v_st], (looked >> v_st) & 1))) break;
            looked ^= 1u << v_st;
          }
        }
        if constexpr (SHARED) {
          if (live < (j + 1) * kKvTile) {
            // rows past the prefix may hold anything (NaN included): zero them so that P = 0 stays 0
            uint8_t* vb = sV + v_st * Sh::kKvBytes;
            for (int row = live - j * kKvTile + lane; row < kKvTile; row += 32)
              for (int h = 0; h < HALVES; ++h) {
                uint4* d = reinterpret_cast<uint4*>(vb + h * Sh::kKvHalf + row * 128);
#pragma unroll
                for (int c = 0; c < 8; ++c) d[c] = make_uint4(0u, 0u, 0u, 0u);
              }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        const bool more = j + 1 < n_kv;
        bool k_ready = false;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int nw = w ? n1 : n0;
          if (j < nw) {
            if (!(ok = wait_all(&p_full[w], p_ph[w]))) break;
            p_ph[w] ^= 1;
            tc_fence_after_sync();
            pv(w, j > 0 ? 1u : 0u);
            // the V stage is free once the last PV of this tile has run
            if (w == 1 || n1 <= j) commit(&v_empty[v_st]);
          }
          if (j + 1 < nw) {
            if (!k_ready) {  // K_{t+1} is waited for only after PV0_t is on its way
              if (!(ok = wait_all(&k_full[k_st], k_ph))) break;
              tc_fence_after_sync();
              k_ready = true;
            }
            qk(w);
          }
        }
        if (!ok) break;
        if (more) {
          commit(&k_empty[k_st]);
          if (j + 2 == n_kv) commit(q_free);  // the unit's last QK is issued
          if (++k_st == kKStages) k_st = 0, k_ph ^= 1;
        }
        if (++v_st == kVStages) v_st = 0, v_ph ^= 1;
      }
      if (!ok) break;
    }
    if (!ok && issued) {
      // wait (bounded) for every UMMA this warp issued before TMEM is freed
      commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, &g_status_prefill);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ UMMA issuer
    regs_dec<kOther>();
    constexpr uint32_t kIdQK = umma_idesc_bf16_f32(kRows, kKvTile, false, false);
    constexpr uint32_t kIdPV = umma_idesc_bf16_f32(kRows, D, false, true);
    bool issued = false;
    auto qk = [&](int w, uint32_t t) {  // S_w = Q_w K_t^T
      if (lane == 0) {
        const uint32_t qbase = smem_u32(sQ + w * Sh::kQBytes);
        const uint32_t kbase = smem_u32(sK + (t % kKStages) * Sh::kKBytes);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t within = (kk & 3) * 32;
          umma_bf16(tmem + w * kKvTile, umma_desc_sw128(qbase + (kk >> 2) * Sh::kQHalf + within, 16, 1024),
                    umma_desc_sw128(kbase + (kk >> 2) * Sh::kKvHalf + within, 16, 1024), kIdQK, kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[w]);
      }
    };
    auto pv = [&](int w, uint32_t t, bool first) {  // O_w (+)= P_w V_t, P_w from the first 64 columns of S_w
      if (lane == 0) {
        const uint32_t vbase = smem_u32(sV + (t % kVStages) * Sh::kKvBytes);
        const uint32_t o_tmem = tmem + 2 * kKvTile + w * D;
#pragma unroll
        for (int kk = 0; kk < kKvTile / 16; ++kk)
          umma_bf16_tmem_a(o_tmem, tmem + w * kKvTile + kk * 8,
                           umma_desc_sw128(vbase + kk * 2048, Sh::kKvHalf, 1024), kIdPV, (!first || kk > 0) ? 1u : 0u);
        umma_commit(&pv_done[w]);
      }
    };
    uint32_t t_base = 0, n_units = 0, np[2] = {0u, 0u};  // tiles, units, p_full phases consumed
    uint32_t k = 0;
    bool ok = true;
    Unit it;
    while (ok) {
      const int r = next_unit(k, it);
      if (r <= 0) {
        ok = r == 0;
        break;
      }
      const int nw[2] = {it.n0, it.n1};
      if (!wait_all(q_full, n_units & 1) || !wait_all(&k_full[t_base % kKStages], (t_base / kKStages) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      qk(0, t_base);
      if (it.n1 > 0) qk(1, t_base);
      if (lane == 0) {
        umma_commit(&k_empty[t_base % kKStages]);
        if (it.n_kv == 1) umma_commit(q_free);  // the unit's last QK is issued
      }
      issued = true;
      __syncwarp();
      for (int j = 0; ok && j < it.n_kv; ++j) {
        const uint32_t t = t_base + j;
        const int vst = t % kVStages;
        if (!wait_all(&v_full[vst], (t / kVStages) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int tok0 = j * kKvTile;
        if (tok0 + kKvTile > it.L) {
          // rows past the sequence end may hold anything (NaN included): zero them so that P = 0 stays 0
          uint8_t* vb = sV + vst * Sh::kKvBytes;
          for (int row = (it.L - tok0) + lane; row < kKvTile; row += 32)
            for (int h = 0; h < HALVES; ++h) {
              uint4* d = reinterpret_cast<uint4*>(vb + h * Sh::kKvHalf + row * 128);
#pragma unroll
              for (int c = 0; c < 8; ++c) d[c] = make_uint4(0u, 0u, 0u, 0u);
            }
          fence_proxy_async_smem();
          __syncwarp();
        }
        const bool more = j + 1 < it.n_kv;
        bool k_ready = false;
        for (int w = 0; w < 2; ++w) {
          if (j < nw[w]) {
            if (!wait_all(&p_full[w], np[w] & 1)) {
              ok = false;
              break;
            }
            ++np[w];
            tc_fence_after_sync();
            pv(w, t, j == 0);
            // the V stage is free once the last PV of this tile has run
            if (lane == 0 && (w == 1 || nw[1] <= j)) umma_commit(&v_empty[vst]);
          }
          if (more && j + 1 < nw[w]) {
            if (!k_ready) {  // K_{t+1} is waited for only after PV0_t is on its way
              if (!wait_all(&k_full[(t + 1) % kKStages], ((t + 1) / kKStages) & 1)) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
              k_ready = true;
            }
            qk(w, t + 1);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0 && more) {
          umma_commit(&k_empty[(t + 1) % kKStages]);
          if (j + 2 == it.n_kv) umma_commit(q_free);  // the unit's last QK is issued
        }
        __syncwarp();
      }
      t_base += it.n_kv;
      ++n_units;
    }
    if (!ok && issued) {
      // wait (bounded) for every UMMA this warp issued before TMEM is freed
      if (lane == 0) umma_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, &g_status_prefill);
    }
  } else if (warp == kMmaWarp + 1) {
    // ------------------------------------------------------------ query loader
    regs_dec<kOther>();
    if (lane == 0) tma_prefetch_desc(&tmQ);
    uint32_t n_units = 0, n_two = 0, k = 0;
    Unit it;
    while (next_unit(k, it) > 0) {
      // the previous unit's query tiles stay until its last QK has completed
      if (n_units > 0 && !wait_all(q_free, (n_units - 1) & 1)) break;
      const int ntiles = it.n1 > 0 ? 2 : 1;
      if (WINDOW || SHARED) {  // a box per lane: one thread takes 0.1 us for each
        if (lane == 0) mbar_arrive_expect_tx(q_full, (uint32_t)(ntiles * Sh::kQBytes));
        __syncwarp();
        const uint64_t pol = l2_policy_evict_first();
        for (int i = lane; i < ntiles * p.r * HALVES; i += 32) {
          const int h = i % HALVES, hh = i / HALVES % p.r, w = i / HALVES / p.r;
          tma_load_3d(sQ + w * Sh::kQBytes + h * Sh::kQHalf + hh * p.Tq * 128, &tmQ, q_full, h * 64, it.g * p.r + hh,
                      it.q0 + (2 * it.pair + w) * p.Tq, pol);
        }
      } else if (lane == 0) {
        if (!KV8) mbar_arrive_expect_tx(q_full, (uint32_t)(ntiles * Sh::kQBytes));
        const uint64_t pol = l2_policy_evict_first();
        for (int w = 0; w < ntiles; ++w) {
          if (KV8) mbar_arrive_expect_tx(&x8.q_raw[w], (uint32_t)Sh::kQBytes);
          const int qi0 = (2 * it.pair + w) * p.Tq;
          for (int hh = 0; hh < p.r; ++hh)
            for (int h = 0; h < HALVES; ++h)
              tma_load_3d(sQ + w * Sh::kQBytes + h * Sh::kQHalf + hh * p.Tq * 128, &tmQ, KV8 ? &x8.q_raw[w] : q_full,
                          h * 64, it.g * p.r + hh, it.q0 + qi0, pol);
        }
      }
      __syncwarp();
      ++n_units;
      n_two += ntiles - 1;
    }
    if (*abort_flag && n_units > 0) {
      mbar_wait(KV8 ? &x8.q_raw[0] : q_full, (n_units - 1) & 1, &g_status_prefill);
      if (KV8 && n_two > 0) mbar_wait(&x8.q_raw[1], (n_two - 1) & 1, &g_status_prefill);
    }
  } else if (warp == kMmaWarp + 2) {
    // ------------------------------------------------------------ unit fetcher
    // claims units from the global list, heaviest first, and publishes them to
    // the other warps through the two-slot unit ring; -1 ends the walk.  Unit k is
    // claimed only once every warp has taken unit k - 1: one unit of lookahead, so
    // that at the end of the list no CTA holds small units that an idle CTA could run.
    regs_dec<kOther>();
    uint32_t k = 0;
    [[maybe_unused]] int at = share.begin, group = share.group;
    [[maybe_unused]] PfGroup now = share.now;
    for (;;) {
      const int slot = k & 1;
      if (k >= 1 && !wait_all(&unit_empty[(k - 1) & 1], ((k - 1) >> 1) & 1)) break;
      // parts: about as many as CTAs.  One that claims a second while it runs its first takes it
      // from a CTA that starts a little later (2 x 256 queries beside 32 decodes: 147 or 173 us)
      if (SPLIT && k >= 1 && !wait_all(q_free, (k - 1) & 1)) break;
      int u = 0;
      Unit it;
      if constexpr (SHARED) {
        if (at < share.end) {
          while (at - share.x >= now.units * now.tiles && group + 1 < p.num_groups) {
            share.x += now.units * now.tiles;
            share.unit += now.units;
            unsigned bad = 0;
            bool decreases;
            now = pf_group(p, ++group, &bad, &decreases);
            pf_lead(p, now);
          }
          const int pairs = now.units / p.G, unit = (at - share.x) / now.tiles;
          it.s = now.leader;
          it.g = unit / pairs;
          it.pair = unit - it.g * pairs;
          it.L = now.tokens;
          it.q_len = now.n;
          it.q0 = now.q0;
          it.n_pages = (now.tokens - 1) / p.bs + 1;
          it.j0 = (at - share.x) - unit * now.tiles;
          it.n_kv = it.n0 = min(now.tiles - it.j0, share.end - at);
          it.n1 = (2 * it.pair + 1) * p.Tq < now.n ? it.n0 : 0;
          it.part = share.unit + unit + blockIdx.x;
          at += it.n_kv;
        } else {
          u = -1;
        }
      } else {
        if (lane == 0) u = atomicAdd(p.unit_head, 1);
        u = __shfl_sync(0xffffffffu, u, 0);
      }
      if constexpr (SHARED) {
      } else if (u < units) {
        bool some;  // false: nothing to compute
        if constexpr (SPLIT)
          some = pf_unit(p, u, splits.y, rest, splits.x, it);
        else
          some = pf_unit(p, u, it);
        if (!some) continue;
      } else {
        u = -1;
      }
      // Windows: nothing is noted of the unit yet.  Cleared here, in front of what every reader of the slot waits for:
      // a unit without a partial tile, or a query tile whose own tiles have none, waits for nothing of warp 15.  Every
      // softmax group has written out the unit before the last one, the slot's, as it has taken the last one.
      if constexpr (WINDOW) {
        if (lane < kOddWords) xw.odd[slot][lane] = 0u;
        if (lane == 0) xw.any_odd[slot] = 0;
        __syncwarp();
      }
      if (lane == 0) {
        if (u >= 0) unit_info[slot] = it;
        unit_slot[slot] = u;
        mbar_arrive(&unit_full[slot]);  // release: the unit's fields are visible to every waiter
      }
      __syncwarp();
      ++k;
      if (u < 0) break;
    }
  } else if (WINDOW && warp > kMmaWarp) {
    // ------------------------------------------------------------ windows: V rows that not every query sees
    // Rows that none sees may hold anything: zeros, so that P = 0 stays 0 (also those behind the sequence's
    // end).  Rows that some see become zeros when they hold an infinity or
    // NaN, and are noted.
    regs_dec<kOther>();
    uint32_t t = 0, k = 0;
    bool ok = true;
    Unit it;
    if constexpr (WINDOW) {
      while (ok && next_unit(k, it) > 0) {
        const int slot = (k - 1) & 1;  // (the fetcher has cleared its bits)
        const int p_first = pf_first_query(p, it), p_last = pf_last_query(p, it);
        for (int j = 0; j < it.n_kv; ++j, ++t) {
          const int tok0 = pf_tile(it, j) * kKvTile, st = t % kVStages;
          // (every tile is waited for and given back: a wait tells a phase from the next one only)
          if (!wait_all(&v_full[st], (t / kVStages) & 1)) {
            ok = false;
            break;
          }
          if (!pf_partial(it, j)) {
            if (lane == 0) mbar_arrive(&v_empty[st]);
            continue;
          }
          uint8_t* tile = sV + st * Sh::kKvBytes;
          auto in_tile = [&](int t) { return min(max(max(t, 0) - tok0, 0), kKvTile); };  // (t: to -2^31, of the largest windows)
          // rows that none sees: between the first tokens and the first query's oldest key, and behind the last query
          const int low = in_tile(it.w.sinks), old = max(in_tile(p_first - p.window + 1), low);
          const int leave = max(in_tile(p_last - p.window + 1), old), end = in_tile(p_last + 1);
          zero_rows<D>(tile, low, old, lane);
          zero_rows<D>(tile, end, kKvTile, lane);
          // rows that some see: those that leave the window of some queries, and those behind the first query
          auto note = [&](int row) {
            const int tok = tok0 + row, i = tok > p_first ? 2 * p.Tq + tok - p_first - 1 : tok - (p_first - p.window + 1);
            atomicOr(&xw.odd[slot][i / 32], 1u << (i % 32));
            *reinterpret_cast<volatile int*>(&xw.any_odd[slot]) = 1;
          };
          const int next = in_tile(p_first + 1);
          look_at_rows<D>(tile, old, leave, lane, note);
          look_at_rows<D>(tile, next, min(low, end), lane, note);  // (first tokens behind the first query)
          look_at_rows<D>(tile, max(next, leave), end, lane, note);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&xw.v_ready[st]);
            mbar_arrive(&v_empty[st]);
          }
        }
      }
    }
  } else if (warp > kMmaWarp) {
    regs_dec<kOther>();  // idle: give the registers to the softmax groups
  } else {
    // ------------------------------------------------------------ softmax groups
    regs_inc<KV8 ? kRegsSoftmax8 : WINDOW || SHARED ? kRegsSoftmaxU : kRegsSoftmax>();
    const int w = warp >> 2;                    // query tile of this group
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_tmem = lane_base + w * kKvTile;
    const uint32_t o_tmem = lane_base + 2 * kKvTile + w * D;
    const float sl2 = p.scale_log2;
    // max of sl2 * s = |sl2| * max(sgn * s); a zero scale makes every visible score zero (uniform weights)
    const float sgn = sl2 < 0.f ? -1.f : sl2 > 0.f ? 1.f : 0.f;
    // > 0, so that a hidden key's -inf stays -inf (8-bit cache: the tile's factors are held above zero)
    const float asl2 = sl2 != 0.f ? fabsf(sl2) : KV8 ? 0.f : 1.f;
    // windows: rows in 32-byte stores where out allows them (whole sectors: half the time of 16-byte ones)
    [[maybe_unused]] const bool wide_out = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    uint32_t ns = 0, npv = 0, k = 0;            // s_full phases consumed, PVs of this group, units read
    bool ok = true;
    Unit it;
    // 8-bit cache: a unit is taken, and its query rows are split, before the unit in front
    // of it is written out, so that the tensor cores have the next QK meanwhile.
    [[maybe_unused]] uint32_t t_base = 0, n_split = 0;  // K/V tiles of the units before, query tiles split
    [[maybe_unused]] float row_factor = 0.f, next_factor = 0.f;  // |sl2| without the query row's scaling
    [[maybe_unused]] int nan_slot = 0;                           // of the unit in hand
    [[maybe_unused]] bool have = false;
    [[maybe_unused]] Unit next;
    [[maybe_unused]] auto advance = [&]() {
      have = next_unit(k, next) > 0;
      if (!have || (w ? next.n1 : next.n0) == 0) return;
      if (!wait_all(&x8.q_raw[w], n_split & 1)) {
        ok = false;
        return;
      }
      ++n_split;
      next_factor = asl2 * split_query_row<D>(sQ + w * Sh::kQBytes, row);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x8.q_full[w]);
    };
    if constexpr (KV8) advance();
    auto take = [&]() -> bool {
      if constexpr (KV8) {
        it = next;
        row_factor = next_factor;
        nan_slot = (k - 1) % kNanUnits;
        return have;
      } else {
        return next_unit(k, it) > 0;
      }
    };
    while (ok && take()) {
      const int nkv = w ? it.n1 : it.n0;
      [[maybe_unused]] const uint32_t t0 = t_base;
      t_base += it.n_kv;
      if (nkv == 0) {                           // no second query tile in this unit
        if constexpr (KV8) advance();
        continue;
      }
      const int L = it.L - pf_first(it) * kKvTile, q_len = it.q_len;  // positions from the unit's first key on
      const int hh = row / p.Tq;
      const int qi0 = (2 * it.pair + w) * p.Tq;
      const int qi = qi0 + (row - hh * p.Tq);
      const bool row_valid = qi < q_len;
      // position of the tile's first query token (shared prefixes: every row sees every key)
      const int p_min = SHARED ? L - 1 : L - q_len + qi0;
      const int p_max = SHARED ? L - 1 : L - q_len + min(q_len - 1, qi0 + p.Tq - 1);
      const int p_row = row_valid && !SHARED ? (L - q_len + qi) : p_max;
      // (windows: a row may see no key of its first tiles; a part of a shared prefix may hold none
      // with a score within fp32's range)
      float m_run = WINDOW || SHARED ? kNoScore : -INFINITY, l_run = 0.f;
      for (int j = 0; j < nkv; ++j) {
        if (!wait_all(&s_full[w], ns & 1)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after_sync();
        const int tok0 = pf_tile(it, j) * kKvTile;
        // Visible keys of this row in this tile form a prefix: t <= p_row.
        const int vis = tok0 + kKvTile - 1 > p_min ? min(max(p_row - tok0 + 1, 0), kKvTile) : kKvTile;
        // (windows: but for the keys [hole, hole + hole_len))
        [[maybe_unused]] int hole = 0, hole_len = 0;
        if constexpr (WINDOW) {
          hole = min(max(it.w.sinks - tok0, 0), kKvTile);
          hole_len = max(min(max(p_row - p.window + 1, 0) - tok0, kKvTile) - hole, 0);
        }
        const bool lean = vis == kKvTile && sgn > 0.f && hole_len == 0;   // the common case: no mask, positive scale
        // the row's 128 scores, read once
        uint32_t sv[kKvTile];
#pragma unroll
        for (int c = 0; c < kKvTile; c += 32) tmem_ld32(s_tmem + c, sv + c);
        tmem_ld_wait();
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = -INFINITY;
        if (WINDOW || SHARED) {
          // the same (below) in pieces: of most tiles with hidden keys, one or two of the four need a look
          if (!lean) {
            if (sgn <= 0.f) {
#pragma unroll
              for (int c = 0; c < kKvTile; ++c) sv[c] = __float_as_uint(__uint_as_float(sv[c]) * sgn);
            }
#pragma unroll
            for (int q = 0; q < kKvTile; q += 32) {
              if (vis < q + 32) {
#pragma unroll
                for (int c = q; c < q + 32; ++c)
                  if (c >= vis) sv[c] = 0xff800000u;
              }
              if (WINDOW && hole_len > 0 && hole < q + 32 && hole + hole_len > q) {
#pragma unroll
                for (int c = q; c < q + 32; ++c)
                  if ((unsigned)(c - hole) < (unsigned)hole_len) sv[c] = 0xff800000u;
              }
            }
          }
        } else if (!lean) {
          // fold the mask (a select: NaN-safe) and a negative scale's sign into the
          // scores once, so that one code path serves every tile
#pragma unroll
          for (int c = 0; c < kKvTile; ++c)
            sv[c] = c < vis ? __float_as_uint(__uint_as_float(sv[c]) * sgn) : 0xff800000u;
        }
        [[maybe_unused]] float fac[8];  // 8-bit cache: log2 units per unit of S, for each 16 tokens
        float m_new;
        if constexpr (KV8) {
          // (written before the K tile's barrier, which the UMMA issuer waited for before S)
          const float4 f0 = x8.ks[(t0 + j) % kKScaleSlots][0], f1 = x8.ks[(t0 + j) % kKScaleSlots][1];
          const float ks[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) fac[i] = ks[i] * row_factor;
          if (!lean) {
            // > 0, so that a hidden key's -inf stays -inf; NaN passes for keys that are seen
#pragma unroll
            for (int i = 0; i < 8; ++i) fac[i] = 16 * i < vis ? max_nan(fac[i], 1.17549435e-38f) : 1.f;
          }
          float top = m_run;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float g = mx[i];
#pragma unroll
            for (int c = 16 * i; c < 16 * i + 16; c += 2) g = max3f(g, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            mx[i] = g * fac[i];
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) top = max3f(top, mx[i], mx[i + 1]);
          m_new = top;
        } else {
#pragma unroll
          for (int c = 0; c < kKvTile; c += 2)
            mx[(c >> 1) & 7] = max3f(mx[(c >> 1) & 7], __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
          const float mxa = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
          m_new = fmaxf(m_run, mxa == -INFINITY ? -INFINITY : mxa * asl2);
        }
        const bool grow = m_new > m_run + 8.0f;   // rescale only when the max grew past 2^8
        float alpha = 1.f;
        if (grow) {
          alpha = exp2_approx(m_run - m_new);
          m_run = m_new;
        }
        if (j >= 1 && __any_sync(0xffffffffu, grow)) {
          // PV_w_{j-1} has completed: it was issued before QK_w_j, whose result we hold
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_tmem + c * 32, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(o_tmem + c * 32, ov);
          }
        }
        l_run *= alpha;
        // P = exp2(s * |sl2| - m) as bf16 pairs (2^-8 of each weight: V is bf16, and the two have one type in the
        // instruction; the row sum is of the fp32 weights; even token in the low half), packed in
        // place into sv[0, 64) and stored over the first 64 columns of S_w
        const float neg_m = -m_run;
        uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};   // row sums, as packed pairs
        const uint64_t asl2_2 = f2_pack(asl2, asl2), neg_m2 = f2_pack(neg_m, neg_m);
        // per pair: one packed FMA, two exponentials, one packed add, one bf16x2 convert
        // (a hidden key is -inf here and m_run is finite: without windows after tile 0, where every row sees
        // key 0: its exponential is exactly 0)
#pragma unroll
        for (int c = 0; c < kKvTile; c += 2) {
          float x0, x1;
          const uint64_t f2 = KV8 ? f2_pack(fac[KV8 ? c >> 4 : 0], fac[KV8 ? c >> 4 : 0]) : asl2_2;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), f2, neg_m2), x0, x1);
          const float e0 = exp2_approx(x0);
          const float e1 = exp2_approx(x1);
          ls2[(c >> 1) & 3] = f2_add(ls2[(c >> 1) & 3], f2_pack(e0, e1));
          sv[c >> 1] = pack_bf16x2(e0, e1);
        }
        tmem_st32(s_tmem, sv);
        tmem_st32(s_tmem + 32, sv + 32);
        float ls[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(ls2[i], ls[2 * i], ls[2 * i + 1]);
        l_run += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&p_full[w]);
      }
      if (!ok) break;
      if constexpr (KV8) {
        advance();
        if (!ok) break;
      }
      npv += nkv;
      if (!wait_all(&pv_done[w], (npv - 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const float inv = 1.0f / l_run;
      const int head = it.g * p.r + hh;
      __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(p.out) + ((size_t)(it.q0 + qi) * p.H + head) * D;
      if constexpr (SPLIT) {
        const int tag = *reinterpret_cast<volatile int*>(&x8.tag[nan_slot]);
        if (tag) {
          const int rest = __ldcg(p.item_count) * p.G - __ldcg(p.splits).y;
          write_part<D>(p, tag, rest, w, row, o_tmem, inv, m_run + log2f(l_run), x8.nan_any[nan_slot] != 0,
                        x8.nan_first[nan_slot], p_row - (L - q_len + 2 * it.pair * p.Tq));
          tc_fence_before_sync();  // O_w may be overwritten
          join_parts<D>(p, tag, rest, w, row, lane, row_valid ? orow : nullptr,
                        row_valid && p.lse_out ? p.lse_out + (size_t)(it.q0 + qi) * p.H + head : nullptr);
          continue;
        }
      }
      if constexpr (SHARED) {
        if (threadIdx.x == 0) {
          int2* unit = p.unit_parts + (it.part - blockIdx.x);
          if (it.j0 == 0) unit->x = it.part;
          if (it.j0 + it.n_kv == (it.L - 1) / kKvTile + 1) unit->y = it.part;
        }
        const size_t at = ((size_t)it.part * 2 + w) * kRows + row;
        float* to = p.part_out + at * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(o_tmem + c * 32, ov);
          tmem_ld_wait();
          if (row_valid) {
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * inv);
#pragma unroll
            for (int i = 0; i < 32; i += 8) st_global_v8(to + c * 32 + i, ov + i);
          }
        }
        if (row_valid) p.part_lse[at] = m_run + log2f(l_run);
      }
      if constexpr (WINDOW) {
        const int slot = (k - 1) & 1;
        if (*reinterpret_cast<volatile int*>(&xw.any_odd[slot]))
          add_odd_tokens<D>(p, it, xw.odd[slot], o_tmem,
                            row_valid ? reinterpret_cast<const __nv_bfloat16*>(p.q) + ((size_t)(it.q0 + qi) * p.H + head) * D
                                      : nullptr,
                            p_row, m_run);
      }
#pragma unroll 1
      for (int c = 0; c < (SHARED ? 0 : D / 32); ++c) {
        uint32_t ov[32];
        tmem_ld32(o_tmem + c * 32, ov);
        tmem_ld_wait();
        if (row_valid) {
          if (WINDOW && wide_out) {
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[e] = pack_bf16x2(__uint_as_float(ov[i + 2 * e]) * inv, __uint_as_float(ov[i + 2 * e + 1]) * inv);
              st_global_v8(orow + c * 32 + i, v);
            }
            continue;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 v;
            v.x = pack_bf16x2(__uint_as_float(ov[i]) * inv, __uint_as_float(ov[i + 1]) * inv);
            v.y = pack_bf16x2(__uint_as_float(ov[i + 2]) * inv, __uint_as_float(ov[i + 3]) * inv);
            v.z = pack_bf16x2(__uint_as_float(ov[i + 4]) * inv, __uint_as_float(ov[i + 5]) * inv);
            v.w = pack_bf16x2(__uint_as_float(ov[i + 6]) * inv, __uint_as_float(ov[i + 7]) * inv);
            *reinterpret_cast<uint4*>(orow + c * 32 + i) = v;
          }
        }
      }
      if constexpr (KV8) {
        if (*reinterpret_cast<volatile int*>(&x8.nan_any[nan_slot]) && row_valid) {
          const int rel = p_row - (L - q_len + 2 * it.pair * p.Tq);
#pragma unroll 1
          for (int d = 0; d < D; ++d)
            if (x8.nan_first[nan_slot][d] <= rel) orow[d] = __ushort_as_bfloat16(0x7fff);
        }
      }
      if (row_valid && p.lse_out) p.lse_out[(size_t)(it.q0 + qi) * p.H + head] = (m_run + log2f(l_run)) * kLn2;
      // the next unit's first PV_w overwrites O_w: every lane has read it
      tc_fence_before_sync();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (p.wait_at_exit) pdl_wait();  // complete only after the decode grid in front of this one
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int prefill_status(uint32_t* bits, int clear) {
  unsigned int v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_status_prefill, sizeof(v));
  if (e == cudaSuccess && clear) {
    unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_status_prefill, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  *bits |= v;
  return METIS_OK;
}

// (sequence, query-tile pair) items: at most ceil(T / (2 Tq)) + S
static size_t prefill_max_items(int num_seqs, int num_tokens, int Tq) {
  return (size_t)(num_tokens + 2 * Tq - 1) / (2 * Tq) + (size_t)num_seqs;
}

// 8-bit cache: memory for parts of units, behind the item list: counters, lse and rows.
static size_t prefill_split_offset(size_t max_items) { return align_up(256 + max_items * sizeof(int4), 256); }

static size_t prefill_split_bytes(int parts, int D) {
  return align_up((size_t)parts * 2 * (kRows / 32) * sizeof(int), 256) + (size_t)parts * 2 * kRows * (1 + D) * sizeof(float);
}

// ... for how many parts.  None where the chunks' units (all of one sequence, as far as the
// host knows) fill two rounds of the SMs, would not be split, or the sequences are short.
static int prefill_max_parts(int num_tokens, int Tq, int G, int cap, int sms) {
  const long long units = (long long)std::max(1, num_tokens / (2 * Tq)) * G;
  if (units >= 2 * sms) return 0;
  const int parts = 2 * units <= sms ? sms : 4 * sms;
  return pf_splits(units, sms, (cap - 1) / kKvTile + 1, parts) > 1 ? parts : 0;
}

// The schedule kernel, then `between(p)` (the decodes of a mixed batch, or
// nothing), then the chunk kernel.
template <int D, bool KV8, bool SPLIT, bool WINDOW, bool SHARED, typename Between>
static int launch_prefill(const PrefillParams& p0, const void* q, const void* k_cache, const void* v_cache,
                          void* workspace, size_t max_items, int sms, cudaStream_t st, Between between) {
  PrefillParams p = p0;
  int* count = reinterpret_cast<int*>(workspace);
  int4* items = reinterpret_cast<int4*>(reinterpret_cast<char*>(workspace) + 256);
  p.items = items;
  p.item_count = count;
  p.unit_head = count + 1;
  if (p.skip_decodes && !SHARED) {
    p.dec_ctas = count + 2;
    p.dec_next = count + 3;
    p.wait_at_exit = 1;
  }
  if (SPLIT) {
    char* at = reinterpret_cast<char*>(workspace) + prefill_split_offset(max_items);
    p.splits = reinterpret_cast<int2*>(count + 4);
    p.parts_done = reinterpret_cast<int*>(at);
    at += align_up((size_t)p.max_parts * 2 * (kRows / 32) * sizeof(int), 256);
    p.part_lse = reinterpret_cast<float*>(at);
    at += (size_t)p.max_parts * 2 * kRows * sizeof(float);
    p.part_out = reinterpret_cast<float*>(at);
  }
  p.num_sms = sms;
  p.D = D;
  p.kv_token_bytes = 2 * p.G * D * (KV8 ? 1 : 2);
  CUtensorMap tmQ, tmK, tmV;
  const uint64_t qdims[3] = {(uint64_t)D, (uint64_t)p.H, (uint64_t)p.T};
  const uint64_t qstr[2] = {(uint64_t)D * 2, (uint64_t)p.H * D * 2};
  const uint32_t qbox[3] = {64, 1, (uint32_t)p.Tq};
  int rc = encode_tiled(&tmQ, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, qdims, qstr, qbox, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  const uint64_t kdims[3] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.num_blocks * p.bs};
  constexpr uint64_t kElem = KV8 ? 1 : 2;
  const uint64_t kstr[2] = {D * kElem, (uint64_t)p.G * D * kElem};
  const uint32_t kbox[3] = {KV8 ? D : 64, 1, (uint32_t)p.bs};
  const CUtensorMapDataType kind = KV8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle k_sw = KV8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  rc = encode_tiled(&tmK, kind, 3, k_cache, kdims, kstr, kbox, k_sw);
  if (rc) return rc;
  // staged V codes are read back row by row: plain rows
  rc = encode_tiled(&tmV, kind, 3, v_cache, kdims, kstr, kbox, KV8 ? CU_TENSOR_MAP_SWIZZLE_NONE : k_sw);
  if (rc) return rc;
  // a programmatic dependent of the kernel before it (e.g. the paged K/V write): its
  // launch overlaps that kernel's tail
  if (!SHARED) {
    rc = launch_dependent(prefill_schedule_kernel, dim3(1), dim3(kSchedThreads), 0, st, "prefill_schedule_kernel launch",
                          p, items, count, (int)max_items);
    if (rc) return rc;
  }
  rc = between(p);
  if (rc) return rc;
  constexpr int smem = PfShape<D, KV8>::kSmem;
  static int done = 0;
  auto kern = prefill_bf16_kernel<D, KV8, SPLIT, WINDOW, SHARED>;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem, &done);
  if (rc) return rc;
  // the warpgroups' register targets draw on the launch allocation: refuse to launch
  // a build whose allocation is smaller (the raising warps would wait forever)
  static int regs_checked = 0;
  if (!regs_checked) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, reinterpret_cast<const void*>(kern));
    if (e != cudaSuccess) return fail(METIS_E_CUDA, "cudaFuncGetAttributes: %s", cudaGetErrorString(e));
    if (fa.numRegs < kRegsLaunch)
      return fail(METIS_E_CUDA, "prefill kernel built with %d registers per thread, %d needed", fa.numRegs,
                  kRegsLaunch);
    regs_checked = 1;
  }
  // persistent: at most one CTA per SM, each taking units from the list as it goes
  // (beside the decodes: the CTAs past the SMs they keep start as their CTAs finish)
  const size_t grid = SPLIT || SHARED ? (size_t)sms : std::min<size_t>(max_items * p.G, (size_t)std::max(sms, 1));
  return launch_dependent(kern, dim3((unsigned)grid), dim3(kPfThreads), smem, st, "prefill_bf16_kernel launch", tmQ,
                          tmK, tmV, p);
}

}  // namespace metis

using namespace metis;

extern "C" size_t metis_prefill_workspace_bytes(int num_seqs, int num_tokens, int num_heads, int num_kv_heads) {
  if (num_seqs <= 0 || num_tokens <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads) return 0;
  const int r = num_heads / num_kv_heads;
  if (r > kRows) return 0;
  return 256 + prefill_max_items(num_seqs, num_tokens, kRows / r) * sizeof(int4);
}

extern "C" size_t metis_prefill_fp8_workspace_bytes(int num_seqs, int num_tokens, int num_heads, int num_kv_heads,
                                                    int head_dim, int max_seq_len) {
  const size_t need = metis_prefill_workspace_bytes(num_seqs, num_tokens, num_heads, num_kv_heads);
  if (!need || (head_dim != 64 && head_dim != 128) || max_seq_len <= 0) return need;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return need;
  }
  const int Tq = kRows / (num_heads / num_kv_heads);
  const int parts = prefill_max_parts(num_tokens, Tq, num_kv_heads, max_seq_len, sms);
  if (!parts) return need;
  return prefill_split_offset(prefill_max_items(num_seqs, num_tokens, Tq)) + prefill_split_bytes(parts, head_dim);
}

namespace metis {

// Both entry points: fp8.k_cache is NULL for a bf16 cache, else k_cache and the codes are one.
static int prefill_chunk(const void* q, const int32_t* cu_q_lens, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse_out, int num_seqs,
                         int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size, int max_blocks,
                         int num_blocks, int dtype, float scale, int max_seq_len, void* workspace,
                         size_t workspace_bytes, void* stream, const Fp8Cache& fp8, int window = 0, int sinks = 0) {
  if (num_seqs < 0 || num_tokens < 0) return fail(METIS_E_SHAPE, "num_seqs and num_tokens must be >= 0");
  if (num_seqs == 0 || num_tokens == 0) return METIS_OK;
  if (!q || !cu_q_lens || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return fail(METIS_E_NULL, "q, cu_q_lens, k_cache, v_cache, block_table, seq_lens and out are required");
  if (num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks <= 0 ||
      num_blocks <= 0 || max_seq_len <= 0)
    return fail(METIS_E_SHAPE, "sizes must be positive");
  if (num_heads % num_kv_heads) return fail(METIS_E_SHAPE, "num_heads %% num_kv_heads != 0");
  if ((long long)max_blocks * block_size > 0x7fffffffLL || (long long)num_blocks * block_size > 0x7fffffffLL)
    return fail(METIS_E_SHAPE, "max_blocks * block_size and num_blocks * block_size must fit in int32");
  if (dtype != METIS_BF16) return fail(METIS_E_UNSUPPORTED, "prefill is built for bf16");
  if (head_dim != 64 && head_dim != 128) return fail(METIS_E_UNSUPPORTED, "head_dim must be 64 or 128");
  if (block_size != 16 && block_size != 32 && block_size != 64)
    return fail(METIS_E_UNSUPPORTED, "block_size must be 16, 32 or 64");
  const int r = num_heads / num_kv_heads;
  if (r != 1 && r != 2 && r != 4 && r != 8 && r != 16)
    return fail(METIS_E_UNSUPPORTED, "num_heads / num_kv_heads must be 1, 2, 4, 8 or 16");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(cu_q_lens, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse_out, 4))
    return fail(METIS_E_ALIGN, "tensors must be 16-byte aligned (index arrays and lse_out: 4-byte)");
  if (!(scale == scale)) return fail(METIS_E_SHAPE, "scale is NaN");
  const size_t need = metis_prefill_workspace_bytes(num_seqs, num_tokens, num_heads, num_kv_heads);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
    return fail(METIS_E_WORKSPACE, "workspace must hold %zu bytes (256-byte aligned)", need);
  const size_t max_items = prefill_max_items(num_seqs, num_tokens, kRows / r);
  if (max_items * num_kv_heads > 0x7fffffffull) return fail(METIS_E_SHAPE, "too many query tiles");

  PrefillParams p{};
  p.cu_q_lens = cu_q_lens;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.lse_out = lse_out;
  p.S = num_seqs;
  p.T = num_tokens;
  p.H = num_heads;
  p.G = num_kv_heads;
  p.r = r;
  p.Tq = kRows / r;
  p.bs = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.cap = (int)std::min<long long>((long long)max_blocks * block_size, (long long)max_seq_len);
  p.scale_log2 = scale * kLog2e;
  p.window = window;
  p.sinks = sinks;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // Single-token sequences (the decodes of a mixed batch) go through the decode
  // kernel, which streams their K/V at the memory rate (a 128-row query tile would
  // hold r valid rows of them).  It runs beside the chunk kernel: the schedule
  // kernel gives it a share of the SMs in proportion to the decodes' bytes against
  // the chunks' FLOPs, its other CTAs exit at once, and the chunk kernel -- launched
  // behind it, which it allows only after its CTAs waited for the schedule -- takes
  // the remaining SMs at once and the decodes' SMs as they finish.  Head ratios
  // above 8 stay on the chunk path.
  p.fp8 = fp8;
  p.skip_decodes = r <= 8 && num_seqs <= 65535;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "querying the SM count: %s", cudaGetErrorString(e));
  sms = std::max(sms, 1);
  auto between = [&](const PrefillParams& pp) -> int {
    if (!pp.skip_decodes) return METIS_OK;
    if (fp8.k_cache)
      return launch_decode_fp8_rows_beside(q, fp8, block_table, seq_lens, cu_q_lens, num_tokens, out, lse_out, num_seqs,
                                           num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks,
                                           scale, pp.cap, pp.dec_ctas, pp.dec_next, sms, st);
    return launch_decode_rows_beside(q, k_cache, v_cache, block_table, seq_lens, cu_q_lens, num_tokens, out, lse_out,
                                     num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks,
                                     scale, pp.cap, window, sinks, pp.dec_ctas, pp.dec_next, sms, st);
  };
  auto launch = [&](auto dim, auto kv8, auto split, auto windowed) {
    return launch_prefill<decltype(dim)::value, decltype(kv8)::value, decltype(split)::value,
                          decltype(windowed)::value, false>(p, q, k_cache, v_cache, workspace, max_items, sms, st, between);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  using Yes = std::true_type;
  using No = std::false_type;
  if (window) return head_dim == 128 ? launch(D128{}, No{}, No{}, Yes{}) : launch(D64{}, No{}, No{}, Yes{});
  if (!fp8.k_cache) return head_dim == 128 ? launch(D128{}, No{}, No{}, No{}) : launch(D64{}, No{}, No{}, No{});
  p.max_parts = prefill_max_parts(num_tokens, p.Tq, num_kv_heads, p.cap, sms);
  if (p.max_parts > 0 &&
      workspace_bytes >= prefill_split_offset(max_items) + prefill_split_bytes(p.max_parts, head_dim))
    return head_dim == 128 ? launch(D128{}, Yes{}, Yes{}, No{}) : launch(D64{}, Yes{}, Yes{}, No{});
  return head_dim == 128 ? launch(D128{}, Yes{}, No{}, No{}) : launch(D64{}, Yes{}, No{}, No{});
}

}  // namespace metis

namespace metis {

// The parts of the shared prefixes of a batch of decodes (shared_prefix.cu).
int launch_shared_prefix(const SharedArgs& a, SharedPlan* plan, SharedOwn* own, int2* unit_parts, float* part_lse,
                         float* part_out, int sms, cudaStream_t st) {
  PrefillParams p{};
  p.cu_q_lens = a.cu_group_seqs;
  p.prefix_lens = a.prefix_lens;
  p.num_groups = a.num_groups;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.S = p.T = a.S;
  p.H = a.H;
  p.G = a.G;
  p.r = a.H / a.G;
  p.Tq = kRows / p.r;
  p.bs = a.bs;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.cap = a.cap;
  p.scale_log2 = a.scale * kLog2e;
  p.plan = plan;
  p.own = own;
  p.unit_parts = unit_parts;
  p.kv_token_bytes = 4 * a.G * a.D;
  p.part_lse = part_lse;
  p.part_out = part_out;
  auto none = [](const PrefillParams&) { return METIS_OK; };
  return a.D == 128 ? launch_prefill<128, false, false, false, true>(p, a.q, a.k_cache, a.v_cache, part_out, 0, sms, st, none)
                    : launch_prefill<64, false, false, false, true>(p, a.q, a.k_cache, a.v_cache, part_out, 0, sms, st, none);
}

}  // namespace metis

extern "C" int metis_paged_attn_prefill_chunk(const void* q, const int32_t* cu_q_lens, const void* k_cache,
                                              const void* v_cache, const int32_t* block_table,
                                              const int32_t* seq_lens, void* out, float* lse_out, int num_seqs,
                                              int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                              int block_size, int max_blocks, int num_blocks, int dtype, float scale,
                                              int max_seq_len, void* workspace, size_t workspace_bytes,
                                              void* stream) {
  clear_error();
  return prefill_chunk(q, cu_q_lens, k_cache, v_cache, block_table, seq_lens, out, lse_out, num_seqs, num_tokens,
                       num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks, dtype, scale, max_seq_len,
                       workspace, workspace_bytes, stream, Fp8Cache{});
}

extern "C" int metis_paged_attn_prefill_chunk_window(const void* q, const int32_t* cu_q_lens, const void* k_cache,
                                                     const void* v_cache, const int32_t* block_table,
                                                     const int32_t* seq_lens, void* out, float* lse_out, int num_seqs,
                                                     int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                                     int block_size, int max_blocks, int num_blocks, int dtype,
                                                     float scale, int window, int sinks, int max_seq_len,
                                                     void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  if (num_seqs > 0 && num_tokens > 0 && (window <= 0 || sinks < 0))
    return fail(METIS_E_SHAPE, "window must be positive and sinks >= 0");
  return prefill_chunk(q, cu_q_lens, k_cache, v_cache, block_table, seq_lens, out, lse_out, num_seqs, num_tokens,
                       num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks, dtype, scale, max_seq_len,
                       workspace, workspace_bytes, stream, Fp8Cache{}, window, sinks);
}

extern "C" int metis_paged_attn_prefill_chunk_fp8(const void* q, const int32_t* cu_q_lens, const void* k_cache,
                                                  const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                                                  const int32_t* block_table, const int32_t* seq_lens, void* out,
                                                  float* lse_out, int num_seqs, int num_tokens, int num_heads,
                                                  int num_kv_heads, int head_dim, int block_size, int max_blocks,
                                                  int num_blocks, int dtype, float scale, int max_seq_len,
                                                  void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  if (num_seqs > 0 && num_tokens > 0 && (!k_cache || !k_scale || !v_scale))
    return fail(METIS_E_NULL, "k_cache, k_scale and v_scale are required");
  return prefill_chunk(q, cu_q_lens, k_cache, v_cache, block_table, seq_lens, out, lse_out, num_seqs, num_tokens,
                       num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks, dtype, scale, max_seq_len,
                       workspace, workspace_bytes, stream, Fp8Cache{k_cache, v_cache, k_scale, v_scale});
}
