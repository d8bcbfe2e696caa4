// Decode items one after another on a warp of its own, its loads running on across them: for many items of
// few tokens each, where a CTA per item would spend its time on starting (lengths, block ids, the first
// loads) and joining its warps.  512 windows of 128 tokens on 8 KV heads (268 MB): 54 us, 5.0 TB/s, where a
// CTA per item takes 81.  What is lost to the copy rate goes with the number of items, at equal boxes per byte (windows
// of 64 tokens 4.5 TB/s, 128 5.0, 500 6.3): an item's length, table entries and query are loads in series, of which
// only the first two run ahead of the item in hand.
#pragma once

#include "decode_items.cuh"

namespace metis {

// kStreamWarps warps of a CTA, each with a ring of stages of its own: 192 KB in flight on an SM.
constexpr int kStreamWarps = 8;
template <int D>
constexpr int stream_stages() {
  return D == 128 ? 3 : 6;
}
template <int D>
constexpr int stream_smem_bytes() {
  return bf16_decode_smem_bytes<D, kStreamWarps, stream_stages<D>()>();
}

// An item: the units of `span` of KV head g of sequence s.  part: the caller's.
struct StreamItem {
  int s, g, part, n;  // n: its units (0: no item)
  WindowSpan span;
  int row0, row1;     // lane l: TMA rows of the units 32 b + l and 32 (b + 1) + l, b the window being issued
};

// The warp's walk over the items that next(item) hands it (false: no more; called by the whole warp), each
// given to store(item, state) when its units are done.  The units of the item in hand and of the next one are
// issued in one order, so the ring stays full over an item's end.  Returns false when a wait gave up.
template <int D, typename Next, typename Store>
__device__ __forceinline__ bool decode_stream(const CUtensorMap& tmK, const CUtensorMap& tmV, const DecodeParams& p,
                                              uint8_t* ring, uint64_t* bars, int lane, unsigned int* status, Next next,
                                              Store store) {
  using Shape = Bf16DecodeShape<D>;
  constexpr int HALVES = Shape::kHalves, STAGES = stream_stages<D>(), STAGE_BYTES = Shape::kStageBytes;
  const uint64_t policy = l2_policy_evict_first();
  int in_st = 0, out_st = 0, in_flight = 0;  // ring positions of the next load and of the next unit to compute
  uint32_t out_ph = 0;

  // TMA row of the item's unit k; -kUnit (a box outside the tensor, read as zeros) marks a bad block id
  auto row_of = [&](const StreamItem& it, int k) -> int {
    if (k >= it.n) return -kUnit;
    const int tok = it.span.token(k), page = tok / p.bs;
    const int b = checked_block(p.block_table + (size_t)it.s * p.max_blocks, page, p.num_blocks, status);
    return b < 0 ? -kUnit : b * p.bs + (tok - page * p.bs);
  };
  auto fetch = [&](StreamItem& it) {
    if (!next(it)) {
      it.n = 0;
      return;
    }
    it.n = it.span.units();
    it.row0 = row_of(it, lane);
    it.row1 = row_of(it, 32 + lane);
  };
  auto issue = [&](StreamItem& it, int k) {  // in order k = 0, 1, 2, ...
    if (k > 0 && (k & 31) == 0) {
      it.row0 = it.row1;
      it.row1 = row_of(it, k + 32 + lane);
    }
    const int row = __shfl_sync(0xffffffffu, it.row0, k & 31);
    uint8_t* base = ring + in_st * STAGE_BYTES;
    if (lane == 0) mbar_arrive_expect_tx(&bars[in_st], STAGE_BYTES);
    __syncwarp();
    if (lane < 2 * HALVES)
      tma_load_3d(base + lane * kBoxBytes, lane < HALVES ? &tmK : &tmV, &bars[in_st], (lane % HALVES) * 64, it.g, row,
                  policy);
    if (++in_st == STAGES) in_st = 0;
    ++in_flight;
  };

  StreamItem now, then;
  int now_k = 0, then_k = 0;  // units issued of each
  fetch(now);
  while (now_k < now.n && in_flight < STAGES) issue(now, now_k++);
  bool ok = true;
  DecodeWarp<D> state;
  while (now.n > 0) {
    state.begin(p, now.s, now.g, lane);
    fetch(then);
    then_k = 0;
    while (then_k < then.n && in_flight < STAGES) issue(then, then_k++);  // (only behind the last unit of `now`)
    for (int k = 0; k < now.n; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[out_st], out_ph, status));  // leave the loop together
      if (!ok) break;
      state.unit(smem_u32(ring + out_st * STAGE_BYTES), now.span.token(k), now.span, p.scale_log2, lane);
      __syncwarp();
      if (++out_st == STAGES) out_st = 0, out_ph ^= 1;
      --in_flight;
      if (now_k < now.n)
        issue(now, now_k++);
      else if (then_k < then.n)
        issue(then, then_k++);
    }
    if (!ok) break;
    store(now, state);
    now = then;
    now_k = then_k;
  }
  if (!ok) {
    // let this warp's loads still in flight land (bounded) before the memory goes away
    for (; in_flight > 0; --in_flight) {
      mbar_wait(&bars[out_st], out_ph, status);
      if (++out_st == STAGES) out_st = 0, out_ph ^= 1;
    }
  }
  return ok;
}

}  // namespace metis
