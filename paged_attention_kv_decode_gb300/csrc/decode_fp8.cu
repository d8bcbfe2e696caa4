// Decode attention over an 8-bit paged cache: e4m3 codes with one power-of-two scale per
// page and KV head (cache_fp8.cu writes it).  For query head h over its KV head g
//
//   z_t = scale * 2^kb(t) * (q_h . code_K(t)),  out = sum_t softmax(z)_t 2^vb(t) code_V(t)
//
// with kb, vb the scale exponents of the page that holds token t.
//
// Memory-bound: 2 G D bytes per cached token against 4 H D operations.  The structure is
// that of the bf16 kernel in decode.cu -- one CTA per (partition, KV head, sequence), the
// group's query heads share each K/V byte, each warp fills a private ring with TMA tile
// loads and keeps its own softmax state -- with what the codes change:
//
//   * A unit is 32 tokens (two m16 tiles): at one byte per element the 16-token units of
//     the bf16 kernel would halve the bytes behind each softmax step.
//   * Codes become fp16 in registers (cvt.e4m3x2 -> f16x2, exact); the products are fp16
//     mma.sync with fp32 accumulation (an e4m3 mma.sync runs as the same conversions and fp16
//     products, of more operands: 13 % slower).  K: a 32-bit piece of ldmatrix holds four
//     consecutive dims of a token, so dims are dealt to the k-slots in that order and the
//     query is loaded to match.  V: ldmatrix.trans of 16-bit pairs gives {two dims} x {two
//     tokens}; one byte permute splits it into the even and the odd dim's token pair, so an
//     m16 tile of output rows is 8 even dims followed by 8 odd ones.
//   * The query row is scaled by a power of two into fp16's range (its largest element in
//     [2^14, 2^15)): exact for bf16 elements down to 2^-29 of the largest, and below that
//     off by at most 2^-39 of it.  fp32 queries are split into two fp16 parts (22 bits).
//   * bf16 queries: a token's weight takes V's page scale along, 2^(z + vb - M), so that P V
//     accumulates straight into O; its reference M, the running maximum of z + vb minus 14,
//     leaves fp16 the range down to 2^-38 of the largest.  M follows the pages' scales, not the
//     values that the weights meet: a page 2^kWide below the largest one so far would lose
//     weights that count in columns where the large page holds zeros.  Its weights are of z
//     alone, each tile against its own maximum, and its products join O in fp32 with the page's
//     factor.  So a weight is off by at most 2^-11 of itself or 2^-27 of the largest one.  The
//     sum of weights has a reference of its own, m, of z alone.
//   * fp32 queries: weights are two fp16 parts too, and each tile's P V lands in a fresh
//     accumulator that joins O with the page's factor.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "../../include/metis_attn.h"
#include "cluster.cuh"
#include "common.cuh"
#include "decode.cuh"
#include "fp8.cuh"
#include "host.h"

namespace metis {

__device__ unsigned int g_status_decode_fp8 = 0;

struct DecodeFp8Params {
  DecodeParams d;
  const uint8_t* k_scale;  // [num_blocks, G]
  const uint8_t* v_scale;
};

constexpr int kUnit8 = 32;       // tokens per pipeline unit (two m16 tiles)
constexpr float kRefDown = 14.f; // softmax reference below the running maximum, log2 units
constexpr float kUndoRefDown = 1.f / 16384.f;  // 2^-kRefDown
constexpr int kMaxJoin = 8;          // partitions of an item that a cluster takes
constexpr int kMinJoinTokens = 128;  // ... in a call that asked for none: tokens in each at least
// bf16 queries: a page whose V scale is further than this (log2) below the largest so far keeps it
// out of its weights, which costs a weight 2^-(39 - kWide) of the largest at most
constexpr int kWide = 12;
constexpr float kSlack = 16.f;   // bf16 queries: the sums' reference moves when it is exceeded by 2^16

template <int D>
struct Fp8DecodeShape {
  static constexpr int kTileBytes = kUnit8 * D;     // K or V of one unit
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kSteps = D / 16;             // 16-dim chunks of a row
};

template <int D, int NW, int STAGES>
constexpr int fp8_decode_smem_bytes() {
  return 1024 + NW * STAGES * (Fp8DecodeShape<D>::kStageBytes + 8);
}

// Byte offset of 16-byte chunk c of row `row` in a TMA tile of D-byte rows: 128-byte
// swizzle for 128-byte rows, 64-byte swizzle for 64-byte rows.
template <int D>
__device__ __forceinline__ uint32_t tile_chunk(int row, int c) {
  return row * D + ((c ^ (D == 128 ? (row & 7) : ((row >> 1) & 3))) << 4);
}

// The part of (lo, hi) that fp16 `packed` left over, scaled by 2^11, as fp16
__device__ __forceinline__ uint32_t pack_f16x2_rest(float lo, float hi, uint32_t packed) {
  const float2 v = unpack_f16x2(packed);
  return pack_f16x2((lo - v.x) * 2048.f, (hi - v.y) * 2048.f);
}

// A warp's units of one work item, the tokens [t0, t1) of KV head g of sequence s, and the
// loads of their K and V into the warp's ring.
// Lane l holds unit k = 32 * window + l of the current window: the TMA row of its page(s)
// and the scale bytes (k0, v0, k1, v1); and the block ids of the next window's unit.
// -box (a box outside the tensor, read as zeros) stands for a bad block id or a page past
// the range.  Ids, then loads of K and V, then scales (and the caller's query): the item's
// first bytes wait for one lookup only.
template <int D, int NW, int STAGES>
struct Fp8Units {
  using Shape = Fp8DecodeShape<D>;
  const CUtensorMap *tmK, *tmV;
  const DecodeFp8Params& pp;
  const int32_t* bt_row;
  uint8_t* ring;      // this warp's stages
  uint64_t* bars;
  int g, t1, warp, lane, u0, n_my, box;
  int st;             // stage of the unit to consume, which the unit STAGES later takes
  uint32_t phase;     // ... and the parity of its barrier
  bool small_pages;   // two pages per unit, else part of one
  int cur0, cur1, id0, id1;  // TMA rows of the window being issued, ids of the next one
  uint32_t cur_sc, next_sc;  // scale bytes alike
  uint32_t use_sc;           // scale bytes of the window being consumed
  uint64_t policy;

  __device__ __forceinline__ Fp8Units(const CUtensorMap& tmK_, const CUtensorMap& tmV_, const DecodeFp8Params& pp_,
                                      uint8_t* smem, uint64_t* bars_, int g_, int s, int t0, int t1_, int warp_,
                                      int lane_, int kb)
      : tmK(&tmK_), tmV(&tmV_), pp(pp_), bt_row(pp_.d.block_table + (size_t)s * pp_.d.max_blocks),
        ring(smem + warp_ * STAGES * Shape::kStageBytes), bars(bars_ + warp_ * STAGES), g(g_), t1(t1_), warp(warp_),
        lane(lane_) {
    // this warp's units: u0 + warp + k * NW, k < n_my
    u0 = t0 / kUnit8;
    const int n_units = (t1 - u0 * kUnit8 + kUnit8 - 1) / kUnit8;
    n_my = warp < n_units ? (n_units - warp + NW - 1) / NW : 0;
    st = kb % STAGES;
    phase = (kb / STAGES) & 1;
    small_pages = pp.d.bs == 16;
    box = small_pages ? 16 : kUnit8;
    policy = l2_policy_evict_first();
    int b0, b1;
    load_ids(lane, b0, b1);
    load_ids(32 + lane, id0, id1);
    check_ids(lane, b0, b1);
    set_rows(lane, b0, b1);
    for (int k = 0; k < STAGES && k < n_my; ++k) load(k, (st + k) % STAGES);
    next_sc = 0;
    cur_sc = use_sc = load_scales(b0, b1);
  }

  __device__ __forceinline__ int first_token(int k) const { return (u0 + warp + k * NW) * kUnit8; }
  __device__ __forceinline__ uint32_t tile() const { return smem_u32(ring + st * Shape::kStageBytes); }

  // Scale bytes (k0, v0, k1, v1) of unit k, the next to be consumed (all lanes)
  __device__ __forceinline__ uint32_t scales(int k) {
    // the window being issued is STAGES units ahead: still the same one where a window begins
    if ((k & 31) == 0) use_sc = cur_sc;
    return __shfl_sync(0xffffffffu, use_sc, k & 31);
  }

  // Wait for the next unit (all lanes).  False: the wait gave up.
  __device__ __forceinline__ bool wait() {
    return __all_sync(0xffffffffu, mbar_wait(&bars[st], phase, &g_status_decode_fp8));
  }

  // Unit k is consumed: load the one that takes its stage.
  __device__ __forceinline__ void release(int k) {
    __syncwarp();
    const int n = k + STAGES;
    if (n < n_my) {
      if ((n & 31) == 0) {
        set_rows(n + lane, id0, id1);  // (checked with their scales, half a window ago)
        cur_sc = next_sc;
        load_ids(n + 32 + lane, id0, id1);
      }
      load(n, st);
      if ((n & 31) == 16) {            // the next window's ids are here by now
        check_ids(n + 16 + lane, id0, id1);
        next_sc = load_scales(id0, id1);
      }
    }
    if (++st == STAGES) {
      st = 0;
      phase ^= 1;
    }
  }

  // The wait for unit k gave up: drain the loads still in flight (bounded) before the ring is reused.
  __device__ __forceinline__ void drain(int k) {
    for (int n = k + 1; n < n_my && n < k + STAGES; ++n) {
      if (++st == STAGES) {
        st = 0;
        phase ^= 1;
      }
      mbar_wait(&bars[st], phase, &g_status_decode_fp8);
    }
  }

  __device__ __forceinline__ void load_ids(int k, int& b0, int& b1) const {  // -1: no such page
    b0 = b1 = -1;
    if (k >= n_my) return;
    const int tok = first_token(k);
    b0 = bt_row[tok / pp.d.bs];
    if (small_pages && tok + 16 < t1) b1 = bt_row[tok / 16 + 1];
  }

  __device__ __forceinline__ int check_id(int b, bool wanted) const {  // a bad id (flagged) becomes -1
    if (b >= 0 && b < pp.d.num_blocks) return b;
    if (wanted) atomicOr(&g_status_decode_fp8, METIS_STATUS_BAD_BLOCK_ID);
    return -1;
  }

  __device__ __forceinline__ void check_ids(int k, int& b0, int& b1) const {
    b0 = check_id(b0, k < n_my);
    b1 = check_id(b1, k < n_my && small_pages && first_token(k) + 16 < t1);
  }

  __device__ __forceinline__ void set_rows(int k, int b0, int b1) {  // of the (checked) ids of unit k
    cur0 = b0 < 0 ? -box : b0 * pp.d.bs + first_token(k) % pp.d.bs;
    cur1 = b1 < 0 ? -box : b1 * 16;
  }

  // (k0, v0, k1, v1); a bad page has scale 1, the second page of a unit that has one the first's
  __device__ __forceinline__ uint32_t load_scales(int b0, int b1) const {
    uint32_t sc = 0x7f7fu;
    if (b0 >= 0) {
      const size_t at = (size_t)b0 * pp.d.G + g;
      sc = ld_byte(pp.k_scale + at) | (ld_byte(pp.v_scale + at) << 8);
    }
    sc |= sc << 16;
    if (small_pages && b1 >= 0) {
      const size_t at = (size_t)b1 * pp.d.G + g;
      sc = (sc & 0xffffu) | (ld_byte(pp.k_scale + at) << 16) | (ld_byte(pp.v_scale + at) << 24);
    }
    return sc;
  }

  // K and V of unit k of the current window into a stage (all lanes)
  __device__ __forceinline__ void load(int k, int stage) {
    uint8_t* base = ring + stage * Shape::kStageBytes;
    uint64_t* bar = &bars[stage];
    if (lane == 0) mbar_arrive_expect_tx(bar, Shape::kStageBytes);
    const int r0 = __shfl_sync(0xffffffffu, cur0, k & 31);
    const int r1 = __shfl_sync(0xffffffffu, cur1, k & 31);
    __syncwarp();
    // one box per lane: lanes 0, 1 the K page(s), lanes 2, 3 the V page(s)
    if (lane < 4 && (small_pages || !(lane & 1)))
      tma_load_3d(base + (lane >> 1) * Shape::kTileBytes + (lane & 1) * (16 * D), lane < 2 ? tmK : tmV, bar, 0, g,
                  (lane & 1) ? r1 : r0, policy);
  }
};

// A sum l relative to 2^m (m = -infinity: of nothing) brought into [1, 2)
__device__ __forceinline__ void normalise_sum(float& l, float& m) {
  const int field = (int)((__float_as_uint(l) >> 23) & 255u);
  if (field == 0 || field == 255) return;  // zero or NaN
  l *= __uint_as_float((uint32_t)(254 - field) << 23);
  m += (float)(field - 127);
}

// The warps' softmax states meet in the ring's memory (every warp is done with it after the
// first sync) and become the item's result through store(cm, cl, co) (combine_and_store's
// arguments).  o(c, i): dim dims(c, i) of the lane for heads 2 q4, 2 q4 + 1, unnormalised
// relative to 2^R0, 2^R1; the sums l0, l1 to 2^m0, 2^m1.  A state leaves with its sum in
// [1, 2) and o against the same power of two, so that no o is larger than the largest |v|
// by more than a factor of two: values up to 2^124 pass the sums over warps.
template <int D, int NW, typename O, typename Sync, typename Store, typename Dims>
__device__ __forceinline__ void combine_fp8(uint8_t* smem, O o, float R0, float R1, float m0, float m1, float l0,
                                            float l1, int warp, int lane, Sync sync, Store store, Dims dims) {
  constexpr int KS = Fp8DecodeShape<D>::kSteps;
  l0 = warp_sum_xor(l0, 4);
  l1 = warp_sum_xor(l1, 4);
  // scores of NaN have left the sum NaN, but not the reference (no comparison with them
  // holds): any finite one makes the state count
  if (l0 != l0) m0 = 0.f;
  if (l1 != l1) m1 = 0.f;
  normalise_sum(l0, m0);
  normalise_sum(l1, m1);
  // 2^(R - m) in two factors: R follows V's scale, and the power itself may be out of range
  const float d0 = m0 == -INFINITY ? 0.f : R0 - m0, d1 = m1 == -INFINITY ? 0.f : R1 - m1;
  const float h0 = fminf(fmaxf(d0, -100.f), 100.f), h1 = fminf(fmaxf(d1, -100.f), 100.f);
  const uint64_t near = f2_pack(exp2_approx(h0), exp2_approx(h1));
  const uint64_t far = f2_pack(exp2_approx(d0 - h0), exp2_approx(d1 - h1));
  sync();  // every warp is done with its ring
  float* cm = reinterpret_cast<float*>(smem);
  float* cl = cm + NW * 8;
  float* co = cl + NW * 8;
  if (lane < 4) {
    cm[warp * 8 + 2 * lane] = m0;
    cm[warp * 8 + 2 * lane + 1] = m1;
    cl[warp * 8 + 2 * lane] = l0;
    cl[warp * 8 + 2 * lane + 1] = l1;
  }
#pragma unroll
  for (int c = 0; c < KS; ++c)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint64_t*>(co + ((size_t)warp * D + dims(c, i)) * 8 + 2 * (lane & 3)) =
          f2_mul(f2_mul(o(c, i), near), far);
  sync();
  store(cm, cl, co);
}

// ---------------------------------------------------------------------------
// bf16 queries
// ---------------------------------------------------------------------------
// One work item; arguments as for decode_bf16_item (decode.cu), store as for combine_fp8.
template <int D, int NW, int STAGES, typename Sync, typename Store>
__device__ __forceinline__ bool decode_fp8_item_bf16(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                                     const DecodeFp8Params& pp, uint8_t* smem, uint64_t* bars, int g,
                                                     int s, int orow, int t0, int t1, int warp, int lane, int& kb,
                                                     Sync sync, Store store) {
  constexpr int KS = Fp8DecodeShape<D>::kSteps;
  const DecodeParams& p = pp.d;
  Fp8Units<D, NW, STAGES> units(tmK, tmV, pp, smem, bars, g, s, t0, t1, warp, lane, kb);

  // q^T as the B operand of S^T = K q^T: lane holds head n = lane / 4; chunk kk's slots
  // are dims 16 kk + 4 (lane % 4) + {0, 1} and + {2, 3}
  const int q4 = lane & 3, rA = lane >> 2;
  uint32_t qf[KS][2];
  float undo;  // what the row's scaling has to be undone by
  {
    const bool live = rA < p.r;
    const __nv_bfloat16* qrow =
        reinterpret_cast<const __nv_bfloat16*>(p.q) + ((size_t)orow * p.H + g * p.r + (live ? rA : 0)) * D + 4 * q4;
    uint2 v[KS];
    uint32_t top = 0;  // bf16 magnitudes order like their bits
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      v[kk] = live ? *reinterpret_cast<const uint2*>(qrow + kk * 16) : make_uint2(0u, 0u);
      top = max_u16x2(max_u16x2(top, v[kk].x & 0x7fff7fffu), v[kk].y & 0x7fff7fffu);
    }
    top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = max(top >> 16, top & 0xffffu);
    // up = 2^(14 - e) for the largest element m 2^e, 1 <= m < 2, and undo = 1 / up, from the
    // exponent field e + 127 (held above 14: a row below 2^-112 is scaled by 2^126)
    const uint32_t field = min(max(top >> 7, 15u), 254u);
    const float up = __uint_as_float((268u - field) << 23);
    undo = __uint_as_float((field - 14u) << 23);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      qf[kk][0] = pack_f16x2(__uint_as_float(v[kk].x << 16) * up, __uint_as_float(v[kk].x & 0xffff0000u) * up);
      qf[kk][1] = pack_f16x2(__uint_as_float(v[kk].y << 16) * up, __uint_as_float(v[kk].y & 0xffff0000u) * up);
    }
  }
  // factor of this thread's score columns, heads 2 q4 and 2 q4 + 1
  const float f0 = p.scale_log2 * __shfl_sync(0xffffffffu, undo, 8 * q4);
  const float f1 = p.scale_log2 * __shfl_sync(0xffffffffu, undo, 8 * q4 + 4);

  float o[KS][4];  // [chunk][even, odd dim of lane / 4] x {head 2 q4, head 2 q4 + 1}, relative to 2^M0, 2^M1
#pragma unroll
  for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float M0 = -INFINITY, M1 = -INFINITY;                      // references of O: z + V's page exponent
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // references of the sums: z

  // ldmatrix rows and chunks: matrices 0, 1 = token rows 0..7, 8..15 of a chunk, 2, 3 of the next
  const int lrow = (lane & 8) + (lane & 7), lchunk = lane >> 4;

  // One unit.  ODD: tiles that are partly outside the range, or pages whose V scale is more
  // than 2^kWide below the largest so far: weights of the scores alone, each tile's against its
  // own maximum, and fresh accumulators that join O with the page's factor.  Everything else
  // runs without a branch but the one of moving references.
  auto consume = [&](auto odd_unit, int tok0, uint32_t sc) {
    constexpr bool ODD = decltype(odd_unit)::value;
    const uint32_t kbase = units.tile();
    const uint32_t vbase = kbase + Fp8DecodeShape<D>::kTileBytes;
    const float vb[2] = {exponent_of_byte((sc >> 8) & 255u), exponent_of_byte(sc >> 24)};

    // S^T (16 tokens x 8 heads, twice) = K codes . q^T, in two chains per tile
    float x[2][4], x2[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[h][i] = x2[h][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KS; kk += 2)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r0, r1, r2, r3, a0, a1, a2, a3;
        ldsm_x4(kbase + tile_chunk<D>(16 * h + lrow, kk + lchunk), r0, r1, r2, r3);
        unpack_e4m3x4(r0, a0, a2);
        unpack_e4m3x4(r1, a1, a3);
        mma_f16_16816(x[h], a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
        unpack_e4m3x4(r2, a0, a2);
        unpack_e4m3x4(r3, a1, a3);
        mma_f16_16816(x2[h], a0, a1, a2, a3, qf[kk + 1][0], qf[kk + 1][1]);
      }
    // V's pieces, on their way during the softmax (ODD: loaded where they are used, to hold fewer registers)
    uint32_t v[KS / 2][2][4];
    auto load_v = [&](int c, int h) {
      ldsm_x4_trans(vbase + tile_chunk<D>(16 * h + lrow, 2 * c + lchunk), v[c][h][0], v[c][h][1], v[c][h][2],
                    v[c][h][3]);
    };
    if (!ODD) {
#pragma unroll
      for (int c = 0; c < KS / 2; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) load_v(c, h);
    }

    // y = z + vb in log2 units (z: the scaled score; ODD: z itself); the thread holds tokens
    // rA, rA + 8 of each tile, heads 2 q4, 2 q4 + 1
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float ks = scale_of_byte((h ? sc >> 16 : sc) & 255u), a = f0 * ks, b = f1 * ks;
      const float e = ODD ? 0.f : vb[h];
      x[h][0] = fmaf(x[h][0] + x2[h][0], a, e);
      x[h][1] = fmaf(x[h][1] + x2[h][1], b, e);
      x[h][2] = fmaf(x[h][2] + x2[h][2], a, e);
      x[h][3] = fmaf(x[h][3] + x2[h][3], b, e);
    }
    [[maybe_unused]] uint32_t v_lo[2], v_hi[2], v_nan[2];  // ODD: which of V's codes count
    if (ODD) {
      // valid tokens of the two tiles (the first tile of a range may start before it)
      const int t = 2 * q4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int nv = h ? min(16, t1 - tok0 - 16) : tok0 < t0 ? 0 : min(16, t1 - tok0);
        if (rA >= nv) x[h][0] = x[h][1] = -INFINITY;
        if (rA + 8 >= nv) x[h][2] = x[h][3] = -INFINITY;
        // Rows past the range may hold anything (NaN codes included): zero them in the V^T
        // fragments so that 0 * NaN cannot poison O.
        v_lo[h] = (t < nv ? 0x0000ffffu : 0u) | (t + 1 < nv ? 0xffff0000u : 0u);
        v_hi[h] = (t + 8 < nv ? 0x0000ffffu : 0u) | (t + 9 < nv ? 0xffff0000u : 0u);
        // a scale of NaN: so is every code
        v_nan[h] = ((h ? sc >> 24 : sc >> 8) & 255u) == 255u ? 0x7f7f7f7fu : 0u;
      }
    }
    // y: the unit's largest z + vb; z: the sums' reference, at least the unit's largest z and
    // above it by at most the exponents' spread (ODD: that z itself, from the tiles' own, zt)
    float y0, y1, z0, z1;
    [[maybe_unused]] float zt0[2], zt1[2];
    if (ODD) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        zt0[h] = warp_max_xor(fmaxf(x[h][0], x[h][2]), 4);
        zt1[h] = warp_max_xor(fmaxf(x[h][1], x[h][3]), 4);
      }
      y0 = fmaxf(zt0[0] + vb[0], zt0[1] + vb[1]);
      y1 = fmaxf(zt1[0] + vb[0], zt1[1] + vb[1]);
      z0 = fmaxf(zt0[0], zt0[1]);
      z1 = fmaxf(zt1[0], zt1[1]);
    } else {
      y0 = warp_max_xor(fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2])), 4);
      y1 = warp_max_xor(fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3])), 4);
      const float vb_min = fminf(vb[0], vb[1]);
      z0 = y0 - vb_min;
      z1 = y1 - vb_min;
    }
    // references move rarely: weights reach 2^15 before O's does
    const bool grow = y0 - kRefDown > M0 + 1.f || z0 > m0 + kSlack || y1 - kRefDown > M1 + 1.f || z1 > m1 + kSlack;
    if (__any_sync(0xffffffffu, grow)) {
      const float N0 = fmaxf(M0, y0 - kRefDown), N1 = fmaxf(M1, y1 - kRefDown);
      const float n0 = fmaxf(m0, z0), n1 = fmaxf(m1, z1);
      const float al0 = exp2_approx(M0 - N0), al1 = exp2_approx(M1 - N1);
      l0 *= exp2_approx(m0 - n0);
      l1 *= exp2_approx(m1 - n1);
      M0 = N0;
      M1 = N1;
      m0 = n0;
      m1 = n1;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        o[i][0] *= al0;
        o[i][1] *= al1;
        o[i][2] *= al0;
        o[i][3] *= al1;
      }
    }
    // P^T (tokens x heads) -> B operand (k = token, n = head) by 8x8 transposes
    uint32_t pb[2][2];
    [[maybe_unused]] float f0t[2], f1t[2];  // ODD: what brings a tile's products to O's reference
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (a tile without a score, or with NaN alone: any finite reference)
      const bool none0 = ODD && zt0[h] == -INFINITY, none1 = ODD && zt1[h] == -INFINITY;
      const float r0 = !ODD ? M0 : none0 ? 0.f : zt0[h] - kRefDown, r1 = !ODD ? M1 : none1 ? 0.f : zt1[h] - kRefDown;
      const float e0 = exp2_approx(x[h][0] - r0), e1 = exp2_approx(x[h][1] - r1);
      const float e2 = exp2_approx(x[h][2] - r0), e3 = exp2_approx(x[h][3] - r1);
      pb[h][0] = movmatrix_trans(pack_f16x2(e0, e1));
      pb[h][1] = movmatrix_trans(pack_f16x2(e2, e3));
      // sums of 2^(z - m): the weights without V's exponent
      if (ODD) {
        f0t[h] = none0 ? 1.f : exp2_approx(r0 + vb[h] - M0);  // at most 2
        f1t[h] = none1 ? 1.f : exp2_approx(r1 + vb[h] - M1);
        l0 = fmaf(e0 + e2, none0 ? 1.f : exp2_approx(r0 - m0), l0);
        l1 = fmaf(e1 + e3, none1 ? 1.f : exp2_approx(r1 - m1), l1);
      } else {
        l0 = fmaf(e0 + e2, exp2_approx(M0 - vb[h] - m0), l0);
        l1 = fmaf(e1 + e3, exp2_approx(M1 - vb[h] - m1), l1);
      }
    }
    // O^T (D x 8 heads) += V^T codes (D x 32 tokens) . P^T
#pragma unroll
    for (int c = 0; c < KS / 2; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (ODD) {
          load_v(c, h);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][h][i] = (v[c][h][i] | v_nan[h]) & (i & 1 ? v_hi[h] : v_lo[h]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t a0, a1, a2, a3;
          unpack_e4m3x4(__byte_perm(v[c][h][2 * u], 0, 0x3120), a0, a1);      // even, odd dims of tokens 0..7
          unpack_e4m3x4(__byte_perm(v[c][h][2 * u + 1], 0, 0x3120), a2, a3);  // ... of tokens 8..15
          if (ODD) {
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16_16816(t, a0, a1, a2, a3, pb[h][0], pb[h][1]);
            float* const acc = o[2 * c + u];
            acc[0] = fmaf(t[0], f0t[h], acc[0]);
            acc[1] = fmaf(t[1], f1t[h], acc[1]);
            acc[2] = fmaf(t[2], f0t[h], acc[2]);
            acc[3] = fmaf(t[3], f1t[h], acc[3]);
          } else {
            mma_f16_16816(o[2 * c + u], a0, a1, a2, a3, pb[h][0], pb[h][1]);
          }
        }
      }
  };

  int k = 0;
  int v_top = 0;  // the largest V scale byte so far
  bool ok = true;
  for (; k < units.n_my; ++k) {
    const uint32_t sc = units.scales(k);
    const int tok0 = units.first_token(k);
    if (!units.wait()) {  // leave the loop together
      ok = false;
      break;
    }
    const int vb0 = (sc >> 8) & 255u, vb1 = sc >> 24;
    v_top = max(v_top, max(vb0, vb1));
    if (tok0 < t0 || tok0 + kUnit8 > t1 || v_top - min(vb0, vb1) > kWide || v_top == 255)
      consume(std::true_type{}, tok0, sc);
    else
      consume(std::false_type{}, tok0, sc);
    units.release(k);
  }
  if (!ok) units.drain(k);

  combine_fp8<D, NW>(smem, [&](int c, int i) { return f2_pack(o[c][2 * i], o[c][2 * i + 1]); }, M0, M1, m0, m1, l0, l1,
                     warp, lane, sync, store, [rA](int c, int i) { return c * 16 + 2 * rA + i; });
  kb += units.n_my;
  return ok;
}

// ---------------------------------------------------------------------------
// fp32 queries
// ---------------------------------------------------------------------------
// The same item for fp32 q and out: two fp16 parts of q and of the weights, and fresh
// accumulators per tile.
template <int D, int NW, int STAGES, typename Sync, typename Store>
__device__ __forceinline__ bool decode_fp8_item_f32(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                                    const DecodeFp8Params& pp, uint8_t* smem, uint64_t* bars, int g,
                                                    int s, int orow, int t0, int t1, int warp, int lane, int& kb,
                                                    Sync sync, Store store) {
  constexpr int KS = Fp8DecodeShape<D>::kSteps;
  const DecodeParams& p = pp.d;
  Fp8Units<D, NW, STAGES> units(tmK, tmV, pp, smem, bars, g, s, t0, t1, warp, lane, kb);

  // q^T as the B operand of S^T = K q^T: lane holds head n = lane / 4; chunk kk's slots
  // are dims 16 kk + 4 (lane % 4) + {0, 1} and + {2, 3}
  const int q4 = lane & 3, rA = lane >> 2;
  uint32_t qf[KS][2], ql[KS][2];
  float undo;  // what the row's scaling has to be undone by
  {
    const bool live = rA < p.r;
    const float* qrow = reinterpret_cast<const float*>(p.q) + ((size_t)orow * p.H + g * p.r + (live ? rA : 0)) * D + 4 * q4;
    float x[KS][4];
    float top = 0.f;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const float4 v = live ? *reinterpret_cast<const float4*>(qrow + kk * 16) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[kk][0] = v.x;
      x[kk][1] = v.y;
      x[kk][2] = v.z;
      x[kk][3] = v.w;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(x[kk][i]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // up = 2^(14 - e) for the largest element m 2^e, 1 <= m < 2, and undo = 1 / up, from the
    // exponent field e + 127 (held above 14: a row below 2^-112 is scaled by 2^126)
    const uint32_t field = min(max(__float_as_uint(top) >> 23, 15u), 254u);
    const float up = __uint_as_float((268u - field) << 23);
    undo = __uint_as_float((field - 14u) << 23);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[kk][i] *= up;
      qf[kk][0] = pack_f16x2(x[kk][0], x[kk][1]);
      qf[kk][1] = pack_f16x2(x[kk][2], x[kk][3]);
      ql[kk][0] = pack_f16x2_rest(x[kk][0], x[kk][1], qf[kk][0]);
      ql[kk][1] = pack_f16x2_rest(x[kk][2], x[kk][3], qf[kk][1]);
    }
  }
  // factor of this thread's score columns, heads 2 q4 and 2 q4 + 1
  const float f0 = p.scale_log2 * __shfl_sync(0xffffffffu, undo, 8 * q4);
  const float f1 = p.scale_log2 * __shfl_sync(0xffffffffu, undo, 8 * q4 + 4);

  uint64_t o[KS][2];  // [chunk][even, odd dim of lane / 4] x {head 2 q4, head 2 q4 + 1}
#pragma unroll
  for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = 0ull;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;


  // ldmatrix rows and chunks: matrices 0, 1 = token rows 0..7, 8..15 of a chunk, 2, 3 of the next
  const int lrow = (((lane >> 3) & 1) << 3) + (lane & 7), lchunk = lane >> 4;

  int k = 0;
  bool ok = true;
  for (; k < units.n_my; ++k) {
    const uint32_t sc = units.scales(k);
    if (!units.wait()) {  // leave the loop together
      ok = false;
      break;
    }
    const int tok0 = units.first_token(k);
    const uint32_t kbase = units.tile();
    const uint32_t vbase = kbase + Fp8DecodeShape<D>::kTileBytes;
    // valid tokens of the two tiles (the first tile of a range may start before it)
    int nv[2];
    nv[0] = tok0 < t0 ? 0 : min(16, t1 - tok0);
    nv[1] = max(0, min(16, t1 - tok0 - 16));

    // S^T (16 tokens x 8 heads, twice) = K codes . q^T
    float acc[2][4], acl[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[h][i] = acl[h][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KS; kk += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r0, r1, r2, r3, a0, a1, a2, a3;
        ldsm_x4(kbase + tile_chunk<D>(16 * h + lrow, kk + lchunk), r0, r1, r2, r3);
        unpack_e4m3x4(r0, a0, a2);
        unpack_e4m3x4(r1, a1, a3);
        mma_f16_16816(acc[h], a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
        mma_f16_16816(acl[h], a0, a1, a2, a3, ql[kk][0], ql[kk][1]);
        unpack_e4m3x4(r2, a0, a2);
        unpack_e4m3x4(r3, a1, a3);
        mma_f16_16816(acc[h], a0, a1, a2, a3, qf[kk + 1][0], qf[kk + 1][1]);
        mma_f16_16816(acl[h], a0, a1, a2, a3, ql[kk + 1][0], ql[kk + 1][1]);
      }
    }

    // online softmax; the thread holds tokens rA, rA + 8 of each tile, heads 2 q4, 2 q4 + 1
    float x[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float kf = scale_of_byte((h ? sc >> 16 : sc) & 255u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = fmaf(acl[h][i], 1.f / 2048.f, acc[h][i]);
        x[h][i] = a * (((i & 1) ? f1 : f0) * kf);
        if (rA + ((i & 2) << 2) >= nv[h]) x[h][i] = -INFINITY;
      }
    }
    const float t0m = warp_max_xor(fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2])), 4) - kRefDown;
    const float t1m = warp_max_xor(fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3])), 4) - kRefDown;
    // weights reach 2^15 before the reference moves
    const bool grow0 = t0m > m0 + 1.f, grow1 = t1m > m1 + 1.f;
    if (__any_sync(0xffffffffu, grow0 || grow1)) {
      const float al0 = grow0 ? exp2_approx(m0 - t0m) : 1.f;
      const float al1 = grow1 ? exp2_approx(m1 - t1m) : 1.f;
      if (grow0) m0 = t0m;
      if (grow1) m1 = t1m;
      l0 *= al0;
      l1 *= al1;
      const uint64_t al = f2_pack(al0, al1);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        o[i][0] = f2_mul(o[i][0], al);
        o[i][1] = f2_mul(o[i][1], al);
      }
    }
    // P^T (tokens x heads) -> B operand (k = token, n = head) by 8x8 transposes
    uint32_t pb[2][2], pl[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = exp2_approx(x[h][i] - ((i & 1) ? m1 : m0));
      l0 += e[0] + e[2];
      l1 += e[1] + e[3];
      const uint32_t a = pack_f16x2(e[0], e[1]), b = pack_f16x2(e[2], e[3]);
      pb[h][0] = movmatrix_trans(a);
      pb[h][1] = movmatrix_trans(b);
      pl[h][0] = movmatrix_trans(pack_f16x2_rest(e[0], e[1], a));
      pl[h][1] = movmatrix_trans(pack_f16x2_rest(e[2], e[3], b));
    }

    // Rows past the range may hold anything (NaN codes included): zero them in the V^T
    // fragments so that 0 * NaN cannot poison O.
    const bool partial = nv[0] < 16 || nv[1] < 16;
    uint32_t vm[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = 2 * q4;
      vm[h][0] = (t < nv[h] ? 0x0000ffffu : 0u) | (t + 1 < nv[h] ? 0xffff0000u : 0u);
      vm[h][1] = (t + 8 < nv[h] ? 0x0000ffffu : 0u) | (t + 9 < nv[h] ? 0xffff0000u : 0u);
    }
    // O^T (D x 8 heads) += 2^vb * V^T codes (D x 16 tokens) . P^T, one fresh accumulator per tile
#pragma unroll
    for (int c = 0; c < KS; c += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[4];
        ldsm_x4_trans(vbase + tile_chunk<D>(16 * h + lrow, c + lchunk), r[0], r[1], r[2], r[3]);
        // 2^vb without the weights' 2^kRefDown: O stays within fp32's range wherever a value does
        const float vf = scale_of_byte((h ? sc >> 24 : sc >> 8) & 255u) * kUndoRefDown;
        const uint64_t vf2 = f2_pack(vf, vf);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t lo = r[2 * u], hi = r[2 * u + 1];
          if (partial) {
            lo &= vm[h][0];
            hi &= vm[h][1];
          }
          uint32_t a0, a1, a2, a3;
          unpack_e4m3x4(__byte_perm(lo, 0, 0x3120), a0, a1);  // even, odd dims of tokens 0..7
          unpack_e4m3x4(__byte_perm(hi, 0, 0x3120), a2, a3);  // ... of tokens 8..15
          float t[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16_16816(t, a0, a1, a2, a3, pb[h][0], pb[h][1]);
          float tl[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16_16816(tl, a0, a1, a2, a3, pl[h][0], pl[h][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = fmaf(tl[i], 1.f / 2048.f, t[i]);
          o[c + u][0] = f2_fma(f2_pack(t[0], t[1]), vf2, o[c + u][0]);
          o[c + u][1] = f2_fma(f2_pack(t[2], t[3]), vf2, o[c + u][1]);
        }
      }
    }
    units.release(k);
  }
  if (!ok) units.drain(k);
  combine_fp8<D, NW>(smem, [&](int c, int i) { return o[c][i]; }, m0 + kRefDown, m1 + kRefDown, m0, m1, l0, l1, warp,
                     lane, sync, store, [rA](int c, int i) { return c * 16 + 2 * rA + i; });
  kb += units.n_my;
  return ok;
}

// Warps per CTA, ring depth per warp and CTAs per SM that the registers allow.  Measured on a
// GB300 (head_dim 128, pages of 16, bf16 queries; items: (sequence, KV head) pairs):
//   unsplit        4 warps, 3 stages, two CTAs per SM: 64 sequences of 512..4096 tokens, 32/8
//                  heads, in 53.6 us (54-56 from box to box); 2 stages and three CTAs 60.9 us (fewer
//                  bytes in flight once the long sequences are alone), 8 warps and one CTA 68 us.
//                  head_dim 64 (half the bytes per unit): 8 warps, 2 stages, two CTAs: the same
//                  batch in 33.6 us, 4 warps and 3 stages 43.9 us
//   few items      up to one per SM: 8 warps, 3 stages: 29 sequences up to 6,000 tokens, 28/4
//                  heads, in 32.9 us, 4 warps 43.6 us
//   many partitions  one warp and 2 stages, twelve CTAs per SM: nothing to combine, and a
//                  partition's start-up (block ids, scales, query) hides behind eleven others:
//                  8 sequences of 32-128 K in 512-token partitions 248 us, 4 warps and 3
//                  stages 361 us before other steps; 16 sequences of 4,096 tokens in as many
//                  30.1 us, 4 warps 37.7 us
//   few partitions  4 warps, 2 stages, three CTAs per SM: 29 sequences up to 6,000 tokens, 28/4
//                  heads, in 1,024-token partitions 26.8 us; 3 stages and two CTAs 32.5 us, 8
//                  warps 39.7 us, one warp 40.9 us
//   a CTA per SM at most, up to 8 partitions  joined in a cluster instead of by a merge kernel:
//                  one sequence of 4,096 tokens in 512-token partitions 8.5 us, 10.7 us with the
//                  merge (but 16 sequences 41.7 us, 37.7 with it: a cluster's CTAs hold their
//                  slots until the last one is done).  No merge, no workspace: an unsplit call
//                  whose items leave SMs idle is split the same way, one sequence of 16,384
//                  tokens 15.7 us (one CTA per item 73.9), eight of 512..4,096 16.5 us (23.8);
//                  by its own length: with a bound of 128 K on 2,048 tokens 7.5 us, in parts of
//                  the bound 14.8.
//                  Partitions of 1,024 tokens and more: 8 warps, 4,096-token ones 24.2 us, 4
//                  warps 32.3 us; not for clusters of more than four over more than half the
//                  SMs, which do not all fit at a time (2 x 4,096: 16.2 us for 10.4)
template <int NW_, int STAGES_, int MIN_CTAS_>
struct Fp8Plan {
  static constexpr int NW = NW_, STAGES = STAGES_, MIN_CTAS = MIN_CTAS_;
};
template <int D>
using Fp8Unsplit = std::conditional_t<D == 128, Fp8Plan<4, 3, 2>, Fp8Plan<8, 2, 2>>;
template <int D>
using Fp8FewItems = std::conditional_t<D == 128, Fp8Plan<8, 3, 1>, Fp8Plan<8, 2, 2>>;
using Fp8ManyParts = Fp8Plan<1, 2, 12>;
using Fp8FewParts = Fp8Plan<4, 2, 3>;
using Fp8JoinLong = Fp8Plan<8, 2, 1>;

template <int D, int NW, int STAGES, typename QT, typename Sync, typename Store>
__device__ __forceinline__ bool decode_fp8_item(const CUtensorMap& tmK, const CUtensorMap& tmV, const DecodeFp8Params& pp,
                                                uint8_t* smem, uint64_t* bars, int g, int s, int orow, int t0, int t1,
                                                int warp, int lane, int& kb, Sync sync, Store store) {
  if constexpr (sizeof(QT) == 4)
    return decode_fp8_item_f32<D, NW, STAGES>(tmK, tmV, pp, smem, bars, g, s, orow, t0, t1, warp, lane, kb, sync, store);
  else
    return decode_fp8_item_bf16<D, NW, STAGES>(tmK, tmV, pp, smem, bars, g, s, orow, t0, t1, warp, lane, kb, sync, store);
}

// A (sequence, KV head)'s partitions are one cluster: their results, normalised rows o
// [r][D] and their lse, are in their CTAs' shared memory at the same addresses, and every
// CTA writes a share of the merged rows, in the order of the partitions.  out = sum of
// o_i 2^(x_i - M) over sum of 2^(x_i - M), x_i the lse in log2 units, M the largest.
template <int D, typename QT, int NT>
__device__ __forceinline__ void join_partitions(const DecodeParams& p, const float* o, const float* lse, int n, int g,
                                                int s) {
  const int parts = p.max_parts, part = blockIdx.y;
  for (int idx = part * NT + threadIdx.x; idx < p.r * (D / 4); idx += parts * NT) {
    const int h = idx / (D / 4), d = (idx - h * (D / 4)) * 4;
    float x[kMaxJoin];
    float4 v[kMaxJoin];
#pragma unroll
    for (int i = 0; i < kMaxJoin; ++i) {
      x[i] = -INFINITY;
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        x[i] = ld_cluster_f32(dsmem_map(smem_u32(lse + h), i)) * kLog2e;
        v[i] = ld_cluster_f32x4(dsmem_map(smem_u32(o + h * D + d), i));
      }
    }
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMaxJoin; ++i) M = fmaxf(M, x[i]);
    float W = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxJoin; ++i) {
      if (x[i] == -INFINITY) continue;
      const float w = exp2_approx(x[i] - M);  // (NaN of a partition stays)
      W += w;
      a0 = fmaf(w, v[i].x, a0);
      a1 = fmaf(w, v[i].y, a1);
      a2 = fmaf(w, v[i].z, a2);
      a3 = fmaf(w, v[i].w, a3);
    }
    const bool empty = n == 0;
    const float inv = empty ? 0.f : 1.f / W;
    const size_t row = (size_t)s * p.H + g * p.r + h;
    store4<QT>(reinterpret_cast<QT*>(p.out) + row * D + d, a0 * inv, a1 * inv, a2 * inv, a3 * inv);
    if (d == 0 && p.lse_out) p.lse_out[row] = empty ? -INFINITY : (M + log2f(W)) * kLn2;
  }
}

// JOIN: the partitions of an item are a cluster along y, else one grid row of all of them.
template <int D, typename QT, typename Plan, bool JOIN>
__global__ void __launch_bounds__(Plan::NW * 32, Plan::MIN_CTAS) decode_fp8_kernel(const __grid_constant__ CUtensorMap tmK,
                                                              const __grid_constant__ CUtensorMap tmV,
                                                              const DecodeFp8Params pp) {
  constexpr int NW = Plan::NW, STAGES = Plan::STAGES;
  constexpr int STAGE_BYTES = Fp8DecodeShape<D>::kStageBytes;
  static_assert(NW * (64 + D * 32) <= NW * STAGES * STAGE_BYTES, "combine area must fit in the ring");
  const DecodeParams& p = pp.d;
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int kb = 0;
  auto sync = [] { __syncthreads(); };
  if constexpr (JOIN) {
    // behind the area of the warps' states (combine_fp8)
    float* jo = reinterpret_cast<float*>(smem + NW * (64 + D * 32));
    float* jl = jo + 8 * D;
    static_assert(NW * (64 + D * 32) + 8 * D * 4 + 32 <= NW * STAGES * STAGE_BYTES, "the partial must fit in the ring");
    const int g = blockIdx.x, part = blockIdx.y, s = blockIdx.z;
    int L = p.seq_lens[s];
    if (L > p.cap) {
      if (threadIdx.x == 0 && part == 0) atomicOr(&g_status_decode_fp8, METIS_STATUS_SEQ_TOO_LONG);
      L = p.cap;
    }
    L = max(L, 0);
    int P = p.partition_size;
    if (P == 0)  // an unsplit call: the sequence, not its bound, in equal parts of whole units
      P = max(kMinJoinTokens, (int)(((unsigned)L + kUnit8 * p.max_parts - 1) / (kUnit8 * p.max_parts) * kUnit8));
    const int n = L / P + (L % P != 0);  // partitions with tokens, at most max_parts
    __syncthreads();                     // the barriers are initialised
    if (part < n)
      decode_fp8_item<D, NW, STAGES, QT>(
          tmK, tmV, pp, smem, bars, g, s, s, part * P, part * P + min(L - part * P, P), warp, lane, kb, sync,
          [&](const float* cm, const float* cl, const float* co) {
            DecodeParams local{};  // one item's partial, in shared memory
            local.D = D;
            local.r = local.H = p.r;
            local.partition_size = P;
            local.max_parts = 1;
            local.part_out = jo;
            local.part_lse = jl;
            combine_and_store<QT, NW>(local, cm, cl, co, 0, 0, 0, 0, threadIdx.x);
          });
    __syncwarp();
    cluster_sync_all();
    join_partitions<D, QT, NW * 32>(p, jo, jl, n, g, s);
    cluster_sync_all();  // nobody leaves while its partial may be read
  } else {
    __shared__ int rank_lens[kMaxRankSeqs];
    __shared__ int rank_found;
    // KV heads vary fastest: the CTAs that read one page's rows (all heads of a token lie side
    // by side) run at about the same time
    const int part = blockIdx.x / p.G, g = blockIdx.x - part * p.G;
    const int s = (p.partition_size == 0 && p.S <= kMaxRankSeqs) ? seq_of_rank(p, blockIdx.y, rank_lens, &rank_found)
                                                                  : (int)blockIdx.y;
    int t0, t1;
    if (!decode_range<QT>(p, part, g, s, s, t0, t1, threadIdx.x, blockDim.x, &g_status_decode_fp8)) return;
    __syncthreads();  // the barriers are initialised
    decode_fp8_item<D, NW, STAGES, QT>(tmK, tmV, pp, smem, bars, g, s, s, t0, t1, warp, lane, kb, sync,
                                       [&](const float* cm, const float* cl, const float* co) {
                                         combine_and_store<QT, NW, true>(p, cm, cl, co, part, g, s, s, threadIdx.x);
                                       });
  }
}

// ---------------------------------------------------------------------------
// the decodes of a mixed chunked-prefill batch, beside the chunk kernel: the scheme of
// decode_rows_beside_kernel (decode.cu)
// ---------------------------------------------------------------------------
// Two groups of six warps with two stages: the mixed batch of 16 chunks of 512 and 48
// decodes takes 291 us and its decodes alone 49 us; four warps and three stages 296 and
// 52 us, three groups of four warps and two stages 288 and 62 us.
constexpr int kDec8Groups = 2;
constexpr int kFp8Warps = 6, kFp8Stages = 2;  // per group

template <int D>
constexpr int dec8_beside_smem_bytes() {
  constexpr int need = 1024 + kDec8Groups * kFp8Warps * kFp8Stages * (Fp8DecodeShape<D>::kStageBytes + 8);
  return need > 116 * 1024 ? need : 116 * 1024;  // never two CTAs on one SM
}

template <int D>
__global__ void __launch_bounds__(kDec8Groups * kFp8Warps * 32, 1)
    decode_fp8_rows_beside_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                                  const DecodeFp8Params pp, const int* n_ctas, int* next_item) {
  constexpr int NW = kFp8Warps, STAGES = kFp8Stages, GT = NW * 32;
  constexpr int STAGE_BYTES = Fp8DecodeShape<D>::kStageBytes;
  static_assert(NW * (64 + D * 32) <= NW * STAGES * STAGE_BYTES, "combine area must fit in the ring");
  const DecodeParams& p = pp.d;
  pdl_wait();  // the schedule kernel (n_ctas, the zeroed counter) and every kernel before it completed
  if ((int)blockIdx.x >= __ldcg(n_ctas)) return;
  pdl_launch_dependents();  // every CTA of the grid has waited by now: the chunk kernel may launch

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ int rank_seq[kMaxRankSeqs];
  __shared__ int lens[kMaxRankSeqs];
  __shared__ int n_dec;
  __shared__ int item_slot[kDec8Groups];
  __shared__ int gave_up[kDec8Groups];  // a warp of the group gave up a wait: the group stops
  // the batch's decodes, longest first (larger batches: in sequence order)
  const bool ranked = p.S <= kMaxRankSeqs;
  if (ranked) {
    if (threadIdx.x == 0) n_dec = 0;
    for (int i = threadIdx.x; i < p.S; i += blockDim.x)
      lens[i] = decode_row(p, i) < 0 ? -1 : min(max(p.seq_lens[i], 0), p.cap);
    __syncthreads();
    for (int c = threadIdx.x; c < p.S; c += blockDim.x) {
      const int Lc = lens[c];
      if (Lc < 0) continue;
      int r = 0;
      for (int k = 0; k < p.S; ++k) r += (lens[k] > Lc) || (lens[k] == Lc && k < c);
      rank_seq[r] = c;
      atomicAdd(&n_dec, 1);
    }
  }
  const int grp = threadIdx.x / GT, tid = threadIdx.x - grp * GT;
  const int warp = tid >> 5, lane = tid & 31;
  uint8_t* gsmem = smem + grp * NW * STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kDec8Groups * NW * STAGES * STAGE_BYTES) + grp * NW * STAGES;
  if (tid == 0) {
    if (grp == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    for (int i = 0; i < NW * STAGES; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
    gave_up[grp] = 0;
  }
  __syncthreads();
  const int n_items = (ranked ? n_dec : p.S) * p.G;
  auto gsync = [grp] { named_barrier_sync(1 + grp, GT); };
  int kb = 0;  // this warp's ring position, across the group's items
  for (;;) {
    fence_proxy_async_smem();  // the combine's stores into the ring come before the next item's loads of the same bytes
    gsync();  // the previous item's combine is done with the ring, and the slot was read
    if (gave_up[grp]) break;  // read after the barrier: the whole group leaves together
    if (tid == 0) item_slot[grp] = atomicAdd(next_item, 1);
    gsync();
    const int it = item_slot[grp];
    if (it >= n_items) break;
    const int rank = it / p.G, g = it - rank * p.G;
    const int s = ranked ? rank_seq[rank] : rank;
    const int orow = decode_row(p, s);
    if (orow < 0) continue;  // not a decode (unranked order only)
    int t0, t1;
    if (!decode_range<__nv_bfloat16>(p, 0, g, s, orow, t0, t1, tid, GT, &g_status_decode_fp8)) continue;
    // A wait that gave up (flagged) is seen by its warp only: every warp of the group
    // still reaches the item's barriers and the next one above, where they all stop.
    if (!decode_fp8_item_bf16<D, NW, STAGES>(tmK, tmV, pp, gsmem, bars, g, s, orow, t0, t1, warp, lane, kb, gsync,
                                             [&](const float* cm, const float* cl, const float* co) {
                                               combine_and_store<__nv_bfloat16, NW>(p, cm, cl, co, 0, g, s, orow, tid);
                                             }) &&
        lane == 0)
      gave_up[grp] = 1;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int decode_fp8_status(uint32_t* bits, int clear) {
  unsigned int v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_status_decode_fp8, sizeof(v));
  if (e == cudaSuccess && clear) {
    unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_status_decode_fp8, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  *bits |= v;
  return METIS_OK;
}

// TMA maps of the K and V codes: boxes of one KV head, a whole row, one page or (pages of
// 32 and 64) 32 tokens of it.
template <int D>
static int encode_kv8_maps(const DecodeParams& p, const void* k_cache, const void* v_cache, CUtensorMap* tmK,
                           CUtensorMap* tmV) {
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.num_blocks * p.bs};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)p.G * D};
  const uint32_t box[3] = {(uint32_t)D, 1, (uint32_t)std::min(p.bs, kUnit8)};
  const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  // a row is 64 or 128 bytes: promoting its fetches to 256 would bring the next head's along,
  // whose own fetch may come too late to use it (2 % slower)
  const CUtensorMapL2promotion promo = CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  int rc = encode_tiled(tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, k_cache, dims, strides, box, sw, promo);
  if (rc) return rc;
  return encode_tiled(tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, v_cache, dims, strides, box, sw, promo);
}

template <int D, typename QT, typename Plan, bool JOIN = false>
static int launch_fp8(const DecodeFp8Params& pp, const void* k_cache, const void* v_cache, cudaStream_t st) {
  CUtensorMap tmK, tmV;
  int rc = encode_kv8_maps<D>(pp.d, k_cache, v_cache, &tmK, &tmV);
  if (rc) return rc;
  constexpr int smem = fp8_decode_smem_bytes<D, Plan::NW, Plan::STAGES>();
  static int done = 0;
  auto kern = decode_fp8_kernel<D, QT, Plan, JOIN>;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem, &done);
  if (rc) return rc;
  const unsigned parts = (unsigned)pp.d.max_parts, G = (unsigned)pp.d.G, S = (unsigned)pp.d.S;
  if (JOIN)
    return launch_dependent_cluster(kern, dim3(G, parts, S), dim3(1, parts, 1), dim3(Plan::NW * 32), (size_t)smem, st,
                                    "decode_fp8_kernel launch", tmK, tmV, pp);
  return launch_dependent(kern, dim3(parts * G, S), dim3(Plan::NW * 32), (size_t)smem, st, "decode_fp8_kernel launch",
                          tmK, tmV, pp);
}

// The plan by the number of items or partitions against the GPU's SMs (seq_lens are not
// known here: partitions count max_seq_len).  *joined: the partitions need no merge.
template <int D, typename QT>
static int launch_fp8(const DecodeFp8Params& pp, const void* k_cache, const void* v_cache, cudaStream_t st,
                      bool* joined) {
  DecodeFp8Params split = pp;
  DecodeParams& p = split.d;
  int tokens = p.partition_size;  // of a partition, at most
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(METIS_E_CUDA, "querying the SM count: %s", cudaGetErrorString(e));
  const long long items = (long long)p.G * p.S;
  if (p.partition_size == 0) {
    if (items > sms) return launch_fp8<D, QT, Fp8Unsplit<D>>(pp, k_cache, v_cache, st);
    // SMs to spare: partitions all the same (no workspace: they are joined)
    p.max_parts = (int)std::min<long long>({kMaxJoin, sms / items, p.cap / kMinJoinTokens});
    if (p.max_parts < 2) return launch_fp8<D, QT, Fp8FewItems<D>>(pp, k_cache, v_cache, st);
    tokens = p.cap / p.max_parts;
  }
  const long long ctas = p.max_parts * items;
  *joined = p.max_parts <= kMaxJoin && ctas <= sms;
  if (*joined && tokens >= 1024 && (2 * ctas <= sms || p.max_parts <= kMaxJoin / 2))
    return launch_fp8<D, QT, Fp8JoinLong, true>(split, k_cache, v_cache, st);
  if (*joined) return launch_fp8<D, QT, Fp8FewParts, true>(split, k_cache, v_cache, st);
  // one warp per partition: where twelve on each SM are filled twice over, and for short ones as
  // soon as the four-warp CTAs would not be on the GPU all at once (three per SM, head_dim 64 four)
  if (ctas >= 24ll * sms || (p.partition_size <= 512 && ctas > (D == 64 ? 4ll : 3ll) * sms))
    return launch_fp8<D, QT, Fp8ManyParts>(pp, k_cache, v_cache, st);
  return launch_fp8<D, QT, Fp8FewParts>(pp, k_cache, v_cache, st);
}

template <int D>
static int launch_beside8(const DecodeFp8Params& pp, const void* k_cache, const void* v_cache, const int* n_ctas,
                          int* next_item, int grid, cudaStream_t st) {
  CUtensorMap tmK, tmV;
  int rc = encode_kv8_maps<D>(pp.d, k_cache, v_cache, &tmK, &tmV);
  if (rc) return rc;
  constexpr int smem = dec8_beside_smem_bytes<D>();
  static int done = 0;
  auto kern = decode_fp8_rows_beside_kernel<D>;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem, &done);
  if (rc) return rc;
  return launch_dependent(kern, dim3((unsigned)grid), dim3(kDec8Groups * kFp8Warps * 32), (size_t)smem, st,
                          "decode_fp8_rows_beside_kernel launch", tmK, tmV, pp, n_ctas, next_item);
}

static DecodeFp8Params fp8_params(const void* q, const Fp8Cache& cache, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* rows, void* out, float* lse_out, int S, int H,
                                  int G, int D, int bs, int max_blocks, int num_blocks, float scale, int cap) {
  DecodeFp8Params pp{};
  DecodeParams& p = pp.d;
  p.q = q;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.lse_out = lse_out;
  p.S = S;
  p.H = H;
  p.G = G;
  p.D = D;
  p.bs = bs;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.r = H / G;
  p.scale_log2 = scale * kLog2e;
  p.max_parts = 1;
  p.cap = cap;
  p.rows = rows;
  pp.k_scale = cache.k_scale;
  pp.v_scale = cache.v_scale;
  return pp;
}

int launch_decode_fp8_rows_beside(const void* q, const Fp8Cache& cache, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* rows, int T, void* out, float* lse_out, int S,
                                  int H, int G, int D, int bs, int max_blocks, int num_blocks, float scale, int cap,
                                  const int* n_ctas, int* next_item, int grid, cudaStream_t st) {
  DecodeFp8Params pp = fp8_params(q, cache, block_table, seq_lens, rows, out, lse_out, S, H, G, D, bs, max_blocks,
                                  num_blocks, scale, cap);
  pp.d.T = T;
  return D == 64 ? launch_beside8<64>(pp, cache.k_cache, cache.v_cache, n_ctas, next_item, grid, st)
                 : launch_beside8<128>(pp, cache.k_cache, cache.v_cache, n_ctas, next_item, grid, st);
}

}  // namespace metis

using namespace metis;

extern "C" int metis_paged_attn_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                                           const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table,
                                           const int32_t* seq_lens, void* out, float* lse_out, int num_seqs,
                                           int num_heads, int num_kv_heads, int head_dim, int block_size,
                                           int max_blocks, int num_blocks, int dtype, float scale, int partition_size,
                                           int max_seq_len, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  if (num_seqs < 0) return fail(METIS_E_SHAPE, "num_seqs < 0");
  if (num_seqs == 0) return METIS_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out)
    return fail(METIS_E_NULL, "q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens and out are required");
  if (num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks <= 0 ||
      num_blocks <= 0 || max_seq_len <= 0)
    return fail(METIS_E_SHAPE, "sizes must be positive");
  if (num_heads % num_kv_heads) return fail(METIS_E_SHAPE, "num_heads %% num_kv_heads != 0");
  if (num_seqs > 65535 || num_kv_heads > 65535) return fail(METIS_E_SHAPE, "num_seqs and num_kv_heads must be <= 65535");
  if ((long long)max_blocks * block_size > 0x7fffffffLL || (long long)num_blocks * block_size > 0x7fffffffLL)
    return fail(METIS_E_SHAPE, "max_blocks * block_size and num_blocks * block_size must fit in int32");
  if (head_dim != 64 && head_dim != 128) return fail(METIS_E_UNSUPPORTED, "head_dim must be 64 or 128");
  if (block_size != 16 && block_size != 32 && block_size != 64)
    return fail(METIS_E_UNSUPPORTED, "block_size must be 16, 32 or 64");
  if (dtype != METIS_F32 && dtype != METIS_BF16) return fail(METIS_E_UNSUPPORTED, "dtype must be METIS_F32 or METIS_BF16");
  if (num_heads / num_kv_heads > 8) return fail(METIS_E_UNSUPPORTED, "num_heads / num_kv_heads must be <= 8");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse_out, 4))
    return fail(METIS_E_ALIGN, "tensors must be 16-byte aligned (block_table, seq_lens, lse_out: 4-byte; scales: any)");
  if (partition_size < 0 || (partition_size % 16))
    return fail(METIS_E_SHAPE, "partition_size must be 0 or a positive multiple of 16");
  if (!(scale == scale)) return fail(METIS_E_SHAPE, "scale is NaN");

  const int eff_len = effective_max_len(max_seq_len, max_blocks, block_size);
  const size_t parts = split_parts(eff_len, partition_size);
  if (parts > 0x7fffffff / (size_t)num_kv_heads) return fail(METIS_E_SHAPE, "too many partitions");
  const size_t need = metis_decode_workspace_bytes(num_seqs, num_heads, head_dim, eff_len, partition_size);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(METIS_E_WORKSPACE, "workspace must hold %zu bytes (256-byte aligned)", need);

  const Fp8Cache cache = {k_cache, v_cache, k_scale, v_scale};
  DecodeFp8Params pp = fp8_params(q, cache, block_table, seq_lens, nullptr, out, lse_out, num_seqs, num_heads,
                                  num_kv_heads, head_dim, block_size, max_blocks, num_blocks, scale, eff_len);
  DecodeParams& p = pp.d;
  p.partition_size = partition_size;
  if (parts) {
    const size_t units = (size_t)num_seqs * num_heads * parts;
    p.max_parts = (int)parts;
    p.part_out = reinterpret_cast<float*>(workspace);
    p.part_lse = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                          align_up(units * head_dim * sizeof(float), 256));
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int rc;
  bool joined = false;
  if (dtype == METIS_F32)
    rc = head_dim == 64 ? launch_fp8<64, float>(pp, k_cache, v_cache, st, &joined)
                        : launch_fp8<128, float>(pp, k_cache, v_cache, st, &joined);
  else
    rc = head_dim == 64 ? launch_fp8<64, __nv_bfloat16>(pp, k_cache, v_cache, st, &joined)
                        : launch_fp8<128, __nv_bfloat16>(pp, k_cache, v_cache, st, &joined);
  if (rc) return rc;
  if (parts && !joined)
    rc = launch_merge_ex(p.part_out, p.part_lse, seq_lens, partition_size, out, lse_out, num_seqs, num_heads, head_dim,
                         p.max_parts, dtype, 0, st);
  return rc;
}
