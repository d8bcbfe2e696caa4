// One work item of a paged decode -- one KV head of one sequence over a span of its tokens -- for the
// kernels that share it: plain, beside chunks, windowed (decode.cu, decode_window.cu), and of a
// warp that walks items (decode_stream.cuh).
#pragma once

#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "decode.cuh"
#include "host.h"

namespace metis {

// ---------------------------------------------------------------------------
// bf16 decode: TMA page units + mma.sync
// ---------------------------------------------------------------------------
constexpr int kUnit = 16;              // tokens per pipeline unit (one m16 tile)
constexpr int kBoxBytes = kUnit * 128; // one 16-token x 64-dim bf16 box, 128-byte rows

template <int D>
struct Bf16DecodeShape {
  static constexpr int kHalves = D / 64;
  static constexpr int kStageBytes = 2 * kHalves * kBoxBytes;  // K halves, then V halves
  static constexpr int kSteps = D / 16;                        // QK k-steps == PV m-tiles
};

template <int D, int NW, int STAGES>
constexpr int bf16_decode_smem_bytes() {
  return 1024 + NW * STAGES * Bf16DecodeShape<D>::kStageBytes + NW * STAGES * 8;
}

// bf16 decode configuration: warps per CTA and ring depth per warp.
#ifndef METIS_DECODE_WARPS
#define METIS_DECODE_WARPS 4
#endif
#ifndef METIS_DECODE_STAGES
#define METIS_DECODE_STAGES 3
#endif
constexpr int kBf16Warps = METIS_DECODE_WARPS;
constexpr int kBf16Stages = METIS_DECODE_STAGES;


// The tokens [t0, t1), in units that start on multiples of kUnit.
struct RangeSpan {
  static constexpr bool kHole = false;
  int t0, t1;
  __host__ __device__ __forceinline__ int units() const {
    return (t1 - t0 / kUnit * kUnit + kUnit - 1) / kUnit;
  }
  __host__ __device__ __forceinline__ int token(int i) const { return (t0 / kUnit + i) * kUnit; }  // first of unit i
  // the tokens one by one: nth(begin()) .. nth(end() - 1)
  __host__ __device__ __forceinline__ int begin() const { return t0; }
  __host__ __device__ __forceinline__ int end() const { return t1; }
  __host__ __device__ __forceinline__ int nth(int i) const { return i; }
};

// The tokens [0, h0) and [h1, t1): a sequence's first ones and its recent ones.  Only units with such
// tokens are visited, so the pages in between need not exist.  An item may take the units
// [first, first + n) of them.
struct WindowSpan {
  static constexpr bool kHole = true;
  int first, n;
  int low_units, skip;  // units with first tokens that come before the recent ones' units; units in between
  int h0, h1, t1;
  __host__ __device__ __forceinline__ int units() const { return n; }
  __host__ __device__ __forceinline__ int token(int i) const {
    i += first;
    return (i < low_units ? i : i + skip) * kUnit;
  }
  __host__ __device__ __forceinline__ bool hidden(int t) const { return t >= h0 && t < h1; }
  __host__ __device__ __forceinline__ int begin() const { return 0; }
  __host__ __device__ __forceinline__ int end() const { return h0 + t1 - h1; }
  __host__ __device__ __forceinline__ int nth(int i) const { return i < h0 ? i : i - h0 + h1; }
  // part `part` of `parts` equal ones (whole units); false: it is empty
  __host__ __device__ __forceinline__ bool take(int part, int parts) {
    const int len = (n + parts - 1) / parts;
    first = part * len;
    n = n - first < len ? n - first : len;
    return n > 0;
  }
};

// What a query behind L tokens sees (L > 0): the last `window` and the first `sinks` of them.
__host__ __device__ __forceinline__ WindowSpan window_span(int L, int window, int sinks) {
  WindowSpan w;
  w.h1 = L > window ? L - window : 0;
  w.h0 = sinks < w.h1 ? sinks : w.h1;
  w.t1 = L;
  const int low = w.h0 / kUnit + (w.h0 % kUnit != 0), recent = w.h1 / kUnit;
  w.low_units = low < recent ? low : recent;
  w.skip = recent - w.low_units;
  w.first = 0;
  w.n = w.low_units + (L / kUnit + (L % kUnit != 0) - recent);
  return w;
}

// A warp's running softmax over units of 16 tokens: the group's query rows (up to 8 heads) against one KV
// head.  q^T is the B operand of S^T = K q^T: a lane holds head n = lane / 4, dims 2*(lane%4) (+1, +8, +9);
// of O^T (D x 8 heads) the rows lane / 4 (+8) of each 16 and the heads 2*(lane%4) (+1), whose maxima (log2
// units) and sums m, l are.
template <int D>
struct DecodeWarp {
  static constexpr int KS = Bf16DecodeShape<D>::kSteps, HALVES = Bf16DecodeShape<D>::kHalves;
  uint32_t qf[KS][2];
  float o[KS][4];
  float m0, m1, l0, l1;

  // Query row orow, KV head g: an empty state.
  __device__ __forceinline__ void begin(const DecodeParams& p, int orow, int g, int lane) {
    const int q4 = lane & 3, rA = lane >> 2;
    const bool live = rA < p.r;
    const __nv_bfloat16* qrow =
        reinterpret_cast<const __nv_bfloat16*>(p.q) + ((size_t)orow * p.H + g * p.r + (live ? rA : 0)) * D;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      qf[kk][0] = live ? *reinterpret_cast<const uint32_t*>(qrow + kk * 16 + 2 * q4) : 0u;
      qf[kk][1] = live ? *reinterpret_cast<const uint32_t*>(qrow + kk * 16 + 8 + 2 * q4) : 0u;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = kNoScore;
    l0 = l1 = 0.f;
  }

  // The unit whose K (and behind it V) boxes are at kbase and whose first token is tok0.
  template <typename Span>
  __device__ __forceinline__ void unit(uint32_t kbase, int tok0, const Span& span, float sl2, int lane) {
    const int q4 = lane & 3, rA = lane >> 2;
    const int nv = min(kUnit, span.t1 - tok0);  // tokens in this unit before the span's end, >= 1
    const uint32_t vbase = kbase + HALVES * kBoxBytes;

    // S^T (16 tokens x 8 heads) = K (16 x D) . q^T (D x 8), in two independent
    // accumulation chains (even / odd k-steps) to halve the dependent-MMA latency
    float sacc[4] = {0.f, 0.f, 0.f, 0.f};
    {
      float sacc2[4] = {0.f, 0.f, 0.f, 0.f};
      const int j = lane >> 3;
      const int row = ((j & 1) << 3) + (lane & 7);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        const int c = kk * 2 + (j >> 1);
        const uint32_t addr = kbase + (c >> 3) * kBoxBytes + row * 128 + ((((c & 7) ^ (row & 7))) << 4);
        uint32_t a0, a1, a2, a3;
        ldsm_x4(addr, a0, a1, a2, a3);
        mma_bf16_16816((kk & 1) ? sacc2 : sacc, a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sacc[i] += sacc2[i];
    }

    // online softmax over this unit; the thread holds tokens rA, rA+8 of heads 2*q4, 2*q4+1
    float s0 = sacc[0] * sl2, s1 = sacc[1] * sl2, s2 = sacc[2] * sl2, s3 = sacc[3] * sl2;
    if (rA >= nv) s0 = s1 = -INFINITY;
    if (rA + 8 >= nv) s2 = s3 = -INFINITY;
    bool holed = false;  // the unit holds tokens between the first ones and the recent ones
    if constexpr (Span::kHole) {
      holed = tok0 < span.h1 && tok0 + kUnit > span.h0;
      if (span.hidden(tok0 + rA)) s0 = s1 = -INFINITY;
      if (span.hidden(tok0 + rA + 8)) s2 = s3 = -INFINITY;
    }
    const float mn0 = fmaxf(m0, warp_max_xor(fmaxf(s0, s2), 4));
    const float mn1 = fmaxf(m1, warp_max_xor(fmaxf(s1, s3), 4));
    const float al0 = exp2_approx(m0 - mn0), al1 = exp2_approx(m1 - mn1);
    const float p0 = exp2_approx(s0 - mn0), p1 = exp2_approx(s1 - mn1);
    const float p2 = exp2_approx(s2 - mn0), p3 = exp2_approx(s3 - mn1);
    l0 = l0 * al0 + (p0 + p2);
    l1 = l1 * al1 + (p1 + p3);
    m0 = mn0;
    m1 = mn1;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      o[i][0] *= al0;
      o[i][1] *= al1;
      o[i][2] *= al0;
      o[i][3] *= al1;
    }
    // P^T (tokens x heads) -> B operand (k = token, n = head) by 8x8 transposes.  The weights are rounded to bf16, which
    // the product's instruction takes (2^-8 of each; rows' error against float64 about 2.0e-3, of which 1.7e-3 is the
    // rounding of out); their sum l is that of the fp32 ones.
    const uint32_t pb0 = movmatrix_trans(pack_bf16x2(p0, p1));
    const uint32_t pb1 = movmatrix_trans(pack_bf16x2(p2, p3));

    // Rows of tokens that are not the item's may hold anything (NaN included): zero
    // them in the V^T fragments so that 0 * garbage cannot poison O.
    uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
    if (nv < kUnit) {
      const int t = 2 * q4;
      mlo = (t < nv ? 0x0000ffffu : 0u) | (t + 1 < nv ? 0xffff0000u : 0u);
      mhi = (t + 8 < nv ? 0x0000ffffu : 0u) | (t + 9 < nv ? 0xffff0000u : 0u);
    }
    if constexpr (Span::kHole) {
      if (holed) {
        const int t = tok0 + 2 * q4;
        mlo &= (span.hidden(t) ? 0u : 0x0000ffffu) | (span.hidden(t + 1) ? 0u : 0xffff0000u);
        mhi &= (span.hidden(t + 8) ? 0u : 0x0000ffffu) | (span.hidden(t + 9) ? 0u : 0xffff0000u);
      }
    }
    // O^T (D x 8 heads) += V^T (D x 16 tokens) . P^T (16 tokens x 8 heads)
    {
      const int j = lane >> 3;
      const int row = ((j >> 1) << 3) + (lane & 7);
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const int c = mt * 2 + (j & 1);
        const uint32_t addr = vbase + (c >> 3) * kBoxBytes + row * 128 + ((((c & 7) ^ (row & 7))) << 4);
        uint32_t a0, a1, a2, a3;
        ldsm_x4_trans(addr, a0, a1, a2, a3);
        mma_bf16_16816(o[mt], a0 & mlo, a1 & mlo, a2 & mhi, a3 & mhi, pb0, pb1);
      }
    }
  }
};

// One work item of the bf16 decode: the tokens of `span` of KV head g of sequence s
// (query row orow), run by NW warps (warp 0 .. NW - 1 of the caller's
// group) over their NW x STAGES TMA ring at
// smem with its barriers at bars.  kb: this warp's ring position before the item
// (ring stages and barrier phases run on across the items of a persistent group),
// advanced past the item's units.  status: the calling file's device status word.
// sync(): a barrier over the group's threads.  store(cm, cl, co): takes the warps'
// states (combine_and_store's) behind such a barrier.
// The combine step reuses the ring: the caller syncs the group before the next
// item's loads.  Returns false when a wait gave up.
template <int D, int NW, int STAGES, typename Span, typename Sync, typename Store>
__device__ __forceinline__ bool decode_bf16_item(const CUtensorMap& tmK, const CUtensorMap& tmV, const DecodeParams& p,
                                                 uint8_t* smem, uint64_t* bars, int g, int s, int orow,
                                                 const Span& span, int warp, int lane, int& kb, unsigned int* status,
                                                 Sync sync, Store store) {
  using Shape = Bf16DecodeShape<D>;
  constexpr int HALVES = Shape::kHalves;
  constexpr int STAGE_BYTES = Shape::kStageBytes;
  constexpr int KS = Shape::kSteps;

  // this warp's units: warp + k * NW, k < n_my
  const int n_units = span.units();
  const int n_my = warp < n_units ? (n_units - warp + NW - 1) / NW : 0;
  const int32_t* bt_row = p.block_table + (size_t)s * p.max_blocks;

  // Lane l holds the TMA row coordinate (block * bs + slot) of unit k = 32 * batch + l;
  // -kUnit (a box entirely outside the tensor, read as zeros) marks a bad block id.
  auto row_coord = [&](int k) -> int {
    if (k >= n_my) return -kUnit;
    const int tok = span.token(warp + k * NW);
    const int page = tok / p.bs;
    const int b = checked_block(bt_row, page, p.num_blocks, status);
    return b < 0 ? -kUnit : b * p.bs + (tok - page * p.bs);
  };
  int win_cur = row_coord(lane);
  int win_next = row_coord(32 + lane);
  const uint64_t policy = l2_policy_evict_first();

  auto issue = [&](int k) {  // called by all lanes, in order k = 0, 1, 2, ...
    if (k > 0 && (k & 31) == 0) {
      win_cur = win_next;
      win_next = row_coord(k + 32 + lane);
    }
    const int row = __shfl_sync(0xffffffffu, win_cur, k & 31);
    const int st = (kb + k) % STAGES;
    uint8_t* base = smem + (warp * STAGES + st) * STAGE_BYTES;
    uint64_t* bar = &bars[warp * STAGES + st];
    if (lane == 0) mbar_arrive_expect_tx(bar, STAGE_BYTES);
    __syncwarp();
    // one box per lane: a single thread issues TMA instructions far slower than several
    if (lane < 2 * HALVES) {
      const int h = lane % HALVES;
      tma_load_3d(base + lane * kBoxBytes, lane < HALVES ? &tmK : &tmV, bar, h * 64, g, row, policy);
    }
  };

  DecodeWarp<D> state;
  state.begin(p, orow, g, lane);

  const int prologue = n_my < STAGES ? n_my : STAGES;
  for (int k = 0; k < prologue; ++k) issue(k);

  int k = 0;
  bool ok = true;
  for (; k < n_my; ++k) {
    const int st = (kb + k) % STAGES;
    const bool landed = mbar_wait(&bars[warp * STAGES + st], ((kb + k) / STAGES) & 1, status);
    if (!__all_sync(0xffffffffu, landed)) {  // leave the loop together
      ok = false;
      break;
    }
    const int tok0 = span.token(warp + k * NW);
    state.unit(smem_u32(smem + (warp * STAGES + st) * STAGE_BYTES), tok0, span, p.scale_log2, lane);
    __syncwarp();
    if (k + STAGES < n_my) issue(k + STAGES);
  }
  if (!ok) {
    // drain this warp's loads still in flight (bounded) before the ring is reused
    for (int kk = k + 1; kk < n_my && kk < k + STAGES; ++kk) {
      const int st = (kb + kk) % STAGES;
      mbar_wait(&bars[warp * STAGES + st], ((kb + kk) / STAGES) & 1, status);
    }
  }

  const int q4 = lane & 3, rA = lane >> 2;
  const float l0 = warp_sum_xor(state.l0, 4), l1 = warp_sum_xor(state.l1, 4);
  sync();  // every warp is done with its ring

  float* cm = reinterpret_cast<float*>(smem);
  float* cl = cm + NW * 8;
  float* co = cl + NW * 8;
  if (lane < 4) {
    cm[warp * 8 + 2 * lane] = state.m0;
    cm[warp * 8 + 2 * lane + 1] = state.m1;
    cl[warp * 8 + 2 * lane] = l0;
    cl[warp * 8 + 2 * lane + 1] = l1;
  }
#pragma unroll
  for (int mt = 0; mt < KS; ++mt) {
    const int d0 = mt * 16 + rA;
    float* c0 = co + ((size_t)warp * D + d0) * 8 + 2 * q4;
    float* c1 = c0 + 8 * 8;
    c0[0] = state.o[mt][0];
    c0[1] = state.o[mt][1];
    c1[0] = state.o[mt][2];
    c1[1] = state.o[mt][3];
  }
  sync();
  store(cm, cl, co);
  kb += n_my;
  return ok;
}

// ---------------------------------------------------------------------------
// joining the parts of an item
// ---------------------------------------------------------------------------
constexpr int kMaxParts = 8;  // of an item: the CTAs of a cluster

// One row's running result: a sum of o_i 2^(x_i - M) and of 2^(x_i - M), x_i the lse of part i in log2
// units and o_i its normalised values.
struct JoinedRow {
  float M = -INFINITY, W = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
  __device__ __forceinline__ void add(float x, const float4& v) {
    if (x == -INFINITY) return;  // an empty part: its values may be anything
    const float top = fmaxf(M, x), keep = exp2_approx(M - top), w = exp2_approx(x - top);  // (NaN stays, in W)
    M = top;
    W = fmaf(W, keep, w);
    a0 = fmaf(a0, keep, w * v.x);
    a1 = fmaf(a1, keep, w * v.y);
    a2 = fmaf(a2, keep, w * v.z);
    a3 = fmaf(a3, keep, w * v.w);
  }
};

// The item's `n` parts that hold tokens, rows o [r][D] and their lse (natural log) in the shared memory
// of the CTAs 0 .. n - 1 of this cluster.  Each of the cluster's `parts` CTAs writes a share of the rows.
template <int D, typename OutT, int NT>
__device__ __forceinline__ void join_parts_of_item(const DecodeParams& p, const float* o, const float* lse, int part,
                                                   int parts, int n, int g, int orow) {
  for (int idx = part * NT + threadIdx.x; idx < p.r * (D / 4); idx += parts * NT) {
    const int h = idx / (D / 4), d = (idx - h * (D / 4)) * 4;
    JoinedRow row;
    float x[kMaxParts];
    float4 v[kMaxParts];
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) {
      x[i] = -INFINITY;
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        x[i] = ld_cluster_f32(dsmem_map(smem_u32(lse + h), i)) * kLog2e;
        v[i] = ld_cluster_f32x4(dsmem_map(smem_u32(o + h * D + d), i));
      }
    }
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) row.add(x[i], v[i]);
    const bool empty = n == 0;  // no part with a token
    const float inv = empty ? 0.f : 1.f / row.W;
    const size_t at = (size_t)orow * p.H + g * p.r + h;
    store4<OutT>(reinterpret_cast<OutT*>(p.out) + at * D + d, row.a0 * inv, row.a1 * inv, row.a2 * inv, row.a3 * inv);
    if (d == 0 && p.lse_out) p.lse_out[at] = empty ? -INFINITY : (row.M + log2f(row.W)) * kLn2;
  }
}

// One of `parts` CTAs (a cluster along y) that share an item of one (sequence, KV head): its part of the
// units of `span`, then the join.  `has`: the sequence has tokens in the span.  The ring holds the partial:
// o, then the lse, behind the warps' states.
template <int D, int NW, int STAGES>
__device__ __forceinline__ void decode_joined_item(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                                   const DecodeParams& p, uint8_t* smem, uint64_t* bars, int g, int s,
                                                   int part, int parts, bool has, WindowSpan span,
                                                   unsigned int* status) {
  constexpr int STAGE_BYTES = Bf16DecodeShape<D>::kStageBytes;
  static_assert(NW * (64 + D * 32) + 8 * D * 4 + 32 <= NW * STAGES * STAGE_BYTES, "the partial must fit in the ring");
  float* jo = reinterpret_cast<float*>(smem + NW * (64 + D * 32));
  float* jl = jo + 8 * D;
  int n = 0, kb = 0;
  if (has) {
    const int len = (span.n + parts - 1) / parts;
    n = (span.n + len - 1) / len;  // parts with units
    if (span.take(part, parts))
      decode_bf16_item<D, NW, STAGES>(tmK, tmV, p, smem, bars, g, s, s, span, threadIdx.x >> 5, threadIdx.x & 31, kb,
                                      status, [] { __syncthreads(); },
                                      [&](const float* cm, const float* cl, const float* co) {
                                        DecodeParams local{};  // one item's partial, in shared memory
                                        local.D = D;
                                        local.r = local.H = p.r;
                                        local.partition_size = 1;
                                        local.max_parts = 1;
                                        local.part_out = jo;
                                        local.part_lse = jl;
                                        combine_and_store<__nv_bfloat16, NW>(local, cm, cl, co, 0, 0, 0, 0,
                                                                             threadIdx.x);
                                      });
  }
  __syncwarp();
  cluster_sync_all();
  join_parts_of_item<D, __nv_bfloat16, NW * 32>(p, jo, jl, part, parts, n, g, s);
  __syncwarp();
  cluster_sync_all();  // nobody leaves while its partial may be read
}

// ---------------------------------------------------------------------------
// fp32 decode on FMA units
// ---------------------------------------------------------------------------
constexpr int kF32Warps = 8;

// The item (KV head g of sequence s over `span`) of a CTA of kF32Warps warps
template <int D, typename Span>
__device__ __forceinline__ void decode_f32_item(const float* k_cache, const float* v_cache, const DecodeParams& p,
                                                int part, int g, int s, const Span& span, unsigned int* status) {
  constexpr int DPL = D / 32;  // dims per lane
  __shared__ float cm[kF32Warps * 8], cl[kF32Warps * 8];
  __shared__ float co[kF32Warps * D * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const float* q = reinterpret_cast<const float*>(p.q) + ((size_t)s * p.H + (size_t)g * p.r) * D;
  float qv[8][DPL];
#pragma unroll
  for (int h = 0; h < 8; ++h)
#pragma unroll
    for (int i = 0; i < DPL; ++i) qv[h][i] = h < p.r ? q[h * D + lane * DPL + i] * p.scale_log2 : 0.f;

  float m[8], l[8], o[8][DPL];
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    m[h] = kNoScore;
    l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < DPL; ++i) o[h][i] = 0.f;
  }
  const int32_t* bt_row = p.block_table + (size_t)s * p.max_blocks;
  const size_t row_stride = (size_t)p.G * D;
  // The warp's tokens, number warp, + kF32Warps, ... of the span, in groups of kF32Batch: the block ids
  // and K/V rows of a group are loaded together, then folded in one at a time in token
  // order (the same order as without grouping).
  constexpr int kF32Batch = D == 64 ? 8 : 4;
  const int end = span.end();
  for (int ib = span.begin() + warp; ib < end; ib += kF32Batch * kF32Warps) {
    float kv[kF32Batch][DPL], vv[kF32Batch][DPL];
#pragma unroll
    for (int u = 0; u < kF32Batch; ++u) {
      const int i = ib + u * kF32Warps;
      int b = -1, page = 0, t = 0;
      if (i < end) {
        t = span.nth(i);
        page = t / p.bs;
        b = checked_block(bt_row, page, p.num_blocks, status);
      }
      if (b >= 0) {
        const size_t off = ((size_t)b * p.bs + (t - page * p.bs)) * row_stride + (size_t)g * D + lane * DPL;
#pragma unroll
        for (int d = 0; d < DPL; ++d) {
          kv[u][d] = k_cache[off + d];
          vv[u][d] = v_cache[off + d];
        }
      } else {
#pragma unroll
        for (int d = 0; d < DPL; ++d) kv[u][d] = vv[u][d] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kF32Batch; ++u) {
      if (ib + u * kF32Warps >= end) break;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        if (h < p.r) {
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < DPL; ++i) dot = fmaf(qv[h][i], kv[u][i], dot);
          dot = warp_sum_xor(dot, 1);
          const float mn = fmaxf(m[h], dot);
          const float al = exp2_approx(m[h] - mn);
          const float pr = exp2_approx(dot - mn);
          l[h] = l[h] * al + pr;
#pragma unroll
          for (int i = 0; i < DPL; ++i) o[h][i] = fmaf(pr, vv[u][i], o[h][i] * al);
          m[h] = mn;
        }
      }
    }
  }
  if (lane == 0) {
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      cm[warp * 8 + h] = m[h];
      cl[warp * 8 + h] = l[h];
    }
  }
#pragma unroll
  for (int h = 0; h < 8; ++h)
#pragma unroll
    for (int i = 0; i < DPL; ++i) co[((size_t)warp * D + lane * DPL + i) * 8 + h] = o[h][i];
  __syncthreads();
  combine_and_store<float, kF32Warps, true>(p, cm, cl, co, part, g, s, s, threadIdx.x);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// CTAs that share an item of up to `tokens` tokens: as many as the SMs take at once (kItemCtasPerSm each), with at
// least kMinPartTokens each.  (Windows of 1,024 over 8 sequences of 8 KV heads: 11.3 us, a CTA each 13.9; one
// sequence with a window of 4,096: 9.9 and 40.7.)
constexpr int kItemCtasPerSm = 2;
constexpr int kMinPartTokens = 128;

inline int item_parts(long long items, int tokens, int sms) {
  const long long fit = items > 0 ? kItemCtasPerSm * (long long)sms / items : 1;
  return (int)std::max<long long>(1, std::min<long long>({kMaxParts, fit, tokens / kMinPartTokens}));
}

// TMA maps of the K and V caches: 16-token x 64-dim boxes of one KV head.
template <int D>
inline int encode_kv_maps(const DecodeParams& p, const void* k_cache, const void* v_cache, CUtensorMap* tmK,
                          CUtensorMap* tmV) {
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.num_blocks * p.bs};
  const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)p.G * D * 2};
  const uint32_t box[3] = {64, 1, (uint32_t)kUnit};
  int rc = encode_tiled(tmK, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, k_cache, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  return encode_tiled(tmV, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v_cache, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace metis
