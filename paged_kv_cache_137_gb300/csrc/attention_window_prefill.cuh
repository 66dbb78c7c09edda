// Prefill attention with a sliding window and sinks, and over block-scaled
// E4M3 caches, on the 5th-generation tensor cores.
//
// The chunk of sequence s is its last n positions; the query at position p
// sees p' <= p with p' > p - window or p' < sinks (window 0: every p' <= p).
//   out = softmax(q . K^T * scale) V  over what it sees.
//
// A CTA takes 256 query rows of one KV head as two tiles of 128 (M of an
// MMA).  Row r of a chunk is head r % G of position r / G: the G query heads
// that share a KV head share its K/V tiles, and 256 rows span 256 / G
// positions only, so that with a window little more than its own keys is
// read and multiplied.  The keys those rows see are walked in steps of 64, as
// four chunks of 16 each: the sinks' chunks, then those from the first row's
// window on; blocks between are not looked up.
//
// Warps 0-3 and 4-7 do the softmax of tile A and B (a thread a row, TMEM lane
// = row), warp 8 drives TMA, warp 9 issues the MMAs:
//   S_t = Q K_t^T  (128 x 64, into one of two TMEM buffers per tile)
//   P_t = 2^(S_t scale - m)  (16 bit, over the S buffer it came from)
//   O  += P_t V_t  (128 x D, A operand from TMEM)
// S_{t+2} is issued when P_t V_t is done, so the tensor core stays two steps
// ahead of the softmax.  O stays in TMEM; a row's reference m moves only when
// its running maximum has grown by 2^8, and then its O is rescaled.  The pool
// rows (and scales) of 32 chunks are fetched a lane each, a batch ahead, and
// the boxes of a step go out a lane each.
//
// E4M3 caches are widened to f16 in shared memory by four warps.  With block
// scales a step has one power of two R per K and V, the exponent of the
// largest of its four chunks' scales, and a chunk is widened as e4m3 * (scale
// / R): exact in f16 as long as scale / R is a power of two of at least 2^-15
// (below that a chunk's smallest values lose bits to f16's subnormals: an
// error of at most 2^-24 R per value, R within the same 64 keys).  R of K joins
// the logit scale; R of V joins the exponent of P, whose reference m is then
// that of s + log2 R, and the row sum takes sum(P) / R, so that O and l keep
// one reference.
//
// Sums, maxima and O are fp32; P is rounded to the MMA's type (the cache's,
// f16 for E4M3: 2^-8 or 2^-11 of a weight), bf16 queries of an E4M3 cache to
// f16.  V rows that no row of the CTA sees are zeroed in shared memory (a
// weight of 0 times what they hold must be 0).  Every wait is bounded; a CTA
// whose wait gives up writes NaN rows, waits for its copies and MMAs in
// flight and frees its TMEM.
#pragma once

#include <atomic>
#include <type_traits>

#include "attention_prefill_umma.cuh"
#include "attention_window.h"

namespace pkv {
namespace tc {
namespace wprefill {

using namespace umma;

constexpr int kChunkKeys = 16;
constexpr int kStepChunks = kKeys / kChunkKeys;   // 4
constexpr int kWide = 3;                          // widened 16-bit buffers (E4M3)
constexpr int kProdWarp = 8, kMmaWarp = 9, kConvWarp = 10, kConvWarps = 4;
constexpr int kScaleRing = 8;

// What the 256 rows of a CTA see: positions [0, sinks) and [w0, last], as
// chunks of 16; the first ns chunks, then those from wb on, n in all.
struct Keys {
  int w0, sinks, last, ns, wb, n;
  __device__ __forceinline__ Keys(int first_pos, int last_pos, int window, int s) {
    last = last_pos;
    w0 = window > 0 ? max(first_pos - window + 1, 0) : 0;
    sinks = window > 0 ? s : 0;
    ns = (min(sinks, w0) + kChunkKeys - 1) / kChunkKeys;
    wb = max(w0 / kChunkKeys, ns);
    n = ns + max(last / kChunkKeys + 1 - wb, 0);
  }
  __device__ __forceinline__ int chunk(int i) const { return i < ns ? i : i - ns + wb; }
  __device__ __forceinline__ bool any_sees(int p) const { return p <= last && (p >= w0 || p < sinks); }
  // every row of some query sees all of step t's 64 keys up to its own end:
  // false where a key of the step may be hidden from all rows
  __device__ __forceinline__ bool inner(int t) const {
    const int p = chunk(kStepChunks * t) * kChunkKeys;
    return kStepChunks * t >= ns && p >= w0 && p + kKeys - 1 <= last;
  }
};

template <typename KV, int D>
struct Shape {
  static constexpr bool kFp8 = std::is_same<KV, E4M3>::value;
  static constexpr int kSlabs = D / 64;                     // 128-byte slabs of a 16-bit row
  static constexpr int kQTile = kRows * D * 2;
  static constexpr int kTile16 = kKeys * D * 2;             // K (or V) of a step, 16 bits
  static constexpr int kStage16 = 2 * kTile16;
  static constexpr int kTile8 = kKeys * D;
  static constexpr int kStage8 = 2 * kTile8;
  static constexpr int kRing = kFp8 ? 4 : 5;                // TMA stages
  static constexpr int kRingBytes = kFp8 ? kRing * kStage8 + kWide * kStage16 : kRing * kStage16;
  static constexpr int kSmem = 1024 + 2 * kQTile + kRingBytes;
  static constexpr int kThreads = 32 * (kFp8 ? kConvWarp + kConvWarps : kConvWarp);
};

using Args = WindowPrefillArgs;

// The largest power of two that is at most x (x > 0), and the scale kept
// within the range block scales have.
__device__ __forceinline__ float pow2_floor(float x) {
  return __uint_as_float(__float_as_uint(x) & 0x7f800000u);
}
__device__ __forceinline__ float clamp_scale(float x) {
  return fminf(fmaxf(x, 9.094947017729282e-13f), 1099511627776.f);   // 2^-40, 2^40
}

// The MMA warp runs its loop with all lanes and predicates each instruction on
// one elected lane: inside a one-lane branch the operands' uniform registers
// would be filled anew before every MMA, which measured about 100 cycles an
// instruction and bound the whole pipeline.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p;
}
// D[tmem] (+)= A[smem] x B[smem], issued where `leader`.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// D[tmem] (+)= A[tmem] x B[smem].
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}

template <typename KV, typename Q, int D, bool BS>
__global__ void __launch_bounds__(Shape<KV, D>::kThreads, 1)
    prefill_window_kernel(const Args a, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap) {
  using S_ = Shape<KV, D>;
  constexpr bool kFp8 = S_::kFp8;
  constexpr bool kBf = std::is_same<KV, BF16>::value;
  constexpr bool kOutBf = std::is_same<Q, BF16>::value;
  constexpr uint32_t kIdQK = idesc(kBf, kRows, kKeys, false);
  constexpr uint32_t kIdPV = idesc(kBf, kRows, D, true);
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int kQSlab = kRows * 128;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // grid: (KV head, sequence, row pair counted from the chunk's end): the
  // pairs with the most keys of every sequence first
  const int kvh = blockIdx.x, s = blockIdx.y;
  const int G = a.group, HQ = a.num_q_heads, T = a.block_size;
  const int ctx = a.ctx_lens[s];
  const int q0 = a.query_start[s];
  const int n = a.query_start[s + 1] - q0;
  if (q0 < 0 || n <= 0 || n > a.total_q - q0) return;   // no rows this call may write
  const int64_t rows = static_cast<int64_t>(n) * G;
  const int npairs = static_cast<int>((rows + 2 * kRows - 1) / (2 * kRows));
  if (ctx < 0 || ctx > a.max_blocks * T || n > ctx || npairs > a.max_q_tiles) {
    // invalid lengths: the chunk's rows of this KV head become NaN
    if (tid == 0 && a.status != nullptr) atomicOr(a.status, kBadLength);
    if (blockIdx.z == 0)
      for (int64_t i = tid; i < rows * D; i += S_::kThreads) {
        const int64_t r = i / D;
        store_elem<Q>(a.out, ((q0 + r / G) * HQ + kvh * G + r % G) * D + i % D, CUDART_NAN_F);
      }
    return;
  }
  const int pair = npairs - 1 - static_cast<int>(blockIdx.z);
  if (pair < 0) return;
  const int first = ctx - n;   // position of the chunk's first query
  // tile X: chunk rows [row0, row0 + 128) of the pair's 256, inside [0, rows)
  const int64_t pair0 = static_cast<int64_t>(pair) * 2 * kRows;
  const int in_pair = static_cast<int>(min(rows - pair0, static_cast<int64_t>(2 * kRows)));
  const int pos_first = first + static_cast<int>(pair0 / G);
  auto pos_of = [&](int r) { return first + static_cast<int>((pair0 + r) / G); };
  const Keys keys(pos_first, pos_of(in_pair - 1), a.window, a.sinks);
  // steps of each tile: up to its last row's position
  const int endA = pos_of(min(in_pair, kRows) - 1) / kChunkKeys + 1;
  const int nA = keys.ns + max(endA - keys.wb, 0);
  const int n_steps = (keys.n + kStepChunks - 1) / kStepChunks;
  const int nt[2] = {max((nA + kStepChunks - 1) / kStepChunks, 1), in_pair > kRows ? n_steps : 0};
  const int steps = max(nt[0], nt[1]);
  const HeadScales hs = head_scales(a.head_scales, a.num_kv_heads, kvh, a.softmax_scale, a.qk_scale,
                                    a.v_scale, 1.f, 1.f);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* q_s = smem;                             // [tile][slab][128 rows][128 B]
  uint8_t* ring = smem + 2 * S_::kQTile;           // 16-bit: [stage][K, V][slab]; E4M3: [stage][K, V]
  uint8_t* wide = ring + S_::kRing * S_::kStage8;  // E4M3: widened [buffer][K, V][slab]
  uint8_t* kv16 = kFp8 ? wide : ring;
  constexpr int kBuf = kFp8 ? kWide : S_::kRing;   // 16-bit K/V buffers
  __shared__ uint64_t full[S_::kRing], empty[S_::kRing], s_full[4], p_full[4], o_done[4], fin;
  __shared__ uint64_t conv_full[kWide], wide_free[kWide];
  __shared__ uint32_t s_ratio[BS ? kScaleRing : 1][2 * kStepChunks];   // half2 pairs: K, then V chunks
  __shared__ float s_ref[BS ? kScaleRing : 1][2];                      // R of K and V
  __shared__ uint32_t tmem_slot;
  __shared__ int s_bad, s_issued;

  if (tid == 0) {
    s_bad = 0;
    s_issued = 0;
    for (int i = 0; i < S_::kRing; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kFp8 ? kConvWarps : 1);
    }
    for (int i = 0; i < kWide; ++i) {
      mbar_init(smem_u32(&conv_full[i]), kConvWarps);
      mbar_init(smem_u32(&wide_free[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), kRows);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    mbar_init(smem_u32(&fin), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kProdWarp) {
    __syncwarp();
    tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // Q rows, zero past the chunk's end, 128-byte-swizzled
  if (warp < 8) {
    const int r = tid;   // row of the pair
    const bool in = r < in_pair;
    const int64_t cr = pair0 + (in ? r : 0);
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const typename Q::raw*>(a.q) +
        ((q0 + cr / G) * static_cast<int64_t>(HQ) + kvh * G + cr % G) * D);
    uint8_t* qx = q_s + (r >> 7) * S_::kQTile;
    uint4 qv[D / 8];   // every load first (one round trip), then the stores
#pragma unroll
    for (int c = 0; c < D / 8; ++c) qv[c] = in ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      uint4 v = qv[c];
      if constexpr (kFp8 && kOutBf) {   // the MMA is f16
        float f[8];
        LoadF32<Q, 8>::run(&v, f);
        v = make_uint4(pack2<false>(f[0], f[1]), pack2<false>(f[2], f[3]), pack2<false>(f[4], f[5]),
                       pack2<false>(f[6], f[7]));
      }
      *reinterpret_cast<uint4*>(qx + (c >> 3) * kQSlab + sw(r & 127, c & 7)) = v;
    }
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == kProdWarp) {
    // ------------------------------------------------------------ producer
    const int32_t* trow = a.tables + static_cast<size_t>(s) * a.max_blocks;
    // lane l of batch b: the pool row (-1: none) and the scales of chunk 32 b + l
    auto fetch = [&](int b, int& row, float2& sc) {
      row = -1;
      sc = make_float2(0.f, 0.f);
      const int i = 32 * b + lane;
      if (i >= keys.n) return;
      const int p = keys.chunk(i) * kChunkKeys;
      const int blk = trow[p / T];
      if (blk < 0 || blk >= a.num_blocks) {
        atomicOr(&s_bad, kBadTable);   // before the step is announced: the rows become NaN
        return;
      }
      const int slab = blk * a.num_kv_heads + kvh;
      row = slab * T + p % T;
      if constexpr (BS) {
        const float2 v = *reinterpret_cast<const float2*>(a.block_scales + 2 * static_cast<size_t>(slab));
        sc = make_float2(clamp_scale(v.x), clamp_scale(v.y));
      }
    };
    int row_cur, row_nxt;
    float2 sc_cur, sc_nxt;
    fetch(0, row_cur, sc_cur);
    fetch(1, row_nxt, sc_nxt);
    // a lane's box of a step: chunk, slab, K or V
    constexpr int kBoxSlabs = kFp8 ? 1 : S_::kSlabs;
    constexpr int kBoxes = kStepChunks * kBoxSlabs * 2;
    const int bv = lane & 1, bsl = (lane >> 1) % kBoxSlabs, bc = (lane >> 1) / kBoxSlabs;
    for (int t = 0; t < steps; ++t) {
      if ((t & 7) == 0 && t > 0) {   // 32 chunks are 8 steps
        row_cur = row_nxt;
        sc_cur = sc_nxt;
        fetch(t / 8 + 1, row_nxt, sc_nxt);
      }
      const int slot = t % S_::kRing;
      const bool ok = t < S_::kRing ||
                      mbar_wait(smem_u32(&empty[slot]), ((t / S_::kRing) - 1) & 1, kWaitNs);
      if (!__all_sync(FULL, ok)) {
        if (lane == 0) atomicOr(&s_bad, kTimeout);
        break;
      }
      const int c0 = (kStepChunks * t) & 31;
      const int row = __shfl_sync(FULL, row_cur, c0 + (bc & 3));
      const bool load = lane < kBoxes && row >= 0;
      if constexpr (BS) {
        float ks = __shfl_sync(FULL, sc_cur.x, c0 + (lane & 3));
        float vs = __shfl_sync(FULL, sc_cur.y, c0 + (lane & 3));
        float x = lane < kStepChunks ? ks : vs;   // lanes 0-3: K scales, 4-7: V scales
        float top = fmaxf(x, __shfl_xor_sync(FULL, x, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
        const float ref = top > 0.f ? pow2_floor(top) : 1.f;
        if (lane < 2 * kStepChunks) {
          const __half2 h = __float2half2_rn(__fdividef(x, ref));
          s_ratio[t % kScaleRing][lane] = *reinterpret_cast<const uint32_t*>(&h);
          if ((lane & 3) == 0) s_ref[t % kScaleRing][lane >> 2] = ref;
        }
      }
      const unsigned boxes = __ballot_sync(FULL, load);
      const uint32_t bar = smem_u32(&full[slot]);
      __syncwarp();   // the scales and any error, before the step is announced
      if (lane == 0)
        mbar_arrive_expect_tx(bar, __popc(boxes) * static_cast<uint32_t>(kChunkKeys * 128));
      __syncwarp();
      if (load) {
        uint8_t* dst = ring + slot * (kFp8 ? S_::kStage8 : S_::kStage16) +
                       bv * (kFp8 ? S_::kTile8 : S_::kTile16) + bsl * kSlab + bc * (kChunkKeys * 128);
        tma_load_2d(smem_u32(dst), bv ? &vmap : &kmap, bsl * 128, row, bar);
      }
      if (lane == 0) s_issued = t + 1;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t leader = elect_one();
    const uint32_t tm = __reduce_max_sync(FULL, tmem);   // uniform for the compiler as well
    const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024);
    const uint64_t k_desc = sw128_desc(smem_u32(kv16), 16, 1024);
    const uint64_t v_desc = sw128_desc(smem_u32(kv16 + S_::kTile16), kSlab, 1024);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(FULL, mbar_wait(smem_u32(bar), parity, kWaitNs));
    };
    auto qk = [&](int X, int t) -> bool {
      const int slot = t % kBuf, b = t & 1, i = 2 * X + b;
      if (!wait(kFp8 ? &conv_full[slot] : &full[slot], (t / kBuf) & 1)) return false;
      // the buffer's step t - 2: its P has been read by P V
      if (t >= 2 && !wait(&o_done[i], ((t >> 1) - 1) & 1)) return false;
      tc_fence_after();
      const uint64_t qd = q_desc + ((X * S_::kQTile) >> 4);
      const uint64_t kd = k_desc + ((slot * S_::kStage16) >> 4);
      const uint32_t d_tmem = tm + 256 * X + 64 * b;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        mma_ss(leader, d_tmem, qd + (((ks >> 2) * kQSlab + 32 * (ks & 3)) >> 4),
               kd + (((ks >> 2) * kSlab + 32 * (ks & 3)) >> 4), kIdQK, ks > 0 ? 1u : 0u);
      commit(leader, smem_u32(&s_full[i]));
      return true;
    };
    auto pv = [&](int X, int t) -> bool {
      const int b = t & 1, i = 2 * X + b;
      if (!wait(&p_full[i], (t >> 1) & 1)) return false;
      tc_fence_after();
      const uint64_t vd = v_desc + (((t % kBuf) * S_::kStage16) >> 4);
      const uint32_t d_tmem = tm + 256 * X + 128, p_tmem = tm + 256 * X + 64 * b;
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)
        mma_ts(leader, d_tmem, p_tmem + 8 * kk, vd + ((2048 * kk) >> 4), kIdPV, (t > 0 || kk > 0) ? 1u : 0u);
      commit(leader, smem_u32(&o_done[i]));
      return true;
    };
    bool ok = true;
    for (int t = 0; t < 2 && ok; ++t)
      for (int X = 0; X < 2 && ok; ++X)
        if (t < nt[X]) ok = qk(X, t);
    for (int t = 0; t < steps && ok; ++t) {
      for (int X = 0; X < 2 && ok; ++X)
        if (t < nt[X]) ok = pv(X, t);
      if (!ok) break;
      commit(leader, smem_u32(kFp8 ? &wide_free[t % kBuf] : &empty[t % kBuf]));
      for (int X = 0; X < 2 && ok; ++X)
        if (t + 2 < nt[X]) ok = qk(X, t + 2);
    }
    if (!ok && lane == 0) atomicOr(&s_bad, kTimeout);
    commit(leader, smem_u32(&fin));
  } else if (kFp8 && warp >= kConvWarp) {
    // ------------------------------------------------------------ converters
    // two warps K, two V; each half of the 64 rows, a 16-byte piece (16
    // elements) a lane at a time
    const int cw = warp - kConvWarp, tv = cw >> 1, half = cw & 1;
    for (int t = 0; t < steps; ++t) {
      const int slot = t % S_::kRing, w = t % kWide;
      const bool ready = mbar_wait(smem_u32(&full[slot]), (t / S_::kRing) & 1, kWaitNs) &&
                         (t < kWide || mbar_wait(smem_u32(&wide_free[w]), ((t / kWide) - 1) & 1, kWaitNs));
      if (!__all_sync(FULL, ready)) {
        if (lane == 0) atomicOr(&s_bad, kTimeout);
        break;
      }
      const uint8_t* src = ring + slot * S_::kStage8 + tv * S_::kTile8;
      uint8_t* dst = wide + w * S_::kStage16 + tv * S_::kTile16;
      const bool inner = keys.inner(t);
#pragma unroll 4
      for (int k = 0; k < 8; ++k) {
        const int u = lane + 32 * k;
        const int row = 32 * half + (u >> 3), c = u & 7;
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        const int p = keys.chunk(kStepChunks * t + (row >> 4)) * kChunkKeys + (row & 15);
        if (tv == 0 || inner || keys.any_sees(p)) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + sw(row, c));
          const uint32_t in[4] = {x.x, x.y, x.z, x.w};
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[2 * e] = e4m3x2_f16x2(in[e] & 0xffffu);
            y[2 * e + 1] = e4m3x2_f16x2(in[e] >> 16);
          }
          if constexpr (BS) {
            const uint32_t rb = s_ratio[t % kScaleRing][tv * kStepChunks + (row >> 4)];
            const __half2 ratio = *reinterpret_cast<const __half2*>(&rb);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __half2 z = __hmul2(*reinterpret_cast<__half2*>(&y[e]), ratio);
              y[e] = *reinterpret_cast<const uint32_t*>(&z);
            }
          }
          lo = make_uint4(y[0], y[1], y[2], y[3]);
          hi = make_uint4(y[4], y[5], y[6], y[7]);
        }
        // head_dim 16 c .. 16 c + 15: slab c / 4, pieces 2 (c % 4) and the next
        uint8_t* d = dst + (c >> 2) * kSlab;
        *reinterpret_cast<uint4*>(d + sw(row, 2 * (c & 3))) = lo;
        *reinterpret_cast<uint4*>(d + sw(row, 2 * (c & 3) + 1)) = hi;
      }
      fence_proxy_async();   // the widened rows, before the tensor core reads them
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&conv_full[w]));
        mbar_arrive(smem_u32(&empty[slot]));
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    // every branch around a warp-wide TMEM access is taken by the whole warp
    const int X = warp >> 2, r = tid & 127, rp = tid;   // tile, TMEM lane, row of the pair
    const int ntx = nt[X];
    const int pos = pos_of(min(rp, in_pair - 1));
    const int w0 = a.window > 0 ? pos - a.window + 1 : 0;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + 256 * X + 128;
    float m_ref = -CUDART_INF_F, l = 0.f;
    bool ok = true;
    for (int t = 0; t < ntx; ++t) {
      const int b = t & 1, i = 2 * X + b;
      if (!__all_sync(FULL, mbar_wait(smem_u32(&s_full[i]), (t >> 1) & 1, kWaitNs))) {
        ok = false;
        break;
      }
      tc_fence_after();
      float sv[64];
      {
        uint32_t h0[32], h1[32];
        const uint32_t ts = tmem + 256 * X + 64 * b + lane_off;
        tmem_ld32_async(ts, h0);
        tmem_ld32_async(ts + 32, h1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          sv[e] = __uint_as_float(h0[e]);
          sv[32 + e] = __uint_as_float(h1[e]);
        }
      }
      float qe = hs.qk, lv = 0.f, inv_v = 1.f;
      if constexpr (BS) {
        // passed already; it orders the producer's scales before this read
        mbar_wait(smem_u32(&conv_full[t % kWide]), (t / kWide) & 1, kWaitNs);
        qe *= s_ref[t % kScaleRing][0];
        const uint32_t vb = __float_as_uint(s_ref[t % kScaleRing][1]);   // a power of two
        lv = static_cast<float>(static_cast<int>(vb >> 23) - 127);
        inv_v = __uint_as_float((254u << 23) - vb);
      }
      // mask: every key of the step lies in one run of positions unless it
      // holds sinks' chunks
      const int p0 = keys.chunk(kStepChunks * t) * kChunkKeys;
      if (!(kStepChunks * t >= keys.ns && p0 >= w0 && p0 + kKeys - 1 <= pos)) {
#pragma unroll
        for (int c = 0; c < kStepChunks; ++c) {
          const int pc = keys.chunk(kStepChunks * t + c) * kChunkKeys;
          const int hi = pos - pc, lo = w0 - pc, sk = keys.sinks - pc;
#pragma unroll
          for (int e = 0; e < kChunkKeys; ++e)
            if (e > hi || (e < lo && e >= sk)) sv[16 * c + e] = -CUDART_INF_F;
        }
      }
      if (!(qe > 0.f)) {   // the maximum below is taken on the raw products
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (sv[e] != -CUDART_INF_F) sv[e] *= qe;
        qe = 1.f;
      }
      float mx8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) mx8[k] = sv[k];
#pragma unroll
      for (int e = 8; e < 64; ++e) mx8[e & 7] = fmaxf(mx8[e & 7], sv[e]);
      const float mx = fmaf(qe, fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                      fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))), lv);
      const bool move = mx > m_ref + kRescaleLog2;
      const bool scale = move && t > 0 && m_ref != -CUDART_INF_F;   // O holds earlier steps
      if (__any_sync(FULL, scale)) {
        const int ip = 2 * X + ((t - 1) & 1);
        if (!__all_sync(FULL, mbar_wait(smem_u32(&o_done[ip]), ((t - 1) >> 1) & 1, kWaitNs))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float f = scale ? ex2(m_ref - mx) : 1.f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tO + lane_off + c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          tmem_st32(tO + lane_off + c, o);
        }
        l *= f;
      }
      if (move) m_ref = mx;
      // a row that has seen nothing yet keeps every weight 0
      const float off = lv - (m_ref == -CUDART_INF_F ? 0.f : m_ref);
      float sum8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum8[k] = 0.f;
      uint32_t w[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float e0 = ex2(fmaf(sv[2 * c], qe, off));
        const float e1 = ex2(fmaf(sv[2 * c + 1], qe, off));
        sum8[(2 * c) & 7] += e0;
        sum8[(2 * c + 1) & 7] += e1;
        w[c] = pack2<kBf>(e0, e1);
      }
      tmem_st32u(tmem + 256 * X + 64 * b + lane_off, w);
      l = fmaf(((sum8[0] + sum8[1]) + (sum8[2] + sum8[3])) + ((sum8[4] + sum8[5]) + (sum8[6] + sum8[7])),
               inv_v, l);
      // V rows that nobody sees (16-bit caches; the converters leave zeros):
      // by tile A's threads, by B's where A has no such step
      if constexpr (!kFp8) {
        if (!keys.inner(t) && r < kKeys && (X == 0 || t >= nt[0])) {
          const int p = keys.chunk(kStepChunks * t + (r >> 4)) * kChunkKeys + (r & 15);
          if (!keys.any_sees(p)) {
            uint8_t* vt = ring + (t % S_::kRing) * S_::kStage16 + S_::kTile16 + r * 128;
#pragma unroll
            for (int c = 0; c < 8 * S_::kSlabs; ++c)
              *reinterpret_cast<uint4*>(vt + (c >> 3) * kSlab + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();   // before the tensor core reads V
          }
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&p_full[i]));
    }
    // epilogue: O / l, after the tile's last P V
    if (ntx > 0) {
      const int tl = ntx - 1;
      ok = __all_sync(FULL, ok && mbar_wait(smem_u32(&o_done[2 * X + (tl & 1)]), (tl >> 1) & 1, kWaitNs));
      tc_fence_after();
      if (!ok) atomicOr(&s_bad, kTimeout);
      const bool bad = !ok || *reinterpret_cast<volatile int*>(&s_bad) != 0;
      const float inv = (l > 0.f || l != l) ? hs.v / l : 0.f;
      const int64_t cr = pair0 + rp;
      typename Q::raw* dst = static_cast<typename Q::raw*>(a.out) +
                             ((q0 + cr / G) * static_cast<int64_t>(HQ) + kvh * G + cr % G) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(tO + lane_off + c, o);
        if (rp < in_pair) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack2<kOutBf>(bad ? CUDART_NAN_F : o[2 * e] * inv,
                                 bad ? CUDART_NAN_F : o[2 * e + 1] * inv);
          uint4* d4 = reinterpret_cast<uint4*>(dst + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) d4[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
      }
    }
  }

  // every MMA done and every copy landed before TMEM and shared memory go
  __syncthreads();
  if (tid == 0) {
    mbar_wait(smem_u32(&fin), 0, kDrainNs);
    if (s_bad) {
      const int issued = s_issued;
      for (int t = max(0, issued - S_::kRing); t < issued; ++t)
        mbar_wait(smem_u32(&full[t % S_::kRing]), (t / S_::kRing) & 1, kDrainNs);
      if (a.status != nullptr) atomicOr(a.status, s_bad);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kProdWarp) {
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename KV, typename Q, int D, bool BS>
pkv_status launch(Args a, const CUtensorMap& kmap, const CUtensorMap& vmap, int32_t max_query_len,
                  cudaStream_t st) {
  using S_ = Shape<KV, D>;
  static_assert(S_::kSmem <= 227 * 1024 - 1024, "ring, queries and the static part fit one SM");
  auto kernel = prefill_window_kernel<KV, Q, D, BS>;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail("windowed prefill: cudaGetDevice", e);
  const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
  if (!bit || !(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S_::kSmem);
    if (e != cudaSuccess) return cuda_fail("windowed prefill: cudaFuncSetAttribute", e);
    configured.fetch_or(bit);
  }
  const int64_t pairs = (static_cast<int64_t>(max_query_len) * a.group + 2 * kRows - 1) / (2 * kRows);
  if (pairs > 65535) return fail(PKV_ERR_UNSUPPORTED, "max_query_len too large");
  a.max_q_tiles = static_cast<int32_t>(pairs);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.num_kv_heads, a.num_seqs, static_cast<unsigned>(pairs));
  cfg.blockDim = dim3(S_::kThreads);
  cfg.dynamicSmemBytes = S_::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, kmap, vmap);
  if (e != cudaSuccess) return cuda_fail("windowed prefill: launch", e);
  return check_launch("windowed prefill");
}

}  // namespace wprefill
}  // namespace tc

template <typename KV, typename Q>
pkv_status launch_window_prefill(const WindowPrefillArgs& a, int head_dim, int32_t max_query_len,
                                 const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t st) {
  if constexpr (std::is_same<KV, E4M3>::value) {
    if (head_dim == 128)
      return a.block_scales ? tc::wprefill::launch<KV, Q, 128, true>(a, kmap, vmap, max_query_len, st)
                            : tc::wprefill::launch<KV, Q, 128, false>(a, kmap, vmap, max_query_len, st);
  } else {
    if (head_dim == 128) return tc::wprefill::launch<KV, Q, 128, false>(a, kmap, vmap, max_query_len, st);
    if (head_dim == 64) return tc::wprefill::launch<KV, Q, 64, false>(a, kmap, vmap, max_query_len, st);
  }
  return fail(PKV_ERR_UNSUPPORTED, "windowed prefill: head_dim not compiled for this cache");
}

}  // namespace pkv
