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
constexpr int kUnitRows = 2 * kRows;              // query rows of a unit
// warps: 0-7 softmax (four a tile), TMA, MMA of tile A and B, scheduler, converters
constexpr int kProdWarp = 8, kMmaWarp = 9, kSchedWarp = 11, kConvWarp = 12, kConvWarps = 4;
constexpr int kScaleRing = 8;

// What the 256 rows of a unit see: positions [0, sinks) and [w0, last], as
// chunks of 16; the first ns chunks, then those from wb on, n in all.
struct Keys {
  int w0, sinks, last, ns, wb, n;
  __device__ __forceinline__ void set(int first_pos, int last_pos, int window, int s) {
    last = last_pos;
    w0 = window > 0 ? max(first_pos - window + 1, 0) : 0;
    sinks = window > 0 ? s : 0;
    ns = (min(sinks, w0) + kChunkKeys - 1) / kChunkKeys;
    wb = max(w0 / kChunkKeys, ns);
    n = ns + max(last / kChunkKeys + 1 - wb, 0);
  }
  __device__ __forceinline__ int chunk(int i) const { return i < ns ? i : i - ns + wb; }
  __device__ __forceinline__ bool any_sees(int p) const { return p <= last && (p >= w0 || p < sinks); }
  // step t's 64 keys are one run that some row sees entirely
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

// A claimed unit as the scheduler announces it.
struct Work {
  int s, kvh, q0, n, ctx, pair;   // s < 0: no more work
  int bad;                        // PKV_DEVICE_* bits met while it ran
};

// 256 rows of one KV head of one chunk, tile X = rows [128 X, 128 X + 128).
struct Unit {
  int s, kvh, q0, row0, in_pair, first;
  Keys keys;
  int nt[2], steps;   // 64-key steps of each tile, and of the K/V stream
  __device__ __forceinline__ Unit(const Work& w, const Args& a) {
    s = w.s;
    kvh = w.kvh;
    q0 = w.q0;
    row0 = w.pair * kUnitRows;
    in_pair = min(w.n * a.group - row0, kUnitRows);
    first = w.ctx - w.n;
    keys.set(pos_of(0, a.group), pos_of(in_pair - 1, a.group), a.window, a.sinks);
    const int endA = pos_of(min(in_pair, kRows) - 1, a.group) / kChunkKeys + 1;
    nt[0] = max((keys.ns + max(endA - keys.wb, 0) + kStepChunks - 1) / kStepChunks, 1);
    steps = (keys.n + kStepChunks - 1) / kStepChunks;
    nt[1] = in_pair > kRows ? steps : 0;
    steps = max(nt[0], nt[1]);
  }
  __device__ __forceinline__ int pos_of(int r, int G) const { return first + (row0 + r) / G; }
  // element offset of row r in q and out
  __device__ __forceinline__ int64_t row_at(int r, const Args& a, int D) const {
    const int i = (row0 + r) / a.group, j = row0 + r - i * a.group;
    return ((static_cast<int64_t>(q0) + i) * a.num_q_heads + kvh * a.group + j) * D;
  }
};

// The largest power of two that is at most x (x > 0), and the scale kept
// within the range block scales have.
__device__ __forceinline__ float pow2_floor(float x) {
  return __uint_as_float(__float_as_uint(x) & 0x7f800000u);
}
__device__ __forceinline__ float clamp_scale(float x) {
  return fminf(fmaxf(x, 9.094947017729282e-13f), 1099511627776.f);   // 2^-40, 2^40
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Ask the hardware for a block of this grid that has not started (its 16-byte
// answer arrives at dst and completes 16 bytes on bar), and read the answer:
// the claimed block's index, or -1 where none is left (then never ask again).
__device__ __forceinline__ void claim_block(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ int claimed_block(const ulonglong2& answer) {
  uint32_t ok, x = 0;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "mov.b128 h, {%2, %3};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "+r"(x)
      : "l"(answer.x), "l"(answer.y));
  return ok ? static_cast<int>(x) : -1;
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
  constexpr int kBuf = kFp8 ? kWide : S_::kRing;            // 16-bit K/V buffers
  // warps that read a unit's description: softmax, TMA, MMA, converters
  constexpr int kReaders = 8 + 1 + 2 + (kFp8 ? kConvWarps : 0);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group, T = a.block_size;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* q_s = smem;                             // [tile][slab][128 rows][128 B]
  uint8_t* ring = smem + 2 * S_::kQTile;           // 16-bit: [stage][K, V][slab]; E4M3: [stage][K, V]
  uint8_t* wide = ring + S_::kRing * S_::kStage8;  // E4M3: widened [buffer][K, V][slab]
  uint8_t* kv16 = kFp8 ? wide : ring;
  __shared__ uint64_t full[S_::kRing], empty[S_::kRing], conv_full[kWide], wide_free[kWide];
  __shared__ uint64_t q_full[2], s_full[4], p_full[4], o_done[4], o_free[2], fin;
  __shared__ uint64_t work_full[2], work_empty[2], claim_bar;
  __shared__ ulonglong2 s_answer;
  __shared__ Work s_work[2];
  __shared__ uint32_t s_ratio[BS ? kScaleRing : 1][2 * kStepChunks];   // half2 pairs: K, then V chunks
  __shared__ float s_ref[BS ? kScaleRing : 1][2];                      // R of K and V
  __shared__ uint32_t tmem_slot;
  __shared__ int s_timeout, s_issued, s_finished, s_claimed;

  if (tid == 0) {
    s_timeout = s_issued = s_finished = s_claimed = 0;
    for (int i = 0; i < S_::kRing; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kFp8 ? kConvWarps : 2);   // converters, or both MMA warps
    }
    for (int i = 0; i < kWide; ++i) {
      mbar_init(smem_u32(&conv_full[i]), kConvWarps);
      mbar_init(smem_u32(&wide_free[i]), 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), kRows);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&q_full[i]), kRows);
      mbar_init(smem_u32(&o_free[i]), kRows);
      mbar_init(smem_u32(&work_full[i]), 1);
      mbar_init(smem_u32(&work_empty[i]), kReaders);
    }
    mbar_init(smem_u32(&claim_bar), 1);
    mbar_init(smem_u32(&fin), 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProdWarp && lane < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &vmap : &kmap))
                 : "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // a warp-wide bounded wait
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(FULL, mbar_wait(smem_u32(bar), parity, kWaitNs));
  };
  // the k-th unit of this CTA: false where there is none (or a wait gave up)
  auto next_work = [&](int k, Work& w) -> bool {
    if (!wait(&work_full[k & 1], (k >> 1) & 1)) {
      if (lane == 0) atomicOr(&s_timeout, 1);
      return false;
    }
    w = s_work[k & 1];
    return w.s >= 0;
  };
  auto release_work = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&work_empty[k & 1]));
  };
  auto give_up = [&]() {
    if (lane == 0) atomicOr(&s_timeout, 1);
  };

  if (warp == kSchedWarp) {
    // ----------------------------------------------------------- scheduler
    // Unit x of the grid is KV head x % N_kv of slot x / N_kv; sequence s has
    // the slots from (query_start[s] * G) / 256 + s on, at least as many as
    // its 256-row pairs, the last pair (the most keys) first.
    int x = blockIdx.x, k = 0, asked = 0;
    while (true) {
      if (!(k < 2 || wait(&work_empty[k & 1], ((k >> 1) - 1) & 1))) {
        give_up();
        break;
      }
      Work w{-1, 0, 0, 0, 0, 0, 0};
      while (true) {   // until a unit with rows, or the end
        if (x < 0) {   // ask for one more block
          if (lane == 0) {
            mbar_arrive_expect_tx(smem_u32(&claim_bar), 16);
            claim_block(smem_u32(&s_answer), smem_u32(&claim_bar));
          }
          __syncwarp();
          if (!wait(&claim_bar, asked & 1)) {
            give_up();
            break;
          }
          ++asked;
          x = claimed_block(s_answer);
          fence_proxy_async();   // the answer is read: the next one may replace it
          __syncwarp();
          if (x < 0) break;
        }
        const int slot = x / a.num_kv_heads;
        w.kvh = x - slot * a.num_kv_heads;
        x = -1;
        auto slot0 = [&](int s) { return static_cast<int>(static_cast<int64_t>(a.query_start[s]) * G / kUnitRows) + s; };
        int lo = 0, hi = a.num_seqs;   // the last sequence whose slots start at or before `slot`
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32;
          const int s = lo + lane * step;
          const unsigned le = __ballot_sync(FULL, s < hi && slot0(s) <= slot);
          const int c = __popc(le);
          if (c == 0) break;
          lo += (c - 1) * step;
          hi = min(lo + step, hi);
        }
        const int q0 = a.query_start[lo], n = a.query_start[lo + 1] - q0, ctx = a.ctx_lens[lo];
        const int at = slot - slot0(lo);
        if (at < 0 || q0 < 0 || n <= 0 || n > a.total_q - q0) continue;   // no rows this call may write
        const int pairs = static_cast<int>((static_cast<int64_t>(n) * G + kUnitRows - 1) / kUnitRows);
        if (at >= pairs) continue;
        w.q0 = q0;
        w.n = n;
        w.ctx = ctx;
        w.pair = pairs - 1 - at;
        if (ctx < 0 || ctx > a.max_blocks * T || n > ctx || n > a.max_q_tiles) {
          // invalid lengths: the unit's rows become NaN (w.s stays -1)
          if (lane == 0 && a.status != nullptr) atomicOr(a.status, kBadLength);
          const int r0 = w.pair * kUnitRows, rows = min(n * G - r0, kUnitRows);
          for (int i = lane; i < rows * D; i += 32) {
            const int r = r0 + i / D;
            store_elem<Q>(a.out, ((static_cast<int64_t>(q0) + r / G) * a.num_q_heads + w.kvh * G + r % G) * D + i % D,
                          CUDART_NAN_F);
          }
          continue;
        }
        w.s = lo;
        break;
      }
      __syncwarp();
      if (lane == 0) {
        s_work[k & 1] = w;
        if (w.s >= 0) s_claimed = k + 1;
        mbar_arrive(smem_u32(&work_full[k & 1]));
      }
      ++k;
      if (w.s < 0) break;
    }
  } else if (warp == kProdWarp) {
    // ------------------------------------------------------------ producer
    // a lane's box of a step: chunk, slab, K or V
    constexpr int kBoxSlabs = kFp8 ? 1 : S_::kSlabs;
    constexpr int kBoxes = kStepChunks * kBoxSlabs * 2;
    const int bv = lane & 1, bsl = (lane >> 1) % kBoxSlabs, bc = (lane >> 1) / kBoxSlabs;
    int g = 0;   // steps of the K/V stream so far
    bool ok = true;
    Work w;
    for (int k = 0; ok && next_work(k, w); ++k) {
      const Unit u(w, a);
      const int32_t* trow = a.tables + static_cast<size_t>(u.s) * a.max_blocks;
      // lane l of batch b: the pool row (-1: none) and the scales of chunk 32 b + l
      auto fetch = [&](int b, int& row, float2& sc) {
        row = -1;
        sc = make_float2(0.f, 0.f);
        const int i = 32 * b + lane;
        if (i >= u.keys.n) return;
        const int p = u.keys.chunk(i) * kChunkKeys;
        const int blk = trow[p / T];
        if (blk < 0 || blk >= a.num_blocks) {
          atomicOr(&s_work[k & 1].bad, kBadTable);   // before the step is announced: the rows become NaN
          return;
        }
        const int slab = blk * a.num_kv_heads + u.kvh;
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
      for (int t = 0; t < u.steps; ++t, ++g) {
        if ((t & 7) == 0 && t > 0) {   // 32 chunks are 8 steps
          row_cur = row_nxt;
          sc_cur = sc_nxt;
          fetch(t / 8 + 1, row_nxt, sc_nxt);
        }
        const int slot = g % S_::kRing;
        if (g >= S_::kRing && !wait(&empty[slot], ((g / S_::kRing) - 1) & 1)) {
          give_up();
          ok = false;
          break;
        }
        const int c0 = (kStepChunks * t) & 31;
        const int row = __shfl_sync(FULL, row_cur, c0 + (bc & 3));
        const bool load = lane < kBoxes && row >= 0;
        if constexpr (BS) {
          const float ks = __shfl_sync(FULL, sc_cur.x, c0 + (lane & 3));
          const float vs = __shfl_sync(FULL, sc_cur.y, c0 + (lane & 3));
          const float x = lane < kStepChunks ? ks : vs;   // lanes 0-3: K scales, 4-7: V scales
          float top = fmaxf(x, __shfl_xor_sync(FULL, x, 1));
          top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
          const float ref = top > 0.f ? pow2_floor(top) : 1.f;
          if (lane < 2 * kStepChunks) {
            const __half2 h = __float2half2_rn(__fdividef(x, ref));
            s_ratio[g % kScaleRing][lane] = *reinterpret_cast<const uint32_t*>(&h);
            if ((lane & 3) == 0) s_ref[g % kScaleRing][lane >> 2] = ref;
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
        if (lane == 0) s_issued = g + 1;
      }
      release_work(k);
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ---------------------------------------------------------- MMA issuers
    // one warp a tile: its waits do not hold up the other tile's MMAs
    const int X = warp - kMmaWarp;
    const uint32_t leader = elect_one();
    const uint32_t tm = __reduce_max_sync(FULL, tmem) + 256 * X;   // uniform for the compiler as well
    const uint64_t q_desc = sw128_desc(smem_u32(q_s + X * S_::kQTile), 16, 1024);
    const uint64_t k_desc = sw128_desc(smem_u32(kv16), 16, 1024);
    const uint64_t v_desc = sw128_desc(smem_u32(kv16 + S_::kTile16), kSlab, 1024);
    uint64_t* kv_full = kFp8 ? conv_full : full;
    uint64_t* kv_free = kFp8 ? wide_free : empty;
    int g = 0, c = 0, units = 0;   // stream steps, this tile's steps and units so far
    bool ok = true;
    Work w;
    for (int k = 0; ok && next_work(k, w); ++k) {
      const Unit u(w, a);
      release_work(k);
      const int nt = X ? u.nt[1] : u.nt[0];
      auto qk = [&](int t) -> bool {
        const int slot = (g + t) % kBuf, i = 2 * X + ((c + t) & 1), use = (c + t) >> 1;
        if (!wait(&kv_full[slot], ((g + t) / kBuf) & 1)) return false;
        // the buffer's step before: its P has been read by P V
        if (use >= 1 && !wait(&o_done[i], (use - 1) & 1)) return false;
        tc_fence_after();
        const uint64_t kd = k_desc + ((slot * S_::kStage16) >> 4);
        const uint32_t d_tmem = tm + 64 * ((c + t) & 1);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss(leader, d_tmem, q_desc + (((ks >> 2) * kQSlab + 32 * (ks & 3)) >> 4),
                 kd + (((ks >> 2) * kSlab + 32 * (ks & 3)) >> 4), kIdQK, ks > 0 ? 1u : 0u);
        commit(leader, smem_u32(&s_full[i]));
        return true;
      };
      auto pv = [&](int t) -> bool {
        const int slot = (g + t) % kBuf, i = 2 * X + ((c + t) & 1);
        if (!wait(&p_full[i], ((c + t) >> 1) & 1)) return false;
        // O of the unit before has been read
        if (t == 0 && units > 0 && !wait(&o_free[X], (units - 1) & 1)) return false;
        tc_fence_after();
        const uint64_t vd = v_desc + ((slot * S_::kStage16) >> 4);
        const uint32_t p_tmem = tm + 64 * ((c + t) & 1);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(leader, tm + 128, p_tmem + 8 * kk, vd + ((2048 * kk) >> 4), kIdPV, (t > 0 || kk > 0) ? 1u : 0u);
        commit(leader, smem_u32(&o_done[i]));
        commit(leader, smem_u32(&kv_free[slot]));
        return true;
      };
      if (nt > 0) {
        ok = wait(&q_full[X], units & 1) && qk(0) && (nt < 2 || qk(1));
        for (int t = 0; t < nt && ok; ++t) ok = pv(t) && (t + 2 >= nt || qk(t + 2));
        ++units;
      }
      // the stream's steps that only the other tile reads
      for (int t = nt; t < u.steps && ok; ++t) {
        const int slot = (g + t) % kBuf;
        ok = wait(&kv_full[slot], ((g + t) / kBuf) & 1);
        if (ok && lane == 0) mbar_arrive(smem_u32(&kv_free[slot]));
      }
      if (!ok) give_up();
      g += u.steps;
      c += nt;
    }
    commit(leader, smem_u32(&fin));
  } else if (kFp8 && warp >= kConvWarp) {
    // ------------------------------------------------------------ converters
    // two warps K, two V; each half of the 64 rows, a 16-byte piece (16
    // elements) a lane at a time
    const int cw = warp - kConvWarp, tv = cw >> 1, half = cw & 1;
    int g = 0;
    bool ok = true;
    Work w;
    for (int k = 0; ok && next_work(k, w); ++k) {
      const Unit u(w, a);
      release_work(k);
      for (int t = 0; t < u.steps; ++t, ++g) {
        const int slot = g % S_::kRing, b = g % kWide;
        if (!wait(&full[slot], (g / S_::kRing) & 1) ||
            (g >= kWide && !wait(&wide_free[b], ((g / kWide) - 1) & 1))) {
          give_up();
          ok = false;
          break;
        }
        const uint8_t* src = ring + slot * S_::kStage8 + tv * S_::kTile8;
        uint8_t* dst = wide + b * S_::kStage16 + tv * S_::kTile16;
        const bool inner = u.keys.inner(t);
#pragma unroll 4
        for (int i = 0; i < 8; ++i) {
          const int e = lane + 32 * i;
          const int row = 32 * half + (e >> 3), c = e & 7;
          uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
          const int p = u.keys.chunk(kStepChunks * t + (row >> 4)) * kChunkKeys + (row & 15);
          if (tv == 0 || inner || u.keys.any_sees(p)) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + sw(row, c));
            const uint32_t in[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[2 * j] = e4m3x2_f16x2(in[j] & 0xffffu);
              y[2 * j + 1] = e4m3x2_f16x2(in[j] >> 16);
            }
            if constexpr (BS) {
              const uint32_t rb = s_ratio[g % kScaleRing][tv * kStepChunks + (row >> 4)];
              const __half2 ratio = *reinterpret_cast<const __half2*>(&rb);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const __half2 z = __hmul2(*reinterpret_cast<__half2*>(&y[j]), ratio);
                y[j] = *reinterpret_cast<const uint32_t*>(&z);
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
          mbar_arrive(smem_u32(&conv_full[b]));
          mbar_arrive(smem_u32(&empty[slot]));
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    // every branch around a warp-wide TMEM access is taken by the whole warp
    const int X = warp >> 2, r = tid & 127, rp = tid;   // tile, TMEM lane, row of the pair
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tX = tmem + 256 * X + lane_off, tO = tX + 128;
    uint8_t* qx = q_s + X * S_::kQTile;
    constexpr int kPieces = D / 8;            // 16-byte pieces of a row
    constexpr int kPer = kRows / (kRows / kPieces);
    // The tile's query rows, a 16-byte piece a thread: a warp reads whole rows
    auto load_q = [&](const Unit& u) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = r / kPieces + i * (kRows / kPieces), c = r % kPieces;
        uint8_t* d = qx + (c >> 3) * kQSlab + sw(row, c & 7);
        const int rr = kRows * X + row;
        if (rr < u.in_pair)
          cp_async16(smem_u32(d), static_cast<const typename Q::raw*>(a.q) + u.row_at(rr, a, D) + 8 * c);
        else
          *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);   // past the chunk's end
      }
    };
    auto announce_q = [&]() {
      cp_async_wait();
      if constexpr (kFp8 && kOutBf) {   // the MMA is f16: the thread's own pieces
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int row = r / kPieces + i * (kRows / kPieces), c = r % kPieces;
          uint4* d = reinterpret_cast<uint4*>(qx + (c >> 3) * kQSlab + sw(row, c & 7));
          uint4 v = *d;
          float f[8];
          LoadF32<Q, 8>::run(&v, f);
          *d = make_uint4(pack2<false>(f[0], f[1]), pack2<false>(f[2], f[3]), pack2<false>(f[4], f[5]),
                          pack2<false>(f[6], f[7]));
        }
      }
      fence_proxy_async();
      mbar_arrive(smem_u32(&q_full[X]));
    };
    int g = 0, c = 0;   // stream steps and this tile's steps so far
    bool ok = true;
    Work w;
    bool more = next_work(0, w);
    if (more) {
      const Unit u(w, a);
      if (X == 0 || u.nt[1] > 0) {
        load_q(u);
        announce_q();
      }
    }
    for (int k = 0; more && ok; ++k) {
      const Unit u(w, a);
      const int ntx = X ? u.nt[1] : u.nt[0];
      const HeadScales hs = head_scales(a.head_scales, a.num_kv_heads, u.kvh, a.softmax_scale, a.qk_scale,
                                        a.v_scale, 1.f, 1.f);
      const int pos = u.pos_of(min(rp, u.in_pair - 1), G);
      const int w0 = a.window > 0 ? pos - a.window + 1 : 0;
      float m_ref = -CUDART_INF_F, l = 0.f;
      bool q_next = false;
      for (int t = 0; t < ntx; ++t) {
        const int b = (c + t) & 1, i = 2 * X + b;
        if (!wait(&s_full[i], ((c + t) >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sv[64];
        {
          uint32_t h0[32], h1[32];
          tmem_ld32_async(tX + 64 * b, h0);
          tmem_ld32_async(tX + 64 * b + 32, h1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            sv[e] = __uint_as_float(h0[e]);
            sv[32 + e] = __uint_as_float(h1[e]);
          }
        }
        if (t == ntx - 1) {
          // the tile's last S is there, so its queries are done with: the
          // next unit's may take their place
          more = next_work(k + 1, w);
          if (more) {
            const Unit v(w, a);
            if (X == 0 || v.nt[1] > 0) {
              load_q(v);
              q_next = true;
            }
          }
        }
        float qe = hs.qk, lv = 0.f, inv_v = 1.f;
        if constexpr (BS) {
          // passed already; it orders the producer's scales before this read
          wait(&conv_full[(g + t) % kWide], ((g + t) / kWide) & 1);
          qe *= s_ref[(g + t) % kScaleRing][0];
          const uint32_t vb = __float_as_uint(s_ref[(g + t) % kScaleRing][1]);   // a power of two
          lv = static_cast<float>(static_cast<int>(vb >> 23) - 127);
          inv_v = __uint_as_float((254u << 23) - vb);
        }
        // mask: every key of the step lies in one run of positions unless it
        // holds sinks' chunks
        const int p0 = u.keys.chunk(kStepChunks * t) * kChunkKeys;
        if (!(kStepChunks * t >= u.keys.ns && p0 >= w0 && p0 + kKeys - 1 <= pos)) {
#pragma unroll
          for (int ch = 0; ch < kStepChunks; ++ch) {
            const int pc = u.keys.chunk(kStepChunks * t + ch) * kChunkKeys;
            const int hi = pos - pc, lo = w0 - pc, sk = u.keys.sinks - pc;
#pragma unroll
            for (int e = 0; e < kChunkKeys; ++e)
              if (e > hi || (e < lo && e >= sk)) sv[16 * ch + e] = -CUDART_INF_F;
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
        for (int j = 0; j < 8; ++j) mx8[j] = sv[j];
#pragma unroll
        for (int e = 8; e < 64; ++e) mx8[e & 7] = fmaxf(mx8[e & 7], sv[e]);
        const float mx = fmaf(qe, fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                        fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))), lv);
        const bool move = mx > m_ref + kRescaleLog2;
        const bool scale = move && t > 0 && m_ref != -CUDART_INF_F;   // O holds earlier steps
        if (__any_sync(FULL, scale)) {
          const int ip = 2 * X + ((c + t - 1) & 1);
          if (!wait(&o_done[ip], ((c + t - 1) >> 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f = scale ? ex2(m_ref - mx) : 1.f;
#pragma unroll 1
          for (int e0 = 0; e0 < D; e0 += 32) {
            float o[32];
            tmem_ld32(tO + e0, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(tO + e0, o);
          }
          l *= f;
        }
        if (move) m_ref = mx;
        // a row that has seen nothing yet keeps every weight 0
        const float off = lv - (m_ref == -CUDART_INF_F ? 0.f : m_ref);
        float sum8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum8[j] = 0.f;
        uint32_t pw[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float e0 = ex2(fmaf(sv[2 * e], qe, off));
          const float e1 = ex2(fmaf(sv[2 * e + 1], qe, off));
          sum8[(2 * e) & 7] += e0;
          sum8[(2 * e + 1) & 7] += e1;
          pw[e] = pack2<kBf>(e0, e1);
        }
        tmem_st32u(tX + 64 * b, pw);
        l = fmaf(((sum8[0] + sum8[1]) + (sum8[2] + sum8[3])) + ((sum8[4] + sum8[5]) + (sum8[6] + sum8[7])),
                 inv_v, l);
        // V rows that nobody sees (16-bit caches; the converters leave zeros);
        // both tiles' threads write them, each before its own P V
        if constexpr (!kFp8) {
          if (!u.keys.inner(t) && r < kKeys) {
            const int p = u.keys.chunk(kStepChunks * t + (r >> 4)) * kChunkKeys + (r & 15);
            if (!u.keys.any_sees(p)) {
              uint8_t* vt = ring + ((g + t) % S_::kRing) * S_::kStage16 + S_::kTile16 + r * 128;
#pragma unroll
              for (int e = 0; e < 8 * S_::kSlabs; ++e)
                *reinterpret_cast<uint4*>(vt + (e >> 3) * kSlab + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async();   // before the tensor core reads V
            }
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&p_full[i]));
      }
      if (!ok) {
        give_up();
        break;
      }
      if (ntx == 0) {   // tile B has no rows in this unit
        more = next_work(k + 1, w);
        if (more) {
          const Unit v(w, a);
          if (v.nt[1] > 0) {
            load_q(v);
            q_next = true;
          }
        }
      }
      if (q_next) announce_q();
      // epilogue: O / l, after the tile's last P V
      if (ntx > 0) {
        const int cl = c + ntx - 1;
        if (!wait(&o_done[2 * X + (cl & 1)], (cl >> 1) & 1)) {
          give_up();
          ok = false;
          break;
        }
        tc_fence_after();
        const bool bad = *reinterpret_cast<volatile int*>(&s_work[k & 1].bad) != 0;
        const float inv = bad ? CUDART_NAN_F : (l > 0.f || l != l) ? hs.v / l : 0.f;
        typename Q::raw* dst = static_cast<typename Q::raw*>(a.out) + u.row_at(min(rp, u.in_pair - 1), a, D);
#pragma unroll 1
        for (int e0 = 0; e0 < D; e0 += 32) {
          float o[32];
          tmem_ld32(tO + e0, o);
          if (e0 + 32 == D) {   // O is in registers: the next unit's first P V may replace it
            tc_fence_before();
            mbar_arrive(smem_u32(&o_free[X]));
          }
          if (rp < u.in_pair) {
            uint32_t ow[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              ow[e] = pack2<kOutBf>(bad ? CUDART_NAN_F : o[2 * e] * inv, bad ? CUDART_NAN_F : o[2 * e + 1] * inv);
            uint4* d4 = reinterpret_cast<uint4*>(dst + e0);
#pragma unroll
            for (int e = 0; e < 4; ++e) d4[e] = make_uint4(ow[4 * e], ow[4 * e + 1], ow[4 * e + 2], ow[4 * e + 3]);
          }
        }
        if (r == 0 && bad && a.status != nullptr) atomicOr(a.status, s_work[k & 1].bad);
      }
      if (rp == 0) s_finished = k + 1;
      release_work(k);
      g += u.steps;
      c += ntx;
    }
  }

  // every MMA done and every copy landed before TMEM and shared memory go
  __syncthreads();
  if (tid == 0) {
    mbar_wait(smem_u32(&fin), 0, kDrainNs);
    if (s_timeout) {
      const int issued = s_issued;
      for (int t = max(0, issued - S_::kRing); t < issued; ++t)
        mbar_wait(smem_u32(&full[t % S_::kRing]), (t / S_::kRing) & 1, kDrainNs);
      if (a.status != nullptr) atomicOr(a.status, kTimeout);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s_timeout) {
    // the units this CTA claimed and did not finish (a claimed unit keeps its
    // description until every reader is done with it)
    for (int k = max(s_finished - 1, 0); k < s_claimed; ++k) {
      const Work w = s_work[k & 1];
      if (w.s < 0 || k + 2 < s_claimed) continue;
      const int r0 = w.pair * kUnitRows, rows = min(w.n * G - r0, kUnitRows);
      for (int i = tid; i < rows * D; i += S_::kThreads) {
        const int r = r0 + i / D;
        store_elem<Q>(a.out, ((static_cast<int64_t>(w.q0) + r / G) * a.num_q_heads + w.kvh * G + r % G) * D + i % D,
                      CUDART_NAN_F);
      }
    }
  }
  if (warp == kMmaWarp) {
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
  // every sequence's slots of 256 rows (see the scheduler), one block each;
  // the blocks that start claim the others one by one
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.group;
  const int64_t units = (rows / kUnitRows + a.num_seqs) * a.num_kv_heads;
  if (rows > INT32_MAX || units > INT32_MAX)
    return fail(PKV_ERR_UNSUPPORTED, "windowed prefill: too many query rows in one call");
  a.max_q_tiles = max_query_len;   // the longest chunk the caller allows
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units));
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
