// Prefill attention with a sliding window and sinks, and over block-scaled
// E4M3 caches, on the 5th-generation tensor cores.
//
// The chunk of sequence s is its last n positions; the query at position p
// sees p' <= p with p' > p - window or p' < sinks (window 0: every p' <= p).
//   out = softmax(q . K^T * scale) V  over what it sees.
//
// A unit of work is 256 query rows of one KV head as two tiles of 128 (M of an
// MMA).  Row r of a chunk is head r % G of position r / G: the G query heads
// that share a KV head share its K/V tiles, and 256 rows span 256 / G
// positions only, so that with a window little more than its own keys is
// read and multiplied.  The keys those rows see are walked in steps of 64, as
// four chunks of 16 each: the sinks' chunks, then those from the first row's
// window on; blocks between are not looked up.
//
// One CTA of 16 warps lives on each SM and claims units as it goes (cluster
// launch control).  Warps 0-3 and 4-7 do the softmax of tile A and B (a thread
// a row, TMEM lane = row), warp 8 drives TMA, warps 9 and 10 issue the MMAs,
// warp 11 claims and describes units, warps 12-15 load queries, widen E4M3 and
// write the output of a unit while the next one runs:
//   S_t = Q K_t^T  (128 x 64, into one of two TMEM buffers per tile)
//   P_t = 2^(S_t scale - m)  (16 bit, over the S buffer it came from)
//   O  += P_t V_t  (128 x D, A operand from TMEM)
// S_{t+2} is issued when P_t V_t is done, so the tensor core stays two steps
// ahead of the softmax.  O stays in TMEM; a row's reference m moves only when
// its running maximum has grown by 2^8, and then its O is rescaled.  The pool
// rows (and scales) of 32 chunks are fetched a lane each, a batch ahead, and
// the boxes of a step go out a lane each.
//
// Measured (GB300, 152 SMs), of 1870 TFLOP/s that a library product reaches:
//   one prompt of 8,192, 32 query / 8 KV heads, window 2,048, bf16:  189 us, 1273 TFLOP/s
//   16 chunks of 512, 28 / 4 heads, window 1,024, bf16:               84 us, 1050 TFLOP/s
//   16 block-scaled E4M3 chunks of 512 over 1,024 to 4,096 tokens:   238 us,  924 TFLOP/s
// What bounds it: a step of both tiles takes 1,300 to 1,450 cycles.  With N =
// 64 its Q K^T reads 6 KB of shared memory per MMA of 32 tensor cycles (1,280
// cycles a step at 128 bytes a cycle, with P V); the 16 TMA boxes of a step
// cost their warp about 80 cycles each; and the two issuing warps wait on
// barriers between.  Half the MMA work alone takes 4% off, a quarter of the
// boxes alone 3%, both 16%.  Keys in steps of 128 do not fit TMEM beside O
// with two buffers.
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
constexpr int kUnitRows = 2 * kRows;              // query rows of a unit
// warps: 0-7 softmax (four a tile), TMA, MMA of tile A and B, scheduler, four helpers
constexpr int kProdWarp = 8, kMmaWarp = 9, kSchedWarp = 11, kHelpWarp = 12;
constexpr int kThreadsW = 512;
constexpr int kWideK = 2, kWideV = 3;             // widened K and V buffers (E4M3)
constexpr int kScaleRing = 16;                    // steps whose scales are kept: more than are in flight

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
  static constexpr int kTile = kKeys * D * KV::bytes;       // as it is stored
  static constexpr int kStage = 2 * kTile;                  // K, then V
  static constexpr int kRing = 5;                           // TMA stages
  static constexpr int kWideBytes = kFp8 ? (kWideK + kWideV) * kTile16 : 0;
  static constexpr int kSmem = 1024 + 2 * kQTile + kRing * kStage + kWideBytes;
  // 16-bit K and V of a step as the MMAs see them: the ring's stages, or the
  // widened buffers
  static constexpr int kBufK = kFp8 ? kWideK : kRing, kBufV = kFp8 ? kWideV : kRing;
  static constexpr int kStrideK = kFp8 ? kTile16 : kStage, kStrideV = kStrideK;
};

using Args = WindowPrefillArgs;

// 256 rows of one KV head of one chunk, as the scheduler announces them: tile X
// is rows [128 X, 128 X + 128).
struct Work {
  int s, kvh, q0, row0, in_pair;   // s < 0: no more work; row0: the unit's first chunk row
  int pos0, rem0;                  // that row is head rem0 of position pos0
  int n;                           // of the chunk
  Keys keys;
  int nt[2], steps;                // 64-key steps of each tile, and of the K/V stream
  int bad;                         // PKV_DEVICE_* bits met while it ran
  __device__ __forceinline__ void set(int seq, int kv_head, int q_first, int len, int ctx, int pair, const Args& a) {
    const int G = a.group;
    s = seq;
    kvh = kv_head;
    q0 = q_first;
    n = len;
    row0 = pair * kUnitRows;
    in_pair = min(len * G - row0, kUnitRows);
    const int first = ctx - len;
    pos0 = first + row0 / G;
    rem0 = row0 % G;
    keys.set(pos0, first + (row0 + in_pair - 1) / G, a.window, a.sinks);
    const int endA = (first + (row0 + min(in_pair, kRows) - 1) / G) / kChunkKeys + 1;
    nt[0] = max((keys.ns + max(endA - keys.wb, 0) + kStepChunks - 1) / kStepChunks, 1);
    steps = (keys.n + kStepChunks - 1) / kStepChunks;
    nt[1] = in_pair > kRows ? steps : 0;
    steps = max(nt[0], nt[1]);
    bad = 0;
  }
  // position and head of row r (< 256) of the unit; inv_g = 1 / G.  rem0 + r is
  // small, so that the product with half a row added falls on the right side.
  __device__ __forceinline__ void place(int r, int G, float inv_g, int* pos, int* head) const {
    const int i = static_cast<int>((static_cast<float>(rem0 + r) + 0.5f) * inv_g);
    *pos = pos0 + i;
    *head = rem0 + r - i * G;
  }
  // element offset of head j at position pos in q and out
  __device__ __forceinline__ int64_t at(int pos, int j, const Args& a, int D) const {
    const int64_t row = static_cast<int64_t>(q0) + (pos - pos0) + row0 / a.group;
    return (row * a.num_q_heads + kvh * a.group + j) * D;
  }
};

// A place in a ring of N buffers and the parity of its use.
template <int N>
struct RingPos {
  int slot = 0;
  uint32_t par = 0;
  bool used = false;   // the buffer has been used before
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      par ^= 1;
      used = true;
    }
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

// Two fp32 operations in one instruction, and the largest of three.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {   // NaN if one is
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
__global__ void __launch_bounds__(kThreadsW, 1)
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
  constexpr int kRing = S_::kRing, kBufK = S_::kBufK, kBufV = S_::kBufV;
  constexpr int kReaders = 15;   // warps that read a unit's description: all but the scheduler

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group, HQ = a.num_q_heads, T = a.block_size;
  const float inv_g = 1.f / static_cast<float>(G);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* q_s = smem;                             // [tile][slab][128 rows][128 B]
  uint8_t* ring = smem + 2 * S_::kQTile;           // [stage][K, V](16-bit: [slab])
  uint8_t* wide = ring + kRing * S_::kStage;       // E4M3: widened K buffers, then V's
  uint8_t* k16 = kFp8 ? wide : ring;
  uint8_t* v16 = kFp8 ? wide + kWideK * S_::kTile16 : ring + S_::kTile;
  __shared__ uint64_t full[kRing], empty[kRing];
  __shared__ uint64_t k_full[kWideK], k_free[kWideK], v_full[kWideV], v_free[kWideV];   // E4M3
  __shared__ uint64_t q_full[2], q_free[2], s_full[4], p_full[4], o_done[4], o_free[2], l_full[2], fin;
  __shared__ uint64_t work_full[2], work_empty[2], claim_bar;
  __shared__ ulonglong2 s_answer;
  __shared__ Work s_work[2];
  __shared__ __half s_ratio[BS ? kScaleRing : 1][2 * kStepChunks];   // scale / R: K, then V chunks
  __shared__ __align__(8) float s_ref[BS ? kScaleRing : 1][2];                      // R of K and V
  __shared__ float s_inv[2][kRows];                                    // 1 / l of a finished row
  __shared__ uint32_t tmem_slot;
  __shared__ int s_timeout, s_issued, s_finished, s_claimed;

  if (tid == 0) {
    s_timeout = s_issued = s_finished = s_claimed = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kFp8 ? 4 : 1);   // the helper warps, or the P V warp
    }
    for (int i = 0; i < kWideK; ++i) {
      mbar_init(smem_u32(&k_full[i]), 2);   // the two warps that widen K
      mbar_init(smem_u32(&k_free[i]), 2);   // both MMA warps
    }
    for (int i = 0; i < kWideV; ++i) {
      mbar_init(smem_u32(&v_full[i]), 2);
      mbar_init(smem_u32(&v_free[i]), 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), kRows);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&q_full[i]), kFp8 ? kRows : 2 * kRows);   // helper threads (and their copies)
      mbar_init(smem_u32(&q_free[i]), 1);
      mbar_init(smem_u32(&o_free[i]), kRows);
      mbar_init(smem_u32(&l_full[i]), kRows);
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
    if (__all_sync(FULL, mbar_try_wait(smem_u32(bar), parity))) return true;
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
    // Unit x of the grid is KV head x % N_kv of slot x / N_kv; of more than 32
    // sequences, s has the slots from (query_start[s] * G) / 256 + s on, at
    // least as many as its 256-row pairs, the last pair (the most keys) first.
    int x = blockIdx.x, k = 0, asked = 0;
    // Up to 32 sequences are taken longest first, lane s keeping sequence s and
    // its first slot in that order: a long unit that starts last would leave
    // the other SMs idle.
    const bool few = a.num_seqs <= 32;
    int my_q0 = 0, my_n = 0, my_ctx = 0, my_units = 0, my_slot = 0;
    if (few) {
      if (lane < a.num_seqs) {
        my_q0 = a.query_start[lane];
        my_n = a.query_start[lane + 1] - my_q0;
        my_ctx = a.ctx_lens[lane];
        if (my_q0 >= 0 && my_n >= 0 && my_n <= a.total_q - my_q0)
          my_units = static_cast<int>((static_cast<int64_t>(my_n) * G + kUnitRows - 1) / kUnitRows);
        else if (a.status != nullptr)   // rows outside the inputs: none that this call may write
          atomicOr(a.status, kBadLength);
      }
      for (int o = 0; o < a.num_seqs; ++o) {
        const int ctx = __shfl_sync(FULL, my_ctx, o), units = __shfl_sync(FULL, my_units, o);
        if (ctx > my_ctx || (ctx == my_ctx && o < lane)) my_slot += units;
      }
    }
    while (true) {
      if (!(k < 2 || wait(&work_empty[k & 1], ((k >> 1) - 1) & 1))) {
        give_up();
        break;
      }
      Work w;
      w.s = -1;
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
        const int kvh = x - slot * a.num_kv_heads;
        x = -1;
        int lo = 0, q0, n, ctx, at, pairs;
        if (few) {
          const unsigned here = __ballot_sync(FULL, slot >= my_slot && slot - my_slot < my_units);
          if (here == 0) continue;   // more blocks than units
          lo = __ffs(here) - 1;
          q0 = __shfl_sync(FULL, my_q0, lo);
          n = __shfl_sync(FULL, my_n, lo);
          ctx = __shfl_sync(FULL, my_ctx, lo);
          pairs = __shfl_sync(FULL, my_units, lo);
          at = slot - __shfl_sync(FULL, my_slot, lo);
        } else {
          auto slot0 = [&](int s) {
            return static_cast<int>(static_cast<int64_t>(a.query_start[s]) * G / kUnitRows) + s;
          };
          int hi = a.num_seqs;   // the last sequence whose slots start at or before `slot`
          while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int s = lo + lane * step;
            const unsigned le = __ballot_sync(FULL, s < hi && slot0(s) <= slot);
            const int c = __popc(le);
            if (c == 0) break;
            lo += (c - 1) * step;
            hi = min(lo + step, hi);
          }
          q0 = a.query_start[lo];
          n = a.query_start[lo + 1] - q0;
          ctx = a.ctx_lens[lo];
          at = slot - slot0(lo);
          if (q0 < 0 || n < 0 || n > a.total_q - q0) {   // rows outside the inputs: none that this call may write
            if (lane == 0 && a.status != nullptr) atomicOr(a.status, kBadLength);
            continue;
          }
          if (at < 0) continue;
          pairs = static_cast<int>((static_cast<int64_t>(n) * G + kUnitRows - 1) / kUnitRows);
          if (at >= pairs) continue;
        }
        const int pair = pairs - 1 - at;
        if (ctx < 0 || ctx > a.max_blocks * T || n > ctx || n > a.max_q_tiles) {
          // invalid lengths: the unit's rows become NaN
          if (lane == 0 && a.status != nullptr) atomicOr(a.status, kBadLength);
          const int r0 = pair * kUnitRows, rows = min(n * G - r0, kUnitRows);
          for (int i = lane; i < rows * D; i += 32) {
            const int r = r0 + i / D;
            store_elem<Q>(a.out, ((static_cast<int64_t>(q0) + r / G) * a.num_q_heads + kvh * G + r % G) * D + i % D,
                          CUDART_NAN_F);
          }
          continue;
        }
        w.set(lo, kvh, q0, n, ctx, pair, a);
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
    RingPos<kRing> at;
    bool ok = true;
    Work w;
    for (int k = 0; ok && next_work(k, w); ++k) {
      const Work& u = w;
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
      for (int t = 0; t < u.steps; ++t, ++g, at.next()) {
        if ((t & 7) == 0 && t > 0) {   // 32 chunks are 8 steps
          row_cur = row_nxt;
          sc_cur = sc_nxt;
          fetch(t / 8 + 1, row_nxt, sc_nxt);
        }
        const int slot = at.slot;
        if (at.used && !wait(&empty[slot], at.par ^ 1)) {
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
            s_ratio[g % kScaleRing][lane] = __float2half_rn(__fdividef(x, ref));
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
          uint8_t* dst = ring + slot * S_::kStage + bv * S_::kTile + bsl * kSlab + bc * (kChunkKeys * 128);
          tma_load_2d(smem_u32(dst), bv ? &vmap : &kmap, bsl * 128, row, bar);
        }
        if (lane == 0) s_issued = g + 1;
      }
      release_work(k);
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ---------------------------------------------------------- MMA issuers
    // No vote in a wait: an instruction is its leader's, and votes added up in
    // a warp's chain.  A lane whose wait gives up goes on without waiting to
    // the end of the unit, where the lanes agree to stop (what it issues until
    // then stays within the CTA's shared memory and TMEM).
    bool late = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!late) late = !mbar_wait(smem_u32(bar), parity, kWaitNs);
    };
    const uint32_t leader = elect_one();
    const uint32_t tm = __reduce_max_sync(FULL, tmem);   // uniform for the compiler as well
    const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024);
    const uint64_t k_desc = sw128_desc(smem_u32(k16), 16, 1024);
    const uint64_t v_desc = sw128_desc(smem_u32(v16), kSlab, 1024);
    // S of a step of tile X from K buffer `slot`, into buffer `to` of the tile
    auto qk = [&](int X, int slot, int to) {
      const uint64_t kd = k_desc + static_cast<uint32_t>(slot * (S_::kStrideK >> 4));
      const uint32_t d_tmem = tm + 256 * X + 64 * to;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        mma_ss(leader, d_tmem, q_desc + ((X * S_::kQTile + (ks >> 2) * kQSlab + 32 * (ks & 3)) >> 4),
               kd + (((ks >> 2) * kSlab + 32 * (ks & 3)) >> 4), kIdQK, ks > 0 ? 1u : 0u);
      commit(leader, smem_u32(&s_full[2 * X + to]));
    };
    // O += P V of a step of tile X, P in buffer `from`, V in buffer `slot`
    auto pv = [&](int X, int slot, int from, bool first) {
      const uint64_t vd = v_desc + static_cast<uint32_t>(slot * (S_::kStrideV >> 4));
      const uint32_t o_tmem = tm + 256 * X + 128, p_tmem = tm + 256 * X + 64 * from;
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)
        mma_ts(leader, o_tmem, p_tmem + 8 * kk, vd + ((2048 * kk) >> 4), kIdPV, (!first || kk > 0) ? 1u : 0u);
      commit(leader, smem_u32(&o_done[2 * X + from]));
    };
    // The work is split by tile for E4M3 caches and by product for 16-bit ones:
    //   one prompt of 8,192, window 2,048, bf16: 198 us by tile, 190 by product
    //   16 chunks of 512, window 1,024, bf16:     91 us,           86
    //   16 block-scaled chunks of 512:           270 us,          340
    // By product no warp waits for a P V before it comes to the next Q K^T, but
    // the tiles keep step, and both wait when a widened buffer comes late.
    Work w;
    if constexpr (kFp8) {
      const int X = warp - kMmaWarp;
      RingPos<kBufK> kp;   // of the next Q K^T
      RingPos<kBufV> vp;   // of the next P V
      RingPos<2> sq, sp;   // S / P buffers of the next Q K^T and the next P V
      int units = 0;       // of this tile so far
      for (int k = 0; next_work(k, w); ++k) {
        const int nt = X ? w.nt[1] : w.nt[0], steps = w.steps;
        release_work(k);
        auto next_qk = [&](bool last) {
          wait(&k_full[kp.slot], kp.par);
          // the buffer's step before: its P has been read by P V
          if (sq.used) wait(&o_done[2 * X + sq.slot], sq.par ^ 1);
          tc_fence_after();
          qk(X, kp.slot, sq.slot);
          commit(leader, smem_u32(&k_free[kp.slot]));
          if (last) commit(leader, smem_u32(&q_free[X]));
          kp.next();
          sq.next();
        };
        if (nt > 0) {
          wait(&q_full[X], units & 1);
          next_qk(nt == 1);
          if (nt > 1) next_qk(nt == 2);
          for (int t = 0; t < nt; ++t) {
            // O of the unit before has been read
            if (t == 0 && units > 0) wait(&o_free[X], (units - 1) & 1);
            wait(&p_full[2 * X + sp.slot], sp.par);
            tc_fence_after();
            pv(X, vp.slot, sp.slot, t == 0);
            commit(leader, smem_u32(&v_free[vp.slot]));
            vp.next();
            sp.next();
            if (t + 2 < nt) next_qk(t + 3 == nt);
          }
          ++units;
        }
        // the stream's steps that only the other tile reads
        for (int t = nt; t < steps; ++t) {
          wait(&k_full[kp.slot], kp.par);
          wait(&v_full[vp.slot], vp.par);
          if (lane == 0) {
            mbar_arrive(smem_u32(&k_free[kp.slot]));
            mbar_arrive(smem_u32(&v_free[vp.slot]));
          }
          kp.next();
          vp.next();
        }
        if (__any_sync(FULL, late)) {
          give_up();
          break;
        }
      }
    } else if (warp == kMmaWarp) {
      RingPos<kRing> at;       // stage of the stream
      RingPos<2> buf[2];       // each tile's next S / P buffer
      int units[2] = {0, 0};   // of each tile so far
      for (int k = 0; next_work(k, w); ++k) {
        const int nt[2] = {w.nt[0], w.nt[1]}, steps = w.steps;
        release_work(k);
        for (int t = 0; t < steps; ++t) {
          wait(&full[at.slot], at.par);
#pragma unroll
          for (int X = 0; X < 2; ++X) {
            if (t >= nt[X]) continue;
            if (t == 0) {
              wait(&q_full[X], units[X] & 1);
              fence_proxy_async();   // copies by threads, before the tensor core reads them
            }
            // the buffer's step before: its P has been read by P V
            if (buf[X].used) wait(&o_done[2 * X + buf[X].slot], buf[X].par ^ 1);
            tc_fence_after();
            qk(X, at.slot, buf[X].slot);
            if (t + 1 == nt[X]) commit(leader, smem_u32(&q_free[X]));
            buf[X].next();
          }
          at.next();
        }
        units[0] += nt[0] > 0;
        units[1] += nt[1] > 0;
        if (__any_sync(FULL, late)) {
          give_up();
          break;
        }
      }
    } else {
      RingPos<kRing> at;
      RingPos<2> buf[2];
      int units[2] = {0, 0};
      for (int k = 0; next_work(k, w); ++k) {
        const int nt[2] = {w.nt[0], w.nt[1]}, steps = w.steps;
        const Keys keys = w.keys;
        // steps [inner0, inner1) have no V row that nobody sees
        const int inner0 = (keys.ns + (keys.wb * kChunkKeys < keys.w0) + kStepChunks - 1) / kStepChunks;
        const int inner1 = (keys.ns + max((keys.last + 1) / kChunkKeys - keys.wb, 0)) / kStepChunks;
        release_work(k);
        for (int t = 0; t < steps; ++t) {
          if (t < inner0 || t >= inner1) {   // such rows become zeros while P is made
            constexpr int kPieces = 8 * S_::kSlabs;   // 16-byte pieces of a row, a lane each
            uint8_t* vt = ring + at.slot * S_::kStage + S_::kTile + (lane % kPieces >> 3) * kSlab + (lane & 7) * 16;
            wait(&full[at.slot], at.par);
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = keys.chunk(kStepChunks * t + 2 * h + (lane >> 4));
              const uint32_t none = __ballot_sync(FULL, !keys.any_sees(c * kChunkKeys + (lane & 15)));
              if (none != 0)
                for (int r = lane / kPieces; r < 32; r += 32 / kPieces)
                  if (none >> r & 1u)
                    *reinterpret_cast<uint4*>(vt + (32 * h + r) * 128) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();   // before the tensor core reads V
            __syncwarp();
          }
#pragma unroll
          for (int X = 0; X < 2; ++X) {
            if (t >= nt[X]) continue;
            // O of the unit before has been read
            if (t == 0 && units[X] > 0) wait(&o_free[X], (units[X] - 1) & 1);
            wait(&p_full[2 * X + buf[X].slot], buf[X].par);
            tc_fence_after();
            pv(X, at.slot, buf[X].slot, t == 0);
            buf[X].next();
          }
          // (the stage's K has been read as well: P follows from S)
          commit(leader, smem_u32(&empty[at.slot]));
          at.next();
        }
        units[0] += nt[0] > 0;
        units[1] += nt[1] > 0;
        if (__any_sync(FULL, late)) {
          give_up();
          break;
        }
      }
    }
    commit(leader, smem_u32(&fin));
  } else if (warp >= kHelpWarp) {
    // -------------------------------------------------------------- helpers
    // Four warps load the queries of each unit, write its output, and, for
    // E4M3 caches, widen its K (two warps) and V (the other two).  A unit's
    // queries follow as soon as the last S of the unit before is done; its
    // first two steps are widened before that unit's output is waited for.
    const int hw = warp - kHelpWarp, ht = tid - 32 * kHelpWarp;
    constexpr int kPieces = D / 8;                 // 16-byte pieces of a query row
    constexpr int kRowStep = kRows / kPieces;      // rows the 128 threads cover at a time
    const int qc = ht % kPieces, qr = ht / kPieces;
    const int di = kRowStep / G, dj = kRowStep - di * G;
    const int64_t step = (static_cast<int64_t>(di) * HQ + dj) * D, wrap = static_cast<int64_t>(HQ - G) * D;
    // rows qr, qr + kRowStep, .. of tile X: eight rows on, a piece keeps its
    // place in the swizzle
    auto load_q = [&](const Work& u, int X) {
      uint32_t d = smem_u32(q_s + X * S_::kQTile + (qc >> 3) * kQSlab + sw(qr, qc & 7));
      int pos, j;
      u.place(kRows * X + qr, G, inv_g, &pos, &j);
      const typename Q::raw* src = static_cast<const typename Q::raw*>(a.q) + u.at(pos, j, a, D) + 8 * qc;
      const int rows = u.in_pair - kRows * X;   // of the tile inside the chunk
#pragma unroll 4
      for (int row = qr; row < kRows; row += kRowStep) {
        if (row < rows) cp_async16(d, src);
        else asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(d), "r"(0) : "memory");
        d += kRowStep * 128;
        src += step;
        j += dj;
        if (j >= G) {
          j -= G;
          src += wrap;
        }
      }
    };
    auto announce_q = [&](int X) {
      if constexpr (!kFp8) {
        // the copies announce themselves, so that this unit's output need not
        // wait for the next one's queries; who waits for them fences
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&q_full[X])) : "memory");
        mbar_arrive(smem_u32(&q_full[X]));
        return;
      }
      cp_async_wait();
      if constexpr (kFp8 && kOutBf) {   // the MMA is f16: the thread's own pieces
        uint8_t* qx = q_s + X * S_::kQTile + (qc >> 3) * kQSlab;
#pragma unroll 4
        for (int row = qr; row < kRows; row += kRowStep) {
          uint4* d = reinterpret_cast<uint4*>(qx + sw(row, qc & 7));
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
    int g = 0;   // steps widened so far
    int units[2] = {0, 0}, loads[2] = {0, 0};
    int last_buf[2] = {1, 1};   // S / P buffer of the tile's last step so far
    uint32_t last_par[2] = {1, 1};
    auto queries = [&](const Work& u) -> bool {
#pragma unroll
      for (int X = 0; X < 2; ++X) {
        if (X == 1 && u.nt[1] == 0) continue;
        // the tile's last S of the unit before is done
        if (loads[X] > 0 && !wait(&q_free[X], (loads[X] - 1) & 1)) return false;
        load_q(u, X);
        announce_q(X);
        ++loads[X];
      }
      return true;
    };
    // Steps [t0, t1) of a unit, widened; each warp half of the 64 rows of K or
    // V, a 16-byte piece (16 elements) a lane at a time.  Lanes of the upper
    // head_dim half store their two pieces in the other order: the two halves'
    // slabs share banks.
    const int tv = hw >> 1, half = hw & 1;
    RingPos<kRing> at;
    int buf = 0;
    uint32_t buf_par = 0;
    bool buf_used = false;
    auto widen = [&](const Work& u, int t0, int t1) -> bool {
      uint64_t* done = tv ? v_full : k_full;
      uint64_t* freed = tv ? v_free : k_free;
      const int bufs = tv ? kWideV : kWideK;
      const int rl = lane >> 3, cc = lane & 7;   // row of four, piece of its 8
      const bool upper = cc >= 4;
      for (int t = t0; t < t1; ++t) {
        if (!wait(&full[at.slot], at.par)) return false;
        if (buf_used && !wait(&freed[buf], buf_par ^ 1)) return false;
        const uint8_t* src = ring + at.slot * S_::kStage + tv * S_::kTile;
        uint8_t* dst = (tv ? v16 : k16) + buf * S_::kTile16 + (cc >> 2) * kSlab;
        __half2 ratio[2];
        if constexpr (BS) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            ratio[e] = __half2half2(s_ratio[g % kScaleRing][tv * kStepChunks + 2 * half + e]);
        }
        auto piece = [&](int i, const uint4& x) {
          const int row = 32 * half + 4 * i + rl;
          const uint32_t in[4] = {x.x, x.y, x.z, x.w};
          uint32_t y[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[2 * j] = e4m3x2_f16x2(in[j] & 0xffffu);
            y[2 * j + 1] = e4m3x2_f16x2(in[j] >> 16);
          }
          if constexpr (BS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __half2 z = __hmul2(*reinterpret_cast<__half2*>(&y[j]), ratio[i >> 2]);
              y[j] = *reinterpret_cast<const uint32_t*>(&z);
            }
          }
          // head_dim 16 cc .. 16 cc + 15: pieces 2 (cc % 4) and the next of slab cc / 4
          const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
          *reinterpret_cast<uint4*>(dst + sw(row, 2 * (cc & 3) + upper)) = upper ? hi : lo;
          *reinterpret_cast<uint4*>(dst + sw(row, 2 * (cc & 3) + !upper)) = upper ? lo : hi;
        };
        if (tv == 0 || u.keys.inner(t)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = *reinterpret_cast<const uint4*>(src + sw(32 * half + 16 * h + 4 * i + rl, cc));
#pragma unroll
            for (int i = 0; i < 4; ++i) piece(4 * h + i, x[i]);
          }
        } else {   // V rows that nobody sees become zeros
          for (int i = 0; i < 8; ++i) {
            const int row = 32 * half + 4 * i + rl;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (u.keys.any_sees(u.keys.chunk(kStepChunks * t + (row >> 4)) * kChunkKeys + (row & 15)))
              x = *reinterpret_cast<const uint4*>(src + sw(row, cc));
            piece(i, x);
          }
        }
        fence_proxy_async();   // the widened rows, before the tensor core reads them
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&done[buf]));
          mbar_arrive(smem_u32(&empty[at.slot]));
        }
        at.next();
        ++g;
        if (++buf == bufs) {
          buf = 0;
          buf_par ^= 1;
          buf_used = true;
        }
      }
      return true;
    };
    // O / l of unit u (the CTA's k-th) into its rows.  Lane pairs swap 16-byte
    // pieces, so that two lanes store 32 bytes of one row.
    auto output = [&](const Work& u, int k) -> bool {
#pragma unroll
      for (int X = 0; X < 2; ++X) {
        const int nt = X ? u.nt[1] : u.nt[0];
        if (nt == 0) continue;
        // the buffer and parity of the tile's last step: nt steps on
        last_par[X] ^= ((last_buf[X] + nt) >> 1) & 1;
        last_buf[X] = (last_buf[X] + nt) & 1;
        if (!wait(&l_full[X], units[X] & 1) || !wait(&o_done[2 * X + last_buf[X]], last_par[X])) return false;
        tc_fence_after();
        const int r = 32 * hw + lane;   // TMEM lane, row of the tile
        const bool bad = *reinterpret_cast<volatile int*>(&s_work[k & 1].bad) != 0;
        const float inv = s_inv[X][r];
        // rows of the pair of lanes: r & ~1 and the next
        typename Q::raw* dst[2];
        bool in[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = kRows * X + (r & ~1) + e;
          in[e] = rr < u.in_pair;
          int pos, j;
          u.place(min(rr, u.in_pair - 1), G, inv_g, &pos, &j);
          dst[e] = static_cast<typename Q::raw*>(a.out) + u.at(pos, j, a, D) + 8 * (lane & 1);
        }
        const uint32_t tO = tmem + 256 * X + 128 + (static_cast<uint32_t>(32 * hw) << 16);
#pragma unroll 1
        for (int e0 = 0; e0 < D; e0 += 32) {
          float o[32];
          tmem_ld32(tO + e0, o);
          if (e0 + 32 == D) {   // O is in registers: the next unit's first P V may replace it
            tc_fence_before();
            mbar_arrive(smem_u32(&o_free[X]));
          }
          uint32_t ow[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            ow[e] = pack2<kOutBf>(bad ? CUDART_NAN_F : o[2 * e] * inv, bad ? CUDART_NAN_F : o[2 * e + 1] * inv);
#pragma unroll
          for (int p = 0; p < 2; ++p) {   // pieces 2 p and 2 p + 1 of these 32 columns
            uint32_t even[4], odd[4];     // what goes to the pair's first and second row
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t mine0 = ow[8 * p + e], mine1 = ow[8 * p + 4 + e];
              const uint32_t got = __shfl_xor_sync(FULL, (lane & 1) ? mine0 : mine1, 1);
              even[e] = (lane & 1) ? got : mine0;
              odd[e] = (lane & 1) ? mine1 : got;
            }
            if (in[0]) *reinterpret_cast<uint4*>(dst[0] + e0 + 16 * p) = make_uint4(even[0], even[1], even[2], even[3]);
            if (in[1]) *reinterpret_cast<uint4*>(dst[1] + e0 + 16 * p) = make_uint4(odd[0], odd[1], odd[2], odd[3]);
          }
        }
        if (r == 0 && bad && a.status != nullptr) atomicOr(a.status, s_work[k & 1].bad);
        ++units[X];
      }
      if (ht == 0) s_finished = k + 1;
      return true;
    };
    Work u, v;   // the unit at hand and the next
    bool more = next_work(0, u), ok = true;
    if (more) ok = queries(u) && (!kFp8 || widen(u, 0, min(2, u.steps)));
    for (int k = 0; more && ok; ++k) {
      if (kFp8) ok = widen(u, min(2, u.steps), u.steps);
      if (!ok) break;
      more = next_work(k + 1, v);
      if (more) ok = queries(v) && (!kFp8 || widen(v, 0, min(2, v.steps)));
      if (ok) ok = output(u, k);
      release_work(k);
      u = v;
    }
    if (!ok) {
      cp_async_wait();
      give_up();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    // every branch around a warp-wide TMEM access is taken by the whole warp
    const int X = warp >> 2, r = tid & 127, rp = tid;   // tile, TMEM lane, row of the pair
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tX = tmem + 256 * X + lane_off, tO = tX + 128;
    RingPos<2> sp;             // S / P buffer
    RingPos<kWideV> av;        // widened V buffer
    int g = 0, units = 0;      // stream steps and this tile's units so far
    bool ok = true;
    Work u;
    for (int k = 0; ok && next_work(k, u); ++k) {
      release_work(k);
      const int ntx = X ? u.nt[1] : u.nt[0];
      const HeadScales hs = head_scales(a.head_scales, a.num_kv_heads, u.kvh, a.softmax_scale, a.qk_scale,
                                        a.v_scale, 1.f, 1.f);
      int pos, head;
      u.place(min(rp, u.in_pair - 1), G, inv_g, &pos, &head);
      const int w0 = a.window > 0 ? pos - a.window + 1 : 0;
      // steps [whole0, whole1) lie in one run of keys the row sees entirely
      const int whole0 = (u.keys.ns + max(max(w0 + kChunkKeys - 1, 0) / kChunkKeys - u.keys.wb, 0) + kStepChunks - 1) / kStepChunks;
      const int whole1 = ((pos + 1) / kChunkKeys - u.keys.wb + u.keys.ns) / kStepChunks;
      float m_ref = -CUDART_INF_F, l = 0.f;
      for (int t = 0; t < ntx; ++t) {
        const int b = sp.slot, i = 2 * X + b;
        if (!wait(&s_full[i], sp.par)) {
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
        float qe = hs.qk, lv = 0.f, inv_v = 1.f;
        // V widened (before this step's P V, which follows P); it also orders
        // the producer's scales before their read
        if (kFp8 && !wait(&v_full[av.slot], av.par)) {
          ok = false;
          break;
        }
        if constexpr (BS) {
          const float2 ref = *reinterpret_cast<const float2*>(s_ref[(g + t) % kScaleRing]);
          qe *= ref.x;
          const uint32_t vb = __float_as_uint(ref.y);   // a power of two
          lv = static_cast<float>(static_cast<int>(vb >> 23) - 127);
          inv_v = __uint_as_float((254u << 23) - vb);
        }
        // elsewhere, a bit per key of a chunk
        if (t < whole0 || t >= whole1) {
          auto below = [](int x) { return (1u << min(max(x, 0), kChunkKeys)) - 1u; };   // the first x keys
#pragma unroll
          for (int ch = 0; ch < kStepChunks; ++ch) {
            const int pc = u.keys.chunk(kStepChunks * t + ch) * kChunkKeys;
            const uint32_t seen = below(pos - pc + 1) & (~below(w0 - pc) | below(u.keys.sinks - pc));
#pragma unroll
            for (int e = 0; e < kChunkKeys; ++e)
              if (!(seen & (1u << e))) sv[16 * ch + e] = -CUDART_INF_F;
          }
        }
        if (!(qe > 0.f)) {   // the maximum below is taken on the raw products
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (sv[e] != -CUDART_INF_F) sv[e] *= qe;
          qe = 1.f;
        }
        float mx4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx4[j] = sv[j];
#pragma unroll
        for (int e = 4; e < 60; e += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) mx4[j] = max3(mx4[j], sv[e + j], sv[e + 4 + j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mx4[j] = max3(mx4[j], sv[60 + j], sv[60 + j]);
        const float mx = fmaf(qe, max3(max3(mx4[0], mx4[1], mx4[2]), mx4[3], mx4[3]), lv);
        const bool move = mx > m_ref + kRescaleLog2;
        const bool scale = move && t > 0 && m_ref != -CUDART_INF_F;   // O holds earlier steps
        if (__any_sync(FULL, scale)) {
          if (!wait(&o_done[2 * X + (b ^ 1)], sp.par ^ (b ^ 1))) {   // the step before
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
        const float2 qe2 = make_float2(qe, qe), off2 = make_float2(off, off);
        float2 sum2[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sum2[j] = make_float2(0.f, 0.f);
        uint32_t pw[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float2 x = fma2(make_float2(sv[2 * e], sv[2 * e + 1]), qe2, off2);
          x.x = ex2(x.x);
          x.y = ex2(x.y);
          sum2[e & 3] = add2(sum2[e & 3], x);
          pw[e] = pack2<kBf>(x.x, x.y);
        }
        tmem_st32u(tX + 64 * b, pw);
        const float2 sum = add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3]));
        l = fmaf(sum.x + sum.y, inv_v, l);
        tc_fence_before();
        mbar_arrive(smem_u32(&p_full[i]));
        sp.next();
        if (kFp8) av.next();
      }
      if (kFp8)
        for (int t = ntx; t < u.steps; ++t) av.next();   // the stream's steps of the other tile
      if (ok && ntx > 0) {
        // the row's factor for the helpers, who are done with the unit before
        ok = units == 0 || wait(&o_free[X], (units - 1) & 1);
        if (ok) {
          s_inv[X][r] = (l > 0.f || l != l) ? hs.v / l : 0.f;
          mbar_arrive(smem_u32(&l_full[X]));
        }
        ++units;
      }
      g += u.steps;
    }
    if (!ok) give_up();
  }

  // every MMA done and every copy landed before TMEM and shared memory go
  __syncthreads();
  if (tid == 0) {
    mbar_wait(smem_u32(&fin), 0, kDrainNs);
    if (s_timeout) {
      const int issued = s_issued;
      for (int t = max(0, issued - kRing); t < issued; ++t)
        mbar_wait(smem_u32(&full[t % kRing]), (t / kRing) & 1, kDrainNs);
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
      for (int i = tid; i < w.in_pair * D; i += kThreadsW) {
        const int r = w.row0 + i / D;
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
  static_assert(S_::kSmem <= 227 * 1024 - 2000, "ring, queries and the static part fit one SM");
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
  if (rows > INT32_MAX || units > INT32_MAX || a.group > 1024)
    return fail(PKV_ERR_UNSUPPORTED, "windowed prefill: too many query rows in one call, or query heads per KV head");
  a.max_q_tiles = max_query_len;   // the longest chunk the caller allows
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units));
  cfg.blockDim = dim3(kThreadsW);
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
