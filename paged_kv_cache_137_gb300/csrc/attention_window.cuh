// Decode attention over what a sliding window and a few first tokens (sinks)
// leave visible, and over E4M3 caches with a scale per (block, KV head).
//
// For the G query heads of one KV head of a sequence of ctx positions,
//   o = sum_{p visible} w_p V[p],  w = softmax(q . K[p] * scale),
// p visible iff p < ctx and (p >= ctx - window or p < sinks); a window of 0
// sees everything.  With block scales, K[p] and V[p] are the stored values
// times the scales of p's block.
//
// The visible positions are walked in chunks of 16, the tokens of one
// m16n8k16 MMA: the sinks' chunks, then the window's.  Only their blocks are
// looked up and read, so table entries of blocks nobody sees may be stale.  A
// (sequence, KV head)'s chunks are shared out evenly over its splits, a
// split's over the four warps of its CTA.  A warp streams its chunks through a
// ring of its own: one lane each asks TMA for the 16 rows of K and of V (the
// 128-byte swizzle keeps ldmatrix free of conflicts), completion by expect-tx
// mbarriers, no barrier between warps until the merge.  Block ids (and
// scales) of 32 chunks are fetched a lane each, 32 chunks ahead.  The products
// take the head-columns form: S^T = K q^T and O^T += V^T P^T with the tokens,
// then head_dim, as the MMA's 16 rows and 8 query heads as its columns; groups
// of 9 to 16 heads keep two column sets per K and V fragment.
//
// A chunk lies in one block, so its two scales are scalars.  The K scale joins
// the logit scale.  The V scale vs joins the exponent of P: with m the running
// maximum of s + log2(vs), P = 2^(s + log2(vs) - m) <= 1 keeps all the bits of
// its 16-bit form however far the blocks' scales lie apart, and the row sum
// takes P / vs, so that O and l keep one reference.
//
// Sums, maxima and O are fp32; q and P are rounded to the MMA's 16-bit type
// (the cache's, f16 for E4M3), off by a relative 2^-8 (bf16) or 2^-11 (f16) at
// most.
//
// Measured (GB300; a plain copy reaches 6,779 GB/s), visible K/V bytes:
//   8 contexts of 16,384 to 32,768, 32 / 32 heads, window 4,096, f16:  81 us, 6,670 GB/s
//   512 block-scaled contexts of 64 to 8,192, 64 / 8 heads:           293 us, 5,850 GB/s
//   64 contexts of 256 to 4,096, 28 / 4 heads, window 1,024, bf16:     26 us, 4,810 GB/s
//   4 block-scaled contexts of up to 128, 32 / 8 heads:               4.3 us
// DRAM counters agree with the visible bytes within 3%.  Short calls are
// latency: a chunk is about 0.85 us of one warp (copy, two MMA chains, softmax
// between), whatever the depth of its ring, and a launch with a unit's first
// lookups about 3 us.
#pragma once

#include <atomic>
#include <type_traits>

#include "attention_tc_launch.cuh"
#include "attention_window.h"

namespace pkv {
namespace tc {

constexpr int kChunk = 16;   // tokens of a chunk: the MMA's rows

// A chunk of K or V in shared memory: its rows in lines of 128 bytes, swizzled
// by TMA.  A line is half a 256-byte row, a row, or two rows of 64 bytes (the
// pool seen as rows of 128): ldmatrix meets eight different bank groups each way.
template <typename KV, int D>
struct ChunkGeom {
  static constexpr int kRowBytes = D * KV::bytes;
  static constexpr int kPieces = kRowBytes / 16;   // 16-byte pieces of a row
  static constexpr int kLineRows = kRowBytes < 128 ? 128 / kRowBytes : 1;
  static constexpr int kTileBytes = kChunk * kRowBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;   // K and V
  static_assert(kTileBytes % 1024 == 0, "the swizzle repeats every 1024 bytes");
  // piece c of row r
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    if constexpr (kLineRows == 1) return swz<kRowBytes / 128>(r, c);
    else return swz<1>(r / kLineRows, r % kLineRows * kPieces + c);
  }
  // the box of the chunk that starts at pool row `row`
  __device__ static __forceinline__ void fetch(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
    if constexpr (kRowBytes <= 128) tma_load_2d(dst, map, 0, row / kLineRows, bar);
    else tma_load_3d(dst, map, 0, 0, row, bar);
  }
};

// The visible positions of a query at position ctx - 1, as chunks.
struct Span {
  int ctx, w0, s0;   // positions [0, s0) and [w0, ctx)
  int ns, wb, n;     // the first ns chunks, then those from wb on: n in all
  __device__ __forceinline__ Span(int c, int window, int sinks) {
    ctx = c;
    w0 = window > 0 ? max(c - window, 0) : 0;
    s0 = min(sinks, w0);
    ns = (s0 + kChunk - 1) / kChunk;
    wb = max(w0 / kChunk, ns);
    n = ns + max((c + kChunk - 1) / kChunk - wb, 0);
  }
  __device__ __forceinline__ int chunk(int i) const { return i < ns ? i : i - ns + wb; }
  __device__ __forceinline__ bool sees(int p) const { return p < ctx && (p >= w0 || p < s0); }
  // every position of the 16 from p on
  __device__ __forceinline__ bool sees_all(int p) const {
    return p + kChunk <= ctx && (p >= w0 || p + kChunk <= s0);
  }
};

// A warp's running softmax state of 8 * NH heads (lane (g, q4): heads
// 8 nh + 2 q4 + j, O^T rows g and g + 8 of each 16-row tile).
template <int D, int NH>
struct WindowState {
  float o[NH][D / 16][4];
  float m[NH][2], l[NH][2];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n) o[h][n][0] = o[h][n][1] = o[h][n][2] = o[h][n][3] = 0.f;
      m[h][0] = m[h][1] = -CUDART_INF_F;
      l[h][0] = l[h][1] = 0.f;
    }
  }
};

// 2^x by the hardware approximation (relative error about 2^-22, 0 at -inf).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A block scale within the range it is promised in.
__device__ __forceinline__ float block_scale(float x) {
  return fminf(fmaxf(x, 9.094947017729282e-13f), 1099511627776.f);   // 2^-40, 2^40
}
__device__ __forceinline__ float finite_or_0(float m) { return m == -CUDART_INF_F ? 0.f : m; }

// One chunk folded into the state; kt, vt: its 16 rows of K and V, pos: the
// position of row 0, qk: logit scale (log2 domain), vs: the block's V scale
// (BS).
// Returns true if V rows were zeroed (generic writes the caller fences before
// TMA refills the stage).
template <typename KV, int D, int NH, bool BS>
__device__ __forceinline__ bool chunk_step(WindowState<D, NH>& st,
                                           const uint32_t (&qb)[NH][D / 16][2], const uint8_t* kt,
                                           uint8_t* vt, const Span& span, int pos, float qk, float vs,
                                           int lane) {
  using G_ = ChunkGeom<KV, D>;
  constexpr bool kFp8 = std::is_same<KV, E4M3>::value;
  constexpr bool kBf = std::is_same<KV, BF16>::value;
  constexpr int KS = D / 16, P = G_::kPieces;
  constexpr unsigned FULL = 0xffffffffu;
  const int g = lane >> 2;
  bool zeroed = false;
  const bool whole = span.sees_all(pos);
  if (!whole) {   // a weight of 0 times what an unseen row holds must be 0
    for (int i = lane; i < kChunk * P; i += 32) {
      const int r = i / P;
      if (!span.sees(pos + r))
        *reinterpret_cast<uint4*>(vt + G_::at(r, i % P)) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    zeroed = true;
  }
  const uint32_t kbase = smem_u32(kt), vbase = smem_u32(vt);
  const int li = lane & 7, mi = lane >> 3;
  const int rk = (mi & 1) * 8 + li;

  // S^T = K q^T
  // (in two chains of half the length: one warp's MMAs are latency)
  float sc[NH][4], sd[NH][4];
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[h][e] = sd[h][e] = 0.f;
  if constexpr (!kFp8) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a0, a1, a2, a3;
      ldsm_x4(kbase + G_::at(rk, 2 * ks + (mi >> 1)), a0, a1, a2, a3);
#pragma unroll
      for (int h = 0; h < NH; ++h)
        mma16816<kBf>(ks & 1 ? sd[h] : sc[h], a0, a1, a2, a3, qb[h][ks][0], qb[h][ks][1]);
    }
  } else {
#pragma unroll
    for (int ks = 0; ks < KS; ks += 2) {   // one load serves two k-steps
      uint32_t w[4];
      ldsm_x4(kbase + G_::at(rk, ks + (mi >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t a0 = e4m3x2_f16x2(w[2 * k] & 0xffffu), a1 = e4m3x2_f16x2(w[2 * k + 1] & 0xffffu);
        const uint32_t a2 = e4m3x2_f16x2(w[2 * k] >> 16), a3 = e4m3x2_f16x2(w[2 * k + 1] >> 16);
#pragma unroll
        for (int h = 0; h < NH; ++h)
          mma16816<false>(k ? sd[h] : sc[h], a0, a1, a2, a3, qb[h][ks + k][0], qb[h][ks + k][1]);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[h][e] += sd[h][e];

  // online softmax over the tokens (rows g, g + 8) of heads 2 q4 + j
  const bool see0 = whole || span.sees(pos + g), see1 = whole || span.sees(pos + g + 8);
  const float lv = BS ? __log2f(vs) : 0.f, inv_v = BS ? __frcp_rn(vs) : 1.f;
  uint32_t pb[NH][2];
  float corr[NH][2];
  bool moved = false;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    float p[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float v0 = see0 ? fmaf(sc[h][j], qk, lv) : -CUDART_INF_F;
      const float v1 = see1 ? fmaf(sc[h][2 + j], qk, lv) : -CUDART_INF_F;
      float mx = fmaxf(v0, v1);
      mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
      const float mn = fmaxf(st.m[h][j], mx);
      const float ref = finite_or_0(mn);   // every logit so far -inf: all weights 0
      corr[h][j] = ex2_approx(st.m[h][j] - ref);
      p[j] = ex2_approx(v0 - ref);
      p[2 + j] = ex2_approx(v1 - ref);
      st.m[h][j] = mn;
      st.l[h][j] = st.l[h][j] * corr[h][j] + (p[j] + p[2 + j]) * inv_v;
      moved = moved || corr[h][j] != 1.f;
    }
    // P^T as the B operand: the transposes of its two 8 x 8 blocks
    pb[h][0] = movmatrix_t(pack2<kBf>(p[0], p[1]));
    pb[h][1] = movmatrix_t(pack2<kBf>(p[2], p[3]));
  }
  // where no maximum of the warp's heads grew, every factor is exactly 1
  if (__any_sync(FULL, moved)) {
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        st.o[h][mt][0] *= corr[h][0];
        st.o[h][mt][1] *= corr[h][1];
        st.o[h][mt][2] *= corr[h][0];
        st.o[h][mt][3] *= corr[h][1];
      }
  }

  // O^T += V^T P^T
  if constexpr (!kFp8) {
    const int rv = (mi >> 1) * 8 + li;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      uint32_t a0, a1, a2, a3;
      ldsm_x4_t(vbase + G_::at(rv, 2 * mt + (mi & 1)), a0, a1, a2, a3);
#pragma unroll
      for (int h = 0; h < NH; ++h) mma16816<kBf>(st.o[h][mt], a0, a1, a2, a3, pb[h][0], pb[h][1]);
    }
  } else {
    // a register holds tokens 2 q4, 2 q4 + 1 of head_dim pair (2 g, 2 g + 1)
#pragma unroll
    for (int mt = 0; mt < D / 16; mt += 2) {
      uint32_t w[4];   // (tokens 0-7, mt), (8-15, mt), (0-7, mt + 1), (8-15, mt + 1)
      ldsm_x4_t(vbase + G_::at(rk, mt + (mi >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x0 = prmt(w[2 * k], 0x3120), x1 = prmt(w[2 * k + 1], 0x3120);
        const uint32_t a0 = e4m3x2_f16x2(x0 & 0xffffu), a1 = e4m3x2_f16x2(x0 >> 16);
        const uint32_t a2 = e4m3x2_f16x2(x1 & 0xffffu), a3 = e4m3x2_f16x2(x1 >> 16);
#pragma unroll
        for (int h = 0; h < NH; ++h) mma16816<false>(st.o[h][mt + k], a0, a1, a2, a3, pb[h][0], pb[h][1]);
      }
    }
  }
  return zeroed;
}

// The state to the merge buffers mS, lS [warp][16], oS [warp][16][D] (heads <
// G).
template <typename KV, int D, int NH>
__device__ __forceinline__ void publish_window(const WindowState<D, NH>& st, float* mS, float* lS,
                                               float* oS, int warp, int G, int lane) {
  constexpr bool kFp8 = std::is_same<KV, E4M3>::value;
  const int g = lane >> 2, q4 = lane & 3;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float l = st.l[h][j];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (g == 0) {   // a NaN sum keeps a finite maximum, so that the merge does not skip it
        mS[warp * 16 + 8 * h + 2 * q4 + j] = l == l ? st.m[h][j] : 0.f;
        lS[warp * 16 + 8 * h + 2 * q4 + j] = l;
      }
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int head = 8 * h + 2 * q4 + (e & 1);
        if (head < G) oS[(warp * 16 + head) * D + out_row_t<kFp8>(mt, g, e >> 1)] = st.o[h][mt][e];
      }
  }
}

// Write the CTA's combined state (its W warps' in mS, lS, oS): the output
// of a lone split, else the split's partial; the last split of the pair to
// arrive (an atomic count, never a wait) merges them all in split order.
// stage: `cap` floats of shared memory the merge may use.
template <typename Q, int D, int W>
__device__ __forceinline__ void finish_unit(const WindowArgs& a, const float* mS, const float* lS,
                                            const float* oS, int kvh, int seq, int split, int nsplit,
                                            int bad_bits, float v_scale, float* stage, int cap,
                                            int* s_last) {
  const int tid = threadIdx.x, G = a.group;
  const size_t head0 = static_cast<size_t>(seq) * a.num_q_heads + static_cast<size_t>(kvh) * G;
  if (tid == 0 && bad_bits != 0 && a.status != nullptr) atomicOr(a.status, bad_bits);
  for (int i = tid; i < G * D; i += 32 * W) {
    const int row = i / D, d = i % D;
    float M, L, A;
    combine_warps(mS, lS, oS, W, 16, row, d, D, M, L, A);
    A *= v_scale;
    if (nsplit == 1) {
      const float o = bad_bits ? CUDART_NAN_F : (L > 0.f || L != L) ? A / L : 0.f;
      store_elem<Q>(a.out, (head0 + row) * D + d, o);
    } else {
      const size_t pidx = (head0 + row) * a.max_splits + split;
      a.ws_acc[pidx * D + d] = bad_bits ? CUDART_NAN_F : A;
      if (d == 0) {
        a.ws_m[pidx] = M;
        a.ws_l[pidx] = bad_bits ? CUDART_NAN_F : L;
      }
    }
  }
  if (nsplit == 1) return;
  int* counter = &a.counters[static_cast<size_t>(seq) * a.num_kv_heads + kvh];
  __threadfence();
  __syncthreads();
  if (tid == 0) *s_last = atomicAdd(counter, 1) == nsplit - 1;
  __syncthreads();
  if (!*s_last) return;
  __threadfence();
  merge_splits<Q, D, 32 * W>(a, head0, nsplit, a.max_splits, 0, stage, cap);
  if (tid == 0) atomicExch(counter, 0);
}

// Warps per CTA by the CTAs of the call that share an SM: a chunk is about a
// microsecond of one warp's latency, so an SM wants its 12 (rows of 256 bytes:
// rings of 16 KiB a warp) or 16 warps (12 KiB) whether its work is one unit or
// several.  The rings take 192 KiB of an SM either way.
template <typename KV, int D, int NH>
constexpr int window_warps(int c) {
  // (two column sets of heads leave registers for 12 warps as well)
  constexpr bool wide = NH > 1 || ChunkGeom<KV, D>::kStageBytes >= 8192;
  return c <= 1 ? (wide ? 12 : 16) : c == 2 ? (wide ? 6 : 8) : kWarps;
}
template <typename KV, int D>
constexpr int window_stages() { return ChunkGeom<KV, D>::kStageBytes >= 8192 ? 2 : 3; }
template <typename KV, int D, int NH, int W>
constexpr int window_ctas() {
  constexpr int warps = NH == 1 && ChunkGeom<KV, D>::kStageBytes < 8192 ? 16 : 12;
  return warps / W < 1 ? 1 : warps / W;
}

template <typename KV, typename Q, int D, int NH, bool BS, int W>
__global__ void __launch_bounds__(32 * W, window_ctas<KV, D, NH, W>())
    decode_window_kernel(const WindowArgs a, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  using G_ = ChunkGeom<KV, D>;   // one warp's stage: 16 tokens of K, then of V
  constexpr int NS = window_stages<KV, D>();
  constexpr int KS = D / 16;
  constexpr unsigned FULL = 0xffffffffu;
  const int kvh = blockIdx.x, seq = blockIdx.y, split = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q4 = lane & 3;
  if (warp == 0 && lane < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &vmap : &kmap))
                 : "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int G = a.group, T = a.block_size;
  const int ctx = a.ctx_lens[seq];
  uint32_t qb[NH][KS][2];
  const typename Q::raw* qrows = static_cast<const typename Q::raw*>(a.q) +
      (static_cast<size_t>(seq) * a.num_q_heads + static_cast<size_t>(kvh) * G) * D;
#pragma unroll
  for (int h = 0; h < NH; ++h) load_qt<KV, Q, D>(qb[h], qrows + 8 * h * D, G - 8 * h, g, q4);
  const HeadScales hs = head_scales(a.head_scales, a.num_kv_heads, kvh, a.softmax_scale, a.qk_scale,
                                    a.v_scale, 1.f, 1.f);
  const bool bad_ctx = ctx < 0 || ctx > a.max_blocks * T;
  const Span span(bad_ctx ? 0 : ctx, a.window, a.sinks);
  const int nsplit = max(1, (span.n + a.part_chunks - 1) / a.part_chunks);
  if (split >= nsplit) return;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t s_bar[W][NS];
  __shared__ int s_bad[W], s_last;
  uint8_t* ring = smem + warp * NS * G_::kStageBytes;
  uint64_t* bar = s_bar[warp];
  if (lane < NS) mbar_init(smem_u32(&bar[lane]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  fence_proxy_async();
  __syncwarp();

  // the split's chunks [c0, c1), the warp's [wa, wa + n) of them
  const int64_t n_all = span.n;
  const int c0 = static_cast<int>(split * n_all / nsplit);
  const int c1 = static_cast<int>((split + 1) * n_all / nsplit);
  const int wa = c0 + warp * (c1 - c0) / W;
  const int n = c0 + (warp + 1) * (c1 - c0) / W - wa;
  const int32_t* trow = a.tables + static_cast<size_t>(seq) * a.max_blocks;
  int bad = bad_ctx ? kBadLength : 0;
  // lane l of batch b: the pool row (-1: a bad table entry) and the scales of
  // the warp's chunk 32 b + l
  auto fetch = [&](int b, int& row, float2& scales) {
    row = -1;
    const int i = 32 * b + lane;
    if (i >= n) return;
    const int p = span.chunk(wa + i) * kChunk;
    const int blk = trow[p / T];
    if (blk < 0 || blk >= a.num_blocks) {
      bad |= kBadTable;
      return;
    }
    const int slab = blk * a.num_kv_heads + kvh;
    row = slab * T + p % T;
    if constexpr (BS) {
      const float2 x = *reinterpret_cast<const float2*>(a.block_scales + 2 * static_cast<size_t>(slab));
      scales = make_float2(block_scale(x.x), block_scale(x.y));
    }
  };
  int row_cur = -1, row_nxt = -1;
  float2 sc_cur = make_float2(0.f, 0.f), sc_nxt = sc_cur;
  fetch(0, row_cur, sc_cur);
  auto issue = [&](int i, int base, int slot) {   // base: the first chunk of the current batch
    const int row = __shfl_sync(FULL, i - base < 32 ? row_cur : row_nxt, i & 31);
    const uint32_t b = smem_u32(&bar[slot]);
    if (lane == 0) mbar_arrive_expect_tx(b, row >= 0 ? G_::kStageBytes : 0);
    __syncwarp();
    if (lane < 2 && row >= 0)
      G_::fetch(smem_u32(ring + slot * G_::kStageBytes + lane * G_::kTileBytes), lane ? &vmap : &kmap, row, b);
  };
  for (int i = 0; i < NS && i < n; ++i) issue(i, 0, i);
  fetch(1, row_nxt, sc_nxt);

  WindowState<D, NH> st;
  st.reset();
  int s = 0;
  uint32_t par = 0;
  for (int i = 0; i < n; ++i) {
    if ((i & 31) == 0 && i > 0) {
      row_cur = row_nxt;
      sc_cur = sc_nxt;
      fetch(i / 32 + 1, row_nxt, sc_nxt);
    }
    if (!__all_sync(FULL, stage_wait(smem_u32(&bar[s]), par, a.wait_ns))) {
      // wait (bounded) for the copies still in flight before the ring is reused
      bad |= kTimeout;
      if (lane == 0)
        for (int t = i; t < n && t < i + NS; ++t) mbar_wait(smem_u32(&bar[t % NS]), (t / NS) & 1, kDrainNs);
      break;
    }
    const int row = __shfl_sync(FULL, row_cur, i & 31);
    float ks = 1.f, vs = 1.f;
    if constexpr (BS) {
      ks = __shfl_sync(FULL, sc_cur.x, i & 31);
      vs = __shfl_sync(FULL, sc_cur.y, i & 31);
    }
    if (row >= 0) {
      uint8_t* kt = ring + s * G_::kStageBytes;
      if (chunk_step<KV, D, NH, BS>(st, qb, kt, kt + G_::kTileBytes, span, span.chunk(wa + i) * kChunk,
                                    hs.qk * ks, vs, lane))
        fence_proxy_async();   // the zeroed rows, before TMA refills the stage
    }
    __syncwarp();
    if (i + NS < n) issue(i + NS, i & ~31, s);
    if (++s == NS) {
      s = 0;
      par ^= 1;
    }
  }

  bad = __reduce_or_sync(FULL, bad);
  if (lane == 0) s_bad[warp] = bad;
  __syncthreads();   // every ring is idle: the merge takes its place
  float* mS = reinterpret_cast<float*>(smem);
  float* lS = mS + W * 16;
  float* oS = lS + W * 16;
  constexpr int kCap = W * NS * G_::kStageBytes / 4;
  static_assert(kCap >= 2 * W * 16 + W * 16 * D, "the warp merge reuses the rings");
  publish_window<KV, D, NH>(st, mS, lS, oS, warp, G, lane);
  __syncthreads();
  int bad_bits = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) bad_bits |= s_bad[w];
  finish_unit<Q, D, W>(a, mS, lS, oS, kvh, seq, split, nsplit, bad_bits, hs.v,
                       reinterpret_cast<float*>(smem), kCap, &s_last);
}

template <typename KV, typename Q, int D, int NH, bool BS, int W>
pkv_status launch_window_form(const WindowArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              cudaStream_t st) {
  constexpr int smem = W * window_stages<KV, D>() * ChunkGeom<KV, D>::kStageBytes + 1024;
  auto kernel = decode_window_kernel<KV, Q, D, NH, BS, W>;
  static std::atomic<uint64_t> configured{0};   // the shared-memory opt-in is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail("windowed decode: cudaGetDevice", e);
  const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
  if (!bit || !(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return cuda_fail("windowed decode: cudaFuncSetAttribute", e);
    configured.fetch_or(bit);
  }
  const dim3 grid(a.num_kv_heads, a.num_seqs, a.max_splits);
  e = launch_dependent(kernel, grid, 32 * W, smem, st, a, kmap, vmap);
  if (e != cudaSuccess) return cuda_fail("windowed decode: launch", e);
  return check_launch("windowed decode (tensor core)");
}

template <typename KV, typename Q, int D, int NH, bool BS>
pkv_status launch_window_w(const WindowArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                           cudaStream_t st) {
  if (a.ctas_per_sm <= 1)
    return launch_window_form<KV, Q, D, NH, BS, window_warps<KV, D, NH>(1)>(a, kmap, vmap, st);
  if (a.ctas_per_sm == 2)
    return launch_window_form<KV, Q, D, NH, BS, window_warps<KV, D, NH>(2)>(a, kmap, vmap, st);
  return launch_window_form<KV, Q, D, NH, BS, kWarps>(a, kmap, vmap, st);
}

template <typename KV, typename Q, int D>
pkv_status launch_window_d(const WindowArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                           cudaStream_t st) {
  if constexpr (std::is_same<KV, E4M3>::value) {
    if (a.block_scales)
      return a.group <= 8 ? launch_window_w<KV, Q, D, 1, true>(a, kmap, vmap, st)
                          : launch_window_w<KV, Q, D, 2, true>(a, kmap, vmap, st);
  }
  return a.group <= 8 ? launch_window_w<KV, Q, D, 1, false>(a, kmap, vmap, st)
                      : launch_window_w<KV, Q, D, 2, false>(a, kmap, vmap, st);
}

}  // namespace tc

template <typename KV, typename Q>
pkv_status launch_window_tc(const WindowArgs& a, int head_dim, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, cudaStream_t st) {
  if (head_dim == 128) return tc::launch_window_d<KV, Q, 128>(a, kmap, vmap, st);
  if (head_dim == 64) return tc::launch_window_d<KV, Q, 64>(a, kmap, vmap, st);
  return fail(PKV_ERR_UNSUPPORTED, "windowed decode: head_dim not compiled for the tensor-core kernel");
}

}  // namespace pkv
