// CUDA-core form of windowed and block-scaled decode attention: fp32 caches,
// and any other when the CUDA-core kernels are asked for.  The same chunks,
// splits and merge as attention_window.cuh; the W warps of a CTA take the
// chunks of its split in turn, two lanes share a token in the q.k phase
// (head_dim / 2 elements each) and the lanes split head_dim for p.V.  All G
// heads (padded to GM) go together, so a K/V element is read once per CTA.  The
// block's V scale multiplies p in fp32.  Everything is fp32.
//
// Bound by a warp's latency per chunk (copies, then GM sums over 16 lanes), so a
// chunk's K and V and the next one's block id are in flight together.  Measured
// (GB300): 4 contexts of up to 128, window 33, 4 / 4 heads, fp32: 3.7 us; 295
// contexts of 136 to 409, 7 / 1 heads: 24.5 us; 16 of 611, 56 / 8 heads: 19.6 us.
#pragma once

#include "attention_window.cuh"

namespace pkv {

template <typename KV, typename Q, int D, int GM, int W>
__global__ void __launch_bounds__(32 * W) decode_window_simt_kernel(const WindowArgs a) {
  using namespace tc;
  constexpr int DQ = D / 2, DV = D / 32;
  constexpr int KB = 32;        // K elements a lane has in flight
  constexpr int VB = 32 / DV;   // V rows (of DV elements a lane) in flight
  constexpr unsigned FULL = 0xffffffffu;
  using raw = typename KV::raw;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int kvh = blockIdx.x, seq = blockIdx.y, split = blockIdx.z;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = a.group, T = a.block_size;
  const int ctx = a.ctx_lens[seq];
  const bool bad_ctx = ctx < 0 || ctx > a.max_blocks * T;
  const Span span(bad_ctx ? 0 : ctx, a.window, a.sinks);
  const int nsplit = max(1, (span.n + a.part_chunks - 1) / a.part_chunks);
  if (split >= nsplit) return;
  const HeadScales hs = head_scales(a.head_scales, a.num_kv_heads, kvh, a.softmax_scale, a.qk_scale,
                                    a.v_scale, 1.f, 1.f);
  const int64_t n_all = span.n;
  const int c0 = static_cast<int>(split * n_all / nsplit);
  const int c1 = static_cast<int>((split + 1) * n_all / nsplit);

  __shared__ float q_s[GM][D];
  __shared__ float p_s[W][kChunk][GM];
  extern __shared__ __align__(16) float merge_s[];   // [2][W][16], [W][16][D]
  __shared__ int s_bad, s_last;
  if (threadIdx.x == 0) s_bad = bad_ctx ? kBadLength : 0;
  for (int i = threadIdx.x; i < GM * D; i += 32 * W) {
    const int j = i / D, d = i % D;
    q_s[j][d] = j < G ? load_elem<Q>(a.q, (static_cast<size_t>(seq) * a.num_q_heads + kvh * G + j) * D + d) * hs.qk
                      : 0.f;
  }
  __syncthreads();

  float m[GM], lsum[GM], acc[GM][DV];
#pragma unroll
  for (int j = 0; j < GM; ++j) {
    m[j] = -CUDART_INF_F;
    lsum[j] = 0.f;
#pragma unroll
    for (int e = 0; e < DV; ++e) acc[j][e] = 0.f;
  }
  const int tok = lane % kChunk, part = lane / kChunk;
  const int32_t* trow = a.tables + static_cast<size_t>(seq) * a.max_blocks;
  bool bad = false;
  int next = c0 + warp < c1 ? trow[span.chunk(c0 + warp) * kChunk / T] : 0;
  for (int c = c0 + warp; c < c1; c += W) {
    const int pos = span.chunk(c) * kChunk;
    const int blk = next;
    if (c + W < c1) next = trow[span.chunk(c + W) * kChunk / T];
    if (blk < 0 || blk >= a.num_blocks) {   // the same for the whole warp
      bad = true;
      break;
    }
    const size_t slab = static_cast<size_t>(blk) * a.num_kv_heads + kvh;
    const size_t base = (slab * T + pos % T) * D;
    float ks = 1.f, vs = 1.f;
    if (a.block_scales) {
      ks = block_scale(a.block_scales[2 * slab]);
      vs = block_scale(a.block_scales[2 * slab + 1]);
    }
    float s[GM];
#pragma unroll
    for (int j = 0; j < GM; ++j) s[j] = 0.f;
    // a row that nobody sees is never read: its weight is 0, its V counts as 0
    const raw* vp = static_cast<const raw*>(a.v_cache) + base + lane * DV;
    float vf[VB][DV];
    auto fetch_v = [&](int t0) {
#pragma unroll
      for (int t = 0; t < VB; ++t) {
#pragma unroll
        for (int e = 0; e < DV; ++e) vf[t][e] = 0.f;
        if (span.sees(pos + t0 + t)) LoadF32<KV, DV>::run(vp + static_cast<size_t>(t0 + t) * D, vf[t]);
      }
    };
    const raw* kp = static_cast<const raw*>(a.k_cache) + base + static_cast<size_t>(tok) * D + part * DQ;
#pragma unroll 1
    for (int d0 = 0; d0 < DQ; d0 += KB) {
      float kf[KB];
#pragma unroll
      for (int i = 0; i < KB; i += 8) LoadF32<KV, 8>::run(kp + d0 + i, kf + i);
      if (d0 + KB == DQ) fetch_v(0);   // on their way beside the last of K
#pragma unroll
      for (int j = 0; j < GM; ++j)
#pragma unroll
        for (int e = 0; e < KB; ++e) s[j] = fmaf(q_s[j][part * DQ + d0 + e], kf[e], s[j]);
    }
    const bool seen = span.sees(pos + tok);
    float corr[GM];
#pragma unroll
    for (int j = 0; j < GM; ++j) {
      s[j] += __shfl_xor_sync(FULL, s[j], kChunk);
      const float sj = seen ? s[j] * ks : -CUDART_INF_F;
      float bm = sj;
#pragma unroll
      for (int off = 1; off < kChunk; off <<= 1) bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, off));
      const float mn = fmaxf(m[j], bm), ref = finite_or_0(mn);
      const float p = exp2f(sj - ref);
      float ps = p;
#pragma unroll
      for (int off = 1; off < kChunk; off <<= 1) ps += __shfl_xor_sync(FULL, ps, off);
      corr[j] = exp2f(m[j] - ref);
      lsum[j] = lsum[j] * corr[j] + ps;
      m[j] = mn;
      if (part == 0) p_s[warp][tok][j] = p * vs;
    }
#pragma unroll
    for (int j = 0; j < GM; ++j)
#pragma unroll
      for (int e = 0; e < DV; ++e) acc[j][e] *= corr[j];
    __syncwarp();
#pragma unroll
    for (int t0 = 0; t0 < kChunk; t0 += VB) {
      if (t0 > 0) fetch_v(t0);
#pragma unroll
      for (int t = 0; t < VB; ++t)
#pragma unroll
        for (int j = 0; j < GM; ++j) {
          const float pj = p_s[warp][t0 + t][j];
#pragma unroll
          for (int e = 0; e < DV; ++e) acc[j][e] = fmaf(pj, vf[t][e], acc[j][e]);
        }
    }
    __syncwarp();
  }
  if (bad && lane == 0) atomicOr(&s_bad, kBadTable);
  float* mS = merge_s;
  float* lS = mS + W * 16;
  float* oS = lS + W * 16;
#pragma unroll
  for (int j = 0; j < GM; ++j) {
    if (lane == 0) {
      mS[warp * 16 + j] = lsum[j] == lsum[j] ? m[j] : 0.f;   // a NaN sum reaches the merge
      lS[warp * 16 + j] = lsum[j];
    }
#pragma unroll
    for (int e = 0; e < DV; ++e) oS[(warp * 16 + j) * D + lane * DV + e] = acc[j][e];
  }
  __syncthreads();
  finish_unit<Q, D, W>(a, mS, lS, oS, kvh, seq, split, nsplit, s_bad, hs.v, merge_s, W * 16 * (D + 2), &s_last);
}

template <typename KV, typename Q, int D, int GM, int W>
cudaError_t launch_window_simt_w(const WindowArgs& a, cudaStream_t st) {
  constexpr int smem = W * 16 * (D + 2) * 4;
  auto kernel = decode_window_simt_kernel<KV, Q, D, GM, W>;
  if constexpr (smem > 32 * 1024) {   // more than the default with the static part: opted in, per device
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
    if (!bit || !(configured.load() & bit)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      configured.fetch_or(bit);
    }
  }
  return tc::launch_dependent(kernel, dim3(a.num_kv_heads, a.num_seqs, a.max_splits), 32 * W, smem, st, a);
}

// Eight warps where at most two CTAs share an SM: a warp's chunk is latency.
template <typename KV, typename Q, int D, int GM>
cudaError_t launch_window_simt_g(const WindowArgs& a, cudaStream_t st) {
  return a.ctas_per_sm <= 2 ? launch_window_simt_w<KV, Q, D, GM, 8>(a, st) : launch_window_simt_w<KV, Q, D, GM, 4>(a, st);
}

template <typename KV, typename Q, int D>
pkv_status launch_window_simt_d(const WindowArgs& a, cudaStream_t st) {
  cudaError_t e;
  if (a.group <= 1) e = launch_window_simt_g<KV, Q, D, 1>(a, st);
  else if (a.group <= 4) e = launch_window_simt_g<KV, Q, D, 4>(a, st);
  else if (a.group <= 8) e = launch_window_simt_g<KV, Q, D, 8>(a, st);
  else e = launch_window_simt_g<KV, Q, D, 16>(a, st);
  if (e != cudaSuccess) return cuda_fail("windowed decode: launch", e);
  return check_launch("windowed decode (CUDA cores)");
}

template <typename KV, typename Q>
pkv_status launch_window_simt(const WindowArgs& a, int head_dim, cudaStream_t st) {
  if (head_dim == 128) return launch_window_simt_d<KV, Q, 128>(a, st);
  if (head_dim == 64) return launch_window_simt_d<KV, Q, 64>(a, st);
  return fail(PKV_ERR_UNSUPPORTED, "windowed decode: head_dim not compiled");
}

}  // namespace pkv
