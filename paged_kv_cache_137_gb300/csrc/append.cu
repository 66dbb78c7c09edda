// Append with rotation: the new tokens' keys and values through the block
// table, keys and queries rotated by their position on the way.
//
// The chunk of sequence s is its last n_s logical positions, as in prefill
// attention; the foundry page on paged block allocation, "In and out": the
// step writes the new tokens' K/V into reserved slots.  With r = rotary_dim
// and the table row (cos a_i, sin a_i) of the token's position, i < r / 2, the
// pair (x0, x1) of index i becomes
//   (x0 cos a_i - x1 sin a_i,  x0 sin a_i + x1 cos a_i),
// each product and the sum rounded to fp32 (no fused multiply-add, so that
// the value does not depend on how a compiler contracts it), then rounded
// once to the cache's type.
//
// Block-scaled E4M3 caches keep one power-of-two scale per (block, KV head,
// K|V).  E4M3 is a floating format, so a power of two loses no mantissa bit
// and a block whose scale grows is requantised exactly except where a value
// becomes subnormal.  The block's scale after the call is
//   S = max(S_before, 2^e),  e = the least with amax(new) <= 448 * 2^e,
// S_before counting only where the block holds earlier tokens; if S grew, the
// earlier bytes b become e4m3(b * S_before / S).
//
// Both forms are bound by memory traffic (prompts) or by latency (a decode
// step).  A thread owns 16 elements of a row, both halves of its 8 pairs, so
// that a rotation never leaves the thread; 16 (head_dim 128) or 32 tokens and
// a group of rows share a CTA, and a thread keeps its angles in registers
// while it walks the rows of its token.  A (block, KV head, K|V) of a
// block-scaled cache is one warp's (two for blocks of 32; D / 16 lanes where
// there is one new token): the maximum is a reduction over its lanes, and
// nobody else writes that block's bytes or its scale.
//
// Measured (GB300; a plain copy reaches 6,779 GB/s):
//   64 new tokens, 28 query / 4 KV heads, bf16:                 3.7 us (latency: the table entry, then the row)
//   6,400 tokens of chunks, 28 / 4 heads, bf16:                24.4 us, 5,590 GB/s
//   512 new tokens, 64 / 8 heads, into a block-scaled cache:    5.5 us, 3,670 GB/s
//   40,000 tokens of prompts, 64 / 8 heads, block-scaled:       260 us, 5,910 GB/s
// DRAM counters of the last: 0.82 GB read and 0.68 GB written, what it has to.
#include <algorithm>
#include <type_traits>

#include <math_constants.h>

#include "attention.h"
#include "device_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kMinScaleExp = -40, kMaxScaleExp = 40;   // exponents a block scale may take

struct AppendArgs {
  void* cache[2];            // K, V
  const void* src[2];        // K, V [total][n_kv][D], rows src_stride apart
  int64_t src_stride[2];
  const void* q;             // [total][n_q][D], rows q_stride apart, or NULL
  void* q_out;               // [total][n_q][D]
  int64_t q_stride;
  float* block_scales;       // [num_blocks][n_kv][2], or NULL
  float inv_scale[2];
  const float* head_scales;  // [4][n_kv], or NULL
  const int32_t* tables;
  const int32_t* ctx_lens;
  const int32_t* query_start;  // [num_seqs + 1], or NULL: one token each
  const float* angles;       // [max_position][rotary]: cosines, then sines
  int32_t max_position, rotary, interleaved;
  int32_t max_blocks, num_seqs, total, max_len, n_q, n_kv, block_size, num_blocks;
  int32_t rows_per_cta;      // rows (heads) a thread walks
  int32_t row_groups;
  int32_t row_ctas;          // CTAs of the row form in grid.x; the rest take block units
  int32_t block_parts;       // CTAs of one touched block
  int* status;
};

// The chunk of sequence s: rows [row0, row0 + n) of the inputs at positions
// first ..; n = 0 where there is nothing to write.
struct Chunk {
  int32_t row0, n, first;
  bool bad;   // invalid lengths: nothing is written, its q_out rows (n of them) become NaN
};
__device__ __forceinline__ Chunk chunk_of(const AppendArgs& a, int s) {
  Chunk c{s, 1, 0, false};
  const int ctx = a.ctx_lens[s];
  if (a.query_start != nullptr) {
    c.row0 = a.query_start[s];
    const int end = a.query_start[s + 1];
    // rows outside the inputs: nothing this call may touch
    if (c.row0 < 0 || end < c.row0 || end > a.total) return {0, 0, 0, true};
    c.n = end - c.row0;
  } else if (ctx == 0) {
    c.first = -1;   // no token: the q_out row becomes zero
    return c;
  }
  c.bad = ctx < 0 || ctx > a.max_blocks * a.block_size || c.n > ctx || c.n > a.max_len ||
          (a.rotary > 0 && ctx > a.max_position);
  c.first = ctx - c.n;
  return c;
}

// 8 elements as they are stored.
template <typename Tag>
struct Raw8 {
  uint4 w[Tag::bytes / 2];
};
template <typename Tag>
__device__ __forceinline__ Raw8<Tag> load_raw8(const void* base, size_t idx) {
  Raw8<Tag> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const typename Tag::raw*>(base) + idx);
#pragma unroll
  for (int i = 0; i < Tag::bytes / 2; ++i) r.w[i] = p[i];
  return r;
}

// A thread's unit of a row: two groups of 8 elements, at p0 and p1, and how
// they turn.  Neighbouring units hold neighbouring groups, so that a warp's
// 16-byte accesses make whole 128-byte lines.  Half-split pairs join the two
// groups; adjacent pairs lie within a group.
struct UnitPlace {
  int p0, p1;
  bool t0, t1;   // the group is rotated (half-split: both or neither)
};
__device__ __forceinline__ UnitPlace unit_place(int u, int head_dim, int rotary, bool interleaved) {
  UnitPlace w;
  if (interleaved) {
    w.p0 = 8 * u;
    w.p1 = head_dim / 2 + 8 * u;
    w.t0 = w.p0 < rotary;
    w.t1 = w.p1 < rotary;
  } else if (u < rotary / 16) {
    w.p0 = 8 * u;
    w.p1 = rotary / 2 + 8 * u;
    w.t0 = w.t1 = true;
  } else {
    w.p0 = rotary + 8 * (u - rotary / 16);
    w.p1 = w.p0 + (head_dim - rotary) / 2;
    w.t0 = w.t1 = false;
  }
  return w;
}

// The unit's 8 angles at a position: half-split pair i of 8 (elements p0 + i
// and p1 + i), or the four adjacent pairs of each group.
__device__ __forceinline__ const float* angle_row(const AppendArgs& a, int pos) {
  return a.angles + static_cast<size_t>(pos) * a.rotary;
}
__device__ __forceinline__ void load_angles(const AppendArgs& a, const float* row, const UnitPlace& w,
                                            float (&c)[8], float (&s)[8]) {
  const int half = a.rotary / 2;
  if (a.interleaved) {
    if (w.t0) {
      LoadF32<F32, 4>::run(row + w.p0 / 2, c);
      LoadF32<F32, 4>::run(row + half + w.p0 / 2, s);
    }
    if (w.t1) {
      LoadF32<F32, 4>::run(row + w.p1 / 2, c + 4);
      LoadF32<F32, 4>::run(row + half + w.p1 / 2, s + 4);
    }
  } else if (w.t0) {
    LoadF32<F32, 8>::run(row + w.p0, c);
    LoadF32<F32, 8>::run(row + half + w.p0, s);
  }
}

// x and y (the unit's two groups) as fp32, rotated.
__device__ __forceinline__ void rotate(float (&x)[8], float (&y)[8], const float (&c)[8],
                                       const float (&s)[8], bool interleaved, const UnitPlace& w) {
  auto turn = [](float& p, float& q, float cs, float sn) {
    const float a = __fsub_rn(__fmul_rn(p, cs), __fmul_rn(q, sn));
    const float b = __fadd_rn(__fmul_rn(p, sn), __fmul_rn(q, cs));
    p = a;
    q = b;
  };
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (w.t0) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
      if (w.t1) turn(y[2 * i], y[2 * i + 1], c[4 + i], s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[i], y[i], c[i], s[i]);
  }
}

// 8 fp32 values to the destination type (times inv for E4M3), rounded once.
template <typename Dst>
__device__ __forceinline__ void store_f8(const float (&f)[8], void* base, size_t idx, float inv) {
  if constexpr (std::is_same<Dst, E4M3>::value) {
    uint2 p;
    uint16_t* h = reinterpret_cast<uint16_t*>(&p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = f32x2_to_e4m3x2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv));
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + idx) = p;
  } else {
    Raw8<Dst> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) store_elem<Dst>(&r, i, f[i]);
    uint4* d = reinterpret_cast<uint4*>(static_cast<typename Dst::raw*>(base) + idx);
#pragma unroll
    for (int i = 0; i < Dst::bytes / 2; ++i) d[i] = r.w[i];
  }
}

template <typename Src, typename Dst>
__device__ __forceinline__ void store_raw8(const Raw8<Src>& r, void* base, size_t idx, float inv) {
  store8<Src, Dst>(&r, static_cast<typename Dst::raw*>(base) + idx, inv);
}

// ------------------------------------------------------------------ rows
// One (token tile, row group): a thread walks rows_per_cta rows of its token,
// rows being the query heads, then (unless the cache is block-scaled) the K
// heads and the V heads.
template <typename Src, typename Dst, int D, bool BS>
__device__ __forceinline__ void append_rows(const AppendArgs& a, int cta) {
  constexpr int kUnits = D / 16;
  constexpr int kTok = kThreads / kUnits;
  constexpr int kU = 4;   // rows whose loads are in flight together
  const int u = threadIdx.x % kUnits;
  const int tile = cta / a.row_groups;
  const int row_first = (cta - tile * a.row_groups) * a.rows_per_cta;
  const int n_rows = a.n_q + (BS ? 0 : 2 * a.n_kv);
  const int row_end = min(row_first + a.rows_per_cta, n_rows);
  int seq, in_chunk;
  const int t = tile * kTok + threadIdx.x / kUnits;
  if (a.query_start == nullptr) {
    seq = t;
    in_chunk = 0;
    if (seq >= a.num_seqs) return;
  } else {
    seq = blockIdx.z;
    in_chunk = t;
  }
  const Chunk c = chunk_of(a, seq);
  if (in_chunk >= c.n) {
    if (c.bad && c.n == 0 && a.status != nullptr) atomicOr(a.status, PKV_DEVICE_BAD_LENGTH);
    return;
  }
  const size_t tok = static_cast<size_t>(c.row0) + in_chunk;
  if (c.bad || c.first < 0) {
    if (c.bad && a.status != nullptr) atomicOr(a.status, PKV_DEVICE_BAD_LENGTH);
    // (a chunk longer than max_len has more rows than the grid has tokens)
    const float fill = c.bad ? CUDART_NAN_F : 0.f;
    const int64_t step = (static_cast<int64_t>(a.max_len) + kTok - 1) / kTok * kTok;
    for (int64_t i = in_chunk; i < c.n; i += step)
      for (int r = row_first; r < min(row_end, a.n_q); ++r)
        for (int e = 0; e < 16; ++e)
          store_elem<Src>(a.q_out, ((c.row0 + i) * a.n_q + r) * D + 16 * u + e, fill);
    return;
  }
  const int pos = c.first + in_chunk;
  const UnitPlace w = unit_place(u, D, a.rotary, a.interleaved != 0);
  const int p0 = w.p0, p1 = w.p1;
  const bool turned = w.t0 || w.t1;
  int blk = -1;
  if (!BS && row_end > a.n_q) {
    blk = a.tables[static_cast<size_t>(seq) * a.max_blocks + pos / a.block_size];
    if (blk < 0 || blk >= a.num_blocks) {
      blk = -1;   // the token's K and V are not written
      if (a.status != nullptr) atomicOr(a.status, PKV_DEVICE_BAD_TABLE);
    }
  }
  float cs[8], sn[8];
  if (turned) load_angles(a, angle_row(a, pos), w, cs, sn);
  for (int r0 = row_first; r0 < row_end; r0 += kU) {
    Raw8<Src> x[kU], y[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int r = r0 + k;
      if (r >= row_end) continue;
      const void* base;
      size_t at;
      if (r < a.n_q) {
        base = a.q;
        at = tok * a.q_stride + static_cast<size_t>(r) * D;
      } else {
        const int which = r - a.n_q >= a.n_kv;
        const int h = r - a.n_q - (which ? a.n_kv : 0);
        base = a.src[which];
        at = tok * a.src_stride[which] + static_cast<size_t>(h) * D;
      }
      x[k] = load_raw8<Src>(base, at + p0);
      y[k] = load_raw8<Src>(base, at + p1);
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int r = r0 + k;
      if (r >= row_end) continue;
      const bool is_q = r < a.n_q;
      const int which = !is_q && r - a.n_q >= a.n_kv;
      const int h = is_q ? r : r - a.n_q - (which ? a.n_kv : 0);
      if (!is_q && blk < 0) continue;
      size_t dst;
      float inv = 1.f;
      if (is_q) {
        dst = (tok * a.n_q + h) * D;
      } else {
        dst = ((static_cast<size_t>(blk) * a.n_kv + h) * a.block_size + pos % a.block_size) * D;
        inv = a.head_scales ? a.head_scales[(2 + which) * a.n_kv + h] : a.inv_scale[which];
      }
      if (turned && !which) {
        float fx[8], fy[8];
        LoadF32<Src, 8>::run(&x[k], fx);
        LoadF32<Src, 8>::run(&y[k], fy);
        rotate(fx, fy, cs, sn, a.interleaved != 0, w);
        if (is_q) {
          store_f8<Src>(fx, a.q_out, dst + p0, 1.f);
          store_f8<Src>(fy, a.q_out, dst + p1, 1.f);
        } else {
          store_f8<Dst>(fx, a.cache[0], dst + p0, inv);
          store_f8<Dst>(fy, a.cache[0], dst + p1, inv);
        }
      } else if (is_q) {
        store_raw8<Src, Src>(x[k], a.q_out, dst + p0, 1.f);
        store_raw8<Src, Src>(y[k], a.q_out, dst + p1, 1.f);
      } else {
        store_raw8<Src, Dst>(x[k], a.cache[which], dst + p0, inv);
        store_raw8<Src, Dst>(y[k], a.cache[which], dst + p1, inv);
      }
    }
  }
}

// ----------------------------------------------------------------- blocks
// The least e with amax <= 448 * 2^e: 448 = 1.75 * 2^8, so e is the exponent
// of amax less 8, one more where its mantissa exceeds 1.75.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kMinScaleExp), kMaxScaleExp);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The scale of a block after new rows of maximum m (S_before 0 where the block
// holds nothing or its scale is no number).
__device__ __forceinline__ float grown_scale(float before, float m) { return fmaxf(before, scale_for(m)); }
__device__ __forceinline__ float valid_scale(float s) { return s > 0.f && s <= 1099511627776.f ? s : 0.f; }   // 2^40

// max(m, |x|) over finite x: an infinity saturates, a NaN stays, neither sets
// the scale.
__device__ __forceinline__ float amax8(const float (&x)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = fabsf(x[i]);
    m = v <= 3.402823466e38f ? fmaxf(m, v) : m;
  }
  return m;
}

// Earlier rows [0, r0) of a block whose scale grew, rounded again; lanes `lane`
// of `lanes`, a 16-byte piece each.
template <int D>
__device__ __forceinline__ void requantise(uint8_t* base, int r0, float ratio, int lane, int lanes) {
  for (int i = lane; i < r0 * (D / 16); i += lanes) {
    uint8_t* p = base + 16 * static_cast<size_t>(i);
    float x[8], y[8];
    LoadF32<E4M3, 8>::run(p, x);
    LoadF32<E4M3, 8>::run(p + 8, y);
    store_f8<E4M3>(x, p, 0, ratio);
    store_f8<E4M3>(y, p, 8, ratio);
  }
}

// One new token: the D / 16 lanes of a (sequence, KV head, K|V) hold its row.
template <typename Src, int D>
__device__ __forceinline__ void append_token(const AppendArgs& a, int seq, int h, int which) {
  constexpr int kUnits = D / 16;
  constexpr unsigned FULL = 0xffffffffu;
  const int u = threadIdx.x % kUnits;
  const int T = a.block_size;
  const bool in = seq < a.num_seqs;
  const Chunk c = in ? chunk_of(a, seq) : Chunk{0, 0, -1, false};
  const bool good = in && !c.bad && c.first >= 0;
  if (in && c.bad && u == 0 && a.status != nullptr) atomicOr(a.status, PKV_DEVICE_BAD_LENGTH);
  const UnitPlace w = unit_place(u, D, a.rotary, a.interleaved != 0);
  float x[8], y[8], m = 0.f, before = 0.f;
  const int row = good ? c.first % T : 0;
  float* scale_at = nullptr;   // NULL: a bad table entry
  size_t slab = 0;
  if (good) {   // the row and its angles beside the table entry and the scale
    const int blk = a.tables[static_cast<size_t>(seq) * a.max_blocks + c.first / T];
    if (blk >= 0 && blk < a.num_blocks) {
      slab = static_cast<size_t>(blk) * a.n_kv + h;
      scale_at = a.block_scales + slab * 2 + which;
      if (row > 0) before = valid_scale(*scale_at);
    }
    const typename Src::raw* p = static_cast<const typename Src::raw*>(a.src[which]) +
                                 static_cast<size_t>(c.row0) * a.src_stride[which] + static_cast<size_t>(h) * D;
    LoadF32<Src, 8>::run(p + w.p0, x);
    LoadF32<Src, 8>::run(p + w.p1, y);
    if (which == 0 && (w.t0 || w.t1)) {
      float cs[8], sn[8];
      load_angles(a, angle_row(a, c.first), w, cs, sn);
      rotate(x, y, cs, sn, a.interleaved != 0, w);
    }
    m = amax8(y, amax8(x, m));
  }
#pragma unroll
  for (int o = kUnits / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
  __syncwarp();   // every lane of a row has read the old scale
  if (!good) return;
  if (scale_at == nullptr) {
    if (u == 0 && a.status != nullptr) atomicOr(a.status, PKV_DEVICE_BAD_TABLE);
    return;
  }
  const float scale = grown_scale(before, m), inv = __frcp_rn(scale);
  uint8_t* base = static_cast<uint8_t*>(a.cache[which]) + slab * T * D;
  store_f8<E4M3>(x, base, static_cast<size_t>(row) * D + w.p0, inv);
  store_f8<E4M3>(y, base, static_cast<size_t>(row) * D + w.p1, inv);
  if (scale > before) {
    if (row > 0) requantise<D>(base, row, __fdiv_rn(before, scale), u, kUnits);
    if (u == 0) *scale_at = scale;
  }
}

// Chunks: 16 rows of one (touched block, KV head, K|V) per warp, kept as they
// came in registers between the maximum and the rounding; a block of 32 is two
// warps', which share their maximum (named barrier, both come by).  A CTA's
// warps are of one block, K heads before V heads, and share the angles of its
// rows in shared memory: read per head, they were as many bytes as the rows.
template <typename Src, int D>
__device__ __forceinline__ void append_block(const AppendArgs& a, int seq, int j, int part, float* s_angles,
                                             float* s_max) {
  constexpr int kUnits = D / 16;
  constexpr int kRows = 32 / kUnits;      // rows per pass
  constexpr int kPasses = 16 / kRows;
  constexpr unsigned FULL = 0xffffffffu;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = lane % kUnits, sub = lane / kUnits;
  const int T = a.block_size, warps = T / 16;
  const Chunk c = chunk_of(a, seq);
  if (c.bad) {
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, PKV_DEVICE_BAD_LENGTH);
    return;
  }
  if (c.n == 0) return;
  const int lb = c.first / T + j;
  const int end = c.first + c.n;
  if (static_cast<int64_t>(lb) * T >= end) return;
  const int r0 = max(c.first - lb * T, 0), r1 = min(end - lb * T, T);   // the new rows
  const int unit = (part * (kThreads / 32) + warp) / warps, half = warp % warps;
  const int which = unit >= a.n_kv, h = unit - which * a.n_kv;
  const bool mine = unit < 2 * a.n_kv;
  const UnitPlace w = unit_place(u, D, a.rotary, a.interleaved != 0);
  const bool turned = which == 0 && (w.t0 || w.t1);
  // the rows, the table entry and the angles are all on their way at once
  Raw8<Src> xr[kPasses], yr[kPasses];
  float m = 0.f;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = 16 * half + kRows * p + sub;
    if (!mine || row < r0 || row >= r1) continue;
    const size_t tok = static_cast<size_t>(c.row0) + (lb * T + row - c.first);
    const size_t at = tok * a.src_stride[which] + static_cast<size_t>(h) * D;
    xr[p] = load_raw8<Src>(a.src[which], at + w.p0);
    yr[p] = load_raw8<Src>(a.src[which], at + w.p1);
  }
  const int blk = a.tables[static_cast<size_t>(seq) * a.max_blocks + lb];
  if (a.rotary > 0 && part * (kThreads / 32) / warps < a.n_kv) {   // a K head among them
    const float4* src = reinterpret_cast<const float4*>(angle_row(a, lb * T + r0));
    float4* dst = reinterpret_cast<float4*>(s_angles + r0 * a.rotary);
    for (int i = threadIdx.x; i < (r1 - r0) * a.rotary / 4; i += kThreads) dst[i] = src[i];
  }
  __syncthreads();
  if (!mine) return;
  // the rotated values of pass p, computed for the maximum and again for the
  // rounding: kept, they would take twice the registers and half the warps
  auto values = [&](int p, float (&x)[8], float (&y)[8]) {
    LoadF32<Src, 8>::run(&xr[p], x);
    LoadF32<Src, 8>::run(&yr[p], y);
    if (turned) {
      float cs[8], sn[8];
      load_angles(a, s_angles + (16 * half + kRows * p + sub) * a.rotary, w, cs, sn);
      rotate(x, y, cs, sn, a.interleaved != 0, w);
    }
  };
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = 16 * half + kRows * p + sub;
    if (row < r0 || row >= r1) continue;
    float x[8], y[8];
    values(p, x, y);
    m = amax8(y, amax8(x, m));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
  if (blk < 0 || blk >= a.num_blocks) {   // the same for both warps of a block
    if (lane == 0 && a.status != nullptr) atomicOr(a.status, PKV_DEVICE_BAD_TABLE);
    return;
  }
  const size_t slab = static_cast<size_t>(blk) * a.n_kv + h;
  float* scale_at = a.block_scales + slab * 2 + which;
  const float before = r0 > 0 ? valid_scale(*scale_at) : 0.f;
  if (T > 16) {
    if (lane == 0) s_max[warp] = m;
    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");   // both have read the scale too
    m = fmaxf(m, s_max[warp ^ 1]);
  } else {
    __syncwarp();   // every lane has read it
  }
  const float scale = grown_scale(before, m), inv = __frcp_rn(scale);
  uint8_t* base = static_cast<uint8_t*>(a.cache[which]) + slab * T * D;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = 16 * half + kRows * p + sub;
    if (row < r0 || row >= r1) continue;
    float x[8], y[8];
    values(p, x, y);
    store_f8<E4M3>(x, base, static_cast<size_t>(row) * D + w.p0, inv);
    store_f8<E4M3>(y, base, static_cast<size_t>(row) * D + w.p1, inv);
  }
  if (scale > before && r0 > 0)
    requantise<D>(base, r0, __fdiv_rn(before, scale), lane + 32 * half, 32 * warps);
  if (lane == 0 && half == 0) *scale_at = scale;
}

template <typename Src, typename Dst, int D, bool BS>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  // launched as a programmatic dependent: the previous kernel in the stream
  // may still be reading what this one writes, or writing what it reads
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cta = blockIdx.x;
  if (!BS || cta < a.row_ctas) {
    append_rows<Src, Dst, D, BS>(a, cta);
  } else {
    if (a.query_start == nullptr) {
      const int per = 2 * a.n_kv;
      const int i = (cta - a.row_ctas) * (kThreads * 16 / D) + threadIdx.x / (D / 16);
      const int seq = i / per, hw = i - seq * per;
      append_token<Src, D>(a, seq, hw >> 1, hw & 1);
    } else {
      __shared__ __align__(16) float s_angles[32 * D];   // up to 32 rows of up to head_dim
      __shared__ float s_max[kThreads / 32];
      const int i = cta - a.row_ctas;
      append_block<Src, D>(a, blockIdx.z, i / a.block_parts, i % a.block_parts, s_angles, s_max);
    }
  }
}

template <typename Src, typename Dst, int D, bool BS>
pkv_status launch_append(AppendArgs a, cudaStream_t st) {
  constexpr int kTok = kThreads / (D / 16);
  const int rows = a.n_q + (BS ? 0 : 2 * a.n_kv);
  const bool one = a.query_start == nullptr;
  const int64_t tiles = (static_cast<int64_t>(one ? a.num_seqs : a.max_len) + kTok - 1) / kTok;
  // a decode step has few tokens: one batch of loads per thread, the rows
  // spread over more CTAs; many tokens fill the GPU with whole tokens
  const int64_t tokens = one ? a.num_seqs : a.total;
  // (rows per CTA of 12 and 36: 6,400 tokens of 36 rows 24.3 and 28.0 us,
  // 40,000 of 64 rows 282 and 264 us)
  const int most = tokens >= 16384 ? 36 : tokens >= 4096 ? 12 : 4;
  a.row_groups = rows > 0 ? (rows + most - 1) / most : 1;
  a.rows_per_cta = std::max((rows + a.row_groups - 1) / a.row_groups, 1);
  const int64_t row_ctas = rows > 0 ? tiles * a.row_groups : 0;
  int64_t block_ctas = 0;
  if (BS) {
    constexpr int kWarps = kThreads / 32;
    if (one) {
      block_ctas = (static_cast<int64_t>(a.num_seqs) * 2 * a.n_kv * (D / 16) + kThreads - 1) / kThreads;
    } else {
      a.block_parts = (2 * a.n_kv * (a.block_size / 16) + kWarps - 1) / kWarps;
      const int64_t touched = (a.max_len + static_cast<int64_t>(a.block_size) - 2) / a.block_size + 1;
      block_ctas = touched * a.block_parts;
    }
  }
  const int64_t ctas = row_ctas + block_ctas;
  if (ctas > INT32_MAX)
    return fail(PKV_ERR_UNSUPPORTED, "pkv_append: too many tokens in one call");
  if (ctas == 0) return PKV_OK;
  a.row_ctas = static_cast<int32_t>(row_ctas);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, one ? 1 : a.num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // between a decode step's attention kernels the SMs keep their split of L1
  // and shared memory; many tokens want their angles in L1 (6,400 tokens: 24.3
  // us, 29.6 with the least L1)
  attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
  attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
  cfg.attrs = attr;
  cfg.numAttrs = tokens < 4096 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel<Src, Dst, D, BS>, a);
  if (e != cudaSuccess) return cuda_fail("pkv_append: launch", e);
  return check_launch("pkv_append");
}

template <typename Src, typename Dst, bool BS>
pkv_status launch_append_d(const AppendArgs& a, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? launch_append<Src, Dst, 128, BS>(a, st)
                         : launch_append<Src, Dst, 64, BS>(a, st);
}

// --------------------------------------------------- scales of copied blocks
constexpr int kMaxScaleLayers = 128;
constexpr int kMaxScalePairs = 1024;

struct CopyScalesArgs {
  float* scales[kMaxScaleLayers];
  int32_t src[kMaxScalePairs];
  int32_t dst[kMaxScalePairs];
  int32_t per_block;   // floats of one block: 2 * n_kv
};

// grid: (pair, layer); each CTA copies the scales of one block.
__global__ void __launch_bounds__(32) copy_scales_kernel(const __grid_constant__ CopyScalesArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float* base = a.scales[blockIdx.y];
  const float* s = base + static_cast<size_t>(a.src[blockIdx.x]) * a.per_block;
  float* d = base + static_cast<size_t>(a.dst[blockIdx.x]) * a.per_block;
  for (int i = threadIdx.x; i < a.per_block; i += 32) d[i] = s[i];
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_append(void* k_cache, void* v_cache, float* block_scales, const void* k,
                                 int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                                 const void* q, int64_t q_stride, int32_t num_q_heads,
                                 int32_t src_dtype, const int32_t* block_tables, int32_t max_blocks,
                                 const int32_t* context_lens, const int32_t* query_start,
                                 int32_t num_seqs, int32_t total_tokens, int32_t max_query_len,
                                 const pkv_rope* rope, const pkv_kv_desc* desc, float k_inv_scale,
                                 float v_inv_scale, void* stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (num_seqs < 0 || total_tokens < 0 || max_query_len < 0 || num_q_heads < 0 || max_blocks < 0)
    return fail(PKV_ERR_INVALID_ARG, "negative size");
  const int src_bytes = src_dtype == PKV_E4M3 ? 0 : pkv_dtype_bytes(src_dtype);
  if (src_bytes == 0) return fail(PKV_ERR_INVALID_ARG, "src_dtype must be F32, F16 or BF16");
  const int kv = desc->kv_dtype;
  if (kv != PKV_E4M3 && src_dtype != kv)
    return fail(PKV_ERR_INVALID_ARG, "a 16/32-bit cache needs src_dtype == kv_dtype");
  if (block_scales) {
    if (kv != PKV_E4M3) return fail(PKV_ERR_INVALID_ARG, "block_scales need an E4M3 cache");
    if (desc->head_scales)
      return fail(PKV_ERR_INVALID_ARG, "block_scales and head_scales exclude each other");
    if (!aligned(block_scales, 8)) return fail(PKV_ERR_INVALID_ARG, "block_scales misaligned");
  }
  if (rope) {
    if (rope->rotary_dim < 0 || rope->max_position < 0)
      return fail(PKV_ERR_INVALID_ARG, "pkv_rope sizes must not be negative");
    if (rope->rotary_dim % 16 != 0 || rope->rotary_dim > desc->head_dim)
      return fail(PKV_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16, at most head_dim");
    if (rope->rotary_dim > 0 && (!rope->cos_sin || !aligned(rope->cos_sin, 16)))
      return fail(PKV_ERR_INVALID_ARG, "cos_sin is NULL or not 16-byte aligned");
  }
  if (num_q_heads > 0 && num_q_heads % desc->num_kv_heads != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
  if (num_seqs == 0 || total_tokens == 0 || max_query_len == 0) return PKV_OK;
  if (num_seqs > 65535) return fail(PKV_ERR_UNSUPPORTED, "more than 65535 sequences per call");
  if (max_blocks == 0) return fail(PKV_ERR_INVALID_ARG, "max_blocks is 0");
  if (!query_start && total_tokens != num_seqs)
    return fail(PKV_ERR_INVALID_ARG, "without query_start there is one token per sequence");
  if (static_cast<int64_t>(max_blocks) * desc->block_size > (int64_t{1} << 30))
    return fail(PKV_ERR_UNSUPPORTED, "context longer than 2^30 tokens");
  if (!k_cache || !v_cache || !k || !v || !block_tables || !context_lens)
    return fail(PKV_ERR_INVALID_ARG, "NULL pointer");
  if (num_q_heads > 0 && (!q || !q_out)) return fail(PKV_ERR_INVALID_ARG, "q or q_out is NULL");
  for (const void* p : {static_cast<const void*>(k_cache), static_cast<const void*>(v_cache), k, v})
    if (!aligned(p, 16)) return fail(PKV_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  if (num_q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16)))
    return fail(PKV_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4))
    return fail(PKV_ERR_INVALID_ARG, "tables misaligned");
  const int64_t vec = 16 / src_bytes;   // a row starts on a 16-byte boundary
  const int64_t kv_row = static_cast<int64_t>(desc->num_kv_heads) * desc->head_dim;
  if (k_stride < kv_row || v_stride < kv_row || k_stride % vec != 0 || v_stride % vec != 0)
    return fail(PKV_ERR_INVALID_ARG, "k_stride, v_stride: at least one row, a multiple of 16 bytes");
  if (num_q_heads > 0) {
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * desc->head_dim;
    if (q_stride < q_row || q_stride % vec != 0)
      return fail(PKV_ERR_INVALID_ARG, "q_stride: at least one row, a multiple of 16 bytes");
    // in place each thread reads what it writes; rows elsewhere would be
    // overwritten before another thread reads them
    if (q == q_out && q_stride != q_row)
      return fail(PKV_ERR_INVALID_ARG, "q_out may be q itself only where q is contiguous");
  }
  int* status = device_status_word(&st);
  if (!status) return st;

  AppendArgs a{};
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.src[0] = k;
  a.src[1] = v;
  a.src_stride[0] = k_stride;
  a.src_stride[1] = v_stride;
  a.q = q;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.block_scales = block_scales;
  a.inv_scale[0] = kv == PKV_E4M3 ? k_inv_scale : 1.f;
  a.inv_scale[1] = kv == PKV_E4M3 ? v_inv_scale : 1.f;
  a.head_scales = desc->head_scales;
  a.tables = block_tables;
  a.ctx_lens = context_lens;
  a.query_start = query_start;
  if (rope && rope->rotary_dim > 0) {
    a.angles = rope->cos_sin;
    a.max_position = rope->max_position;
    a.rotary = rope->rotary_dim;
    a.interleaved = rope->interleaved != 0;
  }
  a.max_blocks = max_blocks;
  a.num_seqs = num_seqs;
  a.total = total_tokens;
  // no chunk that is written is longer than the inputs or than a context
  a.max_len = std::min({max_query_len, total_tokens, max_blocks * desc->block_size});
  a.n_q = num_q_heads;
  a.n_kv = desc->num_kv_heads;
  a.block_size = desc->block_size;
  a.num_blocks = desc->num_blocks;
  a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int D = desc->head_dim;
  if (block_scales) {
    switch (src_dtype) {
      case PKV_F32: return launch_append_d<F32, E4M3, true>(a, D, s);
      case PKV_F16: return launch_append_d<F16, E4M3, true>(a, D, s);
      default: return launch_append_d<BF16, E4M3, true>(a, D, s);
    }
  }
  if (kv == PKV_E4M3) {
    switch (src_dtype) {
      case PKV_F32: return launch_append_d<F32, E4M3, false>(a, D, s);
      case PKV_F16: return launch_append_d<F16, E4M3, false>(a, D, s);
      default: return launch_append_d<BF16, E4M3, false>(a, D, s);
    }
  }
  switch (kv) {
    case PKV_F32: return launch_append_d<F32, F32, false>(a, D, s);
    case PKV_F16: return launch_append_d<F16, F16, false>(a, D, s);
    default: return launch_append_d<BF16, BF16, false>(a, D, s);
  }
}

extern "C" pkv_status pkv_copy_block_scales(float* const* block_scales, int32_t num_layers,
                                            const int32_t* src_dst, int32_t n_pairs,
                                            const pkv_kv_desc* desc, void* stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (desc->kv_dtype != PKV_E4M3) return fail(PKV_ERR_INVALID_ARG, "block_scales need an E4M3 cache");
  if (n_pairs < 0) return fail(PKV_ERR_INVALID_ARG, "n_pairs is negative");
  if (n_pairs == 0) return PKV_OK;
  if (num_layers <= 0 || num_layers > kMaxScaleLayers)
    return fail(PKV_ERR_INVALID_ARG, "num_layers must be in [1, 128]");
  if (!block_scales || !src_dst) return fail(PKV_ERR_INVALID_ARG, "NULL pointer");
  for (int32_t l = 0; l < num_layers; ++l)
    if (!block_scales[l] || !aligned(block_scales[l], 8))
      return fail(PKV_ERR_INVALID_ARG, "block_scales: NULL or misaligned layer pointer");
  for (int32_t i = 0; i < 2 * n_pairs; ++i)
    if (src_dst[i] < 0 || src_dst[i] >= desc->num_blocks)
      return fail(PKV_ERR_INVALID_ARG, "block id out of range");
  CopyScalesArgs a{};
  for (int32_t l = 0; l < num_layers; ++l) a.scales[l] = block_scales[l];
  a.per_block = 2 * desc->num_kv_heads;
  for (int32_t base = 0; base < n_pairs; base += kMaxScalePairs) {
    const int32_t n = std::min(kMaxScalePairs, n_pairs - base);
    for (int32_t i = 0; i < n; ++i) {
      a.src[i] = src_dst[2 * (base + i)];
      a.dst[i] = src_dst[2 * (base + i) + 1];
    }
    copy_scales_kernel<<<dim3(n, num_layers), 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
    st = check_launch("pkv_copy_block_scales");
    if (st != PKV_OK) return st;
  }
  return PKV_OK;
}
