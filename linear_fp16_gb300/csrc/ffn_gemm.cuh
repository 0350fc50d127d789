// The matrix products of the feed-forward block and of its gradients on the
// 5th-generation tensor cores (tcgen05), head dtype binary16 or bfloat16:
//
//   gated      g = x Wg^T + bg, u = x Wu^T + bu, h = act(g) u   (one pass)
//              A = x [M,K], B = Wg | Wu [N,K]; both contracted along their
//              rows (K-major)
//   dx         dx = sum_p D_p W_p, p = 1 or 2 products into one sum
//              A = D_p [M,N] K-major, B = W_p [N,K] contracted over its
//              rows' index (MN-major: the layout in memory is the transpose
//              of what the product needs, and the tensor core reads it so)
//   dW         dW_q = D_q^T x, q = 1 or 2 outputs
//              A = D_q [M,N] and B = x [M,K], both MN-major
//
// A persistent CTA (or a CTA pair on one 256-row tile, 2-SM MMA) per SM walks
// output tiles.  Warp roles as in the linear's GEMM: epilogue warps, one
// thread that issues the MMAs, one or two that issue the TMA loads.  A sum stays
// in TMEM (FP32 accumulators) over a chunk of K, unlike in the linear's kernel,
// which promotes every 1024 elements: these operators' outputs are rounded once
// from the FP32 value to 11 or 8 bits and carry no 2-ulp rule (chunks: see
// ffn_chunk_k).  The accumulators of two tiles fit TMEM, so the epilogue of a
// tile runs under the main loop of the next.  Bound by the tensor pipe under the
// power cap where K is long (GB300, bfloat16, 8192 x 14336 x 4096: gated with g
// and u 1.12 - 1.16 ms, 1.66 - 1.71 PFLOP/s; dx and both dW 2.25 - 2.34 ms, 1.64 -
// 1.71 PFLOP/s), by operand loads from L2 (about 80 GB/s per SM) and the start-up
// where one wave of tiles holds the problem.
//
// The gated tile: half of the tile's BN accumulator columns hold gate
// columns and half the same columns of up, so that one thread has g and u
// of an output side by side, and x's tile is read from shared memory once
// for both.  In a CTA pair each CTA loads half of the B rows: the even one
// gate rows, the odd one up rows.
//
// MN-major operands: a TMA box is 64 (contiguous) x 64 (K) elements with the
// 128-byte swizzle; boxes of a tile lie 8 KB apart (the descriptor's leading
// offset), groups of 8 K rows 1 KB apart (its stride offset), and a K step
// of 16 is 2 KB.
#pragma once

#include <type_traits>

#include "epilogue.cuh"
#include "pack.cuh"
#include "ptx.cuh"

namespace poot {

enum FfnAct : int { kActSilu = 0, kActGeluTanh = 1, kActGeluErf = 2 };

constexpr int kFfnBM = 128;
constexpr int kFfnBK = 64;  // one 128-byte swizzle row
// Epilogue warps; then the MMA issuer; then the TMA producer, in the gated
// kernel one per operand.  The gated kernel takes eight epilogue warps with 168
// registers and two staging boxes each, the gradients sixteen with one (GB300:
// gated 1417 x 520 x 1280 9.9 us with eight, 10.8 with sixteen, 4096 x 4096 x
// 1024 with g and u 48.6 and 50.5; gradients 6 x 8320 x 470 29.8 and 27.0, 112
// x 4480 x 2531 61 and 55, 1024 x 1024 x 768 14.8 and 15.4).
__host__ __device__ constexpr int ffn_epi_warps(bool gated) { return gated ? 8 : 16; }
__host__ __device__ constexpr int ffn_threads(bool gated) { return (ffn_epi_warps(gated) + (gated ? 3 : 2)) * 32; }
constexpr int kFfnMaxBN = 256;
// Elements of K summed in TMEM.  An MMA truncates where it adds 16 products to
// the running sum, always towards zero: sums of one sign come out low by 6.3e-9
// of themselves per term (mean over many outputs on GB300: 5.4e-5 over 8192 terms,
// 1.7e-3 over 262144, where one rounding is 4.9e-4 in binary16 and 3.9e-3 in
// bfloat16).  Chunks keep that at an eighth of the rounding in binary16 and at a
// twentieth in bfloat16 (measured: 5e-5 and 2e-4 at any length).  Longer sums
// are added up over chunks in FP32, rounded to nearest, in a scratch of the CTA
// (128 KB, from L2) by the epilogue warps under the main loop of the next chunk.
// (8192 for bfloat16 too: 2480 -> 2560 us for the gradients of 8192 x 14336 x
// 4096, whose dx sums 28672 terms.)
__host__ __device__ constexpr int ffn_chunk_k(int dtype) { return dtype == kEpiBf16 ? 32768 : 8192; }
constexpr int kFfnMaxStages = 8;
constexpr uint32_t kFfnTmemCols = 2 * kFfnMaxBN;

// Eight consecutive head-dtype elements p[0 .. n) (n <= 8, the rest zero) at
// any 2-byte alignment.
__device__ __forceinline__ uint4 ffn_load8(const uint16_t* __restrict__ p, int n) {
  if (n >= 8) return pack_load8(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j >> 1] |= (uint32_t)__ldg(p + j) << ((j & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows that no wide load fits: the two 16-byte vectors around p, shifted into
// place, where both lie inside the memory [lo, hi) that the matrix spans.
// (Eight 2-byte loads a lane made such kernels bound by their number.)  In
// three steps, so that a caller has several pairs on their way at a time.
__device__ __forceinline__ bool ffn_wide_ok(const uint16_t* p, const void* lo, const void* hi) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15);
  return a0 >= reinterpret_cast<uintptr_t>(lo) && a0 + 32 <= reinterpret_cast<uintptr_t>(hi);
}
struct FfnPair {
  uint4 u, v;
};
__device__ __forceinline__ FfnPair ffn_wide_load(const uint16_t* p) {
  const uint4* a0 = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
  return {__ldg(a0), __ldg(a0 + 1)};
}
__device__ __forceinline__ uint4 ffn_wide_shift(const uint16_t* p, const FfnPair& r) {
  const uint32_t sh = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
  uint32_t w[8] = {r.u.x, r.u.y, r.u.z, r.u.w, r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = (sh & 8u) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = (sh & 4u) ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (sh & 2u) << 3);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// eight elements p[0 .. n) at any alignment, the rest zero
__device__ __forceinline__ uint4 ffn_load8_any(const uint16_t* __restrict__ p, int n, const void* lo, const void* hi) {
  if (n < 8 || !ffn_wide_ok(p, lo, hi)) return ffn_load8(p, n);
  return ffn_wide_shift(p, ffn_wide_load(p));
}

template <int DT>
__device__ __forceinline__ void ffn_unpack8(const uint4& v, float (&f)[8]) {
  const float2 a = ep_unpack_t<DT>(v.x), b = ep_unpack_t<DT>(v.y), c = ep_unpack_t<DT>(v.z), d = ep_unpack_t<DT>(v.w);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y; f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}
template <int DT>
__device__ __forceinline__ uint4 ffn_pack8(const float (&f)[8]) {
  return make_uint4(ep_pack_t<DT>(f[0], f[1]), ep_pack_t<DT>(f[2], f[3]), ep_pack_t<DT>(f[4], f[5]),
                    ep_pack_t<DT>(f[6], f[7]));
}

// Activations in FP32 and their derivatives, from the formulas (s is the
// logistic function):
//   silu       t s(t)                     s + t s (1 - s)
//   gelu_tanh  t s(z), z = a (t + b t^3)  s + t s (1 - s) z'
//              a = 2 sqrt(2/pi), b = 0.044715: the tanh form 0.5 t (1 +
//              tanh(z / 2)) written with the logistic function
//   gelu_erf   t P(t), P the normal distribution function; P + t p(t), p the
//              normal density
// Values, their lower tails included, carry a relative error of at most 2^-15
// (exponents of up to 130 rounded to FP32), far below the one rounding to 11 or
// 8 bits that follows; the derivatives' two terms likewise.  Below 2^-126 the
// error is FP32's subnormal step, far below bfloat16's.
// Where s (1 - s) is 0 in FP32 z' may overflow: the second term is then
// dropped, as in the limit.
// 2^x for x <= 0.  Subnormal results are kept for bfloat16, whose range they lie
// in: 2^(x + 24) times 2^-24, within 2^-20 (the sum's rounding; the instruction
// that keeps them itself takes three more around it: 7540 x 1845 with bias
// gradients 47.5 us against 45.4).  binary16 products of 2^-126 round to zero
// either way, so its form drops them.
template <int DT>
__device__ __forceinline__ float act_exp2(float x) {
  float y;
  if constexpr (DT != kEpiF16) x += 24.0f;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return DT == kEpiF16 ? y : y * 5.9604644775390625e-8f;
}
__device__ __forceinline__ float act_rcp(float x) {  // of 1 and more (its result is never subnormal here)
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// s(z), from e = exp(-|z|) <= 1: 1 / (1 + e), or e / (1 + e) below zero, which
// keeps its relative precision where 1 / (1 + exp(-z)) would pass FP32's
// range (z < -87); `q` is s (1 - s) = e / (1 + e)^2
template <int DT>
__device__ __forceinline__ float act_sigmoid(float z, float& q) {
  const float e = act_exp2<DT>(-kLog2e * fabsf(z));
  const float r = act_rcp(1.0f + e), er = e * r;
  q = er * r;
  return z < 0.0f ? er : r;
}
template <int DT>
__device__ __forceinline__ float act_sigmoid(float z) {
  float q;
  return act_sigmoid<DT>(z, q);
}

// The normal distribution function P(t) and e = exp(-t^2 / 2).  With x = |t| /
// sqrt 2, P(-|t|) = erfcx(x) / 2 exp(-x^2), where erfcx(x) = exp(x^2) erfc(x) is
// smooth; erfcx / 2 is a polynomial of degree 7 without constant term in k = 1 /
// (1 + x / 2), fitted to the least maximum of the relative error on 0 <= x <=
// 9.9 (linear programming on 4200 points): 1.3e-6.  Beyond, exp(-x^2) is below
// FP32's range.  So the lower tail keeps its relative precision, the upper
// is 1 minus it, and the density of the derivative shares the exponential.
template <int DT>
__device__ __forceinline__ float act_normal(float t, float& e) {
  const float x = fabsf(t) * 0.70710678118654752f;
  const float k = act_rcp(fmaf(0.5f, x, 1.0f));
  e = act_exp2<DT>(-kLog2e * x * x);
  float q = fmaf(0.04424222412682183f, k, -0.17885875741623095f);
  q = fmaf(q, k, 0.19529158283855405f);
  q = fmaf(q, k, 0.018470059767194402f);
  q = fmaf(q, k, 0.14092733335201088f);
  q = fmaf(q, k, 0.1387589425987517f);
  q = fmaf(q, k, 0.14116796674491414f) * k * e;
  return t < 0.0f ? q : 1.0f - q;
}

template <int ACT, int DT>
__device__ __forceinline__ float act_value_t(float t) {
  if constexpr (ACT == kActSilu) {
    return t * act_sigmoid<DT>(t);
  } else if constexpr (ACT == kActGeluTanh) {
    return t * act_sigmoid<DT>(1.5957691216057308f * fmaf(0.044715f * t * t, t, t));
  } else {
    float e;
    return t * act_normal<DT>(t, e);
  }
}
template <int DT>
__device__ __forceinline__ float act_value(int act, float t) {
  return act == kActSilu ? act_value_t<kActSilu, DT>(t)
                         : (act == kActGeluTanh ? act_value_t<kActGeluTanh, DT>(t) : act_value_t<kActGeluErf, DT>(t));
}

// value in v, derivative in d
template <int ACT, int DT>
__device__ __forceinline__ void act_both_t(float t, float& v, float& d) {
  if constexpr (ACT == kActGeluErf) {
    float e;
    const float p = act_normal<DT>(t, e);
    v = t * p;
    d = e != 0.0f ? fmaf(t * 0.3989422804014327f, e, p) : p;
  } else {
    float z = t, dz = 1.0f;
    if constexpr (ACT == kActGeluTanh) {
      const float t2 = t * t;
      z = 1.5957691216057308f * fmaf(0.044715f * t2, t, t);
      dz = 1.5957691216057308f * fmaf(0.134145f, t2, 1.0f);
    }
    float q;
    const float s = act_sigmoid<DT>(z, q);
    v = t * s;
    d = q != 0.0f ? fmaf(t * q, dz, s) : s;
  }
}

// Division of n < 2^31 by a divisor known on the host (Granlund and Montgomery,
// "Division by invariant integers using multiplication"): a tile's
// coordinates take six, and the first tile's stand before its first load.
struct FfnDiv {
  uint32_t d = 1, mul = 1, shift = 0;
  FfnDiv() = default;
  explicit FfnDiv(uint32_t d_) : d(d_) {
    while ((uint64_t(1) << shift) < d) ++shift;
    mul = static_cast<uint32_t>((((uint64_t(1) << shift) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// One family of tiles: the products of one kind, with their operands.
// gated: a[0] = x, b = Wg, Wu, y = h, g, u.  dx: a = D_p, b = W_p, y[0] = dx.
// dW: a = D_q, b[0] = x, y = dW_q.
struct FfnJob {
  // the first tile's load needs these
  int tiles_per_out, split, group_m, num_n, num_m;
  int kb_part;       // K blocks (SUB * 64 elements) of one part
  int kb_total;      // over all parts
  int kb_split;      // K blocks of a range (the last may be shorter); split ranges, tiles of their own
  FfnDiv by_out, by_split, by_span, by_group, by_rest;  // tiles_per_out, split, group_m num_n, group_m, the last group's
  // the epilogue these
  int M, N;          // rows and columns of one output (gated: of h)
  int tiles;
  int tma_store;     // outputs stored by TMA; 0: plain stores
  uint16_t* y[3];    // row pitch N
};

// tile t -> (K range, output, M block, N block).  Groups of group_m M blocks
// are walked column by column, odd groups from the far end, so that CTAs
// running together share rows of both operands in L2.
struct FfnTile {
  int s, g, mb, nb;
  __device__ __forceinline__ FfnTile(const FfnJob& j, uint32_t t) {
    const uint32_t q = j.by_out.div(t), tl = t - q * (uint32_t)j.tiles_per_out;
    g = (int)j.by_split.div(q);
    s = (int)q - g * j.split;
    const int span = j.group_m * j.num_n, group = (int)j.by_span.div(tl), first_m = group * j.group_m;
    const uint32_t local = tl - (uint32_t)(group * span);
    const bool rest = j.num_m - first_m < j.group_m;
    nb = (int)(rest ? j.by_rest.div(local) : j.by_group.div(local));
    mb = first_m + (int)local - nb * (rest ? j.num_m - first_m : j.group_m);
    if (group & 1) nb = j.num_n - 1 - nb;
  }
};

struct FfnMaps {
  CUtensorMap a[2][2], b[2][2], y[2][3];  // [job][operand]
  CUtensorMap partial[2];                 // FP32 [slabs][M][N], rows of a 16-byte pitch
};

// Bias gradients, done by the epilogue warps before their first tile: db[o] =
// sum over rows of either FP32 row-block sums (the gate's gradient leaves
// them) or the rows of D itself.
struct FfnBiasGrad {
  const float* sums;   // [rows][outputs][pitch], pitch = N rounded up to 8, or nullptr
  const uint16_t* d;   // [rows][N] head dtype, rows ld apart, or nullptr
  long long ld;
  long long rows;
  int outputs, N;      // outputs: 0 (none), 1 or 2
  uint16_t* out[2];    // either may be nullptr
};

struct FfnDeal {     // see FfnSchedule
  int first;         // the job with the longer tiles
  int rounds, rest;  // its tiles: full rounds over all CTAs (pairs), and what is left
  int extra, base;   // tiles of the other job dealt to CTAs it leaves short: each, all
  int rounds1, rest1;  // the other job's tiles after those
  int tiles1;        // the other job's tiles
};

// (a kernel's first reads of its arguments miss every cache: what the first
// tile needs stands together)
struct FfnGemmArgs {
  FfnDeal deal;
  int bn;            // accumulator columns of a tile (gated: bn / 2 columns of h)
  int cols;          // output columns of a tile
  int stages;
  int act, save;
  FfnJob job[2];     // gated: job 0; gradients: dx, dW (either may have no tiles)
  const uint16_t* bias[2];  // gated: bg, bu or nullptr
  FfnBiasGrad bias_grad;
  float4* scratch;   // sums of earlier chunks, kFfnScratchBytes a CTA; nullptr: no sum has two
};
constexpr int kFfnScratchBytes = kFfnBM * kFfnMaxBN * 4;

// The tiles of one CTA (or pair): its round-robin share of the job with the
// longer tiles (deal.first); then, where that leaves it one tile short of
// others, `extra` tiles of the other job (as many as take the time of one);
// then its round-robin share of the rest of the other job.  count(job) tiles,
// the i-th is tile(job, i).
struct FfnSchedule {
  int first, unit, units, r, extra, base, n0, n1;
  __device__ __forceinline__ FfnSchedule(const FfnDeal& d, int unit_, int units_)
      : first(d.first), unit(unit_), units(units_), r(d.rest), extra(0), base(d.base) {
    if (r != 0 && unit >= r && d.extra > 0) {  // those that exist
      const int start = unit - r, step = units - r;
      extra = d.extra;
      if (start + (extra - 1) * step >= d.tiles1) extra = start < d.tiles1 ? (d.tiles1 - 1 - start) / step + 1 : 0;
    }
    n0 = d.rounds + (unit < r ? 1 : 0);
    n1 = extra + d.rounds1 + (unit < d.rest1 ? 1 : 0);
  }
  __device__ __forceinline__ int count(int job) const { return job == first ? n0 : n1; }
  __device__ __forceinline__ int tile(int job, int i) const {
    if (job == first) return i * units + unit;
    return i < extra ? i * (units - r) + (unit - r) : base + (i - extra) * units + unit;
  }
};

// Shared memory: operand ring, then the epilogue warps' staging boxes and the
// biases of a tile's columns, then barriers.
struct FfnLayout {
  static constexpr int RING_BYTES = 192 * 1024;
  static constexpr int STG_BYTES = 32 * 32 * 2;
  static constexpr int OFF_STG = RING_BYTES;
  static constexpr int STG_BOXES = 16;  // 32 x 32 output boxes, shared out among the epilogue warps
  static constexpr int OFF_BIAS = OFF_STG + STG_BOXES * STG_BYTES;  // [accumulator][box][gate, up][32]
  static constexpr int OFF_BAR = OFF_BIAS + 2 * 4 * 2 * 32 * 2;
  static constexpr int NUM_BARS = 2 * kFfnMaxStages + 5;  // full, empty, acc full x2, acc empty x2, drain
  static constexpr int OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int DYN_BYTES = OFF_ABORT + 4 + 1024;
  static_assert(OFF_BAR % 8 == 0, "mbarriers are 8-byte objects");
  static_assert(DYN_BYTES <= 232448, "more shared memory than a CTA can have");
};

// 64-element sub-blocks of K per stage.  A CTA pair takes two, so that the
// issuing thread waits and commits once per eight MMAs (one wait and commit
// per four leaves gaps in the tensor pipe); a single CTA takes one, for a
// deeper ring on the small problems it serves.
__host__ __device__ constexpr int ffn_sub(int cl) { return cl == 2 ? 2 : 1; }
// K blocks of a chunk
__host__ __device__ constexpr int ffn_chunk_kb(int cl, int dtype) { return ffn_chunk_k(dtype) / (kFfnBK * ffn_sub(cl)); }
__host__ __device__ constexpr int ffn_a_bytes(int cl) { return kFfnBM * kFfnBK * 2 * ffn_sub(cl); }
__host__ __device__ constexpr int ffn_b_bytes(int cl, int bn) { return bn / cl * kFfnBK * 2 * ffn_sub(cl); }
__host__ __device__ constexpr int ffn_stages(int cl, int bn) {
  return FfnLayout::RING_BYTES / (ffn_a_bytes(cl) + ffn_b_bytes(cl, bn)) < kFfnMaxStages
             ? FfnLayout::RING_BYTES / (ffn_a_bytes(cl) + ffn_b_bytes(cl, bn))
             : kFfnMaxStages;
}

// Shared-memory matrix descriptor of an MN-major operand in the 128-byte
// swizzle: 64-element chunks of the contiguous dimension 8 KB apart (leading
// byte offset), 8-row groups along K 1 KB apart (stride byte offset).
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Loads `rows` x 64 (K) elements of one operand into consecutive shared
// memory: K-major in one box of `rows` rows, MN-major in boxes of 64.
template <int CL>
__device__ __forceinline__ void ffn_load(bool mn, uint32_t dst, const CUtensorMap* map, uint32_t bar, int row0,
                                         int rows, int k0) {
  if (mn) {
    for (int r = 0; r < rows; r += 64) {
      if constexpr (CL == 2) tma_load_2d_pair(dst + (uint32_t)r * 128u, map, bar, row0 + r, k0);
      else tma_load_2d(dst + (uint32_t)r * 128u, map, bar, row0 + r, k0);
    }
  } else {
    if constexpr (CL == 2) tma_load_2d_pair(dst, map, bar, k0, row0);
    else tma_load_2d(dst, map, bar, k0, row0);
  }
}

// the epilogue warps of a gradient kernel
__device__ __forceinline__ void ffn_epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(ffn_epi_warps(false) * 32) : "memory"); }

// Bias gradients by the epilogue warps of all CTAs: a CTA takes consecutive
// groups of 8 columns (of all outputs, side by side), a lane every so-many-th
// row of one group.  Lanes of a group meet by shuffles, warps in shared
// memory, in a fixed order.  FP32 sums, one rounding.
template <int DT>
__device__ __forceinline__ void ffn_bias_grad(const FfnBiasGrad& b, float* red, int cta, int ctas) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_out = (b.N + 7) / 8;             // groups of one output
  const int groups = per_out * b.outputs;
  const int share = (groups + ctas - 1) / ctas;
  const int g0 = cta * share, g1 = min(groups, g0 + share);
  for (int base = g0; base < g1; base += 32) {
    const int n = min(32, g1 - base);            // groups of this round
    int width = 1;                               // lanes side by side on them
    while (width < n) width *= 2;
    const int g = lane & (width - 1);
    constexpr int kWarps = ffn_epi_warps(false);
    const int step = kWarps * 32 / width;  // rows read at one time
    const int o = (base + g) / per_out, c = ((base + g) - o * per_out) * 8, nc = min(8, b.N - c);
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.0f;
    if (g < n) {
      const long long r0 = warp * (32 / width) + lane / width;
      if (b.sums != nullptr) {
        const int pitch = per_out * 8;
        const float* p = b.sums + (size_t)o * pitch + c;
        const size_t stride = (size_t)b.outputs * pitch;
#pragma unroll 4
        for (long long r = r0; r < b.rows; r += step) {
          const float4* q = reinterpret_cast<const float4*>(p + (size_t)r * stride);
          const float4 u = __ldg(q), v = __ldg(q + 1);
          s[0] += u.x; s[1] += u.y; s[2] += u.z; s[3] += u.w;
          s[4] += v.x; s[5] += v.y; s[6] += v.z; s[7] += v.w;
        }
      } else {
        const uint16_t *p = b.d + c, *hi = b.d + (b.rows - 1) * b.ld + b.N;
        // (columns past N, inside the row's pitch, are added up and not stored;
        // the last row's may not be there)
        const bool vec = c + 8 <= b.ld && b.ld % 8 == 0 && (reinterpret_cast<uintptr_t>(b.d) & 15u) == 0;
#pragma unroll 4
        for (long long r = r0; r < b.rows; r += step) {
          const uint4 v = vec && (nc == 8 || r + 1 < b.rows) ? __ldg(reinterpret_cast<const uint4*>(p + r * b.ld))
                              : ffn_load8_any(p + r * b.ld, nc, b.d, hi);
          float f[8];
          ffn_unpack8<DT>(v, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] += f[j];
        }
      }
    }
    for (int off = width; off < 32; off *= 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], off);
    }
    if (lane < n) {
#pragma unroll
      for (int j = 0; j < 8; ++j) red[(warp * 32 + lane) * 9 + j] = s[j];
    }
    ffn_epi_sync();
    if ((int)threadIdx.x < n * 8) {
      const int gg = threadIdx.x >> 3, j = threadIdx.x & 7;
      const int oo = (base + gg) / per_out, col = ((base + gg) - oo * per_out) * 8 + j;
      uint16_t* out = oo ? b.out[1] : b.out[0];
      if (col < b.N && out != nullptr) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += red[(w * 32 + gg) * 9 + j];
        out[col] = (uint16_t)ep_pack_t<DT>(t, 0.0f);
      }
    }
    ffn_epi_sync();
  }
}

// A lane's 32 sums of a box in the scratch of FfnGemmArgs: `p` is its first
// float4, the next ones follow 32 apart (a warp's lanes side by side).
__device__ __forceinline__ void ffn_store_scratch(float4* p, const uint32_t (&r)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    p[j * 32] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                            __uint_as_float(r[4 * j + 3]));
}
// r += what stands there
__device__ __forceinline__ void ffn_add_scratch(const float4* p, uint32_t (&r)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 v = p[j * 32];
    r[4 * j] = __float_as_uint(v.x + __uint_as_float(r[4 * j]));
    r[4 * j + 1] = __float_as_uint(v.y + __uint_as_float(r[4 * j + 1]));
    r[4 * j + 2] = __float_as_uint(v.z + __uint_as_float(r[4 * j + 2]));
    r[4 * j + 3] = __float_as_uint(v.w + __uint_as_float(r[4 * j + 3]));
  }
}

// CHUNKS: some sum has more than one chunk (host: FfnSpace).  A form of its own,
// because the code for it costs the others 2 - 3% (1024 x 1024 x 768 gradients
// 16.4 -> 17.0 us).
template <int CL, bool GATED, int DT, bool CHUNKS>
__global__ void __launch_bounds__(ffn_threads(GATED), 1)
    ffn_gemm_kernel(const __grid_constant__ FfnMaps maps, const __grid_constant__ FfnGemmArgs args) {
  using L = FfnLayout;
  constexpr bool PAIR = CL == 2;
  constexpr int EPI_WARPS = ffn_epi_warps(GATED), MMA_WARP = EPI_WARPS, PROD_WARP = EPI_WARPS + 1;  // A's; then B's
  constexpr int STG = L::STG_BOXES / EPI_WARPS;  // staging boxes of a warp
  constexpr int SUB = ffn_sub(CL);
  constexpr int A_BYTES = ffn_a_bytes(CL);
  constexpr int A_SUB = A_BYTES / SUB;
  const int BN = args.bn;
  const int STAGES = args.stages;
  const int B_BYTES = ffn_b_bytes(CL, BN);
  const int B_SUB = B_BYTES / SUB;
  const int STAGE_BYTES = A_BYTES + B_BYTES;
  const uint32_t crank = PAIR ? cluster_ctarank() : 0u;
  const uint32_t rank = crank & 1u;
  const bool leader = rank == 0;
  const int unit = (int)(blockIdx.x / CL);
  const int units = (int)(gridDim.x / CL);
  const int tile_rows = CL * kFfnBM;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bar0 = sbase + L::OFF_BAR;
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (kFfnMaxStages + s); };
  auto bar_cfull = [&](int a) { return bar0 + 8u * (2 * kFfnMaxStages + a); };
  auto bar_cempty = [&](int a) { return bar0 + 8u * (2 * kFfnMaxStages + 2 + a); };
  const uint32_t bar_drain = bar0 + 8u * (2 * kFfnMaxStages + 4);
  auto stage_a = [&](int s) { return sbase + (uint32_t)(s * STAGE_BYTES); };
  auto stage_b = [&](int s) { return sbase + (uint32_t)(s * STAGE_BYTES + A_BYTES); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_TMEM_SLOT);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full(s), 1u);
      mbar_init(bar_empty(s), 1u);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar_cfull(a), 1u);
      mbar_init(bar_cempty(a), (uint32_t)(CL * EPI_WARPS));
    }
    mbar_init(bar_drain, 1u);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_addr(tmem_slot), kFfnTmemCols);
      tmem_relinquish_alloc_permit_pair();
    } else {
      tmem_alloc(smem_addr(tmem_slot), kFfnTmemCols);
      tmem_relinquish_alloc_permit();
    }
  }
  grid_dep_launch();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers exist before any remote signal
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  // Each role waits for the previous grid itself, just before it touches
  // global memory: the schedule and the first tile's coordinates (reads of
  // arguments that miss every cache) are then done by the time it ends.
  // (Prefetching the tensor maps in the prologue made it 1 us longer.)
  const FfnSchedule sched(args.deal, unit, units);
  if (warp >= PROD_WARP) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      // JI: 0 dx (or the gated block), 1 dW.  A's producer arms the stage's
      // barrier for both operands' bytes; B's may land before that (the
      // phase stays open until the arrival).
      auto load_job = [&](auto ji_tag, auto op_tag) {
        constexpr int ji = decltype(ji_tag)::value;
        constexpr bool IS_A = (decltype(op_tag)::value & 1) != 0, IS_B = (decltype(op_tag)::value & 2) != 0;
        const FfnJob& job = args.job[ji];
        const int tiles = sched.count(ji);
        for (int ti = 0; ti < tiles && ok; ++ti) {
          const FfnTile tile(job, (uint32_t)sched.tile(ji, ti));
          const int kb0 = tile.s * job.kb_split, kb1 = min(job.kb_total, kb0 + job.kb_split);
          const int arow = tile.mb * tile_rows + (int)rank * kFfnBM;
          const int brow = tile.nb * args.cols + (GATED ? 0 : (int)rank * (BN / CL));
          for (int kb = kb0; kb < kb1; ++kb) {
            if (issued == 0) grid_dep_wait();
            if (issued >= STAGES && !mbar_wait(bar_empty(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
            const uint32_t fb = bar_full(stage);
            const uint32_t fbl = PAIR ? map_to_cta(fb, 0u) : fb;  // both CTAs' bytes complete on the even CTA's barrier
            if (IS_A && leader) mbar_arrive_expect_tx(fb, (uint32_t)(CL * STAGE_BYTES));
            const int part = kb >= job.kb_part ? 1 : 0;  // (one part: kb never gets there)
            const int kc = (kb - part * job.kb_part) * (SUB * kFfnBK);
#pragma unroll
            for (int h = 0; h < SUB; ++h) {
              const int k0 = kc + h * kFfnBK;
              if constexpr (IS_A)
                ffn_load<CL>(!GATED && ji == 1, stage_a(stage) + (uint32_t)(h * A_SUB),
                             &maps.a[ji][GATED ? 0 : (ji == 1 ? tile.g : part)], fbl, arow, kFfnBM, k0);
              if constexpr (IS_B) {
                const uint32_t db = stage_b(stage) + (uint32_t)(h * B_SUB);
                ffn_load<CL>(!GATED, db, &maps.b[ji][GATED ? (PAIR ? (int)rank : 0) : (ji == 1 ? 0 : part)], fbl, brow,
                             GATED ? BN / 2 : BN / CL, k0);
                if constexpr (GATED && !PAIR)
                  ffn_load<CL>(false, db + (uint32_t)(BN / 2) * 128u, &maps.b[0][1], fbl, brow, BN / 2, k0);
              }
            }
            ++issued;
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
        }
      };
      auto load_jobs = [&](auto op) {
        const std::integral_constant<int, 0> j0;
        const std::integral_constant<int, 1> j1;
        if (GATED || args.deal.first == 0) {
          load_job(j0, op);
          if constexpr (!GATED) load_job(j1, op);
        } else {
          load_job(j1, op);
          load_job(j0, op);
        }
      };
      if constexpr (!GATED) load_jobs(std::integral_constant<int, 3>{});
      else if (warp == PROD_WARP) load_jobs(std::integral_constant<int, 1>{});
      else load_jobs(std::integral_constant<int, 2>{});
      // the last loads land before the CTA can exit (in a pair the odd CTA is
      // held by the closing cluster barrier)
      if (leader) {
        int s = stage;
        uint32_t ph = phase;
        for (int i = 0; i < STAGES && i < issued; ++i) {
          if (s == 0) { s = STAGES - 1; ph ^= 1u; } else { --s; }
          mbar_wait(bar_full(s), ph, nullptr);
        }
      }
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      // (reads no global memory: the waits below are limited in time, and that
      // of the previous grid must not count)
      grid_dep_wait();
      int stage = 0;
      uint32_t phase = 0;
      int buf = 0;
      uint32_t buf_phase = 0;
      bool ok = true;
      // dx tiles and dW tiles each have a loop of their own, whose operand
      // order and instruction descriptor are constants: with the order chosen
      // per tile the issuing thread leaves gaps in the tensor pipe (8192 x
      // 4096 x 14336, both gradients: 1073 us against 1006)
      auto issue_job = [&](auto ji_tag) {
        constexpr int ji = decltype(ji_tag)::value;
        constexpr bool A_MN = !GATED && ji == 1, B_MN = !GATED;
        // 16 elements along K: 32 bytes inside the swizzle row (K-major), two
        // 8-row groups (MN-major)
        constexpr uint32_t AK = A_MN ? 2048u >> 4 : 2u, BKS = B_MN ? 2048u >> 4 : 2u;
        const FfnJob& job = args.job[ji];
        const uint32_t idesc = idesc_f16_f32acc(PAIR ? 2 * kFfnBM : kFfnBM, (uint32_t)BN) |
                               (DT == kEpiBf16 ? ((1u << 7) | (1u << 10)) : 0u) |
                               (A_MN ? (1u << 15) : 0u) | (B_MN ? (1u << 16) : 0u);
        const int tiles = sched.count(ji);
        for (int ti = 0; ti < tiles && ok; ++ti) {
          const uint32_t q = job.by_out.div((uint32_t)sched.tile(ji, ti));
          const int s = (int)(q - job.by_split.div(q) * (uint32_t)job.split);
          const int kb0 = s * job.kb_split, kb1 = min(job.kb_total, kb0 + job.kb_split);
          for (int kc = kb0;;) {  // chunks
            const int kend = CHUNKS ? min(kb1, kc + ffn_chunk_kb(CL, DT)) : kb1;
            if (!mbar_wait(bar_cempty(buf), buf_phase ^ 1u, abort_flag)) { ok = false; break; }
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem_base + (uint32_t)(buf * kFfnMaxBN);
            uint32_t acc = 0;
            for (int kb = kc; kb < kend; ++kb) {
              if (!mbar_wait(bar_full(stage), phase, abort_flag)) { ok = false; break; }
              tc_fence_after_sync();
#pragma unroll
              for (int h = 0; h < SUB; ++h) {
                const uint32_t sa = stage_a(stage) + (uint32_t)(h * A_SUB), sb = stage_b(stage) + (uint32_t)(h * B_SUB);
                const uint64_t ad = A_MN ? sdesc_mnmajor_sw128(sa) : sdesc_kmajor_sw128(sa);
                const uint64_t bd = B_MN ? sdesc_mnmajor_sw128(sb) : sdesc_kmajor_sw128(sb);
#pragma unroll
                for (int k = 0; k < kFfnBK / 16; ++k) {
                  if constexpr (PAIR) umma_f16_pair(d_tmem, ad + AK * k, bd + BKS * k, idesc, acc);
                  else umma_f16(d_tmem, ad + AK * k, bd + BKS * k, idesc, acc);
                  acc = 1u;
                }
              }
              if constexpr (PAIR) umma_commit_pair(bar_empty(stage), 3);
              else umma_commit(bar_empty(stage));
              if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            if constexpr (PAIR) umma_commit_pair(bar_cfull(buf), 3);
            else umma_commit(bar_cfull(buf));
            if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            if (!CHUNKS || (kc = kend) >= kb1) break;
          }
          if (!ok) break;
        }
      };
      if (GATED || args.deal.first == 0) {
        issue_job(std::integral_constant<int, 0>{});
        if constexpr (!GATED) issue_job(std::integral_constant<int, 1>{});
      } else {
        issue_job(std::integral_constant<int, 1>{});
        issue_job(std::integral_constant<int, 0>{});
      }
      // every MMA this thread issued has finished before TMEM is released
      if constexpr (PAIR) umma_commit_pair(bar_drain, 1);
      else umma_commit(bar_drain);
      mbar_wait(bar_drain, 0u, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;   // TMEM lanes 32q .. 32q+31
    const int part = warp >> 2;
    // this warp's 32-column boxes of a tile: part, part + EPI_WARPS / 4, ...
    const int boxes = args.cols / 32;
    uint8_t* const stg0 = smem + L::OFF_STG + warp * STG * L::STG_BYTES;
    int sbox = 0;  // staging box to fill next
    int buf = 0;
    uint32_t buf_phase = 0;
    grid_dep_wait();
    if (!GATED && args.bias_grad.outputs > 0)
      // (16 x 32 x 9 FP32 over the staging boxes of all epilogue warps)
      ffn_bias_grad<DT>(args.bias_grad, reinterpret_cast<float*>(smem + L::OFF_STG), (int)blockIdx.x, (int)gridDim.x);
    const int tiles0 = sched.count(sched.first), tiles = tiles0 + (GATED ? 0 : sched.count(1 - sched.first));
    for (int ti = 0; ti < tiles; ++ti) {
      const int ji = ti < tiles0 ? sched.first : 1 - sched.first, t = sched.tile(ji, ti < tiles0 ? ti : ti - tiles0);
      const FfnJob& job = args.job[ji];
      const int M = job.M, N = job.N;
      const FfnTile tile(job, (uint32_t)t);
      const int s = tile.s, g = tile.g, nb = tile.nb;
      const int m0 = tile.mb * tile_rows + (int)rank * kFfnBM + q * 32, n0 = nb * args.cols;

      // The 32 x 32 box at (m0, nc) of output `o`, this lane's row given as
      // 16 packed pairs value(0) .. value(15), through the staging box: 64
      // bytes a row, chunk j at j ^ ((row >> 1) & 3) (TMA's 64-byte swizzle).
      auto store_box = [&](int o, int nc, auto&& value) {
        if (lane == 0) bulk_wait_group_read<STG - 1>();  // the box's last store has read it
        __syncwarp();
        uint8_t* const stg = stg0 + sbox * L::STG_BYTES;
        sbox = sbox + 1 == STG ? 0 : sbox + 1;
        uint8_t* rowp = stg + lane * 64;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(rowp + (j ^ ((lane >> 1) & 3)) * 16) =
              make_uint4(value(4 * j), value(4 * j + 1), value(4 * j + 2), value(4 * j + 3));
        if (job.tma_store) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&maps.y[ji][o], smem_addr(stg), nc, m0);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          uint16_t* const yo = o == 0 ? job.y[0] : (o == 1 ? job.y[1] : job.y[2]);
          const int rows = min(32, M - m0);
          // lane: column of the box; rows advance by pointer
          auto store_elements = [&] {
            if (nc + lane < N) {
              uint16_t* dst = yo + (size_t)m0 * N + nc + lane;
              const uint8_t* src = stg + (lane & 7) * 2;
#pragma unroll 8
              for (int rr = 0; rr < rows; ++rr, dst += N)
                *dst = *reinterpret_cast<const uint16_t*>(src + rr * 64 + (((lane >> 3) ^ ((rr >> 1) & 3)) << 4));
            }
          };
          if constexpr (GATED) {
            // words of E elements, E rows of one instruction; N is a multiple of E
            auto store_words = [&](auto word) {
              using W = decltype(word);
              constexpr int E = sizeof(W) / 2;
              const int c = lane % (32 / E) * E, r0 = lane / (32 / E);
              if (nc + c < N) {
                uint16_t* dst = yo + (size_t)(m0 + r0) * N + nc + c;
#pragma unroll 2
                for (int rr = r0; rr < rows; rr += E, dst += (size_t)E * N)
                  *reinterpret_cast<W*>(dst) =
                      *reinterpret_cast<const W*>(stg + rr * 64 + (((c >> 3) ^ ((rr >> 1) & 3)) << 4) + (c & 7) * 2);
              }
            };
            // The widest stores that every row's start allows: three outputs of 840 x 7772 x 288
            // take 19.8 us so, 26.0 in single elements. The gradients' one output a job gains
            // nothing, and the longer code costs that kernel registers (48.6 -> 51 us at 4648 x 4173 x 609).
            const uintptr_t align = reinterpret_cast<uintptr_t>(yo) | (uintptr_t)((uint32_t)N * 2u);
            if ((align & 7u) == 0) store_words(uint2{});
            else if ((align & 3u) == 0) store_words(uint32_t{});
            else store_elements();
          } else {
            store_elements();
          }
          __syncwarp();
        }
      };
      // a box of FP32 sums to the partial sums, as two 32 x 16 boxes (64 bytes
      // a row, the same swizzle)
      auto store_partial = [&](const uint32_t (&r)[32], int slab, int nc) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (lane == 0) bulk_wait_group_read<STG - 1>();
          __syncwarp();
          uint8_t* const stg = stg0 + sbox * L::STG_BYTES;
          sbox = sbox + 1 == STG ? 0 : sbox + 1;
          uint8_t* rowp = stg + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = 16 * h + 4 * j;
            *reinterpret_cast<uint4*>(rowp + (j ^ ((lane >> 1) & 3)) * 16) = make_uint4(r[c], r[c + 1], r[c + 2], r[c + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&maps.partial[ji], smem_addr(stg), nc + 16 * h, m0, slab);
            bulk_commit_group();
          }
        }
      };

      const int sum_kb = CHUNKS ? min(job.kb_split, job.kb_total - s * job.kb_split) : 0;
      const bool chunked = CHUNKS && sum_kb > ffn_chunk_kb(CL, DT);
      uint32_t taddr;
      auto wait_sums = [&] {
        const bool got = mbar_wait_long(bar_cfull(buf), buf_phase, abort_flag);
        if (!__all_sync(0xffffffffu, got)) return false;
        tc_fence_after_sync();
        taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kFfnMaxBN);
        return true;
      };
      const bool rows_in = m0 < M;  // warp-uniform
      // The scratch of accumulator columns 32 b .. 32 b + 31, this warp's rows: a
      // lane writes and reads its own row's 32 sums there.  (Gated: gate columns, then up.)
      auto scratch = [&](int b) {
        return args.scratch + (size_t)blockIdx.x * (kFfnScratchBytes / 16) + ((b * 4 + q) * 8) * 32 + lane;
      };
      // this warp is done with the accumulator: its sums are in registers
      auto release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) mbar_arrive_cluster(map_to_cta(bar_cempty(buf), 0u));
          else mbar_arrive(bar_cempty(buf));
        }
      };
      bool ok = true;
      if constexpr (CHUNKS) {
        // all chunks but the last: added up in the scratch
#pragma unroll 1
        for (int c = 0; c < (sum_kb - 1) / ffn_chunk_kb(CL, DT); ++c) {
          ok = wait_sums();
          if (!ok) break;
#pragma unroll 1
          for (int bx = part; bx < boxes && rows_in && n0 + bx * 32 < N; bx += EPI_WARPS / 4) {
#pragma unroll 1
            for (int b = bx; b < (GATED ? BN / 32 : bx + 1); b += BN / 64) {
              uint32_t r[32];
              tmem_ld_32x32b_x32(taddr + (uint32_t)(b * 32), r);
              tmem_ld_wait();
              if (c > 0) ffn_add_scratch(scratch(b), r);
              ffn_store_scratch(scratch(b), r);
            }
          }
          release();
          if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
        }
      }
      if (!ok || !wait_sums()) break;
      bool held = true;
#pragma unroll 1
      for (int bx = part; bx < boxes; bx += EPI_WARPS / 4) {
        const int nc = n0 + bx * 32;
        if (nc >= N || !rows_in) break;  // warp-uniform: nothing of the box is in the output
        uint32_t r[32];
        tmem_ld_32x32b_x32(taddr + (uint32_t)(bx * 32), r);
        if constexpr (GATED) {
          uint32_t r2[32];
          tmem_ld_32x32b_x32(taddr + (uint32_t)(BN / 2 + bx * 32), r2);
          const bool biased = args.bias[0] != nullptr || args.bias[1] != nullptr;
          uint16_t* const sbias = reinterpret_cast<uint16_t*>(smem + L::OFF_BIAS) + (buf * 4 + bx) * 64;
          if (biased && job.split == 1) {
            // lane l fetches the biases of column nc + l.  The four warps of a
            // box write the same values; the slot is this accumulator's, whose
            // next tile starts only after all warps have released it.
            const int col = nc + lane;
            sbias[lane] = (args.bias[0] != nullptr && col < N) ? __ldg(args.bias[0] + col) : (uint16_t)0;
            sbias[32 + lane] = (args.bias[1] != nullptr && col < N) ? __ldg(args.bias[1] + col) : (uint16_t)0;
            __syncwarp();
          }
          tmem_ld_wait();
          if (chunked) {
            ffn_add_scratch(scratch(bx), r);
            ffn_add_scratch(scratch(BN / 64 + bx), r2);
          }
          const bool last_box = bx + EPI_WARPS / 4 >= boxes;
          if (job.split > 1) {
            if (last_box) release();
            held = !last_box;
            store_partial(r, s, nc);
            store_partial(r2, job.split + s, nc);
            continue;
          }
          if (biased) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float gv[8], uv[8];
              ffn_unpack8<DT>(reinterpret_cast<const uint4*>(sbias)[j], gv);
              ffn_unpack8<DT>(reinterpret_cast<const uint4*>(sbias)[4 + j], uv);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                r[8 * j + k] = __float_as_uint(__uint_as_float(r[8 * j + k]) + gv[k]);
                r2[8 * j + k] = __float_as_uint(__uint_as_float(r2[8 * j + k]) + uv[k]);
              }
            }
          }
          // (after the biases: their slot is the accumulator's)
          if (last_box) release();
          held = !last_box;
          if (args.save) {
            store_box(1, nc, [&](int i) { return ep_pack_t<DT>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])); });
            store_box(2, nc, [&](int i) { return ep_pack_t<DT>(__uint_as_float(r2[2 * i]), __uint_as_float(r2[2 * i + 1])); });
          }
          auto gate = [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            store_box(0, nc, [&](int i) {
              return ep_pack_t<DT>(act_value_t<ACT, DT>(__uint_as_float(r[2 * i])) * __uint_as_float(r2[2 * i]),
                                   act_value_t<ACT, DT>(__uint_as_float(r[2 * i + 1])) * __uint_as_float(r2[2 * i + 1]));
            });
          };
          if (args.act == kActSilu) gate(std::integral_constant<int, kActSilu>{});
          else if (args.act == kActGeluTanh) gate(std::integral_constant<int, kActGeluTanh>{});
          else gate(std::integral_constant<int, kActGeluErf>{});
        } else {
          tmem_ld_wait();
          if (chunked) ffn_add_scratch(scratch(bx), r);
          if (bx + EPI_WARPS / 4 >= boxes) {
            release();
            held = false;
          }
          if (job.split > 1) store_partial(r, g * job.split + s, nc);
          else
            store_box(g, nc, [&](int i) { return ep_pack_t<DT>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])); });
        }
      }
      if (held) release();
      if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
    }
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  if (warp == MMA_WARP) {
    tc_fence_after_sync();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, kFfnTmemCols);
    else tmem_dealloc(tmem_base, kFfnTmemCols);
  }
}

}  // namespace poot
