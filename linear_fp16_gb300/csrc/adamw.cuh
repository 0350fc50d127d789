// An AdamW step over a list of tensors, in one pass:
//
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every operation is FP32, rounded on its own in the order written (no fused
// multiply-adds), so a step gives the same bits whatever kernel, list or device
// computes it: what 8-bit codes need, whose neighbours lie percents apart.
//
// States in 8 bits: blocks of 256 consecutive elements of a tensor with one FP32
// scale s each.
//   m       = s c |c|,  c in -127 .. 127    s = max |m| / 127^2
//   sqrt(v) = s c^2,    c in 0 .. 255       s = max sqrt(v) / 255^2
// The codes are nearest in c.  Squares give small values of a block finer steps
// than a linear code: the smallest nonzero one is 6e-5 (m) and 1.5e-5 (sqrt v) of
// the block's largest.  A nonzero sqrt(v) keeps a code of at least 1: as 0 it would leave
// eps alone to divide m.
//
// A warp takes 256 elements at a time, eight a lane, so that a block's maxima are
// two warp reductions.  Bound by HBM: bfloat16 parameters and gradients move 22
// bytes an element with states in FP32, 10 with states in 8 bits.
#pragma once

#include <cmath>

#include "clip.cuh"

namespace poot {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamBlock = 256;     // elements of a scale, and of a warp's turn
constexpr int kAdamTable = 384;     // tensors of one launch
constexpr int kAdamTableFew = 48;   // short lists: less to pass to the launch

template <int T>
struct AdamTable {
  void* p[T];
  const void* g[T];
  void* m[T];
  void* v[T];
  float* ms[T];
  float* vs[T];
  void* copy[T];
  long long n[T];
  long long first[T + 1];  // first chunk of 256 elements of each tensor
  float decay[T];          // 1 - lr wd; with lr on the device wd
  unsigned char types[T];  // GradDtype of p, g << 2, copy << 4; kAdamVec
  int count;
};
constexpr int kAdamVec = 64;  // every pointer is on a boundary of four elements

struct AdamArgs {
  // read on the device where not nullptr
  const float* lr_dev;
  const long long* step_dev;
  const float* grad_scale_dev;
  double lr, log_b1, log_b2;
  long long step;
  float b1, omb1, b2, omb2, eps, grad_scale;
  float minus_zero;             // -0, unknown to the compiler: see adam_product
  float step_size, root_scale;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};

// Eight elements of a lane: two fours 128 apart (VEC), or every 32nd; `n` of the
// chunk's 256 exist, the others are zero.
template <int DT, bool VEC>
struct AdamLoad {
  uint32_t w[DT == kGradF32 ? 8 : 4];
  __device__ __forceinline__ void load(const void* base, long long e0, int n, int lane) {
    if constexpr (VEC && DT == kGradF32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + e0) + lane;
      const uint4 a = p[0], b = p[32];
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else if constexpr (VEC) {
      const uint2* p = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + e0) + lane;
      const uint2 a = p[0], b = p[32];
      w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
    } else if constexpr (DT == kGradF32) {
      const uint32_t* p = static_cast<const uint32_t*>(base) + e0;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j * 32 + lane < n ? p[j * 32 + lane] : 0u;
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(base) + e0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int a = j * 64 + lane, b = a + 32;
        w[j] = (a < n ? (uint32_t)p[a] : 0u) | (b < n ? (uint32_t)p[b] << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (DT == kGradF32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = ep_unpack_t<DT>(w[j]);
        f[2 * j] = a.x;
        f[2 * j + 1] = a.y;
      }
    }
  }
};

template <int DT, bool VEC>
__device__ __forceinline__ void adam_store(void* base, long long e0, int n, int lane, const float (&f)[8]) {
  if constexpr (VEC && DT == kGradF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + e0) + lane;
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[32] = make_float4(f[4], f[5], f[6], f[7]);
  } else if constexpr (VEC) {
    uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + e0) + lane;
    p[0] = make_uint2(ep_pack_t<DT>(f[0], f[1]), ep_pack_t<DT>(f[2], f[3]));
    p[32] = make_uint2(ep_pack_t<DT>(f[4], f[5]), ep_pack_t<DT>(f[6], f[7]));
  } else {
    using E = GradElem<DT>;
    typename E::type* p = static_cast<typename E::type*>(base) + e0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * 32 + lane < n) p[j * 32 + lane] = E::round(f[j]);
  }
}

// ---- codes -------------------------------------------------------------------
template <bool VEC>
struct AdamCodes {
  uint32_t w[2];  // byte j & 3 of word j >> 2
  __device__ __forceinline__ void load(const void* base, long long e0, int n, int lane) {
    const unsigned char* p = static_cast<const unsigned char*>(base) + e0;
    if constexpr (VEC) {
      w[0] = reinterpret_cast<const uint32_t*>(p)[lane];
      w[1] = reinterpret_cast<const uint32_t*>(p)[32 + lane];
    } else {
      w[0] = w[1] = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 32 + lane < n) w[j >> 2] |= (uint32_t)p[j * 32 + lane] << (8 * (j & 3));
    }
  }
  __device__ __forceinline__ void store(void* base, long long e0, int n, int lane) const {
    unsigned char* p = static_cast<unsigned char*>(base) + e0;
    if constexpr (VEC) {
      reinterpret_cast<uint32_t*>(p)[lane] = w[0];
      reinterpret_cast<uint32_t*>(p)[32 + lane] = w[1];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 32 + lane < n) p[j * 32 + lane] = (unsigned char)(w[j >> 2] >> (8 * (j & 3)));
    }
  }
};

// Two FP32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 adam_add(float2 a, float2 b) {
  add_f32x2(a.x, a.y, b.x, b.y);
  return a;
}
__device__ __forceinline__ float2 adam_mul(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 s, t;\n\t"
      "mov.b64 s, {%2, %3};\n\t"
      "mov.b64 t, {%4, %5};\n\t"
      "mul.rn.f32x2 s, s, t;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 adam_fma(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 s, t, u;\n\t"
      "mov.b64 s, {%2, %3};\n\t"
      "mov.b64 t, {%4, %5};\n\t"
      "mov.b64 u, {%6, %7};\n\t"
      "fma.rn.f32x2 s, s, t, u;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 adam_both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 adam_neg(float2 v) { return make_float2(-v.x, -v.y); }

// Bytes j and j + 1 of a word as floats: in the low bits of 2^23's, which is then
// taken off (conversions run at an eighth of the rate).
__device__ __forceinline__ float2 adam_bytes(uint32_t w, int j, float off) {
  const float2 t = make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | (j & 3))),
                               __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | ((j & 3) + 1))));
  return adam_add(t, adam_both(off));
}
// w ^ 0x80808080: c + 128 in 0 .. 255
__device__ __forceinline__ float2 adam_m(uint32_t w, int j, float scale) {
  const float2 c = adam_bytes(w ^ 0x80808080u, j, -8388736.0f);
  // (c |c| is exact)
  return adam_mul(adam_both(scale), make_float2(__fmul_rn(c.x, fabsf(c.x)), __fmul_rn(c.y, fabsf(c.y))));
}
__device__ __forceinline__ float2 adam_root(uint32_t w, int j, float scale) {
  const float2 c = adam_bytes(w, j, -8388608.0f);
  return adam_mul(adam_both(scale), adam_mul(c, c));
}

// The scale of a block whose largest value has the bits `most` (as integers, those of
// absolute values order like the values, infinities and NaN above), and what
// turns a value into the square of its code.  A block that is not finite gets
// the scale NaN, and so reads as NaN throughout.
struct AdamScale {
  float scale, inverse;
};
template <int TOP>
__device__ __forceinline__ AdamScale adam_scale(uint32_t most) {
  constexpr float kSquare = TOP * TOP, kPart = 1.0 / (TOP * TOP);
  const float f = __uint_as_float(most);
  if (most >= 0x7f800000u) return {NAN, 0.0f};
  // (below 2^-110, where the inverse would overflow, a block counts as zero; sqrt(v) is above 2^-75 or zero)
  if (f < 7.703719777548943e-34f) return {0.0f, 0.0f};
  return {__fmul_rn(f, kPart), __fmul_rn(__frcp_rn(f), kSquare)};
}

// Two integers c nearest to sqrt(y), y in 0 .. 255^2 (1 + 2^-22): c + 1 from y > (c + 1/2)^2 on.
// The square root is approximate; taken 2^-10 low, its rounding is the result or
// one less, and the comparison, exact in FP32, decides.
__device__ __forceinline__ uint2 adam_code(float2 y) {
  float2 s;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(y.x));
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(y.y));
  // 2^23: the sum's low bits are the rounded value
  const float2 t = adam_add(adam_add(s, adam_both(-0.0009765625f)), adam_both(8388608.0f));
  const float2 c = adam_add(t, adam_both(-8388608.0f));
  const float2 edge = adam_add(adam_fma(c, c, c), adam_both(0.25f));
  return make_uint2((__float_as_uint(t.x) & 0xffu) + (y.x > edge.x ? 1u : 0u),
                    (__float_as_uint(t.y) & 0xffu) + (y.y > edge.y ? 1u : 0u));
}

struct AdamHyper {
  float b1, omb1, b2, omb2, eps, grad_scale, step_size, root_scale, lr, minus_zero;
};

// a b rounded, for a sum: the assembler fuses a packed product with the addition behind it, .rn or
// not, but not a product that is one already (adding -0 changes nothing).
__device__ __forceinline__ float2 adam_product(const AdamHyper& h, float2 a, float b) {
  return adam_fma(a, adam_both(b), adam_both(h.minus_zero));
}

// sqrt(v) correctly rounded, for v of 2^-100 .. 2^100: from an approximate 1 /
// sqrt(v) one coupled Newton step for sqrt and half its reciprocal, then the
// remainder v - g^2, exact in an FMA, added back (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).
__device__ __forceinline__ float2 adam_sqrt(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(v.x));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(v.y));
  float2 g = adam_mul(v, y), h = adam_mul(y, adam_both(0.5f));
  const float2 e = adam_fma(adam_neg(h), g, adam_both(0.5f));
  g = adam_fma(g, e, g);
  h = adam_fma(h, e, h);
  return adam_fma(adam_fma(adam_neg(g), g, v), h, g);
}

// m / d rounded to nearest likewise, for d of 2^-60 .. 2^60 and m of 2^-75 or more (below, the
// remainder may be subnormal and the last place off by one).
__device__ __forceinline__ float2 adam_div(float2 m, float2 d) {
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  const float2 n = adam_neg(d);
  r = adam_fma(adam_fma(n, r, adam_both(1.0f)), r, r);
  const float2 q = adam_mul(m, r);
  return adam_fma(adam_fma(n, q, m), r, q);
}

// A lane's eight elements: m and v updated, sqrt(v) and the new p.  All 32 lanes call it.
__device__ __forceinline__ void adam_update(const AdamHyper& h, float decay, const float (&gs)[8], float (&p)[8],
                                            float (&m)[8], float (&v)[8], float (&root)[8]) {
  float lo = INFINITY, hi = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 g = adam_mul(make_float2(gs[j], gs[j + 1]), adam_both(h.grad_scale));
    const float2 a = adam_add(adam_product(h, make_float2(m[j], m[j + 1]), h.b1), adam_product(h, g, h.omb1));
    const float2 b = adam_add(adam_product(h, make_float2(v[j], v[j + 1]), h.b2),
                              adam_product(h, adam_mul(g, g), h.omb2));
    m[j] = a.x;
    m[j + 1] = a.y;
    v[j] = b.x;
    v[j + 1] = b.y;
    lo = fminf(lo, fminf(b.x, b.y));
    hi = fmaxf(hi, fmaxf(b.x, b.y));
  }
  // (NaN comes through either way.  Zeros, of elements that have had no gradient yet, take the second.)
  const bool plain = lo >= 7.888609052210118e-31f && hi <= 1.2676506002282294e30f && h.eps <= 1e15f;
  if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 r = adam_sqrt(make_float2(v[j], v[j + 1]));
      const float2 d = adam_add(adam_product(h, r, h.root_scale), adam_both(h.eps));
      const float2 q = adam_div(make_float2(m[j], m[j + 1]), d);
      const float2 n = adam_add(adam_product(h, make_float2(p[j], p[j + 1]), decay), adam_product(h, q, -h.step_size));
      root[j] = r.x;
      root[j + 1] = r.y;
      p[j] = n.x;
      p[j + 1] = n.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      root[j] = __fsqrt_rn(v[j]);
      const float q = __fdiv_rn(m[j], __fadd_rn(__fmul_rn(root[j], h.root_scale), h.eps));
      p[j] = __fsub_rn(__fmul_rn(p[j], decay), __fmul_rn(q, h.step_size));
    }
  }
}

// NaN where either is
__device__ __forceinline__ float adam_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct AdamTensor {
  void* p;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  void* copy;
  long long n;
  float decay;
  int copy_dtype;
};

// 256 elements from e0 on (`n` of them exist).
template <int PD, int GD, int BITS, bool VEC>
__device__ __forceinline__ void adam_chunk(const AdamTensor& t, const AdamHyper& h, long long e0, int n, int lane) {
  AdamLoad<PD, VEC> lp;
  AdamLoad<GD, VEC> lg;
  lg.load(t.g, e0, n, lane);
  lp.load(t.p, e0, n, lane);
  float p[8], g[8], m[8], v[8], root[8];
  if constexpr (BITS == 32) {
    AdamLoad<kGradF32, VEC> lm, lv;
    lm.load(t.m, e0, n, lane);
    lv.load(t.v, e0, n, lane);
    lg.get(g);
    lp.get(p);
    lm.get(m);
    lv.get(v);
    adam_update(h, t.decay, g, p, m, v, root);
    adam_store<kGradF32, VEC>(t.m, e0, n, lane, m);
    adam_store<kGradF32, VEC>(t.v, e0, n, lane, v);
  } else {
    AdamCodes<VEC> cm, cv;
    cm.load(t.m, e0, n, lane);
    cv.load(t.v, e0, n, lane);
    const long long block = e0 / kAdamBlock;
    const float ms = t.ms[block], vs = t.vs[block];
    lg.get(g);
    lp.get(p);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 a = adam_m(cm.w[j >> 2], j, ms), r = adam_root(cv.w[j >> 2], j, vs), b = adam_mul(r, r);
      m[j] = a.x;
      m[j + 1] = a.y;
      v[j] = b.x;
      v[j + 1] = b.y;
    }
    adam_update(h, t.decay, g, p, m, v, root);
    float most_m = 0.0f, most_r = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      most_m = adam_max(most_m, fabsf(m[j]));
      most_r = adam_max(most_r, root[j]);
    }
    // (elements that do not exist are zeros times the scale: NaN in a block that was not finite, as it stays)
    const AdamScale sm = adam_scale<127>(__reduce_max_sync(0xffffffffu, __float_as_uint(most_m)));
    const AdamScale sv = adam_scale<255>(__reduce_max_sync(0xffffffffu, __float_as_uint(most_r)));
    cm.w[0] = cm.w[1] = cv.w[0] = cv.w[1] = 0u;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint2 c = adam_code(adam_mul(make_float2(fabsf(m[j]), fabsf(m[j + 1])), adam_both(sm.inverse)));
      const uint2 k = adam_code(adam_mul(make_float2(root[j], root[j + 1]), adam_both(sv.inverse)));
      const uint32_t c0 = m[j] < 0.0f ? 0u - c.x : c.x, c1 = m[j + 1] < 0.0f ? 0u - c.y : c.y;
      const uint32_t k0 = root[j] > 0.0f ? max(k.x, 1u) : k.x, k1 = root[j + 1] > 0.0f ? max(k.y, 1u) : k.y;
      // bytes 0 of four words
      cm.w[j >> 2] |= __byte_perm(c0, c1, (j & 2) ? 0x4000 : 0x0040) & ((j & 2) ? 0xffff0000u : 0xffffu);
      cv.w[j >> 2] |= __byte_perm(k0, k1, (j & 2) ? 0x4000 : 0x0040) & ((j & 2) ? 0xffff0000u : 0xffffu);
    }
    cm.store(t.m, e0, n, lane);
    cv.store(t.v, e0, n, lane);
    if (lane == 0) {
      t.ms[block] = sm.scale;
      t.vs[block] = sv.scale;
    }
  }
  adam_store<PD, VEC>(t.p, e0, n, lane, p);
  if (PD == kGradF32 && t.copy != nullptr) {
    if (t.copy_dtype == kGradF16) adam_store<kGradF16, VEC>(t.copy, e0, n, lane, p);
    else adam_store<kGradBf16, VEC>(t.copy, e0, n, lane, p);
  }
}

template <int BITS, bool VEC>
__device__ __forceinline__ void adam_dispatch(int types, const AdamTensor& t, const AdamHyper& h, long long e0, int n,
                                              int lane) {
  switch (types & 15) {
    case kGradF16 | kGradF16 << 2: return adam_chunk<kGradF16, kGradF16, BITS, VEC>(t, h, e0, n, lane);
    case kGradF16 | kGradBf16 << 2: return adam_chunk<kGradF16, kGradBf16, BITS, VEC>(t, h, e0, n, lane);
    case kGradF16 | kGradF32 << 2: return adam_chunk<kGradF16, kGradF32, BITS, VEC>(t, h, e0, n, lane);
    case kGradBf16 | kGradF16 << 2: return adam_chunk<kGradBf16, kGradF16, BITS, VEC>(t, h, e0, n, lane);
    case kGradBf16 | kGradBf16 << 2: return adam_chunk<kGradBf16, kGradBf16, BITS, VEC>(t, h, e0, n, lane);
    case kGradBf16 | kGradF32 << 2: return adam_chunk<kGradBf16, kGradF32, BITS, VEC>(t, h, e0, n, lane);
    case kGradF32 | kGradF16 << 2: return adam_chunk<kGradF32, kGradF16, BITS, VEC>(t, h, e0, n, lane);
    case kGradF32 | kGradBf16 << 2: return adam_chunk<kGradF32, kGradBf16, BITS, VEC>(t, h, e0, n, lane);
    default: return adam_chunk<kGradF32, kGradF32, BITS, VEC>(t, h, e0, n, lane);
  }
}

// The factors of a step, in 64 bits: 1 - b^t = -expm1(t log b).
__host__ __device__ inline void adam_factors(double lr, double log_b1, double log_b2, double t, float* step_size,
                                             float* root_scale) {
  *step_size = (float)(lr / -expm1(t * log_b1));
  *root_scale = (float)(1.0 / sqrt(-expm1(t * log_b2)));
}

// The tensor of chunk c.
template <int T>
__device__ __forceinline__ int adam_find(const long long (&first)[T], int count, long long c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A block has consecutive chunks of all tensors', dealt out in equal shares, and its
// warps take them in turn.
template <int T, int BITS>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamTable<T> t, const AdamArgs a) {
  __shared__ AdamHyper shared;
  grid_dep_wait();
  grid_dep_launch();
  AdamHyper h{a.b1, a.omb1, a.b2, a.omb2, a.eps, a.grad_scale, a.step_size, a.root_scale, 0.0f, a.minus_zero};
  if (a.lr_dev != nullptr || a.step_dev != nullptr || a.grad_scale_dev != nullptr) {
    if (threadIdx.x == 0) {
      const double lr = a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr;
      adam_factors(lr, a.log_b1, a.log_b2, (double)(a.step_dev != nullptr ? *a.step_dev : a.step), &h.step_size,
                   &h.root_scale);
      if (a.grad_scale_dev != nullptr) h.grad_scale = *a.grad_scale_dev;
      h.lr = (float)lr;
      shared = h;
    }
    __syncthreads();
    h = shared;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long chunks = t.first[t.count];
  const long long c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
  int k = adam_find(t.first, t.count, c0);
  for (long long c = c0 + warp; c < c1; c += kAdamWarps) {
    while (c >= t.first[k + 1]) ++k;
    AdamTensor x;
    x.p = t.p[k];
    x.g = t.g[k];
    x.m = t.m[k];
    x.v = t.v[k];
    x.ms = t.ms[k];
    x.vs = t.vs[k];
    x.copy = t.copy[k];
    x.n = t.n[k];
    x.decay = a.lr_dev != nullptr ? fmaf(-h.lr, t.decay[k], 1.0f) : t.decay[k];
    const int types = t.types[k];
    x.copy_dtype = (types >> 4) & 3;
    const long long e0 = (c - t.first[k]) * kAdamBlock;
    const long long left = x.n - e0;
    if ((types & kAdamVec) && left >= kAdamBlock) adam_dispatch<BITS, true>(types, x, h, e0, kAdamBlock, lane);
    else adam_dispatch<BITS, false>(types, x, h, e0, (int)min(left, (long long)kAdamBlock), lane);
  }
}

// ---- the values that 8-bit states stand for ----------------------------------------
template <int T>
struct AdamValueTable {
  const void* m[T];
  const void* v[T];
  const float* ms[T];
  const float* vs[T];
  float* mo[T];
  float* vo[T];
  long long n[T];
  long long first[T + 1];
  unsigned char vec[T];
  int count;
};

template <bool VEC>
__device__ __forceinline__ void adam_expand(const void* m, const void* v, float ms, float vs, float* mo, float* vo,
                                            long long e0, int n, int lane) {
  AdamCodes<VEC> cm, cv;
  cm.load(m, e0, n, lane);
  cv.load(v, e0, n, lane);
  float fm[8], fv[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 a = adam_m(cm.w[j >> 2], j, ms), r = adam_root(cv.w[j >> 2], j, vs), b = adam_mul(r, r);
    fm[j] = a.x;
    fm[j + 1] = a.y;
    fv[j] = b.x;
    fv[j + 1] = b.y;
  }
  adam_store<kGradF32, VEC>(mo, e0, n, lane, fm);
  adam_store<kGradF32, VEC>(vo, e0, n, lane, fv);
}

template <int T>
__global__ void __launch_bounds__(kAdamThreads) adamw_values_kernel(const __grid_constant__ AdamValueTable<T> t) {
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long chunks = t.first[t.count];
  const long long c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
  int k = adam_find(t.first, t.count, c0);
  for (long long c = c0 + warp; c < c1; c += kAdamWarps) {
    while (c >= t.first[k + 1]) ++k;
    const long long block = c - t.first[k], e0 = block * kAdamBlock, left = t.n[k] - e0;
    const float ms = t.ms[k][block], vs = t.vs[k][block];
    if (t.vec[k] && left >= kAdamBlock)
      adam_expand<true>(t.m[k], t.v[k], ms, vs, t.mo[k], t.vo[k], e0, kAdamBlock, lane);
    else
      adam_expand<false>(t.m[k], t.v[k], ms, vs, t.mo[k], t.vo[k], e0, (int)min(left, (long long)kAdamBlock), lane);
  }
}

}  // namespace poot
