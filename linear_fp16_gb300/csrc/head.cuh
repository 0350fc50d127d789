// The rows of a vocabulary head: softmax cross entropy and its gradient on the
// logits z = x W^T + b of a tile, in registers (a lane has a row).
//
//   loss_i = lse_i - z_i,t(i),  lse_i = log sum_v exp z_iv
//   q_iv   = dloss_i (exp(z_iv - lse_i) - [v = t(i)])
//
// Exponentials are taken in base 2: with m = max z log2(e), rounded once, a tile's
// sum is sum 2^(z log2(e) - m) (one fused multiply-add and one ex2 an element),
// and (m, sum) pairs join without another rounding of m.  ex2 is within 2 ulp.
#pragma once

#include <cmath>

#include "epilogue.cuh"
#include "ptx.cuh"

namespace poot {

constexpr float kHeadLog2e = 1.4426950408889634f;
constexpr float kHeadLn2 = 0.6931471805599453f;
constexpr int kHeadChunkK = 1024;  // terms of a logit summed in TMEM (lse)
constexpr int kHeadParts = 4;      // (maximum, sum) pairs of a row and tile: one for each warp on it

struct HeadArgs {
  const uint16_t* bias;      // of the launch's first column, or nullptr
  const long long* target;   // [M]
  long long ignore;
  int vocab;                 // all columns
  int col0;                  // the launch's first
  // lse
  float2* partial;           // [tile along V][kHeadParts][M]: maximum times log2(e), sum
  float* picked;             // [M]: the target's logit
  // dz
  const float* lse;          // [M]
  const float* dloss;        // [M], elements dloss_stride apart
  long long dloss_stride;
  float* sums;               // [row blocks of 32][pitch]: column sums of q, or nullptr
  int sums_pitch;            // the launch's columns rounded up to 8
  const float* scale;        // dz: scale[0] goes into q; scaled: scale[1] takes it out
  // scaled
  int sum_dx;                // dx is stored as FP32 sums
  int accumulate;            // and added to those of earlier launches
};

// The column among all of a row with target t, or -1 (ignored, or outside the vocabulary).
__device__ __forceinline__ int head_target(const HeadArgs& h, long long t) {
  return t != h.ignore && t >= 0 && t < h.vocab ? (int)t : -1;
}

__device__ __forceinline__ float head_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// z += 32 columns' biases in shared memory
__device__ __forceinline__ void head_add(float (&z)[32], const float* bias) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 v = reinterpret_cast<const float4*>(bias)[j];
    z[4 * j] += v.x;
    z[4 * j + 1] += v.y;
    z[4 * j + 2] += v.z;
    z[4 * j + 3] += v.w;
  }
}

// Writes z[d] of the lanes whose d is in 0 .. 31.
__device__ __forceinline__ void head_pick(const float (&z)[32], int d, float* out, int row) {
  const bool here = (unsigned)d < 32u;
  if (!__any_sync(0xffffffffu, here)) return;
  float v = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) v = j == d ? z[j] : v;
  if (here) out[row] = v;
}

// What a sum's exponents are taken relative to: the maximum, or 0 where that is
// infinite (the sum is then 0, infinite or NaN, as the formula's).
__device__ __forceinline__ float head_base(float top2) { return fabsf(top2) <= 3.402823466e38f ? top2 : 0.0f; }

__device__ __forceinline__ float head_exp_sum(const float (&z)[32], float base) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 32; ++j) s[j & 3] += head_exp2(fmaf(z[j], kHeadLog2e, -base));
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// (m, s) of two sets of logits joined: m the larger maximum, s relative to it.
// An infinite maximum takes the sums that have it (+inf: infinite or NaN).
__device__ __forceinline__ float2 head_join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float base = head_base(m);
  // (a side without finite logits: 2^-inf = 0 times its sum of 0, or NaN)
  const float fa = a.x == m ? 1.0f : head_exp2(a.x - base), fb = b.x == m ? 1.0f : head_exp2(b.x - base);
  return make_float2(m, a.y * fa + b.y * fb);
}

// dz: what a row needs.  p is computed 2^14 times too large, which keeps it
// down to 2^-140 (ex2 drops subnormal results; bfloat16 reaches 2^-133).
constexpr float kHeadLift = 14.0f, kHeadLiftScale = 16384.0f;
struct HeadRow {
  float lse2, scale;  // of the lifted p
  int target;
  bool used;
};
// As it is loaded, a tile ahead: nothing waits for the values before their tile.
struct HeadRowRaw {
  long long target;
  float lse, dloss;
};
__device__ __forceinline__ HeadRowRaw head_row_load(const HeadArgs& h, int row, int rows) {
  HeadRowRaw r{h.ignore, 0.0f, 0.0f};
  if (row < rows) {
    r.target = __ldg(h.target + row);
    r.lse = __ldg(h.lse + row);
    r.dloss = __ldg(h.dloss + row * h.dloss_stride);
  }
  return r;
}
__device__ __forceinline__ HeadRow head_row(const HeadArgs& h, const HeadRowRaw& raw, float scale) {
  HeadRow r;
  r.used = raw.target != h.ignore;
  r.lse2 = fmaf(raw.lse, kHeadLog2e, -kHeadLift);
  const bool inside = raw.target >= 0 && raw.target < h.vocab;
  r.scale = inside ? raw.dloss * (scale / kHeadLiftScale) : NAN;
  r.target = inside && r.used ? (int)raw.target - h.col0 : -1;
  return r;
}

// r: 32 logits of the launch's columns nc .. -> q, times the scale.
__device__ __forceinline__ void head_gradient(uint32_t (&r)[32], const HeadRow& h, int nc) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float p = head_exp2(fmaf(__uint_as_float(r[j]), kHeadLog2e, -h.lse2)) * h.scale;
    r[j] = h.used ? __float_as_uint(p) : 0u;
  }
  const int d = h.target - nc;
  if (!__any_sync(0xffffffffu, (unsigned)d < 32u)) return;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j == d) r[j] = __float_as_uint(__uint_as_float(r[j]) - h.scale * kHeadLiftScale);
}

// Sums over the warp's rows of 32 columns: lane l gets column l's.  Each step halves
// the columns of a lane and adds the other half's of the lane opposite.  FP32, in a fixed order.
__device__ __forceinline__ float head_column_sum(uint32_t (&r)[32], int lane) {
#pragma unroll
  for (int off = 16; off > 0; off /= 2) {
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const uint32_t keep = upper ? r[i + off] : r[i], send = upper ? r[i] : r[i + off];
      r[i] = __float_as_uint(__uint_as_float(keep) + __uint_as_float(__shfl_xor_sync(0xffffffffu, send, off)));
    }
  }
  return __uint_as_float(r[0]);
}

}  // namespace poot
