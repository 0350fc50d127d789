// The memory-bound steps around the feed-forward products: the gate's
// gradient, column sums (bias gradients), the second half of a split-K
// product, row repacking for operands TMA cannot read in place.
#pragma once

#include "ffn_gemm.cuh"
#include "pack.cuh"

namespace poot {

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

constexpr int kColThreads = 256;
constexpr int kColWidth = 256;  // columns of a block: 32 lanes x 8
constexpr int kColRows = 64;    // rows of a block: 8 warps x 8

struct GateGradArgs {
  const uint16_t *dh, *g, *u;
  long long ld_dh, ld_g, ld_u;
  uint16_t *dg, *du;  // row pitch ldo, 16-byte aligned rows
  long long ldo;
  float* colsum;      // [row blocks][2][N] FP32, or nullptr
  int M, N, act;
};

// dg = dh u act'(g), du = dh act(g), in FP32, each rounded once to the head
// dtype: they are operands of the tensor core, which takes 16-bit values.
// The bias gradients sum the unrounded values.  A block covers 64 rows x 256
// columns, a lane eight columns of eight rows; column sums go through
// registers, then shared memory, in a fixed order.  Bound by its five
// streams (three read, two written).
template <int DT, bool SUMS>
__global__ void __launch_bounds__(kColThreads) gate_grad_kernel(const GateGradArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned cblocks = (a.N + kColWidth - 1) / kColWidth;
  const int cb = blockIdx.x % cblocks, rb = blockIdx.x / cblocks;
  const int c = cb * kColWidth + lane * 8;
  const int n = min(8, a.N - c);  // columns of this lane (<= 0: none)
  const long long row0 = (long long)rb * kColRows + warp;
  float sg[8], su[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sg[j] = su[j] = 0.0f;
  grid_dep_wait();
  grid_dep_launch();
  if (n > 0) {
#pragma unroll 2
    for (int i = 0; i < kColRows / 8; ++i) {
      const long long row = row0 + i * 8;
      if (row >= a.M) break;
      float dh[8], g[8], u[8], dg[8], du[8];
      ffn_unpack8<DT>(ffn_load8(a.dh + row * a.ld_dh + c, n), dh);
      ffn_unpack8<DT>(ffn_load8(a.g + row * a.ld_g + c, n), g);
      ffn_unpack8<DT>(ffn_load8(a.u + row * a.ld_u + c, n), u);
      auto grad = [&](auto act) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v, d;
          act_both_t<decltype(act)::value>(g[j], v, d);
          dg[j] = dh[j] * u[j] * d;
          du[j] = dh[j] * v;
        }
      };
      if (a.act == kActSilu) grad(std::integral_constant<int, kActSilu>{});
      else if (a.act == kActGeluTanh) grad(std::integral_constant<int, kActGeluTanh>{});
      else grad(std::integral_constant<int, kActGeluErf>{});
      if constexpr (SUMS) {
#pragma unroll
        for (int j = 0; j < 8; ++j) { sg[j] += dg[j]; su[j] += du[j]; }
      }
      // whole chunks: the rows' pad columns may be written (never read)
      *reinterpret_cast<uint4*>(a.dg + row * a.ldo + c) = ffn_pack8<DT>(dg);
      *reinterpret_cast<uint4*>(a.du + row * a.ldo + c) = ffn_pack8<DT>(du);
    }
  }
  if constexpr (SUMS) {
    __shared__ float red[8][kColWidth];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) red[warp][lane * 8 + j] = o ? su[j] : sg[j];
      __syncthreads();
      const int col = cb * kColWidth + threadIdx.x;
      if (col < a.N) {
        float s = red[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < 8; ++w) s += red[w][threadIdx.x];
        a.colsum[((size_t)rb * 2 + o) * a.N + col] = s;
      }
    }
  }
}

struct ColSumArgs {
  const uint16_t* d;
  long long ld;
  float* colsum;  // [row blocks][N]
  int M, N;
};

// FP32 column sums of D [M, N] over blocks of 64 rows.
template <int DT>
__global__ void __launch_bounds__(kColThreads) col_sum_kernel(const ColSumArgs a) {
  __shared__ float red[8][kColWidth];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned cblocks = (a.N + kColWidth - 1) / kColWidth;
  const int cb = blockIdx.x % cblocks, rb = blockIdx.x / cblocks;
  const int c = cb * kColWidth + lane * 8;
  const int n = min(8, a.N - c);
  const long long row0 = (long long)rb * kColRows + warp;
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.0f;
  grid_dep_wait();
  grid_dep_launch();
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < kColRows / 8; ++i) {
      const long long row = row0 + i * 8;
      if (row < a.M) {
        float d[8];
        ffn_unpack8<DT>(ffn_load8(a.d + row * a.ld + c, n), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += d[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) red[warp][lane * 8 + j] = s[j];
  __syncthreads();
  const int col = cb * kColWidth + threadIdx.x;
  if (col < a.N) {
    float t = red[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) t += red[w][threadIdx.x];
    a.colsum[(size_t)rb * a.N + col] = t;
  }
}

struct ColFinishArgs {
  const float* colsum;  // [blocks][outputs][N]
  uint16_t* out[2];     // either may be nullptr
  int blocks, outputs, N, dtype;
};

// Adds the row blocks' sums in order; one rounding to the head dtype.
__global__ void __launch_bounds__(256) col_finish_kernel(const ColFinishArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.outputs * a.N) return;
  const int o = i / a.N, col = i - o * a.N;
  uint16_t* out = o ? a.out[1] : a.out[0];
  if (out == nullptr) return;
  const size_t step = (size_t)a.outputs * a.N;
  const float* p = a.colsum + i;
  float s = 0.0f;
  for (int b = 0; b < a.blocks; ++b) s += __ldg(p + b * step);
  out[col] = (uint16_t)(ep_pack(s, 0.0f, a.dtype) & 0xffffu);
}

struct FfnReduceArgs {
  const float* ws;  // [outputs][S][M][N] (gated: outputs 2, gate and up)
  uint16_t* y[3];   // gated: h, g, u (g and u may be nullptr); else the outputs
  const uint16_t* bias[2];
  long long MN;
  int S, N, outputs, dtype, act, gated;
};

// Second half of a split product: the S partial sums of an element are added
// in order; then the gated epilogue or one rounding.
__global__ void __launch_bounds__(256) ffn_reduce_kernel(const FfnReduceArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int dt = a.dtype;
  const long long total = a.gated ? a.MN : a.outputs * a.MN;
  const bool vec = a.N % 4 == 0;  // then every 4 consecutive elements lie in one row
  const long long units = vec ? total / 4 : total;
  const int w = vec ? 4 : 1;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < units; i += gridDim.x * 256LL) {
    const long long e = i * w;
    const int o = (int)(e / a.MN);
    const long long off = e - o * a.MN;
    float s[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !a.gated) break;
      const float* p = a.ws + ((long long)(a.gated ? h : o) * a.S) * a.MN + off;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < a.S; ++k, p += a.MN) {
        if (vec) {
          const float4 t = __ldg(reinterpret_cast<const float4*>(p));
          v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
        } else {
          v.x += __ldg(p);
        }
      }
      s[h][0] = v.x; s[h][1] = v.y; s[h][2] = v.z; s[h][3] = v.w;
    }
    auto put = [&](uint16_t* y, const float (&f)[4]) {
      const uint32_t lo = ep_pack(f[0], f[1], dt), hi = ep_pack(f[2], f[3], dt);
      if (!vec) {
        y[off] = (uint16_t)(lo & 0xffffu);
      } else if ((reinterpret_cast<uintptr_t>(y) & 7u) == 0) {
        *reinterpret_cast<uint2*>(y + off) = make_uint2(lo, hi);
      } else {
        y[off] = (uint16_t)lo; y[off + 1] = (uint16_t)(lo >> 16);
        y[off + 2] = (uint16_t)hi; y[off + 3] = (uint16_t)(hi >> 16);
      }
    };
    if (a.gated) {
      const int col = (int)(off % a.N);
      float h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < w) {
          if (a.bias[0] != nullptr) s[0][j] += ep_widen(__ldg(a.bias[0] + col + j), dt);
          if (a.bias[1] != nullptr) s[1][j] += ep_widen(__ldg(a.bias[1] + col + j), dt);
        }
        h[j] = j < w ? act_value(a.act, s[0][j]) * s[1][j] : 0.0f;
      }
      if (a.y[1] != nullptr) { put(a.y[1], s[0]); put(a.y[2], s[1]); }
      put(a.y[0], h);
    } else {
      put(o ? a.y[1] : a.y[0], s[0]);
    }
  }
}

// K == 0: g = bg, u = bu in every row.
__global__ void __launch_bounds__(256) gated_bias_kernel(const FfnReduceArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int dt = a.dtype;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < a.MN; i += gridDim.x * 256LL) {
    const int col = (int)(i % a.N);
    const float g = a.bias[0] != nullptr ? ep_widen(__ldg(a.bias[0] + col), dt) : 0.0f;
    const float u = a.bias[1] != nullptr ? ep_widen(__ldg(a.bias[1] + col), dt) : 0.0f;
    const uint32_t gu = ep_pack(g, u, dt);
    if (a.y[1] != nullptr) {
      a.y[1][i] = (uint16_t)gu;
      a.y[2][i] = (uint16_t)(gu >> 16);
    }
    a.y[0][i] = (uint16_t)ep_pack(act_value(a.act, g) * u, 0.0f, dt);
  }
}

struct FfnPackArgs {
  const uint16_t* src[4];
  uint16_t* dst[4];      // row pitch ldd (a multiple of 8), 16-byte aligned
  long long ld[4], ldd[4], rows[4];
  int cols[4];
  int count;
};

// Copies up to four matrices into rows of a 16-byte pitch, 16 bytes a thread;
// the pad columns are written as zeros and never read (the tensor maps end at
// the matrix's own columns).
__global__ void __launch_bounds__(256) ffn_pack_kernel(const FfnPackArgs a) {
  grid_dep_wait();
  grid_dep_launch();
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (t >= a.count) break;
    const long long cpr = a.ldd[t] / 8, total = a.rows[t] * cpr;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
      const long long r = i / cpr;
      const int c = (int)(i - r * cpr) * 8;
      const uint4 v = ffn_load8(a.src[t] + r * a.ld[t] + c, a.cols[t] - c);
      *reinterpret_cast<uint4*>(a.dst[t] + r * a.ldd[t] + c) = v;
    }
  }
}

}  // namespace poot
