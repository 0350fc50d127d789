// The gated block for up to 16 rows of x (a decode step): a stream of both
// weights.
//
// A block owns 16 output columns, i.e. 16 rows of Wg and the same 16 of Wu;
// its warps split K.  Per step of 32 along K lane (r = lane / 4, t = lane % 4)
// loads the 16-byte vectors [r][k + 8t ..) and [r + 8][k + 8t ..) of both
// weights and x[r][k + 8t ..) (x[r + 8] too when M > 8).  The summation order
// is free, so K is permuted inside a step: these registers then are the A (W)
// and B (x^T) fragments of two m16n8k16 MMAs per weight, without shuffles,
// and both weights share the x fragments.  Warps meet in shared memory in a
// fixed order; one thread holds g and u of an output and finishes it.
// Bound by HBM: 4 K bytes per output column.
#pragma once

#include "ffn_elem.cuh"
#include "mma.cuh"

namespace poot {

struct GatedGemvArgs {
  const uint16_t *x, *wg, *wu;
  const uint16_t* bias[2];
  uint16_t* y[3];  // h, g, u
  long long ldx;
  int M, N, K, act, save;
};

// VEC: x and the weights 16-byte aligned, K and ldx multiples of 8; else
// elements are gathered at whatever alignment each row has.
template <int DT, bool VEC>
__device__ __forceinline__ uint4 gemv_w8(const uint16_t* __restrict__ p, int n) {
  if constexpr (VEC) return ldg_stream_16(p);
  else return ffn_load8(p, n);
}

// NT: 8-column blocks of tokens (1: M <= 8, 2: M <= 16)
template <int NT, int WARPS, int DT, bool VEC>
__global__ void __launch_bounds__(WARPS * 32) gated_gemv_kernel(const GatedGemvArgs a) {
  constexpr int MT = 8 * NT;
  __shared__ float red[WARPS][2][16][MT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, t = lane & 3;
  const int K = a.K, N = a.N, M = a.M;
  const int n0 = blockIdx.x * 16;
  const int slice = ((K + WARPS * 32 - 1) / (WARPS * 32)) * 32;
  const int k_begin = min(K, warp * slice), k_end = min(K, k_begin + slice);
  const bool okA = n0 + r < N, okB = n0 + r + 8 < N, okx0 = r < M, okx1 = NT > 1 && r + 8 < M;
  const size_t rowA = (size_t)(okA ? n0 + r : 0) * K, rowB = (size_t)(okB ? n0 + r + 8 : 0) * K;
  const uint16_t* __restrict__ gA = a.wg + rowA;
  const uint16_t* __restrict__ gB = a.wg + rowB;
  const uint16_t* __restrict__ uA = a.wu + rowA;
  const uint16_t* __restrict__ uB = a.wu + rowB;
  const uint16_t* __restrict__ x0 = a.x + (okx0 ? r : 0) * a.ldx;
  const uint16_t* __restrict__ x1 = a.x + (okx1 ? r + 8 : 0) * a.ldx;
  grid_dep_wait();
  grid_dep_launch();

  float dg[NT][4], du[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[q][i] = du[q][i] = 0.0f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  constexpr int U = 4;  // steps of 32 along K in flight
  for (int k0 = k_begin; k0 < k_end; k0 += 32 * U) {
    uint4 vga[U], vgb[U], vua[U], vub[U], vx[U][NT];
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int k = k0 + 32 * s + 8 * t;
      const int n = k_end - k;  // VEC: whole vectors only (K % 8 == 0)
      const bool in = n > 0;
      vga[s] = in && okA ? gemv_w8<DT, VEC>(gA + k, n) : zero;
      vgb[s] = in && okB ? gemv_w8<DT, VEC>(gB + k, n) : zero;
      vua[s] = in && okA ? gemv_w8<DT, VEC>(uA + k, n) : zero;
      vub[s] = in && okB ? gemv_w8<DT, VEC>(uB + k, n) : zero;
      vx[s][0] = in && okx0 ? (VEC ? __ldg(reinterpret_cast<const uint4*>(x0 + k)) : ffn_load8(x0 + k, n)) : zero;
      if (NT > 1)
        vx[s][NT - 1] = in && okx1 ? (VEC ? __ldg(reinterpret_cast<const uint4*>(x1 + k)) : ffn_load8(x1 + k, n)) : zero;
    }
#pragma unroll
    for (int s = 0; s < U; ++s) {
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        mma_16816_f32<DT>(dg[q], vga[s].x, vgb[s].x, vga[s].y, vgb[s].y, vx[s][q].x, vx[s][q].y);
        mma_16816_f32<DT>(du[q], vua[s].x, vub[s].x, vua[s].y, vub[s].y, vx[s][q].x, vx[s][q].y);
        mma_16816_f32<DT>(dg[q], vga[s].z, vgb[s].z, vga[s].w, vgb[s].w, vx[s][q].z, vx[s][q].w);
        mma_16816_f32<DT>(du[q], vua[s].z, vub[s].z, vua[s].w, vub[s].w, vx[s][q].z, vx[s][q].w);
      }
    }
  }
  // D[n][m]: i = 0, 1 -> (n = r, m = 2t + i); i = 2, 3 -> (n = r + 8, m = 2t + i - 2)
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = r + (i < 2 ? 0 : 8), m = 8 * q + 2 * t + (i & 1);
      red[warp][0][n][m] = dg[q][i];
      red[warp][1][n][m] = du[q][i];
    }
  __syncthreads();
  // consecutive threads take consecutive columns of one token
  for (int o = threadIdx.x; o < 16 * M; o += WARPS * 32) {
    const int n = o & 15, m = o >> 4;
    const int col = n0 + n;
    if (col >= N) continue;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      g += red[w][0][n][m];
      u += red[w][1][n][m];
    }
    if (a.bias[0] != nullptr) g += ep_widen(__ldg(a.bias[0] + col), DT);
    if (a.bias[1] != nullptr) u += ep_widen(__ldg(a.bias[1] + col), DT);
    const size_t at = (size_t)m * N + col;
    const uint32_t gu = ep_pack_t<DT>(g, u);
    if (a.save) {
      a.y[1][at] = (uint16_t)gu;
      a.y[2][at] = (uint16_t)(gu >> 16);
    }
    a.y[0][at] = (uint16_t)ep_pack_t<DT>(act_value(a.act, g) * u, 0.0f);
  }
}

}  // namespace poot
