// The gated block for up to 16 rows of x (a decode step): a stream of both
// weights, bound by HBM (4 K bytes per output column).
//
// gated_gemv_kernel: operands on 16-byte boundaries.  A block, one or two per
// SM, owns an equal share of consecutive output columns, whatever their number
// (its last columns may fill only part of an MMA: what is not there is not
// loaded), and walks it in passes of up to 16 columns; its warps split K.  Lane
// (r = lane / 4, t = lane % 4) takes, per step of 32 along K and group of 8
// columns, the vectors Wg[n + r][k + 8t ..) and Wu[n + r][k + 8t ..) and
// x[r][k + 8t ..) (x[r + 8] too when M > 8).  The summation order is free, so
// K is permuted inside a step: these registers then are the A fragment (rows
// 0-7 of the MMA: gate, 8-15: up) and the B fragment (x^T) of two m16n8k16
// MMAs, without shuffles, and a thread ends up with g and u of the same
// output.  The weights pass through a ring of cp.async copies whose slots a
// lane fills and reads alone (no barriers): the bytes in flight per SM are
// the ring's 192 KB, whatever registers can hold, and they keep flowing over
// the ends of passes.  Warps meet in shared memory in a fixed order.
//
// gated_gemv_any_kernel: any alignment (rows gathered by smaller loads).
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
  int kw;  // warps that split K
};

// Two blocks of eight warps per SM, beside which the next launch's blocks find
// room to start; where those would have fewer than a group of 8 columns each,
// one block of sixteen warps (GB300, two blocks against one: 16 x 14336 x 4096
// 41.5 and 45.2 us, 8 x 4096 x 4096 13.7 and 15.3; 1 x 14336 x 4096 38.2 and
// 39.1 in a loop on one set of weights, 40.3 and 39.9 where they change from
// call to call; 16 x 1024 x 4096 10.1 and 7.7, 1 x 1024 x 768 3.1 and 2.7).
constexpr int kGgSub = 2;    // groups of 8 columns per pass
constexpr int kGgSteps = 2;  // steps of 32 along K per ring slot
constexpr int kGgRing = 3;   // slots
constexpr int kGgSlot = kGgSteps * kGgSub * 2 * 512;  // bytes of a warp's slot
__host__ __device__ constexpr int gg_ring_bytes(int warps) { return warps * kGgRing * kGgSlot; }
__host__ __device__ constexpr int gg_red_floats(int nt, int warps) { return warps * kGgSub * 16 * (8 * nt + 1); }
__host__ __device__ constexpr int gg_smem_bytes(int nt, int warps) { return gg_ring_bytes(warps) + gg_red_floats(nt, warps) * 4; }
static_assert(gg_smem_bytes(2, 16) <= 232448 && 2 * (gg_smem_bytes(2, 8) + 1024) <= 233472, "shared memory of an SM");

// biases, then one rounding of each result
template <int DT>
__device__ __forceinline__ void gg_finish(const GatedGemvArgs& a, float g, float u, int m, int col) {
  if (a.bias[0] != nullptr) g += ep_widen(__ldg(a.bias[0] + col), DT);
  if (a.bias[1] != nullptr) u += ep_widen(__ldg(a.bias[1] + col), DT);
  const size_t at = (size_t)m * a.N + col;
  if (a.save) {
    const uint32_t gu = ep_pack_t<DT>(g, u);
    a.y[1][at] = (uint16_t)gu;
    a.y[2][at] = (uint16_t)(gu >> 16);
  }
  a.y[0][at] = (uint16_t)ep_pack_t<DT>(act_value<DT>(a.act, g) * u, 0.0f);
}

// NT: 8-column blocks of tokens (1: M <= 8, 2: M <= 16)
template <int NT, int DT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) gated_gemv_kernel(const GatedGemvArgs a) {
  constexpr int MT = 8 * NT;
  extern __shared__ __align__(16) uint8_t gg_smem[];
  float* red = reinterpret_cast<float*>(gg_smem + gg_ring_bytes(WARPS));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, t = lane & 3;
  const int K = a.K, N = a.N, M = a.M;
  // this block's columns, this warp's K range (a multiple of a slot's)
  const int per = N / (int)gridDim.x, extra = N % (int)gridDim.x;
  const int c_begin = (int)blockIdx.x * per + min((int)blockIdx.x, extra);
  const int c_end = c_begin + per + ((int)blockIdx.x < extra ? 1 : 0);
  constexpr int KS = 32 * kGgSteps;
  // K is split over a.kw warps (as many as have a slot's worth of it, a power
  // of two); the warps are WARPS / kw teams, each with every (WARPS / kw)-th pass
  const int kw = a.kw, teams = WARPS / kw, team = warp / kw;
  const int slice = ((K + kw * KS - 1) / (kw * KS)) * KS;
  const int k_begin = min(K, (warp & (kw - 1)) * slice), k_end = min(K, k_begin + slice);
  const int kchunks = (k_end - k_begin + KS - 1) / KS;
  const int passes = (c_end - c_begin + 8 * kGgSub - 1) / (8 * kGgSub);
  const int rounds = (passes + teams - 1) / teams;
  const int total = rounds * kchunks;  // (a team's last round may be past the last pass: nothing is loaded)
  const uint32_t ring = smem_addr(gg_smem) + (uint32_t)(warp * kGgRing * kGgSlot + lane * 16);
  const bool okx0 = r < M, okx1 = NT > 1 && r + 8 < M;
  const uint16_t* __restrict__ x0 = a.x + (okx0 ? r : 0) * a.ldx;
  const uint16_t* __restrict__ x1 = a.x + (okx1 ? r + 8 : 0) * a.ldx;
  grid_dep_wait();
  grid_dep_launch();

  // slot layout: vector (step, group, weight) of lane l at ((step * kGgSub + group) * 2 + weight) * 512 + 16 l
  const ptrdiff_t up = a.wu - a.wg;
  auto issue = [&](int p, int c, int slot) {
    const int n0 = c_begin + p * 8 * kGgSub, k0 = k_begin + c * KS;
    const uint32_t dst = ring + (uint32_t)(slot * kGgSlot);
    const uint16_t* src = a.wg + (size_t)(n0 + r) * K + (k0 + 8 * t);
    if (n0 + 8 * kGgSub <= c_end && k0 + KS <= k_end) {
      // all there: addresses advance by immediates
#pragma unroll
      for (int g = 0; g < kGgSub; ++g, src += (size_t)8 * K) {
        const uint16_t* usrc = src + up;
        static_assert(kGgSteps == 2, "two steps below");
        const uint32_t gd = dst + (uint32_t)(g * 1024);
        cp_async_16_at<0, 0>(gd, src);
        cp_async_16_at<512, 0>(gd, usrc);
        cp_async_16_at<kGgSub * 1024, 64>(gd, src);
        cp_async_16_at<kGgSub * 1024 + 512, 64>(gd, usrc);
      }
      return;
    }
#pragma unroll
    for (int s = 0; s < kGgSteps; ++s) {
#pragma unroll
      for (int g = 0; g < kGgSub; ++g) {
        const int n = n0 + 8 * g;
        if (n < c_end) {  // warp-uniform
          const bool in = n + r < c_end && k0 + 32 * s + 8 * t < k_end;  // K % 8 == 0: a vector is all in or all out
          const uint16_t* q = in ? src + (size_t)(8 * g) * K + 32 * s : a.wg;
          const uint32_t at = dst + (uint32_t)(((s * kGgSub + g) * 2) * 512);
          cp_async_16(at, q, in ? 16u : 0u);
          cp_async_16(at + 512, in ? q + up : a.wu, in ? 16u : 0u);
        }
      }
    }
  };
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load_x = [&](int c, uint4 (&v)[kGgSteps][NT]) {
#pragma unroll
    for (int s = 0; s < kGgSteps; ++s) {
      const int k = k_begin + c * KS + 32 * s + 8 * t;
      v[s][0] = okx0 && k < k_end ? __ldg(reinterpret_cast<const uint4*>(x0 + k)) : zero;
      if (NT > 1) v[s][NT - 1] = okx1 && k < k_end ? __ldg(reinterpret_cast<const uint4*>(x1 + k)) : zero;
    }
  };

  int ip = team, ic = 0;  // next chunk to issue
  auto issue_next = [&](int slot) {
    if (ip < passes && kchunks > 0) {
      issue(ip, ic, slot);
      if (++ic == kchunks) { ic = 0; ip += teams; }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kGgRing - 1; ++i) issue_next(i);
  int slot = 0, fill = kGgRing - 1;
  uint4 vx[kGgSteps][NT];
  if (total > 0) load_x(0, vx);

  for (int rd = 0; rd < rounds; ++rd) {
    const int p = rd * teams + team;
    float d[kGgSub][NT][4];
#pragma unroll
    for (int g = 0; g < kGgSub; ++g)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[g][q][i] = 0.0f;
    const int n0 = c_begin + p * 8 * kGgSub;
    for (int c = 0; c < kchunks; ++c) {
      issue_next(fill);
      cp_async_wait_group<kGgRing - 1>();  // this chunk's copies have landed
      uint4 nx[kGgSteps][NT];
      load_x(c + 1 == kchunks ? 0 : c + 1, nx);
      const uint8_t* src = gg_smem + warp * kGgRing * kGgSlot + slot * kGgSlot + lane * 16;
#pragma unroll
      for (int s = 0; s < kGgSteps; ++s) {
#pragma unroll
        for (int g = 0; g < kGgSub; ++g) {
          if (n0 + 8 * g < c_end) {
            const uint4 wg = *reinterpret_cast<const uint4*>(src + ((s * kGgSub + g) * 2) * 512);
            const uint4 wu = *reinterpret_cast<const uint4*>(src + ((s * kGgSub + g) * 2 + 1) * 512);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
              mma_16816_f32<DT>(d[g][q], wg.x, wu.x, wg.y, wu.y, vx[s][q].x, vx[s][q].y);
              mma_16816_f32<DT>(d[g][q], wg.z, wu.z, wg.w, wu.w, vx[s][q].z, vx[s][q].w);
            }
          }
        }
      }
#pragma unroll
      for (int s = 0; s < kGgSteps; ++s)
#pragma unroll
        for (int q = 0; q < NT; ++q) vx[s][q] = nx[s][q];
      slot = slot + 1 == kGgRing ? 0 : slot + 1;
      fill = fill + 1 == kGgRing ? 0 : fill + 1;
    }
    // D rows 0-7: gate of column r, rows 8-15: up; columns 2t, 2t + 1: tokens
    if (rd > 0) __syncthreads();  // the previous round has been read
#pragma unroll
    for (int g = 0; g < kGgSub; ++g)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[((warp * kGgSub + g) * 16 + r + (i < 2 ? 0 : 8)) * (MT + 1) + 8 * q + 2 * t + (i & 1)] = d[g][q][i];
    __syncthreads();
    for (int o = threadIdx.x; o < teams * 8 * kGgSub * M; o += WARPS * 32) {
      const int n = o & (8 * kGgSub - 1), j = (o / (8 * kGgSub)) & (teams - 1), m = o / (8 * kGgSub * teams);
      const int col = c_begin + (rd * teams + j) * 8 * kGgSub + n;
      if (col >= c_end) continue;
      float g = 0.0f, u = 0.0f;
#pragma unroll 4
      for (int w = 0; w < kw; ++w) {
        const float* e = red + (((j * kw + w) * kGgSub + (n >> 3)) * 16 + (n & 7)) * (MT + 1) + m;
        g += e[0];
        u += e[8 * (MT + 1)];
      }
      gg_finish<DT>(a, g, u, m, col);
    }
  }
  cp_async_wait_all();
}

// Any alignment: a block owns 16 columns, its warps split K; a lane gathers
// the eight elements of a vector by the widest loads its row allows.
template <int NT, int WARPS, int DT>
__global__ void __launch_bounds__(WARPS * 32) gated_gemv_any_kernel(const GatedGemvArgs a) {
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
  const uint16_t *ge = a.wg + (size_t)N * K, *ue = a.wu + (size_t)N * K, *xe = a.x + (M - 1) * a.ldx + K;
  grid_dep_wait();
  grid_dep_launch();

  float dg[NT][4], du[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[q][i] = du[q][i] = 0.0f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  constexpr int U = 2;  // steps of 32 along K in flight
  for (int k0 = k_begin; k0 < k_end; k0 += 32 * U) {
    uint4 vga[U], vgb[U], vua[U], vub[U], vx[U][NT];
    const int kf = k0 + 8 * t, kl = kf + 32 * (U - 1);  // this lane's first and last vector
    if (okB && kl + 8 <= k_end && ffn_wide_ok(gA + kf, a.wg, ge) && ffn_wide_ok(gB + kl, a.wg, ge) &&
        ffn_wide_ok(uA + kf, a.wu, ue) && ffn_wide_ok(uB + kl, a.wu, ue)) {
      FfnPair p[U][4];
#pragma unroll
      for (int s = 0; s < U; ++s) {
        const int k = kf + 32 * s;
        p[s][0] = ffn_wide_load(gA + k);
        p[s][1] = ffn_wide_load(gB + k);
        p[s][2] = ffn_wide_load(uA + k);
        p[s][3] = ffn_wide_load(uB + k);
      }
#pragma unroll
      for (int s = 0; s < U; ++s) {
        const int k = kf + 32 * s;
        vga[s] = ffn_wide_shift(gA + k, p[s][0]);
        vgb[s] = ffn_wide_shift(gB + k, p[s][1]);
        vua[s] = ffn_wide_shift(uA + k, p[s][2]);
        vub[s] = ffn_wide_shift(uB + k, p[s][3]);
      }
    } else {
#pragma unroll
      for (int s = 0; s < U; ++s) {
        const int k = kf + 32 * s, n = k_end - k;
        vga[s] = n > 0 && okA ? ffn_load8(gA + k, n) : zero;
        vgb[s] = n > 0 && okB ? ffn_load8(gB + k, n) : zero;
        vua[s] = n > 0 && okA ? ffn_load8(uA + k, n) : zero;
        vub[s] = n > 0 && okB ? ffn_load8(uB + k, n) : zero;
      }
    }
    // (rows of x that are not there read the first one's, and give zeros)
    if (kl + 8 <= k_end && ffn_wide_ok(x0 + kf, a.x, xe) && ffn_wide_ok(x0 + kl, a.x, xe) &&
        (NT == 1 || (ffn_wide_ok(x1 + kf, a.x, xe) && ffn_wide_ok(x1 + kl, a.x, xe)))) {
      FfnPair p[U][NT];
#pragma unroll
      for (int s = 0; s < U; ++s) {
        p[s][0] = ffn_wide_load(x0 + kf + 32 * s);
        if (NT > 1) p[s][NT - 1] = ffn_wide_load(x1 + kf + 32 * s);
      }
#pragma unroll
      for (int s = 0; s < U; ++s) {
        vx[s][0] = okx0 ? ffn_wide_shift(x0 + kf + 32 * s, p[s][0]) : zero;
        if (NT > 1) vx[s][NT - 1] = okx1 ? ffn_wide_shift(x1 + kf + 32 * s, p[s][NT - 1]) : zero;
      }
    } else {
#pragma unroll
      for (int s = 0; s < U; ++s) {
        const int k = kf + 32 * s, n = k_end - k;
        vx[s][0] = n > 0 && okx0 ? ffn_load8(x0 + k, n) : zero;
        if (NT > 1) vx[s][NT - 1] = n > 0 && okx1 ? ffn_load8(x1 + k, n) : zero;
      }
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
    gg_finish<DT>(a, g, u, m, col);
  }
}

}  // namespace poot
