// The memory-bound steps around the feed-forward products: the gate's
// gradient, the second half of a split-K product, row repacking for operands
// TMA cannot read in place.
#pragma once

#include "ffn_gemm.cuh"

namespace poot {

struct FfnPackArgs {
  const uint16_t* src[4];
  uint16_t* dst[4];      // row pitch ldd (a multiple of 8), 16-byte aligned
  long long ld[4], ldd[4];
  int rows[4], cols[4];
  int count;
};

// Copies up to four matrices into rows of a 16-byte pitch.  A warp takes 1024
// elements of a row, four chunks a lane in flight.  The pad columns are
// written as zeros and never read (the tensor maps end at the matrix's own
// columns).  Blocks `block` of `blocks`.
constexpr int kPackSpan = 1024;
__device__ __forceinline__ void ffn_pack_rows(const FfnPackArgs& a, int block, int blocks) {
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)blocks * 8;
  long long skip = 0;  // this warp's first unit in the next matrix: units are dealt on over all of them
  const long long me = (long long)block * 8 + (threadIdx.x >> 5);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (t >= a.count) break;
    const uint32_t spans = (uint32_t)(a.cols[t] + kPackSpan - 1) / kPackSpan;
    const long long units = (long long)a.rows[t] * spans;
    const uint16_t *lo = a.src[t], *hi = lo + (long long)(a.rows[t] - 1) * a.ld[t] + a.cols[t];
    long long i = me - skip;
    if (i < 0) i += warps;
    for (; i < units; i += warps) {
      // (a row index fits 32 bits; 64-bit division only where the units do not)
      const long long r = units <= 0x7fffffffLL ? (long long)((uint32_t)i / spans) : i / spans;
      const int c0 = (int)(i - r * spans) * kPackSpan + lane * 8;
      const uint16_t* s = a.src[t] + r * a.ld[t];
      uint16_t* d = a.dst[t] + r * a.ldd[t];
      if (c0 + 3 * 256 + 8 <= a.cols[t] && ffn_wide_ok(s + c0, lo, hi) && ffn_wide_ok(s + c0 + 3 * 256, lo, hi)) {
        FfnPair v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = ffn_wide_load(s + c0 + j * 256);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(d + c0 + j * 256) = ffn_wide_shift(s + c0 + j * 256, v[j]);
      } else {
        for (int c = c0; c < min(a.cols[t], c0 + kPackSpan); c += 256)
          *reinterpret_cast<uint4*>(d + c) = ffn_load8_any(s + c, a.cols[t] - c, lo, hi);
      }
    }
    skip = (skip + units) % warps;
  }
}

__global__ void __launch_bounds__(256) ffn_pack_kernel(const FfnPackArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  ffn_pack_rows(a, blockIdx.x, gridDim.x);
}

constexpr int kGateThreads = 256;
constexpr int kGateWidth = 256;  // columns of a block: 32 lanes x 8

struct GateGradArgs {
  const uint16_t *dh, *g, *u;
  long long ld_dh, ld_g, ld_u;
  uint16_t *dg, *du;  // row pitch ldo, 16-byte aligned rows
  long long ldo;
  float* sums;        // [row blocks][2][N rounded up to 8] FP32 column sums, or nullptr
  int M, N, act;
  int rows;           // rows of a block, a multiple of 16
  int blocks;         // blocks of the gradient; the grid's others repack
  FfnPackArgs pack;
};

// dg = dh u act'(g), du = dh act(g), in FP32, each rounded once to the head
// dtype: they are operands of the tensor core, which takes 16-bit values.
// The bias gradients sum the unrounded values: column sums of a block go
// through registers, then shared memory, in a fixed order.  A lane has eight
// columns of every eighth row, two rows in flight.  Bound by its five streams
// (three read, two written).  VEC: rows on 16-byte boundaries.
template <int DT, bool SUMS, bool VEC>
__global__ void __launch_bounds__(kGateThreads, 4) gate_grad_kernel(const __grid_constant__ GateGradArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  if ((int)blockIdx.x >= a.blocks) {
    ffn_pack_rows(a.pack, (int)blockIdx.x - a.blocks, (int)gridDim.x - a.blocks);
    return;
  }
  // rows of a lane in flight: one where two would not fit 64 registers (four
  // blocks an SM; 7540 x 1845 with sums: 62 us with two blocks, 38 so)
  constexpr int ROWS = SUMS && !VEC ? 1 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned cblocks = (a.N + kGateWidth - 1) / kGateWidth;
  const int cb = blockIdx.x % cblocks, rb = blockIdx.x / cblocks;
  const int c = cb * kGateWidth + lane * 8;
  const int n = min(8, a.N - c);  // columns of this lane (<= 0: none)
  const long long row_end = min((long long)a.M, ((long long)rb + 1) * a.rows);
  float sg[8], su[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sg[j] = su[j] = 0.0f;
  const long long last = a.M - 1;
  const uint16_t *eh = a.dh + last * a.ld_dh + a.N, *eg = a.g + last * a.ld_g + a.N, *eu = a.u + last * a.ld_u + a.N;
  auto load = [&](const uint16_t* p, const uint16_t* lo, const uint16_t* hi) {
    return VEC ? ldg_stream_16(p) : ffn_load8_any(p, n, lo, hi);
  };
  // rows no pair of vectors of which leaves the matrices
  auto wide = [&](long long row) {
    return n == 8 && ffn_wide_ok(a.dh + row * a.ld_dh + c, a.dh, eh) && ffn_wide_ok(a.g + row * a.ld_g + c, a.g, eg) &&
           ffn_wide_ok(a.u + row * a.ld_u + c, a.u, eu);
  };
  auto grad = [&](auto act, const uint4& vh, const uint4& vg, const uint4& vu, long long row) {
    float dh[8], g[8], u[8], dg[8], du[8];
    ffn_unpack8<DT>(vh, dh);
    ffn_unpack8<DT>(vg, g);
    ffn_unpack8<DT>(vu, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v, d;
      act_both_t<decltype(act)::value, DT>(g[j], v, d);
      dg[j] = dh[j] * u[j] * d;
      du[j] = dh[j] * v;
      if constexpr (SUMS) {
        sg[j] += dg[j];
        su[j] += du[j];
      }
    }
    // whole chunks: the rows' pad columns may be written (never read)
    *reinterpret_cast<uint4*>(a.dg + row * a.ldo + c) = ffn_pack8<DT>(dg);
    *reinterpret_cast<uint4*>(a.du + row * a.ldo + c) = ffn_pack8<DT>(du);
  };
  auto rows = [&](auto act) {
    for (long long row = (long long)rb * a.rows + warp; row < row_end; row += ROWS * 8) {
      const bool two = ROWS == 2 && row + 8 < row_end;
      const uint16_t *ph = a.dh + row * a.ld_dh + c, *pg = a.g + row * a.ld_g + c, *pu = a.u + row * a.ld_u + c;
      if (!VEC && ROWS == 1 && wide(row)) {
        const FfnPair h0 = ffn_wide_load(ph), g0 = ffn_wide_load(pg), u0 = ffn_wide_load(pu);
        grad(act, ffn_wide_shift(ph, h0), ffn_wide_shift(pg, g0), ffn_wide_shift(pu, u0), row);
        continue;
      }
      if (!VEC && two && wide(row) && wide(row + 8)) {
        const uint16_t *qh = ph + 8 * a.ld_dh, *qg = pg + 8 * a.ld_g, *qu = pu + 8 * a.ld_u;
        const FfnPair h0 = ffn_wide_load(ph), g0 = ffn_wide_load(pg), u0 = ffn_wide_load(pu);
        const FfnPair h1 = ffn_wide_load(qh), g1 = ffn_wide_load(qg), u1 = ffn_wide_load(qu);
        grad(act, ffn_wide_shift(ph, h0), ffn_wide_shift(pg, g0), ffn_wide_shift(pu, u0), row);
        grad(act, ffn_wide_shift(qh, h1), ffn_wide_shift(qg, g1), ffn_wide_shift(qu, u1), row + 8);
        continue;
      }
      const uint4 h0 = load(ph, a.dh, eh), g0 = load(pg, a.g, eg), u0 = load(pu, a.u, eu);
      uint4 h1 = make_uint4(0, 0, 0, 0), g1 = h1, u1 = h1;
      if (two) {
        h1 = load(ph + 8 * a.ld_dh, a.dh, eh);
        g1 = load(pg + 8 * a.ld_g, a.g, eg);
        u1 = load(pu + 8 * a.ld_u, a.u, eu);
      }
      grad(act, h0, g0, u0, row);
      if (two) grad(act, h1, g1, u1, row + 8);
    }
  };
  if (n > 0) {
    if (a.act == kActSilu) rows(std::integral_constant<int, kActSilu>{});
    else if (a.act == kActGeluTanh) rows(std::integral_constant<int, kActGeluTanh>{});
    else rows(std::integral_constant<int, kActGeluErf>{});
  }
  if constexpr (SUMS) {
    __shared__ float red[8][kGateWidth];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) red[warp][lane * 8 + j] = o ? su[j] : sg[j];
      __syncthreads();
      const int col = cb * kGateWidth + threadIdx.x;
      if (col < a.N) {
        float s = red[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < 8; ++w) s += red[w][threadIdx.x];
        a.sums[((size_t)rb * 2 + o) * ((a.N + 7) / 8 * 8) + col] = s;
      }
    }
  }
}

struct FfnReduceArgs {
  const float* ws;  // [outputs][S][M][ldw] (gated: outputs 2, gate and up)
  uint16_t* y[3];   // gated: h, g, u (g and u may be nullptr); else the outputs
  const uint16_t* bias[2];
  long long M;
  int S, N, ldw, outputs, dtype, act, gated;
};

// Second half of a split product: the S partial sums of an element are added
// in order; then the gated epilogue or one rounding.  Four columns a thread
// (the workspace's rows are padded to that).
__global__ void __launch_bounds__(256) ffn_reduce_kernel(const FfnReduceArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int dt = a.dtype, quads = a.ldw / 4;
  const long long per = a.M * quads, total = a.gated ? per : a.outputs * per, slab = a.M * a.ldw;
  const bool vec = a.N % 4 == 0;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const int o = i >= per ? 1 : 0;  // (at most two outputs)
    const long long e = i - o * per;
    const long long row = e <= 0x7fffffffLL ? (long long)((uint32_t)e / (uint32_t)quads) : e / quads;
    const int col = (int)(e - row * quads) * 4;
    const int n = min(4, a.N - col);
    float s[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !a.gated) break;
      const float* p = a.ws + (long long)(a.gated ? h : o) * a.S * slab + row * a.ldw + col;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int k = 0; k < a.S; ++k) {
        const float4 t = __ldg(reinterpret_cast<const float4*>(p + k * slab));
        v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
      }
      s[h][0] = v.x; s[h][1] = v.y; s[h][2] = v.z; s[h][3] = v.w;
    }
    const long long off = row * a.N + col;
    auto put = [&](uint16_t* y, const float (&f)[4]) {
      const uint32_t lo = ep_pack(f[0], f[1], dt), hi = ep_pack(f[2], f[3], dt);
      if (vec && (reinterpret_cast<uintptr_t>(y) & 7u) == 0) {
        *reinterpret_cast<uint2*>(y + off) = make_uint2(lo, hi);
      } else {
        const uint16_t w[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) y[off + j] = w[j];
      }
    };
    if (a.gated) {
      float h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < n) {
          if (a.bias[0] != nullptr) s[0][j] += ep_widen(__ldg(a.bias[0] + col + j), dt);
          if (a.bias[1] != nullptr) s[1][j] += ep_widen(__ldg(a.bias[1] + col + j), dt);
        }
        h[j] = j < n ? act_value<kEpiBf16>(a.act, s[0][j]) * s[1][j] : 0.0f;
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
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < a.M * a.N; i += gridDim.x * 256LL) {
    const int col = (int)(i % a.N);
    const float g = a.bias[0] != nullptr ? ep_widen(__ldg(a.bias[0] + col), dt) : 0.0f;
    const float u = a.bias[1] != nullptr ? ep_widen(__ldg(a.bias[1] + col), dt) : 0.0f;
    const uint32_t gu = ep_pack(g, u, dt);
    if (a.y[1] != nullptr) {
      a.y[1][i] = (uint16_t)gu;
      a.y[2][i] = (uint16_t)(gu >> 16);
    }
    a.y[0][i] = (uint16_t)ep_pack(act_value<kEpiBf16>(a.act, g) * u, 0.0f, dt);
  }
}

}  // namespace poot
