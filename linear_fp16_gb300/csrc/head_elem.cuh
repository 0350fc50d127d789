// The memory-bound steps around the products of a vocabulary head: the rows' loss
// from the tiles' maxima and sums, the scale and the operands of the
// gradients, the last rounding of sums.
#pragma once

#include "ffn_elem.cuh"
#include "head.cuh"

namespace poot {

struct HeadLossArgs {
  const float2* partial;  // [parts][M]
  const float* picked;    // [M], written where the target is inside the vocabulary
  const long long* target;
  float *loss, *lse;      // lse may be nullptr
  long long ignore, M;
  int vocab, parts;
};

constexpr int kHeadLossThreads = 256;

// Joins a row's pairs in a fixed order: ROWS rows a block, 256 / ROWS threads on
// each.  Bound by the latency of the pairs' reads (32 bytes a row and tile; 4096 rows of 128
// tiles, 17 MB, 9 us by itself).
template <int ROWS>
__global__ void __launch_bounds__(kHeadLossThreads) head_loss_kernel(const HeadLossArgs a) {
  constexpr int GROUPS = kHeadLossThreads / ROWS;
  __shared__ float2 red[kHeadLossThreads];
  grid_dep_wait();
  grid_dep_launch();
  const int group = threadIdx.x / ROWS;
  const long long row = (long long)blockIdx.x * ROWS + threadIdx.x % ROWS;
  float2 v = make_float2(-INFINITY, 0.0f);
  if (row < a.M) {
#pragma unroll 8
    for (int p = group; p < a.parts; p += GROUPS) v = head_join(v, __ldg(a.partial + p * a.M + row));
  }
  red[threadIdx.x] = v;
#pragma unroll
  for (int g = GROUPS / 2; g > 0; g /= 2) {
    __syncthreads();
    if (group < g) red[threadIdx.x] = v = head_join(v, red[threadIdx.x + g * ROWS]);
  }
  if (group != 0 || row >= a.M) return;
  // (m is a logit times log2(e): taken back in 64 bits, its rounding to 32 has cancelled in the sum)
  const double lse = (double)v.x * 0.6931471805599453 + (double)logf(v.y);
  if (a.lse != nullptr) a.lse[row] = (float)lse;
  const long long t = __ldg(a.target + row);
  a.loss[row] = t == a.ignore ? 0.0f : (t >= 0 && t < a.vocab ? (float)(lse - (double)__ldg(a.picked + row)) : NAN);
}

struct HeadPrepArgs {
  const float* dloss;
  long long dloss_stride;
  const long long* target;
  long long ignore;
  long long rows;
  float* scale;          // [2], see HeadArgs
  const uint16_t* x;     // rows ld apart
  uint16_t* xc;          // copy, row pitch ldc (a multiple of 8); nullptr: none
  long long ld, ldc;
  int cols;
  int copy_blocks;       // after block 0, these copy x; the rest repack
  FfnPackArgs pack;
};

// Before the gradients.  Block 0: the power of two that brings the largest
// finite |dloss| of the rows in use to [2^14, 2^15), and its inverse.  The next
// blocks copy x with zeros in ignored rows: q is zero there, but as an operand of
// dW's product zero times what such a row holds (padding is often left
// unwritten) need not be.  The others repack W where TMA cannot read it.  Bound by HBM where W
// is repacked (333 x 32003 x 770, 102 MB: 19 us).
__global__ void __launch_bounds__(256) head_prep_kernel(const __grid_constant__ HeadPrepArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0) {
    __shared__ uint32_t red[8];
    uint32_t most = 0;
    auto take = [&](float d) {
      const uint32_t u = __float_as_uint(fabsf(d));
      if (u < 0x7f800000u) most = max(most, u);
    };
    if (a.dloss_stride == 0) {
      take(__ldg(a.dloss));
    } else {
#pragma unroll 4
      for (long long r = threadIdx.x; r < a.rows; r += 256) {
        const bool used = __ldg(a.target + r) != a.ignore;
        take(used ? __ldg(a.dloss + r * a.dloss_stride) : 0.0f);
      }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) red[warp] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < 8; ++w) most = max(most, red[w]);
      // (both powers stay inside FP32's normal range; all zero: as for 1)
      const int e = most == 0 ? 0 : max((int)(most >> 23) - 127, -100);
      a.scale[0] = __uint_as_float((uint32_t)(14 - e + 127) << 23);
      a.scale[1] = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
    }
    return;
  }
  const int block = (int)blockIdx.x - 1;
  if (block >= a.copy_blocks) {
    ffn_pack_rows(a.pack, block - a.copy_blocks, (int)gridDim.x - 1 - a.copy_blocks);
    return;
  }
  const uint16_t *lo = a.x, *hi = a.x + (a.rows - 1) * a.ld + a.cols;
  const int spans = (a.cols + kPackSpan - 1) / kPackSpan;
  const long long units = a.rows * spans, warps = (long long)a.copy_blocks * 8;
  for (long long i = (long long)block * 8 + warp; i < units; i += warps) {
    const long long r = units <= 0x7fffffffLL ? (long long)((uint32_t)i / (uint32_t)spans) : i / spans;
    const int c0 = (int)(i - r * spans) * kPackSpan + lane * 8;
    const uint16_t* s = a.x + r * a.ld;
    uint16_t* d = a.xc + r * a.ldc;
    const bool used = __ldg(a.target + r) != a.ignore;
#pragma unroll
    for (int j = 0; j < kPackSpan / 256; ++j) {
      const int c = c0 + j * 256;
      if (c < a.cols)
        *reinterpret_cast<uint4*>(d + c) = used ? ffn_load8_any(s + c, a.cols - c, lo, hi) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

struct HeadReduceArgs {
  const float* ws;  // [S][M][ldw]
  uint16_t* y;      // [M][N]
  const float* scale;
  long long M;
  int S, N, ldw, dtype;
};

// FP32 sums -> their total in order, times scale[1], rounded once.  Bound by their reads
// (333 x 770, eight sums: 5 us, launch included).
static __global__ void __launch_bounds__(256) head_reduce_kernel(const HeadReduceArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const float scale = a.scale[1];
  const int quads = a.ldw / 4;
  const long long total = a.M * quads, slab = a.M * a.ldw;
  const bool vec = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7u) == 0;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long row = i <= 0x7fffffffLL ? (long long)((uint32_t)i / (uint32_t)quads) : i / quads;
    const int col = (int)(i - row * quads) * 4;
    const float* p = a.ws + row * a.ldw + col;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < a.S; ++k) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(p + k * slab));
      v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
    }
    const uint32_t u0 = ep_pack(v.x * scale, v.y * scale, a.dtype), u1 = ep_pack(v.z * scale, v.w * scale, a.dtype);
    uint16_t* y = a.y + row * a.N + col;
    if (vec) {
      *reinterpret_cast<uint2*>(y) = make_uint2(u0, u1);
    } else {
      const uint16_t w[4] = {(uint16_t)u0, (uint16_t)(u0 >> 16), (uint16_t)u1, (uint16_t)(u1 >> 16)};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < a.N) y[j] = w[j];
    }
  }
}

}  // namespace poot
