// Clipping by the global norm over a list of gradient tensors:
//
//   norm  = sqrt(sum over all tensors of sum g^2)
//   scale = min(1, max_norm / (norm + 1e-6))
//   out   = RN(g * scale)          (in place where dst == src)
//
// Every block sums the squares of its 32 KB pieces into one FP64 partial; then,
// in a second launch or after the grid barrier of a cooperative one, it adds
// all partials in the same order (so all blocks see the same scale, and the
// result does not depend on which block comes first) and scales its pieces,
// the last one first: those are what L2, or in the cooperative form the
// registers, still hold.  Bound by HBM: the tensors are read for the norm, read
// again, from L2 as far as it holds them, and written.  Lists beyond kClipTable
// tensors take several launches of each half.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "epilogue.cuh"
#include "ptx.cuh"

namespace poot {

enum GradDtype : int { kGradF16 = 0, kGradBf16 = 1, kGradF32 = 2 };

constexpr int kClipThreads = 256;
constexpr int kClipPieceBytes = 32 * 1024;
constexpr int kClipVectors = kClipPieceBytes / 16 / kClipThreads;  // a thread's vectors of a piece
// Two blocks of 100 registers without spills, half of the next piece in flight
// while half of this one is worked on (1.4 GB on GB300: 632 us; three blocks
// 661, spilling; four without the overlap 649)
constexpr int kClipBlocksPerSm = 2;
constexpr int kClipTable = 512;      // tensors of one launch
constexpr int kClipTableFew = 64;    // short lists: less to pass to the launch

template <int T>
struct ClipTable {
  const void* src[T];
  void* dst[T];
  long long n[T];
  int first[T + 1];  // first piece of each tensor
  unsigned char dtype[T];
  int count;
};

struct ClipArgs {
  double* partial;     // of all launches
  int part0;           // first partial of this launch (sum) or 0
  int parts;           // partials in all (scale)
  float max_norm;
  float* norm;
  int write_norm;      // this launch's block 0 writes the norm
};

template <int DT>
struct GradElem {
  using type = uint16_t;
  static __device__ __forceinline__ uint16_t round(float v) { return (uint16_t)ep_pack_t<DT>(v, 0.0f); }
};
template <>
struct GradElem<kGradF32> {
  using type = float;
  static __device__ __forceinline__ float round(float v) { return v; }
};

// the FP32 values of a 16-byte vector
template <int DT>
__device__ __forceinline__ void grad_unpack(const uint4& v, float (&f)[DT == kGradF32 ? 4 : 8]) {
  if constexpr (DT == kGradF32) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = ep_unpack_t<DT>(w[i]);
      f[2 * i] = a.x;
      f[2 * i + 1] = a.y;
    }
  }
}
template <int DT>
__device__ __forceinline__ uint4 grad_pack(const float (&f)[DT == kGradF32 ? 4 : 8]) {
  if constexpr (DT == kGradF32) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    return make_uint4(ep_pack_t<DT>(f[0], f[1]), ep_pack_t<DT>(f[2], f[3]), ep_pack_t<DT>(f[4], f[5]),
                      ep_pack_t<DT>(f[6], f[7]));
  }
}

// One piece of a tensor: elements before the first 16-byte boundary of the
// source, whole vectors, the rest.
struct ClipPiece {
  const char* src;
  char* dst;
  int dtype, size, head, nv, tail0, n;
};

template <int T>
__device__ __forceinline__ ClipPiece clip_piece(const ClipTable<T>& t, int c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  ClipPiece p;
  p.dtype = t.dtype[lo];
  p.size = p.dtype == kGradF32 ? 4 : 2;
  const int per = kClipPieceBytes / p.size;
  const long long e0 = (long long)(c - t.first[lo]) * per;
  p.n = (int)min((long long)per, t.n[lo] - e0);
  p.src = static_cast<const char*>(t.src[lo]) + e0 * p.size;
  p.dst = static_cast<char*>(t.dst[lo]) + e0 * p.size;
  p.head = min(p.n, (int)((16 - (reinterpret_cast<uintptr_t>(p.src) & 15u)) & 15u) / p.size);
  p.nv = (p.n - p.head) / (16 / p.size);
  p.tail0 = p.head + p.nv * (16 / p.size);
  return p;
}

// One thread's share of a piece: vectors, and at most one element of its
// ragged ends (thread t < head the t-th, thread 8 + t the t-th after the
// vectors; zero bits where there is none).
struct ClipShare {
  uint4 v[kClipVectors];
  uint32_t edge;
};
constexpr int kClipHalf = kClipVectors / 2;

__device__ __forceinline__ int clip_edge(const ClipPiece& p) {  // its element, or -1
  const int t = threadIdx.x;
  if (t < 8) return t < p.head ? t : -1;
  return t - 8 < p.n - p.tail0 ? p.tail0 + t - 8 : -1;
}

// half h of the vectors (zeros past the end), and the edge with the first
template <int H>
__device__ __forceinline__ void clip_load(const ClipPiece& p, ClipShare& x) {
  const uint4* pv = reinterpret_cast<const uint4*>(p.src + p.head * p.size) + threadIdx.x;
#pragma unroll
  for (int u = H * kClipHalf; u < (H + 1) * kClipHalf; ++u)
    x.v[u] = u * kClipThreads + (int)threadIdx.x < p.nv ? pv[u * kClipThreads] : make_uint4(0u, 0u, 0u, 0u);
  if constexpr (H == 0) {
    const int e = clip_edge(p);
    x.edge = 0u;
    if (e >= 0)
      x.edge = p.size == 4 ? reinterpret_cast<const uint32_t*>(p.src)[e]
                           : (uint32_t)reinterpret_cast<const uint16_t*>(p.src)[e];
  }
}

template <int DT>
__device__ __forceinline__ float grad_bits(uint32_t e) {
  return DT == kGradF32 ? __uint_as_float(e) : ep_widen((uint16_t)e, DT);
}

// Sum of squares of half a share, of values times `scale`, in FP32 (at most 33
// elements).
template <int DT, int H>
__device__ __forceinline__ float clip_sum_scaled(const ClipShare& x, float scale) {
  constexpr int V = DT == kGradF32 ? 4 : 8;
  float s = 0.0f;
#pragma unroll
  for (int u = H * kClipHalf; u < (H + 1) * kClipHalf; ++u) {
    float f[V];
    grad_unpack<DT>(x.v[u], f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float t = f[j] * scale;
      s = fmaf(t, t, s);
    }
  }
  if constexpr (H == 0) {
    const float t = grad_bits<DT>(x.edge) * scale;
    s = fmaf(t, t, s);
  }
  return s;
}

// Sum of squares of half a share.  Where the FP32 sum leaves the middle of
// its range (bfloat16 and binary32 reach 3e38 and 1e-45, their squares do
// not), the values are scaled by a power of two first: 2^-70 keeps 33 squares
// of the largest below 2^127, 2^100 the square of the smallest above 2^-126.
template <int DT, int H>
__device__ __forceinline__ double clip_sum(const ClipShare& x) {
  const float s = clip_sum_scaled<DT, H>(x, 1.0f);
  if (s > 1e-30f && s < 1e37f) return (double)s;
  if (s <= 1e-30f) {
    constexpr float kUp = 1.2676506002282294e30f;                           // 2^100
    return (double)clip_sum_scaled<DT, H>(x, kUp) * 6.223015277861142e-61;  // 2^-200
  }
  constexpr float kDown = 8.470329472543003e-22f;                           // 2^-70 (NaN comes through)
  return (double)clip_sum_scaled<DT, H>(x, kDown) * 1.3937965749081639e42;  // 2^140
}
template <int H>
__device__ __forceinline__ double clip_sum(int dt, const ClipShare& x) {
  return dt == kGradF16 ? clip_sum<kGradF16, H>(x) : (dt == kGradBf16 ? clip_sum<kGradBf16, H>(x) : clip_sum<kGradF32, H>(x));
}

template <int DT, int H>
__device__ __forceinline__ void clip_scale(const ClipPiece& p, const ClipShare& x, float scale) {
  using E = GradElem<DT>;
  using T = typename E::type;
  constexpr int V = 16 / sizeof(T);
  T* o = reinterpret_cast<T*>(p.dst);
  T* ov = o + p.head + (int)threadIdx.x * V;
  const bool vec = (reinterpret_cast<uintptr_t>(ov) & 15u) == 0;  // source and destination share 16-byte boundaries
#pragma unroll
  for (int u = H * kClipHalf; u < (H + 1) * kClipHalf; ++u) {
    if (u * kClipThreads + (int)threadIdx.x < p.nv) {
      float f[V];
      grad_unpack<DT>(x.v[u], f);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] *= scale;
      if (vec) {
        *reinterpret_cast<uint4*>(ov + u * kClipThreads * V) = grad_pack<DT>(f);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) ov[u * kClipThreads * V + j] = E::round(f[j]);
      }
    }
  }
  if constexpr (H == 0) {
    const int e = clip_edge(p);
    if (e >= 0) o[e] = E::round(grad_bits<DT>(x.edge) * scale);
  }
}
template <int H>
__device__ __forceinline__ void clip_scale(const ClipPiece& p, const ClipShare& x, float scale) {
  if (p.dtype == kGradF16) clip_scale<kGradF16, H>(p, x, scale);
  else if (p.dtype == kGradBf16) clip_scale<kGradBf16, H>(p, x, scale);
  else clip_scale<kGradF32, H>(p, x, scale);
}

enum ClipMode : int { kClipBoth = 0, kClipSum = 1, kClipScale = 2 };

// Sum of a warp's values.
__device__ __forceinline__ double clip_warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <int T, int MODE>
__global__ void __launch_bounds__(kClipThreads, kClipBlocksPerSm)
    clip_kernel(const __grid_constant__ ClipTable<T> t, const ClipArgs a) {
  __shared__ double red[kClipThreads];
  __shared__ float s_scale;
  grid_dep_wait();
  grid_dep_launch();
  const int pieces = t.first[t.count];
  const int mine = (int)blockIdx.x < pieces ? (pieces - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  auto nth = [&](int k) { return clip_piece(t, (int)blockIdx.x + k * (int)gridDim.x); };
  // half of the next piece is on its way while half of this one is worked on
  ClipShare x;
  ClipPiece p;
  if constexpr (MODE != kClipScale) {
    double acc = 0.0;
    if (mine > 0) {
      p = nth(0);
      clip_load<0>(p, x);
      clip_load<1>(p, x);
      for (int k = 0;;) {
        const int dt = p.dtype;
        const bool more = ++k < mine;
        if (more) p = nth(k);
        acc += clip_sum<0>(dt, x);
        if (more) clip_load<0>(p, x);
        acc += clip_sum<1>(dt, x);
        if (!more) break;
        clip_load<1>(p, x);
      }

    }
    // FP64 is slow here (two lanes a cycle per SM): one warp adds the block's
    // sums, and below one lane takes the root and the quotient (9 MB: 13.7 us
    // with all threads doing so, 9.1 so)
    red[threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.x < 32) {
      double s = red[threadIdx.x];
#pragma unroll
      for (int w = 1; w < kClipThreads / 32; ++w) s += red[w * 32 + threadIdx.x];
      s = clip_warp_sum(s);
      if (threadIdx.x == 0) a.partial[a.part0 + blockIdx.x] = s;
    }
  }
  if constexpr (MODE == kClipSum) return;
  if constexpr (MODE == kClipBoth) cooperative_groups::this_grid().sync();
  if (threadIdx.x < 32) {
    double acc = 0.0;
    for (int i = threadIdx.x; i < a.parts; i += 32) acc += a.partial[i];
    acc = clip_warp_sum(acc);
    if (threadIdx.x == 0) {
      const double norm = sqrt(acc);
      const double q = (double)a.max_norm / (norm + 1e-6);
      s_scale = (float)(q > 1.0 ? 1.0 : q);  // NaN stays NaN
      if (blockIdx.x == 0 && a.write_norm) *a.norm = (float)norm;
    }
  }
  __syncthreads();
  const float scale = s_scale;
  if (mine == 0) return;
  // from the last piece down: x holds it after the sums
  int k = mine - 1;
  if constexpr (MODE == kClipScale) {
    p = nth(k);
    clip_load<0>(p, x);
    clip_load<1>(p, x);
  }
  // times one changes nothing: a tensor clipped in place stays as it is, and
  // is not read again
  auto load = [&](auto h) {
    if (!(scale == 1.0f && p.src == p.dst)) clip_load<decltype(h)::value>(p, x);
  };
  const std::integral_constant<int, 0> h0;
  const std::integral_constant<int, 1> h1;
  for (;;) {
    const ClipPiece q = p;
    const bool more = --k >= 0, skip = scale == 1.0f && q.src == q.dst;
    if (more) p = nth(k);
    if (!skip) clip_scale<0>(q, x, scale);
    if (more) load(h0);
    if (!skip) clip_scale<1>(q, x, scale);
    if (!more) break;
    load(h1);
  }
}

}  // namespace poot
