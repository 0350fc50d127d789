// Clipping by the global norm over a list of gradient tensors:
//
//   norm  = sqrt(sum over all tensors of sum g^2)
//   scale = min(1, max_norm / (norm + 1e-6))
//   out   = RN(g * scale)          (in place where dst == src)
//
// Two launches: sums of squares, one FP64 partial per block, over 32 KB
// pieces of the tensors; then every block adds the partials in the same
// order (so all see the same scale, and the result does not depend on which
// block finishes first) and scales its pieces, last pieces first: those are
// what L2 still holds.  Bound by HBM: the tensors are read once for the norm,
// then read (from L2 as far as it holds them) and written once.
#pragma once

#include "epilogue.cuh"
#include "ptx.cuh"

namespace poot {

enum GradDtype : int { kGradF16 = 0, kGradBf16 = 1, kGradF32 = 2 };

constexpr int kClipThreads = 256;
constexpr int kClipPieceBytes = 32 * 1024;
constexpr int kClipTable = 512;  // tensors of one launch

struct ClipTable {
  const void* src[kClipTable];
  void* dst[kClipTable];
  long long n[kClipTable];
  int first[kClipTable + 1];  // first piece of each tensor
  unsigned char dtype[kClipTable];
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

__device__ __forceinline__ int clip_find(const ClipTable& t, int piece) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= piece) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int DT>
struct GradElem {
  using type = uint16_t;
  static __device__ __forceinline__ float load(const uint16_t* p) { return ep_widen(*p, DT); }
  static __device__ __forceinline__ uint16_t round(float v) { return (uint16_t)ep_pack_t<DT>(v, 0.0f); }
};
template <>
struct GradElem<kGradF32> {
  using type = float;
  static __device__ __forceinline__ float load(const float* p) { return *p; }
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

// Sum of squares of p[0 .. n) by one block's threads (each its own share).
// FP32 over at most 64 elements at a time, then FP64.  Where FP32 squares
// leave their range (bfloat16 and binary32 reach 3e38), the same elements are
// squared in FP64.
template <int DT>
__device__ __forceinline__ double clip_sum_piece(const void* src, int n) {
  using E = GradElem<DT>;
  using T = typename E::type;
  constexpr int V = 16 / sizeof(T), U = kClipPieceBytes / 16 / kClipThreads;
  const T* p = static_cast<const T*>(src);
  const int tid = threadIdx.x;
  double acc = 0.0;
  auto slow = [&](float f) { return (double)f * (double)f; };
  auto in_range = [](float s) { return s > 1e-30f && s < 1e37f; };
  // elements before the first 16-byte boundary, whole vectors, the rest
  const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / (int)sizeof(T));
  const int nv = (n - head) / V;
  const int tail0 = head + nv * V;
  const uint4* pv = reinterpret_cast<const uint4*>(p + head);
  for (int b = 0; b < nv; b += kClipThreads * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u * kClipThreads + tid;
      v[u] = i < nv ? __ldg(pv + i) : make_uint4(0u, 0u, 0u, 0u);
    }
    float s = 0.0f;
    uint32_t any = 0u;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[V];
      grad_unpack<DT>(v[u], f);
      any |= v[u].x | v[u].y | v[u].z | v[u].w;
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(f[j], f[j], s);
    }
    if (in_range(s)) {
      acc += (double)s;
    } else if (any != 0u) {
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        const int i = b + u * kClipThreads + tid;
        if (i < nv)
          for (int j = 0; j < V; ++j) acc += slow(E::load(reinterpret_cast<const T*>(pv + i) + j));
      }
    }
  }
  if (tid < head) acc += slow(E::load(p + tid));
  if (tid < n - tail0) acc += slow(E::load(p + tail0 + tid));
  return acc;
}

__global__ void __launch_bounds__(kClipThreads) clip_sum_kernel(const __grid_constant__ ClipTable t, const ClipArgs a) {
  __shared__ double red[kClipThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  double acc = 0.0;
  const int pieces = t.first[t.count];
  for (int c = blockIdx.x; c < pieces; c += gridDim.x) {
    const int i = clip_find(t, c);
    const int dt = t.dtype[i];
    const int per = kClipPieceBytes / (dt == kGradF32 ? 4 : 2);
    const long long e0 = (long long)(c - t.first[i]) * per;
    const int n = (int)min((long long)per, t.n[i] - e0);
    if (dt == kGradF16) acc += clip_sum_piece<kGradF16>(static_cast<const uint16_t*>(t.src[i]) + e0, n);
    else if (dt == kGradBf16) acc += clip_sum_piece<kGradBf16>(static_cast<const uint16_t*>(t.src[i]) + e0, n);
    else acc += clip_sum_piece<kGradF32>(static_cast<const float*>(t.src[i]) + e0, n);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = red[0];
#pragma unroll
    for (int w = 1; w < kClipThreads / 32; ++w) s += red[w];
    a.partial[a.part0 + blockIdx.x] = s;
  }
}

template <int DT>
__device__ __forceinline__ void clip_scale_piece(const void* src, void* dst, int n, float scale) {
  using E = GradElem<DT>;
  using T = typename E::type;
  constexpr int V = 16 / sizeof(T), U = kClipPieceBytes / 16 / kClipThreads;
  const T* p = static_cast<const T*>(src);
  T* o = static_cast<T*>(dst);
  const int tid = threadIdx.x;
  const uintptr_t ps = reinterpret_cast<uintptr_t>(p), os = reinterpret_cast<uintptr_t>(o);
  if (((ps ^ os) & 15u) != 0) {  // source and destination rows never share a 16-byte boundary
    for (int i = tid; i < n; i += kClipThreads) o[i] = E::round(E::load(p + i) * scale);
    return;
  }
  const int head = min(n, (int)((16 - (ps & 15u)) & 15u) / (int)sizeof(T));
  const int nv = (n - head) / V;
  const int tail0 = head + nv * V;
  const uint4* pv = reinterpret_cast<const uint4*>(p + head);
  uint4* ov = reinterpret_cast<uint4*>(o + head);
  for (int b = 0; b < nv; b += kClipThreads * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u * kClipThreads + tid;
      if (i < nv) v[u] = pv[i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u * kClipThreads + tid;
      if (i < nv) {
        float f[V];
        grad_unpack<DT>(v[u], f);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] *= scale;
        ov[i] = grad_pack<DT>(f);
      }
    }
  }
  if (tid < head) o[tid] = E::round(E::load(p + tid) * scale);
  if (tid < n - tail0) o[tail0 + tid] = E::round(E::load(p + tail0 + tid) * scale);
}

__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const __grid_constant__ ClipTable t, const ClipArgs a) {
  __shared__ double red[kClipThreads / 32];
  __shared__ float s_scale;
  grid_dep_wait();
  grid_dep_launch();
  double acc = 0.0;
  for (int i = threadIdx.x; i < a.parts; i += kClipThreads) acc += a.partial[i];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = red[0];
#pragma unroll
    for (int w = 1; w < kClipThreads / 32; ++w) s += red[w];
    const double norm = sqrt(s);
    const double q = (double)a.max_norm / (norm + 1e-6);
    s_scale = (float)(q > 1.0 ? 1.0 : q);  // NaN stays NaN
    if (blockIdx.x == 0 && a.write_norm) *a.norm = (float)norm;
  }
  __syncthreads();
  const float scale = s_scale;
  const int pieces = t.first[t.count];
  for (int k = blockIdx.x; k < pieces; k += gridDim.x) {
    const int c = pieces - 1 - k;
    const int i = clip_find(t, c);
    // times one changes nothing: a tensor clipped in place stays as it is
    if (scale == 1.0f && t.src[i] == t.dst[i]) continue;
    const int dt = t.dtype[i];
    const int per = kClipPieceBytes / (dt == kGradF32 ? 4 : 2);
    const long long e0 = (long long)(c - t.first[i]) * per;
    const int n = (int)min((long long)per, t.n[i] - e0);
    const long long o16 = e0 * 2, o32 = e0 * 4;
    const char* s = static_cast<const char*>(t.src[i]);
    char* d = static_cast<char*>(t.dst[i]);
    if (dt == kGradF16) clip_scale_piece<kGradF16>(s + o16, d + o16, n, scale);
    else if (dt == kGradBf16) clip_scale_piece<kGradBf16>(s + o16, d + o16, n, scale);
    else clip_scale_piece<kGradF32>(s + o32, d + o32, n, scale);
  }
}

}  // namespace poot
