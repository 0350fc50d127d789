// Host-side pieces shared by the library's translation units: the CUDA error
// of the calling thread, the device query, launches, tensor-map encoding and
// the per-stream workspace.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <functional>
#include <map>
#include <mutex>
#include <thread>
#include <utility>
#include <vector>

#include "poot_linear.h"

namespace poot_host {

inline thread_local cudaError_t t_last_cuda_error = cudaSuccess;

using EncodeTiledFn = decltype(&cuTensorMapEncodeTiled);
inline EncodeTiledFn g_encode_tiled = nullptr;
inline std::mutex g_encode_mu;

inline int cuda_fail(cudaError_t e) {
  t_last_cuda_error = e;
  return POOT_ERR_CUDA;
}

// Whether `dev` is an sm_103 device, and its SM count; looks up the driver's
// tensor-map encoder on first use.
inline int device_query(int dev, int* sms) {
  int major = 0, minor = 0;
  cudaError_t e;
  if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return cuda_fail(e);
  if (major != 10 || minor != 3) return POOT_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_encode_mu);
  if (g_encode_tiled == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return cuda_fail(e);
    if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cuda_fail(cudaErrorNotSupported);
    g_encode_tiled = reinterpret_cast<EncodeTiledFn>(fn);
  }
  return POOT_OK;
}

// The feed-forward kernels' device error word on the current device, read
// and cleared (poot_ffn.cu).
cudaError_t take_ffn_device_error(unsigned int* word);

// Launch with programmatic stream serialisation (see grid_dep_wait in
// ptx.cuh): the kernel may be scheduled while the previous kernel in the
// stream drains; it waits for that kernel before touching global memory.
// cluster_x > 1 launches clusters of that many CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_clustered(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             unsigned cluster_x, Args&&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  std::memset(attr, 0, sizeof(attr));
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster_x > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster_x;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                   Args&&... args) {
  return launch_clustered(kernel, grid, block, smem, stream, 1u, std::forward<Args>(args)...);
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  if (a == nullptr || b == nullptr || abytes <= 0 || bbytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

// [slabs][outer][inner] tensor of FP32, box [1][box_outer][box_inner].
inline bool encode_3d_f32(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t slabs,
                   uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[3] = {inner, outer, slabs};
  const cuuint64_t strides[2] = {inner * 4, inner * outer * 4};
  const cuuint32_t box[3] = {box_inner, box_outer, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides,
                                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Row-major [outer, inner] tensor of 2-byte elements (binary16, or bfloat16
// when bf16), rows `pitch` elements apart (default inner), box [box_outer,
// box_inner].
inline bool encode_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
               uint32_t box_outer, CUtensorMapSwizzle swizzle, bool bf16 = false, uint64_t pitch = 0) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {(pitch != 0 ? pitch : inner) * 2};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode_tiled(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                    2, const_cast<void*>(base), dims,
                                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// [slabs][outer][inner] tensor of 2-byte elements, box [1][box_outer][box_inner]
// (each box stays inside one slab: stores clip at `outer` per slab).
inline bool encode_3d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t slabs,
               uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle, bool bf16) {
  const cuuint64_t dims[3] = {inner, outer, slabs};
  const cuuint64_t strides[2] = {inner * 2, inner * outer * 2};
  const cuuint32_t box[3] = {box_inner, box_outer, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode_tiled(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                    3, const_cast<void*>(base), dims, strides, box, estr,
                                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// ---- workspaces -------------------------------------------------------------
struct Workspace {
  std::mutex mu;  // held by the call that uses the buffer, see WorkspaceLease
  void* ptr = nullptr;
  size_t bytes = 0;
};
inline std::mutex g_ws_mu;  // guards the map and the retired list, never held while a buffer's is taken
// key: (device, stream, thread): the thread is part of the key only for
// cudaStreamPerThread, one handle that names a different stream in each thread
struct WorkspaceKey {
  int dev;
  cudaStream_t stream;
  std::thread::id thread;
  bool operator<(const WorkspaceKey& o) const {
    if (dev != o.dev) return dev < o.dev;
    if (stream != o.stream) return std::less<cudaStream_t>()(stream, o.stream);
    return thread < o.thread;
  }
};
inline std::map<WorkspaceKey, Workspace> g_ws;  // (its elements never move)
inline std::vector<void*> g_ws_retired;

struct WorkspaceRelease {
  ~WorkspaceRelease() {
    for (auto& kv : g_ws)
      if (kv.second.ptr != nullptr) cudaFree(kv.second.ptr);
    for (void* p : g_ws_retired) cudaFree(p);
  }
};
inline WorkspaceRelease g_ws_release;

// Workspace of a call (split-K partial sums, packed operands, dg and du, the
// clip's partial sums).  Outside stream capture: one buffer per (device,
// stream; thread for cudaStreamPerThread), grown by doubling and kept for the
// life of the process (a buffer outgrown is kept too, as work queued earlier
// may still read it).  A call writes the buffer with one launch and reads it
// with a later one, so the order of a stream's launches alone does not make it
// safe to share: two host threads could queue A1 B1 A2 B2.  The lease holds
// the buffer's lock until the call has queued its last launch; calls of other
// threads on that stream wait on the host meanwhile.  Under capture: a
// graph-owned allocation (cudaMallocAsync / cudaFreeAsync on the capturing
// stream become memory nodes of the graph), so that a graph never shares a
// buffer with calls made outside it.  nullptr: no workspace (and no lock).
struct WorkspaceLease {
  void* ptr = nullptr;
  bool graph_owned = false;
  cudaStream_t stream = nullptr;
  std::unique_lock<std::mutex> lock;
  // After the call's last launch, or on any early return before it: a
  // graph-owned workspace is freed on its stream, a buffer's lock is given up.
  cudaError_t release() {
    cudaError_t e = cudaSuccess;
    if (graph_owned) e = cudaFreeAsync(ptr, stream);
    graph_owned = false;
    if (lock.owns_lock()) lock.unlock();
    return e;
  }
  WorkspaceLease() = default;
  WorkspaceLease(const WorkspaceLease&) = delete;
  WorkspaceLease& operator=(const WorkspaceLease&) = delete;
  WorkspaceLease(WorkspaceLease&& o) noexcept
      : ptr(o.ptr), graph_owned(o.graph_owned), stream(o.stream), lock(std::move(o.lock)) {
    o.graph_owned = false;
  }
  WorkspaceLease& operator=(WorkspaceLease&& o) noexcept {
    if (this != &o) {
      (void)release();
      ptr = o.ptr;
      graph_owned = o.graph_owned;
      stream = o.stream;
      lock = std::move(o.lock);
      o.graph_owned = false;
    }
    return *this;
  }
  ~WorkspaceLease() { (void)release(); }
};

inline WorkspaceLease stream_workspace(int dev, cudaStream_t stream, size_t bytes) {
  WorkspaceLease lease;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) {
    (void)cudaGetLastError();
    return lease;
  }
  if (cs != cudaStreamCaptureStatusNone) {
    if (cs != cudaStreamCaptureStatusActive || cudaMallocAsync(&lease.ptr, bytes, stream) != cudaSuccess) {
      (void)cudaGetLastError();
      lease.ptr = nullptr;
      return lease;
    }
    lease.graph_owned = true;
    lease.stream = stream;
    return lease;
  }
  const std::thread::id tid = stream == cudaStreamPerThread ? std::this_thread::get_id() : std::thread::id();
  Workspace* ws;
  {
    std::lock_guard<std::mutex> lock(g_ws_mu);
    ws = &g_ws[WorkspaceKey{dev, stream, tid}];
  }
  std::unique_lock<std::mutex> held(ws->mu);
  if (ws->bytes < bytes) {
    const auto whole = [](size_t v) { return (v + (size_t(1) << 20) - 1) & ~((size_t(1) << 20) - 1); };
    size_t want = whole(bytes > 2 * ws->bytes ? bytes : 2 * ws->bytes);
    void* p = nullptr;
    cudaError_t e = cudaMalloc(&p, want);
    if (e != cudaSuccess && whole(bytes) < want) {  // no room to double: what the call needs
      (void)cudaGetLastError();
      want = whole(bytes);
      e = cudaMalloc(&p, want);
    }
    if (e != cudaSuccess) {
      (void)cudaGetLastError();  // the caller goes without, or reports it
      return lease;
    }
    if (ws->ptr != nullptr) {
      std::lock_guard<std::mutex> lock(g_ws_mu);
      g_ws_retired.push_back(ws->ptr);
    }
    ws->ptr = p;
    ws->bytes = want;
  }
  lease.ptr = ws->ptr;
  lease.lock = std::move(held);
  return lease;
}

}  // namespace poot_host
