// The library's per-stream workspace with the CUDA runtime replaced by host
// functions: a buffer belongs to one call at a time.  Prints one line per
// failed check; exits 0 when all hold.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <thread>

#include "host.cuh"

static std::atomic<int> g_fail_allocs{0}, g_capturing{0}, g_async_frees{0};

// the few runtime functions the workspace calls
extern "C" {
cudaError_t cudaMalloc(void** p, size_t n) {
  if (g_fail_allocs > 0) {
    --g_fail_allocs;
    return cudaErrorMemoryAllocation;
  }
  *p = std::malloc(n);
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
  std::free(p);
  return cudaSuccess;
}
cudaError_t cudaMallocAsync(void** p, size_t n, cudaStream_t) {
  *p = std::malloc(n);
  return cudaSuccess;
}
cudaError_t cudaFreeAsync(void* p, cudaStream_t) {
  ++g_async_frees;
  std::free(p);
  return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
  *s = g_capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
}

static int g_bad = 0;
static void check(bool ok, const char* what) {
  if (!ok) {
    std::printf("FAILED: %s\n", what);
    ++g_bad;
  }
}

static cudaStream_t handle(uintptr_t v) { return reinterpret_cast<cudaStream_t>(v); }

// whether another thread can lease `stream`'s workspace now (it waits 0.2 s
// for it); `after` then runs, and the thread is joined
template <typename F>
static bool other_thread_gets(cudaStream_t stream, F&& after) {
  std::atomic<bool> got{false};
  std::thread t([&] {
    poot_host::WorkspaceLease l = poot_host::stream_workspace(0, stream, 64);
    got = l.ptr != nullptr;
  });
  for (int i = 0; i < 200 && !got; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  const bool now = got;
  after();
  t.join();
  check(got, "the other thread gets the workspace in the end");
  return now;
}

int main() {
  using poot_host::stream_workspace;
  using poot_host::WorkspaceLease;
  const cudaStream_t a = handle(0x1000), b = handle(0x2000);
  auto nothing = [] {};
  {
    WorkspaceLease l = stream_workspace(0, a, 64);
    check(l.ptr != nullptr, "a workspace");
    check(!other_thread_gets(a, [&] { (void)l.release(); }), "a second call on the stream waits for the first's release");
    WorkspaceLease m;
    m = stream_workspace(0, a, 64);
    WorkspaceLease n(std::move(m));
    check(!other_thread_gets(a, [&] { (void)n.release(); }), "a lease moved on still holds the workspace");
    WorkspaceLease o = stream_workspace(0, a, 64);
    check(other_thread_gets(b, nothing), "another stream has a workspace of its own");
  }
  check(other_thread_gets(a, nothing), "a lease gives its workspace up where it ends");
  {
    // the buffer of another thread's call is not replaced while that call uses it
    WorkspaceLease l = stream_workspace(0, a, 64);
    void* const p = l.ptr;
    (void)l.release();
    WorkspaceLease big = stream_workspace(0, a, size_t(8) << 20);
    check(big.ptr != nullptr && big.ptr != p, "a larger buffer");
  }
  {
    // 8 MB held: doubled to 16 where there is room, else what is asked for
    g_fail_allocs = 1;
    WorkspaceLease l = stream_workspace(0, a, size_t(9) << 20);
    check(l.ptr != nullptr && g_fail_allocs == 0, "a buffer that cannot be doubled grows to what the call needs");
  }
  {
    g_fail_allocs = 1;
    WorkspaceLease l = stream_workspace(0, a, size_t(64) << 20);
    check(l.ptr == nullptr, "no workspace where none can be had");
    WorkspaceLease again = stream_workspace(0, a, 64);  // (the same thread: a lock kept would hang here)
    check(again.ptr != nullptr, "a lease that failed holds nothing");
  }
  {
    g_capturing = 1;
    WorkspaceLease l = stream_workspace(0, a, 64), m = stream_workspace(0, a, 64);
    check(l.ptr != nullptr && m.ptr != nullptr && l.ptr != m.ptr, "graph-owned workspaces are their call's alone");
    g_capturing = 0;
    check(other_thread_gets(a, nothing), "a graph-owned workspace holds no lock");
  }
  check(g_async_frees == 2, "graph-owned workspaces are freed");
  {
    WorkspaceLease l = stream_workspace(0, cudaStreamPerThread, 64);
    check(other_thread_gets(cudaStreamPerThread, nothing), "cudaStreamPerThread is another stream in another thread");
  }
  if (g_bad == 0) std::printf("ok\n");
  return g_bad == 0 ? 0 : 1;
}
