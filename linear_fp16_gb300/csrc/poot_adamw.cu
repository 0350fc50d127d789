// C ABI of the AdamW step (include/poot_train.h): argument checks, tables and
// launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <vector>

#include "poot_train.h"
#include "adamw.cuh"
#include "host.cuh"

namespace {

using namespace poot;
using namespace poot_host;

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxElements = int64_t(1) << 40;

struct AdamDevice {
  bool ready = false;
  int status = POOT_OK;
  int sms = 0;
  int blocks[2] = {0, 0};  // that run at one time: states in 32, in 8 bits
};
int adam_smem_bytes(bool small) { return small ? kAdamSmem : 0; }
std::mutex g_mu;
AdamDevice g_devices[kMaxDevices];

int adam_device(AdamDevice** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return POOT_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_mu);
  AdamDevice& d = g_devices[dev];
  if (!d.ready) {
    const int q = device_query(dev, &d.sms);
    if (q == POOT_ERR_CUDA) return q;
    if (q == POOT_OK) {
      for (int b = 0; b < 2; ++b) {
        int few = 0, many = 0;
        auto fewer = b == 0 ? adamw_kernel<kAdamTableFew, 32> : adamw_kernel<kAdamTableFew, 8>;
        auto more = b == 0 ? adamw_kernel<kAdamTable, 32> : adamw_kernel<kAdamTable, 8>;
        const int smem = adam_smem_bytes(b == 1);
        if ((e = cudaFuncSetAttribute(fewer, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(more, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
            (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&few, fewer, kAdamThreads, smem)) != cudaSuccess ||
            (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&many, more, kAdamThreads, smem)) != cudaSuccess)
          return cuda_fail(e);
        d.blocks[b] = std::max(1, std::min(few, many)) * d.sms;
      }
    }
    d.status = q;
    d.ready = true;
  }
  *out = &d;
  return d.status;
}

// Memory that a call touches: a range that is written overlaps no other.
struct Ranges {
  struct Range {
    uintptr_t lo, hi;
    bool write;
  };
  std::vector<Range> all;
  void add(const void* p, int64_t bytes, bool write) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p != nullptr && bytes > 0) all.push_back({lo, lo + uintptr_t(bytes), write});
  }
  bool conflict() {
    std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t end_any = 0, end_written = 0;
    for (const Range& r : all) {
      if (r.lo < end_written || (r.write && r.lo < end_any)) return true;
      end_any = std::max(end_any, r.hi);
      if (r.write) end_written = std::max(end_written, r.hi);
    }
    return false;
  }
};

inline int64_t blocks_of(int64_t n) { return (n + kAdamBlock - 1) / kAdamBlock; }
inline int dtype_size(int dtype) { return dtype == POOT_GRAD_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype >= POOT_GRAD_F16 && dtype <= POOT_GRAD_F32; }

// Blocks that share `chunks` out, eight warps each: as many as run at one time while a warp has
// less than kTurns chunks, then one for every kTurns turns, so that SMs that are ahead take more of them.
constexpr int64_t kTurns = 16;
inline unsigned adam_grid(int64_t chunks, int most) {
  const int64_t turns = (chunks + kAdamWarps - 1) / kAdamWarps;
  // (2^20 blocks times the chunks of a launch, below 2^41, stay in 64 bits)
  const int64_t blocks = std::max<int64_t>(std::min<int64_t>(turns, most), turns / kTurns);
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(blocks, int64_t(1) << 20)));
}

template <int T>
cudaError_t step_list(const poot_adamw_tensor* const* t, int count, const poot_adamw_args& p, const AdamArgs& a,
                      int most, cudaStream_t stream) {
  AdamTable<T> table;
  table.count = count;
  table.first[0] = 0;
  const bool small = p.bits == 8;
  for (int i = 0; i < count; ++i) {
    const poot_adamw_tensor& x = *t[i];
    table.p[i] = x.param;
    table.g[i] = x.grad;
    table.m[i] = x.m;
    table.v[i] = x.v;
    table.ms[i] = x.m_scale;
    table.vs[i] = x.v_scale;
    table.copy[i] = x.copy;
    table.n[i] = x.n;
    table.first[i + 1] = table.first[i] + blocks_of(x.n);
    table.decay[i] = static_cast<float>(p.lr_device != nullptr ? x.weight_decay : 1.0 - p.lr * x.weight_decay);
    const bool vec = aligned(x.param, 16) && aligned(x.grad, 16) && aligned(x.m, 16) && aligned(x.v, 16) &&
                     aligned(x.copy, 16);
    table.types[i] = static_cast<unsigned char>(x.param_dtype | x.grad_dtype << 2 |
                                                (x.copy != nullptr ? x.copy_dtype << 4 : 0) | (vec ? kAdamVec : 0));
  }
  return launch(small ? adamw_kernel<T, 8> : adamw_kernel<T, 32>, dim3(adam_grid(table.first[count], most)),
                dim3(kAdamThreads), adam_smem_bytes(small), stream, table, a);
}

int adamw_step(const poot_adamw_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_adamw_args& p = *ap;
  auto in = [](double v, double lo, double hi) { return v >= lo && v < hi; };  // (false for NaN)
  if (p.count < 0 || p.count > POOT_FFN_MAX_SIZE || (p.count > 0 && p.tensors == nullptr) ||
      (p.bits != 32 && p.bits != 8) || !in(p.beta1, 0.0, 1.0) || !in(p.beta2, 0.0, 1.0) || !in(p.eps, 0.0, INFINITY) ||
      (p.step_device == nullptr && p.step < 1) || (p.lr_device == nullptr && !in(p.lr, 0.0, INFINITY)) ||
      (p.grad_scale_device == nullptr && !std::isfinite(p.grad_scale)))
    return POOT_ERR_INVALID_ARG;
  if (!aligned(p.lr_device, 4) || !aligned(p.step_device, 8) || !aligned(p.grad_scale_device, 4))
    return POOT_ERR_MISALIGNED;
  Ranges ranges;
  ranges.add(p.lr_device, 4, false);
  ranges.add(p.step_device, 8, false);
  ranges.add(p.grad_scale_device, 4, false);
  std::vector<const poot_adamw_tensor*> list;
  const bool small = p.bits == 8;
  for (int64_t i = 0; i < p.count; ++i) {
    const poot_adamw_tensor& x = p.tensors[i];
    if (x.n < 0 || x.n > kMaxElements || !dtype_ok(x.param_dtype) || !dtype_ok(x.grad_dtype) ||
        !in(x.weight_decay, 0.0, INFINITY))
      return POOT_ERR_INVALID_ARG;
    if (x.n == 0) continue;
    if (x.param == nullptr || x.grad == nullptr || x.m == nullptr || x.v == nullptr ||
        (small && (x.m_scale == nullptr || x.v_scale == nullptr)) ||
        (x.copy != nullptr && (x.param_dtype != POOT_GRAD_F32 || !dtype_ok(x.copy_dtype) || x.copy_dtype == POOT_GRAD_F32)))
      return POOT_ERR_INVALID_ARG;
    const int ps = dtype_size(x.param_dtype), gs = dtype_size(x.grad_dtype), ss = small ? 1 : 4;
    if (!aligned(x.param, ps) || !aligned(x.grad, gs) || !aligned(x.m, ss) || !aligned(x.v, ss) ||
        (small && (!aligned(x.m_scale, 4) || !aligned(x.v_scale, 4))) || !aligned(x.copy, 2))
      return POOT_ERR_MISALIGNED;
    ranges.add(x.param, x.n * ps, true);
    ranges.add(x.grad, x.n * gs, false);
    ranges.add(x.m, x.n * ss, true);
    ranges.add(x.v, x.n * ss, true);
    if (small) {
      ranges.add(x.m_scale, 4 * blocks_of(x.n), true);
      ranges.add(x.v_scale, 4 * blocks_of(x.n), true);
    }
    ranges.add(x.copy, x.n * 2, true);
    list.push_back(&x);
  }
  if (ranges.conflict()) return POOT_ERR_INVALID_ARG;
  if (list.empty()) return POOT_OK;
  AdamDevice* d;
  const int st = adam_device(&d);
  if (st != POOT_OK) return st;
  AdamArgs a;
  std::memset(&a, 0, sizeof(a));
  a.lr_dev = p.lr_device;
  a.step_dev = reinterpret_cast<const long long*>(p.step_device);
  a.grad_scale_dev = p.grad_scale_device;
  a.lr = p.lr;
  a.log_b1 = std::log(p.beta1);
  a.log_b2 = std::log(p.beta2);
  a.step = p.step;
  a.b1 = static_cast<float>(p.beta1);
  a.omb1 = static_cast<float>(1.0 - p.beta1);
  a.b2 = static_cast<float>(p.beta2);
  a.omb2 = static_cast<float>(1.0 - p.beta2);
  a.eps = static_cast<float>(p.eps);
  a.grad_scale = static_cast<float>(p.grad_scale);
  a.minus_zero = -0.0f;
  if (p.lr_device == nullptr && p.step_device == nullptr)
    adam_factors(p.lr, a.log_b1, a.log_b2, static_cast<double>(p.step), &a.step_size, &a.root_scale);
  const int most = d->blocks[small ? 1 : 0];
  for (size_t i = 0; i < list.size(); i += kAdamTable) {
    const int n = static_cast<int>(std::min<size_t>(kAdamTable, list.size() - i));
    const cudaError_t e = n <= kAdamTableFew ? step_list<kAdamTableFew>(list.data() + i, n, p, a, most, stream)
                                             : step_list<kAdamTable>(list.data() + i, n, p, a, most, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return POOT_OK;
}

template <int T>
cudaError_t values_list(const poot_adamw_codes* const* t, int count, int most, cudaStream_t stream) {
  AdamValueTable<T> table;
  table.count = count;
  table.first[0] = 0;
  for (int i = 0; i < count; ++i) {
    const poot_adamw_codes& x = *t[i];
    table.m[i] = x.m;
    table.v[i] = x.v;
    table.ms[i] = x.m_scale;
    table.vs[i] = x.v_scale;
    table.mo[i] = x.m_out;
    table.vo[i] = x.v_out;
    table.n[i] = x.n;
    table.first[i + 1] = table.first[i] + blocks_of(x.n);
    table.vec[i] = aligned(x.m, 4) && aligned(x.v, 4) && aligned(x.m_out, 16) && aligned(x.v_out, 16);
  }
  return launch(adamw_values_kernel<T>, dim3(adam_grid(table.first[count], most)), dim3(kAdamThreads), 0, stream, table);
}

int adamw_values(const poot_adamw_codes* s, int64_t count, cudaStream_t stream) {
  if (count < 0 || count > POOT_FFN_MAX_SIZE || (count > 0 && s == nullptr)) return POOT_ERR_INVALID_ARG;
  Ranges ranges;
  std::vector<const poot_adamw_codes*> list;
  for (int64_t i = 0; i < count; ++i) {
    const poot_adamw_codes& x = s[i];
    if (x.n < 0 || x.n > kMaxElements) return POOT_ERR_INVALID_ARG;
    if (x.n == 0) continue;
    if (x.m == nullptr || x.v == nullptr || x.m_scale == nullptr || x.v_scale == nullptr || x.m_out == nullptr ||
        x.v_out == nullptr)
      return POOT_ERR_INVALID_ARG;
    if (!aligned(x.m_scale, 4) || !aligned(x.v_scale, 4) || !aligned(x.m_out, 4) || !aligned(x.v_out, 4))
      return POOT_ERR_MISALIGNED;
    ranges.add(x.m, x.n, false);
    ranges.add(x.v, x.n, false);
    ranges.add(x.m_scale, 4 * blocks_of(x.n), false);
    ranges.add(x.v_scale, 4 * blocks_of(x.n), false);
    ranges.add(x.m_out, 4 * x.n, true);
    ranges.add(x.v_out, 4 * x.n, true);
    list.push_back(&x);
  }
  if (ranges.conflict()) return POOT_ERR_INVALID_ARG;
  if (list.empty()) return POOT_OK;
  AdamDevice* d;
  const int st = adam_device(&d);
  if (st != POOT_OK) return st;
  for (size_t i = 0; i < list.size(); i += kAdamTable) {
    const int n = static_cast<int>(std::min<size_t>(kAdamTable, list.size() - i));
    const cudaError_t e = n <= kAdamTableFew ? values_list<kAdamTableFew>(list.data() + i, n, 8 * d->sms, stream)
                                             : values_list<kAdamTable>(list.data() + i, n, 8 * d->sms, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return POOT_OK;
}

// a C entry lets no C++ exception out (host allocations may throw)
template <typename F>
int guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return cuda_fail(cudaErrorMemoryAllocation);
  }
}

}  // namespace

extern "C" {

int poot_adamw_step(const poot_adamw_args* args, poot_stream_t stream) {
  return guarded([&] { return adamw_step(args, reinterpret_cast<cudaStream_t>(stream)); });
}

int poot_adamw_values(const poot_adamw_codes* states, int64_t count, poot_stream_t stream) {
  return guarded([&] { return adamw_values(states, count, reinterpret_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
