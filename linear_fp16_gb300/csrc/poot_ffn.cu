// C ABI of the feed-forward operators (include/poot_ffn.h): argument checks,
// tile plans, workspaces and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <vector>

#include "poot_ffn.h"
#include "clip.cuh"
#include "ffn_elem.cuh"
#include "ffn_gemm.cuh"
#include "ffn_gemv.cuh"
#include "host.cuh"

namespace poot_host {
cudaError_t take_ffn_device_error(unsigned int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, poot::g_device_error, sizeof(*word));
  if (e != cudaSuccess || *word == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(poot::g_device_error, &zero, sizeof(zero));
}
}  // namespace poot_host

namespace {

using namespace poot;
using namespace poot_host;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int kMaxDevices = 64;

struct FfnDevice {
  bool ready = false;
  int status = POOT_OK;
  int dev = 0;
  int sms = 0;
};
std::mutex g_mu;
FfnDevice g_devices[kMaxDevices];

template <int CL, int KIND>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(ffn_gemm_kernel<CL, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              FfnLayout::DYN_BYTES);
}

template <int NT, int DT>
cudaError_t set_gemv_attr() {
  return cudaFuncSetAttribute(gated_gemv_kernel<NT, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              gg_smem_bytes(NT));
}

int ffn_device(FfnDevice** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return POOT_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_mu);
  FfnDevice& d = g_devices[dev];
  if (!d.ready) {
    const int q = device_query(dev, &d.sms);
    if (q == POOT_ERR_CUDA) return q;
    if (q == POOT_OK &&
        ((e = set_attr<1, kFfnGated>()) != cudaSuccess || (e = set_attr<2, kFfnGated>()) != cudaSuccess ||
         (e = set_attr<1, kFfnDx>()) != cudaSuccess || (e = set_attr<2, kFfnDx>()) != cudaSuccess ||
         (e = set_attr<1, kFfnDw>()) != cudaSuccess || (e = set_attr<2, kFfnDw>()) != cudaSuccess ||
         (e = set_gemv_attr<1, kEpiF16>()) != cudaSuccess || (e = set_gemv_attr<1, kEpiBf16>()) != cudaSuccess ||
         (e = set_gemv_attr<2, kEpiF16>()) != cudaSuccess || (e = set_gemv_attr<2, kEpiBf16>()) != cudaSuccess))
      return cuda_fail(e);
    d.dev = dev;
    d.status = q;
    d.ready = true;
  }
  *out = &d;
  return d.status;
}

inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t ceil8(int64_t v) { return (v + 7) / 8 * 8; }
inline unsigned grid_for(int64_t units, int sms) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(units, 256), int64_t(sms) * 8)));
}

// ---- argument checks ---------------------------------------------------------
struct Span {
  const void* p;
  int64_t bytes;
};

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && M <= kMaxDim && N <= kMaxDim && K <= kMaxDim;
}

// bytes of a [rows, cols] matrix of 2-byte elements, rows ld apart
int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld) {
  return rows <= 0 || cols <= 0 ? 0 : 2 * ((rows - 1) * ld + cols);
}

// outputs may overlap neither an input nor one another; 2-byte alignment
int check_spans(std::initializer_list<Span> in, std::initializer_list<Span> out) {
  for (const auto& v : {in, out})
    for (const Span& s : v)
      if (s.p != nullptr && !aligned(s.p, 2)) return POOT_ERR_MISALIGNED;
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    for (const Span& s : in)
      if (overlaps(o->p, o->bytes, s.p, s.bytes)) return POOT_ERR_INVALID_ARG;
    for (const Span* q = out.begin(); q != o; ++q)
      if (overlaps(o->p, o->bytes, q->p, q->bytes)) return POOT_ERR_INVALID_ARG;
  }
  return POOT_OK;
}

// ---- operands ------------------------------------------------------------------
// A matrix as TMA reads it: base 16-byte aligned, pitch a multiple of 8.
struct Operand {
  const void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  bool tma() const { return aligned(p, 16) && ld % 8 == 0; }
};

// Collects the operands that need repacking; `place` lays the copies out from
// `base` and rewrites the operands, `launch_pack` queues the copy.
struct Packer {
  FfnPackArgs a;
  Operand* ops[4];
  size_t bytes = 0;
  Packer() { std::memset(&a, 0, sizeof(a)); }
  void need(Operand* o) {
    if (o->p == nullptr || o->tma()) return;
    const int t = a.count++;
    ops[t] = o;
    a.src[t] = static_cast<const uint16_t*>(o->p);
    a.ld[t] = o->ld;
    a.ldd[t] = ceil8(o->cols);
    a.rows[t] = o->rows;
    a.cols[t] = static_cast<int>(o->cols);
    bytes += round256(size_t(o->rows) * a.ldd[t] * 2);
  }
  void place(char* base) {
    for (int t = 0; t < a.count; ++t) {
      a.dst[t] = reinterpret_cast<uint16_t*>(base);
      ops[t]->p = base;
      ops[t]->ld = a.ldd[t];
      base += round256(size_t(a.rows[t]) * a.ldd[t] * 2);
    }
  }
  cudaError_t run(int sms, cudaStream_t stream) const {
    if (a.count == 0) return cudaSuccess;
    int64_t most = 0;
    for (int t = 0; t < a.count; ++t) most = std::max<int64_t>(most, a.rows[t] * (a.ldd[t] / 8));
    return launch(ffn_pack_kernel, dim3(grid_for(most, sms)), dim3(256), 0, stream, a);
  }
};

// ---- tile plan -------------------------------------------------------------------
struct FfnPlan {
  int cl, bn, split;
};

// Cost model: every CTA (pair) runs ceil(tiles / slots) tiles; a 64-element K
// block of a 128-row tile takes max(2 bn, 128 + bn) cycles of MMA or operand
// reads, divided by the efficiency of the shape; plus a fixed fill and drain.
// A split over K adds the second kernel and its bytes.
FfnPlan plan_ffn(int64_t rows, int64_t cols, int64_t kb, int outputs, bool gated, int sms) {
  static const struct { int cl, bn, eff; } shapes[] = {{2, 256, 100}, {2, 128, 80}, {1, 256, 85}, {1, 128, 70}, {1, 64, 55}};
  FfnPlan best = {1, 64, 1};
  int64_t best_cost = INT64_MAX;
  for (const auto& s : shapes) {
    const int64_t width = gated ? s.bn / 2 : s.bn;
    const int64_t tiles = ceil_div(rows, 128 * s.cl) * ceil_div(cols, width) * outputs;
    const int64_t slots = s.cl == 2 ? sms / 2 : sms;
    const int64_t per_kb = std::max<int64_t>(2 * s.bn, 128 + s.bn);
    for (int S = 1; S <= 16; ++S) {
      if (S > 1 && (kb / S < 8 || tiles * S > 2 * slots)) break;
      const int64_t waves = ceil_div(tiles * S, slots);
      int64_t cost = waves * (ceil_div(kb, S) * per_kb * 100 / s.eff + 1500) + (s.cl == 2 ? 1500 : 0);
      if (S > 1) cost += 6000 + S * rows * cols * outputs * (gated ? 2 : 1) * 4 / 2048;
      if (cost < best_cost) { best_cost = cost; best = {s.cl, s.bn, S}; }
    }
  }
  return best;
}

struct FfnCall {
  int kind;
  Operand a[2], b[2];
  int parts = 1;    // kFfnDx: products in one sum
  int outputs = 1;  // kFfnDw: outputs
  int64_t rows = 0, cols = 0, kext = 0;  // of one output; K extent of one part
  void* y[3] = {nullptr, nullptr, nullptr};
  const void* bias[2] = {nullptr, nullptr};
  int dtype = 0, act = 0, save = 0;
  FfnPlan plan;

  void make_plan(int sms) {
    plan = plan_ffn(rows, cols, ceil_div(kext, kFfnBK) * parts, outputs, kind == kFfnGated, sms);
  }
  size_t partial_bytes() const {
    return plan.split > 1 ? size_t(plan.split) * (kind == kFfnGated ? 2 : outputs) * rows * cols * 4 : 0;
  }
};

template <int CL, int KIND>
cudaError_t launch_ffn(const FfnMaps& m, const FfnGemmArgs& a, int sms, cudaStream_t stream) {
  const int64_t units = std::min<int64_t>(a.num_tiles, sms / CL);
  return launch_clustered(ffn_gemm_kernel<CL, KIND>, dim3(static_cast<unsigned>(units * CL)), dim3(kFfnThreads),
                          FfnLayout::DYN_BYTES, stream, unsigned(CL), m, a);
}

int run_ffn_gemm(const FfnCall& c, const FfnDevice& d, float* partial, cudaStream_t stream) {
  const FfnPlan& p = c.plan;
  const bool gated = c.kind == kFfnGated, bf16 = c.dtype == POOT_DTYPE_BF16;
  const bool a_mn = c.kind == kFfnDw, b_mn = !gated;
  FfnGemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.M = static_cast<int>(c.rows);
  a.N = static_cast<int>(c.cols);
  a.bn = p.bn;
  a.cols = gated ? p.bn / 2 : p.bn;
  a.stages = ffn_stages(p.cl, p.bn);
  a.num_m_blocks = static_cast<int>(ceil_div(c.rows, kFfnBM * p.cl));
  a.num_n_blocks = static_cast<int>(ceil_div(c.cols, a.cols));
  const int64_t bk = kFfnBK * ffn_sub(p.cl);
  a.kb_part = static_cast<int>(ceil_div(c.kext, bk));
  if (int64_t(a.kb_part) * c.parts > INT32_MAX) return POOT_ERR_INVALID_ARG;
  a.kb_total = a.kb_part * c.parts;
  a.kb_split = static_cast<int>(ceil_div(a.kb_total, p.split));
  a.split = static_cast<int>(ceil_div(a.kb_total, a.kb_split));  // no empty range
  // M blocks walked together: their A rows within 32 MB of L2, and at least
  // eight, about the square of tiles that run at one time
  int64_t group = (int64_t(32) << 20) / (2 * c.kext * c.parts * kFfnBM * p.cl);
  group = std::max<int64_t>(8, std::min<int64_t>(group, 64));
  a.group_m = static_cast<int>(std::min<int64_t>(group, a.num_m_blocks));
  const int64_t tpg = int64_t(a.num_m_blocks) * a.num_n_blocks;
  const int64_t tiles = tpg * c.outputs * a.split;
  if (tiles > INT32_MAX) return POOT_ERR_INVALID_ARG;
  a.tiles_per_group = static_cast<int>(tpg);
  a.num_tiles = static_cast<int>(tiles);
  a.dtype = c.dtype;
  a.act = c.act;
  a.save = c.save;
  a.partial = a.split > 1 ? partial : nullptr;
  const int ny = gated ? (c.save ? 3 : 1) : c.outputs;
  a.tma_store = a.split == 1 && c.cols % 8 == 0;
  for (int i = 0; i < ny; ++i) {
    a.y[i] = static_cast<uint16_t*>(c.y[i]);
    if (!aligned(c.y[i], 16)) a.tma_store = 0;
  }
  for (int i = 0; i < 2; ++i) a.bias[i] = static_cast<const uint16_t*>(c.bias[i]);

  FfnMaps m;
  std::memset(&m, 0, sizeof(m));
  const int na = c.kind == kFfnDx ? c.parts : (c.kind == kFfnDw ? c.outputs : 1);
  const int nbm = gated ? 2 : (c.kind == kFfnDx ? c.parts : 1);
  auto encode = [&](CUtensorMap* map, const Operand& o, bool mn, int rows) {
    return encode_2d(map, o.p, o.cols, o.rows, kFfnBK, mn ? kFfnBK : static_cast<uint32_t>(rows),
                     CU_TENSOR_MAP_SWIZZLE_128B, bf16, o.ld);
  };
  for (int i = 0; i < na; ++i)
    if (!encode(&m.a[i], c.a[i], a_mn, kFfnBM)) return cuda_fail(cudaErrorInvalidValue);
  for (int i = 0; i < nbm; ++i)
    if (!encode(&m.b[i], c.b[i], b_mn, p.bn / 2)) return cuda_fail(cudaErrorInvalidValue);
  if (a.tma_store)
    for (int i = 0; i < ny; ++i)
      if (!encode_2d(&m.y[i], c.y[i], c.cols, c.rows, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, bf16))
        return cuda_fail(cudaErrorInvalidValue);
  cudaError_t e;
  const bool pair = p.cl == 2;
  switch (c.kind) {
    case kFfnGated: e = pair ? launch_ffn<2, kFfnGated>(m, a, d.sms, stream) : launch_ffn<1, kFfnGated>(m, a, d.sms, stream); break;
    case kFfnDx: e = pair ? launch_ffn<2, kFfnDx>(m, a, d.sms, stream) : launch_ffn<1, kFfnDx>(m, a, d.sms, stream); break;
    default: e = pair ? launch_ffn<2, kFfnDw>(m, a, d.sms, stream) : launch_ffn<1, kFfnDw>(m, a, d.sms, stream); break;
  }
  if (e != cudaSuccess) return cuda_fail(e);
  if (a.split > 1) {
    FfnReduceArgs r;
    std::memset(&r, 0, sizeof(r));
    r.ws = partial;
    for (int i = 0; i < 3; ++i) r.y[i] = i < ny ? static_cast<uint16_t*>(c.y[i]) : nullptr;
    for (int i = 0; i < 2; ++i) r.bias[i] = a.bias[i];
    r.MN = c.rows * c.cols;
    r.S = a.split;
    r.N = a.N;
    r.outputs = c.outputs;
    r.dtype = c.dtype;
    r.act = c.act;
    r.gated = gated;
    e = launch(ffn_reduce_kernel, dim3(grid_for(r.MN * c.outputs / (c.cols % 4 == 0 ? 4 : 1), d.sms)), dim3(256), 0,
               stream, r);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return POOT_OK;
}

int finish(WorkspaceLease& lease, int rc) {
  const cudaError_t e = lease.release();
  if (rc != POOT_OK) return rc;
  return e == cudaSuccess ? POOT_OK : cuda_fail(e);
}

// ---- the gated block ------------------------------------------------------------
template <int NT>
cudaError_t launch_gated_gemv(const GatedGemvArgs& a, bool bf16, bool vec, int sms, cudaStream_t stream) {
  if (vec) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(sms, a.N)));
    return launch(bf16 ? gated_gemv_kernel<NT, kEpiBf16> : gated_gemv_kernel<NT, kEpiF16>, grid, dim3(kGgWarps * 32),
                  gg_smem_bytes(NT), stream, a);
  }
  const int64_t tiles = ceil_div(a.N, 16);
  const dim3 grid(static_cast<unsigned>(tiles));
  if (tiles < 2 * int64_t(sms))
    return launch(bf16 ? gated_gemv_any_kernel<NT, 16, kEpiBf16> : gated_gemv_any_kernel<NT, 16, kEpiF16>, grid,
                  dim3(16 * 32), 0, stream, a);
  return launch(bf16 ? gated_gemv_any_kernel<NT, 8, kEpiBf16> : gated_gemv_any_kernel<NT, 8, kEpiF16>, grid,
                dim3(8 * 32), 0, stream, a);
}

int gated_gemv(const poot_gated_linear_args& p, int64_t ldx, const FfnDevice& d, cudaStream_t stream) {
  GatedGemvArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = static_cast<const uint16_t*>(p.x);
  a.wg = static_cast<const uint16_t*>(p.wg);
  a.wu = static_cast<const uint16_t*>(p.wu);
  a.bias[0] = static_cast<const uint16_t*>(p.bg);
  a.bias[1] = static_cast<const uint16_t*>(p.bu);
  a.y[0] = static_cast<uint16_t*>(p.h);
  a.y[1] = static_cast<uint16_t*>(p.g);
  a.y[2] = static_cast<uint16_t*>(p.u);
  a.ldx = ldx;
  a.M = static_cast<int>(p.M);
  a.N = static_cast<int>(p.N);
  a.K = static_cast<int>(p.K);
  a.act = p.activation;
  a.save = p.g != nullptr;
  // Warps that split K: never more than there are ring slots of K; and, as
  // far as the block has a pass for each team, so few that a warp's share of a
  // pass is four slots (8 x 8192 x 2048 on GB300: 16.3 us with two slots, 14.1
  // with four)
  const int64_t passes = ceil_div(ceil_div(p.N, std::min<int64_t>(d.sms, p.N)), 8 * kGgSub);
  a.kw = kGgWarps;
  while (a.kw > 1 && (a.kw / 2 * 32 * kGgSteps >= p.K ||
                      (p.K < a.kw * 128 * kGgSteps && 2 * kGgWarps / a.kw <= passes)))
    a.kw /= 2;
  const bool bf16 = p.dtype == POOT_DTYPE_BF16;
  const bool vec = p.K % 8 == 0 && ldx % 8 == 0 && aligned(p.x, 16) && aligned(p.wg, 16) && aligned(p.wu, 16);
  const cudaError_t e = p.M <= 8 ? launch_gated_gemv<1>(a, bf16, vec, d.sms, stream)
                                 : launch_gated_gemv<2>(a, bf16, vec, d.sms, stream);
  return e == cudaSuccess ? POOT_OK : cuda_fail(e);
}

int gated_linear(const poot_gated_linear_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_gated_linear_args& p = *ap;
  const int64_t M = p.M, N = p.N, K = p.K, ldx = p.ldx != 0 ? p.ldx : K;
  if (!sizes_ok(M, N, K) || ldx < K || (p.dtype != POOT_DTYPE_F16 && p.dtype != POOT_DTYPE_BF16) ||
      p.activation < POOT_ACT_SILU || p.activation > POOT_ACT_GELU_ERF || (p.g == nullptr) != (p.u == nullptr))
    return POOT_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return POOT_OK;
  if (p.h == nullptr || (K > 0 && (p.x == nullptr || p.wg == nullptr || p.wu == nullptr))) return POOT_ERR_INVALID_ARG;
  const int64_t out = span_bytes(M, N, N), wb = span_bytes(N, K, K);
  const int rc = check_spans({{p.x, span_bytes(M, K, ldx)}, {p.wg, wb}, {p.wu, wb}, {p.bg, 2 * N}, {p.bu, 2 * N}},
                             {{p.h, out}, {p.g, out}, {p.u, out}});
  if (rc != POOT_OK) return rc;
  FfnDevice* d;
  const int st = ffn_device(&d);
  if (st != POOT_OK) return st;
  if (K == 0) {
    FfnReduceArgs r;
    std::memset(&r, 0, sizeof(r));
    r.y[0] = static_cast<uint16_t*>(p.h);
    r.y[1] = static_cast<uint16_t*>(p.g);
    r.y[2] = static_cast<uint16_t*>(p.u);
    r.bias[0] = static_cast<const uint16_t*>(p.bg);
    r.bias[1] = static_cast<const uint16_t*>(p.bu);
    r.MN = M * N;
    r.N = static_cast<int>(N);
    r.dtype = p.dtype;
    r.act = p.activation;
    const cudaError_t e = launch(gated_bias_kernel, dim3(grid_for(M * N, d->sms)), dim3(256), 0, stream, r);
    return e == cudaSuccess ? POOT_OK : cuda_fail(e);
  }
  if (M <= POOT_GEMV_MAX_M) return gated_gemv(p, ldx, *d, stream);
  FfnCall c;
  c.kind = kFfnGated;
  c.a[0] = {p.x, M, K, ldx};
  c.b[0] = {p.wg, N, K, K};
  c.b[1] = {p.wu, N, K, K};
  c.rows = M;
  c.cols = N;
  c.kext = K;
  c.y[0] = p.h;
  c.y[1] = p.g;
  c.y[2] = p.u;
  c.bias[0] = p.bg;
  c.bias[1] = p.bu;
  c.dtype = p.dtype;
  c.act = p.activation;
  c.save = p.g != nullptr;
  c.make_plan(d->sms);
  Packer pk;
  pk.need(&c.a[0]);
  pk.need(&c.b[0]);
  pk.need(&c.b[1]);
  const size_t partial = round256(c.partial_bytes());
  WorkspaceLease lease;
  if (partial + pk.bytes > 0) {
    lease = stream_workspace(d->dev, stream, partial + pk.bytes);
    if (lease.ptr == nullptr) return cuda_fail(cudaErrorMemoryAllocation);
  }
  char* ws = static_cast<char*>(lease.ptr);
  pk.place(ws + partial);
  const cudaError_t e = pk.run(d->sms, stream);
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  return finish(lease, run_ffn_gemm(c, *d, reinterpret_cast<float*>(ws), stream));
}

int zero(void* p, int64_t bytes, cudaStream_t stream) {
  if (p == nullptr || bytes == 0) return POOT_OK;
  const cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), stream);
  return e == cudaSuccess ? POOT_OK : cuda_fail(e);
}

// The products behind dx and dw: D_q (one or two, TMA-readable) with W_q and x.
struct Grads {
  int count;            // D matrices
  Operand d[2], w[2], x;
  void* dx;
  void* dw[2];
  int64_t M, N, K;
  int dtype;

  FfnCall dx_call, dw_call;
  int ndw = 0;

  void plan(int sms, Packer* pk) {
    if (dx != nullptr && K > 0) {
      FfnCall& c = dx_call;
      c.kind = kFfnDx;
      c.parts = count;
      c.rows = M;
      c.cols = K;
      c.kext = N;
      c.y[0] = dx;
      c.dtype = dtype;
      c.make_plan(sms);
      for (int i = 0; i < count; ++i) pk->need(&w[i]);
    }
    for (int i = 0; i < count; ++i) ndw += dw[i] != nullptr;
    if (K == 0) ndw = 0;
    if (ndw > 0) {
      FfnCall& c = dw_call;
      c.kind = kFfnDw;
      c.outputs = ndw;
      c.rows = N;
      c.cols = K;
      c.kext = M;
      c.dtype = dtype;
      c.make_plan(sms);
      pk->need(&x);
    }
  }
  size_t partial_bytes() const {
    return round256(std::max(dx != nullptr && K > 0 ? dx_call.partial_bytes() : 0, ndw > 0 ? dw_call.partial_bytes() : 0));
  }
  int run(const FfnDevice& dev, float* partial, cudaStream_t stream) {
    if (dx != nullptr && K > 0) {
      for (int i = 0; i < count; ++i) {
        dx_call.a[i] = d[i];
        dx_call.b[i] = w[i];
      }
      const int rc = run_ffn_gemm(dx_call, dev, partial, stream);
      if (rc != POOT_OK) return rc;
    }
    if (ndw > 0) {
      int o = 0;
      for (int i = 0; i < count; ++i) {
        if (dw[i] == nullptr) continue;
        dw_call.a[o] = d[i];
        dw_call.y[o] = dw[i];
        ++o;
      }
      dw_call.b[0] = x;
      return run_ffn_gemm(dw_call, dev, partial, stream);
    }
    return POOT_OK;
  }
};

cudaError_t finish_columns(const float* colsum, int64_t blocks, int outputs, int64_t N, int dtype, void* o0, void* o1,
                           cudaStream_t stream) {
  ColFinishArgs f;
  f.colsum = colsum;
  f.out[0] = static_cast<uint16_t*>(o0);
  f.out[1] = static_cast<uint16_t*>(o1);
  f.blocks = static_cast<int>(blocks);
  f.outputs = outputs;
  f.N = static_cast<int>(N);
  f.dtype = dtype;
  return launch(col_finish_kernel, dim3(static_cast<unsigned>(ceil_div(outputs * N, 256))), dim3(256), 0, stream, f);
}

int gated_linear_backward(const poot_gated_linear_backward_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_gated_linear_backward_args& p = *ap;
  const int64_t M = p.M, N = p.N, K = p.K;
  const int64_t ldx = p.ldx != 0 ? p.ldx : K, ld_dh = p.ld_dh != 0 ? p.ld_dh : N, ld_g = p.ld_g != 0 ? p.ld_g : N,
                ld_u = p.ld_u != 0 ? p.ld_u : N;
  if (!sizes_ok(M, N, K) || ldx < K || ld_dh < N || ld_g < N || ld_u < N ||
      (p.dtype != POOT_DTYPE_F16 && p.dtype != POOT_DTYPE_BF16) || p.activation < POOT_ACT_SILU ||
      p.activation > POOT_ACT_GELU_ERF)
    return POOT_ERR_INVALID_ARG;
  const bool want_dw = p.dwg != nullptr || p.dwu != nullptr, want_db = p.dbg != nullptr || p.dbu != nullptr;
  if (M > 0 && N > 0 && (p.dx != nullptr || want_dw || want_db)) {
    if (p.dh == nullptr || p.g == nullptr || p.u == nullptr) return POOT_ERR_INVALID_ARG;
    if (K > 0 && p.dx != nullptr && (p.wg == nullptr || p.wu == nullptr)) return POOT_ERR_INVALID_ARG;
    if (K > 0 && want_dw && p.x == nullptr) return POOT_ERR_INVALID_ARG;
  }
  const int64_t wb = span_bytes(N, K, K);
  const int rc = check_spans({{p.dh, span_bytes(M, N, ld_dh)},
                              {p.x, span_bytes(M, K, ldx)},
                              {p.wg, wb},
                              {p.wu, wb},
                              {p.g, span_bytes(M, N, ld_g)},
                              {p.u, span_bytes(M, N, ld_u)}},
                             {{p.dx, span_bytes(M, K, K)}, {p.dwg, wb}, {p.dwu, wb}, {p.dbg, 2 * N}, {p.dbu, 2 * N}});
  if (rc != POOT_OK) return rc;
  if (p.dx == nullptr && !want_dw && !want_db) return POOT_OK;
  FfnDevice* d;
  const int st = ffn_device(&d);
  if (st != POOT_OK) return st;
  if (M == 0 || N == 0) {
    int z = POOT_OK;
    for (const Span& s : {Span{p.dx, span_bytes(M, K, K)}, Span{p.dwg, wb}, Span{p.dwu, wb}, Span{p.dbg, 2 * N},
                          Span{p.dbu, 2 * N}})
      if (z == POOT_OK) z = zero(const_cast<void*>(s.p), s.bytes, stream);
    return z;
  }
  Grads g;
  g.count = 2;
  g.w[0] = {p.wg, N, K, K};
  g.w[1] = {p.wu, N, K, K};
  g.x = {p.x, M, K, ldx};
  g.dx = p.dx;
  g.dw[0] = p.dwg;
  g.dw[1] = p.dwu;
  g.M = M;
  g.N = N;
  g.K = K;
  g.dtype = p.dtype;
  Packer pk;
  g.plan(d->sms, &pk);
  const int64_t Np = ceil8(N), row_blocks = ceil_div(M, kColRows);
  if (ceil_div(N, kColWidth) * row_blocks > INT32_MAX) return POOT_ERR_INVALID_ARG;
  const size_t dbytes = round256(size_t(M) * Np * 2), partial = g.partial_bytes();
  const size_t cbytes = want_db ? round256(size_t(row_blocks) * 2 * N * 4) : 0;
  WorkspaceLease lease = stream_workspace(d->dev, stream, 2 * dbytes + partial + cbytes + pk.bytes);
  if (lease.ptr == nullptr) return cuda_fail(cudaErrorMemoryAllocation);
  char* ws = static_cast<char*>(lease.ptr);
  g.d[0] = {ws, M, N, Np};
  g.d[1] = {ws + dbytes, M, N, Np};
  float* const part = reinterpret_cast<float*>(ws + 2 * dbytes);
  float* const colsum = reinterpret_cast<float*>(ws + 2 * dbytes + partial);
  pk.place(ws + 2 * dbytes + partial + cbytes);
  cudaError_t e = pk.run(d->sms, stream);
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  GateGradArgs ga;
  ga.dh = static_cast<const uint16_t*>(p.dh);
  ga.g = static_cast<const uint16_t*>(p.g);
  ga.u = static_cast<const uint16_t*>(p.u);
  ga.ld_dh = ld_dh;
  ga.ld_g = ld_g;
  ga.ld_u = ld_u;
  ga.dg = reinterpret_cast<uint16_t*>(ws);
  ga.du = reinterpret_cast<uint16_t*>(ws + dbytes);
  ga.ldo = Np;
  ga.colsum = want_db ? colsum : nullptr;
  ga.M = static_cast<int>(M);
  ga.N = static_cast<int>(N);
  ga.act = p.activation;
  const dim3 grid(static_cast<unsigned>(ceil_div(N, kColWidth) * row_blocks));
  const bool bf16 = p.dtype == POOT_DTYPE_BF16;
  auto kern = bf16 ? (want_db ? gate_grad_kernel<kEpiBf16, true> : gate_grad_kernel<kEpiBf16, false>)
                   : (want_db ? gate_grad_kernel<kEpiF16, true> : gate_grad_kernel<kEpiF16, false>);
  e = launch(kern, grid, dim3(kColThreads), 0, stream, ga);
  if (e == cudaSuccess && want_db)
    e = finish_columns(colsum, row_blocks, 2, N, p.dtype, p.dbg, p.dbu, stream);
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  return finish(lease, g.run(*d, part, stream));
}

int linear_backward(const poot_linear_backward_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_linear_backward_args& p = *ap;
  const int64_t M = p.M, N = p.N, K = p.K;
  const int64_t ldx = p.ldx != 0 ? p.ldx : K, ld_dy = p.ld_dy != 0 ? p.ld_dy : N;
  if (!sizes_ok(M, N, K) || ldx < K || ld_dy < N || (p.dtype != POOT_DTYPE_F16 && p.dtype != POOT_DTYPE_BF16))
    return POOT_ERR_INVALID_ARG;
  if (M > 0 && N > 0 && (p.dx != nullptr || p.dw != nullptr || p.db != nullptr)) {
    if (p.dy == nullptr || (K > 0 && p.dx != nullptr && p.w == nullptr) || (K > 0 && p.dw != nullptr && p.x == nullptr))
      return POOT_ERR_INVALID_ARG;
  }
  const int64_t wb = span_bytes(N, K, K);
  const int rc = check_spans({{p.dy, span_bytes(M, N, ld_dy)}, {p.x, span_bytes(M, K, ldx)}, {p.w, wb}},
                             {{p.dx, span_bytes(M, K, K)}, {p.dw, wb}, {p.db, 2 * N}});
  if (rc != POOT_OK) return rc;
  if (p.dx == nullptr && p.dw == nullptr && p.db == nullptr) return POOT_OK;
  FfnDevice* d;
  const int st = ffn_device(&d);
  if (st != POOT_OK) return st;
  if (M == 0 || N == 0) {
    int z = zero(p.dx, span_bytes(M, K, K), stream);
    if (z == POOT_OK) z = zero(p.dw, wb, stream);
    return z == POOT_OK ? zero(p.db, 2 * N, stream) : z;
  }
  Grads g;
  g.count = 1;
  g.d[0] = {p.dy, M, N, ld_dy};
  g.w[0] = {p.w, N, K, K};
  g.x = {p.x, M, K, ldx};
  g.dx = p.dx;
  g.dw[0] = p.dw;
  g.dw[1] = nullptr;
  g.M = M;
  g.N = N;
  g.K = K;
  g.dtype = p.dtype;
  Packer pk;
  g.plan(d->sms, &pk);
  if (K > 0 && (p.dx != nullptr || p.dw != nullptr)) pk.need(&g.d[0]);
  const int64_t row_blocks = ceil_div(M, kColRows);
  if (ceil_div(N, kColWidth) * row_blocks > INT32_MAX) return POOT_ERR_INVALID_ARG;
  const size_t partial = g.partial_bytes();
  const size_t cbytes = p.db != nullptr ? round256(size_t(row_blocks) * N * 4) : 0;
  WorkspaceLease lease;
  if (partial + cbytes + pk.bytes > 0) {
    lease = stream_workspace(d->dev, stream, partial + cbytes + pk.bytes);
    if (lease.ptr == nullptr) return cuda_fail(cudaErrorMemoryAllocation);
  }
  char* ws = static_cast<char*>(lease.ptr);
  pk.place(ws + partial + cbytes);
  cudaError_t e = pk.run(d->sms, stream);
  if (e == cudaSuccess && p.db != nullptr) {
    ColSumArgs ca;
    ca.d = static_cast<const uint16_t*>(p.dy);
    ca.ld = ld_dy;
    ca.colsum = reinterpret_cast<float*>(ws + partial);
    ca.M = static_cast<int>(M);
    ca.N = static_cast<int>(N);
    const dim3 grid(static_cast<unsigned>(ceil_div(N, kColWidth) * row_blocks));
    e = launch(p.dtype == POOT_DTYPE_BF16 ? col_sum_kernel<kEpiBf16> : col_sum_kernel<kEpiF16>, grid, dim3(kColThreads),
               0, stream, ca);
    if (e == cudaSuccess) e = finish_columns(ca.colsum, row_blocks, 1, N, p.dtype, p.db, nullptr, stream);
  }
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  return finish(lease, g.run(*d, reinterpret_cast<float*>(ws), stream));
}

// ---- clipping ----------------------------------------------------------------------
int clip_grad_norm(const poot_grad_tensor* t, int64_t count, float max_norm, float* norm, cudaStream_t stream) {
  if (count < 0 || count > kMaxDim || norm == nullptr || (count > 0 && t == nullptr) || !(max_norm >= 0.0f))
    return POOT_ERR_INVALID_ARG;
  if (!aligned(norm, 4)) return POOT_ERR_MISALIGNED;
  struct Range {
    uintptr_t lo, hi;
    int64_t index;  // -1: the norm
    bool write;
  };
  std::vector<Range> ranges;
  ranges.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + 4, -1, true});
  int64_t pieces_all = 0;
  for (int64_t i = 0; i < count; ++i) {
    const poot_grad_tensor& g = t[i];
    if (g.dtype < POOT_GRAD_F16 || g.dtype > POOT_GRAD_F32 || g.n < 0 || g.n > (int64_t(1) << 40))
      return POOT_ERR_INVALID_ARG;
    if (g.n == 0) continue;
    if (g.src == nullptr || g.dst == nullptr) return POOT_ERR_INVALID_ARG;
    const int size = g.dtype == POOT_GRAD_F32 ? 4 : 2;
    if (!aligned(g.src, size) || !aligned(g.dst, size)) return POOT_ERR_MISALIGNED;
    const uintptr_t s = reinterpret_cast<uintptr_t>(g.src), o = reinterpret_cast<uintptr_t>(g.dst);
    ranges.push_back({s, s + uintptr_t(g.n) * size, i, g.src == g.dst});
    if (g.src != g.dst) ranges.push_back({o, o + uintptr_t(g.n) * size, i, true});
    pieces_all += ceil_div(g.n, kClipPieceBytes / size);
  }
  if (pieces_all > INT32_MAX) return POOT_ERR_INVALID_ARG;
  // a written range overlaps nothing else: sorted by start, every range that
  // reaches past a later one's start conflicts if either is written
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end_any = 0, end_written = 0;
  for (const Range& r : ranges) {
    if (r.lo < end_written || (r.write && r.lo < end_any)) return POOT_ERR_INVALID_ARG;
    end_any = std::max(end_any, r.hi);
    if (r.write) end_written = std::max(end_written, r.hi);
  }
  FfnDevice* d;
  const int st = ffn_device(&d);
  if (st != POOT_OK) return st;
  const int max_blocks = d->sms * 4;
  const int64_t launches = std::max<int64_t>(1, ceil_div(count, kClipTable));
  WorkspaceLease lease = stream_workspace(d->dev, stream, size_t(launches) * max_blocks * sizeof(double));
  if (lease.ptr == nullptr) return cuda_fail(cudaErrorMemoryAllocation);
  ClipArgs a;
  a.partial = static_cast<double*>(lease.ptr);
  a.max_norm = max_norm;
  a.norm = norm;
  a.write_norm = 0;
  a.part0 = 0;
  a.parts = 0;
  ClipTable table;
  auto fill = [&](int64_t first) {
    int64_t k = first;
    table.count = 0;
    table.first[0] = 0;
    for (; k < count && table.count < kClipTable; ++k) {
      const poot_grad_tensor& g = t[k];
      if (g.n == 0) continue;
      const int i = table.count++;
      table.src[i] = g.src;
      table.dst[i] = g.dst;
      table.n[i] = g.n;
      table.dtype[i] = static_cast<unsigned char>(g.dtype);
      table.first[i + 1] =
          table.first[i] + static_cast<int>(ceil_div(g.n, kClipPieceBytes / (g.dtype == POOT_GRAD_F32 ? 4 : 2)));
    }
    return k;
  };
  auto blocks_for = [&]() {
    return static_cast<unsigned>(std::max(1, std::min(table.first[table.count], max_blocks)));
  };
  cudaError_t e = cudaSuccess;
  bool more = true;
  for (int64_t k = 0; more && e == cudaSuccess;) {
    k = fill(k);
    more = k < count;
    const unsigned blocks = blocks_for();
    a.part0 = a.parts;
    e = launch(clip_sum_kernel, dim3(blocks), dim3(kClipThreads), 0, stream, table, a);
    a.parts += static_cast<int>(blocks);
  }
  more = true;
  for (int64_t k = 0; more && e == cudaSuccess;) {
    const bool single = count <= kClipTable;  // the table still holds the one launch's tensors
    a.write_norm = k == 0;
    k = single ? count : fill(k);
    more = k < count;
    e = launch(clip_scale_kernel, dim3(blocks_for()), dim3(kClipThreads), 0, stream, table, a);
  }
  return finish(lease, e == cudaSuccess ? POOT_OK : cuda_fail(e));
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

int poot_gated_linear(const poot_gated_linear_args* args, poot_stream_t stream) {
  return guarded([&] { return gated_linear(args, reinterpret_cast<cudaStream_t>(stream)); });
}

int poot_gated_linear_backward(const poot_gated_linear_backward_args* args, poot_stream_t stream) {
  return guarded([&] { return gated_linear_backward(args, reinterpret_cast<cudaStream_t>(stream)); });
}

int poot_linear_backward(const poot_linear_backward_args* args, poot_stream_t stream) {
  return guarded([&] { return linear_backward(args, reinterpret_cast<cudaStream_t>(stream)); });
}

int poot_clip_grad_norm(const poot_grad_tensor* tensors, int64_t count, float max_norm, float* norm,
                        poot_stream_t stream) {
  return guarded([&] { return clip_grad_norm(tensors, count, max_norm, norm, reinterpret_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
