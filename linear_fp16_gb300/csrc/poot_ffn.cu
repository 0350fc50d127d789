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
#include "ffn_plan.cuh"
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

constexpr int kMaxDevices = 64;

struct FfnDevice : DeviceInfo {
  bool ready = false;
  int status = POOT_OK;
  int clip_blocks = 0;  // blocks of the cooperative clip that run at one time
};
std::mutex g_mu;
FfnDevice g_devices[kMaxDevices];

template <int CL, bool GATED>
cudaError_t set_attr() {
  for (auto kernel : {ffn_gemm_kernel<CL, GATED, kEpiF16, false>, ffn_gemm_kernel<CL, GATED, kEpiF16, true>,
                      ffn_gemm_kernel<CL, GATED, kEpiBf16, false>, ffn_gemm_kernel<CL, GATED, kEpiBf16, true>}) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FfnLayout::DYN_BYTES);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int NT, int DT>
cudaError_t set_gemv_attr() {
  const cudaError_t e = cudaFuncSetAttribute(gated_gemv_kernel<NT, DT, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             gg_smem_bytes(NT, 16));
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(gated_gemv_kernel<NT, DT, 8>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, gg_smem_bytes(NT, 8));
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
        ((e = set_attr<1, true>()) != cudaSuccess || (e = set_attr<2, true>()) != cudaSuccess ||
         (e = set_attr<1, false>()) != cudaSuccess || (e = set_attr<2, false>()) != cudaSuccess ||
         (e = set_gemv_attr<1, kEpiF16>()) != cudaSuccess || (e = set_gemv_attr<1, kEpiBf16>()) != cudaSuccess ||
         (e = set_gemv_attr<2, kEpiF16>()) != cudaSuccess || (e = set_gemv_attr<2, kEpiBf16>()) != cudaSuccess))
      return cuda_fail(e);
    if (q == POOT_OK) {
      int few = 0, many = 0;
      if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&few, clip_kernel<kClipTableFew, kClipBoth>, kClipThreads,
                                                             0)) != cudaSuccess ||
          (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&many, clip_kernel<kClipTable, kClipBoth>, kClipThreads,
                                                             0)) != cudaSuccess)
        return cuda_fail(e);
      d.clip_blocks = std::min(std::min(few, many), kClipBlocksPerSm) * d.sms;
      if (d.clip_blocks == 0) return cuda_fail(cudaErrorCooperativeLaunchTooLarge);
    }
    d.dev = dev;
    d.status = q;
    d.ready = true;
  }
  *out = &d;
  return d.status;
}

template <int CL, bool GATED>
cudaError_t launch_ffn(const FfnMaps& m, const FfnGemmArgs& a, bool bf16, int64_t units, cudaStream_t stream) {
  auto pick = [&](auto chunks) {
    constexpr bool C = decltype(chunks)::value;
    return bf16 ? ffn_gemm_kernel<CL, GATED, kEpiBf16, C> : ffn_gemm_kernel<CL, GATED, kEpiF16, C>;
  };
  return launch_clustered(a.scratch != nullptr ? pick(std::true_type{}) : pick(std::false_type{}),
                          dim3(static_cast<unsigned>(units * CL)), dim3(ffn_threads(GATED)), FfnLayout::DYN_BYTES, stream,
                          unsigned(CL), m, a);
}

// The products of this unit's kernels (see ffn_plan.cuh).
int run_ffn_products(const FfnProduct* const* ps, int count, const FfnPlan& p, const FfnEpilogue& ep,
                     const FfnBiasGrad* bg, char* ws, const FfnDevice& d, cudaStream_t stream) {
  const bool gated = count > 0 && ps[0]->gated;
  return run_products(
      ps, count, p, ep, bg, ws, d,
      [&](const FfnMaps& m, const FfnGemmArgs& a, bool bf16, int64_t units) {
        const bool pair = p.cl == 2;
        if (gated)
          return pair ? launch_ffn<2, true>(m, a, bf16, units, stream) : launch_ffn<1, true>(m, a, bf16, units, stream);
        return pair ? launch_ffn<2, false>(m, a, bf16, units, stream) : launch_ffn<1, false>(m, a, bf16, units, stream);
      },
      [&](const FfnProduct& q, const FfnJob& j, const float* partial) {
        FfnReduceArgs r;
        std::memset(&r, 0, sizeof(r));
        r.ws = partial;
        for (int o = 0; o < 3; ++o) r.y[o] = j.y[o];
        for (int o = 0; o < 2; ++o) r.bias[o] = static_cast<const uint16_t*>(ep.bias[o]);
        r.M = q.rows;
        r.S = j.split;
        r.N = j.N;
        r.ldw = static_cast<int>(ceil_div(q.cols, 4) * 4);
        r.outputs = q.outputs;
        r.dtype = ep.dtype;
        r.act = ep.act;
        r.gated = q.gated;
        return launch(ffn_reduce_kernel, dim3(grid_for(r.M * (r.ldw / 4) * q.outputs, d.sms)), dim3(256), 0, stream, r);
      });
}

// ---- the gated block ------------------------------------------------------------
template <int NT, int WARPS>
cudaError_t launch_gated_gemv_vec(const GatedGemvArgs& a, bool bf16, unsigned blocks, cudaStream_t stream) {
  return launch(bf16 ? gated_gemv_kernel<NT, kEpiBf16, WARPS> : gated_gemv_kernel<NT, kEpiF16, WARPS>, dim3(blocks),
                dim3(WARPS * 32), gg_smem_bytes(NT, WARPS), stream, a);
}

template <int NT>
cudaError_t launch_gated_gemv(GatedGemvArgs a, bool bf16, bool vec, int sms, cudaStream_t stream) {
  if (vec) {
    const bool two = a.N >= 8 * 2 * sms;
    const int warps = two ? 8 : 16;
    const int64_t blocks = std::min<int64_t>(two ? 2 * sms : sms, a.N);
    // Warps that split K: never more than there are ring slots of K; and, as
    // far as the block has a pass for each team, so few that a warp's share of a
    // pass is four slots (8 x 8192 x 2048 on GB300: 16.3 us with two slots, 14.1
    // with four)
    const int64_t passes = ceil_div(ceil_div(a.N, blocks), 8 * kGgSub);
    a.kw = warps;
    while (a.kw > 1 && (a.kw / 2 * 32 * kGgSteps >= a.K ||
                        (a.K < a.kw * 128 * kGgSteps && 2 * warps / a.kw <= passes)))
      a.kw /= 2;
    return two ? launch_gated_gemv_vec<NT, 8>(a, bf16, static_cast<unsigned>(blocks), stream)
               : launch_gated_gemv_vec<NT, 16>(a, bf16, static_cast<unsigned>(blocks), stream);
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
  const bool bf16 = p.dtype == POOT_DTYPE_BF16;
  const bool vec = p.K % 8 == 0 && ldx % 8 == 0 && aligned(p.x, 16) && aligned(p.wg, 16) && aligned(p.wu, 16);
  const cudaError_t e = p.M <= 8 ? launch_gated_gemv<1>(a, bf16, vec, d.sms, stream)
                                 : launch_gated_gemv<2>(a, bf16, vec, d.sms, stream);
  return e == cudaSuccess ? POOT_OK : cuda_fail(e);
}

int gated_linear(const poot_gated_linear_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_gated_linear_args& p = *ap;
  const int64_t M = p.M, N = p.N, K = p.K;
  int64_t ldx;
  if (!sizes_ok(M, N, K) || !row_pitch(M, K, p.ldx, &ldx) ||
      (p.dtype != POOT_DTYPE_F16 && p.dtype != POOT_DTYPE_BF16) ||
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
    r.M = M;
    r.N = static_cast<int>(N);
    r.dtype = p.dtype;
    r.act = p.activation;
    const cudaError_t e = launch(gated_bias_kernel, dim3(grid_for(M * N, d->sms)), dim3(256), 0, stream, r);
    return e == cudaSuccess ? POOT_OK : cuda_fail(e);
  }
  if (M <= POOT_GEMV_MAX_M) return gated_gemv(p, ldx, *d, stream);
  FfnProduct q;
  q.gated = true;
  q.a[0] = {p.x, M, K, ldx};
  q.b[0] = {p.wg, N, K, K};
  q.b[1] = {p.wu, N, K, K};
  q.rows = M;
  q.cols = N;
  q.kext = K;
  q.y[0] = p.h;
  q.y[1] = p.g;
  q.y[2] = p.u;
  FfnEpilogue ep;
  ep.dtype = p.dtype;
  ep.act = p.activation;
  ep.save = p.g != nullptr;
  ep.bias[0] = p.bg;
  ep.bias[1] = p.bu;
  const FfnProduct* const ps[1] = {&q};
  FfnPlan plan = plan_ffn(ps, 1, d->sms);
  Packer pk;
  pk.need(&q.a[0]);
  pk.need(&q.b[0]);
  pk.need(&q.b[1]);
  size_t space;
  WorkspaceLease lease;
  if (!lease_products(ps, 1, &plan, p.dtype, pk.bytes, *d, stream, &space, &lease))
    return cuda_fail(cudaErrorMemoryAllocation);
  char* ws = static_cast<char*>(lease.ptr);
  pk.place(ws + space);
  const cudaError_t e = pk.run(d->sms, stream);
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  return finish(lease, run_ffn_products(ps, 1, plan, ep, nullptr, ws, *d, stream));
}

// The products behind dx and dw of D_q (one or two) with W_q and x.
struct Grads {
  FfnProduct dx, dw;
  const FfnProduct* ps[2];
  int count = 0;
  FfnPlan plan;

  // d: the D matrices (their addresses may be filled in later, by set_d)
  void make(int nd, const Operand* d, const Operand* w, const Operand& x, void* dxp, void* const* dwp, int64_t M,
            int64_t N, int64_t K, int sms, Packer* pk) {
    if (dxp != nullptr && K > 0) {
      dx.parts = nd;
      dx.rows = M;
      dx.cols = K;
      dx.kext = N;
      dx.y[0] = dxp;
      for (int i = 0; i < nd; ++i) {
        dx.a[i] = d[i];
        dx.b[i] = w[i];
        pk->need(&dx.b[i]);
      }
      ps[count++] = &dx;
    }
    dw.outputs = 0;
    if (K > 0)
      for (int i = 0; i < nd; ++i)
        if (dwp[i] != nullptr) {
          dw.a[dw.outputs] = d[i];
          dw.y[dw.outputs++] = dwp[i];
        }
    if (dw.outputs > 0) {
      dw.mn_a = true;
      dw.rows = N;
      dw.cols = K;
      dw.kext = M;
      dw.b[0] = x;
      pk->need(&dw.b[0]);
      ps[count++] = &dw;
    }
    plan = plan_ffn(ps, count, sms);
  }
  int run(const FfnEpilogue& ep, const FfnBiasGrad* bg, char* ws, const FfnDevice& dev, cudaStream_t stream) const {
    return run_ffn_products(ps, count, plan, ep, bg, ws, dev, stream);
  }
};

int gated_linear_backward(const poot_gated_linear_backward_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_gated_linear_backward_args& p = *ap;
  const int64_t M = p.M, N = p.N, K = p.K;
  int64_t ldx, ld_dh, ld_g, ld_u;
  if (!sizes_ok(M, N, K) || !row_pitch(M, K, p.ldx, &ldx) || !row_pitch(M, N, p.ld_dh, &ld_dh) ||
      !row_pitch(M, N, p.ld_g, &ld_g) || !row_pitch(M, N, p.ld_u, &ld_u) ||
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
  // without columns dx, dwg and dwu have no elements: a launch needs a product or a bias gradient
  if (((p.dx == nullptr && !want_dw) || K == 0) && !want_db) return POOT_OK;
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
  // Rows of a block of the gate's gradient: 64, less while the blocks are
  // fewer than four per SM
  int rows = 64;
  while (rows > 16 && ceil_div(M, rows) * ceil_div(N, kGateWidth) < 4 * int64_t(d->sms)) rows /= 2;
  const int64_t Np = ceil8(N), row_blocks = ceil_div(M, rows), gate_blocks = row_blocks * ceil_div(N, kGateWidth);
  if (gate_blocks > INT32_MAX / 2) return POOT_ERR_INVALID_ARG;
  Packer pk;
  Grads g;
  const Operand dmat[2] = {{nullptr, M, N, Np}, {nullptr, M, N, Np}}, w[2] = {{p.wg, N, K, K}, {p.wu, N, K, K}};
  void* const dwp[2] = {p.dwg, p.dwu};
  g.make(2, dmat, w, {p.x, M, K, ldx}, p.dx, dwp, M, N, K, d->sms, &pk);
  const size_t dbytes = round256(size_t(M) * Np * 2);
  const size_t sbytes = want_db ? round256(size_t(row_blocks) * 2 * Np * 4) : 0;
  size_t space;
  WorkspaceLease lease;
  if (!lease_products(g.ps, g.count, &g.plan, p.dtype, 2 * dbytes + sbytes + pk.bytes, *d, stream, &space, &lease))
    return cuda_fail(cudaErrorMemoryAllocation);
  char* const ws = static_cast<char*>(lease.ptr);
  char* const dgp = ws;
  char* const dup = ws + dbytes;
  float* const sums = reinterpret_cast<float*>(ws + 2 * dbytes + space);
  pk.place(ws + 2 * dbytes + space + sbytes);
  g.dx.a[0].p = dgp;
  g.dx.a[1].p = dup;
  for (int i = 0; i < g.dw.outputs; ++i) g.dw.a[i].p = g.dw.y[i] == p.dwg ? dgp : dup;
  GateGradArgs ga;
  std::memset(&ga, 0, sizeof(ga));
  ga.dh = static_cast<const uint16_t*>(p.dh);
  ga.g = static_cast<const uint16_t*>(p.g);
  ga.u = static_cast<const uint16_t*>(p.u);
  ga.ld_dh = ld_dh;
  ga.ld_g = ld_g;
  ga.ld_u = ld_u;
  ga.dg = reinterpret_cast<uint16_t*>(dgp);
  ga.du = reinterpret_cast<uint16_t*>(dup);
  ga.ldo = Np;
  ga.sums = want_db ? sums : nullptr;
  ga.M = static_cast<int>(M);
  ga.N = static_cast<int>(N);
  ga.act = p.activation;
  ga.rows = rows;
  ga.blocks = static_cast<int>(gate_blocks);
  ga.pack = pk.a;
  const dim3 grid(static_cast<unsigned>(gate_blocks + pk.blocks(d->sms)));
  const bool vec = N % 8 == 0 && ld_dh % 8 == 0 && ld_g % 8 == 0 && ld_u % 8 == 0 && aligned(p.dh, 16) &&
                   aligned(p.g, 16) && aligned(p.u, 16);
  auto pick = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return want_db ? (vec ? gate_grad_kernel<DT, true, true> : gate_grad_kernel<DT, true, false>)
                   : (vec ? gate_grad_kernel<DT, false, true> : gate_grad_kernel<DT, false, false>);
  };
  auto kern = p.dtype == POOT_DTYPE_BF16 ? pick(std::integral_constant<int, kEpiBf16>{})
                                         : pick(std::integral_constant<int, kEpiF16>{});
  const cudaError_t e = launch(kern, grid, dim3(kGateThreads), 0, stream, ga);
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  FfnEpilogue ep;
  ep.dtype = p.dtype;
  FfnBiasGrad bg;
  std::memset(&bg, 0, sizeof(bg));
  if (want_db) {
    bg.sums = sums;
    bg.rows = row_blocks;
    bg.outputs = 2;
    bg.N = static_cast<int>(N);
    bg.out[0] = static_cast<uint16_t*>(p.dbg);
    bg.out[1] = static_cast<uint16_t*>(p.dbu);
  }
  return finish(lease, g.run(ep, &bg, ws + 2 * dbytes, *d, stream));
}

int linear_backward(const poot_linear_backward_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_linear_backward_args& p = *ap;
  const int64_t M = p.M, N = p.N, K = p.K;
  int64_t ldx, ld_dy;
  if (!sizes_ok(M, N, K) || !row_pitch(M, K, p.ldx, &ldx) || !row_pitch(M, N, p.ld_dy, &ld_dy) ||
      (p.dtype != POOT_DTYPE_F16 && p.dtype != POOT_DTYPE_BF16))
    return POOT_ERR_INVALID_ARG;
  if (M > 0 && N > 0 && (p.dx != nullptr || p.dw != nullptr || p.db != nullptr)) {
    if (p.dy == nullptr || (K > 0 && p.dx != nullptr && p.w == nullptr) || (K > 0 && p.dw != nullptr && p.x == nullptr))
      return POOT_ERR_INVALID_ARG;
  }
  const int64_t wb = span_bytes(N, K, K);
  const int rc = check_spans({{p.dy, span_bytes(M, N, ld_dy)}, {p.x, span_bytes(M, K, ldx)}, {p.w, wb}},
                             {{p.dx, span_bytes(M, K, K)}, {p.dw, wb}, {p.db, 2 * N}});
  if (rc != POOT_OK) return rc;
  if (((p.dx == nullptr && p.dw == nullptr) || K == 0) && p.db == nullptr) return POOT_OK;
  FfnDevice* d;
  const int st = ffn_device(&d);
  if (st != POOT_OK) return st;
  if (M == 0 || N == 0) {
    int z = zero(p.dx, span_bytes(M, K, K), stream);
    if (z == POOT_OK) z = zero(p.dw, wb, stream);
    return z == POOT_OK ? zero(p.db, 2 * N, stream) : z;
  }
  Packer pk;
  Operand dy = {p.dy, M, N, ld_dy};
  Grads g;
  const Operand w = {p.w, N, K, K};
  g.make(1, &dy, &w, {p.x, M, K, ldx}, p.dx, &p.dw, M, N, K, d->sms, &pk);
  if (g.count > 0) pk.need(&dy);
  size_t space;
  WorkspaceLease lease;
  if (!lease_products(g.ps, g.count, &g.plan, p.dtype, pk.bytes, *d, stream, &space, &lease))
    return cuda_fail(cudaErrorMemoryAllocation);
  char* const ws = static_cast<char*>(lease.ptr);
  pk.place(ws + space);
  g.dx.a[0] = g.dw.a[0] = dy;
  const cudaError_t e = pk.run(d->sms, stream);
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  FfnEpilogue ep;
  ep.dtype = p.dtype;
  FfnBiasGrad bg;
  std::memset(&bg, 0, sizeof(bg));
  if (p.db != nullptr) {
    bg.d = static_cast<const uint16_t*>(dy.p);  // the repacked rows where there are any
    bg.ld = dy.ld;
    bg.rows = M;
    bg.outputs = 1;
    bg.N = static_cast<int>(N);
    bg.out[0] = static_cast<uint16_t*>(p.db);
  }
  return finish(lease, g.run(ep, &bg, ws, *d, stream));
}

// ---- clipping ----------------------------------------------------------------------
// The table of `count` tensors; returns the launch's blocks.
template <int T>
int fill_clip(ClipTable<T>* table, const poot_grad_tensor* t, int64_t count, int max_blocks) {
  int n = 0;
  table->first[0] = 0;
  for (int64_t k = 0; k < count; ++k) {
    const poot_grad_tensor& g = t[k];
    if (g.n == 0) continue;
    table->src[n] = g.src;
    table->dst[n] = g.dst;
    table->n[n] = g.n;
    table->dtype[n] = static_cast<unsigned char>(g.dtype);
    table->first[n + 1] =
        table->first[n] + static_cast<int>(ceil_div(g.n, kClipPieceBytes / (g.dtype == POOT_GRAD_F32 ? 4 : 2)));
    ++n;
  }
  table->count = n;
  return std::max(1, std::min(table->first[n], max_blocks));
}

// One list: two launches, the second started by the first's end; or, beyond
// eight pieces a resident block (80 MB), one cooperative launch, whose second
// half starts from what its blocks read last (GB300: 9 MB 8.7 us in two
// launches, 9.3 in one; 18 MB in 12 tensors 9.2 and 11.4; 60 MB 29.6 both;
// 500 MB 242 and 235; 1.4 GB 654 and 631).
template <int T>
int clip_list(const poot_grad_tensor* t, int64_t count, ClipArgs a, int max_blocks, cudaStream_t stream) {
  ClipTable<T> table;
  const int blocks = fill_clip(&table, t, count, max_blocks);
  a.parts = blocks;
  cudaError_t e;
  if (table.first[table.count] > 8 * max_blocks) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kClipThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    std::memset(&attr, 0, sizeof(attr));
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, clip_kernel<T, kClipBoth>, table, a);
  } else {
    e = launch(clip_kernel<T, kClipSum>, dim3(blocks), dim3(kClipThreads), 0, stream, table, a);
    if (e == cudaSuccess) e = launch(clip_kernel<T, kClipScale>, dim3(blocks), dim3(kClipThreads), 0, stream, table, a);
  }
  return e == cudaSuccess ? POOT_OK : cuda_fail(e);
}

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
  const int max_blocks = d->clip_blocks;
  const int64_t launches = std::max<int64_t>(1, ceil_div(count, kClipTable));
  WorkspaceLease lease = stream_workspace(d->dev, stream, size_t(launches) * max_blocks * sizeof(double));
  if (lease.ptr == nullptr) return cuda_fail(cudaErrorMemoryAllocation);
  ClipArgs a;
  a.partial = static_cast<double*>(lease.ptr);
  a.max_norm = max_norm;
  a.norm = norm;
  a.write_norm = 1;
  a.part0 = 0;
  a.parts = 0;
  if (count <= kClipTableFew) return finish(lease, clip_list<kClipTableFew>(t, count, a, max_blocks, stream));
  if (count <= kClipTable) return finish(lease, clip_list<kClipTable>(t, count, a, max_blocks, stream));
  ClipTable<kClipTable> table;
  cudaError_t e = cudaSuccess;
  for (int64_t k = 0; k < count && e == cudaSuccess; k += kClipTable) {
    const int blocks = fill_clip(&table, t + k, std::min<int64_t>(kClipTable, count - k), max_blocks);
    a.part0 = a.parts;
    e = launch(clip_kernel<kClipTable, kClipSum>, dim3(blocks), dim3(kClipThreads), 0, stream, table, a);
    a.parts += blocks;
  }
  for (int64_t k = 0; k < count && e == cudaSuccess; k += kClipTable) {
    const int blocks = fill_clip(&table, t + k, std::min<int64_t>(kClipTable, count - k), max_blocks);
    a.write_norm = k == 0;
    e = launch(clip_kernel<kClipTable, kClipScale>, dim3(blocks), dim3(kClipThreads), 0, stream, table, a);
  }
  return finish(lease, e == cudaSuccess ? POOT_OK : cuda_fail(e));
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
