// C ABI of the vocabulary head's loss and its gradients (include/poot_train.h):
// argument checks, pieces of the vocabulary, workspaces and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "poot_train.h"
#include "ffn_plan.cuh"
#include "head_elem.cuh"

namespace poot_host {
cudaError_t take_head_device_error(unsigned int* word) {
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

struct HeadDevice : DeviceInfo {
  bool ready = false;
  int status = POOT_OK;
};
std::mutex g_mu;
HeadDevice g_devices[kMaxDevices];

template <int CL, int DT>
cudaError_t set_attr() {
  for (auto kernel : {ffn_gemm_kernel<CL, kFfnLse, DT, true>, ffn_gemm_kernel<CL, kFfnDz, DT, false>,
                      ffn_gemm_kernel<CL, kFfnDz, DT, true>, ffn_gemm_kernel<CL, kFfnScaled, DT, false>,
                      ffn_gemm_kernel<CL, kFfnScaled, DT, true>}) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FfnLayout::DYN_BYTES);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int head_device(HeadDevice** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return POOT_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_mu);
  HeadDevice& d = g_devices[dev];
  if (!d.ready) {
    const int q = device_query(dev, &d.sms);
    if (q == POOT_ERR_CUDA) return q;
    if (q == POOT_OK && ((e = set_attr<1, kEpiF16>()) != cudaSuccess || (e = set_attr<2, kEpiF16>()) != cudaSuccess ||
                         (e = set_attr<1, kEpiBf16>()) != cudaSuccess || (e = set_attr<2, kEpiBf16>()) != cudaSuccess))
      return cuda_fail(e);
    d.dev = dev;
    d.status = q;
    d.ready = true;
  }
  *out = &d;
  return d.status;
}

template <int MODE, bool CHUNKS>
cudaError_t launch_mode(const FfnMaps& m, const FfnHeadGemmArgs& a, bool bf16, int cl, int64_t units,
                        cudaStream_t stream) {
  auto kernel = cl == 2 ? (bf16 ? ffn_gemm_kernel<2, MODE, kEpiBf16, CHUNKS> : ffn_gemm_kernel<2, MODE, kEpiF16, CHUNKS>)
                        : (bf16 ? ffn_gemm_kernel<1, MODE, kEpiBf16, CHUNKS> : ffn_gemm_kernel<1, MODE, kEpiF16, CHUNKS>);
  return launch_clustered(kernel, dim3(static_cast<unsigned>(units * cl)), dim3(ffn_threads(false)),
                          FfnLayout::DYN_BYTES, stream, unsigned(cl), m, a);
}

template <int MODE>
cudaError_t launch_head(const FfnMaps& m, const FfnGemmArgs& base, const HeadArgs& head, bool bf16, int cl,
                        int64_t units, cudaStream_t stream) {
  FfnHeadGemmArgs a;
  static_cast<FfnGemmArgs&>(a) = base;
  a.head = head;
  if constexpr (MODE == kFfnLse) {
    return launch_mode<MODE, true>(m, a, bf16, cl, units, stream);
  } else {
    return base.scratch != nullptr ? launch_mode<MODE, true>(m, a, bf16, cl, units, stream)
                                   : launch_mode<MODE, false>(m, a, bf16, cl, units, stream);
  }
}

// Without columns the logits are the biases: products with operands of zeros,
// eight columns wide, in the workspace.
struct ZeroOperands {
  size_t xb = 0, wb = 0;
  ZeroOperands(int64_t M, int64_t V, int64_t K)
      : xb(K == 0 ? round256(size_t(M) * 16) : 0), wb(K == 0 ? round256(size_t(V) * 16) : 0) {}
  size_t bytes() const { return xb + wb; }
  cudaError_t place(char* at, Operand* x, Operand* w, cudaStream_t stream) const {
    if (bytes() == 0) return cudaSuccess;
    x->p = at;
    w->p = at + xb;
    x->cols = w->cols = x->ld = w->ld = 8;
    return cudaMemsetAsync(at, 0, bytes(), stream);
  }
};

// Elements whose multiple the pitch of a copy is: 128 bytes, a row's part of a
// K block then lies in as few sectors as it can (2047 x 32003 x 770, the products alone: 97 us
// with rows of 1552 bytes, 75 with rows of 1664 and a shorter epilogue).
constexpr int64_t kHeadPitch = 64;

// Tiles of the logits.  One M block on a W of some size is a stream of W: single CTAs, whose
// short A leaves the ring to W, and the widest tile unless a narrower one deals the columns out
// more evenly.  Times in microseconds: HBM's, or a CTA's rounds of tiles, whose K blocks arrive
// 2.5 us after they are asked for, a ring full at a time (GB300, one row, 131072 x 4096: 224 wide 163 us, 128
// wide 170, 96 wide 188, 64 wide 280; 256 wide 212 with 128 rows of A in a stage).
FfnPlan plan_logits(const FfnProduct& q, int sms) {
  const FfnProduct* const ps[1] = {&q};
  FfnPlan best = plan_ffn(ps, 1, sms, false);
  const double bytes = 2.0 * double(q.cols) * double(q.kext);
  if (q.rows > kFfnBM || bytes < 8e6) return best;
  best.cl = 1;
  double best_time = 1e300;
  for (int bn = kFfnMaxBN; bn >= 128; bn -= 32) {
    const int stage = static_cast<int>(ceil8(std::min<int64_t>(q.rows, kFfnBM))) * kFfnBK * 2 + ffn_b_bytes(1, bn);
    const double rounds = double(ceil_div(ceil_div(q.cols, bn), sms));
    const double t = std::max(bytes / 6.6e6, rounds * double(ceil_div(q.kext, kFfnBK)) * 2.5 /
                                                 std::min(FfnLayout::RING_BYTES / stage, kFfnMaxStages));
    if (t < 0.97 * best_time) {
      best_time = t;
      best.bn = bn;
    }
  }
  return best;
}

// ---- the loss --------------------------------------------------------------------
template <int ROWS>
cudaError_t launch_loss(const HeadLossArgs& a, cudaStream_t stream) {
  return launch(head_loss_kernel<ROWS>, dim3(static_cast<unsigned>(ceil_div(a.M, ROWS))), dim3(kHeadLossThreads), 0,
                stream, a);
}

int linear_cross_entropy(const poot_linear_cross_entropy_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_linear_cross_entropy_args& p = *ap;
  const int64_t M = p.M, V = p.V, K = p.K;
  int64_t ldx;
  if (!sizes_ok(M, V, K) || !row_pitch(M, K, p.ldx, &ldx) ||
      (p.dtype != POOT_DTYPE_F16 && p.dtype != POOT_DTYPE_BF16) || (M > 0 && V == 0))
    return POOT_ERR_INVALID_ARG;
  if (M == 0) return POOT_OK;
  if (p.target == nullptr || p.loss == nullptr || (K > 0 && (p.x == nullptr || p.w == nullptr)))
    return POOT_ERR_INVALID_ARG;
  if (!aligned(p.target, 8) || !aligned(p.loss, 4) || !aligned(p.lse, 4)) return POOT_ERR_MISALIGNED;
  const int rc = check_spans({{p.x, span_bytes(M, K, ldx)}, {p.w, span_bytes(V, K, K)}, {p.b, 2 * V}, {p.target, 8 * M}},
                             {{p.loss, 4 * M}, {p.lse, 4 * M}});
  if (rc != POOT_OK) return rc;
  HeadDevice* d;
  const int st = head_device(&d);
  if (st != POOT_OK) return st;
  const int64_t Kz = K == 0 ? 8 : K;
  FfnProduct q;
  q.logits = true;
  q.a[0] = {p.x, M, K, ldx};
  q.b[0] = {p.w, V, K, K};
  q.rows = M;
  q.cols = V;
  q.kext = Kz;
  const FfnProduct* const ps[1] = {&q};
  const FfnPlan plan = plan_logits(q, d->sms);
  Packer pk(kHeadPitch);
  if (K > 0) {
    pk.need(&q.a[0]);
    pk.need(&q.b[0]);
  }
  const ZeroOperands zeros(M, V, K);
  const int64_t parts = ceil_div(V, plan.bn) * kHeadParts;
  const size_t pbytes = round256(size_t(parts) * M * sizeof(float2)), tbytes = round256(size_t(M) * 4);
  WorkspaceLease lease = stream_workspace(d->dev, stream, pbytes + tbytes + pk.bytes + zeros.bytes());
  if (lease.ptr == nullptr) return cuda_fail(cudaErrorMemoryAllocation);
  char* const ws = static_cast<char*>(lease.ptr);
  cudaError_t e = zeros.place(ws + pbytes + tbytes, &q.a[0], &q.b[0], stream);
  pk.place(ws + pbytes + tbytes);
  if (e == cudaSuccess) e = pk.run(d->sms, stream);
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  HeadArgs h;
  std::memset(&h, 0, sizeof(h));
  h.bias = static_cast<const uint16_t*>(p.b);
  h.target = reinterpret_cast<const long long*>(p.target);
  h.ignore = p.ignore_index;
  h.vocab = static_cast<int>(V);
  h.partial = reinterpret_cast<float2*>(ws);
  h.picked = reinterpret_cast<float*>(ws + pbytes);
  FfnEpilogue ep;
  ep.dtype = p.dtype;
  const int r = run_products(
      ps, 1, plan, ep, nullptr, nullptr, *d,
      [&](const FfnMaps& m, const FfnGemmArgs& a, bool bf16, int64_t units) {
        return launch_head<kFfnLse>(m, a, h, bf16, plan.cl, units, stream);
      },
      [](const FfnProduct&, const FfnJob&, const float*) { return cudaSuccess; });
  if (r != POOT_OK) return finish(lease, r);
  HeadLossArgs l;
  l.partial = h.partial;
  l.picked = h.picked;
  l.target = h.target;
  l.loss = p.loss;
  l.lse = p.lse;
  l.ignore = h.ignore;
  l.M = M;
  l.vocab = h.vocab;
  l.parts = static_cast<int>(parts);
  // rows of a block: 32 (a warp's loads side by side), 8 (whole sectors) while the blocks do not fill the SMs
  e = M >= 32 * int64_t(d->sms) ? launch_loss<32>(l, stream)
                                : (M >= 16 ? launch_loss<8>(l, stream) : launch_loss<1>(l, stream));
  return finish(lease, e == cudaSuccess ? POOT_OK : cuda_fail(e));
}

// ---- its gradients -----------------------------------------------------------------
// Columns of a piece: q of a piece takes at most 256 MB, pieces of about equal
// width, multiples of 256 (a tile).
constexpr int64_t kHeadPieceBytes = int64_t(256) << 20;
int64_t piece_columns(int64_t M, int64_t V) {
  const int64_t most = std::max<int64_t>(kHeadPieceBytes / (2 * M) / 256 * 256, 512);
  const int64_t pieces = ceil_div(V, most);
  return std::min(V, ceil_div(ceil_div(V, pieces), 256) * 256);
}

int linear_cross_entropy_backward(const poot_linear_cross_entropy_backward_args* ap, cudaStream_t stream) {
  if (ap == nullptr) return POOT_ERR_INVALID_ARG;
  const poot_linear_cross_entropy_backward_args& p = *ap;
  const int64_t M = p.M, V = p.V, K = p.K;
  int64_t ldx;
  if (!sizes_ok(M, V, K) || !row_pitch(M, K, p.ldx, &ldx) ||
      (p.dtype != POOT_DTYPE_F16 && p.dtype != POOT_DTYPE_BF16) || (M > 0 && V == 0) || p.dloss_stride < 0 ||
      (M > 1 && p.dloss_stride > kMaxSpan / M))
    return POOT_ERR_INVALID_ARG;
  const bool want = p.dx != nullptr || p.dw != nullptr || p.db != nullptr;
  if (M > 0 && want &&
      (p.dloss == nullptr || p.target == nullptr || p.lse == nullptr || (K > 0 && (p.x == nullptr || p.w == nullptr))))
    return POOT_ERR_INVALID_ARG;
  if (!aligned(p.dloss, 4) || !aligned(p.target, 8) || !aligned(p.lse, 4)) return POOT_ERR_MISALIGNED;
  const int64_t wb = span_bytes(V, K, K);
  const int rc = check_spans({{p.dloss, M > 0 ? 4 * ((M - 1) * p.dloss_stride + 1) : 0},
                              {p.x, span_bytes(M, K, ldx)},
                              {p.w, wb},
                              {p.b, 2 * V},
                              {p.target, 8 * M},
                              {p.lse, 4 * M}},
                             {{p.dx, span_bytes(M, K, K)}, {p.dw, wb}, {p.db, 2 * V}});
  if (rc != POOT_OK) return rc;
  const bool want_dx = p.dx != nullptr && K > 0, want_dw = p.dw != nullptr && K > 0, want_db = p.db != nullptr;
  if (!want_dx && !want_dw && !want_db) return POOT_OK;
  HeadDevice* d;
  const int st = head_device(&d);
  if (st != POOT_OK) return st;
  if (M == 0) {
    const int z = zero(p.dw, wb, stream);
    return z == POOT_OK ? zero(p.db, 2 * V, stream) : z;
  }
  const int64_t Vc = piece_columns(M, V), ldq = ceil_div(Vc, kHeadPitch) * kHeadPitch, Kz = K == 0 ? 8 : K;
  // operands: x (copied where dW reads it, see head_prep_kernel), W
  const int64_t ldxc = ceil_div(K, kHeadPitch) * kHeadPitch;
  Operand x = {p.x, M, K, ldx}, w = {p.w, V, K, K};
  Packer pk(kHeadPitch);
  size_t xbytes = 0;
  if (K > 0) {
    if (want_dw) xbytes = round256(size_t(M) * ldxc * 2);
    else pk.need(&x);
    pk.need(&w);
  }
  const ZeroOperands zeros(M, V, K);
  // the logits of a piece, then its products
  FfnProduct z, dx, dw;
  z.logits = true;
  z.rows = M;
  z.kext = Kz;
  z.ldy = ldq;
  z.cols = Vc;
  const FfnProduct* const zs[1] = {&z};
  const FfnPlan zplan = plan_logits(z, d->sms);
  const FfnProduct* ps[2];
  int count = 0;
  if (want_dx) {
    dx.rows = M;
    dx.cols = K;
    dx.kext = Vc;
    dx.y[0] = p.dx;
    dx.sum = Vc < V;
    ps[count++] = &dx;
  }
  if (want_dw) {
    dw.mn_a = true;
    dw.rows = Vc;
    dw.cols = K;
    dw.kext = M;
    ps[count++] = &dw;
  }
  FfnPlan plan = plan_ffn(ps, count, d->sms);
  FfnSpace zspace(zs, 1, zplan, p.dtype, d->sms);
  // column sums of q, of 32 rows each
  const int64_t sum_blocks = want_db ? ceil_div(M, 32) : 0;
  const size_t sbytes = round256(size_t(sum_blocks) * ceil8(Vc) * 4);
  const size_t qbytes = round256(size_t(M) * ldq * 2);
  size_t space;
  WorkspaceLease lease;
  if (!lease_products(ps, count, &plan, p.dtype, 256 + qbytes + zspace.bytes() + sbytes + xbytes + pk.bytes + zeros.bytes(), *d,
                      stream, &space, &lease))
    return cuda_fail(cudaErrorMemoryAllocation);
  char* at = static_cast<char*>(lease.ptr);
  auto take = [&](size_t bytes) {
    char* const r = at;
    at += bytes;
    return r;
  };
  char* const pws = take(space);
  float* const scale = reinterpret_cast<float*>(take(256));
  char* const q = take(qbytes);
  char* const zws = take(zspace.bytes());
  float* const sums = reinterpret_cast<float*>(take(sbytes));
  uint16_t* const xc = reinterpret_cast<uint16_t*>(take(xbytes));
  HeadPrepArgs pa;
  std::memset(&pa, 0, sizeof(pa));
  pa.dloss = p.dloss;
  pa.dloss_stride = p.dloss_stride;
  pa.target = reinterpret_cast<const long long*>(p.target);
  pa.ignore = p.ignore_index;
  pa.rows = M;
  pa.scale = scale;
  if (xbytes != 0) {
    pa.x = static_cast<const uint16_t*>(p.x);
    pa.ld = ldx;
    pa.xc = xc;
    pa.ldc = ldxc;
    pa.cols = static_cast<int>(K);
    pa.copy_blocks = static_cast<int>(std::min<int64_t>(ceil_div(M * ceil_div(K, kPackSpan), 8), int64_t(d->sms) * 8));
    x = {xc, M, K, pa.ldc};
  }
  cudaError_t e = zeros.place(at, &x, &w, stream);
  pk.place(take(pk.bytes));
  pa.pack = pk.a;
  if (e == cudaSuccess)
    e = launch(head_prep_kernel, dim3(static_cast<unsigned>(1 + pa.copy_blocks + pk.blocks(d->sms))), dim3(256), 0,
               stream, pa);
  if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  HeadArgs h;
  std::memset(&h, 0, sizeof(h));
  h.target = pa.target;
  h.ignore = p.ignore_index;
  h.vocab = static_cast<int>(V);
  h.lse = p.lse;
  h.dloss = p.dloss;
  h.dloss_stride = p.dloss_stride;
  h.scale = scale;
  FfnEpilogue ep;
  ep.dtype = p.dtype;
  auto reduce = [&](void* y, const float* sums, int64_t rows, int64_t cols, int S) {
    HeadReduceArgs r;
    std::memset(&r, 0, sizeof(r));
    r.ws = sums;
    r.y = static_cast<uint16_t*>(y);
    r.scale = scale;
    r.M = rows;
    r.S = S;
    r.N = static_cast<int>(cols);
    r.ldw = static_cast<int>(ceil_div(cols, 4) * 4);
    r.dtype = p.dtype;
    return launch(head_reduce_kernel, dim3(grid_for(rows * (r.ldw / 4), d->sms)), dim3(256), 0, stream, r);
  };
  for (int64_t c0 = 0; c0 < V; c0 += Vc) {
    const int64_t cols = std::min(Vc, V - c0);
    const Operand wc = {static_cast<const uint16_t*>(w.p) + c0 * w.ld, cols, w.cols, w.ld};
    const Operand qc = {q, M, cols, ldq};
    h.bias = p.b == nullptr ? nullptr : static_cast<const uint16_t*>(p.b) + c0;
    h.col0 = static_cast<int>(c0);
    h.sums = want_db ? sums : nullptr;
    h.sums_pitch = static_cast<int>(ceil8(cols));
    z.a[0] = x;
    z.b[0] = wc;
    z.cols = cols;
    z.y[0] = q;
    int r = run_products(
        zs, 1, zplan, ep, nullptr, zws, *d,
        [&](const FfnMaps& m, const FfnGemmArgs& a, bool bf16, int64_t units) {
          return launch_head<kFfnDz>(m, a, h, bf16, zplan.cl, units, stream);
        },
        [](const FfnProduct&, const FfnJob&, const float*) { return cudaSuccess; });
    if (r != POOT_OK) return finish(lease, r);
    dx.kext = cols;
    dx.a[0] = qc;
    dx.b[0] = wc;
    dw.rows = cols;
    dw.a[0] = qc;
    dw.b[0] = x;
    dw.y[0] = static_cast<uint16_t*>(p.dw) + c0 * K;
    h.sum_dx = dx.sum;
    h.accumulate = c0 > 0;
    FfnBiasGrad bg;
    std::memset(&bg, 0, sizeof(bg));
    if (want_db) {
      bg.outputs = 1;
      bg.N = static_cast<int>(cols);
      bg.out[0] = static_cast<uint16_t*>(p.db) + c0;
      bg.sums = sums;
      bg.rows = sum_blocks;
    }
    r = run_products(
        ps, count, plan, ep, &bg, pws, *d,
        [&](const FfnMaps& m, const FfnGemmArgs& a, bool bf16, int64_t units) {
          return launch_head<kFfnScaled>(m, a, h, bf16, plan.cl, units, stream);
        },
        [&](const FfnProduct& g, const FfnJob& j, const float* sums) {
          return reduce(g.y[0], sums, g.rows, g.cols, j.split);
        });
    if (r != POOT_OK) return finish(lease, r);
  }
  if (dx.sum && want_dx) {
    e = reduce(p.dx, reinterpret_cast<const float*>(pws), M, K, 1);
    if (e != cudaSuccess) return finish(lease, cuda_fail(e));
  }
  return finish(lease, POOT_OK);
}

}  // namespace

extern "C" {

int poot_linear_cross_entropy(const poot_linear_cross_entropy_args* args, poot_stream_t stream) {
  return guarded([&] { return linear_cross_entropy(args, reinterpret_cast<cudaStream_t>(stream)); });
}

int poot_linear_cross_entropy_backward(const poot_linear_cross_entropy_backward_args* args, poot_stream_t stream) {
  return guarded([&] { return linear_cross_entropy_backward(args, reinterpret_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
