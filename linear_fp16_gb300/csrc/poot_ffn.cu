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

// Sizes: the kernels round them up to tiles, vectors and warps' shares of K (at
// most 2304 more, the repacking's two spans of a row) in 32 bits
constexpr int64_t kMaxDim = POOT_FFN_MAX_SIZE;
static_assert(kMaxDim + 2304 < (int64_t(1) << 31), "32-bit index arithmetic");
constexpr int kMaxDevices = 64;

struct FfnDevice {
  bool ready = false;
  int status = POOT_OK;
  int dev = 0;
  int sms = 0;
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

// Elements that a matrix spans, gaps between its rows included: no more than any
// address space holds, so that byte counts and end addresses stay in 64 bits.
constexpr int64_t kMaxSpan = int64_t(1) << 50;

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && M <= kMaxDim && N <= kMaxDim && K <= kMaxDim && M * N <= kMaxSpan &&
         M * K <= kMaxSpan && N * K <= kMaxSpan;
}

// The row pitch `ld` of an argument (0: contiguous rows) into *out; false: none
// that a [rows, cols] matrix can have.  A single row has no pitch, whatever ld
// says: it gets one that suits TMA.
bool row_pitch(int64_t rows, int64_t cols, int64_t ld, int64_t* out) {
  if (ld == 0) ld = cols;
  if (ld < cols || (rows > 1 && ld > kMaxSpan / rows)) return false;
  *out = rows > 1 ? ld : (cols + 7) / 8 * 8;
  return true;
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
    a.rows[t] = static_cast<int>(o->rows);
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
  // eight warps a block, a unit (see ffn_pack_rows) a warp while they last
  int blocks(int sms) const {
    int64_t units = 0;
    for (int t = 0; t < a.count; ++t) units += int64_t(a.rows[t]) * ceil_div(a.cols[t], kPackSpan);
    return static_cast<int>(std::min<int64_t>(ceil_div(units, 8), int64_t(sms) * 8));
  }
  cudaError_t run(int sms, cudaStream_t stream) const {
    if (a.count == 0) return cudaSuccess;
    return launch(ffn_pack_kernel, dim3(static_cast<unsigned>(blocks(sms))), dim3(256), 0, stream, a);
  }
};

// ---- tile plan -------------------------------------------------------------------
struct FfnPlan {
  int cl = 1, bn = 64;
  int split[2] = {1, 1};
};

// One family of products (see FfnJob) before it is planned.
struct FfnProduct {
  bool gated = false, mn_a = false;
  Operand a[2], b[2];
  int parts = 1, outputs = 1;
  int64_t rows = 0, cols = 0, kext = 0;  // of one output; K extent of one part
  void* y[3] = {nullptr, nullptr, nullptr};
  int64_t kb() const { return ceil_div(kext, kFfnBK) * parts; }
  size_t partial_bytes(int split) const {
    return split > 1 ? round256(size_t(split) * (gated ? 2 : outputs) * rows * ceil_div(cols, 4) * 16) : 0;
  }
};

// Time of a plan, in microseconds, from a model: a tile takes its K blocks at
// the shape's rate plus a fill, or its epilogue where that is longer; the tiles
// fill the CTAs (pairs) as FfnSchedule deals them; all of it takes at least the
// operands' time from HBM; a split adds the second kernel and the partial sums'
// traffic.  The constants are a fit to GB300 timings of single and paired
// products of 17 .. 8192 rows under every tile and split; they rank plans, and
// are not the times of the present kernels.
struct FfnShape {
  int cl, bn;
  double per_kb;  // 64 elements of K
};
constexpr FfnShape kFfnShapes[] = {{2, 256, 0.264}, {2, 128, 0.244}, {1, 256, 0.335}, {1, 128, 0.281}, {1, 64, 0.236}};

inline const FfnShape& shape_of(const FfnPlan& p) {
  for (const FfnShape& s : kFfnShapes)
    if (s.cl == p.cl && s.bn == p.bn) return s;
  return kFfnShapes[0];
}

// Time of a tile of `kb` 64-element K blocks among others of its kind: its
// products, or its share of HBM for 128 rows of output.
inline double tile_time(const FfnShape& s, int64_t kb, int64_t cols) {
  return std::max(double(kb) * s.per_kb + 0.23, double(cols) * 128 * 2 / 39.5e3);
}

double plan_time(const FfnProduct* const* ps, int count, const FfnShape& s, const int* split, int sms, double bytes) {
  const int64_t slots = sms / s.cl;
  int64_t tiles[2] = {0, 0}, kbs[2] = {1, 1};
  double tile[2] = {0, 0}, last = 0, added = s.cl == 2 ? 0.39 : 0.0;
  for (int i = 0; i < count; ++i) {
    const FfnProduct& q = *ps[i];
    const int64_t width = q.gated ? s.bn / 2 : s.bn;
    const int64_t kb = ceil_div(q.kext, kFfnBK * s.cl) * q.parts;
    kbs[i] = ceil_div(kb, split[i]);
    const int64_t S = ceil_div(kb, kbs[i]);
    const double main = double(kbs[i] * s.cl) * s.per_kb + 0.23;
    const double epi = 0.137 * double(width) / 128.0;
    tiles[i] = ceil_div(q.rows, kFfnBM * s.cl) * ceil_div(q.cols, width) * q.outputs * S;
    tile[i] = std::max(main, epi);
    last = std::max(last, std::min(main, epi));
    if (S > 1) added += 1.7 + double(S) * double(q.rows) * double(q.cols) * q.outputs * (q.gated ? 2 : 1) * 1.75e-6;
  }
  double t;
  if (count < 2) {
    t = double(ceil_div(tiles[0], slots)) * tile[0];
  } else {
    double dealt[2];
    for (int i = 0; i < 2; ++i) dealt[i] = tile_time(s, kbs[i] * s.cl, s.bn);
    const int f = dealt[1] > dealt[0] ? 1 : 0, o = 1 - f;
    const int64_t r = tiles[f] % slots, extra = r != 0 ? static_cast<int64_t>(dealt[f] / dealt[o] + 0.5) : 0;
    const int64_t common = ceil_div(std::max<int64_t>(0, tiles[o] - extra * (slots - r)), slots);
    const int64_t taken = r != 0 ? std::min(extra, ceil_div(tiles[o], slots - r)) : 0;
    t = std::max(double(ceil_div(tiles[f], slots)) * tile[f], double(tiles[f] / slots) * tile[f] + double(taken) * tile[o]) +
        double(common) * tile[o];
  }
  return std::max(t + last, bytes / 5.95e6) + added;
}

FfnPlan plan_ffn(const FfnProduct* const* ps, int count, int sms) {
  double bytes = 0;
  for (int i = 0; i < count; ++i) {
    const FfnProduct& q = *ps[i];
    const int na = q.mn_a ? q.outputs : q.parts, nb = q.gated ? 2 : q.parts;
    bytes += 2.0 * (double(q.rows) * q.kext * na + double(q.cols) * q.kext * nb + double(q.rows) * q.cols * q.outputs);
  }
  FfnPlan best;
  double best_time = 1e300;
  for (const FfnShape& s : kFfnShapes) {
    int split[2] = {1, 1};
    double t = plan_time(ps, count, s, split, sms, bytes);
    // splits, one product after the other, while its tiles leave CTAs idle
    for (int i = 0; i < count; ++i) {
      const FfnProduct& q = *ps[i];
      const int64_t tiles = ceil_div(q.rows, kFfnBM * s.cl) * ceil_div(q.cols, q.gated ? s.bn / 2 : s.bn) * q.outputs;
      for (int S = 2; S <= 16 && tiles * S <= 2 * (sms / s.cl) && q.kb() >= 4 * S; S *= 2) {
        int trial[2] = {split[0], split[1]};
        trial[i] = S;
        const double u = plan_time(ps, count, s, trial, sms, bytes);
        if (u < t) {
          t = u;
          split[i] = S;
        }
      }
    }
    if (t < best_time) {
      best_time = t;
      best.cl = s.cl;
      best.bn = s.bn;
      best.split[0] = split[0];
      best.split[1] = split[1];
    }
  }
  return best;
}

struct FfnEpilogue {
  int dtype = 0, act = 0, save = 0;
  const void* bias[2] = {nullptr, nullptr};
};

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

// K blocks of product `q` under plan `p`: of one part, of a range (its split's
// ranges but the last)
inline int64_t plan_kb_part(const FfnProduct& q, const FfnPlan& p) { return ceil_div(q.kext, kFfnBK * ffn_sub(p.cl)); }
inline int64_t plan_kb_split(const FfnProduct& q, const FfnPlan& p, int i) {
  return ceil_div(plan_kb_part(q, p) * q.parts, p.split[i]);
}

// Workspace of products under plan `p`: each one's partial sums, then the
// CTAs' scratch where a sum has more than one chunk (see FfnGemmArgs).
struct FfnSpace {
  size_t partial[2] = {0, 0}, scratch = 0;
  size_t bytes() const { return partial[0] + partial[1] + scratch; }
  FfnSpace(const FfnProduct* const* ps, int count, const FfnPlan& p, int dtype, int sms) {
    for (int i = 0; i < count; ++i) {
      partial[i] = ps[i]->partial_bytes(p.split[i]);
      if (plan_kb_split(*ps[i], p, i) > ffn_chunk_kb(p.cl, dtype)) scratch = size_t(sms) * kFfnScratchBytes;
    }
  }
};

// Leases the workspace of products under *plan, and `more` bytes behind them;
// *space is what the products take.  Where the device has no room for it, the
// products go unsplit.  false: no room even so.
bool lease_products(const FfnProduct* const* ps, int count, FfnPlan* plan, int dtype, size_t more, const FfnDevice& d,
                    cudaStream_t stream, size_t* space, WorkspaceLease* lease) {
  for (;;) {
    *space = FfnSpace(ps, count, *plan, dtype, d.sms).bytes();
    if (*space + more == 0) return true;
    *lease = stream_workspace(d.dev, stream, *space + more);
    if (lease->ptr != nullptr) return true;
    if (plan->split[0] == 1 && plan->split[1] == 1) return false;
    plan->split[0] = plan->split[1] = 1;
  }
}

// Runs up to two products (dx and dW) in one launch, with the
// bias gradients `bg` (may be nullptr) beside them, then the second halves of
// split products.  `ws`: workspace as FfnSpace lays it out.
int run_products(const FfnProduct* const* ps, int count, const FfnPlan& p, const FfnEpilogue& ep,
                 const FfnBiasGrad* bg, char* ws, const FfnDevice& d, cudaStream_t stream) {
  const FfnSpace space(ps, count, p, ep.dtype, d.sms);
  float* const partial[2] = {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + space.partial[0])};
  const bool bf16 = ep.dtype == POOT_DTYPE_BF16;
  FfnGemmArgs a;
  FfnMaps m;
  std::memset(&a, 0, sizeof(a));
  std::memset(&m, 0, sizeof(m));
  a.bn = p.bn;
  a.stages = ffn_stages(p.cl, p.bn);
  const bool gated = count > 0 && ps[0]->gated;
  a.cols = gated ? p.bn / 2 : p.bn;
  a.act = ep.act;
  a.save = ep.save;
  for (int i = 0; i < 2; ++i) a.bias[i] = static_cast<const uint16_t*>(ep.bias[i]);
  if (bg != nullptr) a.bias_grad = *bg;
  if (space.scratch != 0) a.scratch = reinterpret_cast<float4*>(ws + space.partial[0] + space.partial[1]);
  const int64_t units_max = d.sms / p.cl;
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    const FfnProduct& q = *ps[i];
    const int ji = q.mn_a ? 1 : 0;
    FfnJob& j = a.job[ji];
    j.M = static_cast<int>(q.rows);
    j.N = static_cast<int>(q.cols);
    j.num_m = static_cast<int>(ceil_div(q.rows, kFfnBM * p.cl));
    j.num_n = static_cast<int>(ceil_div(q.cols, a.cols));
    const int64_t kb_part = plan_kb_part(q, p);
    if (kb_part * q.parts > INT32_MAX) return POOT_ERR_INVALID_ARG;
    // (one part: the part index never advances)
    j.kb_part = q.parts > 1 ? static_cast<int>(kb_part) : INT32_MAX;
    j.kb_total = static_cast<int>(kb_part * q.parts);
    j.kb_split = static_cast<int>(plan_kb_split(q, p, i));
    j.split = static_cast<int>(ceil_div(j.kb_total, j.kb_split));  // no empty range
    // M blocks walked together: their A rows within 32 MB of L2, and at least
    // eight, about the square of tiles that run at one time
    int64_t group = (int64_t(32) << 20) / (2 * q.kext * q.parts * kFfnBM * p.cl);
    group = std::max<int64_t>(8, std::min<int64_t>(group, 64));
    j.group_m = static_cast<int>(std::min<int64_t>(group, j.num_m));
    const int64_t tpo = int64_t(j.num_m) * j.num_n, tiles = tpo * q.outputs * j.split;
    total += tiles;
    if (total > INT32_MAX / 4) return POOT_ERR_INVALID_ARG;
    j.tiles_per_out = static_cast<int>(tpo);
    j.tiles = static_cast<int>(tiles);
    j.by_out = FfnDiv(static_cast<uint32_t>(tpo));
    j.by_split = FfnDiv(static_cast<uint32_t>(j.split));
    j.by_span = FfnDiv(static_cast<uint32_t>(j.group_m) * static_cast<uint32_t>(j.num_n));
    j.by_group = FfnDiv(static_cast<uint32_t>(j.group_m));
    j.by_rest = FfnDiv(static_cast<uint32_t>((j.num_m - 1) % j.group_m + 1));
    const int ny = q.gated ? (ep.save ? 3 : 1) : q.outputs;
    j.tma_store = j.split == 1 && q.cols % 8 == 0;
    for (int o = 0; o < ny; ++o) {
      j.y[o] = static_cast<uint16_t*>(q.y[o]);
      if (!aligned(q.y[o], 16)) j.tma_store = 0;
    }
    auto encode = [&](CUtensorMap* map, const Operand& o, bool mn, int rows) {
      return encode_2d(map, o.p, o.cols, o.rows, kFfnBK, mn ? kFfnBK : static_cast<uint32_t>(rows),
                       CU_TENSOR_MAP_SWIZZLE_128B, bf16, o.ld);
    };
    const int na = q.gated ? 1 : (q.mn_a ? q.outputs : q.parts), nb = q.gated ? 2 : (q.mn_a ? 1 : q.parts);
    bool ok = true;
    for (int o = 0; o < na; ++o) ok = ok && encode(&m.a[ji][o], q.a[o], q.mn_a, kFfnBM);
    for (int o = 0; o < nb; ++o) ok = ok && encode(&m.b[ji][o], q.b[o], !q.gated, p.bn / 2);
    if (j.tma_store)
      for (int o = 0; o < ny; ++o)
        ok = ok && encode_2d(&m.y[ji][o], q.y[o], q.cols, q.rows, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, bf16);
    if (j.split > 1)
      ok = ok && encode_3d_f32(&m.partial[ji], partial[i], ceil_div(q.cols, 4) * 4, q.rows,
                               uint64_t(j.split) * (q.gated ? 2 : q.outputs), 16, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (!ok) return cuda_fail(cudaErrorInvalidValue);
  }
  for (FfnJob& j : a.job) {
    if (j.tiles > 0) continue;
    j.tiles_per_out = 1;
    j.split = 1;
  }
  // without bias gradients no more CTAs than tiles
  const int64_t units = a.bias_grad.outputs > 0 ? units_max : std::min<int64_t>(total, units_max);
  FfnDeal& deal = a.deal;
  if (count == 2) {
    double t[2];
    for (int i = 0; i < 2; ++i) t[i] = tile_time(shape_of(p), int64_t(a.job[i].kb_split) * p.cl, a.cols);
    deal.first = t[1] > t[0] ? 1 : 0;
    deal.extra = static_cast<int>(std::min(t[deal.first] / t[1 - deal.first] + 0.5, 1e6));
  } else if (count == 1) {
    deal.first = ps[0]->mn_a ? 1 : 0;
  }
  deal.rounds = static_cast<int>(a.job[deal.first].tiles / units);
  deal.rest = static_cast<int>(a.job[deal.first].tiles % units);
  deal.tiles1 = a.job[1 - deal.first].tiles;
  const int64_t dealt = deal.rest != 0 ? std::min<int64_t>(int64_t(deal.extra) * (units - deal.rest), deal.tiles1) : 0;
  deal.base = static_cast<int>(dealt);
  deal.rounds1 = static_cast<int>((deal.tiles1 - dealt) / units);
  deal.rest1 = static_cast<int>((deal.tiles1 - dealt) % units);
  const bool pair = p.cl == 2;
  cudaError_t e;
  if (gated) e = pair ? launch_ffn<2, true>(m, a, bf16, units, stream) : launch_ffn<1, true>(m, a, bf16, units, stream);
  else e = pair ? launch_ffn<2, false>(m, a, bf16, units, stream) : launch_ffn<1, false>(m, a, bf16, units, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  for (int i = 0; i < count; ++i) {
    const FfnProduct& q = *ps[i];
    const FfnJob& j = a.job[q.mn_a ? 1 : 0];
    if (j.split == 1) continue;
    FfnReduceArgs r;
    std::memset(&r, 0, sizeof(r));
    r.ws = partial[i];
    for (int o = 0; o < 3; ++o) r.y[o] = j.y[o];
    for (int o = 0; o < 2; ++o) r.bias[o] = a.bias[o];
    r.M = q.rows;
    r.S = j.split;
    r.N = j.N;
    r.ldw = static_cast<int>(ceil_div(q.cols, 4) * 4);
    r.outputs = q.outputs;
    r.dtype = ep.dtype;
    r.act = ep.act;
    r.gated = q.gated;
    e = launch(ffn_reduce_kernel, dim3(grid_for(r.M * (r.ldw / 4) * q.outputs, d.sms)), dim3(256), 0,
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
  return finish(lease, run_products(ps, 1, plan, ep, nullptr, ws, *d, stream));
}

int zero(void* p, int64_t bytes, cudaStream_t stream) {
  if (p == nullptr || bytes == 0) return POOT_OK;
  const cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), stream);
  return e == cudaSuccess ? POOT_OK : cuda_fail(e);
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
    return run_products(ps, count, plan, ep, bg, ws, dev, stream);
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
