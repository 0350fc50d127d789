// Host side of the products of ffn_gemm.cuh, shared by the translation units
// that launch them: argument checks on spans, operands and their repacking,
// tile plans, workspaces, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "poot_ffn.h"
#include "ffn_elem.cuh"
#include "ffn_gemm.cuh"
#include "host.cuh"

namespace poot_host {

using namespace poot;

struct DeviceInfo {
  int dev = 0;
  int sms = 0;
};

// Sizes: the kernels round them up to tiles, vectors and warps' shares of K (at
// most 2304 more, the repacking's two spans of a row) in 32 bits
constexpr int64_t kMaxDim = POOT_FFN_MAX_SIZE;
static_assert(kMaxDim + 2304 < (int64_t(1) << 31), "32-bit index arithmetic");

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

inline bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && M <= kMaxDim && N <= kMaxDim && K <= kMaxDim && M * N <= kMaxSpan &&
         M * K <= kMaxSpan && N * K <= kMaxSpan;
}

// The row pitch `ld` of an argument (0: contiguous rows) into *out; false: none
// that a [rows, cols] matrix can have.  A single row has no pitch, whatever ld
// says: it gets one that suits TMA.
inline bool row_pitch(int64_t rows, int64_t cols, int64_t ld, int64_t* out) {
  if (ld == 0) ld = cols;
  if (ld < cols || (rows > 1 && ld > kMaxSpan / rows)) return false;
  *out = rows > 1 ? ld : (cols + 7) / 8 * 8;
  return true;
}

// bytes of a [rows, cols] matrix of 2-byte elements, rows ld apart
inline int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld) {
  return rows <= 0 || cols <= 0 ? 0 : 2 * ((rows - 1) * ld + cols);
}

// outputs may overlap neither an input nor one another; 2-byte alignment
inline int check_spans(std::initializer_list<Span> in, std::initializer_list<Span> out) {
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
  int64_t unit;  // elements whose multiple a copy's pitch is
  explicit Packer(int64_t unit_ = 8) : unit(unit_) { std::memset(&a, 0, sizeof(a)); }
  void need(Operand* o) {
    if (o->p == nullptr || o->tma()) return;
    const int t = a.count++;
    ops[t] = o;
    a.src[t] = static_cast<const uint16_t*>(o->p);
    a.ld[t] = o->ld;
    a.ldd[t] = ceil_div(o->cols, unit) * unit;
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
  bool logits = false;  // both operands K-major, one product (the vocabulary head's)
  Operand a[2], b[2];
  int parts = 1, outputs = 1;
  int64_t rows = 0, cols = 0, kext = 0;  // of one output; K extent of one part
  void* y[3] = {nullptr, nullptr, nullptr};
  int64_t ldy = 0;      // row pitch of y; 0: contiguous
  bool sum = false;     // the output stays FP32 sums, added up over launches
  int64_t kb() const { return ceil_div(kext, kFfnBK) * parts; }
  size_t partial_bytes(int split) const {
    return split > 1 || sum ? round256(size_t(split) * (gated ? 2 : outputs) * rows * ceil_div(cols, 4) * 16) : 0;
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

inline double plan_time(const FfnProduct* const* ps, int count, const FfnShape& s, const int* split, int sms, double bytes) {
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

inline FfnPlan plan_ffn(const FfnProduct* const* ps, int count, int sms, bool may_split = true) {
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
      for (int S = 2; may_split && !q.sum && S <= 16 && tiles * S <= 2 * (sms / s.cl) && q.kb() >= 4 * S; S *= 2) {
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
inline bool lease_products(const FfnProduct* const* ps, int count, FfnPlan* plan, int dtype, size_t more, const DeviceInfo& d,
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
// launch_kernel(maps, args, bf16, units) launches the kernel of the products,
// launch_reduce(product, job, partial sums) the second half of a split one.
template <typename Kernel, typename Reduce>
int run_products(const FfnProduct* const* ps, int count, const FfnPlan& p, const FfnEpilogue& ep,
                 const FfnBiasGrad* bg, char* ws, const DeviceInfo& d, Kernel&& launch_kernel, Reduce&& launch_reduce) {
  const FfnSpace space(ps, count, p, ep.dtype, d.sms);
  float* const partial[2] = {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + space.partial[0])};
  const bool bf16 = ep.dtype == POOT_DTYPE_BF16;
  FfnGemmArgs a;
  FfnMaps m;
  std::memset(&a, 0, sizeof(a));
  std::memset(&m, 0, sizeof(m));
  a.bn = p.bn;
  a.a_rows = kFfnBM;
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
    const int ny = q.gated ? (ep.save ? 3 : 1) : (q.y[0] != nullptr ? q.outputs : 0);
    const int64_t ldy = q.ldy != 0 ? q.ldy : q.cols;
    j.tma_store = j.split == 1 && !q.sum && ldy % 8 == 0;
    for (int o = 0; o < ny; ++o) {
      j.y[o] = static_cast<uint16_t*>(q.y[o]);
      if (!aligned(q.y[o], 16)) j.tma_store = 0;
    }
    if (q.logits && p.cl == 1 && q.rows < kFfnBM) {
      a.a_rows = static_cast<int>(ceil8(q.rows));
      a.stages = std::min(FfnLayout::RING_BYTES / (a.a_rows * kFfnBK * 2 * ffn_sub(1) + ffn_b_bytes(1, p.bn)), kFfnMaxStages);
    }
    auto encode = [&](CUtensorMap* map, const Operand& o, bool mn, int rows) {
      return encode_2d(map, o.p, o.cols, o.rows, kFfnBK, mn ? kFfnBK : static_cast<uint32_t>(rows),
                       CU_TENSOR_MAP_SWIZZLE_128B, bf16, o.ld);
    };
    const int na = q.gated ? 1 : (q.mn_a ? q.outputs : q.parts), nb = q.gated ? 2 : (q.mn_a ? 1 : q.parts);
    bool ok = true;
    for (int o = 0; o < na; ++o) ok = ok && encode(&m.a[ji][o], q.a[o], q.mn_a, a.a_rows);
    for (int o = 0; o < nb; ++o) ok = ok && encode(&m.b[ji][o], q.b[o], !q.gated && !q.logits, q.logits ? p.bn / p.cl : p.bn / 2);
    if (j.tma_store)
      for (int o = 0; o < ny; ++o)
        ok = ok && encode_2d(&m.y[ji][o], q.y[o], q.cols, q.rows, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, bf16, ldy);
    if (j.split > 1 || q.sum)
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
  const cudaError_t e = launch_kernel(m, a, bf16, units);
  if (e != cudaSuccess) return cuda_fail(e);
  for (int i = 0; i < count; ++i) {
    const FfnProduct& q = *ps[i];
    const FfnJob& j = a.job[q.mn_a ? 1 : 0];
    if (j.split == 1 || q.sum) continue;
    const cudaError_t r = launch_reduce(q, j, partial[i]);
    if (r != cudaSuccess) return cuda_fail(r);
  }
  return POOT_OK;
}

inline int finish(WorkspaceLease& lease, int rc) {
  const cudaError_t e = lease.release();
  if (rc != POOT_OK) return rc;
  return e == cudaSuccess ? POOT_OK : cuda_fail(e);
}

inline int zero(void* p, int64_t bytes, cudaStream_t stream) {
  if (p == nullptr || bytes == 0) return POOT_OK;
  const cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), stream);
  return e == cudaSuccess ? POOT_OK : cuda_fail(e);
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

}  // namespace poot_host
