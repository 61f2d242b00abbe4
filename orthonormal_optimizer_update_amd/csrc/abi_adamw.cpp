// C-ABI entry points of AdamW and the gradients' norm: argument checks, tables of
// tensors and launches.  No device allocation, no host synchronisation.
#include <math.h>

#include <limits>

#include "../../include/ortho.h"
#include "adamw.h"
#include "plan.h"

using namespace ortho;

namespace {

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

bool consecutive(const ortho_mat& a) { return a.rows == 1 || a.ld == a.cols; }

uint32_t pitch(const ortho_mat& a) { return a.rows == 1 ? 0 : static_cast<uint32_t>(a.ld); }

constexpr int64_t kMaxUnits = int64_t{1} << 30;  // of one launch over more than one tensor

AdamwScalars scalars(const ortho_adamw& h) {
  AdamwScalars s{};
  s.b1 = static_cast<float>(h.beta1);
  s.c1 = static_cast<float>(1.0 - h.beta1);
  s.b2 = static_cast<float>(h.beta2);
  s.c2 = static_cast<float>(1.0 - h.beta2);
  s.eps = static_cast<float>(h.eps);
  s.lr = h.lr;
  s.wd = h.weight_decay;
  s.log_b1 = log(h.beta1);
  s.log_b2 = log(h.beta2);
  const double t = static_cast<double>(h.step < 1 ? 1 : h.step);
  s.keep = static_cast<float>(1.0 - h.lr * h.weight_decay);
  s.size = static_cast<float>(h.lr / -expm1(t * s.log_b1));
  s.root = static_cast<float>(1.0 / sqrt(-expm1(t * s.log_b2)));
  s.step = h.step;
  s.seed_lo = static_cast<uint32_t>(h.seed);
  s.seed_hi = static_cast<uint32_t>(h.seed >> 32);
  s.lr_dev = h.lr_dev;
  s.step_dev = h.step_dev;
  s.factor = h.factor;
  return s;
}

int32_t kind_of(const ortho_mat& x, const ortho_mat& g) {
  return (x.dtype == ORTHO_BF16 ? kBf16Weight : 0) | (g.dtype == ORTHO_BF16 ? kBf16Gradient : 0);
}

// A launch's table while it is filled.
template <typename Table>
struct Filling {
  typedef decltype(Table::units) Unit;
  Table a{};
  int count = 0;
  bool fits(int64_t units) const {
    return count < Table::kMost && (sizeof(Unit) == 8 || a.units + units <= kMaxUnits);
  }
  auto& add(int64_t units) {
    a.first[count] = a.units;
    a.units += static_cast<Unit>(units);
    return a.t[count++];
  }
  void close() {
    for (int i = count; i < kLanes; ++i) a.first[i] = std::numeric_limits<Unit>::max();
  }
  void clear() {
    count = 0;
    a.units = 0;
  }
};

}  // namespace

extern "C" {

size_t ortho_grad_norm_workspace_size(int32_t count) { return grad_norm_ws_bytes(count); }

ortho_status grad_norm(int32_t count, const ortho_mat* G, double max_norm, float* out, void* ws,
                       size_t ws_bytes, void* stream) {
  const ortho_status st = validate_grad_norm(count, G, max_norm, out, ws, ws_bytes);
  if (st != ORTHO_OK) return st;
  static_assert(kNormPerLaunch == NormParts::kMost, "");
  double* const part = static_cast<double*>(ws);
  Filling<NormParts> f;
  int parts = 0;
  auto flush = [&]() -> hipError_t {
    if (f.count == 0) return hipSuccess;
    f.close();
    const int groups = static_cast<int>(f.a.units < kNormGroups ? f.a.units : kNormGroups);
    f.a.part = part + parts;
    parts += groups;
    const hipError_t e = launch_grad_norm_parts(f.a, groups, as_stream(stream));
    f.clear();
    return e;
  };
  for (int32_t i = 0; i < count; ++i) {
    const bool flat = consecutive(G[i]);
    const int64_t rows = flat ? 1 : G[i].rows, cols = flat ? G[i].rows * G[i].cols : G[i].cols;
    const Deal d = deal(rows, cols, G[i].dtype == ORTHO_BF16 ? 32 : 16);
    if (!f.fits(d.units) && flush() != hipSuccess) return ORTHO_E_HIP;
    f.add(d.units) = {G[i].data, G[i].ld, cols, static_cast<int32_t>(rows), static_cast<int32_t>(d.across),
                      d.lanes, G[i].dtype == ORTHO_BF16};
  }
  if (flush() != hipSuccess) return ORTHO_E_HIP;
  return launch_grad_norm_join(part, parts, max_norm, out, as_stream(stream)) == hipSuccess ? ORTHO_OK
                                                                                           : ORTHO_E_HIP;
}

ortho_status adamw_step(int32_t count, const ortho_mat* X, const ortho_mat* G, const ortho_mat* M,
                        const ortho_mat* V, const ortho_mat* SM, const ortho_mat* SV,
                        const ortho_adamw* h, void* stream) {
  const ortho_status st = validate_adamw(count, X, G, M, V, SM, SV, h);
  if (st != ORTHO_OK) return st;
  const bool stochastic = h->stochastic != 0;
  Filling<AdamwFlat> flat;
  Filling<AdamwRows> rows;
  flat.a.h = rows.a.h = scalars(*h);
  auto flush_flat = [&]() -> hipError_t {
    if (flat.count == 0) return hipSuccess;
    flat.close();
    const hipError_t e = launch_adamw_flat(flat.a, stochastic, as_stream(stream));
    flat.clear();
    return e;
  };
  auto flush_rows = [&]() -> hipError_t {
    if (rows.count == 0) return hipSuccess;
    rows.close();
    int kind = rows.a.t[0].kind;
    for (int i = 0; i < rows.count; ++i)
      if (rows.a.t[i].kind != kind || rows.a.t[i].sm == nullptr) kind = -1;
    const hipError_t e = launch_adamw_rows(rows.a, kind, stochastic, as_stream(stream));
    rows.clear();
    return e;
  };
  for (int32_t i = 0; i < count; ++i) {
    const bool codes = M[i].dtype == ORTHO_E4M3;
    if (!codes && consecutive(X[i]) && consecutive(G[i]) && consecutive(M[i]) && consecutive(V[i])) {
      const int64_t n = X[i].rows * X[i].cols, units = (n + kUnit - 1) / kUnit;
      if (!flat.fits(units) && flush_flat() != hipSuccess) return ORTHO_E_HIP;
      flat.add(units) = {X[i].data, G[i].data, static_cast<float*>(M[i].data), static_cast<float*>(V[i].data),
                         n, i, kind_of(X[i], G[i])};
      continue;
    }
    // (a quarter: what ends a row takes longer than padding does; 2331 x 1537 in codes with
    // fp32 gradients in pieces of 2048 columns 12.7 us, of 256, an eighth, 14.0)
    const Deal d = deal(X[i].rows, X[i].cols, 8, 4);
    if (!rows.fits(d.units) && flush_rows() != hipSuccess) return ORTHO_E_HIP;
    RowTensor& t = rows.add(d.units);
    t = {};
    t.x = X[i].data;
    t.g = G[i].data;
    t.m = M[i].data;
    t.v = V[i].data;
    t.ldx = pitch(X[i]);
    t.ldg = pitch(G[i]);
    t.ldm = pitch(M[i]);
    t.ldv = pitch(V[i]);
    if (codes) {
      t.sm = static_cast<float*>(SM[i].data);
      t.sv = static_cast<float*>(SV[i].data);
      t.ldsm = pitch(SM[i]);
      t.ldsv = pitch(SV[i]);
    }
    t.rows = static_cast<int32_t>(X[i].rows);
    t.cols = static_cast<int32_t>(X[i].cols);
    t.across = static_cast<int32_t>(d.across);
    t.lanes = d.lanes;
    t.index = i;
    t.kind = kind_of(X[i], G[i]);
  }
  if (flush_flat() != hipSuccess || flush_rows() != hipSuccess) return ORTHO_E_HIP;
  return ORTHO_OK;
}

}  // extern "C"
