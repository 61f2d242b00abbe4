// C-ABI entry points of the 8-bit operators: argument checks and launches.  No
// allocation, no host synchronisation.
#include "../../include/ortho.h"
#include "fp8.h"
#include "plan.h"

using namespace ortho;

namespace {

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

int64_t esz(const ortho_mat& a) {
  return a.dtype == ORTHO_F32 ? 4 : (a.dtype == ORTHO_BF16 ? 2 : 1);
}

// Whether every row of the matrix starts at a multiple of `bytes`.
bool rows_at(const ortho_mat* a, int64_t bytes) {
  return a == nullptr || (reinterpret_cast<uintptr_t>(a->data) % bytes == 0 && a->ld * esz(*a) % bytes == 0);
}

void* data_of(const ortho_mat* a) { return a ? a->data : nullptr; }
int64_t ld_of(const ortho_mat* a) { return a ? a->ld : 0; }

ortho_status done(hipError_t e) { return e == hipSuccess ? ORTHO_OK : ORTHO_E_HIP; }

}  // namespace

extern "C" {

ortho_status fp8_quantize(ortho_mat X, int32_t block_rows, const ortho_mat* Q, const ortho_mat* S,
                          const ortho_mat* QT, const ortho_mat* ST, void* stream) {
  const ortho_status st = validate_fp8_quantize(X, block_rows, Q, S, QT, ST);
  if (st != ORTHO_OK) return st;
  QuantArgs a{};
  a.x = X.data;
  a.ldx = X.ld;
  a.q = static_cast<uint8_t*>(data_of(Q));
  a.ldq = ld_of(Q);
  a.qt = static_cast<uint8_t*>(data_of(QT));
  a.ldqt = ld_of(QT);
  a.s = data_of(S);
  a.lds = ld_of(S);
  a.st = data_of(ST);
  a.ldst = ld_of(ST);
  a.m = static_cast<int>(X.rows);
  a.n = static_cast<int>(X.cols);
  const bool e8m0 = (S ? S : ST)->dtype == ORTHO_E8M0;
  return done(launch_fp8_quantize(a, X.dtype == ORTHO_BF16, e8m0, block_rows != 1, as_stream(stream)));
}

ortho_status rms_norm_fp8(ortho_mat X, const ortho_mat* Res, ortho_mat W, float eps,
                          const ortho_mat* Sum, const ortho_mat* Y, ortho_mat Q, ortho_mat S,
                          void* stream) {
  const ortho_status st = validate_rms_norm_fp8(X, Res, W, eps, Sum, Y, Q, S);
  if (st != ORTHO_OK) return st;
  NormArgs a{};
  a.x = X.data;
  a.ldx = X.ld;
  a.res = data_of(Res);
  a.ldres = ld_of(Res);
  a.w = W.data;
  a.w_bf = W.dtype == ORTHO_BF16;
  a.sum = data_of(Sum);
  a.ldsum = ld_of(Sum);
  a.y = data_of(Y);
  a.ldy = ld_of(Y);
  a.q = static_cast<uint8_t*>(Q.data);
  a.ldq = Q.ld;
  a.s = S.data;
  a.lds = S.ld;
  a.eps = eps;
  a.m = static_cast<int>(X.rows);
  a.n = static_cast<int>(X.cols);
  return done(launch_rms_norm_fp8(a, X.dtype == ORTHO_BF16, S.dtype == ORTHO_E8M0, as_stream(stream)));
}

size_t ortho_rms_norm_backward_workspace_size(int64_t m, int64_t n) {
  NormGradPlan p;
  return plan_norm_grad(m, n, &p) ? p.total_bytes : 0;
}

ortho_status rms_norm_backward(ortho_mat dY, ortho_mat X, ortho_mat W, float eps,
                               const ortho_mat* dSum, ortho_mat dX, ortho_mat dW, void* ws,
                               size_t ws_bytes, void* stream) {
  const ortho_status st = validate_rms_norm_backward(dY, X, W, eps, dSum, dX, dW, ws, ws_bytes);
  if (st != ORTHO_OK) return st;
  NormGradPlan plan;
  plan_norm_grad(X.rows, X.cols, &plan);
  NormGradArgs a{};
  a.dy = dY.data;
  a.lddy = dY.ld;
  a.x = X.data;
  a.ldx = X.ld;
  a.w = W.data;
  a.w_bf = W.dtype == ORTHO_BF16;
  a.dsum = data_of(dSum);
  a.lddsum = ld_of(dSum);
  a.dx = dX.data;
  a.lddx = dX.ld;
  a.dw = static_cast<float*>(dW.data);
  a.part = static_cast<float*>(ws);
  a.ldpart = plan.ld;
  a.eps = eps;
  a.m = static_cast<int>(X.rows);
  a.n = static_cast<int>(X.cols);
  a.groups = plan.groups;
  return done(launch_rms_norm_backward(a, X.dtype == ORTHO_BF16, as_stream(stream)));
}

size_t ortho_fp8_matmul_workspace_size(int64_t m, int64_t n, int64_t k) {
  Fp8MatmulPlan p;
  return plan_fp8_matmul(m, n, k, &p) ? p.total_bytes : 0;
}

ortho_status fp8_matmul(ortho_mat A, ortho_mat SA, ortho_mat B, ortho_mat SB, ortho_mat C,
                        const ortho_mat* Add, void* ws, size_t ws_bytes, void* stream) {
  const ortho_status st = validate_fp8_matmul(A, SA, B, SB, C, Add, ws, ws_bytes);
  if (st != ORTHO_OK) return st;
  Fp8GemmArgs a{};
  a.a = static_cast<const uint8_t*>(A.data);
  a.lda = A.ld;
  a.sa = {SA.data, SA.ld, SA.rows == A.rows ? 0 : 7};
  a.b = static_cast<const uint8_t*>(B.data);
  a.ldb = B.ld;
  a.sb = {SB.data, SB.ld, SB.rows == B.rows ? 0 : 7};
  a.c = C.data;
  a.ldc = C.ld;
  a.add = data_of(Add);
  a.ldadd = ld_of(Add);
  a.add_bf = Add && Add->dtype == ORTHO_BF16;
  a.M = static_cast<int>(A.rows);
  a.N = static_cast<int>(B.rows);
  a.K = static_cast<int>(A.cols);
  constexpr int64_t kMaxLd = 1 << 22;   // 256 rows within 32-bit byte offsets, scales' rows too
  a.dma = rows_at(&A, 16) && rows_at(&B, 16) && A.ld <= kMaxLd && B.ld <= kMaxLd &&
          SA.ld <= kMaxLd / 4 && SB.ld <= kMaxLd / 4;
  static_assert(kFewRows == kFewRowsMax, "");
  Fp8MatmulPlan plan;
  plan_fp8_matmul(A.rows, B.rows, A.cols, &plan);
  a.e8m0 = SA.dtype == ORTHO_E8M0;
  a.c_bf = C.dtype == ORTHO_BF16;
  a.splits = plan.splits;
  a.kchunk = plan.kchunk;
  a.part = plan.splits > 1 ? static_cast<float*>(ws) : nullptr;
  a.ldp = plan.ldp;
  return done(launch_fp8_matmul(a, as_stream(stream)));
}

}  // extern "C"
