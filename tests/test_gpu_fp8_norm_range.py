"""rms_norm_fp8 where a row times the weight leaves fp32's range though the result
is an ordinary number."""

import pytest
import torch

import fp8_ref as ref
from orthonormal_optimizer_update_amd import api
from parity_util import note
from test_gpu_fp8 import TYPES, U32, check_norm, half, normal

pytestmark = pytest.mark.gpu

SCALES = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    api.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(3, 200), (5, 1000), (4, 2048), (3, 4096), (2, 8192), (2, 16384), (2, 20000)])
def test_rows_times_weight_beyond_fp32(m, n, dtype, scale):
    """Rows of about 2^55 (2^110 n is a number) with weights of about 2^75 in every
    fifth block: their products are about 2^130, the results about 2^75.  Rows of 1
    beside them."""
    x = normal(1, m, n, dtype)
    x[0] *= 2.0 ** 55
    x[-1] *= 2.0 ** 55
    w = 1 + 0.1 * normal(3, 1, n)
    for b in range(0, n, 640):
        w[:, b:b + 128] *= 2.0 ** 75
    note(f"rms_norm_fp8 range {m}x{n} {dtype} {scale}")
    y = torch.empty(m, n, dtype=TYPES[dtype], device="cuda")
    Q, S = api.rms_norm_fp8(x.cuda(), w.cuda(), y_out=y, scale_dtype=SCALES[scale])
    torch.cuda.synchronize()
    assert torch.all(torch.isfinite(ref.e4m3_values(Q)))
    check_norm(x, None, w, 1e-6, Q, S, None, y)


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(3, 200), (5, 1000), (3, 4096), (2, 20000)])
def test_rows_times_weight_below_fp32(m, n, dtype, scale):
    """Rows of about 2^-55 (2^-110 is a normal number) without an eps, with weights of
    about 2^-80 and 2^-100: their products are subnormal or zero, the results about
    2^-80 and 2^-100."""
    x = normal(1, m, n, dtype)
    x[0] *= 2.0 ** -55
    x[-1] *= 2.0 ** -55
    w = 1 + 0.1 * normal(3, 1, n)
    for b in range(0, n, 640):
        w[:, b:b + 128] *= 2.0 ** -80
        w[:, b + 128:b + 256] *= 2.0 ** -100
    note(f"rms_norm_fp8 range below {m}x{n} {dtype} {scale}")
    y = torch.empty(m, n, dtype=TYPES[dtype], device="cuda")
    Q, S = api.rms_norm_fp8(x.cuda(), w.cuda(), eps=0.0, y_out=y, scale_dtype=SCALES[scale])
    torch.cuda.synchronize()
    check_norm(x, None, w, 0.0, Q, S, None, y)


def test_infinite_weights_and_rows_beside_large_products():
    """An infinite result is a NaN code and leaves its block's others their scale; an
    infinite row is zero but for itself."""
    n = 512
    x, w = normal(1, 4, n), 1 + 0.1 * normal(2, 1, n)
    x[1] *= 2.0 ** 55
    w[:, :128] *= 2.0 ** 75
    w[0, 7], w[0, 300] = float("inf"), float("-inf")
    x[3, 20] = float("inf")
    note("rms_norm_fp8 infinite weights")
    Q, S = api.rms_norm_fp8(x.cuda(), w.cuda())
    torch.cuda.synchronize()
    qv, sv = ref.e4m3_values(Q), ref.scale_values(S)
    bad = torch.zeros(3, n, dtype=torch.bool)
    bad[:, 7], bad[:, 300] = True, True
    assert torch.equal(torch.isnan(qv[:3]), bad)
    plain = w.clone()
    plain[0, 7], plain[0, 300] = 0.0, 0.0
    q = Q.view(torch.uint8)[:3].clone()
    q[:, 7], q[:, 300] = 0, 0
    check_norm(x[:3], None, plain, 1e-6, q.view(torch.float8_e4m3fn), S[:3], None, None)
    # 0 times an infinite weight, and the infinite element itself
    bad = torch.zeros(n, dtype=torch.bool)
    bad[7], bad[300], bad[20] = True, True, True
    assert torch.equal(torch.isnan(qv[3]), bad) and torch.all(sv[3] == 1)
    assert torch.all(torch.nan_to_num(qv[3]) == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(3, 200), (5, 1000), (2200, 1000), (4, 2048), (3, 4096), (1100, 8192), (2, 16384), (2, 20000)])
def test_gradient_of_rows_far_from_one(m, n, dtype):
    """Rows of 2^-55 without an eps under gradients of 2^-85, and of 2^55 under 2^85:
    products of 2^-140 and 2^140, means of 2^-85 and 2^85; the gradients are 2^-30 and
    2^30.  Ordinary rows beside them, and a zero gradient."""
    x, dy = normal(1, m, n, dtype), normal(2, m, n, dtype, 0.25)
    size = torch.zeros(m, 1)
    size[0], size[m - 1] = -1.0, 1.0
    x, dy = x * torch.exp2(55 * size).to(x.dtype), dy * torch.exp2(85 * size).to(dy.dtype)
    w = 1 + 0.1 * normal(4, 1, n)
    dy += x * torch.exp2(30 * size).to(dy.dtype)   # (so that the mean counts)
    if m > 2:
        dy[1] = 0.0
    note(f"rms_norm_backward far rows {m}x{n} {dtype}")
    dx, dw = api.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=0.0)
    torch.cuda.synchronize()
    wx, ww = ref.rms_norm_backward(dy, x, w, 0.0)
    t = 1 / torch.sqrt(x.double().square().mean(1, keepdim=True))
    h, u = (dy.double() * w.double()).abs(), x.double().abs() * t
    mags = t * (h + u * (h * u).mean(1, keepdim=True))
    tol = 2 * (n + 12) * U32 * mags + half(x.dtype) * wx.abs()
    assert torch.all((dx.cpu().double() - wx).abs() <= tol)
    mw = (dy.double().abs() * u).sum(0, keepdim=True)
    assert torch.all((dw.cpu().double() - ww).abs() <= (m + n / 2 + 10) * U32 * mw)
