"""Paths of the 8-bit operators that sizes, layouts and rows per workgroup
choose: the large tiles at their present bounds, codes at any byte with a bf16
result, NaN under the 8-bit instruction, and rows that share a workgroup."""

import pytest
import torch

import fp8_ref as ref
from orthonormal_optimizer_update_amd import api
from parity_util import note
from test_gpu_fp8 import (TYPES, U32, check_norm, check_product, codes_and_scales, group_tops, half,
                          matmul_reference, normal, padded, untouched, upload)

pytestmark = pytest.mark.gpu

SCALES = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    api.lib()
    torch.cuda.set_device(0)


# from this many elements of a bf16 C on, the tiles are 256 x 256
LARGE_TILES = 256 * 256 * 160


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("m,n,k", [
    (4096, 2560, 640),    # whole tiles, as many as the bound
    (5120, 2560, 128),    # more, still fewer than there are CUs, one block of k
    (3300, 3300, 300),    # ragged, with a short last block
    (20700, 520, 272),
    (2570, 4100, 1111),   # codes' rows that end inside 16 bytes
])
def test_large_tiles(m, n, k, scale):
    assert m * n >= LARGE_TILES
    for bra, brb, with_add in ((1, 128, False), (1, 1, True), (128, 128, True)):
        a, sa = codes_and_scales(m + k, m, k, bra, scale)
        b, sb = codes_and_scales(n + 2 * k, n, k, brb, scale)
        add = normal(9, m, n, "bf16") if with_add else None
        note(f"fp8_matmul {m}x{n}x{k} {scale} blocks {bra}/{brb} bf16 add={with_add}")
        c = api.fp8_matmul(upload(a), sa.cuda(), upload(b), sb.cuda(), add=None if add is None else add.cuda())
        torch.cuda.synchronize()
        want, mags = matmul_reference(a, sa, bra, b, sb, brb)
        check_product(c, want, mags, k, add, group_tops(a, sa, bra, b, sb, brb))


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,extra,offset", [
    (5, 300, 260, 3, 1), (130, 200, 385, 16, 0), (130, 200, 384, 16, 5), (300, 257, 511, 1, 0),
    (260, 260, 200, 8, 0), (70, 130, 2500, 3, 1), (129, 64, 15, 2, 1)])
def test_codes_at_any_byte(m, n, k, extra, offset, out, scale):
    """Codes, scales, Add and C at any element, for either type of C (a bf16 C's
    tiles then copy codes through registers), split over K where there are few
    tiles; nothing is written outside C."""
    for brb in (1, 128):
        a, sa = codes_and_scales(1, m, k, 1, scale)
        b, sb = codes_and_scales(2, n, k, brb, scale)
        other = "f32" if out == "bf16" else "bf16"
        add = normal(3, m, n, other)
        (va, _), (vb, _), (vadd, _) = (padded(t, extra, offset) for t in (a, b, add))
        (vsa, _), (vsb, _) = padded(sa, extra, offset), padded(sb, extra, offset)
        c, buf = padded(torch.zeros(m, n, dtype=TYPES[out]), extra, offset)
        note(f"fp8_matmul strided {m}x{n}x{k} +{extra} @{offset} {scale} blocks 1/{brb} {out}")
        api.fp8_matmul(va, vsa, vb, vsb, c, add=vadd)
        torch.cuda.synchronize()
        want, mags = matmul_reference(a, sa, 1, b, sb, brb)
        tops = group_tops(a, sa, 1, b, sb, brb) if out == "bf16" else None
        check_product(c, want, mags, k, add, tops)
        assert untouched(c, buf)


def test_large_tiles_into_a_strided_result():
    m, n, k = 3300, 3300, 160
    assert m * n >= LARGE_TILES
    a, sa = codes_and_scales(1, m, k, 1, "f32")
    b, sb = codes_and_scales(2, n, k, 128, "f32")
    add = normal(3, m, n, "bf16")
    c, buf = padded(torch.zeros(m, n, dtype=torch.bfloat16), 3, 1)
    note("fp8_matmul large tiles strided")
    api.fp8_matmul(upload(a), sa.cuda(), upload(b), sb.cuda(), c, add=padded(add, 5, 3)[0])
    torch.cuda.synchronize()
    want, mags = matmul_reference(a, sa, 1, b, sb, 128)
    check_product(c, want, mags, k, add, group_tops(a, sa, 1, b, sb, 128))
    assert untouched(c, buf)


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("m,n,k,aligned", [
    (4, 200, 300, True), (300, 300, 300, True), (70, 260, 1000, True), (300, 300, 300, False),
    (3300, 3300, 300, True), (4096, 2560, 256, True)])
def test_nan_reaches_only_its_row_and_column_of_a_bf16_result(m, n, k, aligned, scale):
    """NaN codes at the ends of k (inside the short last block), and a NaN scale,
    under the 8-bit instruction."""
    place = upload if aligned else lambda t: padded(t, 3, 1)[0]
    for brb in (1, 128):
        a, sa = codes_and_scales(1, m, k, 1, scale)
        b, sb = codes_and_scales(2, n, k, brb, scale)
        a.view(torch.uint8)[1, k - 1] = 0x7f
        b.view(torch.uint8)[150, 0] = 0xff
        if scale == "f32":
            sa[3, -1] = float("nan")
        else:
            sa.view(torch.uint8)[3, -1] = 255
        note(f"fp8_matmul NaN {m}x{n}x{k} {scale} blocks 1/{brb} bf16 aligned={aligned}")
        c = api.fp8_matmul(place(a), sa.cuda(), place(b), sb.cuda())
        torch.cuda.synchronize()
        bad = torch.isnan(c).cpu()
        want = torch.zeros(m, n, dtype=torch.bool)
        want[1], want[3], want[:, 150] = True, True, True
        assert torch.equal(bad, want)


# Rows beyond the number of workgroups (8192 for n <= 1024, 2048 to 4096 columns,
# 1024 to 8192, 512 above), and not a multiple of it.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,scale", [(9000, 520, "f32"), (5000, 2049, "e8m0"), (2500, 8192, "f32"),
                                       (1300, 16384, "e8m0"), (1100, 17000, "f32")])
def test_norm_rows_that_share_a_workgroup(m, n, scale, dtype):
    x, res = normal(1, m, n, dtype, 2.0), normal(2, m, n, dtype)
    x *= torch.exp2(torch.arange(m) % 7 - 3.0)[:, None]   # no two neighbours alike
    w = 1 + 0.1 * normal(3, 1, n)
    note(f"rms_norm_fp8 {m}x{n} {dtype} {scale}")
    y = torch.empty_like(x, device="cuda")
    total = x.cuda()   # in place
    Q, S = api.rms_norm_fp8(total, w.cuda(), residual=res.cuda(), sum_out=total, y_out=y, scale_dtype=SCALES[scale])
    torch.cuda.synchronize()
    check_norm(x, res, w, 1e-6, Q, S, total, y)


# (2048 workgroups for n <= 1024, 1024 above)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(5000, 520), (2500, 2049), (2100, 8192), (2100, 9000), (1100, 17000)])
def test_norm_gradient_rows_that_share_a_workgroup(m, n, dtype):
    """dw's terms dy u pass through at most ceil(m / 1024) <= 5 additions in a
    workgroup, 1024 / 16 + 64 among the parts, and 60 roundings in u (sums of 32
    per thread, 6 levels in a wave, 16 waves; the mean, eps, root, reciprocal and
    products): under 256 half steps."""
    x, dy, ds = normal(1, m, n, dtype, 2.0), normal(2, m, n, dtype, 1e-3), normal(3, m, n, dtype, 1e-3)
    x *= torch.exp2(torch.arange(m) % 7 - 3.0)[:, None]
    w = 1 + 0.1 * normal(4, 1, n)
    wx, ww = ref.rms_norm_backward(dy, x, w, 1e-6, ds)
    t = 1 / torch.sqrt(x.double().square().mean(1, keepdim=True) + 1e-6)
    h, u = (dy.double() * w.double()).abs(), x.double().abs() * t
    mags = t * (h + u * (h * u).mean(1, keepdim=True)) + ds.double().abs()
    tol = 2 * (n + 12) * U32 * mags + half(x.dtype) * wx.abs()
    mw = (dy.double().abs() * u).sum(0, keepdim=True)
    for into in ("new", "dy"):
        note(f"rms_norm_backward {m}x{n} {dtype} into {into}")
        tdy = dy.cuda()
        dx, dw = api.rms_norm_backward(tdy, x.cuda(), w.cuda(), dX=tdy if into == "dy" else None, dsum=ds.cuda())
        torch.cuda.synchronize()
        assert torch.all((dx.cpu().double() - wx).abs() <= tol)
        assert torch.all((dw.cpu().double() - ww).abs() <= 256 * U32 * mw)
