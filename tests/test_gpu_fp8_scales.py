"""Block scales at the ends of their types: elements that are representable
although the product of the two scales is not."""

import pytest
import torch

import fp8_ref as ref
from orthonormal_optimizer_update_amd import api
from parity_util import note
from test_gpu_fp8 import TYPES, check_product, group_tops, matmul_reference, padded, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    api.lib()
    torch.cuda.set_device(0)


LEAST = 2.0 ** -9   # smallest positive code


def operand(seed, rows, k, block_rows, patterns, dtype):
    """Codes and scales whose blocks of rows go through `patterns`, pairs of
    (what the codes are, scale)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.zeros(rows, k)
    nkb = ref.cdiv(k, 128)
    s = torch.ones(ref.cdiv(rows, block_rows), nkb)
    for i in range(s.size(0)):
        kind, scale = patterns[i % len(patterns)]
        at = slice(i * block_rows, min((i + 1) * block_rows, rows))
        s[i] = scale
        if kind == "one":         # one smallest code in each block
            q[at, ::128] = LEAST
        elif kind == "full":
            q[at] = 448.0
        elif kind == "normal":
            q[at] = torch.randn(q[at].shape, generator=g)
    q = q.to(torch.float8_e4m3fn)
    if dtype == torch.float8_e8m0fnu:
        b = (torch.log2(s.double()).round() + 127).to(torch.uint8)
        s = b.view(torch.float8_e8m0fnu)
    return q, s


def check(a, sa, bra, b, sb, brb, out, place=upload):
    m, n, k = a.size(0), b.size(0), a.size(1)
    c = api.fp8_matmul(place(a), sa.cuda(), place(b), sb.cuda(), out_dtype=out)
    torch.cuda.synchronize()
    want, mags = matmul_reference(a, sa, bra, b, sb, brb)
    assert torch.all(mags < 3e38)
    tops = group_tops(a, sa, bra, b, sb, brb) if out == torch.bfloat16 else None
    # (from 2^-126 on, steps of 2^-149 are no coarser than what check_product counts)
    assert torch.all((mags == 0) | (mags >= 2.0 ** -126))
    assert torch.all(c.cpu()[mags == 0] == 0)
    check_product(c, want, mags, k, None, tops)


POWERS_A = [("zero", 2.0 ** 127), ("one", 2.0 ** 127), ("full", 2.0 ** -127), ("normal", 1.0)]
POWERS_B = [("one", 2.0 ** 10), ("full", 2.0 ** -23), ("normal", 1.0)]
SIZES = [(5, 384, 300), (29, 400, 128), (40, 390, 1700), (300, 700, 384), (520, 384, 1111)]
LARGE = [(4096, 2560, 256), (3300, 3300, 300)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("m,n,k", SIZES + LARGE)
def test_products_of_scales_beyond_fp32(m, n, k, scale, out):
    """2^127 x 2^10 with sums of zero and of 2^-18, and 2^-127 x 2^-23 with sums of
    448^2 128: the scales' products are infinite and zero, the elements 0, 2^119 (a
    multiple of it for several blocks) and 2^-125.4.  (b's one code meets full rows of
    a: 2^-127 2^10 2^-9 448 = 2^-117.)"""
    dtype = torch.float32 if scale == "f32" else torch.float8_e8m0fnu
    for bra, brb in ((1, 128), (1, 1)) if m > 256 else ((1, 128), (1, 1), (128, 1)):
        a, sa = operand(1, m, k, bra, POWERS_A, dtype)
        b, sb = operand(2, n, k, brb, POWERS_B, dtype)
        note(f"fp8_matmul scales beyond fp32 {m}x{n}x{k} {scale} blocks {bra}/{brb} {out}")
        check(a, sa, bra, b, sb, brb, TYPES[out])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("m,n,k", [(5, 300, 260), (300, 400, 520), (60, 390, 1701), (130, 260, 15), (40, 300, 3), (9, 100, 9)])
def test_products_of_scales_beyond_fp32_with_codes_at_any_byte(m, n, k, scale, out):
    """The same with rows of codes at any byte, and rows shorter than 16."""
    dtype = torch.float32 if scale == "f32" else torch.float8_e8m0fnu
    for bra, brb in ((1, 128), (1, 1)):
        a, sa = operand(1, m, k, bra, POWERS_A, dtype)
        b, sb = operand(2, n, k, brb, POWERS_B if k > 100 else POWERS_B[:1] + POWERS_B[2:], dtype)
        note(f"fp8_matmul scales beyond fp32 at any byte {m}x{n}x{k} {scale} blocks {bra}/{brb} {out}")
        check(a, sa, bra, b, sb, brb, TYPES[out], lambda t: padded(t, 3, 1)[0])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES + LARGE)
def test_subnormal_products_of_fp32_scales(m, n, k, out):
    """3.1e-22 x 1.03e-22 is 22.8 steps of fp32's smallest number, 23 rounded (1%
    off); the element, 448^2 k times it, is a normal number."""
    pa = [("full", 3.1e-22), ("normal", 1.7), ("full", 3.3e-22)]
    pb = [("full", 1.03e-22), ("normal", 0.03)]
    for bra, brb in ((1, 128), (1, 1)):
        a, sa = operand(1, m, k, bra, pa, torch.float32)
        b, sb = operand(2, n, k, brb, pb, torch.float32)
        note(f"fp8_matmul subnormal product of scales {m}x{n}x{k} blocks {bra}/{brb} {out}")
        check(a, sa, bra, b, sb, brb, TYPES[out])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(7, 300, 260), (150, 260, 1100), (4096, 2560, 128), (3300, 3300, 160)])
def test_extreme_scales_change_no_other_element(m, n, k, out):
    """Rows and columns without an extreme scale come out bit for bit as they do
    among moderate ones; negative and zero scales count as they are."""
    g = torch.Generator().manual_seed(3)
    a = torch.randn(m, k, generator=g).to(torch.float8_e4m3fn)
    b = torch.randn(n, k, generator=g).to(torch.float8_e4m3fn)
    sa = torch.rand(m, ref.cdiv(k, 128), generator=g) * 0.02 + 1e-3
    sa[3::5] *= -1
    sa[4] = 0.0
    for brb in (1, 128):
        sb = torch.rand(ref.cdiv(n, brb), ref.cdiv(k, 128), generator=g) * 0.02 + 1e-3
        sb[0::2] *= -1
        note(f"fp8_matmul extreme scales beside others {m}x{n}x{k} blocks 1/{brb} {out}")
        ua, ub = upload(a), upload(b)
        plain = api.fp8_matmul(ua, sa.cuda(), ub, sb.cuda(), out_dtype=TYPES[out])
        wild, rows = sa.clone(), [1, m - 2]
        wild[rows[0]], wild[rows[1]] = 1e-40, 3e38
        mixed = api.fp8_matmul(ua, wild.cuda(), ub, sb.cuda(), out_dtype=TYPES[out])
        torch.cuda.synchronize()
        keep = [i for i in range(m) if i not in rows]
        assert torch.equal(plain[keep], mixed[keep])
        want, mags = matmul_reference(a, sa, 1, b, sb, brb)
        tops = group_tops(a, sa, 1, b, sb, brb) if out == "bf16" else None
        check_product(plain, want, mags, k, None, tops)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(4352, 4608, 256), (4350, 4600, 250), (300, 400, 1700), (20, 300, 700)])
def test_far_scales_in_some_tiles_with_add_in_place(m, n, k, out):
    """C = Add, in tiles that one workgroup takes in turn, with far scales in some."""
    a, sa = operand(1, m, k, 1, POWERS_A, torch.float32)
    b, sb = operand(2, n, k, 128, POWERS_B, torch.float32)
    sa[m // 3:] = 1.0
    add = torch.randn(m, n, generator=torch.Generator().manual_seed(3)).to(TYPES[out])
    note(f"fp8_matmul far scales in some tiles {m}x{n}x{k} {out}")
    c = add.cuda()
    api.fp8_matmul(upload(a), sa.cuda(), upload(b), sb.cuda(), c, add=c)
    torch.cuda.synchronize()
    want, mags = matmul_reference(a, sa, 1, b, sb, 128)
    tops = group_tops(a, sa, 1, b, sb, 128) if out == "bf16" else None
    check_product(c, want, mags, k, add, tops)
