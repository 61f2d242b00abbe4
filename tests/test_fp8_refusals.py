"""Refusals of the 8-bit operators' argument checks that need no GPU."""

import ctypes

import pytest
import torch

from orthonormal_optimizer_update_amd import api
from test_fp8_cpu import BF, C8, DTYPE, E8, F, FAKE, LAYOUT, M, PARAM, SHAPE, WS, ref


def apart(i):
    """Addresses 1 MiB apart."""
    return FAKE + (i << 20)


@pytest.mark.parametrize("scales", [F, E8])
def test_norms_refuse_a_weight_narrower_than_the_data(scales):
    """A bf16 weight goes with bf16 data; an fp32 one with either."""
    L = api.lib()
    for x, w, want in ((F, BF, True), (BF, C8, True), (BF, E8, True), (F, F, False), (BF, F, False), (BF, BF, False)):
        got = L.rms_norm_fp8(M(30, 200, x), None, M(1, 200, w, data=apart(1)), 1e-6, None, None,
                             M(30, 200, C8, data=apart(2)), M(31 if not want else 30, 2, scales, data=apart(3)), None)
        assert (got == DTYPE) == want   # (an accepted pair goes on to the scales' wrong shape)
        ws = ctypes.c_void_p(FAKE)
        got = L.rms_norm_backward(M(30, 200, x), M(30, 200, x, data=apart(1)), M(1, 200, w, data=apart(2)), 1e-6, None,
                                  M(30, 200, x, data=apart(3)), M(1, 200, F, data=apart(4)), ws, 0, None)
        assert (got == DTYPE) == want   # (and to the workspace's size)


# Places of an m x n matrix against another at FAKE with rows of 512 bytes (200
# columns of bf16 take 400): same or fully apart is accepted, else refused.
APART = [(FAKE + (1 << 20), 200), (FAKE + 30 * 512, 256), (FAKE - 30 * 512, 256),   # behind, before
         (FAKE + 400, 256 * 2), (FAKE + 30 * 512 + 112, 200)]
SAME = [(FAKE, 256)]
PARTLY = [(FAKE + 512, 256), (FAKE - 512, 256),      # a row on
          (FAKE + 2, 256), (FAKE - 2, 256),          # a column on
          (FAKE + 29 * 512 + 398, 256),              # the last element alone
          (FAKE, 200), (FAKE, 512),                  # the same start, other rows
          (FAKE + 256, 256), (FAKE + 5 * 512 + 396, 201), (FAKE - 400, 256)]


@pytest.mark.parametrize("place", APART + SAME + PARTLY)
def test_outputs_of_the_norms_that_overlap_an_input_partly(place):
    L, m, n = api.lib(), 30, 200
    data, ld = place
    x, out = M(m, n, BF, ld=256), M(m, n, BF, ld=ld, data=data)
    far, q, s = M(m, n, BF, data=apart(8)), M(m, n, C8, data=apart(9)), M(m, 1, F, data=apart(10))
    w, dw = M(1, n, F, data=apart(11)), M(1, n, F, data=apart(12))
    # (what passes the check of overlaps meets the scales' wrong shape, or no workspace)
    if place == APART[3]:      # every other row's end: rows of 1024 bytes in gaps of 512 bytes' rows
        x = M(m, n, BF, ld=512)
    want = SHAPE if place in APART + SAME else LAYOUT
    assert L.rms_norm_fp8(x, None, w, 1e-6, ref(out), None, q, s, None) == want
    assert L.rms_norm_fp8(far, ref(x), w, 1e-6, ref(out), None, q, s, None) == want
    want = SHAPE if place in APART else LAYOUT      # y has memory of its own
    assert L.rms_norm_fp8(x, None, w, 1e-6, None, ref(out), q, s, None) == want
    assert L.rms_norm_fp8(far, ref(x), w, 1e-6, None, ref(out), q, s, None) == want
    assert L.rms_norm_fp8(far, None, w, 1e-6, ref(x), ref(out), q, s, None) == want
    want = WS if place in APART + SAME else LAYOUT
    for dy, xx, ds in ((x, far, None), (far, x, None), (far, far, x)):
        assert L.rms_norm_backward(dy, xx, w, 1e-6, ref(ds), out, dw, None, 0, None) == want


@pytest.mark.parametrize("place", APART + SAME + PARTLY)
def test_add_that_overlaps_the_product_partly(place):
    m, n, k = 30, 200, 128
    data, ld = place
    add = M(m, n, BF, ld=512 if place == APART[3] else 256)
    c = M(m, n, BF, ld=ld, data=data)
    a, sa = M(m, k, C8, data=apart(8)), M(m, 1, F, data=apart(9))
    b, sb = M(n, k, C8, data=apart(10)), M(n, 1, F, data=apart(11))
    want = WS if place in APART + SAME else LAYOUT
    assert api.lib().fp8_matmul(a, sa, b, sb, c, ref(add), None, 0, None) == want
    # another type of the same start, and one in the second half of its rows
    c = M(m, n, F, ld=128 if n <= 128 else 256)
    assert api.lib().fp8_matmul(a, sa, b, sb, c, ref(add), None, 0, None) == LAYOUT
    c = M(m, n, F, ld=400, data=FAKE + 400)
    add = M(m, n, BF, ld=800)
    assert api.lib().fp8_matmul(a, sa, b, sb, c, ref(add), None, 0, None) == WS


def test_single_rows_that_overlap():
    L, n = api.lib(), 64
    x, w, q, s = M(1, n, F), M(1, n, F, data=apart(1)), M(1, n, C8, data=apart(2)), M(1, 2, F, data=apart(3))
    for data, ld, want in ((FAKE, n, SHAPE), (FAKE, 999, SHAPE), (FAKE + 4, n, LAYOUT), (FAKE + 4 * n, n, SHAPE)):
        assert L.rms_norm_fp8(x, None, w, 1e-6, ref(M(1, n, F, ld=ld, data=data)), None, q, s, None) == want


def test_overlaps_of_the_largest_descriptors():
    """Rows and leading dimensions at their limits: the extent passes 64 bits."""
    L, m, n, ld = api.lib(), 1 << 30, 4, 1 << 40
    x, w, q, s = M(m, n, F, ld=ld), M(1, n, F, data=FAKE - 4096), M(m, n, C8, data=FAKE - 8192), M(m, 2, F, data=FAKE)
    for off, want in ((0, SHAPE), (4, LAYOUT), (16, SHAPE), (4 * ld, LAYOUT), (4 * ld + 16, SHAPE)):
        assert L.rms_norm_fp8(x, None, w, 1e-6, ref(M(m, n, F, ld=ld, data=FAKE + off)), None, q, s, None) == want


def test_workspace_counts_the_bytes_behind_its_address():
    """A tensor that repeats its elements holds only those; a strided one at least
    as many as it has."""
    t = torch.zeros(4, 4)
    ws = torch.zeros(1024, dtype=torch.uint8)
    assert api._check_ws(ws, t) == (ws.data_ptr(), 1024)
    assert api._check_ws(ws.view(torch.float32), t) == (ws.data_ptr(), 1024)
    assert api._check_ws(ws.view(32, 32)[:, :8], t)[1] == 256
    assert api._check_ws(ws[::2], t)[1] == 512
    assert api._check_ws(ws[:1].expand(1 << 20), t)[1] == 1
    assert api._check_ws(ws[:256].view(1, 256).expand(64, 256), t)[1] == 256
    assert api._check_ws(ws[:0], t)[1] == 0


@pytest.mark.parametrize("block_rows", [0, -1, -128])
def test_block_rows_below_one_reach_the_library(block_rows):
    """(Where no outputs are given they are allocated first; then comes what is wrong
    with the call: here the device, on a GPU block_rows.)"""
    with pytest.raises(ValueError, match="GPU"):
        api.fp8_quantize(torch.zeros(4, 256), block_rows=block_rows)


@pytest.mark.gpu
@pytest.mark.parametrize("block_rows", [0, -1, -128, 2, 64, 256])
def test_block_rows_other_than_1_and_128(block_rows):
    with pytest.raises(api.OrthoError) as e:
        api.fp8_quantize(torch.zeros(4, 256, device="cuda"), block_rows=block_rows, transposed=True)
    assert e.value.status == PARAM


def test_limits_of_sizes():
    """2^24 blocks or tiles of 128 x 128, and 2^30 rows or columns."""
    L = api.lib()

    need = api.fp8_matmul_workspace_size
    assert need(1 << 30, 128, 1) > 0 and need(1 << 30, 256, 1) == 0 and need((1 << 30) + 1, 1, 1) == 0
    m, n = 1 << 30, 256
    got = L.fp8_matmul(M(m, 1, C8), M(m, 1, F, data=apart(1)), M(n, 1, C8, data=apart(2)), M(n, 1, F, data=apart(3)),
                       M(m, n, BF, data=apart(4)), None, ctypes.c_void_p(FAKE), 1 << 40, None)
    assert got == SHAPE
    x, q, s = M(1 << 20, 1 << 18, F), M(1 << 20, 1 << 18, C8, data=apart(1)), M(1 << 20, 1 << 11, F, data=apart(2))
    assert L.fp8_quantize(x, 1, ref(q), ref(s), None, None, None) == SHAPE   # 2^24 blocks
