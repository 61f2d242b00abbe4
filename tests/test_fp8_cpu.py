"""The 8-bit operators' argument checks, which need no GPU: documented status
codes before anything touches the device, and the binding's refusals."""

import ctypes

import pytest
import torch

from orthonormal_optimizer_update_amd import api

FAKE = 0x7F0000000000   # never dereferenced: validation fails first
F, BF, C8, E8 = api.ORTHO_F32, api.ORTHO_BF16, api.ORTHO_E4M3, api.ORTHO_E8M0
OK, NULL, SHAPE, DTYPE, LAYOUT, WS, PARAM = 0, 1, 2, 3, 5, 6, 7


def M(rows, cols, dtype, ld=None, data=FAKE):
    return api.OrthoMat(data, rows, cols, ld if ld is not None else cols, dtype)


def ref(m):
    return None if m is None else ctypes.byref(m)


def test_constants():
    assert (F, BF, C8, E8) == (0, 1, 2, 3)


@pytest.mark.parametrize("change,want", [
    (dict(br=2), PARAM), (dict(br=0), PARAM), (dict(x=M(300, 200, BF, data=None)), NULL),
    (dict(x=M(300, 200, C8)), DTYPE), (dict(x=M(300, 200, 9)), DTYPE), (dict(x=M(300, 200, -1)), DTYPE),
    (dict(x=M(0, 200, BF)), SHAPE), (dict(x=M(300, 200, BF, ld=199)), LAYOUT),
    (dict(s=None), NULL), (dict(st=None), NULL), (dict(q=None, s=None, qt=None, st=None), NULL),
    (dict(q=M(300, 200, BF)), DTYPE), (dict(q=M(200, 300, C8)), SHAPE), (dict(q=M(300, 200, C8, data=None)), NULL),
    (dict(q=M(300, 200, C8, ld=100)), LAYOUT), (dict(s=M(300, 1, F)), SHAPE), (dict(s=M(299, 2, F)), SHAPE),
    (dict(s=M(300, 2, BF)), DTYPE), (dict(s=M(300, 2, E8)), DTYPE), (dict(qt=M(300, 200, C8)), SHAPE),
    (dict(st=M(200, 2, F)), SHAPE), (dict(br=128), SHAPE), (dict(s=M(300, 2, F, ld=1)), LAYOUT),
])
def test_quantize_argument_errors(change, want):
    a = dict(x=M(300, 200, BF), br=1, q=M(300, 200, C8), s=M(300, 2, F), qt=M(200, 300, C8), st=M(200, 3, F))
    a.update(change)
    got = api.lib().fp8_quantize(a["x"], a["br"], ref(a["q"]), ref(a["s"]), ref(a["qt"]), ref(a["st"]), None)
    assert got == want


@pytest.mark.parametrize("change,want", [
    (dict(x=M(30, 200, C8)), DTYPE), (dict(x=M(30, 200, BF, data=None)), NULL), (dict(res=M(30, 200, F)), DTYPE),
    (dict(res=M(30, 201, BF)), SHAPE), (dict(w=M(1, 199, F)), SHAPE), (dict(w=M(200, 1, F)), SHAPE),
    (dict(w=M(1, 200, C8)), DTYPE), (dict(eps=-1e-6), PARAM), (dict(eps=float("nan")), PARAM),
    (dict(eps=float("inf")), PARAM), (dict(total=M(29, 200, BF)), SHAPE), (dict(y=M(30, 200, F)), DTYPE),
    (dict(y=M(30, 200, BF, data=None)), NULL), (dict(q=M(30, 200, E8)), DTYPE), (dict(q=M(30, 100, C8)), SHAPE),
    (dict(s=M(30, 1, F)), SHAPE), (dict(s=M(1, 2, F)), SHAPE), (dict(s=M(30, 2, C8)), DTYPE),
    (dict(x=M(30, 32769, BF), w=M(1, 32769, F)), SHAPE),
    (dict(total=M(30, 200, BF, ld=208)), LAYOUT), (dict(y=M(30, 200, BF)), LAYOUT),
])
def test_norm_argument_errors(change, want):
    a = dict(x=M(30, 200, BF), res=M(30, 200, BF), w=M(1, 200, F), eps=1e-6, total=M(30, 200, BF),
             y=M(30, 200, BF, data=FAKE + (1 << 20)), q=M(30, 200, C8), s=M(30, 2, F))
    a.update(change)
    got = api.lib().rms_norm_fp8(a["x"], ref(a["res"]), a["w"], a["eps"], ref(a["total"]), ref(a["y"]),
                                 a["q"], a["s"], None)
    assert got == want
    if a["x"].dtype == F:   # a bf16 weight goes with bf16 data only
        assert api.lib().rms_norm_fp8(M(30, 200, F), None, M(1, 200, BF), 1e-6, None, None, a["q"], a["s"],
                                      None) == DTYPE


@pytest.mark.parametrize("change,want", [
    (dict(dy=M(30, 200, F)), DTYPE), (dict(dy=M(30, 100, BF)), SHAPE), (dict(dx=M(30, 200, F)), DTYPE),
    (dict(dx=M(30, 200, BF, data=None)), NULL), (dict(dw=M(1, 200, BF)), DTYPE), (dict(dw=M(200, 1, F)), SHAPE),
    (dict(ds=M(31, 200, BF)), SHAPE), (dict(eps=-1.0), PARAM), (dict(ws=None), WS), (dict(ws=FAKE + 16), WS),
    (dict(short=1), WS), (dict(x=M(30, 200, E8)), DTYPE), (dict(dx=M(30, 200, BF, ld=208)), LAYOUT),
])
def test_norm_gradient_argument_errors(change, want):
    a = dict(dy=M(30, 200, BF), x=M(30, 200, BF), w=M(1, 200, F), eps=1e-6, ds=M(30, 200, BF),
             dx=M(30, 200, BF), dw=M(1, 200, F), ws=FAKE, short=0)
    a.update(change)
    need = api.rms_norm_backward_workspace_size(30, 200)
    got = api.lib().rms_norm_backward(a["dy"], a["x"], a["w"], a["eps"], ref(a["ds"]), a["dx"], a["dw"],
                                      ctypes.c_void_p(a["ws"]), need - a["short"], None)
    assert got == want


def test_workspace_sizes():
    assert api.rms_norm_backward_workspace_size(0, 10) == 0
    assert api.rms_norm_backward_workspace_size(10, 32769) == 0
    assert api.rms_norm_backward_workspace_size(1, 1) % 256 == 0
    assert api.rms_norm_backward_workspace_size(8192, 4096) >= 4096 * 4
    assert api.fp8_matmul_workspace_size(0, 1, 1) == api.fp8_matmul_workspace_size(1, 1, -1) == 0
    assert api.fp8_matmul_workspace_size(1 << 30, 1 << 30, 1) == 0
    for m, n, k in ((1, 1, 1), (1, 8192, 2048), (2048, 2048, 8200), (16384, 4096, 4096)):
        b = api.fp8_matmul_workspace_size(m, n, k)
        assert b > 0 and b % 256 == 0


@pytest.mark.parametrize("change,want", [
    (dict(a=M(300, 500, BF)), DTYPE), (dict(a=M(300, 500, C8, data=None)), NULL),
    (dict(a=M(300, 499, C8)), SHAPE), (dict(b=M(200, 500, E8)), DTYPE), (dict(b=M(200, 500, C8, ld=499)), LAYOUT),
    (dict(sa=M(300, 3, F)), SHAPE), (dict(sa=M(2, 4, F)), SHAPE), (dict(sa=M(300, 4, E8)), DTYPE),
    (dict(sb=M(200, 4, E8)), DTYPE), (dict(sb=M(3, 4, F)), SHAPE), (dict(sb=M(2, 4, BF)), DTYPE),
    (dict(c=M(200, 300, BF)), SHAPE), (dict(c=M(300, 200, C8)), DTYPE), (dict(add=M(300, 199, F)), SHAPE),
    (dict(add=M(300, 200, C8)), DTYPE), (dict(add=M(300, 200, F)), LAYOUT), (dict(ws=None), WS),
    (dict(ws=FAKE + 128), WS), (dict(short=1), WS), (dict(a=M(0, 500, C8)), SHAPE),
])
def test_matmul_argument_errors(change, want):
    """(Add at C's address with another type is a layout error: the fake
    pointers coincide.)"""
    v = dict(a=M(300, 500, C8), sa=M(300, 4, F), b=M(200, 500, C8), sb=M(2, 4, F), c=M(300, 200, BF),
             add=None, ws=FAKE, short=0)
    v.update(change)
    need = api.fp8_matmul_workspace_size(300, 200, 500)
    got = api.lib().fp8_matmul(v["a"], v["sa"], v["b"], v["sb"], v["c"], ref(v["add"]),
                               ctypes.c_void_p(v["ws"]), need - v["short"], None)
    assert got == want


def test_the_steps_refuse_8_bit_matrices():
    ws = ctypes.c_void_p(FAKE)
    for dt in (C8, E8):
        assert api.lib().newton_schulz(M(64, 48, dt), M(64, 48, dt), 5, None, ws, 1 << 30, None) == DTYPE


def test_binding_refusals():
    """Tensors that are not on a GPU, and what the descriptors cannot express."""
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="GPU"):
        api.fp8_quantize(x)
    with pytest.raises(ValueError, match="GPU"):
        api.rms_norm_fp8(x, torch.zeros(1, 256))
    with pytest.raises(ValueError):
        api.mat(torch.zeros(4, 4, dtype=torch.float8_e4m3fn))


def test_code_rows_are_aligned():
    q = api.fp8_codes(5, 130, "cpu")
    assert q.shape == (5, 130) and q.stride() == (144, 1)
    assert api.fp8_scales(300, 130, "cpu").shape == (300, 2)
    assert api.fp8_scales(300, 130, "cpu", 128, torch.float8_e8m0fnu).shape == (3, 2)


def test_valid_calls_without_gpu_report_hip_error():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    L = api.lib()
    ws = ctypes.c_void_p(FAKE)
    assert L.fp8_quantize(M(4, 8, F), 1, ref(M(4, 8, C8)), ref(M(4, 1, F)), None, None, None) == 8
    assert L.rms_norm_fp8(M(4, 8, F), None, M(1, 8, F), 1e-6, None, None, M(4, 8, C8), M(4, 1, F), None) == 8
    assert L.rms_norm_backward(M(4, 8, F), M(4, 8, F), M(1, 8, F), 1e-6, None, M(4, 8, F), M(1, 8, F), ws,
                               api.rms_norm_backward_workspace_size(4, 8), None) == 8
    assert L.fp8_matmul(M(4, 8, C8), M(4, 1, F), M(6, 8, C8), M(6, 1, F), M(4, 6, F), None, ws,
                        api.fp8_matmul_workspace_size(4, 6, 8), None) == 8
