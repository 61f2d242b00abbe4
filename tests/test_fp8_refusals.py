"""Refusals of the 8-bit operators' argument checks that need no GPU."""

import ctypes

import pytest

from orthonormal_optimizer_update_amd import api
from test_fp8_cpu import BF, C8, DTYPE, E8, F, FAKE, M


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
