"""The 8-bit operators in 64 bits, from their definitions: plain torch on the
host, no code shared with the package."""

from __future__ import annotations

import torch

BLOCK = 128
TOP = 448.0


def cdiv(a, b):
    return -(-a // b)


def e4m3_table():
    """The 256 values of the e4m3 codes (OCP): bias 7, no infinities, 0x7f and
    0xff NaN."""
    out = []
    for c in range(256):
        sign, e, m = -1.0 if c & 128 else 1.0, c >> 3 & 15, c & 7
        if e == 15 and m == 7:
            out.append(float("nan"))
        elif e == 0:
            out.append(sign * m * 2.0 ** -9)
        else:
            out.append(sign * (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


def e4m3_values(codes):
    """float8_e4m3fn tensor -> fp64 values, through the table."""
    return e4m3_table()[codes.cpu().contiguous().view(torch.uint8).long()]


def e8m0_values(scales):
    b = scales.cpu().contiguous().view(torch.uint8).double()
    return torch.where(b == 255, torch.full_like(b, float("nan")), torch.exp2(b - 127))


def scale_values(s):
    return s.cpu().double() if s.dtype == torch.float32 else e8m0_values(s)


def half_step(v):
    """Half the distance between neighbouring e4m3 values around v."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def nearest_e4m3(v):
    """v to the nearest e4m3 value, ties to the even code; |v| <= 448."""
    step = 2 * half_step(v)
    return torch.round(v / step) * step


def expand(s, rows, cols, block_rows):
    return s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def block_tops(x, block_rows):
    """Largest finite magnitude of each block."""
    m, n = x.shape
    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    pad = torch.zeros(cdiv(m, block_rows) * block_rows, cdiv(n, BLOCK) * BLOCK, dtype=torch.float64)
    pad[:m, :n] = a
    return pad.view(cdiv(m, block_rows), block_rows, cdiv(n, BLOCK), BLOCK).amax(dim=(1, 3))


def e8m0_scale(top):
    s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / TOP)))
    # log2 next to a power of two may be off either way: settle by comparison
    s = torch.where(top <= TOP * s / 2, s / 2, s)
    s = torch.where(top > TOP * s, s * 2, s)
    return torch.where(top > 0, s.clamp(min=2.0 ** -126), torch.ones_like(s))


def f32_scale(top):
    return torch.where(top > 0, (top / TOP).clamp(min=2.0 ** -126), torch.ones_like(top))


def rms_norm(r, w, eps):
    r, w = r.double().cpu(), w.double().cpu()
    return r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * w


def rms_norm_backward(dy, x, w, eps, dsum=None):
    dy, x, w = dy.double().cpu(), x.double().cpu(), w.double().cpu()
    t = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    h, u = dy * w, x * t
    dx = t * (h - u * (h * u).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double().cpu()
    return dx, (dy * u).sum(0, keepdim=True)
