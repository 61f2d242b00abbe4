"""AdamW and the gradients' norm in 64 bits, from their definitions: plain torch and numpy on the
host, no code shared with the package.

Rounded results are checked from both sides: with e the bound of what 32-bit arithmetic may be off
by before the rounding R (to nearest, or with given random bits; R is monotone), a result r of the
exact value v holds if R(v - e) <= r <= R(v + e)."""

from __future__ import annotations

import numpy as np
import torch

from fp8_ref import TOP, cdiv, e4m3_values, expand, nearest_e4m3

U = 2.0 ** -24   # half a step of fp32, relative


def mix(h):
    h = h.astype(np.uint32)
    h = (h ^ (h >> np.uint32(16))) * np.uint32(0x7FEB352D)
    h = (h ^ (h >> np.uint32(15))) * np.uint32(0x846CA68B)
    return h ^ (h >> np.uint32(16))


def random_bits(seed, step, tensor, rows, cols, first_row=0):
    """(weight's 16 bits, m's 20, sqrt(v)'s 20) of a tensor's elements in `rows` rows."""
    with np.errstate(over="ignore"):
        gold = np.uint32(0x9E3779B9)
        key = mix(np.array([seed & 0xFFFFFFFF], dtype=np.uint32))
        for word in (seed >> 32, step & 0xFFFFFFFF, step >> 32, tensor):
            key = mix(key ^ mix(np.array([word], dtype=np.uint32) + gold))
        e = np.arange(rows * cols, dtype=np.uint64) + np.uint64(first_row * cols)
        low, high = (e & np.uint64(0xFFFFFFFF)).astype(np.uint32), (e >> np.uint64(32)).astype(np.uint32)
        a = mix(low ^ (key + gold * high))
        b = mix(a + gold)
    out = ((a & 4095) << 4 | (b & 15), a >> 12, b >> 12)
    return tuple(torch.from_numpy(v.astype(np.int64)).view(rows, cols) for v in out)


def round_bf16(v, bits=None):
    """v (64 bits) to bf16 values: nearest even, or by bits out of 2^16, away from zero if they and
    the part that is cut make a whole step."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 8).clamp(min=-133).double())
    if bits is None:
        return torch.round(v / step) * step
    return torch.sign(v) * torch.floor(v.abs() / step + bits.double() / 2 ** 16) * step


def round_e4m3(v, bits=None):
    """|v| <= 448."""
    v = v.clamp(-TOP, TOP)
    if bits is None:
        return nearest_e4m3(v)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * torch.floor(v.abs() / step + bits.double() / 2 ** 20) * step


def state_values(codes, scales):
    rows, cols = codes.shape
    return e4m3_values(codes) * expand(scales.cpu().double(), rows, cols, 1)


def step(x, g, m, v, lr, t, betas, eps, decay, factor=1.0):
    """(value, bound of 32-bit arithmetic's error) of x' before its rounding, m', v'; all fp64.
    The bounds count a rounding (U) for each constant and operation of the formula."""
    b1, b2 = betas
    g = g * factor
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    # g: 1; each product: constant and product; the sum
    em = U * (3 * (b1 * m).abs() + 4 * ((1 - b1) * g).abs()) + 2.0 ** -148
    # g twice, its square, constant, product; the sum.  (what is below 2^-126 loses up to 2^-149 a step)
    ev = U * (3 * b2 * v + 6 * (1 - b2) * g * g) + 2.0 ** -148
    size, root = lr / (1 - b1 ** t), 1 / (1 - b2 ** t) ** 0.5
    low = (v2 - ev).clamp(min=0).sqrt() * root + eps       # smallest divisor
    down = v2.sqrt() * root + eps
    # sqrt 1, root 2, eps 1, sum 1, reciprocal 2 (one unit in the last place), product 1, size 2: ten
    # roundings of the update (a quotient in place of reciprocal and product would be eight)
    update = size * m2 / down
    eu = size * ((m2.abs() + em) / low - m2.abs() / down) + 10 * U * size * (m2.abs() + em) / low
    keep = 1 - lr * decay
    ex = 3 * U * (keep * x).abs() + eu + U * update.abs()
    return (keep * x - update, ex * 1.01), (m2, em * 1.01), (v2, ev * 1.01)


def tops(x):
    """Largest finite magnitude of each 1 x 128 block."""
    rows, cols = x.shape
    pad = torch.zeros(rows, cdiv(cols, 128) * 128, dtype=torch.float64)
    pad[:, :cols] = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    return pad.view(rows, -1, 128).amax(2)


def between(got, low, high):
    """Whether low <= got <= high wherever low and high are numbers, and NaN or the same infinity elsewhere."""
    number = torch.isfinite(low) & torch.isfinite(high)
    ok = torch.where(number, (got >= low) & (got <= high), (got == low) | (torch.isnan(low) & torch.isnan(got)))
    return bool(ok.all())


def check_codes(codes, scales, value, err, bits, least):
    """The codes and scales of `value` (rows x cols, off by err at most before they are taken)."""
    rows, cols = value.shape
    s = scales.cpu().double()
    top, low, high = tops(value), tops((value.abs() - err).clamp(min=0)), tops(value.abs() + err)
    some = top > 0
    # a value that the error reaches zero from may be zero in 32 bits (a square below 2^-149 is, and the
    # bound of v' counts it), and where this holds for all of a block, its scale may be 1 as well
    some &= ~((low == 0) & (s == 1))
    assert bool((s[some] >= (low / TOP * (1 - 2 * U)).clamp(min=2.0 ** -126)[some]).all())
    assert bool((s[some] <= (high / TOP * (1 + 2 * U)).clamp(min=2.0 ** -126)[some]).all())
    assert bool((s[top == 0] == 1).all())
    got = e4m3_values(codes)
    finite = torch.isfinite(value)
    assert bool(torch.isnan(got[~finite]).all())
    each = expand(s, rows, cols, 1)
    q = value / each
    eq = err / each + 3 * U * q.abs()   # 1 / s, the product, and the 2^-6 that is added below 2^-6
    eq = eq + 2.0 ** -30
    lo, hi = round_e4m3(q - eq, bits), round_e4m3(q + eq, bits)
    if least:
        lo = torch.where(value - err > 0, lo.clamp(min=2.0 ** -9), lo.clamp(min=0))
        hi = torch.where(value + err > 0, hi.clamp(min=2.0 ** -9), hi)
    assert between(got[finite], lo[finite], hi[finite])


def norm(gs):
    total = sum(float((g.cpu().double() ** 2).sum()) for g in gs)
    return total ** 0.5
