"""Tokens by expert from their definitions: loops and plain torch in 64 bits on the host, no code
shared with the package."""

from __future__ import annotations

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}   # half a step, relative


def sort(chosen, experts, align):
    """(slot, source, offsets, counts) as lists of whole numbers."""
    tokens, choices = len(chosen), len(chosen[0])
    rows = tokens * choices + experts * (align - 1)
    lists = [[] for _ in range(experts)]
    for t in range(tokens):
        for j in range(choices):
            e = chosen[t][j]
            if 0 <= e < experts:
                lists[e].append(t * choices + j)
    slot, source, offsets, at = [[-1] * choices for _ in range(tokens)], [-1] * rows, [], 0
    for pairs in lists:
        offsets.append(at)
        for i, pair in enumerate(pairs):
            slot[pair // choices][pair % choices] = at + i
            source[at + i] = pair
        at += -(-len(pairs) // align) * align
    return slot, source, offsets + [at], [len(pairs) for pairs in lists]


def combine(y, slot, w, add):
    """(out, the bound of 32-bit sums' error), 64 bits."""
    tokens, choices = slot.shape
    out = torch.zeros(tokens, y.size(1), dtype=torch.float64)
    size = torch.zeros_like(out)
    for t in range(tokens):
        for j in range(choices):
            if 0 <= slot[t, j] < y.size(0):
                term = (1.0 if w is None else w[t, j]) * y[slot[t, j]]
                out[t] += term
                size[t] += term.abs()
        if add is not None:
            out[t] += add[t]
            size[t] += add[t].abs()
    return out, (choices + 2) * U * size


def combine_backward(dout, y, slot, w, rows):
    """(dy with NaN in rows that no pair has, dw, the bound of dw's error), 64 bits."""
    tokens, choices = slot.shape
    dy = torch.full((rows, dout.size(1)), float("nan"), dtype=torch.float64)
    dw, size = torch.zeros(tokens, choices, dtype=torch.float64), torch.zeros(tokens, choices, dtype=torch.float64)
    for t in range(tokens):
        for j in range(choices):
            if 0 <= slot[t, j] < rows:
                dy[slot[t, j]] = (1.0 if w is None else w[t, j]) * dout[t]
                if y is not None:
                    dw[t, j] = (dout[t] * y[slot[t, j]]).sum()
                    size[t, j] = (dout[t] * y[slot[t, j]]).abs().sum()
    # a thread of 64 or more adds n / 64 products at most (rounded up to 8), then ten sums
    return dy, dw, (dout.size(1) / 64 + 8 + 10) * U * size
