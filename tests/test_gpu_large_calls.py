"""AdamW and the tokens by expert in calls large enough to go past the caches, against the same work in
other layouts and in smaller calls, whose results are to be the same bits."""

import pytest
import torch

from orthonormal_optimizer_update_amd import api

pytestmark = pytest.mark.gpu
BF, F, C8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def step(x, g, states, seed, extra=None):
    """One step on copies; rows `extra` elements further apart where given.  The weights and states after it."""
    def place(t):
        if t is None or extra is None or t.dtype == C8 or t.size(1) != x.size(1):
            return None if t is None else t.clone()
        wide = torch.zeros(t.size(0), t.size(1) + extra, dtype=t.dtype, device="cuda")[:, :t.size(1)]
        return wide.copy_(t)
    X, G = [place(x)], [place(g)]
    M, V, SM, SV = ([place(s)] for s in states)
    if extra is not None and states[2] is not None:
        # (a tensor of another kind in the launch)
        X.append(torch.zeros(2, 9, device="cuda")[:, :8])
        G.append(torch.ones(2, 8, device="cuda"))
        M.append(torch.zeros(2, 8, device="cuda"))
        V.append(torch.zeros(2, 8, device="cuda"))
        SM.append(None)
        SV.append(None)
    codes = states[2] is not None
    api.adamw_step(X, G, M, V, 1e-2, 5, weight_decay=0.1, SM=SM if codes else None, SV=SV if codes else None, seed=seed)
    return [t.view(torch.uint8) if t.dtype == C8 else t for t in (X[0], M[0], V[0], SM[0], SV[0]) if t is not None]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("tx", [F, BF])
@pytest.mark.parametrize("tg", [F, BF])
@pytest.mark.parametrize("seed", [None, 17])
def test_adamw(bits, tx, tg, seed):
    rows, cols = 8200, 2049   # (more than 8192 units of 2048, and a part of one)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(rows, cols, generator=gen, device="cuda") * 0.02).to(tx)
    g = (torch.randn(rows, cols, generator=gen, device="cuda") * 1e-3).to(tg)
    g[5] = 0
    g[7, 3:90] = 0
    g[9, 100] = float("inf")
    states = [s[0] if s is not None else None for s in api.adamw_states([x], bits)]
    for _ in range(2):
        got = step(x, g, states, seed)
        for a, b in zip(got, step(x, g, states, seed, extra=8)):
            assert torch.equal(torch.nan_to_num(a, 7.0) if a.is_floating_point() else a,
                               torch.nan_to_num(b, 7.0) if b.is_floating_point() else b)
        x = got[0]
        states = [s.view(C8) if s.dtype == torch.uint8 else s for s in got[1:]] + [None] * (5 - len(got))


def parts(tokens):
    return [slice(i, min(i + 500, tokens)) for i in range(0, tokens, 500)]


@pytest.mark.parametrize("dtype,tokens,n", [(BF, 7500, 1124), (F, 3800, 1124), (BF, 4200, 2048), (F, 2100, 2049)])
def test_rows_by_expert(dtype, tokens, n):
    choices, experts = 8, 12
    gen = torch.Generator(device="cuda").manual_seed(4)
    chosen = torch.randint(-1, experts, (tokens, choices), generator=gen, device="cuda")
    slot, source, offsets, counts = api.expert_sort(chosen, experts, 128)
    rows = source.numel()
    x = torch.randn(tokens, n, generator=gen, device="cuda").to(dtype)
    w = torch.rand(tokens, choices, generator=gen, device="cuda")
    used = int(offsets[-1])

    y = torch.full((rows, n), 3.0, dtype=dtype, device="cuda")
    api.expert_gather(x, slot, offsets, counts, Y=y)
    want = torch.zeros(rows, n, dtype=dtype, device="cuda")
    own = source >= 0
    want[own] = x[(source[own] // choices).long()]
    want[used:] = 3
    assert torch.equal(y, want)

    y = torch.randn(rows, n, generator=gen, device="cuda").to(dtype)
    for add in (None, x):
        out = api.expert_combine(y, slot, w, add)
        for p in parts(tokens):
            assert torch.equal(out[p], api.expert_combine(y, slot[p].contiguous(), w[p], None if add is None else add[p]))
    inplace = x.clone()
    assert torch.equal(api.expert_combine(y, slot, w, inplace, inplace), out)

    dy, dw = api.expert_combine_backward(x, slot, w, offsets, counts, dY=torch.full_like(y, 3.0), Y=y)
    part = torch.full_like(y, 3.0)
    for p in parts(tokens):
        _, d = api.expert_combine_backward(x[p], slot[p].contiguous(), w[p], offsets, counts, dY=part, Y=y)
        assert torch.equal(dw[p], d)
    assert torch.equal(dy, part) and bool((dy[used:] == 3).all())
    kept = y[used:].clone()
    over, d = api.expert_combine_backward(x, slot, w, offsets, counts, dY=y, Y=y)
    assert torch.equal(over[:used], dy[:used]) and torch.equal(d, dw) and torch.equal(over[used:], kept)


@pytest.mark.parametrize("shift", [0, 5])
def test_codes_by_expert(shift):
    tokens, choices, experts, n = 8300, 8, 20, 2048
    gen = torch.Generator(device="cuda").manual_seed(5)
    chosen = torch.randint(-1, experts, (tokens, choices), generator=gen, device="cuda")
    slot, source, offsets, counts = api.expert_sort(chosen, experts, 64)
    x = torch.randint(0, 127, (tokens, n + shift), generator=gen, device="cuda", dtype=torch.uint8)[:, shift:]
    s = torch.rand(tokens, n // 128, generator=gen, device="cuda")
    y, sy = api.expert_gather(x.view(C8), slot, offsets, counts, S=s, rows=source.numel())
    own, used = source >= 0, int(offsets[-1])
    token = (source[own] // choices).long()
    assert torch.equal(y.view(torch.uint8)[own], x[token]) and torch.equal(sy[own], s[token])
    empty = ~own
    empty[used:] = False
    assert not bool(y.view(torch.uint8)[empty].any()) and bool((sy[empty] == 1).all())
