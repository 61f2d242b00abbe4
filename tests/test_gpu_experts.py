"""Tokens sorted by expert and back on the GPU, against their definitions."""

import pytest
import torch

import experts_ref as R
from orthonormal_optimizer_update_amd import api

pytestmark = pytest.mark.gpu
BF, F, C8, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


def choose(gen, tokens, choices, experts, wide=False, dropped=0.2):
    """Experts of uneven popularity, some pairs without one, some with one that does not exist."""
    e = (torch.rand(tokens, choices, generator=gen) ** 2 * experts).long().clamp(max=experts - 1)
    out = torch.rand(tokens, choices, generator=gen)
    e = torch.where(out < dropped / 2, torch.full_like(e, -1), e)
    e = torch.where((out > 1 - dropped / 4), torch.full_like(e, experts), e)
    e = torch.where((out > 1 - dropped / 8), torch.full_like(e, (1 << 33) if wide else 2 ** 31 - 1), e)
    return e if wide else e.int()


SORTS = [(1, 1, 1, 1), (1, 3, 2, 1), (5, 2, 7, 4), (33, 8, 64, 1), (100, 64, 3, 128), (64, 1, 1024, 16), (511, 8, 64, 128),
         (512, 8, 64, 1), (513, 8, 100, 3), (4096, 1, 1, 1), (4097, 1, 5, 4096), (3000, 6, 257, 128), (9000, 2, 1000, 1)]


@pytest.mark.parametrize("case", SORTS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dropped", [0.0, 0.3, 2.0])
def test_sort(case, wide, dropped):
    tokens, choices, experts, align = case
    chosen = choose(torch.Generator().manual_seed(tokens), tokens, choices, experts, wide, dropped)
    if dropped == 2.0:
        chosen.fill_(-1)
    want = R.sort(chosen.tolist(), experts, align)
    ws = api.workspace(api.expert_sort_workspace_size(tokens, choices, experts), "cuda").fill_(255)
    got = api.expert_sort(chosen.cuda(), experts, align, ws=ws)
    for a, b in zip(got, want):
        assert a.cpu().tolist() == b


def test_sort_of_many():
    """More pairs than 1024 tiles of 4096, against torch's stable sort."""
    tokens, choices, experts, align = 700_001, 7, 300, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    chosen = torch.randint(-5, experts + 3, (tokens, choices), generator=gen, device="cuda")
    slot, source, offsets, counts = api.expert_sort(chosen, experts, align)
    ids = chosen.flatten()
    ok = (ids >= 0) & (ids < experts)
    order = torch.sort(torch.where(ok, ids, experts), stable=True)[1][:int(ok.sum())]
    count = torch.stack([(ids == e).sum() for e in range(experts)])
    assert torch.equal(counts.long(), count)
    begin = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum((count + align - 1) // align * align, 0)])
    assert torch.equal(offsets.long(), begin)
    place = torch.arange(order.numel(), device="cuda") - (torch.cumsum(count, 0) - count)[ids[order]] + begin[ids[order]]
    want = torch.full_like(ids, -1)
    want[order] = place
    assert torch.equal(slot.flatten().long(), want)
    rows = torch.full((source.numel(),), -1, dtype=torch.long, device="cuda")
    rows[place] = order
    assert torch.equal(source.long(), rows)


def test_sort_without_sources():
    chosen = choose(torch.Generator().manual_seed(3), 50, 4, 9).cuda()
    want = api.expert_sort(chosen, 9, 8)
    slot, offsets, counts = (torch.empty_like(want[i]) for i in (0, 2, 3))
    ws = api.workspace(256, "cuda")
    status = api.lib().expert_sort(chosen.data_ptr(), 4, 50, 4, 9, 8, slot.data_ptr(), None, offsets.data_ptr(), counts.data_ptr(),
                                   ws.data_ptr(), 256, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    for a, b in zip((slot, offsets, counts), (want[0], want[2], want[3])):
        assert torch.equal(a, b)


def strided(t, pad, shift=0):
    """t's values with rows `pad` elements further apart, `shift` elements into its memory."""
    rows, cols = t.shape
    raw = t.view(torch.uint8) if t.element_size() == 1 else t
    memory = torch.zeros(shift + rows * (cols + pad), dtype=raw.dtype, device="cuda")
    out = memory[shift:].view(rows, cols + pad)[:, :cols]
    out.copy_(raw)
    return out.view(t.dtype)


def bytes_of(t):
    return t.contiguous().view(torch.uint8)


def plan(tokens, choices, experts, align, dropped=0.2, seed=0):
    chosen = choose(torch.Generator().manual_seed(seed + tokens), tokens, choices, experts, dropped=dropped).cuda()
    return api.expert_sort(chosen, experts, align)


SHAPES = [(1, 1, 1, 1, 1), (3, 2, 2, 1, 7), (9, 3, 4, 8, 8), (37, 2, 5, 16, 129), (130, 4, 33, 1, 2001), (64, 8, 64, 128, 256),
          (50, 16, 20, 4, 1024), (7, 9, 3, 2, 5000), (33, 64, 100, 1, 136)]


@pytest.mark.parametrize("case", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3 f32", "e4m3 e8m0"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_gather(case, kind, pad, shift):
    tokens, choices, experts, align, n = case
    slot, source, offsets, counts = plan(*case[:4])
    rows, gen = source.numel() + 2, torch.Generator().manual_seed(5)
    s = sy = None
    raw = torch.randint(0, 256, (tokens, n * 4), generator=gen, dtype=torch.uint8)   # every bit pattern, NaN among them
    x = {"bf16": raw.view(BF)[:, :n], "f32": raw.view(F)}.get(kind, raw.view(C8)[:, :n]).contiguous().cuda()
    y = strided(torch.full((rows, n * x.element_size()), 77, dtype=torch.uint8, device="cuda").view(x.dtype), pad, shift)
    if kind.startswith("e4m3"):
        blocks, st = -(-n // 128), F if kind.endswith("f32") else E8
        s = torch.randint(1, 255, (tokens, blocks), generator=gen, dtype=torch.uint8)
        s = (s.float() if st == F else s.view(E8)).cuda()
        s = strided(s, pad, shift)
        sy = strided(torch.full((rows, blocks * s.element_size()), 77, dtype=torch.uint8, device="cuda").view(st), pad, shift)
    before, before_s = bytes_of(y).clone(), None if sy is None else bytes_of(sy).clone()
    api.expert_gather(strided(x, pad, shift), slot, offsets, counts, y, S=s, SY=sy)
    end, src = int(offsets[-1]), source[:rows - 2]
    for got, want, was, pad_value in ((y, x, before, 0), (sy, s, before_s, 1)):
        if got is None:
            continue
        out = bytes_of(want)[src.clamp(min=0).long() // choices]
        blank = bytes_of(torch.full((1, want.size(1)), float(pad_value), device="cuda").to(want.dtype))
        out = torch.where((src < 0)[:, None], blank, out)
        assert torch.equal(bytes_of(got)[:end], out[:end])
        assert torch.equal(bytes_of(got)[end:], was[end:])   # rows behind the last expert's


@pytest.mark.parametrize("case", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("weights,add", [(None, None), (F, None), (BF, BF), (F, F)])
def test_combine(case, dtype, weights, add):
    tokens, choices, experts, align, n = case
    slot, source, _, _ = plan(*case[:4], dropped=0.5)
    gen, rows = torch.Generator().manual_seed(6), source.numel()
    y = torch.randn(rows, n, generator=gen).to(dtype).cuda()
    y[source < 0] = float("nan")      # no one's rows
    for pad, shift in ((0, 0), (5, 1)):
        w = None if weights is None else strided(torch.rand(tokens, choices, generator=gen).to(weights).cuda(), pad, shift)
        ad = None if add is None else strided(torch.randn(tokens, n, generator=gen).to(add).cuda(), pad, shift)
        if w is not None:
            w[slot < 0] = float("nan")
        out = strided(torch.full((tokens, n), 9.0, dtype=dtype, device="cuda"), pad, shift)
        api.expert_combine(strided(y, pad, shift), slot, w, ad, out)
        want, err = R.combine(y.cpu().double(), slot.cpu(), None if w is None else w.cpu().double(), None if ad is None else ad.cpu().double())
        assert bool(((out.cpu().double() - want).abs() <= err + R.HALF[dtype] * (want.abs() + err)).all())
        if ad is not None and ad.dtype == dtype:   # in place
            api.expert_combine(y, slot, w, ad, ad)
            assert torch.equal(ad, out)


@pytest.mark.parametrize("case", SHAPES)
@pytest.mark.parametrize("dtype,weights", [(BF, F), (F, F), (BF, BF), (F, None)])
def test_combine_backward(case, dtype, weights):
    tokens, choices, experts, align, n = case
    slot, source, offsets, counts = plan(*case[:4], dropped=0.5)
    gen, rows, end = torch.Generator().manual_seed(7), source.numel(), int(offsets[-1])
    y = torch.randn(rows, n, generator=gen).to(dtype).cuda()
    y[source < 0] = float("nan")
    d = torch.randn(tokens, n, generator=gen).to(dtype).cuda()
    for pad, shift in ((0, 0), (5, 1)):
        w = None if weights is None else strided(torch.rand(tokens, choices, generator=gen).to(weights).cuda(), pad, shift)
        dy = strided(torch.full((rows, n), 7.0, dtype=dtype, device="cuda"), pad, shift)
        dw = strided(torch.full((tokens, choices), 7.0, device="cuda"), pad, shift)
        api.expert_combine_backward(strided(d, pad, shift), slot, w, offsets, counts, dy, Y=strided(y, pad, shift), dW=dw)
        want, want_w, err = R.combine_backward(d.cpu().double(), y.cpu().double(), slot.cpu(), None if w is None else w.cpu().double(), rows)
        got, used = dy.cpu().double(), (source >= 0).cpu()
        # one rounding in 32 bits, one to the type
        assert bool(((got - want).abs() <= (R.U + R.HALF[dtype]) * want.abs() * 1.01 + 1e-38)[used].all())
        assert bool((got[:end][~used[:end]] == 0).all()) and bool((got[end:] == 7).all())
        assert bool(((dw.cpu().double() - want_w).abs() <= err).all())
        assert bool((dw.cpu()[slot.cpu() < 0] == 0).all())
        only, none = api.expert_combine_backward(d, slot, w, offsets, counts, rows=rows)
        assert none is None and torch.equal(only[:end], dy[:end])
        same = y.clone()      # the gradient in Y's place
        _, again = api.expert_combine_backward(d, slot, w, offsets, counts, same, Y=same)
        assert torch.equal(same[:end], dy[:end]) and torch.equal(again, dw)


def test_gradients_against_differences():
    """A loss's change over small changes of y, of the weights and of the gathered x."""
    tokens, choices, experts, align, n = 13, 3, 4, 4, 40
    slot, source, offsets, counts = plan(tokens, choices, experts, align, 0.3)
    gen, rows, end = torch.Generator().manual_seed(8), source.numel(), int(offsets[-1])
    x, r = torch.randn(tokens, n, generator=gen).cuda(), torch.randn(tokens, n, generator=gen).cuda()
    w = torch.rand(tokens, choices, generator=gen).cuda()
    y, _ = api.expert_gather(x, slot, offsets, counts, torch.zeros(rows, n, device="cuda"))

    def loss(x, w):      # rows squared on the way; in 64 bits on the host behind the operators
        z, _ = api.expert_gather(x, slot, offsets, counts, torch.zeros(rows, n, device="cuda"))
        return float((api.expert_combine(z * z, slot, w).double() * r.double()).sum())

    dz, dw = api.expert_combine_backward(r, slot, w, offsets, counts, Y=y * y, dY=torch.zeros(rows, n, device="cuda"))
    dx = api.expert_combine(dz * 2 * y, slot, out=torch.empty_like(x))
    h = 2.0 ** -7
    for tensor, grad in ((x, dx), (w, dw)):
        for k in range(20):
            i, j = k * 7 % tensor.size(0), k * 11 % tensor.size(1)
            keep = tensor[i, j].item()
            tensor[i, j] = keep + h
            up = loss(x, w)
            tensor[i, j] = keep - h
            down = loss(x, w)
            tensor[i, j] = keep
            # the loss is a polynomial of degree 2 in x and 1 in w: the difference is exact but for the
            # sums' roundings, of at most choices + 2 of 2^-24 of the terms of one row or of one element
            size = float((r[i].abs().double() * (y[slot[i].clamp(min=0).long()].double() ** 2).sum(0)).sum()) + 1
            assert abs((up - down) / (2 * h) - grad[i, j].item()) < 10 * R.U * size / h + 1e-5


def test_slots_out_of_range_are_no_rows():
    """A caller's slots beyond the matrix are left out, not followed."""
    y, n = torch.randn(6, 64, device="cuda"), 64
    slot = torch.tensor([[0, 6], [5, -7], [2 ** 31 - 1, 1], [-2 ** 31, 1 << 20]], dtype=torch.int32, device="cuda")
    w = torch.full((4, 2), 2.0, device="cuda")
    out = api.expert_combine(y, slot, w)
    want = torch.stack([2 * y[0], 2 * y[5], 2 * y[1], 0 * y[0]])
    assert torch.equal(out, want)
    offsets = torch.tensor([0, 1 << 20, 2 ** 31 - 1], dtype=torch.int32, device="cuda")   # padding far beyond
    counts = torch.tensor([6, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    x = torch.randn(4, n, device="cuda")
    z, _ = api.expert_gather(x, slot, offsets, counts, torch.full((6, n), 3.0, device="cuda"))
    assert torch.equal(z, torch.stack([x[0], x[2], 3 + 0 * x[0], 3 + 0 * x[0], 3 + 0 * x[0], x[1]]))
    dy, dw = api.expert_combine_backward(x, slot, w, offsets, counts, torch.full((6, n), 3.0, device="cuda"), Y=y)
    assert torch.equal(dy[[0, 5, 1]], 2 * x[:3]) and bool((dy[2:5] == 3).all()) and bool((dw[3] == 0).all())


def test_one_expert_takes_all_and_the_same_twice():
    tokens, n = 300, 96
    chosen = torch.full((tokens, 2), 4, dtype=torch.int32, device="cuda")
    slot, source, offsets, counts = api.expert_sort(chosen, 9, 128)
    assert counts.tolist() == [0, 0, 0, 0, 600, 0, 0, 0, 0] and offsets.tolist() == [0] * 5 + [640] * 5
    x = torch.randn(tokens, n, dtype=BF, device="cuda")
    y, _ = api.expert_gather(x, slot, offsets, counts, rows=source.numel())
    assert torch.equal(y[:600:2], x) and torch.equal(y[1:600:2], x) and not bool(y[600:640].any())
    out = api.expert_combine(y, slot, torch.full((tokens, 2), 0.5, device="cuda"))
    assert torch.equal(out, x)


@pytest.mark.parametrize("n", [40, 300, 2001])
def test_tokens_that_all_stay_out(n):
    chosen = torch.full((33, 3), -1, dtype=torch.int64, device="cuda")
    slot, source, offsets, counts = api.expert_sort(chosen, 6, 16)
    assert not bool(counts.any()) and not bool(offsets.any()) and bool((source == -1).all()) and bool((slot == -1).all())
    x, rows = torch.randn(33, n, dtype=BF, device="cuda"), source.numel()
    y, _ = api.expert_gather(x, slot, offsets, counts, torch.full((rows, n), 5.0, dtype=BF, device="cuda"))
    assert bool((y == 5).all())
    y.fill_(float("nan"))
    w = torch.full((33, 3), float("inf"), device="cuda")
    assert not bool(api.expert_combine(y, slot, w).any()) and torch.equal(api.expert_combine(y, slot, w, x), x)
    dy, dw = api.expert_combine_backward(x, slot, w, offsets, counts, torch.full_like(y, 5.0), Y=y)
    assert bool((dy == 5).all()) and not bool(dw.any())


def test_two_graphs_that_share_a_workspace():
    cases = [(3000, 4, 60, 16), (900, 8, 7, 1)]
    ws = api.workspace(max(api.expert_sort_workspace_size(t, k, e) for t, k, e, _ in cases), "cuda")
    gen, graphs, held = torch.Generator(device="cuda").manual_seed(2), [], []
    for t, k, e, align in cases:
        chosen = torch.randint(0, e, (t, k), generator=gen, device="cuda")
        ints = api.expert_sort(chosen, e, align, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.expert_sort(chosen, e, align, *ints, ws=ws)
        graphs.append(graph)
        held.append((chosen, ints, e, align))
    for i in range(4):
        for chosen, _, e, _ in held:
            chosen.copy_(torch.randint(-1, e, chosen.shape, generator=gen, device="cuda"))
        for graph in (graphs if i % 2 else graphs[::-1]):
            graph.replay()
        torch.cuda.synchronize()
        for chosen, ints, e, align in held:
            for a, b in zip(ints, api.expert_sort(chosen, e, align)):
                assert torch.equal(a, b)


def test_rows_beyond_32_bits():
    """Rows of the sorted matrix more than 2^32 bytes in."""
    n, rows = 1 << 16, (1 << 15) + (1 << 10)
    y = torch.zeros(rows, n, dtype=BF, device="cuda")
    slot = torch.tensor([[rows - 1, 0], [rows - 2, 3]], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    counts = torch.tensor([rows], dtype=torch.int32, device="cuda")
    x = torch.randn(2, n, dtype=BF, device="cuda")
    api.expert_gather(x, slot, offsets, counts, y)
    assert torch.equal(y[[rows - 1, 0, rows - 2, 3]], x[[0, 0, 1, 1]]) and int((y != 0).any(1).sum()) == 4
    assert torch.equal(api.expert_combine(y, slot, torch.full((2, 2), 0.5, device="cuda")), x)
    dy, dw = api.expert_combine_backward(x, slot, None, offsets, counts, y, Y=y)
    assert torch.equal(y[[rows - 1, 0, rows - 2, 3]], x[[0, 0, 1, 1]])


def test_captured_and_replayed():
    """The whole way in a graph, replayed with other tokens and experts each time."""
    tokens, choices, experts, align, n = 700, 4, 30, 16, 200
    gen = torch.Generator().manual_seed(9)
    chosen = choose(gen, tokens, choices, experts).cuda()
    x, w = torch.randn(tokens, n, dtype=BF, device="cuda"), torch.rand(tokens, choices, device="cuda")
    rows = api.expert_rows(tokens, choices, experts, align)
    y, out = torch.zeros(rows, n, dtype=BF, device="cuda"), torch.empty_like(x)
    ws = api.workspace(api.expert_sort_workspace_size(tokens, choices, experts), "cuda")
    ints = api.expert_sort(chosen, experts, align, ws=ws)

    def call():
        slot, source, offsets, counts = api.expert_sort(chosen, experts, align, *ints, ws=ws)
        api.expert_gather(x, slot, offsets, counts, y)
        api.expert_combine(y, slot, w, x, out)
        return api.expert_combine_backward(out, slot, w, offsets, counts, Y=y)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dy, dw = call()
    for i in range(4):
        chosen.copy_(choose(gen, tokens, choices, experts, dropped=0.1 * i))
        x.copy_(torch.randn(tokens, n, generator=gen))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*ints, out, dw)] + [dy[:int(ints[2][-1])].clone()]
        dy2, dw2 = call()
        torch.cuda.synchronize()
        for a, b in zip(got, [*ints, out, dw2, dy2[:int(ints[2][-1])]]):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    cases = [(900, 8, 64, 128, 512), (1500, 2, 7, 1, 333)]

    def run(case, seed):
        tokens, choices, experts, align, n = case
        gen = torch.Generator(device="cuda").manual_seed(seed)
        chosen = torch.randint(0, experts, (tokens, choices), generator=gen, device="cuda")
        x = torch.randn(tokens, n, generator=gen, device="cuda")
        slot, source, offsets, counts = api.expert_sort(chosen, experts, align)
        y, _ = api.expert_gather(x, slot, offsets, counts, torch.zeros(source.numel(), n, device="cuda"))
        out = api.expert_combine(y, slot)
        dy, dw = api.expert_combine_backward(out, slot, None, offsets, counts, torch.zeros_like(y), Y=y)
        return slot, source, y, out, dy, dw

    want = [run(c, 1) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], []
    for s, c in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append(run(c, 1))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for p, q in zip(a, b):
            assert torch.equal(p, q)
