"""AdamW over many tensors and the gradients' norm on the GPU, against their definitions in 64 bits."""

import math

import pytest
import torch

import adamw_ref as R
from orthonormal_optimizer_update_amd import api

pytestmark = pytest.mark.gpu
BF, F, C8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
H = dict(lr=1e-2, betas=(0.9, 0.97), eps=1e-8, weight_decay=0.05)


def values(gen, rows, cols, std):
    """Normal values of another size from row to row, every seventh column 0."""
    x = torch.randn(rows, cols, generator=gen, dtype=torch.float64) * std
    x = x * torch.exp(torch.randn(rows, 1, generator=gen, dtype=torch.float64))
    x[:, ::7] = 0
    return x


def placed(x, dtype, ld=None, shift=0):
    """x on the GPU as a matrix with rows `ld` apart, `shift` elements into its memory; the gaps hold 3."""
    rows, cols = x.shape
    ld = cols if ld is None else ld
    raw = x.to(F).to(dtype)
    memory = torch.full((shift + rows * ld,), 3.0, dtype=F, device="cuda").to(dtype)
    out = memory[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    if dtype == C8:
        out.view(torch.uint8).copy_(raw.view(torch.uint8).cuda())
    else:
        out.copy_(raw)
    return memory, out


class Tensor:
    """A tensor with gradient and states, and what a step makes of it in 64 bits."""

    def __init__(self, gen, rows, cols, tx=BF, tg=BF, bits=32, pad=0, shift=0):
        self.shape, self.tx, self.bits = (rows, cols), tx, bits
        ld = cols + pad
        self.gaps = []

        def keep(x, dtype, ld=ld):
            memory, t = placed(x, dtype, ld, shift)
            self.gaps.append((memory, t, memory.clone()))
            return t

        self.x = keep(values(gen, rows, cols, 0.02), tx)
        self.g = keep(values(gen, rows, cols, 1e-3), tg)
        m, v = values(gen, rows, cols, 3e-4), values(gen, rows, cols, 1e-3).abs()
        self.sm = self.sv = None
        if bits == 8:
            blocks = R.cdiv(cols, 128)
            sm, sv = R.tops(m) / R.TOP, R.tops(v) / R.TOP
            sm, sv = torch.where(sm > 0, sm, 1.0).float().double(), torch.where(sv > 0, sv, 1.0).float().double()
            self.m = keep(R.round_e4m3(m / R.expand(sm, rows, cols, 1)), C8)
            self.v = keep(R.round_e4m3(v / R.expand(sv, rows, cols, 1)), C8)
            self.sm, self.sv = keep(sm, F, blocks + pad), keep(sv, F, blocks + pad)
        else:
            self.m, self.v = keep(m, F), keep(v * v, F)

    def start(self):
        x, g = self.x.cpu().double(), self.g.cpu().double()
        if self.bits == 8:
            return x, g, R.state_values(self.m, self.sm), R.state_values(self.v, self.sv) ** 2
        return x, g, self.m.cpu().double(), self.v.cpu().double()

    def gaps_untouched(self):
        for memory, t, before in self.gaps:
            a, b = memory.clone(), before.clone()
            for z in (a, b):
                part = torch.as_strided(z.view(torch.uint8) if z.dtype == C8 else z, t.shape, t.stride(), t.storage_offset())
                part.zero_()
            if not torch.equal(a.view(torch.uint8), b.view(torch.uint8)):
                return False
        return True


def step_and_check(tensors, t=7, seed=None, factor=None, lr=None, tstep=None):
    start = [x.start() for x in tensors]
    any8 = any(x.bits == 8 for x in tensors)
    f = 1.0 if factor is None else float(factor)
    api.adamw_step([x.x for x in tensors], [x.g for x in tensors], [x.m for x in tensors], [x.v for x in tensors],
                   H["lr"] if lr is None else lr, t if tstep is None else tstep, betas=H["betas"], eps=H["eps"],
                   weight_decay=H["weight_decay"], SM=[x.sm for x in tensors] if any8 else None,
                   SV=[x.sv for x in tensors] if any8 else None, seed=seed, factor=factor)
    for i, (x, was) in enumerate(zip(tensors, start)):
        lr_used = H["lr"] if lr is None else float(lr)
        (xn, ex), (mn, em), (vn, ev) = R.step(*was, lr_used, t, H["betas"], H["eps"], H["weight_decay"], f)
        bits = R.random_bits(seed, t, i, *x.shape) if seed is not None else (None, None, None)
        got = x.x.cpu().double()
        if x.tx == BF:
            assert R.between(got, R.round_bf16(xn - ex, bits[0]), R.round_bf16(xn + ex, bits[0])), (i, x.shape)
        else:
            assert R.between(got, xn - ex, xn + ex), (i, x.shape)
        if x.bits == 8:
            root, er = vn.sqrt(), (vn + ev).sqrt() - (vn - ev).clamp(min=0).sqrt()
            R.check_codes(x.m, x.sm, mn, em, bits[1], False)
            R.check_codes(x.v, x.sv, root, er + R.U * root, bits[2], True)
        else:
            assert R.between(x.m.cpu().double(), mn - em, mn + em), (i, x.shape)
            assert R.between(x.v.cpu().double(), vn - ev, vn + ev), (i, x.shape)
        assert x.gaps_untouched()
    return tensors


SHAPES = [(1, 1), (1, 7), (1, 8), (3, 127), (2, 129), (1, 2048), (1, 2049), (17, 100), (5, 1537), (300, 9), (64, 512),
          (129, 2056), (1, 4097)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("tx,tg", [(BF, BF), (BF, F), (F, F), (F, BF)])
@pytest.mark.parametrize("seed", [None, 0x123456789ABCDEF])
def test_shapes(bits, tx, tg, seed):
    gen = torch.Generator().manual_seed(1)
    step_and_check([Tensor(gen, *s, tx, tg, bits) for s in SHAPES], seed=seed)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 0), (5, 1), (0, 3)])
def test_rows_of_any_pitch_at_any_element(bits, pad, shift):
    gen = torch.Generator().manual_seed(2)
    ts = [Tensor(gen, *s, tx, tg, bits, pad, shift) for s in SHAPES for tx, tg in ((BF, F), (F, BF))]
    step_and_check(ts, seed=5 if pad else None)


def test_many_tensors_of_all_kinds_in_one_call():
    """More than a launch's table holds of either, in a mixed order."""
    gen = torch.Generator().manual_seed(3)
    kinds = [(BF, BF, 32, 0), (F, BF, 8, 0), (BF, F, 8, 3), (F, F, 32, 2)]
    ts = [Tensor(gen, 1 + i % 5, 1 + 37 * i % 300, *kinds[i % 4]) for i in range(210)]
    step_and_check(ts, seed=11)


def test_many_units():
    """More units than workgroups are resident, in a table with small tensors around."""
    gen = torch.Generator().manual_seed(4)
    shapes = [(1, 5), (2100, 2048), (3, 3), (700, 6145), (1, 1)]
    for bits in (32, 8):
        step_and_check([Tensor(gen, *s, BF, BF, bits) for s in shapes], seed=1 << 40)


@pytest.mark.parametrize("t", [1, 2, 1000, 10 ** 7, 3 * 2 ** 32 + 5])
def test_steps(t):
    gen = torch.Generator().manual_seed(5)
    kinds = [(F, F, 32), (BF, BF, 8)]
    step_and_check([Tensor(gen, 3, 333, *k) for k in kinds], t=t, seed=9)
    gen = torch.Generator().manual_seed(5)
    step_and_check([Tensor(gen, 3, 333, *k) for k in kinds], t=t, seed=9, lr=torch.tensor([0.03], device="cuda"),
                   tstep=torch.tensor([t], device="cuda"))


@pytest.mark.parametrize("factor", [1.0, 0.25, 1e-3, -2.0, 0.0])
def test_factor(factor):
    gen = torch.Generator().manual_seed(6)
    step_and_check([Tensor(gen, 3, 333, *k) for k in [(F, F, 32), (BF, BF, 8), (BF, F, 32), (F, BF, 8, 1)]],
                   factor=torch.tensor(factor, device="cuda"))


def test_a_factor_of_nan_leaves_all_as_it_was():
    gen = torch.Generator().manual_seed(7)
    ts = [Tensor(gen, 5, 333, *k) for k in [(F, F, 32), (BF, BF, 8), (BF, F, 32, 1)]]
    G = [t.g for t in ts]
    G[1][2, 5] = float("inf")
    out = api.grad_norm(G, 1.0)
    assert math.isinf(out[0].item()) and math.isnan(out[1].item())
    before = [memory.clone() for t in ts for memory, _, _ in t.gaps]
    api.adamw_step([t.x for t in ts], G, [t.m for t in ts], [t.v for t in ts], 0.1, 1, SM=[t.sm for t in ts],
                   SV=[t.sv for t in ts], factor=out[1:])
    for a, b in zip(before, (memory for t in ts for memory, _, _ in t.gaps)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("seed", [None, 3])
def test_infinities_and_nan_stay_where_they_are(bits, seed):
    gen = torch.Generator().manual_seed(8)
    bad = Tensor(gen, 4, 300, F, F, bits)
    gen = torch.Generator().manual_seed(8)
    good = Tensor(gen, 4, 300, F, F, bits)
    places = [(0, 0, float("nan")), (1, 130, float("inf")), (2, 299, -float("inf"))]
    for t in (bad, good):
        for i, j, v in places:
            t.g[i, j] = v if t is bad else 0.0
        api.adamw_step([t.x], [t.g], [t.m], [t.v], 0.1, 3, SM=[t.sm] if bits == 8 else None,
                       SV=[t.sv] if bits == 8 else None, seed=seed)
    hit = torch.zeros(4, 300, dtype=torch.bool)
    for i, j, _ in places:
        hit[i, j] = True
    for name in "xmv":
        a, b = getattr(bad, name).cpu().float(), getattr(good, name).cpu().float()
        if bits == 32 or name == "x":
            assert torch.equal(a[~hit], b[~hit])
        assert bool(torch.isfinite(a[~hit]).all())
    m = bad.m.cpu().float()[hit]
    assert bool((torch.isnan(m) if bits == 8 else ~torch.isfinite(m)).all())
    if bits == 8:   # scales of finite values alone
        assert bool(torch.isfinite(bad.sm).all()) and bool(torch.isfinite(bad.sv).all())
        blocks = torch.ones(4, 3, dtype=torch.bool)
        for i, j, _ in places:
            blocks[i, j // 128] = False
        assert torch.equal(bad.sm.cpu()[blocks], good.sm.cpu()[blocks])


def test_squares_beyond_fp32_do_not_poison_8_bit_states():
    """g^2 is infinite: no update of the weight but its decay, and the kept root stays a number."""
    for bits in (8, 32):
        x, g = torch.full((1, 256), 2.0, device="cuda"), torch.zeros(1, 256, device="cuda")
        g[0, 200] = 1e25
        M, V, SM, SV = api.adamw_states([x], bits)
        for t in range(1, 4):
            api.adamw_step([x], [g], M, V, 0.1, t, SM=SM, SV=SV, weight_decay=0.0)
            g.zero_()
        assert torch.equal(x.cpu(), torch.full((1, 256), 2.0)) or (bits == 8 and abs(x[0, 200].item() - 2) < 1e7 and
                                                                  bool((x[0, :200] == 2).all()))


@pytest.mark.parametrize("std", [1e-22, 1e-20, 1e-18, 1e-16, 1e-13, 1e13, 1e17])
@pytest.mark.parametrize("seed", [None, 6])
def test_gradients_at_the_ends_of_the_range(std, seed):
    """Squares around fp32's smallest numbers, where the root is formed another way, and near its largest."""
    gen = torch.Generator().manual_seed(12)
    ts = [Tensor(gen, 4, 1537, F, F, bits) for bits in (32, 8)]
    for t in ts:
        t.x.mul_(std)
        t.g.mul_(std * 1e3)
        t.m.zero_() if t.bits == 32 else t.m.view(torch.uint8).zero_()
        t.v.zero_() if t.bits == 32 else t.v.view(torch.uint8).zero_()
        t.g[1, 5] = 1e-3        # (one block with a gradient of ordinary size)
        for i, (memory, view, _) in enumerate(t.gaps):
            t.gaps[i] = (memory, view, memory.clone())
    step_and_check(ts, seed=seed)


def test_a_small_root_never_becomes_zero():
    """Beside a large neighbour sqrt(v) is far below the least code, and gets it all the same."""
    for seed in (None, 1, 2):
        x, g = torch.zeros(1, 128, device="cuda"), torch.full((1, 128), 1e-9, device="cuda")
        g[0, 0] = 1.0
        g[0, 1] = 0.0
        M, V, SM, SV = api.adamw_states([x], 8)
        api.adamw_step([x], [g], M, V, 0.1, 1, SM=SM, SV=SV, seed=seed, eps=1e-30)
        v = V[0].float().cpu()
        assert v[0, 0] == 448 and v[0, 1] == 0 and bool((v[0, 2:] == 2.0 ** -9).all())


def test_states_from_the_start_and_several_steps():
    """adamw_states, parameters of any shape, and ten steps against the 64-bit run of the same."""
    gen = torch.Generator().manual_seed(9)
    shapes = [(5,), (), (3, 4, 5, 6), (7, 130), (2, 3, 64)]
    x = [torch.randn(s, generator=gen).cuda() for s in shapes]
    want = [t.cpu().double() for t in x]
    M, V, SM, SV = api.adamw_states(x)
    assert SM is None and SV is None
    m, v = [torch.zeros_like(t) for t in want], [torch.zeros_like(t) for t in want]
    X = api.mats(x)
    for t in range(1, 11):
        g = [torch.randn(s, generator=gen) for s in shapes]
        api.adamw_step(X, [t_.cuda() for t_ in g], M, V, 0.01, t)
        for i in range(len(x)):
            gi = g[i].double()
            m[i] = 0.9 * m[i] + 0.1 * gi
            v[i] = 0.999 * v[i] + 0.001 * gi * gi
            want[i] = want[i] * (1 - 0.01 * 0.01) - 0.01 * (m[i] / (1 - 0.9 ** t)) / (torch.sqrt(v[i] / (1 - 0.999 ** t)) + 1e-8)
    for a, b in zip(x, want):   # at most 15 roundings a step of values of about 4 at most, ten steps
        assert float((a.cpu().double() - b).abs().max()) < 10 * 15 * R.U * 4


def test_rounding_holds_what_is_small_on_the_average():
    """An update of 1/64 of a bf16 step, 256 times: to nearest it is lost, stochastically a step of
    4 +- 0.5 per element is made (256 / 64; standard deviation 2 each, 0.03 over 4096 elements)."""
    x = torch.ones(1, 4096, dtype=BF, device="cuda")
    g = torch.full((1, 4096), 1e-3, dtype=F, device="cuda")
    for seed, moved in ((None, 0.0), (77, 4.0)):
        w = x.clone()
        M, V, _, _ = api.adamw_states([w])
        for t in range(1, 257):   # a constant gradient: the update is lr in each step
            api.adamw_step([w], [g], M, V, 2.0 ** -8 / 64, t, weight_decay=0.0, eps=1e-12, seed=seed)
        mean = float((1 - w.double()).mean()) / 2.0 ** -8
        assert abs(mean - moved) < (0.2 if seed else 1e-9), mean


@pytest.mark.parametrize("bits,seed", [(32, None), (32, 4), (8, None), (8, 4)])
def test_the_same_bits_twice_and_in_any_company(bits, seed):
    """The same tensor alone, among others, and as rows of a wider matrix."""
    def make(pad=0):
        return Tensor(torch.Generator().manual_seed(10), 33, 777, BF, BF, bits, pad)

    def run(ts):
        api.adamw_step([t.x for t in ts], [t.g for t in ts], [t.m for t in ts], [t.v for t in ts], 0.1, 3,
                       SM=[t.sm for t in ts] if bits == 8 else None, SV=[t.sv for t in ts] if bits == 8 else None, seed=seed)
        return ts[0]

    other = Tensor(torch.Generator().manual_seed(11), 900, 1111, BF, BF, bits)
    a, b, c = run([make()]), run([make(), other]), run([make(pad=3)])
    for name in ("x", "m", "v") + (("sm", "sv") if bits == 8 else ()):
        for o in (b, c):
            p, q = getattr(a, name).contiguous(), getattr(o, name).contiguous()
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), name


# ---- the gradients' norm ----


@pytest.mark.parametrize("dtype", [BF, F])
def test_norm(dtype):
    gen = torch.Generator().manual_seed(20)
    shapes = SHAPES + [(1, 8192), (1, 8193), (33, 5000), (2, 32769)]
    for pad, shift in ((0, 0), (3, 1)):
        gs = [placed(values(gen, *s, 1e-3), dtype, s[1] + pad, shift)[1] for s in shapes]
        want = R.norm(gs)
        for most in (want * 2, want / 3, float("inf")):
            out = api.grad_norm(gs, most).cpu().double()
            factor = min(1.0, most / want)
            assert abs(out[0] - want) <= (R.U + 1e-12) * want and abs(out[1] - factor) <= (R.U + 1e-12) * factor


def test_norm_of_many_and_of_mixed_types():
    gen = torch.Generator().manual_seed(21)
    gs = [placed(values(gen, 1 + i % 3, 1 + 31 * i % 500, 10.0 ** (i % 7 - 3)), (BF, F)[i % 2], 600, i % 2)[1] for i in range(300)]
    want = R.norm(gs)
    ws = api.workspace(api.grad_norm_workspace_size(len(gs)), "cuda")
    a = api.grad_norm(gs, 1.0, ws=ws)
    assert abs(a[0].item() - want) <= (R.U + 1e-12) * want
    ws.fill_(255)
    assert torch.equal(a, api.grad_norm(api.mats(gs), 1.0, ws=ws))
    assert torch.equal(a, api.grad_norm(gs, 1.0, out=torch.empty(2, device="cuda")))


@pytest.mark.parametrize("value,norm", [(1e25, 1e25), (1e-30, 1e-30), (0.0, 0.0), (3e38, math.inf)])
def test_norm_at_the_ends_of_the_range(value, norm):
    """Squares beyond fp32; a norm beyond fp32 is infinite but its factor is not lost."""
    g = torch.full((1, 4), value, device="cuda")
    out = api.grad_norm([g], 2.0).cpu().double()
    exact = 2 * g[0, 0].item()
    assert out[0] == pytest.approx(exact if norm < math.inf else math.inf, rel=1e-6)
    assert out[1] == pytest.approx(min(1.0, 2.0 / exact) if exact else 1.0, rel=1e-6)
    g[0, 2] = float("nan")
    out = api.grad_norm([g], 2.0)
    assert bool(torch.isnan(out).all())


def test_overlapping_gradients_are_counted_each():
    g = torch.randn(1, 5000, device="cuda")
    out = api.grad_norm([g, g[:, :100], g[:, 50:]], 1.0)
    assert out[0].item() == pytest.approx(R.norm([g, g[:, :100], g[:, 50:]]), rel=1e-6)


# ---- graphs, streams ----


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_read_step_rate_and_factor_anew(bits):
    def make():
        gen = torch.Generator().manual_seed(30)
        return [Tensor(gen, *s, BF, BF, bits) for s in ((5, 333), (1, 2048), (70, 1000))]

    ts, eager = make(), make()
    lr, t = torch.tensor([0.1], device="cuda"), torch.tensor([1], device="cuda")
    ws, out = api.workspace(api.grad_norm_workspace_size(3), "cuda"), torch.empty(2, device="cuda")
    more = torch.ones(1, dtype=torch.int64, device="cuda")

    def call(q):
        api.grad_norm([x.g for x in q], 1.0, out=out, ws=ws)
        api.adamw_step([x.x for x in q], [x.g for x in q], [x.m for x in q], [x.v for x in q], lr, t,
                       SM=[x.sm for x in q] if bits == 8 else None, SV=[x.sv for x in q] if bits == 8 else None,
                       seed=3, factor=out[1:])

    call(make())
    t.add_(more)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ts)
        t.add_(more)
    torch.cuda.synchronize()
    for i in range(4):
        t.fill_(i + 1)
        lr.fill_(0.1 / (i + 1))
        new = [torch.randn(x.shape, device="cuda") * 10.0 ** (-i) for x in ts]
        for q in (ts, eager):
            for x, n in zip(q, new):
                x.g.copy_(n)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert t.item() == i + 2
        t.fill_(i + 1)
        call(eager)
        torch.cuda.synchronize()
        for a, b in zip(ts, eager):
            for name in ("x", "m", "v"):
                assert torch.equal(getattr(a, name).contiguous().view(torch.uint8), getattr(b, name).contiguous().view(torch.uint8))


def test_two_streams_at_once():
    """Steps on tensors of their own, and norms with workspaces of their own."""
    def make(seed):
        return [Tensor(torch.Generator().manual_seed(seed), 400, 3000, BF, BF, 32)]

    def run(ts, ws, n):
        outs = []
        for t in range(1, n + 1):
            out = api.grad_norm([x.g for x in ts], 0.5, ws=ws)
            api.adamw_step([x.x for x in ts], [x.g for x in ts], [x.m for x in ts], [x.v for x in ts], 0.1, t, factor=out[1:])
            outs.append(out)
        return outs

    want = [make(40), make(41)]
    size = api.grad_norm_workspace_size(1)
    for q in want:
        run(q, api.workspace(size, "cuda"), 6)
    got, wss = [make(40), make(41)], [api.workspace(size, "cuda") for _ in range(2)]
    torch.cuda.synchronize()
    streams, held = [torch.cuda.Stream() for _ in range(2)], []
    for q, ws, s in zip(got, wss, streams):
        with torch.cuda.stream(s):
            held.append(run(q, ws, 6))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0].x, b[0].x) and torch.equal(a[0].v, b[0].v)


def test_offsets_beyond_32_bits():
    """A weight of more than 2^31 elements, and rows further apart than that."""
    n = (1 << 31) + 4099
    x = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.zeros(n, dtype=BF, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g[-5:] = 1.0
    for call in (lambda: api.grad_norm([g]), lambda: api.adamw_step([x], [g], [m], [v], 0.5, 1)):
        with pytest.raises(api.OrthoError) as e:   # (2^30 columns at most)
            call()
        assert e.value.status == 2
    rows = n // 7
    x, g, m, v = (t[-7 * rows:].view(rows, 7) for t in (x, g, m, v))
    assert api.grad_norm([g])[0].item() == pytest.approx(5 ** 0.5)
    api.adamw_step([x], [g], [m], [v], 0.5, 1)
    assert bool((x.flatten()[-5:] == -0.5).all()) and int((x != 0).sum()) == 5
    del x, g, m, v
    wide = torch.zeros(3, 1 << 30, dtype=BF, device="cuda")
    for bits in (32, 8):
        X = [wide[:, :200]]
        M, V, SM, SV = api.adamw_states(X, bits)
        wide.zero_()
        api.adamw_step(X, [torch.ones(3, 200, dtype=BF, device="cuda")], M, V, 0.5, 1, SM=SM, SV=SV, weight_decay=0.0)
        assert bool((wide[:, :200] == -0.5).all()) and not bool(wide[:, 200:400].any())


def test_random_bits_of_more_than_2_to_the_32_elements():
    """Rows around element 2^32, which lies among a thread's eight."""
    cols, rows, seed, t = 8191, (1 << 32) // 8191 + 2, 99, 5
    first = rows - 3
    X, G = (torch.zeros(rows, cols, dtype=BF, device="cuda") for _ in range(2))
    gen = torch.Generator().manual_seed(13)
    x, g = values(gen, 3, cols, 0.02).to(BF), values(gen, 3, cols, 1e-3).to(BF)
    X[first:].copy_(x)
    G[first:].copy_(g)
    M, V, SM, SV = api.adamw_states([X], 8)
    api.adamw_step([X], [G], M, V, H["lr"], t, betas=H["betas"], eps=H["eps"], weight_decay=H["weight_decay"], SM=SM, SV=SV, seed=seed)
    zero = torch.zeros(3, cols, dtype=torch.float64)
    (xn, ex), (mn, em), (vn, ev) = R.step(x.double(), g.double(), zero, zero, H["lr"], t, H["betas"], H["eps"], H["weight_decay"])
    bits = R.random_bits(seed, t, 0, 3, cols, first)
    assert R.between(X[first:].cpu().double(), R.round_bf16(xn - ex, bits[0]), R.round_bf16(xn + ex, bits[0]))
    R.check_codes(M[0][first:], SM[0][first:], mn, em, bits[1], False)
    root, er = vn.sqrt(), (vn + ev).sqrt() - (vn - ev).clamp(min=0).sqrt()
    R.check_codes(V[0][first:], SV[0][first:], root, er + R.U * root, bits[2], True)
    assert not bool(X[:first].any())


def test_two_graphs_that_share_a_workspace():
    """Replayed one after the other, as a program may that runs them on one stream."""
    ws = api.workspace(api.grad_norm_workspace_size(100), "cuda")
    gs = [[torch.randn(3, 1000 + i, device="cuda") for i in range(n)] for n in (100, 3)]
    outs, graphs = [torch.zeros(2, device="cuda") for _ in gs], []
    for g, out in zip(gs, outs):
        api.grad_norm(g, 1.0, out=out, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.grad_norm(g, 1.0, out=out, ws=ws)
        graphs.append(graph)
    for k in range(4):
        for g in gs:
            for t in g:
                t.mul_(1.5)
        for graph in (graphs if k % 2 else graphs[::-1]):
            graph.replay()
        torch.cuda.synchronize()
        for g, out in zip(gs, outs):
            assert torch.equal(out, api.grad_norm(g, 1.0))
