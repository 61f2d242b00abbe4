"""Argument checks of AdamW, the gradients' norm and the tokens by expert, which need no GPU."""

import ctypes
import math

import pytest
import torch

from orthonormal_optimizer_update_amd import api
from test_fp8_cpu import BF, C8, DTYPE, E8, F, FAKE, LAYOUT, M, PARAM, SHAPE, WS, ref

OK, NULL = 0, 1


def at(i, byte=0):
    """Addresses 16 MiB apart."""
    return FAKE + (i << 24) + byte


def array(*mats):
    return (api.OrthoMat * len(mats))(*mats)


def hyper(**kw):
    h = api.OrthoAdamw(0.1, 0.9, 0.99, 1e-8, 0.01, 1, 0, 0, None, None, None)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def tensor(i, rows=30, cols=200, x=BF, g=BF, bits=32, **kw):
    """X, G, M, V, SM, SV of tensor i, far from the others."""
    b = -(-cols // 128)
    s = C8 if bits == 8 else F
    t = dict(X=M(rows, cols, x, data=at(6 * i)), G=M(rows, cols, g, data=at(6 * i + 1)), M=M(rows, cols, s, data=at(6 * i + 2)),
             V=M(rows, cols, s, data=at(6 * i + 3)), SM=M(rows, b, F, data=at(6 * i + 4)), SV=M(rows, b, F, data=at(6 * i + 5)))
    t.update(kw)
    return t


def adamw(tensors, h=None, count=None, scales=True):
    lists = [array(*[t[k] for t in tensors]) for k in ("X", "G", "M", "V", "SM", "SV")]
    if not scales:
        lists[4:] = [None, None]
    # (every call here is refused: what is right in one way is wrong in another that is looked at later)
    return api.lib().adamw_step(len(tensors) if count is None else count, *lists, ref(hyper() if h is None else h), None)


OVERLAP = dict(G=M(30, 200, F, data=at(0, 60)))   # what is looked at last: G in X


@pytest.mark.parametrize("kw,want", [
    (dict(X=M(30, 200, BF, data=None)), NULL), (dict(G=M(30, 200, BF, data=None)), NULL), (dict(SV=M(30, 2, F, data=None)), NULL),
    (dict(X=M(30, 200, C8, data=at(0))), DTYPE), (dict(G=M(30, 200, E8, data=at(1))), DTYPE), (dict(M=M(30, 200, BF, data=at(2))), DTYPE),
    (dict(V=M(30, 200, F, data=at(3))), DTYPE), (dict(SM=M(30, 2, E8, data=at(4))), DTYPE),
    (dict(G=M(30, 201, BF, data=at(1))), SHAPE), (dict(M=M(29, 200, C8, data=at(2))), SHAPE), (dict(SM=M(30, 3, F, data=at(4))), SHAPE),
    (dict(SV=M(1, 2, F, data=at(5))), SHAPE), (dict(X=M(0, 200, BF, data=at(0))), SHAPE),
    (dict(X=M(30, 200, BF, ld=199, data=at(0))), LAYOUT), (OVERLAP, LAYOUT),
])
def test_adamw_refuses(kw, want):
    assert adamw([tensor(0, bits=8, **kw)]) == want
    assert adamw([tensor(1), tensor(0, bits=8, **kw), tensor(2)]) == want


def test_adamw_refuses_far_rows():
    for k in ("X", "G", "M", "V", "SM", "SV"):
        t = tensor(0, bits=8)
        t[k] = M(t[k].rows, t[k].cols, t[k].dtype, ld=1 << 32, data=t[k].data)
        assert adamw([t]) == LAYOUT


def test_adamw_refuses_scalars_inside_the_tensors():
    t = tensor(0, bits=8)
    for k in ("X", "M", "V", "SM", "SV"):
        assert adamw([t], hyper(factor=t[k].data + 8)) == LAYOUT
        assert adamw([t], hyper(lr_dev=t[k].data + 8)) == LAYOUT
        assert adamw([t], hyper(step_dev=t[k].data - 4)) == LAYOUT


def test_adamw_refuses_missing_lists():
    t = tensor(0, bits=8)
    assert adamw([t], scales=False) == NULL
    x = array(t["X"])
    L = api.lib()
    for k in range(5):
        args = [x, x, x, x]
        h = ref(hyper())
        if k < 4:
            args[k] = None
        else:
            h = None
        assert L.adamw_step(1, *args, None, None, h, None) == NULL
    assert adamw([t], count=0) == PARAM and adamw([t], count=-1) == PARAM
    # scales that no tensor needs are not looked at
    assert adamw([tensor(0, SM=M(1, 1, 9, data=None), SV=M(1, 1, 9, data=None), **OVERLAP)]) == LAYOUT


@pytest.mark.parametrize("kw", [
    dict(lr=math.nan), dict(lr=math.inf), dict(lr=1e39), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan),
    dict(eps=0.0), dict(eps=1e-39), dict(eps=-1.0), dict(eps=math.nan), dict(eps=1e39), dict(weight_decay=-0.1), dict(weight_decay=math.inf),
    dict(weight_decay=math.nan), dict(step=0), dict(step=-5)])
def test_adamw_refuses_parameters(kw):
    assert adamw([tensor(0)], hyper(**kw)) == PARAM


@pytest.mark.parametrize("kw", [dict(beta1=0.0), dict(beta2=0.0), dict(eps=2.0 ** -126), dict(step=0, step_dev=FAKE), dict(weight_decay=0.0),
                                dict(lr=0.0), dict(lr=-1.0), dict(step=2 ** 62)])
def test_adamw_takes_parameters(kw):
    assert adamw([tensor(0, **OVERLAP)], hyper(**kw)) == LAYOUT   # (gets as far as the overlap)


@pytest.mark.parametrize("eps,status", [(2.0 ** 100, LAYOUT), (1.01 * 2.0 ** 100, PARAM), (1e38, PARAM)])
def test_adamw_largest_eps(eps, status):
    assert adamw([tensor(0, **OVERLAP)], hyper(eps=eps)) == status


def test_adamw_refuses_too_many_elements():
    n = 1 << 30
    assert adamw([tensor(0, rows=n, cols=1025)]) == SHAPE
    assert api.lib().grad_norm(1, array(M(n, 1025, BF)), 1.0, at(9), at(10), 1 << 20, None) == SHAPE


@pytest.mark.parametrize("bits", [8, 32])
def test_a_tensor_twice_or_partly_in_another_is_refused(bits):
    t, u = tensor(0, bits=bits), tensor(1, bits=bits)
    assert adamw([t, u, t]) == LAYOUT
    names = ["X", "M", "V"] + (["SM", "SV"] if bits == 8 else [])
    for a in names:
        for b in names + ["G"]:
            if a == "X" and b == "X" or a != b:
                last = t[b].data + (t[b].rows * t[b].cols - 1) * {F: 4, BF: 2, C8: 1}[t[b].dtype]   # its last element
                moved = dict(u)
                moved[a] = M(u[a].rows, u[a].cols, u[a].dtype, data=last)
                assert adamw([t, moved]) == LAYOUT, (a, b)
                assert adamw([moved, t]) == LAYOUT, (a, b)


@pytest.mark.parametrize("args,want", [
    (dict(count=0), PARAM), (dict(most=0.0), PARAM), (dict(most=-1.0), PARAM), (dict(most=math.nan), PARAM), (dict(out=None), NULL),
    (dict(g=None), NULL), (dict(out=at(0, 8)), LAYOUT), (dict(ws=None), WS), (dict(size=16383), WS), (dict(ws=at(8, 8)), WS),
    (dict(dtype=C8), DTYPE)])
def test_grad_norm_refuses(args, want):
    a = dict(count=2, most=1.0, out=at(5), ws=at(8), size=16384, g=0, dtype=BF)
    a.update(args)
    g = None if a["g"] is None else array(M(5, 9, a["dtype"], data=at(0)), M(1, 7, F, data=at(1)))
    assert api.lib().grad_norm(a["count"], g, a["most"], a["out"], a["ws"], a["size"], None) == want


def test_grad_norm_workspace():
    size = api.grad_norm_workspace_size
    assert size(0) == 0 and size(-1) == 0 and size(1) == 16384 and size(64) == 16384 and size(65) == 32768


# ---- tokens by expert ----


def test_expert_rows_and_workspace():
    rows, ws = api.expert_rows, api.expert_sort_workspace_size
    assert rows(10, 3, 4, 8) == 30 + 28 and rows(1, 1, 1, 1) == 1
    for bad in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 65, 100, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0), (1, 1, 1, 4097),
                (1 << 30, 1, 1, 1), (1 << 25, 32, 1, 1), ((1 << 30) - 1, 1, 1024, 4096), (1 << 62, 64, 1, 1), (-1, 1, 1, 1)):
        assert rows(*bad) == 0, bad
    assert rows((1 << 30) - 1, 1, 1, 1) == (1 << 30) - 1 and rows((1 << 24) - 1, 64, 1, 1) == 64 * ((1 << 24) - 1)
    assert ws(0, 1, 1) == 0 and ws(1, 1, 1025) == 0 and ws(2048, 1, 64) == 256 and ws(2049, 1, 64) == 2 * 64 * 4
    assert ws((1 << 30) - 1, 1, 1024) <= 1024 * 1024 * 4


def sort(**kw):
    a = dict(chosen=at(0), bytes=4, tokens=30, choices=2, experts=5, align=4, slot=at(1), source=at(2), offsets=at(3), counts=at(4),
             ws=at(5), size=0)   # (no workspace: what is looked at last)
    a.update(kw)
    return api.lib().expert_sort(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(), WS), (dict(source=None), WS), (dict(chosen=None), NULL), (dict(slot=None), NULL), (dict(offsets=None), NULL),
    (dict(counts=None), NULL), (dict(bytes=2), DTYPE), (dict(tokens=0), SHAPE), (dict(choices=65), SHAPE), (dict(experts=0), SHAPE),
    (dict(align=5000), SHAPE), (dict(slot=at(0, 236)), LAYOUT), (dict(slot=at(0, 240)), WS), (dict(source=at(1, 236)), LAYOUT),
    (dict(offsets=at(4, 16)), LAYOUT), (dict(counts=at(3, 20)), LAYOUT), (dict(counts=at(3, 24)), WS), (dict(size=256, ws=at(5, 4)), WS),
    (dict(bytes=8, slot=at(0, 476)), LAYOUT)])
def test_expert_sort_refuses(kw, want):
    assert sort(**kw) == want


def gather(**kw):
    a = dict(X=M(30, 200, C8, data=at(0)), S=M(30, 2, F, data=at(1)), slot=at(2), choices=2, offsets=at(3), counts=at(4), experts=5,
             Y=M(80, 200, C8, data=at(5)), SY=M(80, 2, F, data=at(6)))
    a.update(kw)
    p = lambda m: None if m is None else ref(m)
    return api.lib().expert_gather(a["X"], p(a["S"]), a["slot"], a["choices"], a["offsets"], a["counts"], a["experts"], a["Y"],
                                   p(a["SY"]), None)


@pytest.mark.parametrize("kw,want", [
    (dict(slot=None), NULL), (dict(offsets=None), NULL), (dict(counts=None), NULL), (dict(S=None), NULL), (dict(SY=None), NULL),
    (dict(X=M(30, 200, BF, data=at(0))), DTYPE), (dict(X=M(30, 200, BF, data=at(0)), Y=M(80, 200, BF, data=at(5))), DTYPE),
    (dict(X=M(30, 200, E8, data=at(0))), DTYPE), (dict(Y=M(80, 201, C8, data=at(5))), SHAPE), (dict(choices=0), SHAPE),
    (dict(choices=65), SHAPE), (dict(experts=0), SHAPE), (dict(experts=1025), SHAPE), (dict(S=M(30, 1, F, data=at(1))), SHAPE),
    (dict(SY=M(79, 2, F, data=at(6))), SHAPE), (dict(SY=M(80, 2, E8, data=at(6))), DTYPE), (dict(S=M(1, 2, F, data=at(1))), SHAPE),
    (dict(Y=M(80, 200, C8, data=at(0, 5999))), LAYOUT), (dict(Y=M(80, 200, C8, data=at(2, 239))), LAYOUT),
    (dict(Y=M(80, 200, C8, data=at(3, 23))), LAYOUT), (dict(Y=M(80, 200, C8, data=at(4, 19))), LAYOUT),
    (dict(SY=M(80, 2, F, data=at(5, 15996))), LAYOUT), (dict(SY=M(80, 2, F, data=at(1))), LAYOUT),
    (dict(X=M(1 << 29, 200, C8, data=at(0)), S=M(1 << 29, 2, F, data=at(1))), SHAPE)])
def test_expert_gather_refuses(kw, want):
    assert gather(**kw) == want


def combine(**kw):
    a = dict(Y=M(80, 200, BF, data=at(0)), slot=at(1), choices=2, W=M(30, 2, F, data=at(2)), Add=M(30, 200, F, data=at(3)),
             Out=M(30, 200, BF, data=at(4)))
    a.update(kw)
    p = lambda m: None if m is None else ref(m)
    return api.lib().expert_combine(a["Y"], a["slot"], a["choices"], p(a["W"]), p(a["Add"]), a["Out"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(slot=None), NULL), (dict(Y=M(80, 200, C8, data=at(0))), DTYPE), (dict(Out=M(30, 200, F, data=at(4))), DTYPE),
    (dict(W=M(30, 2, C8, data=at(2))), DTYPE), (dict(Add=M(30, 200, C8, data=at(3))), DTYPE), (dict(choices=3), SHAPE),
    (dict(choices=65), SHAPE), (dict(W=M(29, 2, F, data=at(2))), SHAPE), (dict(Add=M(30, 199, F, data=at(3))), SHAPE),
    (dict(Out=M(30, 199, BF, data=at(4))), SHAPE), (dict(Out=M(30, 200, BF, data=at(0, 31998))), LAYOUT),
    (dict(Add=M(30, 200, BF, data=at(4, 2))), LAYOUT), (dict(Add=M(30, 200, F, data=at(4))), LAYOUT),
    (dict(W=M(30, 2, F, data=at(4, 11996))), LAYOUT), (dict(Out=M(30, 200, BF, data=at(1, 238))), LAYOUT)])
def test_expert_combine_refuses(kw, want):
    assert combine(**kw) == want


def backward(**kw):
    a = dict(dOut=M(30, 200, BF, data=at(0)), slot=at(1), choices=2, W=M(30, 2, F, data=at(2)), offsets=at(3), counts=at(4), experts=5,
             dY=M(80, 200, BF, data=at(5)), Y=M(80, 200, BF, data=at(6)), dW=M(30, 2, F, data=at(7)))
    a.update(kw)
    p = lambda m: None if m is None else ref(m)
    return api.lib().expert_combine_backward(a["dOut"], a["slot"], a["choices"], p(a["W"]), a["offsets"], a["counts"], a["experts"],
                                             a["dY"], p(a["Y"]), p(a["dW"]), None)


@pytest.mark.parametrize("kw,want", [
    (dict(slot=None), NULL), (dict(offsets=None), NULL), (dict(counts=None), NULL), (dict(Y=None), NULL), (dict(dW=None), NULL),
    (dict(dOut=M(30, 200, C8, data=at(0))), DTYPE), (dict(dY=M(80, 200, F, data=at(5))), DTYPE), (dict(Y=M(80, 200, F, data=at(6))), DTYPE),
    (dict(dW=M(30, 2, BF, data=at(7))), DTYPE), (dict(W=M(30, 2, E8, data=at(2))), DTYPE), (dict(Y=M(81, 200, BF, data=at(6))), SHAPE),
    (dict(dW=M(30, 3, F, data=at(7))), SHAPE), (dict(W=M(30, 1, F, data=at(2))), SHAPE), (dict(dY=M(80, 100, BF, data=at(5))), SHAPE),
    (dict(experts=0), SHAPE), (dict(dY=M(80, 200, BF, data=at(0, 11998))), LAYOUT), (dict(dY=M(80, 200, BF, data=at(6, 2))), LAYOUT),
    (dict(dY=M(80, 200, BF, ld=201, data=at(6))), LAYOUT), (dict(dW=M(30, 2, F, data=at(2))), LAYOUT),
    (dict(dW=M(30, 2, F, data=at(0))), LAYOUT), (dict(dW=M(30, 2, F, data=at(5))), LAYOUT), (dict(dW=M(30, 2, F, data=at(6))), LAYOUT),
    (dict(dY=M(80, 200, BF, data=at(3, 22))), LAYOUT), (dict(dW=M(30, 2, F, data=at(1))), LAYOUT)])
def test_expert_combine_backward_refuses(kw, want):
    assert backward(**kw) == want


# ---- the binding ----


def test_tensors_as_matrices():
    f = api.binding().matrix
    t = torch.zeros(4, 6, 8)
    assert f(torch.zeros(())) == (1, 1, 1) and f(torch.zeros(7)) == (1, 7, 7) and f(t) == (4, 48, 48)
    assert f(t[:, 0]) == (4, 8, 48) and f(t[1:2]) == (1, 48, 48)
    assert f(torch.zeros(5, 3)[:, 1:]) == (5, 2, 3) and f(torch.zeros(8, 1, 3)) == (8, 3, 3)
    assert f(torch.zeros(6, 1)[::2]) == (3, 1, 2) and f(torch.zeros(1, 4, 4)[:, :, 0:]) == (1, 16, 16)
    assert f(torch.zeros(1)[::3]) == (1, 1, 1) and f(torch.zeros(0)) == (1, 0, 1)
    assert f(t[:, :3]) == (4, 24, 48)   # rows with gaps between them
    for bad in (t[:, 1:, :3], t[:, :, ::2], t.transpose(0, 1), torch.zeros(8)[::2], torch.zeros(1, 8).expand(3, 8), torch.zeros(8, 4).t(),
                t[:, :, :0]):
        with pytest.raises(ValueError):
            f(bad)
    with pytest.raises(ValueError):
        f(3)


def test_the_binding_wants_a_gpu():
    x = torch.zeros(3, 4)
    for call in (lambda: api.mats([x]), lambda: api.adamw_step([x], [x], [x], [x], 0.1, 1), lambda: api.grad_norm([x]),
                 lambda: api.expert_sort(torch.zeros(2, 2, dtype=torch.int32), 4),
                 lambda: api.expert_gather(x, torch.zeros(3, 1, dtype=torch.int32), x, x, Y=x),
                 lambda: api.expert_combine(x, torch.zeros(3, 1, dtype=torch.int32)),
                 lambda: api.expert_combine_backward(x, torch.zeros(3, 1, dtype=torch.int32), None, x, x, Y=x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="chosen"):
        api.expert_sort(torch.zeros(4, dtype=torch.int32), 4)
    for empty in ([], [None]):
        with pytest.raises(ValueError, match="at least one"):
            api.mats(empty)
        with pytest.raises(ValueError, match="at least one"):
            api.grad_norm(empty)
    with pytest.raises(ValueError):
        api.adamw_states([x], 16)


def test_states_of_any_shape():
    shapes = [(), (5,), (3, 4, 50), (7, 130)]
    M_, V, SM, SV = api.adamw_states([torch.zeros(s) for s in shapes], 8)
    for s, m, v, a, b in zip(shapes, M_, V, SM, SV):
        assert m.shape == v.shape == torch.Size(s) and m.dtype == torch.float8_e4m3fn
        rows, cols, _ = api.binding().matrix(torch.zeros(s))
        assert a.shape == b.shape == (rows, -(-cols // 128)) and bool((a == 1).all())


def test_the_binding_counts_its_arguments():
    b = api.binding()
    for name in ("check", "matrix", "grad_norm", "adamw_step", "expert_sort", "expert_gather", "expert_combine", "expert_combine_backward"):
        with pytest.raises(TypeError):
            getattr(b, name)(*range(30))


@pytest.mark.gpu
class TestRefusalsOfTensors:
    """What the binding raises for tensors that no descriptor can stand for."""

    def z(self, *shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    def test_lists(self):
        z = self.z
        a, cpu = [z(3, 4), z(5)], torch.zeros(3, 4)
        assert len(api.mats(a)) == 2 and api.mats([None, a[0]])[0] is None
        for bad, what in (([cpu, a[0]], "GPU"), ([a[0], cpu], "GPU"), ([z(3, 4).half()], "dtype"), ([z(4, 3).t()], "stride"),
                          ([a[0], 3], "tensor"), ([z(1, 3).expand(4, 3)], "overlap")):
            with pytest.raises(ValueError, match=what):
                api.mats(bad)
            with pytest.raises(ValueError):
                api.grad_norm(bad)
        M, V, _, _ = api.adamw_states(a)
        with pytest.raises(ValueError, match="2 tensors in each list, got 1"):
            api.adamw_step(a, a[:1], M, V, 0.1, 1)
        with pytest.raises(ValueError, match="lr"):
            api.adamw_step(a, [z(3, 4), z(5)], M, V, z(2), 1)
        with pytest.raises(ValueError, match="step"):
            api.adamw_step(a, [z(3, 4), z(5)], M, V, 0.1, z(1))
        with pytest.raises(ValueError, match="factor"):
            api.adamw_step(a, [z(3, 4), z(5)], M, V, 0.1, 1, factor=z(1, dtype=torch.float64))
        with pytest.raises(ValueError, match="GPU"):
            api.adamw_step(a, [z(3, 4), z(5)], M, V, 0.1, 1, factor=torch.ones(1))
        with pytest.raises(TypeError):
            api.adamw_step(a, [z(3, 4), z(5)], M, V, "0.1", 1)
        with pytest.raises(TypeError):
            api.adamw_step(a, [z(3, 4), z(5)], M, V, 0.1, 1.5)
        with pytest.raises(api.OrthoError) as e:       # a gradient that is not there
            api.adamw_step(a, [z(3, 4), None], M, V, 0.1, 1)
        assert e.value.status == NULL
        for out in (z(3), z(2, dtype=torch.bfloat16), z(4)[::2]):
            with pytest.raises(ValueError, match="out"):
                api.grad_norm(a, out=out)
        with pytest.raises(api.OrthoError) as e:
            api.grad_norm(a, ws=z(1).expand(1 << 20))
        assert e.value.status == WS
        assert not any(bool(t.any()) for t in a)

    def test_rows(self):
        z = self.z
        chosen = z(6, 2, dtype=torch.int32)
        for bad in (z(6, 2), z(6, 4, dtype=torch.int64)[:, ::2], z(12, dtype=torch.int32)):
            with pytest.raises(ValueError, match="chosen"):
                api.expert_sort(bad, 4)
        slot, source, offsets, counts = api.expert_sort(chosen, 4)
        for kw in (dict(slot=z(6, 2)), dict(slot=z(5, 2, dtype=torch.int32)), dict(source=z(11, dtype=torch.int32)),
                   dict(offsets=counts), dict(counts=offsets), dict(slot=slot.cpu())):
            with pytest.raises(ValueError, match="GPU" if "slot" in kw and not kw["slot"].is_cuda else next(iter(kw))):
                api.expert_sort(chosen, 4, **kw)
        with pytest.raises(ValueError, match="align"):
            api.expert_sort(chosen, 4, 1 << 33, slot, source, offsets, counts, z(256, dtype=torch.uint8))
        X = z(6, 8)
        with pytest.raises(ValueError, match="rows"):
            api.expert_gather(X, slot, offsets, counts)
        with pytest.raises(ValueError, match="slot"):
            api.expert_gather(X[:5], slot, offsets, counts, rows=12)
        with pytest.raises(ValueError, match="offsets"):
            api.expert_gather(X, slot, counts, counts, rows=12)
        with pytest.raises(ValueError, match="2-D"):
            api.expert_gather(X, slot, offsets, counts, Y=z(12, 8, 1))
        Y, _ = api.expert_gather(X, slot, offsets, counts, rows=12)
        with pytest.raises(api.OrthoError) as e:
            api.expert_combine(Y, slot, z(6, 3))
        assert e.value.status == SHAPE
        with pytest.raises(ValueError, match="slot"):
            api.expert_combine(Y, slot.long(), out=X)
        with pytest.raises(ValueError, match="rows"):
            api.expert_combine_backward(X, slot, None, offsets, counts)
        with pytest.raises(api.OrthoError) as e:
            api.expert_combine_backward(X, slot, None, offsets, counts, rows=12, Y=z(11, 8))
        assert e.value.status == SHAPE
