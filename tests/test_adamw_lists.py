"""Lists of tensors given as what can be gone through only once."""

import pytest
import torch

from orthonormal_optimizer_update_amd import api


class OnAGpu:
    """What the binding is not asked about here: a tensor on GPU 0."""
    device = "cuda:0"

    def get_device(self):
        return 0


@pytest.fixture
def calls(monkeypatch):
    """The arguments of the binding's calls, lists gone through as it does."""
    seen = []

    class Binding:
        def __getattr__(self, name):
            def call(*args):
                seen.append([list(a) if hasattr(a, "__iter__") and not isinstance(a, torch.Tensor) else a for a in args])
                return 0
            return call

    monkeypatch.setattr(api, "_binding", Binding())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    return seen


@pytest.mark.parametrize("make", [list, tuple, iter, lambda x: (t for t in x)])
def test_every_item_reaches_the_binding(calls, make):
    x = [OnAGpu() for _ in range(5)]
    api.grad_norm(make(x), out=torch.empty(2), ws=torch.empty(1))
    assert calls[-1][0] == x
    api.adamw_step(make(x), make(x), make(x), make(x), 0.1, 1, SM=make(x), SV=make(x))
    assert calls[-1][:6] == [x] * 6
    api.adamw_step(make(x), make(x), make(x), make(x), 0.1, 1)
    assert calls[-1][:6] == [x] * 4 + [None, None]


def test_an_empty_iterator_is_refused():
    for call in (lambda: api.grad_norm(iter([])), lambda: api.adamw_step(iter([]), [], [], [], 0.1, 1)):
        with pytest.raises(ValueError, match="at least one"):
            call()


@pytest.mark.gpu
def test_norm_and_step_of_iterators():
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = [torch.randn(3, 50 + i, generator=gen, device="cuda") for i in range(5)]
    ws = api.workspace(api.grad_norm_workspace_size(len(g)), "cuda")
    want = api.grad_norm(g, 1.0)
    assert torch.equal(api.grad_norm(iter(g), 1.0, ws=ws), want)
    assert torch.equal(api.grad_norm((t for t in g), 1.0), want)
    g[0][1, 7] = float("inf")
    assert bool(torch.isnan(api.grad_norm((t for t in g), 1.0, ws=ws)[1]))
    g[0][1, 7] = 0.0
    x, y = [torch.ones_like(t) for t in g], [torch.ones_like(t) for t in g]
    a, b = api.adamw_states(x), api.adamw_states(y)
    api.adamw_step(x, g, a[0], a[1], 0.1, 1)
    api.adamw_step(iter(y), iter(g), iter(b[0]), iter(b[1]), 0.1, 1)
    for p, q in zip(x + a[0] + a[1], y + b[0] + b[1]):
        assert torch.equal(p, q)


@pytest.mark.parametrize("bits", [32, 8])
def test_states_for_an_iterator(bits):
    shapes = [(3,), (4, 5), (2, 3, 64)]
    want = api.adamw_states([torch.zeros(s) for s in shapes], bits)
    got = api.adamw_states((torch.zeros(s) for s in shapes), bits)
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or [t.shape for t in a] == [t.shape for t in b])
