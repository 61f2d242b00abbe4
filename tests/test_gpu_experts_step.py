"""One training step of a mixture-of-experts layer through the operators together: norm, sort, gather of
8-bit rows, the experts' products, weighted combination, its gradient, the experts' weight gradients,
clipping, Muon on the experts' matrices and AdamW on the rest.  Each operator's result is held to 64-bit
arithmetic on the operands that it got."""

import pytest
import torch

import adamw_ref
import experts_ref
import oracle
from fp8_ref import e4m3_values, expand, rms_norm_backward, scale_values
from orthonormal_optimizer_update_amd import api

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24
TOKENS, CHOICES, EXPERTS, ALIGN, D = 500, 2, 5, 128, 256


def product(a, b):
    """a b^T in 64 bits, and the bound of fp32 sums over k of them."""
    return a @ b.t(), (a.shape[1] + 8) * U * (a.abs() @ b.abs().t())


def close(got, want, err):
    assert bool(((got.cpu().double() - want).abs() <= err + 1e-30).all())


@pytest.mark.parametrize("scale_dtype", [torch.float32, torch.float8_e8m0fnu])
def test_a_layers_step(scale_dtype):
    gen = torch.Generator().manual_seed(17)
    rand = lambda *s: torch.randn(*s, generator=gen).cuda()
    x, norm_w, router = rand(TOKENS, D).to(BF), 1 + 0.1 * rand(1, D), 0.1 * rand(EXPERTS, D)
    W = [0.05 * rand(D, D) for _ in range(EXPERTS)]
    r = 1e-2 * rand(TOKENS, D)

    # forward: the norm's codes go to the experts' rows
    y = torch.empty_like(x)
    q, s = api.rms_norm_fp8(x, norm_w, y_out=y, scale_dtype=scale_dtype)
    logits = y.float() @ router.t()
    weights, chosen = torch.topk(torch.softmax(logits, 1), CHOICES, dim=1)
    chosen[::7] = -1                                   # padding of the batch
    weights = weights.contiguous()
    slot, source, offsets, counts = api.expert_sort(chosen, EXPERTS, ALIGN)
    rows = api.expert_rows(TOKENS, CHOICES, EXPERTS, ALIGN)
    xe, se = api.expert_gather(q, slot, offsets, counts, S=s, rows=rows)
    start, count = offsets.tolist(), counts.tolist()   # the one number that the host waits for
    quantized = [api.fp8_quantize(w, block_rows=128, scale_dtype=scale_dtype, transposed=True) for w in W]
    h = torch.zeros(rows, D, device="cuda")
    for e in range(EXPERTS):
        part = slice(start[e], start[e + 1])           # whole blocks of 128: rows of padding are zeros
        if count[e]:
            api.fp8_matmul(xe[part], se[part], quantized[e][0], quantized[e][1], out=h[part])
    residual = x.float()
    out = api.expert_combine(h, slot, weights, add=residual)

    xv = e4m3_values(q) * expand(scale_values(s), TOKENS, D, 1)
    wv = [e4m3_values(k[0]) * expand(scale_values(k[1]), D, D, 128) for k in quantized]
    want, err = torch.zeros(TOKENS, D, dtype=torch.float64), torch.zeros(TOKENS, D, dtype=torch.float64)
    sl, wt = slot.cpu(), weights.cpu().double()
    for t in range(TOKENS):
        for j in range(CHOICES):
            if chosen[t, j] >= 0:
                p, ep = product(xv[t:t + 1], wv[int(chosen[t, j])])
                want[t] += wt[t, j] * p[0]
                err[t] += wt[t, j] * (ep[0] + 4 * U * p[0].abs())
    want += residual.cpu().double()
    close(out, want, err + 4 * U * want.abs())
    assert not bool(h[source[:start[-1]].cpu().numpy().tolist().index(-1)].any())   # padding gives zeros
    for t in range(0, TOKENS, 7):
        assert torch.equal(out[t], residual[t])

    # backward
    dh, dw = api.expert_combine_backward(r, slot, weights, offsets, counts, Y=h, dY=torch.zeros_like(h))
    want_dh, want_dw, err_dw = experts_ref.combine_backward(r.cpu().double(), h.cpu().double(), sl, wt, rows)
    close(dw, want_dw, err_dw)
    used = (source >= 0).cpu()
    close(dh[used.cuda()], want_dh[used], 2 * U * want_dh[used].abs())
    end = start[-1]
    dq, ds, dqt, dst = api.fp8_quantize(dh[:end], scale_dtype=scale_dtype, transposed=True)
    ye, _ = api.expert_gather(y, slot, offsets, counts, rows=rows)
    _, _, yt, st = api.fp8_quantize(ye[:end], scale_dtype=scale_dtype, transposed=True)
    grads, dxe = [], torch.zeros_like(h)
    for e in range(EXPERTS):
        part, blocks = slice(start[e], start[e + 1]), slice(start[e] // 128, start[e + 1] // 128)
        if not count[e]:
            grads.append(torch.zeros(D, D, device="cuda"))
            continue
        g = api.fp8_matmul(dqt[:, part], dst[:, blocks], yt[:, part], st[:, blocks], out_dtype=F)
        a = e4m3_values(dqt[:, part]) * expand(scale_values(dst[:, blocks]), D, part.stop - part.start, 1)
        b = e4m3_values(yt[:, part]) * expand(scale_values(st[:, blocks]), D, part.stop - part.start, 1)
        close(g, *product(a, b))
        grads.append(g)
        api.fp8_matmul(dq[part], ds[part], quantized[e][2], quantized[e][3], out=dxe[part])
    dy = api.expert_combine(dxe, slot)
    sums, es = experts_ref.combine(dxe.cpu().double(), sl, None, None)
    close(dy, sums, es + U * sums.abs())
    dx, dnorm = api.rms_norm_backward(dy.to(BF), x, norm_w)
    want_dx, want_dnorm = rms_norm_backward(dy.to(BF), x, norm_w, 1e-6)
    assert float((dx.cpu().double() - want_dx).norm() / want_dx.norm()) < 2 * 2.0 ** -8
    assert float((dnorm.cpu().double() - want_dnorm).norm() / want_dnorm.norm()) < 1e-5

    # the step: one norm over all gradients; the experts' matrices as a group, the rest together
    drouter = 1e-3 * rand(EXPERTS, D)
    rest, rest_g = [norm_w, router], [dnorm, drouter]
    clip = api.grad_norm(grads + rest_g, 0.1)
    total = adamw_ref.norm(grads + rest_g)
    assert clip[0].item() == pytest.approx(total, rel=1e-6) and clip[1].item() == pytest.approx(min(1, 0.1 / total), rel=1e-6)
    before = [w.cpu().double() for w in W]
    momenta = [torch.zeros_like(w) for w in W]
    api.muon_step_batched(W, grads, momenta, 0.9, 0.01)
    for w, was, g in zip(W, before, grads):
        step = oracle.newton_schulz(g.cpu().double().numpy(), 5)
        moved = torch.from_numpy(step) * 0.01
        assert float((was - w.cpu().double() - moved).norm()) <= 1e-4 * float(moved.norm()) + 1e-6 * float(was.norm())
    was = [t.cpu().double() for t in rest]
    M, V, SM, SV = api.adamw_states(rest, 8)
    api.adamw_step(rest, rest_g, M, V, 0.01, 1, SM=SM, SV=SV, factor=clip[1:])
    for t, w, g in zip(rest, was, rest_g):
        (want, err), _, _ = adamw_ref.step(w, g.cpu().double(), 0 * w, 0 * w, 0.01, 1, (0.9, 0.999), 1e-8, 0.01, float(clip[1]))
        close(t, want, err)
