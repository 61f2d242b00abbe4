"""The 8-bit operators as a training program strings them together around a
step, in HIP graphs, on several streams, and on matrices beyond 32-bit offsets."""

import numpy as np
import pytest
import torch

import fp8_ref as ref
import oracle
from orthonormal_optimizer_update_amd import api
from parity_util import TOL, note, rel, to_host
from test_gpu_fp8 import (UBF, check_codes, check_norm, check_product, codes_and_scales, group_tops, half,
                          matmul_reference, normal, upload)

pytestmark = pytest.mark.gpu

SCALES = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    api.lib()
    torch.cuda.set_device(0)


def values(q, s, block_rows):
    return ref.e4m3_values(q) * ref.expand(ref.scale_values(s), *q.shape, block_rows)


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("T,n_in,n_out", [(200, 256, 384), (1, 300, 140), (515, 192, 130)])
def test_layer_and_step(T, n_in, n_out, scale):
    """norm -> product -> its two gradients -> the norm's gradient -> Muon step
    -> the stepped weight in 8 bits; each stage against 64 bits on what the
    stages before it wrote."""
    sd = SCALES[scale]
    x, res = normal(1, T, n_in, "bf16"), normal(2, T, n_in, "bf16")
    w = 1 + 0.1 * normal(3, 1, n_in)
    W, dy = normal(4, n_out, n_in, "bf16", 0.02), normal(5, T, n_out, "bf16", 1e-3)
    dres = normal(6, T, n_in, "bf16", 1e-3)
    note(f"layer T={T} in={n_in} out={n_out} {scale}")
    tW = W.cuda()
    total, yn = torch.empty(T, n_in, dtype=torch.bfloat16, device="cuda"), None
    yn = torch.empty_like(total)
    Q, S = api.rms_norm_fp8(x.cuda(), w.cuda(), residual=res.cuda(), sum_out=total, y_out=yn, scale_dtype=sd)
    WQ, WS, WQT, WST = api.fp8_quantize(tW, block_rows=128, scale_dtype=sd, transposed=True)
    y = api.fp8_matmul(Q, S, WQ, WS)
    DQ, DS, DQT, DST = api.fp8_quantize(dy.cuda(), scale_dtype=sd, transposed=True)
    dyn = api.fp8_matmul(DQ, DS, WQT, WST)
    YQT, YST = api.fp8_codes(n_in, T, "cuda"), api.fp8_scales(n_in, T, "cuda", 1, sd)
    api.fp8_quantize(yn, QT=YQT, ST=YST)
    G = api.fp8_matmul(DQT, DST, YQT, YST)
    G32 = api.fp8_matmul(DQT, DST, YQT, YST, out_dtype=torch.float32)
    dx, dw = api.rms_norm_backward(dyn, total, w.cuda(), dsum=dres.cuda())
    M = torch.zeros(n_out, n_in, device="cuda")
    before = to_host(tW)
    api.muon_step(tW, G, M, 0.95, 0.02)
    NQ, NS, NQT, NST = api.fp8_quantize(tW, block_rows=128, scale_dtype=sd, transposed=True)
    torch.cuda.synchronize()

    check_norm(x, res, w, 1e-6, Q, S, total, yn)
    check_codes(W, WQ, WS, 128)
    check_codes(W.t().contiguous(), WQT, WST, 128)
    for got, (a, sa, bra), (b, sb, brb) in ((y, (Q, S, 1), (WQ, WS, 128)), (dyn, (DQ, DS, 1), (WQT, WST, 128)),
                                            (G, (DQT, DST, 1), (YQT, YST, 1)), (G32, (DQT, DST, 1), (YQT, YST, 1))):
        want, mags = matmul_reference(a.cpu(), sa.cpu(), bra, b.cpu(), sb.cpu(), brb)
        tops = group_tops(a.cpu(), sa.cpu(), bra, b.cpu(), sb.cpu(), brb) if got.dtype == torch.bfloat16 else None
        check_product(got, want, mags, a.size(1), None, tops)
    # the gradient against the unquantised one: each operand is off by half a
    # step of e4m3, 2^-4 of the element or, near zero, 2^-10 of the scale
    A, B = dy.t().double(), yn.cpu().t().double()
    ea = (A.abs() * 2.0 ** -4).maximum(ref.expand(ref.scale_values(DST), n_out, T, 1) * 2.0 ** -10) * 1.001
    eb = (B.abs() * 2.0 ** -4).maximum(ref.expand(ref.scale_values(YST), n_in, T, 1) * 2.0 ** -10) * 1.001
    bound = ea @ B.abs().t() + A.abs() @ eb.t() + ea @ eb.t()
    assert torch.all((G32.double().cpu() - A @ B.t()).abs() <= bound * (1 + 1e-3))
    wx, ww = ref.rms_norm_backward(dyn, total, w, 1e-6, dres)
    assert rel(to_host(dx), wx.numpy()) <= 2 * UBF and rel(to_host(dw), ww.numpy()) <= 1e-5
    step = oracle.muon_step(before, to_host(G), np.zeros((n_out, n_in)), 0.95, 0.02)
    assert rel(to_host(M), step["M"]) <= TOL["f32"]
    stepped = before + step["dX"]
    # the update carries the Newton-Schulz precision of bf16, the weight one more rounding
    assert rel(to_host(tW), stepped) <= TOL["bf16"]
    check_codes(tW.cpu(), NQ, NS, 128)
    check_codes(tW.cpu().t().contiguous(), NQT, NST, 128)


def graph_case(T, n_in, n_out, scale):
    """State of one captured sequence: inputs, outputs and workspaces."""
    sd = SCALES[scale]
    st = {
        "x": normal(1, T, n_in, "bf16").cuda(), "res": normal(2, T, n_in, "bf16").cuda(),
        "w": (1 + 0.1 * normal(3, 1, n_in)).cuda(), "W": normal(4, n_out, n_in, "bf16", 0.02).cuda(),
        "dy": normal(5, T, n_out, "bf16", 1e-3).cuda(), "acc": torch.zeros(n_out, n_in, device="cuda"),
        "Q": api.fp8_codes(T, n_in, "cuda"), "S": api.fp8_scales(T, n_in, "cuda", 1, sd),
        "WQ": api.fp8_codes(n_out, n_in, "cuda"), "WS": api.fp8_scales(n_out, n_in, "cuda", 128, sd),
        "WQT": api.fp8_codes(n_in, n_out, "cuda"), "WST": api.fp8_scales(n_in, n_out, "cuda", 128, sd),
        "DQ": api.fp8_codes(T, n_out, "cuda"), "DS": api.fp8_scales(T, n_out, "cuda", 1, sd),
        "DQT": api.fp8_codes(n_out, T, "cuda"), "DST": api.fp8_scales(n_out, T, "cuda", 1, sd),
        "YQT": api.fp8_codes(n_in, T, "cuda"), "YST": api.fp8_scales(n_in, T, "cuda", 1, sd),
        "total": torch.empty(T, n_in, dtype=torch.bfloat16, device="cuda"),
        "yn": torch.empty(T, n_in, dtype=torch.bfloat16, device="cuda"),
        "y": torch.empty(T, n_out, dtype=torch.bfloat16, device="cuda"),
        "dyn": torch.empty(T, n_in, dtype=torch.bfloat16, device="cuda"),
        "dx": torch.empty(T, n_in, dtype=torch.bfloat16, device="cuda"),
        "dw": torch.empty(1, n_in, device="cuda"),
    }
    for k, v in st.items():   # what no call writes (the codes' padding) has a value
        if v.dtype == torch.float8_e4m3fn:
            v.view(torch.uint8).zero_()
    sizes = [api.fp8_matmul_workspace_size(T, n_out, n_in), api.fp8_matmul_workspace_size(T, n_in, n_out),
             api.fp8_matmul_workspace_size(n_out, n_in, T)]
    ws = api.workspace(max(sizes), "cuda")
    ws_norm = api.workspace(api.rms_norm_backward_workspace_size(T, n_in), "cuda")

    def call(s):
        api.rms_norm_fp8(s["x"], s["w"], s["Q"], s["S"], residual=s["res"], sum_out=s["total"], y_out=s["yn"])
        api.fp8_quantize(s["W"], s["WQ"], s["WS"], s["WQT"], s["WST"], block_rows=128)
        api.fp8_matmul(s["Q"], s["S"], s["WQ"], s["WS"], s["y"], ws=ws)
        api.fp8_quantize(s["dy"], s["DQ"], s["DS"], s["DQT"], s["DST"])
        api.fp8_matmul(s["DQ"], s["DS"], s["WQT"], s["WST"], s["dyn"], ws=ws)
        api.fp8_quantize(s["yn"], QT=s["YQT"], ST=s["YST"])
        api.fp8_matmul(s["DQT"], s["DST"], s["YQT"], s["YST"], s["acc"], add=s["acc"], ws=ws)
        api.rms_norm_backward(s["dyn"], s["total"], s["w"], s["dx"], s["dw"], ws=ws_norm)

    return st, call


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("T,n_in,n_out,scale", [(7, 512, 640, "f32"), (130, 2048, 256, "e8m0"),
                                                (300, 320, 448, "f32"), (4096, 2048, 4096, "e8m0")])
def test_graph_replays_match_eager_calls(T, n_in, n_out, scale):
    """One captured sequence, replayed three times with new inputs, eager work
    and synchronisations between, bit for bit against the calls made eagerly."""
    st, call = graph_case(T, n_in, n_out, scale)
    note(f"graph T={T} in={n_in} out={n_out} {scale}")
    call({k: v.clone() for k, v in st.items()})
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(st)
    torch.cuda.synchronize()
    for i in range(3):
        st["x"].copy_(normal(10 + i, T, n_in, "bf16"))
        st["dy"].copy_(normal(20 + i, T, n_out, "bf16", 1e-3))
        eager = {k: v.clone() for k, v in st.items()}
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        call(eager)
        torch.cuda.synchronize()
        for k in st:
            assert torch.equal(bits(st[k]), bits(eager[k])), f"replay {i}: {k}"
    del graph


def test_two_streams_at_once():
    """Two sequences side by side on their own streams and workspaces."""
    cases = [graph_case(130, 2048, 256, "f32"), graph_case(300, 320, 448, "e8m0")]
    wants = []
    for st, call in cases:
        e = {k: v.clone() for k, v in st.items()}
        call(e)
        torch.cuda.synchronize()
        wants.append(e)
    note("two streams")
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for (st, call), s in zip(cases, streams):
            st["acc"].zero_()
        torch.cuda.synchronize()
        for (st, call), s in zip(cases, streams):
            with torch.cuda.stream(s):
                call(st)
        torch.cuda.synchronize()
        for (st, _), want in zip(cases, wants):
            for k in st:
                assert torch.equal(bits(st[k]), bits(want[k])), k


def test_offsets_beyond_32_bits():
    """More than 2^32 elements: the last rows come out like the same rows alone."""
    m, n = 140000, 32768
    x = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    rows = torch.cat([torch.arange(0, 3), torch.arange(65530, 65540), torch.arange(131070, 131074),
                      torch.arange(m - 5, m)]).cuda()
    part = normal(1, rows.numel(), n, "bf16").cuda()
    x[rows] = part
    note("fp8_quantize 140000 x 32768")
    Q, S, _, _ = api.fp8_quantize(x)
    q1, s1, _, _ = api.fp8_quantize(part)
    torch.cuda.synchronize()
    assert torch.equal(Q.view(torch.uint8)[rows], q1.view(torch.uint8)) and torch.equal(S[rows], s1)
    w = (1 + 0.1 * normal(2, 1, n)).cuda()
    note("rms_norm_fp8 140000 x 32768")
    y = torch.empty_like(x)
    Q2, S2 = api.rms_norm_fp8(x, w, y_out=y)
    y1 = torch.empty_like(part)
    q2, s2 = api.rms_norm_fp8(part, w, y_out=y1)
    torch.cuda.synchronize()
    assert torch.equal(Q2.view(torch.uint8)[rows], q2.view(torch.uint8))
    assert torch.equal(S2[rows], s2) and torch.equal(y[rows], y1)
    del Q2, S2, y
    b, sb = codes_and_scales(3, 96, n, 128, "f32")
    ub, usb = upload(b), sb.cuda()
    note("fp8_matmul 140000 x 96 x 32768")
    c = api.fp8_matmul(Q, S, ub, usb, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, mags = matmul_reference(q1.cpu(), s1.cpu(), 1, b, sb, 128)
    check_product(c[rows], want, mags, n)
    c = api.fp8_matmul(Q, S, ub, usb)
    torch.cuda.synchronize()
    tops = group_tops(q1.cpu(), s1.cpu(), 1, b, sb, 128)
    check_product(c[rows], want, mags, n, None, tops)


@pytest.mark.parametrize("m", [3, 100, 256])
def test_scales_at_the_ends_of_e8m0(m):
    """Byte 0 (2^-127) against byte 254 (2^127)."""
    n, k = 256, 256
    a, sa = codes_and_scales(1, m, k, 1, "e8m0")
    b, sb = codes_and_scales(2, n, k, 128, "e8m0")
    sa.view(torch.uint8)[:, 0], sb.view(torch.uint8)[:, 0] = 0, 254
    sa.view(torch.uint8)[:, 1], sb.view(torch.uint8)[:, 1] = 254, 0
    note(f"fp8_matmul e8m0 ends m={m}")
    want, mags = matmul_reference(a, sa, 1, b, sb, 128)
    for out in (torch.float32, torch.bfloat16):
        c = api.fp8_matmul(upload(a), sa.cuda(), upload(b), sb.cuda(), out_dtype=out)
        torch.cuda.synchronize()
        tops = group_tops(a, sa, 1, b, sb, 128) if out == torch.bfloat16 else None
        check_product(c, want, mags, k, None, tops)


def test_binding_refuses_mixed_devices_and_layouts():
    x = torch.zeros(4, 256, device="cuda")
    with pytest.raises(ValueError, match="expected every tensor on"):
        api.rms_norm_fp8(x, torch.ones(1, 256))
    with pytest.raises(ValueError, match="workspace"):
        q, s, _, _ = api.fp8_quantize(x)
        api.fp8_matmul(q, s, q, s, ws=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="unit stride"):
        api.fp8_quantize(x.t())
    with pytest.raises(ValueError, match="2-D"):
        api.rms_norm_fp8(x, torch.ones(256, device="cuda"))
    with pytest.raises(ValueError, match="overlap"):
        api.fp8_quantize(x[:1].expand(4, 256))
    with pytest.raises(ValueError, match="dtype"):
        api.fp8_quantize(x.half())
    with pytest.raises(api.OrthoError) as e:
        api.fp8_quantize(x, block_rows=64)
    assert e.value.status in (2, 7)
    with pytest.raises(api.OrthoError):
        api.fp8_quantize(torch.empty(0, 256, device="cuda"))


def test_more_blocks_and_rows_than_one_thread_each():
    """Sizes at which 16 threads per block, or a workgroup per 16 rows of B,
    would pass the 2^32 threads of a launch."""
    m = (1 << 28) + 131
    x = torch.arange(m, device="cuda", dtype=torch.int32).remainder_(7).sub_(3).to(torch.bfloat16)[:, None]
    Q = torch.zeros(m, 1, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    S = torch.zeros(m, 1, dtype=torch.float8_e8m0fnu, device="cuda")
    note(f"fp8_quantize {m} x 1")
    api.fp8_quantize(x, Q, S)
    torch.cuda.synchronize()
    # one element per block: rows of seven repeat, so the last ones and a sample
    # across equal the same rows alone
    part = torch.arange(7, device="cuda").sub(3).to(torch.bfloat16)[:, None]
    q1 = torch.zeros(7, 1, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s1 = torch.zeros(7, 1, dtype=torch.float8_e8m0fnu, device="cuda")
    api.fp8_quantize(part, q1, s1)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(0, m, 65521), torch.arange(m - 1000, m)]).cuda()
    for big, small in ((Q, q1), (S, s1)):
        assert torch.equal(big.view(torch.uint8)[at], small.view(torch.uint8)[at % 7])
    del x, Q, S, at
    n, k = (1 << 25) + 21, 16
    b = torch.arange(n * k, device="cuda", dtype=torch.int32).remainder_(13).sub_(6).to(torch.float8_e4m3fn).view(n, k)
    a = torch.arange(k, device="cuda").sub(8).to(torch.float8_e4m3fn)[None]
    sa = torch.ones(1, 1, device="cuda")
    sb = torch.full((-(-n // 128), 1), 2.0, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        note(f"fp8_matmul 1 x {n} x {k} {dt}")
        c = api.fp8_matmul(a, sa, b, sb, out_dtype=dt)
        torch.cuda.synchronize()
        # integers below 2^11: the products and sums are exact
        want = (b.float() * (2 * a.float())).sum(1)[None].to(dt)
        assert torch.equal(c, want)
