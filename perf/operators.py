"""Measured cases of the 8-bit layer operators: the quantisation of a matrix to e4m3 codes with a
scale for each block of 128, the matrix product of such operands, the RMS norm with the residual's
addition and 8-bit output, and the norm's gradient.

`run` computes them in plain torch operations in 32 bits, or, with `own` set, calls the package."""

import math

import torch

own = False

BLOCK = 128
TOP = 448.0          # largest e4m3 value
LEAST = 2.0 ** -126  # smallest scale
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCALES = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}


def listed():
    return [
        # one token through an MLP's first product while serving: the weight's bytes and the latency count
        dict(name="matmul one token", op="matmul", m=1, n=8192, k=2048, scale="f32", rows_b=False, out="bf16", add=False),
        # a small batch of tokens through the second product of the MLP, residual added
        dict(name="matmul few tokens", op="matmul", m=24, n=2048, k=8192, scale="e8m0", rows_b=False, out="bf16", add=True),
        # sizes that divide by nothing
        dict(name="matmul ragged", op="matmul", m=1000, n=1537, k=1111, scale="f32", rows_b=False, out="bf16", add=False),
        # forward product of the 2048-wide model's MLP on 8192 tokens
        dict(name="matmul forward", op="matmul", m=8192, n=8192, k=2048, scale="f32", rows_b=False, out="bf16", add=False),
        # its weight gradient, accumulated in fp32 over micro-batches of an odd number of tokens
        dict(name="matmul weight gradient", op="matmul", m=8192, n=2048, k=8200, scale="f32", rows_b=True, out="f32", add=True),
        # a 4096 x 4096 weight on a long batch, power-of-two scales
        dict(name="matmul long batch", op="matmul", m=16384, n=4096, k=4096, scale="e8m0", rows_b=False, out="bf16", add=False),
        # a weight just stepped by the optimizer, for the forward product and for the data gradient
        dict(name="quantize weight", op="quantize", m=4096, n=4096, block_rows=128, type="bf16", scale="f32", transposed=True),
        # an output gradient, for the data gradient (by rows) and the weight gradient (by columns)
        dict(name="quantize gradient", op="quantize", m=8191, n=2048, block_rows=1, type="bf16", scale="e8m0", transposed=True),
        # the norm before a projection for one token while serving
        dict(name="norm one token", op="norm", m=1, n=4096, type="bf16", scale="f32", residual=True, y=False),
        # the same in training: the bf16 result is kept for the weight gradient
        dict(name="norm training", op="norm", m=8192, n=4096, type="bf16", scale="f32", residual=True, y=True),
        # gradients of the norm: a short fine-tuning batch, and a training batch
        dict(name="norm gradient short", op="norm_grad", m=37, n=2048, type="bf16", residual=True),
        dict(name="norm gradient training", op="norm_grad", m=8192, n=4096, type="bf16", residual=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "quantize", "norm", "norm_grad"])
    if op == "matmul":
        most = 16384 * 4096 * 4096
        while True:
            m, n, k = _log(rng, 1, 16384), _log(rng, 100, 8192), _log(rng, 100, 8200)
            if rng.random() < 0.5:
                n, k = max(128, n // 128 * 128), max(128, k // 128 * 128)
            if m * n * k <= most:
                break
        grad = rng.random() < 0.3
        return dict(op=op, m=m, n=n, k=k, scale=rng.choice(["f32", "e8m0"]), rows_b=grad,
                    out="f32" if grad else "bf16", add=rng.random() < 0.5)
    m, n = _log(rng, 1, 8192), _log(rng, 128, 4096)
    if rng.random() < 0.5:
        n = max(128, n // 128 * 128)
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "quantize":
        return dict(op=op, m=m, n=n, block_rows=rng.choice([1, 128]), type=kind,
                    scale=rng.choice(["f32", "e8m0"]), transposed=rng.random() < 0.6)
    if op == "norm":
        return dict(op=op, m=m, n=n, type=kind, scale=rng.choice(["f32", "e8m0"]),
                    residual=rng.random() < 0.7, y=rng.random() < 0.5)
    return dict(op=op, m=m, n=n, type=kind, residual=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _up(a, b):
    return -(-a // b)


def _empty_codes(rows, cols, dev):
    """Codes whose rows start at multiples of 16 bytes."""
    return torch.empty(rows, _up(cols, 16) * 16, dtype=torch.float8_e4m3fn, device=dev)[:, :cols]


def _plain_quantize(x, block_rows, scale):
    """Codes (as values of the 8-bit type) and scales of x's blocks."""
    m, n = x.shape
    x = x.float()
    mb, nb = _up(m, block_rows), _up(n, BLOCK)
    pad = torch.zeros(mb * block_rows, nb * BLOCK, device=x.device)
    pad[:m, :n] = x
    t = pad.view(mb, block_rows, nb, BLOCK)
    a = torch.where(torch.isfinite(t), t.abs(), torch.zeros_like(t)).amax(dim=(1, 3))
    if scale == "f32":
        s = torch.clamp(a / TOP, min=LEAST)
    else:
        f, e = torch.frexp(a)  # a = f 2^e, f in [0.5, 1): 448 = 0.875 2^9
        e = torch.clamp(e - 9 + (f > 0.875).to(e.dtype), min=-126)
        s = ((e + 127) << 23).view(torch.float32)  # 2^e
    s = torch.where(a == 0, torch.ones_like(s), s)
    q = (t * (1.0 / s)[:, None, :, None]).reshape(mb * block_rows, nb * BLOCK)[:m, :n]
    return q.to(torch.float8_e4m3fn), s.to(SCALES[scale])


def _plain_values(codes, s, block_rows):
    s = s.float().repeat_interleave(BLOCK, 1)[:, :codes.size(1)]
    return codes.float() * s.repeat_interleave(block_rows, 0)[:codes.size(0)]


def _plain_norm(x, residual, w, scale, want_y):
    r = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    f = r.float()
    y = f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * w.float()
    q, s = _plain_quantize(y, 1, scale)
    return {"sum": None if residual is None else r, "y": y.to(x.dtype) if want_y else None, "q": q, "s": s}


def _plain_norm_grad(dy, x, w, dsum):
    g, f = dy.float(), x.float()
    t = torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)
    u, h = f * t, g * w.float()
    dx = t * (h - u * (h * u).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.float()
    return {"dx": dx.to(x.dtype), "dw": (g * u).sum(0, keepdim=True)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _normal(gen, rows, cols, std, kind):
    return (torch.randn(rows, cols, generator=gen, device="cuda") * std).to(TYPES[kind])


def _activations(gen, rows, cols, kind):
    """Activations: a few channels carry much larger values than the others."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    loud = torch.rand(1, cols, generator=gen, device="cuda") < 0.01
    return torch.where(loud, x * 20.0, x).to(TYPES[kind])


def _gradient(gen, rows, cols, kind):
    """Output gradients: small, and of another size from token to token."""
    size = torch.exp(torch.randn(rows, 1, generator=gen, device="cuda")) * 1e-4
    return (torch.randn(rows, cols, generator=gen, device="cuda") * size).to(TYPES[kind])


def _stored(codes):
    out = _empty_codes(codes.size(0), codes.size(1), codes.device)
    out.view(torch.uint8).copy_(codes.view(torch.uint8))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    state = {"case": c}
    if c["op"] == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        if c["rows_b"]:   # weight gradient: both operands by rows along the tokens
            a, b = _gradient(gen, k, m, "f32").t(), _activations(gen, k, n, "f32").t()
        else:
            a, b = _activations(gen, m, k, "f32"), _normal(gen, n, k, 0.02, "f32")
        br = 1 if c["rows_b"] else BLOCK
        qa, sa = _plain_quantize(a, 1, c["scale"])
        qb, sb = _plain_quantize(b, br, c["scale"])
        state.update(a=_stored(qa), sa=sa, b=_stored(qb), sb=sb,
                     c=torch.empty(m, n, dtype=TYPES[c["out"]], device="cuda"),
                     add=_normal(gen, m, n, 0.01 if c["rows_b"] else 1.0, c["out"]) if c["add"] else None)
        return state
    m, n, kind = c["m"], c["n"], c["type"]
    if c["op"] == "quantize":
        x = _normal(gen, m, n, 0.02, kind) if c["block_rows"] == BLOCK else _gradient(gen, m, n, kind)
        br = c["block_rows"]
        state.update(x=x, q=_empty_codes(m, n, "cuda"),
                     s=torch.empty(_up(m, br), _up(n, BLOCK), dtype=SCALES[c["scale"]], device="cuda"))
        state.update(qt=_empty_codes(n, m, "cuda") if c["transposed"] else None,
                     st=torch.empty(_up(n, br), _up(m, BLOCK), dtype=SCALES[c["scale"]], device="cuda") if c["transposed"] else None)
        return state
    w = 1.0 + 0.1 * torch.randn(1, n, generator=gen, device="cuda")
    x = _activations(gen, m, n, kind)
    other = None
    if c["op"] == "norm":
        if c["residual"]:
            other = _normal(gen, m, n, 1.0, kind)
        state.update(x=x, w=w, residual=other, sum=torch.empty_like(x) if c["residual"] else None,
                     y=torch.empty_like(x) if c["y"] else None, q=_empty_codes(m, n, "cuda"),
                     s=torch.empty(m, _up(n, BLOCK), dtype=SCALES[c["scale"]], device="cuda"))
        return state
    dy = _gradient(gen, m, n, kind)
    if c["residual"]:
        other = _gradient(gen, m, n, kind)
    state.update(dy=dy, x=x, w=w, dsum=other, dx=torch.empty_like(x),
                 dw=torch.empty(1, n, device="cuda"))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(state):
    c = state["case"]
    if own:
        from orthonormal_optimizer_update_amd import api
        if c["op"] == "matmul":
            if "ws" not in state:  # a program keeps its workspace
                state["ws"] = api.workspace(api.fp8_matmul_workspace_size(c["m"], c["n"], c["k"]), state["a"].device)
            api.fp8_matmul(state["a"], state["sa"], state["b"], state["sb"], state["c"], add=state["add"], ws=state["ws"])
            return state["c"]
        if c["op"] == "quantize":
            api.fp8_quantize(state["x"], state["q"], state["s"], state["qt"], state["st"], block_rows=c["block_rows"])
            return {k: state[k] for k in ("q", "s", "qt", "st")}
        if c["op"] == "norm":
            api.rms_norm_fp8(state["x"], state["w"], state["q"], state["s"], eps=EPS,
                             residual=state["residual"], sum_out=state["sum"], y_out=state["y"])
            return {k: state[k] for k in ("sum", "y", "q", "s")}
        if "ws" not in state:
            state["ws"] = api.workspace(api.rms_norm_backward_workspace_size(c["m"], c["n"]), state["x"].device)
        api.rms_norm_backward(state["dy"], state["x"], state["w"], state["dx"], state["dw"], eps=EPS,
                              dsum=state["dsum"], ws=state["ws"])
        return {"dx": state["dx"], "dw": state["dw"]}
    if c["op"] == "matmul":
        p = _plain_values(state["a"], state["sa"], 1) @ _plain_values(state["b"], state["sb"], 1 if c["rows_b"] else BLOCK).t()
        if state["add"] is not None:
            p = p + state["add"].float()
        return p.to(TYPES[c["out"]])
    if c["op"] == "quantize":
        q, s = _plain_quantize(state["x"], c["block_rows"], c["scale"])
        qt, st = _plain_quantize(state["x"].t(), c["block_rows"], c["scale"]) if c["transposed"] else (None, None)
        return {"q": q, "s": s, "qt": qt, "st": st}
    if c["op"] == "norm":
        return _plain_norm(state["x"], state["residual"], state["w"], c["scale"], c["y"])
    return _plain_norm_grad(state["dy"], state["x"], state["w"], state["dsum"])


def work(case):
    c = case
    sb = 4 if c.get("scale") == "f32" else 1
    if c["op"] == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        kb = _up(k, BLOCK)
        out = 2 if c["out"] == "bf16" else 4
        scales = sb * kb * (m + (n if c["rows_b"] else _up(n, BLOCK)))
        return {"bytes": (m + n) * k + scales + m * n * out * (2 if c["add"] else 1), "flops": 2 * m * n * k}
    m, n = c["m"], c["n"]
    e = 2 if c["type"] == "bf16" else 4
    if c["op"] == "quantize":
        br = c["block_rows"]
        one = m * n + sb * _up(m, br) * _up(n, BLOCK)
        two = m * n + sb * _up(n, br) * _up(m, BLOCK)
        return {"bytes": m * n * e + one + (two if c["transposed"] else 0), "flops": 3 * m * n * (2 if c["transposed"] else 1)}
    if c["op"] == "norm":
        each = e * (1 + 2 * c["residual"] + c["y"]) + 1
        return {"bytes": m * n * each + 4 * n + sb * m * _up(n, BLOCK), "flops": 8 * m * n}
    return {"bytes": m * n * e * (3 + c["residual"]) + 8 * n, "flops": 12 * m * n}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def _power(e):
    """2^e in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(v):
    """v to the nearest e4m3 value, ties to even, in 64 bits (|v| <= 448)."""
    _, e = torch.frexp(v)                       # |v| in [2^(e-1), 2^e)
    step = _power(torch.clamp(e - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantize(x, tall, scale):
    """Codes' values and scales, one strip of blocks after another."""
    m, n = x.shape
    q, s = torch.empty_like(x), []
    for j in range(0, n, BLOCK):
        strip = x[:, j:j + BLOCK]
        top = strip.abs().amax(1)
        if tall > 1:
            top = torch.stack([part.amax() for part in top.split(tall)])
        each = top / TOP
        if scale == "e8m0":
            each = _power(torch.ceil(torch.log2(torch.where(each > 0, each, torch.ones_like(each)))))
        each = torch.where(top > 0, each.clamp(min=LEAST), torch.ones_like(each))
        q[:, j:j + BLOCK] = _round_e4m3(strip / each.repeat_interleave(tall)[:m, None])
        s.append(each)
    return q, torch.stack(s, 1)


def exact(case, seed):
    c, state = case, prepare(case, seed)
    if c["op"] == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        total = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        for b, j in enumerate(range(0, k, BLOCK)):
            p = state["a"][:, j:j + BLOCK].double() * state["sa"][:, b:b + 1].double()
            sb = state["sb"][:, b].double()
            sb = sb if c["rows_b"] else sb.repeat_interleave(BLOCK)[:n]
            q = state["b"][:, j:j + BLOCK].double() * sb[:, None]
            total += p @ q.t().contiguous()
        return total if state["add"] is None else total + state["add"].double()
    x = state["x"].double()
    if c["op"] == "quantize":
        q, s = _exact_quantize(x, c["block_rows"], c["scale"])
        qt, st = _exact_quantize(x.t().contiguous(), c["block_rows"], c["scale"]) if c["transposed"] else (None, None)
        return {"q": q, "s": s, "qt": qt, "st": st}
    w, n = state["w"].double(), c["n"]
    if c["op"] == "norm":
        total = x
        if c["residual"]:  # the sum is kept in x's type, and what is kept is normalised
            total = x + state["residual"].double()
            x = total.to(TYPES[c["type"]]).double()
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / n + EPS) * w
        q, s = _exact_quantize(y, 1, c["scale"])
        return {"sum": total if c["residual"] else None, "y": y if c["y"] else None, "q": q, "s": s}
    dy = state["dy"].double()
    root = torch.sqrt((x * x).sum(1, keepdim=True) / n + EPS)
    dw = (dy * x / root).sum(0, keepdim=True)
    dx = dy * w / root - x * ((dy * w * x).sum(1, keepdim=True) / n) / root ** 3
    if state["dsum"] is not None:
        dx = dx + state["dsum"].double()
    return {"dx": dx, "dw": dw}
