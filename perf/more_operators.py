"""Measured cases of the operators around the steps: AdamW over many tensors at once with the
gradients' norm and clipping, tokens sorted by expert and brought back with weights, and the
gradient of that.

`run` computes them in plain torch operations, or, with `own` set, calls the package."""

import math

import torch

own = False

BLOCK = 128
TOP = 448.0          # largest e4m3 value
LEAST = 2.0 ** -126  # smallest scale
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LR, BETAS, EPS, DECAY, STEP = 3e-4, (0.9, 0.95), 1e-8, 0.1, 1000
SEED = 20240229      # of the stochastic rounding


def listed():
    return [
        # the norms' weights of a 12-layer model: what a call costs
        dict(name="adamw norms", op="adamw", shapes="49x1x2048", type="f32", grad="f32", bits=32, clip=0.0, stochastic=False),
        # an embedding with states in 8 bits, its bf16 weights rounded stochastically, the gradients clipped
        dict(name="adamw embedding 8 bits", op="adamw", shapes="1x32768x2048", type="bf16", grad="bf16", bits=8, clip=1.0, stochastic=True),
        # sizes that divide by nothing: small layers, with gradients accumulated in fp32
        dict(name="adamw ragged", op="adamw", shapes="3x1x1,20x1x2001,7x333x1537,5x129x771", type="bf16", grad="f32", bits=8, clip=1.0, stochastic=False),
        # every matrix of the 12-layer, 2048-wide model, states in 32 bits, the gradients clipped
        dict(name="adamw model", op="adamw", shapes="48x2048x2048,12x2048x8192,12x8192x2048", type="bf16", grad="bf16", bits=32, clip=1.0, stochastic=False),
        # a decoding step's tokens
        dict(name="sort few tokens", op="sort", tokens=33, choices=8, experts=64, align=1, wide=False, dropped=0.0),
        # a training batch, each expert's rows padded to whole blocks of 128
        dict(name="sort training", op="sort", tokens=16384, choices=8, experts=128, align=128, wide=True, dropped=0.0),
        # rows at any byte, and tokens that stay out (padding of the batch)
        dict(name="gather ragged", op="gather", tokens=1023, choices=2, experts=8, align=1, n=2001, type="bf16", dropped=0.2),
        # a training batch in 8 bits on its way to the experts' products
        dict(name="gather codes training", op="gather", tokens=8192, choices=8, experts=64, align=128, n=2048, type="e4m3", dropped=0.0),
        # a decoding step's results back to its tokens, the residual added
        dict(name="combine few tokens", op="combine", tokens=16, choices=8, experts=64, align=1, n=4096, type="bf16", add=True, dropped=0.0),
        # a training batch's
        dict(name="combine training", op="combine", tokens=8192, choices=8, experts=64, align=128, n=2048, type="bf16", add=False, dropped=0.0),
        # gradients: a short fine-tuning batch in fp32, and a training batch
        dict(name="combine gradient short", op="combine_grad", tokens=37, choices=3, experts=8, align=1, n=1537, type="f32", dropped=0.1),
        dict(name="combine gradient training", op="combine_grad", tokens=8192, choices=8, experts=64, align=128, n=2048, type="bf16", dropped=0.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "sort", "gather", "combine", "combine_grad"])
    if op == "adamw":
        groups, left = [], 300_000_000
        for _ in range(rng.randint(1, 4)):
            rows, cols = rng.choice([1, _log(rng, 1, 16384)]), _log(rng, 1, 16384)
            if rng.random() < 0.5:
                cols = max(128, cols // 128 * 128)
            count = min(_log(rng, 1, 100), max(1, left // (rows * cols)))
            left -= min(left, count * rows * cols)
            groups.append("%dx%dx%d" % (count, rows, cols))
        return dict(op=op, shapes=",".join(groups), type=rng.choice(["bf16", "bf16", "f32"]), grad=rng.choice(["bf16", "f32"]),
                    bits=rng.choice([8, 32]), clip=rng.choice([0.0, 1.0]), stochastic=rng.random() < 0.5)
    experts = _log(rng, 1, 512)
    choices = min(experts, rng.choice([1, 2, 3, 4, 6, 8, 8, 16]))
    c = dict(op=op, tokens=_log(rng, 1, 16384), choices=choices, experts=experts, align=rng.choice([1, 1, 16, 128]),
             dropped=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "sort":
        return dict(c, wide=rng.random() < 0.5)
    while True:
        n = _log(rng, 64, 8192)
        if rng.random() < 0.5:
            n = max(128, n // 128 * 128)
        if (c["tokens"] * choices + experts * (c["align"] - 1)) * n <= 8192 * 8 * 2048:
            break
        c["tokens"] = max(1, c["tokens"] // 2)
    c["n"] = n
    if op == "gather":
        return dict(c, type=rng.choice(["bf16", "f32", "e4m3"]))
    c["type"] = rng.choice(["bf16", "bf16", "f32"])
    return dict(c, add=rng.random() < 0.5) if op == "combine" else c


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _up(a, b):
    return -(-a // b)


def _mix(h):
    """A 32-bit mix of shifts and products, on int64 tensors or Python integers."""
    h = ((h ^ (h >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    h = ((h ^ (h >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random_bits(rows, cols, tensor, device):
    """The random bits of a tensor's elements: 16 for the weight, 20 each for the two states."""
    key = _mix(SEED & 0xFFFFFFFF)
    for word in (SEED >> 32, STEP & 0xFFFFFFFF, STEP >> 32, tensor):
        key = _mix(key ^ _mix(word + 0x9E3779B9 & 0xFFFFFFFF))
    at = torch.arange(rows * cols, device=device)
    high = at >> 32
    a = _mix((at & 0xFFFFFFFF) ^ (key + high * 0x9E3779B9 & 0xFFFFFFFF))
    b = _mix(a + 0x9E3779B9 & 0xFFFFFFFF)
    shape = (rows, cols)
    return ((a & 0xFFF) << 4 | (b & 15)).view(shape), (a >> 12).view(shape), (b >> 12).view(shape)


def _cut(x, keep_from, bits):
    """|x|'s fp32 bits with random bits below bit `keep_from` added, cut there, and x's sign."""
    low = (1 << keep_from) - 1
    u = (x.abs().view(torch.int32).long() + bits) & ~low
    return torch.copysign(u.int().view(torch.float32), x)


def _to_weight(x, kind, bits):
    if kind == "bf16" and bits is not None:
        return _cut(x, 16, bits).to(torch.bfloat16)
    return x.to(TYPES[kind])


def _to_codes(x, bits, least):
    """Codes and scales of x (rows x cols) by blocks of 1 x 128; `least`: no positive value becomes 0."""
    rows, cols = x.shape
    pad = torch.zeros(rows, _up(cols, BLOCK) * BLOCK, device=x.device)
    pad[:, :cols] = x
    top = pad.view(rows, -1, BLOCK).abs().amax(2)
    s = torch.where(top == 0, torch.ones_like(top), torch.clamp(top / TOP, min=LEAST))
    q = x * (1.0 / s).repeat_interleave(BLOCK, 1)[:, :cols]
    if bits is not None:
        q = q.clamp(-TOP, TOP)
        small = q.abs() < 2.0 ** -6  # steps of 2^-9 from here down
        shift = torch.where(small, 2.0 ** -6, 0.0)
        q = torch.copysign(_cut(q.abs() + shift, 20, bits) - shift, q)
    if least:
        q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn), s


def _of_codes(q, s):
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :q.size(1)]


def _plain_step(x, g, m, v, factor):
    """x' before its rounding, m', v' (fp32)."""
    b1, b2 = BETAS
    g = g.float()
    if factor is not None:
        g = g * factor
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * (g * g)
    down = torch.sqrt(v) / math.sqrt(1.0 - b2 ** STEP) + EPS
    return (1.0 - LR * DECAY) * x.float() - LR / (1.0 - b1 ** STEP) * (m / down), m, v


def _plain_norm(g, most):
    norm = g.double().square().sum().sqrt()
    return torch.stack([norm, torch.where(norm > most, most / norm, torch.ones_like(norm))]).float()


def _plain_adamw(state):
    c = state["case"]
    out = _plain_norm(state["g"], c["clip"]) if c["clip"] else None
    factor = out[1] if c["clip"] else None
    if c["bits"] == 32 and not (c["stochastic"] and c["type"] == "bf16"):   # the tensors lie behind one another
        x, m, v = _plain_step(state["x"], state["g"], state["m"], state["v"], factor)
        state["x"].copy_(x)
        state["m"].copy_(m)
        state["v"].copy_(v)
        return out
    for i, (x, g, m, v) in enumerate(zip(state["xs"], state["gs"], state["ms"], state["vs"])):
        bits = _random_bits(x.size(0), x.size(1), i, x.device) if c["stochastic"] else (None, None, None)
        if c["bits"] == 8:
            sm, sv = state["sms"][i], state["svs"][i]
            xn, mn, vn = _plain_step(x, g, _of_codes(m, sm), _of_codes(v, sv).square(), factor)
            for to, s, value, r, least in ((m, sm, mn, bits[1], False), (v, sv, torch.sqrt(vn), bits[2], True)):
                q, sn = _to_codes(value, r, least)
                to.copy_(q)
                s.copy_(sn)
        else:
            xn, mn, vn = _plain_step(x, g, m, v, factor)
            m.copy_(mn)
            v.copy_(vn)
        x.copy_(_to_weight(xn, c["type"], bits[0]))
    return out


def _rows(c):
    return c["tokens"] * c["choices"] + c["experts"] * (c["align"] - 1)


def _plain_sort(chosen, c):
    pairs, e = c["tokens"] * c["choices"], c["experts"]
    ids = chosen.reshape(-1).long()
    ids = torch.where((ids >= 0) & (ids < e), ids, torch.full_like(ids, e))
    by, order = torch.sort(ids, stable=True)
    count = torch.zeros(e + 1, dtype=torch.long, device=ids.device).scatter_add_(0, ids, torch.ones_like(ids))
    padded = (count[:e] + c["align"] - 1) // c["align"] * c["align"]
    ends, padded_ends = torch.cumsum(count, 0), torch.cumsum(padded, 0)
    begins = torch.cat([padded_ends - padded, padded_ends[-1:]])
    place = torch.arange(pairs, device=ids.device) - (ends - count)[by] + begins[by]
    place = torch.where(by < e, place, torch.full_like(place, _rows(c)))   # (a place behind the last for those that stay out)
    slot = torch.empty_like(ids)
    slot[order] = torch.where(by < e, place, torch.full_like(place, -1))
    source = torch.full((_rows(c) + 1,), -1, dtype=torch.long, device=ids.device)
    source[place] = order
    return {"slot": slot.int().view(c["tokens"], c["choices"]), "source": source[:-1].int(), "offsets": begins.int(),
            "counts": count[:e].int()}


def _plain_gather(x, source, choices):
    y = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    y = torch.where((source < 0)[:, None], torch.zeros((), dtype=y.dtype, device=y.device), y[source.clamp(min=0).long() // choices])
    return y.view(x.dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _shapes(text):
    for part in text.split(","):
        count, rows, cols = (int(v) for v in part.split("x"))
        for _ in range(count):
            yield rows, cols


def _views(shapes, dtype, value=None):
    """A buffer of zeros and its tensors, each from a multiple of 256 elements on."""
    at, total = [], 0
    for rows, cols in shapes:
        at.append(total)
        total += _up(rows * cols, 256) * 256
    flat = torch.zeros(total, dtype=dtype, device="cuda")
    return flat, [flat[a:a + r * k].view(r, k) for a, (r, k) in zip(at, shapes)]


def _fill(gen, views, std, spread):
    """Normal values whose size differs from row to row."""
    for t in views:
        r = torch.randn(t.shape, generator=gen, device="cuda")
        if spread:
            r *= torch.exp(0.5 * torch.randn(t.size(0), 1, generator=gen, device="cuda"))
        t.copy_(r * std)


def _prepare_adamw(c, gen):
    shapes = list(_shapes(c["shapes"]))
    state = {"case": c}
    state["x"], state["xs"] = _views(shapes, TYPES[c["type"]])
    state["g"], state["gs"] = _views(shapes, TYPES[c["grad"]])
    _fill(gen, state["xs"], 0.02, False)
    _fill(gen, state["gs"], 1e-3, True)
    m, ms = _views(shapes, torch.float32)
    v, vs = _views(shapes, torch.float32)
    _fill(gen, ms, 3e-4, True)
    _fill(gen, vs, 1e-3, True)
    v.abs_().add_(1e-5)
    if c["bits"] == 32:
        state.update(m=m, ms=ms, v=v.square_(), vs=vs)
        return state
    blocks = [(rows, _up(cols, BLOCK)) for rows, cols in shapes]
    for name, values in (("m", ms), ("v", vs)):
        codes, state[name + "s"] = _views(shapes, torch.float8_e4m3fn)
        scales, state["s" + name + "s"] = _views(blocks, torch.float32)
        state.update({name: codes, "s" + name: scales})
        for value, q, s in zip(values, state[name + "s"], state["s" + name + "s"]):
            qn, sn = _to_codes(value, None, name == "v")
            q.copy_(qn)
            s.copy_(sn)
    return state


def _chosen(c, gen):
    """Experts of each token, all different, some more popular than others; tokens that stay out have -1."""
    liked = 0.7 * torch.randn(c["experts"], generator=gen, device="cuda")
    score = liked + torch.randn(c["tokens"], c["experts"], generator=gen, device="cuda")
    weight, chosen = torch.topk(score, c["choices"], dim=1)
    out = torch.rand(c["tokens"], 1, generator=gen, device="cuda") < c["dropped"]
    return torch.where(out, torch.full_like(chosen, -1), chosen), torch.softmax(weight, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    if c["op"] == "adamw":
        return _prepare_adamw(c, gen)
    chosen, weights = _chosen(c, gen)
    state = {"case": c}
    if c["op"] == "sort":
        chosen = chosen if c["wide"] else chosen.int()
        state.update(chosen=chosen, slot=torch.empty(c["tokens"], c["choices"], dtype=torch.int32, device="cuda"),
                     source=torch.empty(_rows(c), dtype=torch.int32, device="cuda"),
                     offsets=torch.empty(c["experts"] + 1, dtype=torch.int32, device="cuda"),
                     counts=torch.empty(c["experts"], dtype=torch.int32, device="cuda"))
        return state
    state.update(_plain_sort(chosen, c))
    tokens, rows, n = c["tokens"], _rows(c), c["n"]

    def normal(count):
        return torch.randn(count, n, generator=gen, device="cuda")

    if c["op"] == "gather":
        x = normal(tokens)
        if c["type"] == "e4m3":
            x, s = _to_codes(x, None, False)
            state.update(s=s, sy=torch.zeros(rows, s.size(1), device="cuda"))
            state["y"] = torch.zeros(rows, n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        else:
            x = x.to(TYPES[c["type"]])
            state["y"] = torch.zeros(rows, n, dtype=x.dtype, device="cuda")
        return dict(state, x=x)
    kind = TYPES[c["type"]]
    state.update(weights=weights, y=torch.where((state["source"] < 0)[:, None], torch.zeros((), device="cuda"), normal(rows)).to(kind))
    if c["op"] == "combine":
        state.update(add=normal(tokens).to(kind) if c["add"] else None, out=torch.empty(tokens, n, dtype=kind, device="cuda"))
    else:
        state.update(dout=(1e-3 * normal(tokens)).to(kind), dy=torch.zeros(rows, n, dtype=kind, device="cuda"),
                     dw=torch.empty(tokens, c["choices"], device="cuda"))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _own_adamw(state, api):
    c = state["case"]
    if "mats" not in state:  # a program keeps its parameters' and states' descriptors, and the workspace
        lists = {k: api.mats(state[k]) for k in ("xs", "ms", "vs", "sms", "svs") if k in state}
        state["mats"] = lists
        state["out"] = torch.empty(2, device="cuda")
        state["ws"] = api.workspace(api.grad_norm_workspace_size(len(state["gs"])), state["x"].device)
    lists, grads = state["mats"], api.mats(state["gs"])
    out = None
    if c["clip"]:
        out = api.grad_norm(grads, c["clip"], out=state["out"], ws=state["ws"])
    api.adamw_step(lists["xs"], grads, lists["ms"], lists["vs"], LR, STEP, betas=BETAS, eps=EPS, weight_decay=DECAY,
                   SM=lists.get("sms"), SV=lists.get("svs"), seed=SEED if c["stochastic"] else None,
                   factor=out[1:] if c["clip"] else None)
    return out


def run(state):
    c = state["case"]
    if own:
        from orthonormal_optimizer_update_amd import api
    if c["op"] == "adamw":
        if own:
            out = _own_adamw(state, api)
        else:
            out = _plain_adamw(state)
        return {"norm": out, **{k: state.get(k) for k in ("x", "m", "v", "sm", "sv")}}
    if c["op"] == "sort":
        if not own:
            return _plain_sort(state["chosen"], c)
        if "ws" not in state:
            state["ws"] = api.workspace(api.expert_sort_workspace_size(c["tokens"], c["choices"], c["experts"]), state["chosen"].device)
        api.expert_sort(state["chosen"], c["experts"], c["align"], state["slot"], state["source"], state["offsets"], state["counts"],
                        ws=state["ws"])
        return {k: state[k] for k in ("slot", "source", "offsets", "counts")}
    slot, source, k = state["slot"], state["source"], c["choices"]
    if c["op"] == "gather":
        if own:
            api.expert_gather(state["x"], slot, state["offsets"], state["counts"], state["y"], S=state.get("s"), SY=state.get("sy"))
            return {"y": state["y"], "s": state.get("sy")}
        s = None
        if c["type"] == "e4m3":  # (rows of padding: zeros with a scale of 1; behind the last expert's: as they were)
            pad = (source < 0) & (torch.arange(source.numel(), device=source.device) < state["offsets"][-1])
            s = _plain_gather(state["s"], source, k) + pad[:, None].float()
        return {"y": _plain_gather(state["x"], source, k), "s": s}
    if c["op"] == "combine":
        if own:
            return api.expert_combine(state["y"], slot, state["weights"], add=state["add"], out=state["out"])
        w = torch.where(slot >= 0, state["weights"], torch.zeros((), device=slot.device))
        out = (state["y"][slot.clamp(min=0).long()].float() * w[:, :, None]).sum(1)
        if state["add"] is not None:
            out = out + state["add"].float()
        return out.to(TYPES[c["type"]])
    if own:
        dy, dw = api.expert_combine_backward(state["dout"], slot, state["weights"], state["offsets"], state["counts"], state["dy"],
                                             Y=state["y"], dW=state["dw"])
        return {"dy": dy, "dw": dw}
    valid, pair = slot >= 0, source.clamp(min=0).long()
    dout = state["dout"].float()
    dw = (state["y"][slot.clamp(min=0).long()].float() * dout[:, None, :]).sum(2)
    w = torch.where(source >= 0, state["weights"].reshape(-1)[pair], torch.zeros((), device=slot.device))
    return {"dy": (dout[pair // k] * w[:, None]).to(TYPES[c["type"]]), "dw": torch.where(valid, dw, torch.zeros_like(dw))}


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if c["op"] == "adamw":
        count = sum(r * k for r, k in _shapes(c["shapes"]))
        blocks = sum(r * _up(k, BLOCK) for r, k in _shapes(c["shapes"]))
        states = 16 * count if c["bits"] == 32 else 4 * count + 16 * blocks
        return {"bytes": count * (2 * size[c["type"]] + size[c["grad"]]) + states, "flops": (17 if c["clip"] else 15) * count}
    pairs, rows = c["tokens"] * c["choices"], _rows(c)
    if c["op"] == "sort":
        return {"bytes": pairs * (12 if c["wide"] else 8) + 4 * rows + 8 * c["experts"], "flops": pairs}
    n = c["n"]
    e = size[c["type"]]
    used = pairs * (1 - c["dropped"])
    if c["op"] == "gather":
        row = n * e + (4 * _up(n, BLOCK) if e == 1 else 0)
        return {"bytes": (c["tokens"] + used) * row + 4 * pairs, "flops": 0}
    if c["op"] == "combine":
        return {"bytes": (used + c["tokens"] * (2 if c["add"] else 1)) * n * e + 8 * pairs, "flops": 2 * used * n}
    return {"bytes": (2 * used + c["tokens"]) * n * e + 12 * pairs, "flops": 3 * used * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _power(e):
    """2^e in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(v, bits):
    """v (|v| <= 448) to e4m3 in 64 bits: nearest, ties to even, or down with the chance that its random bits give."""
    _, e = torch.frexp(v)
    step = _power(torch.clamp(e - 1, min=-6) - 3)
    if bits is None:
        return torch.round(v / step) * step
    return torch.sign(v) * torch.floor(v.abs() / step + bits.double() / 2 ** 20) * step


def _exact_codes(x, bits, least):
    rows, cols = x.shape
    q, s = torch.empty_like(x), torch.empty(rows, _up(cols, BLOCK), dtype=x.dtype, device=x.device)
    whole = cols // BLOCK * BLOCK
    for first, last in ((0, whole), (whole, cols)):
        if first == last:
            continue
        part = x[:, first:last].reshape(rows, -1, min(BLOCK, last - first))
        top = part.abs().amax(2, keepdim=True)
        each = torch.where(top > 0, (top / TOP).clamp(min=LEAST), torch.ones_like(top))
        r = None if bits is None else bits[:, first:last].reshape(part.shape)
        code = _round_e4m3((part / each).clamp(-TOP, TOP), r)
        if least:
            code = torch.where(part > 0, code.clamp(min=2.0 ** -9), code)
        q[:, first:last] = code.reshape(rows, -1)
        s[:, first // BLOCK:_up(last, BLOCK)] = each[:, :, 0]
    return q, s


def _exact_adamw(c, state):
    b1, b2 = BETAS
    factor, norm = 1.0, None
    if c["clip"]:
        total = sum(float((g.double() ** 2).sum()) for g in state["g"].split(1 << 26))
        length = math.sqrt(total)
        factor = min(1.0, c["clip"] / length)
        norm = torch.tensor([length, factor], dtype=torch.float64, device="cuda")
    out = {k: torch.zeros(state[k].shape, dtype=torch.float64, device="cuda") for k in ("x", "m", "v", "sm", "sv") if k in state}
    at = scales_at = 0
    for i, x in enumerate(state["xs"]):
        rows, cols = x.shape
        here = slice(at, at + rows * cols)
        at += _up(rows * cols, 256) * 256
        g = state["gs"][i].double() * factor
        m, v = state["ms"][i].double(), state["vs"][i].double()
        if c["bits"] == 8:
            m = m * state["sms"][i].double().repeat_interleave(BLOCK, 1)[:, :cols]
            v = (v * state["svs"][i].double().repeat_interleave(BLOCK, 1)[:, :cols]) ** 2
        m = m + (1 - b1) * (g - m)
        v = v + (1 - b2) * (g * g - v)
        x = x.double() - LR * DECAY * x.double()
        x = x - LR * (m / (1 - b1 ** STEP)) / ((v / (1 - b2 ** STEP)) ** 0.5 + EPS)
        bits = _random_bits(rows, cols, i, x.device) if c["stochastic"] else (None, None, None)
        if c["type"] == "bf16" and bits[0] is not None:
            _, e = torch.frexp(x)
            step = _power(e - 8)
            x = torch.sign(x) * torch.floor(x.abs() / step + bits[0].double() / 2 ** 16) * step
        out["x"][here] = x.view(-1)
        if c["bits"] == 32:
            out["m"][here], out["v"][here] = m.view(-1), v.view(-1)
            continue
        blocks = rows * _up(cols, BLOCK)
        there = slice(scales_at, scales_at + blocks)
        scales_at += _up(blocks, 256) * 256
        for name, value, r in (("m", m, bits[1]), ("v", v.sqrt(), bits[2])):
            q, s = _exact_codes(value, r, name == "v")
            out[name][here], out["s" + name][there] = q.view(-1), s.view(-1)
    return {"norm": norm, **{k: out.get(k) for k in ("x", "m", "v", "sm", "sv")}}


def exact(case, seed):
    c, state = case, prepare(case, seed)
    if c["op"] == "adamw":
        return _exact_adamw(c, state)
    if c["op"] == "sort":
        return None
    slot, k = state["slot"].long(), c["choices"]
    if c["op"] == "gather":
        x = state["x"].double()
        y = torch.zeros(_rows(c) + 1, c["n"], dtype=torch.float64, device="cuda")
        s = None
        if "s" in state:
            s = torch.zeros(_rows(c) + 1, state["s"].size(1), dtype=torch.float64, device="cuda")
            s[:int(state["offsets"][-1])] = 1.0
        for j in range(k):
            y[slot[:, j]] = x   # (those that stay out go to the row behind the last)
            if s is not None:
                s[slot[:, j]] = state["s"].double()
        return {"y": y[:-1], "s": None if s is None else s[:-1]}
    w = state["weights"].double() * (slot >= 0)
    if c["op"] == "combine":
        out = torch.zeros(c["tokens"], c["n"], dtype=torch.float64, device="cuda")
        if state["add"] is not None:
            out += state["add"].double()
        for j in range(k):
            out += w[:, j:j + 1] * state["y"].double()[slot[:, j]]
        return out
    dout = state["dout"].double()
    dy = torch.zeros(_rows(c) + 1, c["n"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(c["tokens"], k, dtype=torch.float64, device="cuda")
    for j in range(k):
        dy[slot[:, j]] = w[:, j:j + 1] * dout
        dw[:, j] = (dout * state["y"][slot[:, j]].double()).sum(1) * (slot[:, j] >= 0)
    return {"dy": dy[:-1], "dw": dw}
