"""Workloads of the operators around a layer's products: the RMS norm with its
residual (its gradients, and its output in 8 bits), rows quantized to 8 bits,
the int8 product with a scale for each token and channel, and the routing of
tokens to experts.

`listed()` names the cases, `draw(rng)` gives more of the same ranges,
`prepare(case, seed)` makes a case's inputs on the GPU, `run(state)` is one
call of the operator (`own` true: this library's; false: elementary torch
operations in 32 bits, rounded once), `exact(case, seed)` the 64-bit value by
definition and `work(case)` the bytes and operations that a call cannot avoid.
Rows in 8 bits come back as the values they stand for, in the input's type.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # A training step's norm of the summed stream, forward and backward.
        dict(name="norm_train_bf16", op="norm", dtype="bf16", R=8192, K=4096, residual=True, wide=False),
        # A width that is no multiple of anything, fp32 weights, the stream as it is.
        dict(name="norm_odd_f16", op="norm", dtype="f16", R=1021, K=1003, residual=False, wide=True),
        # One decoded token: stream summed, normalized and quantized for the next int8 product.
        dict(name="norm_i8_token_bf16", op="norm_i8", dtype="bf16", R=1, K=4096, residual=True, wide=False),
        # A long prompt on the way into the int8 products.
        dict(name="norm_i8_prompt_bf16", op="norm_i8", dtype="bf16", R=4096, K=8192, residual=True, wide=False),
        # The activations of a decode batch before the down projection.
        dict(name="rows_batch_f16", op="rows", dtype="f16", R=16, K=14336),
        # The same of a prompt.
        dict(name="rows_prompt_bf16", op="rows", dtype="bf16", R=4096, K=14336),
        # One token through one projection.
        dict(name="i8_token_bf16", op="i8", out="bf16", M=1, N=4096, K=4096, bias=False),
        # A decode batch through a large projection with a bias.
        dict(name="i8_batch_f16", op="i8", out="f16", M=16, N=8192, K=8192, bias=True),
        # Sizes that no tile divides and rows that start at any byte.
        dict(name="i8_odd_bf16", op="i8", out="bf16", M=777, N=1003, K=2005, bias=True),
        # A prompt through the up projection.
        dict(name="i8_prompt_bf16", op="i8", out="bf16", M=4096, N=14336, K=4096, bias=False),
        # A decode batch's choices: softmax over the experts' logits.
        dict(name="route_batch_f32", op="route", dtype="f32", R=16, E=64, top=6, score="softmax", bias=False,
             groups=1, top_groups=1, best=1, renorm=True, grad=False),
        # A training batch: sigmoid scores, a balancing bias, the best 4 of 8 groups, and the gradient.
        dict(name="route_train_bf16", op="route", dtype="bf16", R=16384, E=256, top=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, best=2, renorm=True, grad=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_i8", "rows", "i8", "i8", "route", "route"))
    if op in ("norm", "norm_i8", "rows"):
        # (a row of one value has a gradient of zeros but for eps: nothing to compare)
        K = _log_int(rng, 16 if op == "norm" else 1, 16384) if rng.random() < 0.5 else 8 * _log_int(rng, 8, 2048)
        R = _log_int(rng, 1, min(16384, 8192 * 4096 // K))
        case = dict(op=op, dtype=rng.choice(("f16", "bf16")), R=R, K=K)
        if op != "rows":
            case.update(residual=rng.random() < 0.5, wide=rng.random() < 0.5)
        return case
    if op == "i8":
        odd = rng.random() < 0.25
        K = _log_int(rng, 1, 4096) if odd else 16 * _log_int(rng, 4, 896)
        N = _log_int(rng, 1, 14336)
        M = _log_int(rng, 1, min(2048 if odd else 8192, 4096 * 14336 * 4096 // (N * K)))
        return dict(op=op, out=rng.choice(("f16", "bf16", "f32")), M=M, N=N, K=K, bias=rng.random() < 0.5)
    groups = rng.choice((1, 1, 2, 4, 8, 16))
    E = groups * _log_int(rng, 2, 512 // groups)
    top_groups = rng.randrange(1, groups + 1)
    renorm, grad = rng.random() < 0.6, rng.random() < 0.5
    # (one renormalized weight is always 1, with a gradient of zeros)
    top = _log_int(rng, 2 if renorm and grad else 1, min(16, top_groups * (E // groups)))
    return dict(op=op, dtype=rng.choice(("f16", "bf16", "f32")), R=_log_int(rng, 1, 16384 * 256 // E), E=E, top=top,
                score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups,
                top_groups=top_groups, best=rng.choice((1, 2)), renorm=renorm, grad=grad)


# ---------------------------------------------------------------- inputs

def _randn(gen, shape, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)


def _stream(gen, R, K, dt):
    """Activations: normal values, and one channel in 200 that is several times larger."""
    loud = 1 + 6 * (torch.rand(K, generator=gen, device="cuda") < 0.005).float()
    return (_randn(gen, (R, K)) * loud).to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if s["op"] in ("norm", "norm_i8", "rows"):
        dt, R, K = DTYPES[s["dtype"]], s["R"], s["K"]
        s["x"] = _stream(gen, R, K, dt)
        if s["op"] == "rows":
            return s
        s["r"] = _stream(gen, R, K, dt) if s["residual"] else None
        s["w"] = (1 + _randn(gen, K, 0.1)).to(torch.float32 if s["wide"] else dt)
        if s["op"] == "norm":
            s["dy"] = _randn(gen, (R, K), 0.1).to(dt)
            s["dh"] = _randn(gen, (R, K), 0.1).to(dt) if s["residual"] else None
            for name in ("x", "r", "w"):
                if s[name] is not None:
                    s[name].requires_grad_()
        return s
    if s["op"] == "i8":
        M, N, K = s["M"], s["N"], s["K"]
        s["x"] = _randn(gen, (M, K), 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["w"] = _randn(gen, (N, K), 36.0).round_().clamp_(-127, 127).to(torch.int8)
        s["sx"] = (0.02 + 0.03 * torch.rand(M, generator=gen, device="cuda"))
        s["sw"] = (0.5 + torch.rand(N, generator=gen, device="cuda")) * (0.03 * K ** -0.5)
        s["b"] = _randn(gen, N, 0.2).to(DTYPES[s["out"]]) if s["bias"] else None
        return s
    R, E = s["R"], s["E"]
    s["logits"] = (_randn(gen, (R, E)) + _randn(gen, E, 0.5)).to(DTYPES[s["dtype"]])
    s["b"] = _randn(gen, E, 0.02) if s["bias"] else None
    if s["grad"]:
        s["dw"] = _randn(gen, (R, s["top"]))
        s["logits"].requires_grad_()
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _values(q, scale, dt):
    """Rows in 8 bits as the values they stand for."""
    return torch.mul(q, scale[:, None], out=torch.empty(q.shape, dtype=dt, device=q.device))


def _own(s):
    if s["op"] == "norm":
        from dense_tiled_gemm_02_amd import norm
        if s["r"] is None:
            y = norm.rms_norm(s["x"], s["w"], eps=EPS)
            return (y.detach(),) + torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
        y, h = norm.rms_norm(s["x"], s["w"], s["r"], eps=EPS)
        dx, dr, dw = torch.autograd.grad((y, h), (s["x"], s["r"], s["w"]), (s["dy"], s["dh"]))
        return y.detach(), h.detach(), dx, dr, dw
    if s["op"] == "norm_i8":
        from dense_tiled_gemm_02_amd import norm
        q, scale, *h = norm.rms_norm_i8(s["x"], s["w"], s["r"], eps=EPS)
        return (_values(q, scale, s["x"].dtype), scale, *h)
    if s["op"] == "rows":
        from dense_tiled_gemm_02_amd import i8
        q, scale = i8.i8_quantize(s["x"])
        return _values(q, scale, s["x"].dtype), scale
    if s["op"] == "i8":
        from dense_tiled_gemm_02_amd import i8
        return i8.i8_matmul(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"], out_dtype=DTYPES[s["out"]])
    from dense_tiled_gemm_02_amd import router
    w, ids = router.route(s["logits"], s["top"], score=s["score"], bias=s["b"], groups=s["groups"],
                          top_groups=s["top_groups"], group_best=s["best"], renormalize=s["renorm"], scale=2.5)
    if not s["grad"]:
        return w, ids
    return w.detach(), ids, torch.autograd.grad(w, s["logits"], s["dw"])[0]


def _plain(s):
    with torch.no_grad():
        if s["op"] == "norm":
            return _plain_norm(s)
        if s["op"] == "norm_i8":
            h, rstd = _plain_stream(s)
            q, scale = _plain_rows(h.float() * rstd * s["w"].float())
            return (_values(q, scale, h.dtype), scale) + (() if s["r"] is None else (h,))
        if s["op"] == "rows":
            q, scale = _plain_rows(s["x"].float())
            return _values(q, scale, s["x"].dtype), scale
        if s["op"] == "i8":
            y = (s["x"].float() @ s["w"].float().t()) * s["sx"][:, None] * s["sw"]
            if s["b"] is not None:
                y += s["b"].float()
            return y.to(DTYPES[s["out"]])
        return _plain_route(s)


def _plain_stream(s):
    """The summed stream, held in the stream's type, and the reciprocal of its root mean square."""
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    return h, torch.rsqrt(h.float().square().mean(1, keepdim=True) + EPS)


def _plain_rows(v):
    scale = v.abs().amax(1) / 127
    q = torch.where(scale[:, None] > 0, v / scale[:, None], 0.0).round().clamp(-127, 127).to(torch.int8)
    return q, scale


def _plain_norm(s):
    h, rstd = _plain_stream(s)
    w, dy = s["w"].float(), s["dy"].float()
    unit = h.float() * rstd
    y = (unit * w).to(h.dtype)
    g = dy * w
    dx = (g - unit * (g * unit).mean(1, keepdim=True)) * rstd
    dw = (dy * unit).sum(0).to(s["w"].dtype)
    if s["r"] is None:
        return y, dx.to(h.dtype), dw
    dx = (dx + s["dh"].float()).to(h.dtype)
    return y, h, dx, dx, dw


def _plain_route(s):
    R, E, top, G = s["R"], s["E"], s["top"], s["groups"]
    l = s["logits"].float()
    # which score is larger is a border: 64 bits; without a bias the logits have the scores' order
    score = torch.softmax(l.double(), 1) if s["score"] == "softmax" else torch.sigmoid(l.double())
    choice = l.double() if s["b"] is None else score + s["b"].double()
    if G > 1:
        of_group = choice if s["best"] == 1 or s["b"] is not None else score
        best = of_group.view(R, G, E // G).sort(dim=-1, descending=True).values[..., :s["best"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :s["top_groups"]]
        inside = torch.zeros(R, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        choice = choice.masked_fill(~inside.repeat_interleave(E // G, 1), -math.inf)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :top]
    score = score.float()
    p = score.gather(1, ids)
    w = p / p.sum(1, keepdim=True) if s["renorm"] else p
    if not s["grad"]:
        return w * 2.5, ids.int()
    dw = s["dw"] * 2.5
    if s["renorm"]:
        dp = (dw - (dw * w).sum(1, keepdim=True)) / p.sum(1, keepdim=True)
    else:
        dp = dw
    if s["score"] == "sigmoid":
        dl = torch.zeros_like(l).scatter_(1, ids, dp * p * (1 - p))
    else:
        dl = torch.zeros_like(l).scatter_(1, ids, dp * p) - score * (dp * p).sum(1, keepdim=True)
        if s["renorm"]:   # the sum over the chosen is zero: the others' gradients are zeros
            dl = torch.zeros_like(l).scatter_(1, ids, dp * p)
    return w * 2.5, ids.int(), dl.to(s["logits"].dtype)


# ---------------------------------------------------------------- by definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if s["op"] == "i8":
            acc = torch.matmul(s["x"].to(torch.float64), s["w"].to(torch.float64).t().contiguous())
            acc *= torch.outer(s["sx"].to(torch.float64), s["sw"].to(torch.float64))
            return acc if s["b"] is None else acc + s["b"].to(torch.float64)
        if s["op"] == "route":
            return _exact_route(s)
        if s["op"] == "rows":
            return _exact_rows(s["x"].to(torch.float64))
        K = s["K"]
        total = s["x"].to(torch.float64)
        if s["r"] is not None:
            total = total + s["r"].to(torch.float64)
        h = total.to(s["x"].dtype).to(torch.float64)   # the stream is held in its type
        w = s["w"].to(torch.float64)
        length = torch.sqrt((h * h).sum(1) / K + EPS)
        y = h / length[:, None] * w
        if s["op"] == "norm_i8":
            return _exact_rows(y) + (() if s["r"] is None else (total,))
        dy = s["dy"].to(torch.float64)
        # y_i = h_i w_i / n, n = sqrt(sum h^2 / K + eps): dn/dh_i = h_i / (K n)
        along = (dy * w * h).sum(1) / (K * length ** 3)
        dx = dy * w / length[:, None] - h * along[:, None]
        dw = (dy * h / length[:, None]).sum(0)
        if s["r"] is None:
            return y, dx, dw
        dx = dx + s["dh"].to(torch.float64)
        return y, total, dx, dx, dw


def _exact_rows(v):
    most = v.abs().max(1).values
    steps = torch.round(v * 127 / most.clamp(min=1e-300)[:, None])
    return steps * (most / 127)[:, None], most / 127


def _exact_route(s):
    l = s["logits"].to(torch.float64)
    R, E, G = s["R"], s["E"], s["groups"]
    if s["score"] == "softmax":
        e = torch.exp(l - l.max(1, keepdim=True).values)
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-l))
    want = p.clone() if s["b"] is None else p + s["b"].to(torch.float64)
    if G > 1:
        part = want.reshape(R, G, E // G).clone()
        strength = torch.zeros(R, G, dtype=torch.float64, device=l.device)
        for _ in range(min(s["best"], E // G)):
            value, at = part.max(-1)
            strength += value
            part.scatter_(-1, at[..., None], -math.inf)
        allowed = torch.zeros(R, G, dtype=torch.bool, device=l.device)
        for _ in range(s["top_groups"]):
            allowed.scatter_(1, _first_max(strength.masked_fill(allowed, -math.inf)), True)
        want = want.reshape(R, G, E // G).masked_fill(~allowed[..., None], -math.inf).reshape(R, E)
    ids = torch.empty(R, s["top"], dtype=torch.int64, device=l.device)
    for j in range(s["top"]):
        ids[:, j:j + 1] = _first_max(want)
        want.scatter_(1, ids[:, j:j + 1], -math.inf)
    chosen = torch.zeros_like(p).scatter_(1, ids, 1.0)
    total = (p * chosen).sum(1, keepdim=True) if s["renorm"] else torch.ones(R, 1, dtype=torch.float64, device=l.device)
    w = 2.5 * p.gather(1, ids) / total
    if not s["grad"]:
        return w, ids.int()
    g = torch.zeros_like(p).scatter_(1, ids, 2.5 * s["dw"].to(torch.float64)) / total   # with respect to the scores
    if s["renorm"]:
        g = g - chosen * (g * p).sum(1, keepdim=True) / total
    if s["score"] == "sigmoid":
        return w, ids.int(), g * p * (1 - p)
    return w, ids.int(), p * (g - (g * p).sum(1, keepdim=True))


def _first_max(v):
    """The lowest index of each row's largest value."""
    at = torch.arange(v.shape[1], device=v.device)
    return torch.where(v == v.max(1, keepdim=True).values, at, v.shape[1]).min(1, keepdim=True).values


# ---------------------------------------------------------------- what a pass cannot avoid

def work(case):
    """Bytes (each input read once, each output written once) and operations of one pass."""
    if case["op"] == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": M * K + N * K + 4 * (M + N) + size * M * N + (size * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if case["op"] == "route":
        R, E, top = case["R"], case["E"], case["top"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": R * (size * E + 8 * top) + (4 * E if case["bias"] else 0)
                + (R * (4 * top + size * E) if case["grad"] else 0), "flops": R * E * (8 if case["grad"] else 4)}
    n = case["R"] * case["K"]
    if case["op"] == "rows":   # the values come back in the input's type
        return {"bytes": 4 * n + 4 * case["R"], "flops": 3 * n}
    weight = case["K"] * (4 if case["wide"] else 2)
    if case["op"] == "norm_i8":
        return {"bytes": (8 if case["residual"] else 4) * n + weight + 4 * case["R"], "flops": 7 * n}
    # x, dy and, with a residual, r and dh; y, the gradients (x's and r's are one) and, with a residual, h
    return {"bytes": (14 if case["residual"] else 8) * n + 2 * weight, "flops": (16 if case["residual"] else 14) * n}
