"""Workloads of the expert-layer operators: the row grouping, the products
grouped by expert, their weight gradient, and the 4-bit matrix-vector product.

`listed()` names the cases, `draw(rng)` gives more of the same ranges,
`prepare(case, seed)` makes a case's inputs on the GPU, `run(state)` is one
call of the operator (`own` true: this library's; false: elementary torch
operations in 32 bits, rounded once), `exact(case, seed)` the 64-bit value by
definition and `work(case)` the bytes and operations that a call cannot avoid.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # Training forward of a large expert layer: 8192 tokens, two experts each.
        dict(name="matmul_train_bf16", op="matmul", dtype="bf16", R=16384, K=4096, N=4096, E=8, trans=False, pad=0),
        # Input gradient (weights read transposed) with many small experts, padded to a capacity.
        dict(name="matmul_dgrad_bf16", op="matmul", dtype="bf16", R=5003, K=1408, N=2048, E=64, trans=True, pad=117),
        # Unaligned feature sizes: the element-wise path.
        dict(name="matmul_odd_f16", op="matmul", dtype="f16", R=777, K=1003, N=517, E=5, trans=False, pad=0),
        # A decode batch through unquantized experts: a few rows for each.
        dict(name="matmul_decode_f16", op="matmul", dtype="f16", R=16, K=1024, N=512, E=8, trans=True, pad=0),
        # Weight gradient of the training layer, into fp32 gradients.
        dict(name="wgrad_train_bf16", op="wgrad", dtype="bf16", out="f32", R=16384, M=4096, N=2048, E=8, pad=0),
        # Weight gradient with many small experts, some without a row.
        dict(name="wgrad_many_f16", op="wgrad", dtype="f16", out="f16", R=4099, M=1024, N=2048, E=64, pad=51),
        # A micro-batch's weight gradient.
        dict(name="wgrad_small_bf16", op="wgrad", dtype="bf16", out="bf16", R=48, M=512, N=256, E=4, pad=0),
        # One token through one 4-bit projection.
        dict(name="w4_token_bf16", op="w4", dtype="bf16", M=1, K=4096, N=4096, E=0, G=128, zeros=False),
        # A decode batch through a large 4-bit projection with zero points.
        dict(name="w4_batch_f16", op="w4", dtype="f16", M=16, K=8192, N=14336, E=0, G=64, zeros=True),
        # A decode batch through 4-bit experts, each row its own.
        dict(name="w4_experts_bf16", op="w4", dtype="bf16", M=32, K=4096, N=2048, E=16, G=32, zeros=False),
        # Router choices of a decode batch.
        dict(name="rows_decode", op="rows", R=64, E=8, wide=True),
        # Router choices of a training batch.
        dict(name="rows_train", op="rows", R=131072, E=128, wide=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _feature(rng, hi, odd):
    """A feature size: a multiple of 8, or any size up to 1200 on the element-wise path."""
    return _log_int(rng, 17, 1200) if odd else 8 * _log_int(rng, 4, hi // 8)


def draw(rng):
    op = rng.choice(("matmul", "matmul", "wgrad", "wgrad", "w4", "w4", "rows"))
    if op == "rows":
        return dict(op=op, R=_log_int(rng, 1, 131072), E=_log_int(rng, 1, 256), wide=rng.random() < 0.5)
    dtype = rng.choice(("f16", "bf16"))
    if op == "w4":
        G = rng.choice((32, 64, 128))
        N = _log_int(rng, 16, 14336)
        K = 32 * _log_int(rng, 4, 256)
        E = 0 if rng.random() < 0.5 else max(1, min(_log_int(rng, 1, 64), 14336 * 8192 // (N * K)))
        return dict(op=op, dtype=dtype, M=_log_int(rng, 1, 32), K=K, N=N, E=E, G=G, zeros=rng.random() < 0.5)
    odd = rng.random() < 0.2
    R = _log_int(rng, 1, 2048 if odd else 16384)
    X, N = _feature(rng, 4096, odd), _feature(rng, 4096 if op == "matmul" else 2048, odd)
    E = max(1, min(_log_int(rng, 1, 128), 8 * 4096 * 2048 // (X * N)))
    pad = rng.randrange(0, R // 8 + 1) if rng.random() < 0.5 else 0
    if op == "matmul":
        return dict(op=op, dtype=dtype, R=R, K=X, N=N, E=E, trans=rng.random() < 0.5, pad=pad)
    return dict(op=op, dtype=dtype, out=rng.choice(("f32", dtype)), R=R, M=X, N=N, E=E, pad=pad)


def _lengths(case, seed):
    """Rows of each expert: a skewed router, as untrained and trained ones are."""
    rng = np.random.default_rng([seed, 11])
    p = np.exp(rng.normal(0.0, 0.6, case["E"]))
    return rng.multinomial(case["R"] - case["pad"], p / p.sum())


def _ids(n, E, seed, dropped):
    rng = np.random.default_rng([seed, 12])
    p = np.exp(rng.normal(0.0, 0.6, E))
    ids = rng.choice(E, size=n, p=p / p.sum())
    if dropped:
        ids[rng.random(n) < 0.02] = -1
    return ids


def _randn(gen, shape, dtype, scale):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "rows":
        ids = _ids(case["R"], case["E"], seed, True)
        s["ids"] = torch.from_numpy(ids).to(torch.int64 if case["wide"] else torch.int32).cuda()
        return s
    dt = DTYPES[case["dtype"]]
    if case["op"] == "w4":
        M, N, K, E, G = case["M"], case["N"], case["K"], case["E"], case["G"]
        lead = (E,) if E else ()
        s["x"] = _randn(gen, (M, K), dt, 1.0)
        s["w"] = torch.randint(0, 256, lead + (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        groups = -(-K // G)
        s["scale"] = (torch.rand(lead + (N, groups), generator=gen, device="cuda") * 0.01 + 0.002).to(dt)
        s["zero"] = torch.randint(4, 12, lead + (N, groups), generator=gen, device="cuda",
                                  dtype=torch.uint8) if case["zeros"] else None
        s["rows"] = None
        s["experts"] = None
        if E:
            ids = _ids(M, E, seed, False)
            s["rows"] = ids.tolist()
            s["experts"] = torch.from_numpy(ids).to(torch.int32).cuda()
        return s
    lens = _lengths(case, seed)
    bounds = np.concatenate([[0], np.cumsum(lens)])
    s["bounds"] = bounds.tolist()
    s["offsets"] = torch.from_numpy(bounds).to(torch.int32).cuda()
    R, N, E = case["R"], case["N"], case["E"]
    if case["op"] == "matmul":
        K = case["K"]
        s["a"] = _randn(gen, (R, K), dt, 1.0)
        if case["trans"]:
            s["b"] = _randn(gen, (E, N, K), dt, K ** -0.5).transpose(1, 2)
        else:
            s["b"] = _randn(gen, (E, K, N), dt, K ** -0.5)
    else:
        s["a"] = _randn(gen, (R, case["M"]), dt, 1.0)
        s["g"] = _randn(gen, (R, N), dt, 0.1)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    if s["op"] == "rows":
        from dense_tiled_gemm_02_amd import grouped
        return grouped.group_rows(s["ids"], s["E"])
    if s["op"] == "matmul":
        from dense_tiled_gemm_02_amd import grouped
        return grouped.grouped_matmul(s["a"], s["b"], s["offsets"])
    if s["op"] == "wgrad":
        from dense_tiled_gemm_02_amd import grouped
        return grouped.grouped_wgrad(s["a"], s["g"], s["offsets"], out_dtype=DTYPES[s["out"]])
    from dense_tiled_gemm_02_amd import w4
    return w4.w4_matvec(s["x"], s["w"], s["scale"], zeros=s["zero"], group=s["G"], experts=s["experts"])


def _plain(s):
    if s["op"] == "rows":
        ids, E, R = s["ids"], s["E"], s["R"]
        key = torch.where((ids >= 0) & (ids < E), ids, E).long()
        member = (key == torch.arange(E + 1, device=ids.device)[:, None]).int()
        before = torch.cumsum(member, 1, dtype=torch.int32)
        count = before[:, -1].long()
        offsets = torch.zeros(E + 2, dtype=torch.int64, device=ids.device)
        offsets[1:] = torch.cumsum(count, 0)
        row = torch.arange(R, device=ids.device)
        order = torch.empty(R, dtype=torch.int32, device=ids.device)
        order[offsets[key] + before[key, row].long() - 1] = row.int()
        return offsets[:E + 1].int(), order
    dt = DTYPES[s["dtype"]]
    if s["op"] == "matmul":
        d = torch.zeros(s["R"], s["N"], dtype=dt, device=s["a"].device)
        for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if hi > lo:
                d[lo:hi] = (s["a"][lo:hi].float() @ s["b"][e].float()).to(dt)
        return d
    if s["op"] == "wgrad":
        d = torch.zeros(s["E"], s["M"], s["N"], dtype=DTYPES[s["out"]], device=s["a"].device)
        for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if hi > lo:
                d[e] = (s["a"][lo:hi].float().t() @ s["g"][lo:hi].float()).to(d.dtype)
        return d
    x = s["x"].float()
    if s["rows"] is None:
        return (x @ _dequant(s["w"], s["scale"], s["zero"], s["G"], s["K"]).t()).to(dt)
    y = torch.zeros(s["M"], s["N"], dtype=dt, device=x.device)
    for e in sorted(set(s["rows"])):
        pick = torch.tensor([i for i, r in enumerate(s["rows"]) if r == e], device=x.device)
        w = _dequant(s["w"][e], s["scale"][e], None if s["zero"] is None else s["zero"][e], s["G"], s["K"])
        y[pick] = (x[pick] @ w.t()).to(dt)
    return y


def _dequant(w, scale, zero, G, K):
    q = torch.stack((w & 15, w >> 4), -1).reshape(w.shape[0], K).float()
    z = zero.float().repeat_interleave(G, 1)[:, :K] if zero is not None else 8.0
    return (q - z) * scale.float().repeat_interleave(G, 1)[:, :K]


# ---------------------------------------------------------------- by definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rows":
        ids = s["ids"].cpu().numpy()
        key = np.where((ids >= 0) & (ids < s["E"]), ids, s["E"])
        offsets = np.searchsorted(np.sort(key), np.arange(s["E"] + 1), side="left")
        order = np.argsort(key, kind="stable")
        return (torch.from_numpy(offsets.astype(np.int32)).cuda(), torch.from_numpy(order.astype(np.int32)).cuda())
    if s["op"] == "w4":
        M, N, K, G = s["M"], s["N"], s["K"], s["G"]
        group = torch.arange(K, device="cuda") // G
        y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        E = s["E"] or 1
        w = s["w"].reshape(E, N, K // 2)
        scale = s["scale"].reshape(E, N, -1)
        rows = np.zeros(M, np.int64) if s["rows"] is None else np.asarray(s["rows"])
        for e in range(E):
            hit = torch.from_numpy(np.nonzero(rows == e)[0]).cuda()
            if hit.numel() == 0:
                continue
            weight = torch.empty(N, K, dtype=torch.float64, device="cuda")
            weight[:, 0::2] = (w[e] % 16).double()
            weight[:, 1::2] = (w[e] // 16).double()
            if s["zero"] is None:
                weight -= 8
            else:
                weight -= s["zero"].reshape(E, N, -1)[e].double()[:, group]
            weight *= scale[e].double()[:, group]
            y[hit] = s["x"][hit].double() @ weight.t()
        return y
    bounds = s["bounds"]
    a = s["a"]
    if s["op"] == "matmul":
        parts = [a[bounds[e]:bounds[e + 1]].double() @ s["b"][e].double() for e in range(s["E"])]
        parts.append(torch.zeros(s["R"] - bounds[-1], s["N"], dtype=torch.float64, device="cuda"))
        return torch.cat(parts)
    return torch.stack([a[bounds[e]:bounds[e + 1]].double().t() @ s["g"][bounds[e]:bounds[e + 1]].double()
                        for e in range(s["E"])])


# ---------------------------------------------------------------- what a pass cannot avoid

def work(case):
    """Bytes (each input read once, each output written once) and operations of
    one pass; every expert counts as used where there are enough rows for it."""
    if case["op"] == "rows":
        return {"bytes": case["R"] * ((8 if case["wide"] else 4) + 4) + 4 * (case["E"] + 1), "flops": 0}
    if case["op"] == "w4":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        used = min(case["E"], M) if case["E"] else 1
        per_group = 3 if case["zeros"] else 2
        return {"bytes": used * (N * K // 2 + N * -(-K // G) * per_group) + 2 * M * (K + N), "flops": 2 * M * N * K}
    R, N, E = case["R"], case["N"], case["E"]
    rows = R - case["pad"]
    if case["op"] == "matmul":
        K = case["K"]
        return {"bytes": 2 * rows * K + 2 * min(E, rows) * K * N + 2 * R * N, "flops": 2 * rows * K * N}
    M = case["M"]
    return {"bytes": 2 * rows * (M + N) + (4 if case["out"] == "f32" else 2) * E * M * N, "flops": 2 * rows * M * N}
