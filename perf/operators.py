"""The feed-forward operators as they are measured: cases, plain forms, 64-bit values.

Three operators, each in its directions:

* ``gated`` / ``gated_backward``: ``H = act(X Wg + bg) * (X Wu + bu)``, both products, the activation and the product
  of the two in one kernel (the training form also returns the pre-activations), and its gradients.
* ``residual`` / ``residual_backward``: ``Y = act(A B + bias) + R`` (the training form also returns ``A B + bias``), and
  its gradients.
* ``clip``: the global norm of a list of gradients and the list scaled to at most ``max_norm``.

Where ``own`` is false ``run`` computes them with elementary torch operations in 32 bits (sums of squares in 64),
rounded once at the end; where it is true it makes the library's calls.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One token of a feed-forward block 4096 -> 16384 (the FFN width of the benchmark): weights streamed once.
        {"name": "gated 1 token", "op": "gated", "M": 1, "N": 16384, "K": 4096, "dtype": "bf16", "out": "bf16",
         "act": "silu", "bias": False, "train": False},
        # A small decoding batch of a narrow block with biases and odd extents.
        {"name": "gated 17 tokens, odd", "op": "gated", "M": 17, "N": 2731, "K": 1001, "dtype": "f16", "out": "f16",
         "act": "gelu", "bias": True, "train": False},
        # A prompt of some hundred tokens, the hidden width 8/3 of the model width (odd).
        {"name": "gated prompt", "op": "gated", "M": 777, "N": 5461, "K": 2048, "dtype": "bf16", "out": "bf16",
         "act": "silu", "bias": False, "train": False},
        # The training forward at the benchmark's FFN shape: H and both pre-activations.
        {"name": "gated training forward", "op": "gated", "M": 8192, "N": 16384, "K": 4096, "dtype": "bf16",
         "out": "bf16", "act": "silu", "bias": False, "train": True},
        # Its backward.
        {"name": "gated backward", "op": "gated_backward", "M": 8192, "N": 16384, "K": 4096, "dtype": "bf16",
         "act": "silu", "bias": False},
        # A small training batch, biases, odd extents.
        {"name": "gated backward, odd", "op": "gated_backward", "M": 1537, "N": 2731, "K": 1024, "dtype": "f16",
         "act": "gelu", "bias": True},
        # The block's second product for one token, added to the residual stream.
        {"name": "residual 1 token", "op": "residual", "M": 1, "N": 4096, "K": 16384, "dtype": "bf16", "out": "bf16",
         "act": "none", "bias": False, "train": False},
        # A decoding batch whose residual stream is kept in fp32.
        {"name": "residual 40 tokens, fp32 stream", "op": "residual", "M": 40, "N": 1024, "K": 2731, "dtype": "f16",
         "out": "f32", "act": "none", "bias": True, "train": False},
        # The second product of a training batch.
        {"name": "residual batch", "op": "residual", "M": 8192, "N": 4096, "K": 16384, "dtype": "bf16", "out": "bf16",
         "act": "none", "bias": False, "train": False},
        # Backward of a square layer with GELU, bias and skip connection.
        {"name": "residual backward", "op": "residual_backward", "M": 4096, "N": 4096, "K": 4096, "dtype": "bf16",
         "act": "gelu", "bias": True},
        # The gradients of a few softplus MLPs (weights 128 x 128 and vectors, fp32, packed one behind the other).
        {"name": "clip small", "op": "clip", "count": 24, "total": 197000, "dtype": "f32", "aligned": False,
         "max_norm": 1.0},
        # The gradients of a stack of feed-forward blocks in one bucket.
        {"name": "clip large", "op": "clip", "count": 48, "total": 600000000, "dtype": "bf16", "aligned": True,
         "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "residual", "residual", "residual_backward", "clip"])
    if op == "clip":
        total = _log(rng, 2000, 600000000)
        count = min(_log(rng, 1, 400), total // 100)
        return {"op": op, "count": count, "total": total, "dtype": rng.choice(["f32", "bf16", "f16"]),
                "aligned": rng.random() < 0.5, "max_norm": rng.choice([1.0, 1.0, 0.25, 1e6])}
    dtype = rng.choice(["bf16", "f16"])
    c = {"op": op, "dtype": dtype, "bias": rng.random() < 0.4}
    if op in ("gated", "gated_backward"):
        c["K"] = _log(rng, 64, 4096)
        c["N"] = _log(rng, 64, 16384)
        c["act"] = rng.choice(["silu", "silu", "gelu", "relu"])
    else:
        c["K"] = _log(rng, 64, 16384)
        c["N"] = _log(rng, 64, 4096)
        c["act"] = rng.choice(["none", "none", "gelu", "silu", "softplus"])
    if op in ("gated", "residual"):
        c["M"] = _log(rng, 1, 8192)
        c["out"] = rng.choice([dtype, dtype, "f32"])
        c["train"] = rng.random() < 0.3
    else:
        c["M"] = _log(rng, 16, 8192)
    return c


def _sizes(case):
    """Element counts of the list's tensors: a fixed mixture of matrices and vectors, odd ones among them."""
    rng = random.Random(case["count"] * 1000003 + case["total"])
    w = [math.exp(rng.uniform(0.0, 3.0)) if i % 3 else 0.02 for i in range(case["count"])]
    s = sum(w)
    sizes = [max(1, int(case["total"] * x / s)) for x in w]
    sizes[-1] += max(0, case["total"] - sum(sizes))
    return sizes


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(gen, rows, cols, std, dtype):
    """rows x cols ~ N(0, std), each row starting at a multiple of 16 bytes."""
    per = 16 // _ES[dtype]
    t = torch.empty((rows, (cols + per - 1) // per * per), device="cuda", dtype=_DT[dtype])
    t.normal_(0.0, std, generator=gen)
    return t[:, :cols]


def _vec(gen, n, std, dtype):
    return torch.empty(n, device="cuda", dtype=_DT[dtype]).normal_(0.0, std, generator=gen)


def _space(rows, cols, dtype):
    per = 16 // _ES[dtype]
    return torch.empty((rows, (cols + per - 1) // per * per), device="cuda", dtype=_DT[dtype])[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case, "op": case["op"]}
    if case["op"] == "clip":
        sizes, offsets, at = _sizes(case), [], 0
        for n in sizes:
            offsets.append(at)
            at += (n + 63) // 64 * 64 if case["aligned"] else n
        flat = torch.zeros(at, device="cuda", dtype=_DT[case["dtype"]])
        flat_out = torch.zeros_like(flat)
        s["grads"] = [flat[o:o + n] for o, n in zip(offsets, sizes)]
        s["outs"] = [flat_out[o:o + n] for o, n in zip(offsets, sizes)]
        if case["aligned"]:
            for g in s["grads"]:
                g.normal_(0.0, 0.01, generator=gen)
        else:
            flat.normal_(0.0, 0.01, generator=gen)
        s["flat"], s["flat_out"] = flat, flat_out
        return s
    M, N, K, dt, bias = case["M"], case["N"], case["K"], case["dtype"], case["bias"]
    out_dt = case.get("out", dt)
    s["X"] = _rows(gen, M, K, 1.0, dt)
    names = ("g", "u") if case["op"].startswith("gated") else ("",)
    for e in names:
        s["W" + e] = _rows(gen, K, N, K ** -0.5, dt)
        s["b" + e] = _vec(gen, N, 0.02, dt) if bias else None
    if case["op"] == "residual":
        s["R"] = _rows(gen, M, N, 1.0, out_dt)
    if case["op"] in ("gated", "residual"):
        s["out"] = _space(M, N, out_dt)
    if case.get("train"):
        for e in names:
            s["Z" + e] = _space(M, N, dt)
    if case["op"].endswith("backward"):
        # the pre-activations that the training forward stored, and the gradient that arrives
        for e in names:
            z = torch.mm(s["X"], s["W" + e])
            s["Z" + e] = _space(M, N, dt)
            s["Z" + e].copy_(z if not bias else z + s["b" + e])
        s["dY"] = _rows(gen, M, N, 1.0, dt)
    return s


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------

def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.7071067811865476))
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "softplus":
        return torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-z.abs()))
    return z


def _act_grad(z, act):
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "softplus":
        return torch.sigmoid(z)
    return torch.ones_like(z)


def run(state):
    case, op = state["case"], state["op"]
    if own:
        return _run_own(state, case, op)
    if op == "clip":
        flat = state["flat"]
        norm = torch.sqrt(torch.sum(torch.square(flat.double())))
        coef = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)
        return {"norm": norm.float(), "grads": (flat.float() * coef.float()).to(flat.dtype)}
    dt, act = state["X"].dtype, case["act"]
    X = state["X"].float()
    if op == "gated":
        zg, zu = X @ state["Wg"].float(), X @ state["Wu"].float()
        if case["bias"]:
            zg, zu = zg + state["bg"].float(), zu + state["bu"].float()
        r = {"H": (_act(zg, act) * zu).to(_DT[case["out"]])}
        if case["train"]:
            r["Zg"], r["Zu"] = zg.to(dt), zu.to(dt)
        return r
    if op == "residual":
        z = X @ state["W"].float()
        if case["bias"]:
            z = z + state["b"].float()
        r = {"Y": (_act(z, act) + state["R"].float()).to(_DT[case["out"]])}
        if case["train"]:
            r["Z"] = z.to(dt)
        return r
    dY = state["dY"].float()
    if op == "gated_backward":
        zg, zu = state["Zg"].float(), state["Zu"].float()
        dzg, dzu = dY * zu * _act_grad(zg, act), dY * _act(zg, act)
        r = {"dX": (dzg @ state["Wg"].float().t() + dzu @ state["Wu"].float().t()).to(dt),
             "dWg": (X.t() @ dzg).to(dt), "dWu": (X.t() @ dzu).to(dt)}
        if case["bias"]:
            r["dbg"], r["dbu"] = dzg.sum(0).to(dt), dzu.sum(0).to(dt)
        return r
    dz = dY * _act_grad(state["Z"].float(), act)
    r = {"dX": (dz @ state["W"].float().t()).to(dt), "dW": (X.t() @ dz).to(dt)}
    if case["bias"]:
        r["db"] = dz.sum(0).to(dt)
    return r


def _run_own(state, case, op):
    import mlp_megakernel_amd as mk
    if op == "clip":
        norm = mk.clip_grad_norm(state["grads"], case["max_norm"], out=state["outs"])
        return {"norm": norm, "grads": state["flat_out"]}
    act, dt = case["act"], state["X"].dtype
    if op == "gated":
        if case["train"]:
            H, (Zg, Zu) = mk.gated_gemm_train(state["X"], state["Wg"], state["Wu"], state["bg"], state["bu"], act=act,
                                              out=state["out"], preact=(state["Zg"], state["Zu"]))
            return {"H": H, "Zg": Zg, "Zu": Zu}
        return {"H": mk.gated_gemm(state["X"], state["Wg"], state["Wu"], state["bg"], state["bu"], act=act,
                                   out=state["out"])}
    if op == "residual":
        if case["train"]:
            Y, Z = mk.gemm_residual_train(state["X"], state["W"], state["R"], state["b"], act=act, out=state["out"],
                                          preact=state["Z"])
            return {"Y": Y, "Z": Z}
        return {"Y": mk.gemm_residual(state["X"], state["W"], state["R"], state["b"], act=act, out=state["out"])}
    if op == "gated_backward":
        g = mk.gated_gemm_backward(state["X"], state["Wg"], state["Wu"], (state["Zg"], state["Zu"]), state["dY"],
                                   act=act, want_dbias=case["bias"], grad_dtype=dt)
        r = {"dX": g.dA, "dWg": g.dBg, "dWu": g.dBu}
        if case["bias"]:
            r["dbg"], r["dbu"] = g.dbias_g, g.dbias_u
        return r
    g = mk.gemm_residual_backward(state["X"], state["W"], state["dY"], preact=state["Z"], act=act,
                                  want_dbias=case["bias"], grad_dtype=dt)
    r = {"dX": g.dA, "dW": g.dB}
    if case["bias"]:
        r["db"] = g.dbias
    return r


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": 2 * n * _ES[case["dtype"]], "flops": 3 * n}
    M, N, K, es = case["M"], case["N"], case["K"], _ES[case["dtype"]]
    os = _ES[case.get("out", case["dtype"])]
    nb = 2 if case["op"].startswith("gated") else 1
    b = es * (M * K + nb * K * N + (nb * N if case["bias"] and not case["op"].endswith("backward") else 0))
    if not case["op"].endswith("backward"):
        b += os * M * N * (2 if case["op"] == "residual" else 1) + (nb * es * M * N if case["train"] else 0)
        return {"bytes": b, "flops": 2 * nb * M * N * K}
    # reads the pre-activations (not needed without an activation) and dY, writes dX, the dW and the bias gradients
    z = 0 if case["op"] == "residual_backward" and case["act"] == "none" else nb
    b += es * ((z + 1) * M * N + M * K + nb * K * N + (nb * N if case["bias"] else 0))
    return {"bytes": b, "flops": 4 * nb * M * N * K}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    D = {k: v.to(torch.float64) for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("out", "flat_out")}
    if case["op"] == "clip":
        v = D["flat"]
        norm = torch.linalg.vector_norm(v)
        top = float(case["max_norm"])
        n = float(norm) + 1e-6
        return {"norm": norm, "grads": v * (top / n) if n > top else v}

    def sigma(z):
        return 1.0 / (1.0 + torch.exp(-z))

    def cdf(z):
        return 0.5 * torch.erfc(-z / math.sqrt(2.0))

    # activation and derivative, each from its definition
    f, df = {
        "none": (lambda z: z, lambda z: z * 0 + 1),
        "relu": (lambda z: torch.where(z > 0, z, z * 0), lambda z: torch.where(z > 0, z * 0 + 1, z * 0)),
        "silu": (lambda z: z * sigma(z), lambda z: sigma(z) + z * sigma(z) * sigma(-z)),
        "gelu": (lambda z: z * cdf(z), lambda z: cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)),
        "softplus": (lambda z: torch.logaddexp(z, z * 0), sigma),
    }[case["act"]]

    def product(w, b):
        z = torch.mm(D["X"], D[w])
        return z.add_(D[b][None, :]) if D.get(b) is not None else z

    if case["op"] == "gated":
        zg, zu = product("Wg", "bg"), product("Wu", "bu")
        r = {"H": f(zg).mul_(zu)}
        if case["train"]:
            r.update(Zg=zg, Zu=zu)
        return r
    if case["op"] == "residual":
        z = product("W", "b")
        r = {"Y": f(z) + D["R"]}
        if case["train"]:
            r["Z"] = z
        return r
    if case["op"] == "gated_backward":
        du = f(D["Zg"]).mul_(D["dY"])
        dg = df(D["Zg"]).mul_(D["Zu"]).mul_(D["dY"])
        Xt = D["X"].t().contiguous()
        r = {"dX": torch.mm(dg, D["Wg"].t().contiguous()) + torch.mm(du, D["Wu"].t().contiguous()),
             "dWg": torch.mm(Xt, dg), "dWu": torch.mm(Xt, du)}
        if case["bias"]:
            r["dbg"], r["dbu"] = torch.sum(dg, dim=0), torch.sum(du, dim=0)
        return r
    dz = df(D["Z"]).mul_(D["dY"])
    r = {"dX": torch.mm(dz, D["W"].t().contiguous()), "dW": torch.mm(D["X"].t().contiguous(), dz)}
    if case["bias"]:
        r["db"] = torch.sum(dz, dim=0)
    return r
