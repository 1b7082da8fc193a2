"""The training operators of the pre-norm gated FFN block, measured case by case.

Five paths: layer norm forward (with the residual add) and backward (with the
reduction of the weight's and bias's gradients), the gated FFN's training
forward (keeping the two projections) and backward, and the Newton-Schulz
orthogonalisation of weight updates (as the Muon optimiser does).

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, with ``own`` true, through the framework's entry points.  ``exact``
gives the same outputs in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
NS = (3.4445, -4.7750, 2.0315)   # Newton-Schulz coefficients a, b, c
NS_EPS = 1e-7
NS_STEPS = 5


def listed():
    return [
        # one decoding batch's worth of tokens at the tiny model width: latency
        {"name": "ln_fwd_tiny", "op": "ln_fwd", "T": 64, "N": 256, "type": "bf16", "params": "bf16", "residual": True},
        # the residual stream of a large model's micro-batch: bandwidth
        {"name": "ln_fwd_large", "op": "ln_fwd", "T": 16384, "N": 8192, "type": "bf16", "params": "f32",
         "residual": True},
        # packed sequences of odd total length, an fp32 stream of odd width (rows not 16-byte aligned)
        {"name": "ln_bwd_ragged_f32", "op": "ln_bwd", "T": 4099, "N": 1021, "type": "f32", "params": "f32",
         "residual": False},
        # the large micro-batch's backward, with the residual's gradient added
        {"name": "ln_bwd_large", "op": "ln_bwd", "T": 16384, "N": 8192, "type": "bf16", "params": "f32",
         "residual": True},
        # a handful of tokens through a Llama 3 8B sized block: the weights' bytes
        {"name": "glu_fwd_few", "op": "glu_fwd", "M": 16, "N": 4096, "O": 14336, "P": 4096, "act": "silu"},
        # a micro-batch of 4096 tokens through the same block: tensor cores
        {"name": "glu_fwd_8b", "op": "glu_fwd", "M": 4096, "N": 4096, "O": 14336, "P": 4096, "act": "silu"},
        # the tiny block: latency
        {"name": "glu_bwd_tiny", "op": "glu_bwd", "M": 64, "N": 256, "O": 1024, "P": 256, "act": "silu"},
        # packed sequences of odd total length, sizes that end inside a tile, GeGLU
        {"name": "glu_bwd_ragged", "op": "glu_bwd", "M": 1003, "N": 2056, "O": 5528, "P": 2056, "act": "gelu_tanh"},
        # the Llama 3 8B sized block's backward
        {"name": "glu_bwd_8b", "op": "glu_bwd", "M": 4096, "N": 4096, "O": 14336, "P": 4096, "act": "silu"},
        # one small weight matrix's update: latency of fifteen dependent products
        {"name": "muon_tiny", "op": "muon", "B": 1, "m": 256, "n": 1024, "type": "bf16"},
        # the stacked down projections of eight small experts (tall matrices), fp32 momentum
        {"name": "muon_experts", "op": "muon", "B": 8, "m": 4096, "n": 1024, "type": "f32"},
        # the Llama 3 8B sized block's W1
        {"name": "muon_8b", "op": "muon", "B": 1, "m": 4096, "n": 14336, "type": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "glu_fwd", "glu_bwd", "muon"])
    if op in ("ln_fwd", "ln_bwd"):
        T, N, kind = _log(rng, 1, 16384), _log(rng, 32, 8192), rng.choice(["bf16", "f32"])
        if kind == "f32":
            T = (T + 1) // 2   # no more bytes than the largest listed case
        return {"op": op, "T": T, "N": N, "type": kind,
                "params": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.5}
    if op in ("glu_fwd", "glu_bwd"):
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 64, 4096, 8), "O": _log(rng, 64, 14336, 8),
                "P": _log(rng, 64, 4096, 8), "act": rng.choice(["silu", "gelu_tanh", "relu", "none"])}
    m, n = _log(rng, 16, 4096), _log(rng, 16, 14336)
    if rng.random() < 0.5:
        m, n = n, m
    case = {"op": op, "B": rng.choice([1, 1, 2, 3, 8]), "m": m, "n": n, "type": rng.choice(["bf16", "f32"])}
    while case["B"] > 1 and case["B"] * m * n * min(m, n) > 4096 * 4096 * 14336:
        case["B"] -= 1
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).add_(mean)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        T, N, act, par = case["T"], case["N"], TYPES[case["type"]], TYPES[case["params"]]
        # a residual stream: channels of different scale and offset, a few of them far larger
        scale = torch.exp(_randn(g, N, std=0.3))
        scale[torch.randint(0, N, (1 + N // 512,), generator=g, device="cuda")] *= 20.0
        offset = _randn(g, N, std=0.1)

        def stream():
            return _randn(g, T, N).mul_(scale).add_(offset).to(act)

        st = {"case": case, "gamma": _randn(g, N, std=0.1, mean=1.0).to(par), "beta": _randn(g, N, std=0.1).to(par)}
        if op == "ln_fwd":
            return st | {"X": stream(), "residual": stream() if case["residual"] else None}
        S = stream()
        f = S.float()
        mean = f.mean(1)
        rstd = (f.var(1, unbiased=False) + EPS).rsqrt()
        return st | {"S": S, "mean": mean, "rstd": rstd, "dY": _randn(g, T, N, std=0.05).to(act),
                     "dS": _randn(g, T, N, std=0.05).to(act) if case["residual"] else None}
    if op in ("glu_fwd", "glu_bwd"):
        M, N, O, P = case["M"], case["N"], case["O"], case["P"]
        bf = torch.bfloat16
        st = {"case": case, "X": _randn(g, M, N).to(bf), "W1": _randn(g, N, O, std=N ** -0.5).to(bf),
              "W3": _randn(g, N, O, std=N ** -0.5).to(bf), "W2": _randn(g, O, P, std=O ** -0.5).to(bf)}
        if op == "glu_bwd":   # what the forward pass kept, and the loss's gradient
            st |= {"G": st["X"] @ st["W1"], "U": st["X"] @ st["W3"], "dY": _randn(g, M, P, std=0.01).to(bf)}
        return st
    B, m, n = case["B"], case["m"], case["n"]
    # momentum: gradient noise and a few strong directions
    r = max(1, min(m, n) // 64)
    G = _randn(g, B, m, n)
    G.baddbmm_(_randn(g, B, m, r), _randn(g, B, r, n), alpha=r ** -0.5)
    G = G.mul_(1e-3).to(TYPES[case["type"]])
    return {"case": case, "G": G[0] if B == 1 else G}


# ------------------------------------------------------------- plain forms
def _act(name, x):
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x ** 3)))
    return torch.clamp_min(x, 0) if name == "relu" else x


def _act_grad(name, x):
    if name == "silu":
        s = torch.sigmoid(x)
        return s * (1 + x * (1 - s))
    if name == "gelu_tanh":
        c = 0.7978845608028654
        t = torch.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    return (x > 0).to(x.dtype) if name == "relu" else torch.ones_like(x)


def _ln_fwd(s):
    X, R = s["X"], s["residual"]
    S = X if R is None else (X.float() + R.float()).to(X.dtype)   # the norm is of S as it is stored
    f = S.float()
    mean = f.mean(1, keepdim=True)
    c = f - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    Y = (c * rstd * s["gamma"].float() + s["beta"].float()).to(X.dtype)
    return {"Y": Y, "S": S, "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _ln_bwd(s):
    dY, r = s["dY"].float(), s["rstd"][:, None]
    xh = (s["S"].float() - s["mean"][:, None]) * r
    g = dY * s["gamma"].float()
    dX = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["dS"] is not None:
        dX = dX + s["dS"].float()
    return {"dX": dX.to(s["dY"].dtype), "dgamma": (dY * xh).sum(0), "dbeta": dY.sum(0)}


def _glu_fwd(s):
    X, bf = s["X"].float(), torch.bfloat16
    G, U = X @ s["W1"].float(), X @ s["W3"].float()
    Y = (_act(s["case"]["act"], G) * U) @ s["W2"].float()
    return {"Y": Y.to(bf), "G": G.to(bf), "U": U.to(bf)}


def _glu_bwd(s):
    act, bf = s["case"]["act"], torch.bfloat16
    dY, X, G, U = s["dY"].float(), s["X"].float(), s["G"].float(), s["U"].float()
    a = _act(act, G)
    dH = dY @ s["W2"].float().t()
    dG, dU = dH * U * _act_grad(act, G), dH * a
    dX = dG @ s["W1"].float().t() + dU @ s["W3"].float().t()
    return {"dX": dX.to(bf), "dW1": (X.t() @ dG).to(bf), "dW3": (X.t() @ dU).to(bf),
            "dW2": ((a * U).t() @ dY).to(bf)}


def _muon(s):
    X = s["G"].float()
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.mT
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + NS_EPS)
    a, b, c = NS
    for _ in range(NS_STEPS):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return {"O": (X.mT if tall else X).to(torch.bfloat16).contiguous()}


_PLAIN = {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "glu_fwd": _glu_fwd, "glu_bwd": _glu_bwd, "muon": _muon}


def _own(s):
    import transformer_ffn_gb300 as tffn
    op = s["case"]["op"]
    if op == "ln_fwd":
        Y, S, mean, rstd = tffn.layer_norm_forward(s["X"], s["gamma"], s["beta"], residual=s["residual"], eps=EPS)
        return {"Y": Y, "S": S, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dX, dgamma, dbeta = tffn.layer_norm_backward(s["dY"], s["S"], s["gamma"], s["mean"], s["rstd"], dS=s["dS"])
        return {"dX": dX, "dgamma": dgamma, "dbeta": dbeta}
    if op == "glu_fwd":
        Y, G, U = tffn.ffn_glu_forward_train(s["X"], s["W1"], s["W3"], s["W2"], s["case"]["act"])
        return {"Y": Y, "G": G, "U": U}
    if op == "glu_bwd":
        dX, dW1, dW3, dW2 = tffn.ffn_glu_backward(s["dY"], s["X"], s["W1"], s["W3"], s["W2"], s["G"], s["U"],
                                                  s["case"]["act"])
        return {"dX": dX, "dW1": dW1, "dW3": dW3, "dW2": dW2}
    return {"O": tffn.muon_orthogonalize(s["G"], steps=NS_STEPS)}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        T, N = case["T"], case["N"]
        e, pe = (4 if case[k] == "f32" else 2 for k in ("type", "params"))
        if op == "ln_fwd":
            return {"bytes": 2 * T * N * e * (2 if case["residual"] else 1) + 8 * T + 2 * N * pe, "flops": 9 * T * N}
        return {"bytes": T * N * e * (4 if case["residual"] else 3) + 8 * T + N * pe + 8 * N, "flops": 14 * T * N}
    if op in ("glu_fwd", "glu_bwd"):
        M, N, O, P = case["M"], case["N"], case["O"], case["P"]
        weights = 2 * O * (2 * N + P)
        if op == "glu_fwd":
            return {"bytes": weights + 2 * M * (N + P + 2 * O), "flops": 2 * M * O * (2 * N + P)}
        return {"bytes": 2 * weights + 2 * M * (2 * N + P + 2 * O), "flops": 2 * M * O * (4 * N + 2 * P)}
    B, m, n = case["B"], min(case["m"], case["n"]), max(case["m"], case["n"])
    e = 4 if case["type"] == "f32" else 2
    # A and A A are symmetric: half of their entries
    return {"bytes": B * m * n * (e + 2), "flops": B * NS_STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)}


# ---------------------------------------------------------------- 64 bits
def _exact_act(name, x):
    """(activation, its derivative) in 64 bits."""
    if name == "relu":
        return torch.relu(x), torch.where(x > 0, 1.0, 0.0).double()
    if name == "none":
        return x, torch.ones_like(x)
    if name == "silu":
        sg = 1 / (1 + torch.exp(-x))
        return x * sg, sg + x * sg * (1 - sg)
    k = math.sqrt(2 / math.pi)
    u, du = k * (x + 0.044715 * x * x * x), k * (1 + 0.134145 * x * x)
    sg = 1 / (1 + torch.exp(-2 * u))       # 0.5 (1 + tanh u)
    return x * sg, sg + 2 * x * sg * (1 - sg) * du


def _exact_muon(G):
    U = G.double()
    flip = U.shape[0] > U.shape[1]
    X = (U.t() if flip else U) / (torch.linalg.vector_norm(U) + NS_EPS)
    a, b, c = NS
    eye = torch.eye(X.shape[0], dtype=torch.float64, device=X.device)
    for _ in range(NS_STEPS):
        A = torch.mm(X, X.t())
        X = torch.mm(a * eye + b * A + c * torch.mm(A, A), X)
    return (X.t() if flip else X).contiguous()


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "ln_fwd":
        X, R = s["X"], s["residual"]
        S = (X if R is None else (X.double() + R.double()).to(X.dtype)).double()
        mean, var = S.mean(1), S.var(1, unbiased=False)
        rstd = 1 / torch.sqrt(var + EPS)
        Y = S.sub(mean[:, None]).mul_(rstd[:, None]).mul_(s["gamma"].double()).add_(s["beta"].double())
        return {"Y": Y, "S": S, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        N, r = case["N"], s["rstd"].double()
        dY, xh = s["dY"].double(), (s["S"].double() - s["mean"].double()[:, None]) * r[:, None]
        g = dY * s["gamma"].double()
        dgamma, dbeta = torch.einsum("tn,tn->n", dY, xh), torch.einsum("tn->n", dY)
        dX = (g * N - g.sum(1)[:, None] - xh * torch.einsum("tn,tn->t", g, xh)[:, None]) * (r / N)[:, None]
        if s["dS"] is not None:
            dX += s["dS"].double()
        return {"dX": dX, "dgamma": dgamma, "dbeta": dbeta}
    if op == "glu_fwd":
        X = s["X"].double()
        G, U = torch.mm(X, s["W1"].double()), torch.mm(X, s["W3"].double())
        return {"Y": torch.mm(_exact_act(case["act"], G)[0] * U, s["W2"].double()), "G": G, "U": U}
    if op == "glu_bwd":
        X, dY, U = s["X"].double(), s["dY"].double(), s["U"].double()
        h, dh = _exact_act(case["act"], s["G"].double())
        dH = torch.mm(dY, s["W2"].double().t())
        dU, dG = dH * h, dH * dh * U
        dX = torch.mm(dG, s["W1"].double().t()).addmm_(dU, s["W3"].double().t())
        return {"dX": dX, "dW1": torch.mm(X.t(), dG), "dW3": torch.mm(X.t(), dU), "dW2": torch.mm((h * U).t(), dY)}
    G = s["G"]
    return {"O": _exact_muon(G) if G.dim() == 2 else torch.stack([_exact_muon(x) for x in G])}
