"""The dense layer's fused operators, as measured workloads.

Five operators that a transformer's feed-forward layer runs, forward, backward
and in its optimiser, each in its plain form (elementary torch operations in
32 bits, rounded once at the end) and, where ``own`` is true, through this
library's entry points:

    linear       C = act(A B^T + bias) + R, optionally with Z = A B^T + bias
    linear_bwd   dA, dB, dbias of act(A B^T + bias) from Z and dC
    gated        C = act(Z_gate) * Z_up, [Z_gate Z_up] = A B^T + bias,
                 B holding N gate rows and then N up rows
    gated_bwd    dA, dB, dbias of it from Z and dC
    ortho        Newton-Schulz orthogonalisation of a batch of matrices

A (M x K) holds tokens, B (N x K, or 2N x K) the weights, all BF16 and
row-major; sums are taken in FP32 or wider.
"""
import math

import torch

own = False

#: Coefficients of the quintic X <- a X + (b X X^T + c (X X^T)^2) X that
#: the optimiser uses, its number of steps and the guard of its division.
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7

ACTS = ("none", "relu", "gelu", "silu")


def listed():
    return [
        # One token through an output projection while serving: the weights
        # are read once, latency counts.
        {"name": "linear_1_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "act": "none", "bias": False,
         "res": True, "z": False},
        # A ragged batch of short prompts with everything switched on, its
        # pre-activations kept for training.
        {"name": "linear_ragged", "op": "linear", "M": 333, "N": 1032, "K": 2056, "act": "gelu", "bias": True,
         "res": True, "z": True},
        # A training batch through a down projection with the residual.
        {"name": "linear_8192", "op": "linear", "M": 8192, "N": 4096, "K": 8192, "act": "none", "bias": True,
         "res": True, "z": False},
        # A small layer's gradients at an odd number of tokens.
        {"name": "linear_bwd_odd", "op": "linear_bwd", "M": 777, "N": 1000, "K": 520, "act": "none", "bias": True},
        # A training batch's gradients through a GELU layer.
        {"name": "linear_bwd_4096", "op": "linear_bwd", "M": 4096, "N": 8192, "K": 4096, "act": "gelu", "bias": True},
        # Four sequences decoding one token each through a gated layer.
        {"name": "gated_4_tokens", "op": "gated", "M": 4, "N": 8192, "K": 4096, "act": "silu", "bias": False,
         "z": False},
        # A short prompt through a gated layer of odd width.
        {"name": "gated_ragged", "op": "gated", "M": 129, "N": 2744, "K": 1032, "act": "gelu", "bias": True,
         "z": True},
        # A training batch through a gated layer, pre-activations kept.
        {"name": "gated_8192", "op": "gated", "M": 8192, "N": 8192, "K": 4096, "act": "silu", "bias": False,
         "z": True},
        # A small gated layer's gradients at an odd number of tokens.
        {"name": "gated_bwd_odd", "op": "gated_bwd", "M": 301, "N": 1384, "K": 512, "act": "gelu", "bias": True},
        # A training batch's gradients through a gated layer.
        {"name": "gated_bwd_4096", "op": "gated_bwd", "M": 4096, "N": 8192, "K": 4096, "act": "silu", "bias": False},
        # The optimiser's update of a stack of small projections.
        {"name": "ortho_stack", "op": "ortho", "batch": 6, "rows": 1032, "cols": 256, "fp32": False},
        # The optimiser's update of one large weight, momentum in FP32.
        {"name": "ortho_4096", "op": "ortho", "batch": 1, "rows": 4096, "cols": 8192, "fp32": True},
    ]


def _log_size(rng, low, high, of):
    """A multiple of `of` in low .. high, spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / of)) * of))


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "gated", "gated_bwd", "ortho"])
    if op == "ortho":
        while True:
            rows, cols = _log_size(rng, 64, 8192, 8), _log_size(rng, 64, 8192, 8)
            batch = rng.choice([1, 2, 3, 5, 8, 12])
            if min(rows, cols) <= 4096 and batch * min(rows, cols) ** 2 * max(rows, cols) <= 4096 * 4096 * 8192:
                return {"op": op, "batch": batch, "rows": rows, "cols": cols, "fp32": rng.random() < 0.5}
    case = {"op": op, "M": _log_size(rng, 1, 8192, 1), "N": _log_size(rng, 64, 8192, 8),
            "K": _log_size(rng, 64, 8192, 8), "act": rng.choice(ACTS), "bias": rng.random() < 0.5}
    if op.endswith("_bwd"):
        case["M"] = min(case["M"], 4096)
        case["K"] = min(case["K"], 4096)
    elif op == "gated":
        case["K"] = min(case["K"], 4096)
    if op == "linear":
        case["N"] = min(case["N"], 4096)
        case["res"] = rng.random() < 0.7
    if op in ("linear", "gated"):
        case["z"] = rng.random() < 0.4
    return case


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "ortho":
        # momentum of a weight: a sum over tokens of gradient times activation
        b, r, c = case["batch"], case["rows"], case["cols"]
        t = 2 * max(r, c)
        g = torch.empty(b, r, c, device="cuda")
        for i in range(b):
            g[i] = _normal(gen, r, t, std=1e-3, dtype=torch.float32) @ _normal(gen, t, c, dtype=torch.float32)
        s["G"] = g if case["fp32"] else g.to(torch.bfloat16)
        if own:
            import dense_gemm_14_amd as lib
            s["lib"] = lib
            s["O"] = torch.empty(b, r, c, device="cuda", dtype=torch.bfloat16)
            s["ws"] = _workspace(lib.newton_schulz_workspace_size(b, r, c))
        return s
    M, N, K = case["M"], case["N"], case["K"]
    rows = 2 * N if case["op"].startswith("gated") else N
    s["A"] = _normal(gen, M, K)
    s["B"] = _normal(gen, rows, K, std=K ** -0.5)
    if case["op"].endswith("_bwd"):
        s["Z"] = _normal(gen, M, rows)   # pre-activations kept by the forward pass
        s["dC"] = _normal(gen, M, N, std=2.0 ** -8)
    else:
        s["bias_v"] = _normal(gen, rows, std=0.5) if case["bias"] else None
        s["R"] = _normal(gen, M, N) if case.get("res") else None
    if own:
        import dense_gemm_14_amd as lib
        s["lib"] = lib
        new = lambda *shape: torch.empty(*shape, device="cuda", dtype=torch.bfloat16)
        s["act_id"] = {"none": lib.ACT_NONE, "relu": lib.ACT_RELU, "gelu": lib.ACT_GELU_TANH,
                       "silu": lib.ACT_SILU}[case["act"]]
        if case["op"].endswith("_bwd"):
            s["dA"], s["dB"] = new(M, K), new(rows, K)
            s["dbias"] = new(rows) if case["bias"] else None
            s["ws"] = _workspace(lib.bias_act_bwd_workspace_size(M, N, K, s["act_id"]) if case["op"] == "linear_bwd"
                                 else lib.gated_bwd_workspace_size(M, N, K))
        else:
            s["C"] = new(M, N)
            s["Zout"] = new(M, rows) if case["z"] else None
            s["ws"] = _workspace(lib.bias_act_res_workspace_size(M, N, K) if case["op"] == "linear"
                                 else lib.gated_workspace_size(M, N, K))
    return s


def _workspace(nbytes):
    return torch.empty(nbytes, device="cuda", dtype=torch.uint8) if nbytes else None


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    lib, op = s["lib"], s["op"]
    if op == "ortho":
        lib.newton_schulz(s["batch"], s["rows"], s["cols"], s["G"], s["O"], STEPS, QUINTIC, EPS, s["ws"])
        return {"O": s["O"]}
    M, N, K = s["M"], s["N"], s["K"]
    if op == "linear":
        lib.gemm_bf16_nt_bias_act_res(M, N, K, s["A"], s["B"], s["bias_v"], s["act_id"], s["R"], s["Zout"], s["C"],
                                      s["ws"])
        return {"C": s["C"], "Z": s["Zout"]} if s["z"] else {"C": s["C"]}
    if op == "gated":
        lib.gemm_bf16_nt_gated(M, N, K, s["A"], s["B"], s["bias_v"], s["act_id"], s["Zout"], s["C"], s["ws"])
        return {"C": s["C"], "Z": s["Zout"]} if s["z"] else {"C": s["C"]}
    call = lib.gemm_bf16_nt_bias_act_bwd if op == "linear_bwd" else lib.gemm_bf16_nt_gated_bwd
    call(M, N, K, s["A"], s["B"], s["Z"], s["act_id"], s["dC"], s["dA"], s["dB"], s["dbias"], s["ws"])
    return {"dA": s["dA"], "dB": s["dB"], "dbias": s["dbias"]} if s["bias"] else {"dA": s["dA"], "dB": s["dB"]}


# ---- plain forms -------------------------------------------------------------

_ROOT = math.sqrt(2.0 / math.pi)


def _act(name, z):
    if name == "relu":
        return z * (z > 0)
    if name == "gelu":
        return z / (1 + torch.exp(-2 * _ROOT * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        s = 1 / (1 + torch.exp(-2 * _ROOT * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * 2 * _ROOT * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def _run_plain(s):
    op, bf16 = s["op"], torch.bfloat16
    if op == "ortho":
        a, b, c = QUINTIC
        out = []
        for g in s["G"]:
            x = g.float()
            x = x / (torch.sqrt((x * x).sum()) + EPS)
            tall = x.shape[0] > x.shape[1]
            x = x.t() if tall else x
            for _ in range(STEPS):
                p = x @ x.t()
                x = a * x + (b * p + c * (p @ p)) @ x
            out.append((x.t() if tall else x).to(bf16))
        return {"O": torch.stack(out)}
    N, act = s["N"], s["act"]
    if op in ("linear", "gated"):
        z = s["A"].float() @ s["B"].float().t()
        if s["bias_v"] is not None:
            z = z + s["bias_v"].float()
        if op == "gated":
            y = _act(act, z[:, :N]) * z[:, N:]
        else:
            y = _act(act, z)
            if s["R"] is not None:
                y = y + s["R"].float()
        return {"C": y.to(bf16), "Z": z.to(bf16)} if s["z"] else {"C": y.to(bf16)}
    z, dc = s["Z"].float(), s["dC"].float()
    if op == "gated_bwd":
        gate, up = z[:, :N], z[:, N:]
        dz = torch.cat([dc * up * _act_grad(act, gate), dc * _act(act, gate)], dim=1)
    else:
        dz = dc * _act_grad(act, z)
    out = {"dA": (dz @ s["B"].float()).to(bf16), "dB": (dz.t() @ s["A"].float()).to(bf16)}
    if s["bias"]:
        out["dbias"] = dz.sum(0).to(bf16)
    return out


# ---- definitions in 64 bits --------------------------------------------------


def exact(case, seed):
    """The same outputs from the operators' definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "ortho":
        a, b, c = QUINTIC
        x = s["G"].double()
        x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS)
        eye = torch.eye(min(case["rows"], case["cols"]), device="cuda", dtype=torch.float64)
        for i in range(x.shape[0]):
            for _ in range(STEPS):
                if case["rows"] <= case["cols"]:
                    q = torch.mm(x[i], x[i].t())
                    x[i] = torch.mm(a * eye + torch.mm(b * eye + c * q, q), x[i])
                else:
                    q = torch.mm(x[i].t(), x[i])
                    x[i] = torch.mm(x[i], a * eye + torch.mm(b * eye + c * q, q))
        return {"O": x}
    N, name = case["N"], case["act"]
    f = {"none": lambda z: z, "relu": lambda z: torch.clamp(z, min=0),
         "gelu": lambda z: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))),
         "silu": lambda z: z * torch.sigmoid(z)}[name]
    if not case["op"].endswith("_bwd"):
        z = torch.mm(s["A"].double(), s["B"].double().t())
        if s["bias_v"] is not None:
            z += s["bias_v"].double()
        y = f(z[:, :N]) * z[:, N:] if case["op"] == "gated" else f(z)
        if s.get("R") is not None:
            y = y + s["R"].double()
        return {"C": y, "Z": z} if case["z"] else {"C": y}
    # the derivative of each element's activation, by torch's own differentiation
    z = s["Z"].double().requires_grad_()
    y = f(z[:, :N]) * z[:, N:] if case["op"] == "gated_bwd" else f(z)
    dz, = torch.autograd.grad(y, z, s["dC"].double())
    out = {"dA": torch.mm(dz, s["B"].double()), "dB": torch.mm(dz.t(), s["A"].double())}
    if case["bias"]:
        out["dbias"] = torch.sum(dz, dim=0)
    return out


def work(case):
    if case["op"] == "ortho":
        b, r, c = case["batch"], case["rows"], case["cols"]
        m, n = min(r, c), max(r, c)
        # the Gram product and its square are symmetric: half of each
        return {"bytes": b * r * c * ((4 if case["fp32"] else 2) + 2),
                "flops": b * STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)}
    M, N, K = case["M"], case["N"], case["K"]
    rows = 2 * N if case["op"].startswith("gated") else N
    if case["op"].endswith("_bwd"):
        keeps_z = case["op"] == "gated_bwd" or case["act"] != "none"
        return {"bytes": 2 * (2 * M * K + 2 * rows * K + M * N + (M * rows if keeps_z else 0) + (rows if case["bias"] else 0)),
                "flops": 4 * M * rows * K}
    return {"bytes": 2 * (M * K + rows * K + M * N * (2 if case.get("res") else 1) + (M * rows if case["z"] else 0)
                          + (rows if case["bias"] else 0)),
            "flops": 2 * M * rows * K}
