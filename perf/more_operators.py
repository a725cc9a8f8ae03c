"""The two ends of a language model, as measured workloads.

What stands around the feed-forward layers when a network is trained or run:
the lookup of the tokens' rows, the normalisation before each layer, and the
loss over the vocabulary, each with its gradients. Each operator is there in
its plain form (elementary torch operations in 32 bits, rounded once at the
end) and, where ``own`` is true, through this library's entry points:

    embed     Y[t] = scale E[ids[t]]
    embed_bwd dE[v] = R[v] + scale sum of dY[t] over the t with ids[t] = v
    norm      Y = (X - mean) rstd gamma + beta, with mean and rstd of each row
    norm_bwd  dX (plus the residual's gradient R), dgamma and dbeta of it
    ce        loss[m] = lse[m] - z[m][targets[m]], lse[m] = log sum exp z[m],
              z = A B^T, without keeping z
    ce_bwd    dA, dB of it for the gradient dloss of each row's loss

An id or a target outside 0 .. vocab - 1 marks a place that is left out: a row
of zeros, a loss of zero, no gradient. A (M x K) holds tokens and B (V x K) the
vocabulary's rows, both BF16; sums are taken in FP32 or wider.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5


def listed():
    return [
        # Four sequences that decode one token each: latency counts.
        {"name": "embed_4_tokens", "op": "embed", "tokens": 4, "vocab": 128000, "cols": 4096, "e": "bf16", "y": "bf16",
         "id64": True, "skip": 0.0},
        # A training batch into an FP32 stream of residuals.
        {"name": "embed_16384", "op": "embed", "tokens": 16384, "vocab": 128000, "cols": 4096, "e": "bf16", "y": "fp32",
         "id64": True, "skip": 0.0},
        # A ragged batch with padding, its gradient added to the one that the
        # tied output projection has left.
        {"name": "embed_bwd_ragged", "op": "embed_bwd", "tokens": 777, "vocab": 32001, "cols": 1000, "e": "bf16",
         "y": "bf16", "id64": False, "skip": 0.1, "base": True},
        # A training batch's gradient of a large table.
        {"name": "embed_bwd_16384", "op": "embed_bwd", "tokens": 16384, "vocab": 128000, "cols": 4096, "e": "bf16",
         "y": "bf16", "id64": True, "skip": 0.0, "base": False},
        # One token while serving.
        {"name": "norm_1_token", "op": "norm", "rows": 1, "cols": 4096, "x": "bf16", "w": "bf16"},
        # A training batch.
        {"name": "norm_8192", "op": "norm", "rows": 8192, "cols": 4096, "x": "bf16", "w": "bf16"},
        # A small layer's gradients, stream and weights in FP32, at an odd
        # number of tokens.
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 301, "cols": 1000, "x": "fp32", "w": "fp32", "res": True},
        # A training batch's gradients, the residual's added.
        {"name": "norm_bwd_8192", "op": "norm_bwd", "rows": 8192, "cols": 4096, "x": "bf16", "w": "bf16", "res": True},
        # One token's score while serving: the vocabulary's rows are read once.
        {"name": "ce_1_token", "op": "ce", "M": 1, "V": 128000, "K": 4096, "id64": True, "skip": 0.0},
        # A training or evaluation batch.
        {"name": "ce_8192", "op": "ce", "M": 8192, "V": 128000, "K": 4096, "id64": True, "skip": 0.0},
        # A ragged batch of a small model, a quarter of it padding, an odd
        # vocabulary.
        {"name": "ce_bwd_ragged", "op": "ce_bwd", "M": 333, "V": 32001, "K": 1032, "id64": False, "skip": 0.25},
        # A training batch's gradients.
        {"name": "ce_bwd_4096", "op": "ce_bwd", "M": 4096, "V": 128000, "K": 4096, "id64": True, "skip": 0.0},
    ]


def _log_size(rng, low, high, of=1):
    """A multiple of `of` in low .. high, spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / of)) * of))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "norm", "norm_bwd", "ce", "ce_bwd"])
    if op.startswith("norm"):
        case = {"op": op, "rows": _log_size(rng, 1, 8192), "cols": _log_size(rng, 64, 8192, 8),
                "x": rng.choice(["bf16", "bf16", "fp32"]), "w": rng.choice(["bf16", "fp32"])}
        while case["rows"] * case["cols"] * (2 if case["x"] == "fp32" else 1) > 8192 * 4096:
            case["rows"] = (case["rows"] + 1) // 2
        if op == "norm_bwd":
            case["res"] = rng.random() < 0.6
        return case
    if op.startswith("embed"):
        case = {"op": op, "tokens": _log_size(rng, 1, 16384), "vocab": _log_size(rng, 64, 128000),
                "cols": _log_size(rng, 64, 4096, 8), "e": rng.choice(["bf16", "bf16", "fp32"]),
                "y": rng.choice(["bf16", "fp32"]), "id64": rng.random() < 0.6, "skip": rng.choice([0.0, 0.1])}
        if op == "embed_bwd":
            case["base"] = rng.random() < 0.5
            while case["vocab"] * case["cols"] * (2 if case["e"] == "fp32" else 1) * (2 if case["base"] else 1) > 128000 * 4096:
                case["vocab"] = case["vocab"] // 2
        return case
    case = {"op": op, "M": _log_size(rng, 1, 8192), "V": _log_size(rng, 64, 128000), "K": _log_size(rng, 64, 4096, 8),
            "id64": rng.random() < 0.6, "skip": rng.choice([0.0, 0.1, 0.5])}
    if op == "ce_bwd":
        case["M"] = min(case["M"], 4096)
    return case


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float64)


def _ids(gen, n, vocab, skip, id64):
    """Token ids as text has them, the k-th most frequent about 1 / k as often
    as the first, and -100 for a share of padding."""
    ids = torch.exp(_uniform(gen, n) * math.log(vocab + 1)).long() - 1
    ids = ids.clamp(0, vocab - 1) * 7919 % vocab      # frequent ones apart
    ids = torch.where(_uniform(gen, n) < skip, torch.full_like(ids, -100), ids)
    return ids if id64 else ids.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s, op = dict(case), case["op"]
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, device="cuda", dtype=dtype)
    if op.startswith("embed"):
        T, V, K = case["tokens"], case["vocab"], case["cols"]
        e, y = _TYPES[case["e"]], _TYPES[case["y"]]
        s["ids"] = _ids(gen, T, V, case["skip"], case["id64"])
        s["scale"] = math.sqrt(K)
        if op == "embed":
            s["E"] = _normal(gen, V, K, std=0.02, dtype=e)
            s["Y"] = new(T, K, dtype=y)
        else:
            s["dY"] = _normal(gen, T, K, std=2.0 ** -12, dtype=y)
            s["R"] = _normal(gen, V, K, std=2.0 ** -8, dtype=e) if case["base"] else None
            s["dE"] = new(V, K, dtype=e)
    elif op.startswith("norm"):
        r, c = case["rows"], case["cols"]
        x, w = _TYPES[case["x"]], _TYPES[case["w"]]
        # a stream of residuals: rows of different sizes, off centre
        size = torch.exp(_normal(gen, r, 1, std=0.5, dtype=torch.float32))
        s["X"] = ((_normal(gen, r, c, dtype=torch.float32) + 0.3) * size).to(x)
        s["gamma"] = (1 + _normal(gen, c, std=0.2, dtype=torch.float32)).to(w)
        if op == "norm":
            s["beta"] = _normal(gen, c, std=0.1, dtype=w)
            s["Y"], s["mean"], s["rstd"] = new(r, c), new(r, dtype=torch.float32), new(r, dtype=torch.float32)
        else:
            f = s["X"].double()
            s["mean"] = f.mean(1).float()
            s["rstd"] = (1 / torch.sqrt(f.var(1, correction=0) + EPS)).float()
            s["dY"] = _normal(gen, r, c, std=2.0 ** -8)
            s["R"] = _normal(gen, r, c, std=2.0 ** -8, dtype=x) if case["res"] else None
            s["dX"], s["dgamma"], s["dbeta"] = new(r, c, dtype=x), new(c, dtype=w), new(c, dtype=w)
    else:
        M, V, K = case["M"], case["V"], case["K"]
        s["B"] = _normal(gen, V, K, std=2 * K ** -0.5)
        s["targets"] = _ids(gen, M, V, case["skip"], case["id64"])
        # tokens that the network has learnt to different degrees: the target's
        # logit raised by 0 to 12
        at = s["targets"].long().clamp(min=0)
        s["A"] = (torch.randn(M, K, generator=gen, device="cuda") +
                  _uniform(gen, M, 1).float() * 3 * s["B"][at].float()).to(torch.bfloat16)
        if op == "ce":
            s["loss"], s["lse"] = new(M, dtype=torch.float32), new(M, dtype=torch.float32)
        else:
            kept = s["targets"] >= 0
            s["dloss"] = kept.float() / kept.sum().clamp(min=1)     # of the mean over the rows
            s["lse"] = torch.where(kept, _lse_of(s["A"], s["B"]), 0.0)
            s["dA"], s["dB"] = new(M, K), new(V, K)
    if own:
        import dense_gemm_14_amd as lib
        s["lib"] = lib
        nbytes = {"embed_bwd": lambda: lib.embedding_bwd_workspace_size(case["tokens"], case["vocab"], case["cols"]),
                  "norm_bwd": lambda: lib.layer_norm_bwd_workspace_size(case["rows"], case["cols"]),
                  "ce": lambda: lib.cross_entropy_workspace_size(case["M"], case["V"], case["K"]),
                  "ce_bwd": lambda: lib.cross_entropy_bwd_workspace_size(case["M"], case["V"], case["K"])}.get(op, int)()
        s["ws"] = torch.empty(nbytes, device="cuda", dtype=torch.uint8) if nbytes else None
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    lib, op, ws = s["lib"], s["op"], s["ws"]
    if op == "embed":
        lib.embedding(s["tokens"], s["vocab"], s["cols"], s["ids"], s["E"], s["Y"], s["scale"])
        return {"Y": s["Y"]}
    if op == "embed_bwd":
        lib.embedding_bwd(s["tokens"], s["vocab"], s["cols"], s["ids"], s["dY"], s["R"], s["dE"], s["scale"], ws)
        return {"dE": s["dE"]}
    if op == "norm":
        lib.layer_norm(s["rows"], s["cols"], s["X"], s["gamma"], s["beta"], s["Y"], s["mean"], s["rstd"], EPS)
        return {"Y": s["Y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_bwd":
        lib.layer_norm_bwd(s["rows"], s["cols"], s["X"], s["gamma"], s["mean"], s["rstd"], s["dY"], s["R"], s["dX"],
                           s["dgamma"], s["dbeta"], ws)
        return {"dX": s["dX"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "ce":
        lib.gemm_bf16_nt_cross_entropy(s["M"], s["V"], s["K"], s["A"], s["B"], s["targets"], s["loss"], s["lse"], ws)
        return {"loss": s["loss"], "lse": s["lse"]}
    lib.gemm_bf16_nt_cross_entropy_bwd(s["M"], s["V"], s["K"], s["A"], s["B"], s["targets"], s["lse"], s["dloss"],
                                       s["dA"], s["dB"], ws)
    return {"dA": s["dA"], "dB": s["dB"]}


# ---- plain forms -------------------------------------------------------------


def _lse_of(A, B):
    """log sum exp of each row of A B^T, which the forward pass leaves."""
    z = A.float() @ B.float().t()
    top = z.amax(1, keepdim=True)
    return top[:, 0] + torch.log(torch.exp(z - top).sum(1))


def _run_plain(s):
    op = s["op"]
    if op == "embed":
        kept = (s["ids"] >= 0)[:, None]
        y = torch.where(kept, s["scale"] * s["E"][s["ids"].long().clamp(min=0)].float(), 0.0)
        return {"Y": y.to(s["Y"].dtype)}
    if op == "embed_bwd":
        kept = (s["ids"] >= 0)[:, None]
        dy = torch.where(kept, s["scale"] * s["dY"].float(), 0.0)
        de = torch.zeros(s["vocab"], s["cols"], device="cuda")
        de.index_add_(0, s["ids"].long().clamp(min=0), dy)
        if s["R"] is not None:
            de = de + s["R"].float()
        return {"dE": de.to(s["dE"].dtype)}
    if op == "norm":
        x = s["X"].float()
        mean = x.sum(1) / s["cols"]
        d = x - mean[:, None]
        rstd = 1 / torch.sqrt((d * d).sum(1) / s["cols"] + EPS)
        y = d * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        return {"Y": y.to(torch.bfloat16), "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        n = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dY"].float()
        g = dy * s["gamma"].float()
        dx = s["rstd"][:, None] * (g - g.sum(1, keepdim=True) / s["cols"] - n * ((g * n).sum(1, keepdim=True) / s["cols"]))
        if s["R"] is not None:
            dx = dx + s["R"].float()
        return {"dX": dx.to(s["dX"].dtype), "dgamma": (dy * n).sum(0).to(s["dgamma"].dtype),
                "dbeta": dy.sum(0).to(s["dbeta"].dtype)}
    a, b, t = s["A"].float(), s["B"].float(), s["targets"].long()
    kept, at = t >= 0, t.clamp(min=0)[:, None]
    z = a @ b.t()
    if op == "ce":
        top = z.amax(1, keepdim=True)
        lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
        loss = lse - z.gather(1, at)[:, 0]
        return {"loss": torch.where(kept, loss, 0.0), "lse": torch.where(kept, lse, 0.0)}
    dz = torch.exp(z - s["lse"][:, None])
    dz.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    dz *= torch.where(kept, s["dloss"], 0.0)[:, None]
    return {"dA": (dz @ b).to(torch.bfloat16), "dB": (dz.t() @ a).to(torch.bfloat16)}


# ---- definitions in 64 bits --------------------------------------------------


def exact(case, seed):
    """The same outputs from the operators' definitions in 64 bits."""
    s, op = prepare(case, seed), case["op"]
    if op in ("embed", "embed_bwd"):
        keep = torch.nonzero(s["ids"] >= 0)[:, 0]
        rows = s["ids"][keep].long()
        if op == "embed":
            out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
            out[keep] = s["E"][rows].double() * math.sqrt(case["cols"])
            return {"Y": out}
        # tokens of one id side by side, their sum the difference of two
        # running sums
        order = torch.argsort(rows, stable=True)
        dy = s["dY"][keep][order].double()
        found, count = torch.unique_consecutive(rows[order], return_counts=True)
        total = torch.cat([torch.zeros(1, case["cols"], dtype=torch.float64, device="cuda"), dy.cumsum(0)])
        end = count.cumsum(0)
        out = torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device="cuda")
        if s["R"] is not None:
            out += s["R"]
        out[found] += (total[end] - total[end - count]) * math.sqrt(case["cols"])
        return {"dE": out}
    if op == "norm":
        x = s["X"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        return {"Y": torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], s["gamma"].double()),
                "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        # through the definition's own derivatives, row statistics included
        x = s["X"].double().requires_grad_()
        gamma = s["gamma"].double().requires_grad_()
        beta = torch.zeros_like(gamma).requires_grad_()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + EPS) * gamma + beta
        dx, dg, db = torch.autograd.grad(y, (x, gamma, beta), s["dY"].double())
        return {"dX": dx if s["R"] is None else dx + s["R"].double(), "dgamma": dg, "dbeta": db}
    M, V = case["M"], case["V"]
    b = s["B"].double()
    keep = torch.nonzero(s["targets"] >= 0)[:, 0]
    first, second = (torch.zeros(M, dtype=torch.float64, device="cuda") for _ in range(2)) if op == "ce" else (
        torch.zeros(M, case["K"], dtype=torch.float64, device="cuda"), torch.zeros_like(b))
    for rows in keep.split(max(1, (1 << 28) // V)):
        a, t = s["A"][rows].double(), s["targets"][rows].long()
        logp = torch.mm(a, b.t())
        if op == "ce":
            lse = torch.logsumexp(logp, 1)
            second[rows] = lse
            first[rows] = lse - logp[torch.arange(len(rows), device="cuda"), t]
        else:
            p = torch.softmax(logp, 1)
            p[torch.arange(len(rows), device="cuda"), t] -= 1
            p *= s["dloss"][rows, None].double()
            first[rows] = torch.mm(p, b)
            second += torch.mm(p.t(), a)
    return {"loss": first, "lse": second} if op == "ce" else {"dA": first, "dB": second}


def _distinct(tokens, vocab):
    """How many different ids `tokens` of _ids have on average."""
    edge = np.log(np.arange(1, vocab + 2, dtype=np.float64)) / math.log(vocab + 1)
    return float(-np.expm1(tokens * np.log1p(-np.minimum(np.diff(edge), 1 - 1e-12))).sum())


def work(case):
    op, size = case["op"], {"bf16": 2, "fp32": 4}
    if op.startswith("embed"):
        T, V, K = case["tokens"], case["vocab"], case["cols"]
        kept, ids = T * (1 - case["skip"]), T * (8 if case["id64"] else 4)
        if op == "embed":
            rows = _distinct(kept, V)
            return {"bytes": ids + rows * K * size[case["e"]] + T * K * size[case["y"]], "flops": kept * K}
        return {"bytes": ids + kept * K * size[case["y"]] + V * K * size[case["e"]] * (2 if case["base"] else 1),
                "flops": 2 * kept * K}
    if op.startswith("norm"):
        n, x, w = case["rows"] * case["cols"], size[case["x"]], size[case["w"]]
        if op == "norm":
            return {"bytes": n * (x + 2) + 2 * case["cols"] * w + 8 * case["rows"], "flops": 7 * n}
        return {"bytes": n * (2 * x + 2 + (x if case["res"] else 0)) + 3 * case["cols"] * w + 8 * case["rows"],
                "flops": 13 * n}
    M, V, K = case["M"], case["V"], case["K"]
    kept = M * (1 - case["skip"])
    targets = M * (8 if case["id64"] else 4)
    if op == "ce":
        return {"bytes": 2 * (kept * K + V * K) + targets + 8 * M, "flops": 2 * kept * V * K}
    # the logits, which nobody has kept, and the two products with their gradient
    return {"bytes": 2 * (kept * K + V * K) + 2 * (M * K + V * K) + targets + 8 * M, "flops": 6 * kept * V * K}
