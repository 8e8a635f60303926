"""What is measured of the embedding-head operators: the matrix product with its epilogue,
layer norm, and the balance loss over cells, each in both directions.

`run` computes an operator in plain torch (fp32 arithmetic, rounded once) or, where `own`
is true, through this repository's binding.  `exact` is the definition in fp64.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


def listed():
    return [
        # One query's hidden state through the projection of a search front end: latency.
        dict(name="linear_one_query", op="linear", dtype="bf16", rows=1, depth=768, cols=768,
             act="none", residual=False, save=False),
        # A batch of queries scored against every cell of the 4096-cell index (bias = the
        # centroids' half norms), fp32 points: ragged rows.
        dict(name="linear_scores_f32", op="linear", dtype="f32", rows=2500, depth=768, cols=4096,
             act="none", residual=False, save=False),
        # The expanding product of a head in training: GELU, pre-activation kept.
        dict(name="linear_gelu_train", op="linear", dtype="bf16", rows=10000, depth=768,
             cols=4096, act="gelu", residual=False, save=True),
        # A corpus encoded in one go: the largest product, with its residual.
        dict(name="linear_corpus", op="linear", dtype="bf16", rows=65536, depth=4096, cols=4096,
             act="silu", residual=True, save=False),
        # Gradients of a small head with odd sizes, fp32.
        dict(name="linear_backward_odd_f32", op="linear_backward", dtype="f32", rows=1001,
             depth=300, cols=129, act="relu"),
        # Gradients of the expanding product over a long batch.
        dict(name="linear_backward_train", op="linear_backward", dtype="bf16", rows=65536,
             depth=768, cols=4096, act="gelu"),
        # The norm in front of one small batch of queries: latency.
        dict(name="layer_norm_queries", op="layer_norm", dtype="bf16", rows=50, depth=768),
        # A corpus normalised before it is clustered.
        dict(name="layer_norm_corpus", op="layer_norm", dtype="f32", rows=262144, depth=768),
        # Gradients of the norm over odd rows, fp32.
        dict(name="layer_norm_backward_odd_f32", op="layer_norm_backward", dtype="f32",
             rows=10007, depth=129),
        # Gradients of the norm at a wide hidden size, long batch.
        dict(name="layer_norm_backward_train", op="layer_norm_backward", dtype="bf16",
             rows=65536, depth=4096),
        # A router's balance term: two of 64 experts a token, some padding rows.
        dict(name="balance_experts", op="balance", dtype="f32", rows=8192, cells=64, top=2,
             pad=0.05),
        # Rows balanced over the 4096 cells of an index, one cell a row.
        dict(name="balance_cells", op="balance", dtype="bf16", rows=65536, cells=4096, top=1,
             pad=0.0),
    ]


def _log_size(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "layer_norm",
                     "layer_norm_backward", "balance"])
    case = dict(op=op, dtype=rng.choice(["bf16", "f32"]), rows=_log_size(rng, 1, 65536))
    if op in ("linear", "linear_backward"):
        case["depth"] = _log_size(rng, 16, 4096)
        case["cols"] = _log_size(rng, 16, 4096)
        if rng.random() < 0.6:  # most real sizes are multiples of eight
            case["depth"] = max(16, case["depth"] // 8 * 8)
            case["cols"] = max(16, case["cols"] // 8 * 8)
        case["act"] = rng.choice(["none", "relu", "gelu", "silu"])
        if op == "linear":
            case["residual"] = rng.random() < 0.5
            case["save"] = rng.random() < 0.5
        most = (1 << 39) // (case["depth"] * case["cols"])
        case["rows"] = max(1, min(case["rows"], most))
    elif op in ("layer_norm", "layer_norm_backward"):
        case["depth"] = _log_size(rng, 1, 8192)
        if rng.random() < 0.6:
            case["depth"] = (case["depth"] + 7) // 8 * 8
        case["rows"] = max(1, min(case["rows"], (1 << 28) // case["depth"]))
    else:
        case["cells"] = _log_size(rng, 2, 8192)
        case["top"] = rng.randint(1, min(8, case["cells"]))
        case["rows"] = max(1, min(case["rows"], (1 << 28) // case["cells"]))
        case["pad"] = rng.choice([0.0, 0.1, 0.5])
    return case


# ------------------------------------------------------------------------------- inputs

def _normal(gen, shape, dtype, scale=1.0, shift=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (t * scale + shift).to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _TYPES[case["dtype"]]
    n = case["rows"]
    if case["op"] in ("linear", "linear_backward"):
        d, m = case["depth"], case["cols"]
        s = {"X": _normal(gen, (n, d), dtype),
             "W": _normal(gen, (m, d), dtype, d ** -0.5),
             "bias": _normal(gen, (m,), torch.float32, 0.1)}
        if case["op"] == "linear":
            s["R"] = _normal(gen, (n, m), dtype) if case["residual"] else None
        else:
            s["Z"] = None
            if case["act"] != "none":  # the pre-activation that the forward pass kept
                s["Z"] = (s["X"] @ s["W"].t() + s["bias"]).to(dtype)
            s["dY"] = _normal(gen, (n, m), dtype, 0.01)
        return s
    if case["op"] in ("layer_norm", "layer_norm_backward"):
        d = case["depth"]
        # hidden states: rows of differing scale with a common offset
        scale = torch.exp(0.5 * torch.randn((n, 1), generator=gen, device="cuda"))
        s = {"X": (torch.randn((n, d), generator=gen, device="cuda") * scale + 0.3).to(dtype),
             "gamma": _normal(gen, (d,), torch.float32, 0.1, 1.0),
             "beta": _normal(gen, (d,), torch.float32, 0.1)}
        if case["op"] == "layer_norm_backward":
            s["dY"] = _normal(gen, (n, d), dtype, 0.01)
            x = s["X"].double()  # the statistics that the forward pass kept
            mean = x.mean(1)
            var = ((x - mean[:, None]) ** 2).mean(1)
            s["mean"], s["rstd"] = mean.float(), (var + _EPS).rsqrt().float()
        return s
    k, top = case["cells"], case["top"]
    S = _normal(gen, (n, k), dtype, 1.5)
    # cells of uneven popularity: the selection is the top scores with a bias per cell
    bias = 0.5 * torch.randn((k,), generator=gen, device="cuda")
    lab = (S.float() + bias).topk(top, dim=1).indices.to(torch.int32)
    if case["pad"] > 0:
        lab[torch.rand((n,), generator=gen, device="cuda") < case["pad"]] = -1
    return {"S": S, "labels": lab.contiguous()}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from exact_lloyd_means_b200 import fk
        n = case["rows"]
        dtype = _TYPES[case["dtype"]]
        dev = "cuda"
        if case["op"] == "linear":
            d, m = case["depth"], case["cols"]
            s["Y"] = torch.empty((n, m), dtype=dtype, device=dev)
            s["Zout"] = torch.empty((n, m), dtype=dtype, device=dev) if case["save"] else None
            s["ws"] = fk.linear_workspace(n, d, m, dtype)
        elif case["op"] == "linear_backward":
            d, m = case["depth"], case["cols"]
            s["dX"] = torch.empty((n, d), dtype=dtype, device=dev)
            s["dW"] = torch.empty((m, d), dtype=dtype, device=dev)
            s["db"] = torch.empty((m,), dtype=torch.float32, device=dev)
            s["ws"] = fk.linear_backward_workspace(n, d, m, dtype)
        elif case["op"] == "layer_norm":
            d = case["depth"]
            s["Y"] = torch.empty((n, d), dtype=dtype, device=dev)
            s["mean"] = torch.empty((n,), dtype=torch.float32, device=dev)
            s["rstd"] = torch.empty((n,), dtype=torch.float32, device=dev)
        elif case["op"] == "layer_norm_backward":
            d = case["depth"]
            s["dX"] = torch.empty((n, d), dtype=dtype, device=dev)
            s["dgamma"] = torch.empty((d,), dtype=torch.float32, device=dev)
            s["dbeta"] = torch.empty((d,), dtype=torch.float32, device=dev)
            s["ws"] = fk.layer_norm_backward_workspace(n, d, dtype)
        else:
            k = case["cells"]
            s["counts"] = torch.empty((k,), dtype=torch.int32, device=dev)
            s["rows"] = torch.empty((1,), dtype=torch.int32, device=dev)
            s["loss"] = torch.empty((1,), dtype=torch.float32, device=dev)
            s["dS"] = torch.empty((n, k), dtype=dtype, device=dev)
            s["ws"] = fk.balance_workspace(n, k, dtype)
    return s


# ---------------------------------------------------------------------------- plain forms

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (
            2 * math.pi) ** -0.5
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain(s):
    case = s["case"]
    op, dtype = case["op"], _TYPES[case["dtype"]]
    if op == "linear":
        z = s["X"].float() @ s["W"].float().t() + s["bias"]
        y = _act(z, case["act"])
        if s["R"] is not None:
            y = y + s["R"].float()
        out = {"Y": y.to(dtype)}
        if case["save"]:
            out["Z"] = z.to(dtype)
        return out
    if op == "linear_backward":
        g = s["dY"].float()
        if case["act"] != "none":
            g = g * _act_slope(s["Z"].float(), case["act"])
        return {"dX": (g @ s["W"].float()).to(dtype), "dW": (g.t() @ s["X"].float()).to(dtype),
                "db": g.sum(0)}
    if op == "layer_norm":
        x = s["X"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1 / torch.sqrt((c * c).mean(1) + _EPS)
        y = c * rstd[:, None] * s["gamma"] + s["beta"]
        return {"Y": y.to(dtype), "mean": mean, "rstd": rstd}
    if op == "layer_norm_backward":
        x, dy = s["X"].float(), s["dY"].float()
        r = s["rstd"][:, None]
        h = (x - s["mean"][:, None]) * r
        w = dy * s["gamma"]
        dx = r * (w - w.mean(1, keepdim=True) - h * (w * h).mean(1, keepdim=True))
        return {"dX": dx.to(dtype), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}
    k, lab = case["cells"], s["labels"]
    kept = (lab >= 0).any(1)
    hit = torch.where(lab >= 0, lab, torch.full_like(lab, k)).long().reshape(-1)
    counts = torch.zeros(k + 1, dtype=torch.int32, device=lab.device)
    counts.index_add_(0, hit, torch.ones_like(hit, dtype=torch.int32))
    counts = counts[:k]
    n = kept.sum(dtype=torch.int32).reshape(1)
    nf = n.clamp(min=1).float()
    f = counts.float() / (nf * case["top"])
    x = s["S"].float()
    e = torch.exp(x - x.max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True) * kept[:, None]
    t = (p * f).sum(1, keepdim=True)
    loss = k / nf * t.sum()
    return {"counts": counts, "rows": n, "loss": loss.reshape(1),
            "dS": (k / nf * p * (f - t)).to(dtype)}


def _kernels(s):
    from exact_lloyd_means_b200 import fk
    case = s["case"]
    op = case["op"]
    if op == "linear":
        fk.fk_linear(s["X"], s["W"], s["Y"], s["ws"], bias=s["bias"], act=case["act"],
                     residual=s["R"], Z=s["Zout"])
        out = {"Y": s["Y"]}
        if case["save"]:
            out["Z"] = s["Zout"]
        return out
    if op == "linear_backward":
        fk.fk_linear_backward(s["dY"], s["X"], s["W"], s["ws"], act=case["act"], Z=s["Z"],
                              dX=s["dX"], dW=s["dW"], dbias=s["db"])
        return {"dX": s["dX"], "dW": s["dW"], "db": s["db"]}
    if op == "layer_norm":
        fk.fk_layer_norm(s["X"], s["gamma"], s["beta"], s["Y"], eps=_EPS, mean=s["mean"],
                         rstd=s["rstd"])
        return {"Y": s["Y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "layer_norm_backward":
        fk.fk_layer_norm_backward(s["dY"], s["X"], s["gamma"], s["mean"], s["rstd"], s["dX"],
                                  s["dgamma"], s["dbeta"], s["ws"])
        return {"dX": s["dX"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    fk.fk_balance_counts(s["labels"], s["counts"], s["rows"])
    fk.fk_balance_loss(s["S"], s["labels"], s["counts"], s["rows"], s["loss"], s["dS"],
                       s["ws"])
    return {"counts": s["counts"], "rows": s["rows"], "loss": s["loss"], "dS": s["dS"]}


def run(state):
    return _kernels(state) if own else _plain(state)


# --------------------------------------------------------------------------------- bounds

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["rows"]
    if case["op"] in ("linear", "linear_backward"):
        d, m = case["depth"], case["cols"]
        if case["op"] == "linear":
            outs = 1 + int(case["save"]) + int(case["residual"])
            return {"bytes": e * (n * d + m * d + outs * n * m) + 4 * m, "flops": 2 * n * d * m}
        ins = 1 + int(case["act"] != "none")
        return {"bytes": e * (2 * n * d + 2 * m * d + ins * n * m) + 4 * m,
                "flops": 4 * n * d * m}
    if case["op"] == "layer_norm":
        d = case["depth"]
        return {"bytes": 2 * e * n * d + 8 * d + 8 * n, "flops": 8 * n * d}
    if case["op"] == "layer_norm_backward":
        d = case["depth"]
        return {"bytes": 3 * e * n * d + 12 * d + 8 * n, "flops": 14 * n * d}
    k, top = case["cells"], case["top"]
    return {"bytes": 2 * e * n * k + 4 * n * top + 4 * k, "flops": 10 * n * k}


# ------------------------------------------------------------------------- the definition

def exact(case, seed):
    """The same outputs from the definition in fp64."""
    i = _inputs(case, seed)
    q = {key: v.double() for key, v in i.items() if v is not None and v.is_floating_point()}
    op = case["op"]
    if op in ("linear", "linear_backward"):
        cdf = lambda v: torch.special.ndtr(v)  # noqa: E731
        sig = lambda v: torch.sigmoid(v)  # noqa: E731
        act = case.get("act")
    if op == "linear":
        z = torch.addmm(q["bias"], q["X"], q["W"].t())
        y = z
        if act == "relu":
            y = z.clamp(min=0)
        elif act == "gelu":
            y = z * cdf(z)
        elif act == "silu":
            y = z * sig(z)
        if i["R"] is not None:
            y = y + q["R"]
        out = {"Y": y}
        if case["save"]:
            out["Z"] = z
        return out
    if op == "linear_backward":
        g = q["dY"]
        if act == "relu":
            g = torch.where(q["Z"] > 0, g, torch.zeros_like(g))
        elif act == "gelu":
            z = q["Z"]
            g = g * (cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        elif act == "silu":
            z = q["Z"]
            g = g * (sig(z) + z * sig(z) * sig(-z))
        return {"dX": torch.mm(g, q["W"]), "dW": torch.mm(g.t(), q["X"]), "db": g.sum(0)}
    if op == "layer_norm":
        x = q["X"]
        mean = x.mean(1, keepdim=True)
        var = ((x - mean).square()).mean(1, keepdim=True)
        rstd = (var + _EPS).rsqrt()
        return {"Y": (x - mean) * rstd * q["gamma"] + q["beta"], "mean": mean[:, 0],
                "rstd": rstd[:, 0]}
    if op == "layer_norm_backward":
        n, d = q["X"].shape
        hat = (q["X"] - q["mean"][:, None]) * q["rstd"][:, None]
        w = q["dY"] * q["gamma"][None]
        a, b = w.sum(1, keepdim=True), (w * hat).sum(1, keepdim=True)
        dx = q["rstd"][:, None] / d * (d * w - a - hat * b)
        return {"dX": dx, "dgamma": (q["dY"] * hat).sum(0), "dbeta": q["dY"].sum(0)}
    k, lab = case["cells"], i["labels"]
    kept = lab.max(1).values >= 0
    flat = lab.reshape(-1)
    counts = torch.bincount(flat[flat >= 0], minlength=k)
    n = int(kept.sum())
    f = counts.double() / (max(n, 1) * case["top"])
    p = torch.softmax(q["S"], 1)
    p[~kept] = 0
    c = k / max(n, 1)
    t = torch.mv(p, f)
    return {"counts": counts.to(torch.int32),
            "rows": torch.tensor([n], dtype=torch.int32, device=lab.device),
            "loss": (c * t.sum()).reshape(1), "dS": c * p * (f[None] - t[:, None])}
