"""Cases for measuring the layer operators: a linear layer with bias,
activation and residual, forward and backward; a gated pair of projections,
forward and backward; the Muon update of a list of matrices.

A scene's attributes may come out of a small network instead of being held per
Gaussian: rows of features (looked up in a table, one row per Gaussian) pass
through linear and gated layers and become SH coefficients or opacities.  The
layers' matrices are trained by orthogonalised momentum, everything else by
Adam.  The same operators serve the layers of language models: wide 16-bit
matrices, a batch of tokens or a single one.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NS_A, NS_B, NS_C, NS_STEPS, NS_EPS = 3.4445, -4.7750, 2.0315, 5, 1e-7
LR, MOMENTUM = 0.02, 0.95


def listed():
    return [
        # one new token through a layer with a residual: a serving step, where the weights' bytes count
        dict(name="linear_step", op="linear", rows=1, ins=4096, outs=4096, type="bf16", act="none", bias=True,
             residual=True, pre=False),
        # SH coefficients (degree 3) of a million Gaussians from 32 features each
        dict(name="linear_scene", op="linear", rows=1_000_000, ins=32, outs=48, type="f32", act="none", bias=True,
             residual=False, pre=False),
        # a training batch of tokens through the first matrix of a feed-forward block
        dict(name="linear_batch", op="linear", rows=8192, ins=4096, outs=11008, type="bf16", act="gelu", bias=True,
             residual=False, pre=True),
        # a few hundred visible Gaussians through a narrow hidden layer
        dict(name="linear_bwd_small", op="linear_bwd", rows=257, ins=35, outs=64, type="f32", act="silu", bias=True),
        # a hidden layer of a million Gaussians' network
        dict(name="linear_bwd_scene", op="linear_bwd", rows=1_000_000, ins=32, outs=64, type="f32", act="relu",
             bias=True),
        # the batch's backward pass, odd sizes throughout
        dict(name="linear_bwd_odd", op="linear_bwd", rows=8191, ins=2049, outs=4097, type="f16", act="gelu",
             bias=True),
        # four sequences take one token each
        dict(name="gated_step", op="gated", rows=4, ins=4096, outs=11008, type="bf16", act="silu", pre=False),
        # a training batch of tokens
        dict(name="gated_batch", op="gated", rows=8192, ins=4096, outs=11008, type="bf16", act="silu", pre=True),
        # its backward pass at half the width
        dict(name="gated_bwd_batch", op="gated_bwd", rows=8192, ins=2048, outs=5504, type="bf16", act="silu"),
        # the matrices of a narrow network over Gaussian features
        dict(name="muon_small", op="muon", count=4, rows=64, cols=48, grad="f32", copy="none", decay=0.0,
             nesterov=True),
        # tall matrices with an odd side, 16-bit gradients and 16-bit copies for the next pass
        dict(name="muon_tall", op="muon", count=24, rows=2048, cols=515, grad="bf16", copy="bf16", decay=0.01,
             nesterov=True),
        # square matrices of wide layers
        dict(name="muon_wide", op="muon", count=3, rows=4096, cols=4096, grad="f32", copy="none", decay=0.1,
             nesterov=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "gated", "gated_bwd", "muon"])
    if op == "muon":
        rows, cols = _log(rng, 8, 4096), _log(rng, 8, 4096)
        side = min(rows, cols)
        most = max(1, min(48, int(2e11 // (side * rows * cols + 1))))
        return dict(op=op, count=rng.randint(1, most), rows=rows, cols=cols, grad=rng.choice(["f32", "f32", "f16", "bf16"]),
                    copy=rng.choice(["none", "bf16", "f16"]), decay=rng.choice([0.0, 0.01]),
                    nesterov=rng.choice([True, True, False]))
    # narrow layers over many Gaussians, wide ones over tokens
    if rng.random() < 0.4:
        ins, outs = rng.choice([_log(rng, 3, 256), 16 * rng.randint(1, 8)]), rng.choice([_log(rng, 3, 256), 48, 64])
        most = 1_000_000
    else:
        ins = rng.choice([_log(rng, 64, 8192), 128 * rng.randint(1, 40)])
        outs = rng.choice([_log(rng, 64, 11008), 128 * rng.randint(1, 64)])
        most = 16384
    most = min(most, int(3.5e11 // (ins * outs)), 200_000_000 // (ins + 2 * outs))
    kind = rng.choice(["f32", "f16", "bf16"])
    if op.startswith("gated"):
        c = dict(op=op, rows=_log(rng, 1, max(1, most // 2)), ins=ins, outs=outs, type=kind,
                 act=rng.choice(["silu", "gelu", "relu", "sigmoid"]))
        if op == "gated":
            c.update(pre=rng.choice([True, False]))
        return c
    c = dict(op=op, rows=_log(rng, 1, most), ins=ins, outs=outs, type=kind,
             act=rng.choice(["none", "relu", "silu", "gelu", "sigmoid"]), bias=rng.choice([True, True, False]))
    if op == "linear":
        c.update(residual=rng.choice([True, False]), pre=c["act"] != "none" and rng.random() < 0.5)
    return c


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    s = {"case": c}

    def normal(shape, scale, dtype):
        return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)

    if c["op"] == "muon":
        shape = (c["count"], c["rows"], c["cols"])
        s["params"] = normal(shape, 0.02, torch.float32)
        s["m"] = normal(shape, 0.01, torch.float32)
        s["grads"] = normal(shape, 0.01, TYPES[c["grad"]])
        s["copies"] = None if c["copy"] == "none" else torch.zeros(shape, dtype=TYPES[c["copy"]], device=DEV)
        return s
    t = TYPES[c["type"]]
    n, k, f = c["rows"], c["ins"], c["outs"]
    both = f * (2 if c["op"].startswith("gated") else 1)   # gate rows, then up rows
    s["x"] = normal((n, k), 1.0, t)
    s["w"] = normal((both, k), k ** -0.5, t)
    s["bias"] = normal((both,), 0.1, torch.float32) if c.get("bias") else None
    if c["op"].endswith("_bwd"):
        s["pre"] = _pre(s)
        s["dout"] = normal((n, f), 0.1, t)
        s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
        s["dbias"] = torch.empty_like(s["bias"]) if c.get("bias") else None
    else:
        s["residual"] = normal((n, f), 1.0, t) if c.get("residual") else None
        s["out"] = torch.empty((n, f), dtype=t, device=DEV)
        s["pre"] = torch.empty((n, both), dtype=t, device=DEV) if c["pre"] else None
    return s


def _pre(s):
    """What the forward pass of these inputs keeps: x w^T + bias in the inputs' type."""
    z = torch.matmul(s["x"].float(), s["w"].float().t())
    return (z if s["bias"] is None else z + s["bias"]).to(s["x"].dtype)


# ---------------------------------------------------------------------------- one pass

_context = []


def _ctx():
    import differentiable_gaussian_splatting_amd as dgs
    if not _context:
        _context.append(dgs.Context())
    return dgs, _context[0]


GELU_S, GELU_C = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    return z / (1.0 + torch.exp(-2.0 * GELU_S * (z + GELU_C * z * z * z)))


def _slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        p = 1.0 / (1.0 + torch.exp(-2.0 * GELU_S * (z + GELU_C * z * z * z)))
        return p + z * p * (1.0 - p) * 2.0 * GELU_S * (1.0 + 3.0 * GELU_C * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 - p) if act == "sigmoid" else p + z * p * (1.0 - p)


def run(s):
    c = s["case"]
    if own:
        dgs, ctx = _ctx()
        if c["op"] == "linear":
            dgs.gs_linear_fwd(ctx, s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], pre=s["pre"],
                              out=s["out"])
            return [s["out"]] + ([s["pre"]] if c["pre"] else [])
        if c["op"] == "linear_bwd":
            dgs.gs_linear_bwd(ctx, s["x"], s["w"], s["dout"], pre=s["pre"], act=c["act"], dx=s["dx"], dw=s["dw"],
                              dbias=s["dbias"])
            return [s["dx"], s["dw"]] + ([s["dbias"]] if c["bias"] else [])
        if c["op"] == "gated":
            dgs.gs_gated_fwd(ctx, s["x"], s["w"], act=c["act"], pre=s["pre"], out=s["out"])
            return [s["out"]] + ([s["pre"]] if c["pre"] else [])
        if c["op"] == "gated_bwd":
            dgs.gs_gated_bwd(ctx, s["x"], s["w"], s["pre"], s["dout"], act=c["act"], dx=s["dx"], dw=s["dw"])
            return [s["dx"], s["dw"]]
        if "lists" not in s:   # a training program describes its buffers once
            s["lists"] = {k: dgs.TensorList(list(s[k])) for k in ("params", "m", "grads", "copies") if s[k] is not None}
        L = s["lists"]
        dgs.gs_muon_tensors(ctx, L["params"], L["m"], L["grads"], lr=LR, momentum=MOMENTUM, nesterov=c["nesterov"],
                            weight_decay=c["decay"], steps=NS_STEPS, copies=L.get("copies"))
        return [s["params"], s["m"]] + ([] if s["copies"] is None else [s["copies"]])

    if c["op"] == "muon":
        g = s["grads"].float()
        s["m"].mul_(MOMENTUM).add_(g)
        x = g + MOMENTUM * s["m"] if c["nesterov"] else s["m"].clone()
        x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + NS_EPS)
        x = _newton_schulz(x if c["rows"] <= c["cols"] else x.transpose(1, 2).contiguous(), NS_STEPS)
        x = x if c["rows"] <= c["cols"] else x.transpose(1, 2)
        s["params"].mul_(1.0 - LR * c["decay"]).sub_(x * (LR * math.sqrt(max(1.0, c["rows"] / c["cols"]))))
        if s["copies"] is None:
            return [s["params"], s["m"]]
        s["copies"].copy_(s["params"])
        return [s["params"], s["m"], s["copies"]]
    t, f = s["x"].dtype, c["outs"]
    x, w = s["x"].float(), s["w"].float()
    if c["op"] in ("linear", "gated"):
        z = torch.matmul(x, w.t())
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, c["act"]) if c["op"] == "linear" else _act(z[:, :f], c["act"]) * z[:, f:]
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(t)] + ([z.to(t)] if c["pre"] else [])
    z, d = s["pre"].float(), s["dout"].float()
    if c["op"] == "linear_bwd":
        dz = d * _slope(z, c["act"])
    else:
        dz = torch.cat([d * z[:, f:] * _slope(z[:, :f], c["act"]), d * _act(z[:, :f], c["act"])], 1)
    out = [torch.matmul(dz, w).to(t), torch.matmul(dz.t(), x).to(t)]
    return out + ([dz.sum(0)] if c.get("bias") else [])


def _newton_schulz(x, left):
    """`left` steps of x = a x + (b G + c G^2) x with G = x x^T, for a stack of matrices no taller than wide."""
    if left == 0:
        return x
    gram = torch.bmm(x, x.transpose(1, 2).contiguous())
    poly = NS_B * gram + NS_C * torch.bmm(gram, gram)
    return _newton_schulz(NS_A * x + torch.bmm(poly, x), left - 1)


def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2, "none": 0}
    if c["op"] == "muon":
        n, side = c["rows"] * c["cols"], min(c["rows"], c["cols"])
        # G and G^2 are symmetric: half of their products are enough
        step = side * n + side ** 3 + 2 * side * n
        return {"bytes": c["count"] * n * (16 + size[c["grad"]] + size[c["copy"]]), "flops": c["count"] * NS_STEPS * step}
    e, n, k, f = size[c["type"]], c["rows"], c["ins"], c["outs"]
    both = f * (2 if c["op"].startswith("gated") else 1)
    weights = both * k * e + (4 * both if c.get("bias") else 0)
    if c["op"].endswith("_bwd"):
        kept = 0 if c["act"] == "none" else n * both * e
        return {"bytes": 2 * n * k * e + 2 * weights + kept + n * f * e, "flops": 4 * n * k * both}
    rows = n * k + n * f + (n * f if c.get("residual") else 0) + (n * both if c["pre"] else 0)
    return {"bytes": weights + rows * e, "flops": 2 * n * k * both}


# ---------------------------------------------------------------------------- the definition in 64 bits

def _exact_act(z, act):
    """Value and slope of the activation."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":   # 1/2 z (1 + tanh u)
        u = GELU_S * (z + GELU_C * z ** 3)
        h = torch.tanh(u)
        return 0.5 * z * (1 + h), 0.5 * (1 + h) + 0.5 * z * (1 - h * h) * GELU_S * (1 + 3 * GELU_C * z * z)
    p = torch.sigmoid(z)
    return (p, p * (1 - p)) if act == "sigmoid" else (z * p, p * (1 + z * (1 - p)))


def exact(case, seed):
    s = prepare(case, seed)
    c, f = s["case"], case.get("outs")
    if c["op"] == "muon":
        ps, ms = [], []
        for p, m, g in zip(s["params"].double(), s["m"].double(), s["grads"].double()):
            m = MOMENTUM * m + g
            u = m if not c["nesterov"] else g + MOMENTUM * m
            x = u / (u.norm() + NS_EPS)
            for _ in range(NS_STEPS):
                if c["rows"] <= c["cols"]:
                    a = x @ x.T
                    x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
                else:
                    a = x.T @ x
                    x = NS_A * x + x @ (NS_B * a + NS_C * (a @ a))
            ps.append(p - LR * c["decay"] * p - LR * max(1.0, c["rows"] / c["cols"]) ** 0.5 * x)
            ms.append(m)
        ps, ms = torch.stack(ps), torch.stack(ms)
        return [ps, ms] + ([ps] if s["copies"] is not None else [])
    x, w = s["x"].double(), s["w"].double()
    if c["op"] in ("linear", "gated"):
        z = x @ w.T
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(z, c["act"])[0] if c["op"] == "linear" else _exact_act(z[:, :f], c["act"])[0] * z[:, f:]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return [y] + ([z] if c["pre"] else [])
    z, d = s["pre"].double(), s["dout"].double()
    if c["op"] == "linear_bwd":
        dz = d * _exact_act(z, c["act"])[1]
    else:
        a, slope = _exact_act(z[:, :f], c["act"])
        dz = torch.cat([d * z[:, f:] * slope, d * a], 1)
    return [dz @ w, dz.T @ x] + ([dz.sum(0)] if c.get("bias") else [])
