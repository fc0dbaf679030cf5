"""Cases for measuring the table and update operators: a lookup of table rows
by index and its gradient, the global norm of a list of gradients with
clipping, and Adam over a list of tensors.

A scene of N Gaussians may hold its SH coefficients in a table of V rows with
an index per Gaussian; a training step then looks the rows up, renders a view,
sums the Gaussians' gradient rows into the table's gradient, clips the whole
gradient to a global norm and updates table and geometry.  The same operators
serve token tables (wide rows, 16-bit types) and parameter lists of layers.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BETA1, BETA2, EPS, LR = 0.9, 0.999, 1e-15, 1e-3


def listed():
    return [
        # 16 sequences take one token each: a serving step's lookup, where latency counts
        dict(name="fwd_step", op="fwd", tokens=16, vocab=32768, width=4096, type="bf16", index="i64", scale=64.0,
             spread="zipf", masked=0.0),
        # a prompt with masked positions, odd sizes throughout
        dict(name="fwd_odd", op="fwd", tokens=8191, vocab=50021, width=1027, type="f16", index="i64", scale=0.5,
             spread="zipf", masked=0.1),
        # the SH rows (degree 3) of a 6M-Gaussian scene from a table of 65536
        dict(name="fwd_scene", op="fwd", tokens=6_000_000, vocab=65536, width=48, type="f32", index="i32", scale=1.0,
             spread="codes", masked=0.0),
        # a few hundred visible Gaussians, SH without its first coefficient
        dict(name="bwd_small", op="bwd", tokens=257, vocab=4096, width=45, row=45, type="f32", grad="f32",
             index="i32", scale=1.0, spread="zipf", masked=0.0, padding=-1),
        # a training batch of tokens over a token table, its first row a padding row
        dict(name="bwd_prompt", op="bwd", tokens=16384, vocab=32768, width=4096, row=4096, type="bf16", grad="f32",
             index="i64", scale=64.0, spread="zipf", masked=0.0, padding=0),
        # the SH columns of a 6M-Gaussian view's gradient rows (59 values each); a quarter of the Gaussians share
        # the background's row
        dict(name="bwd_scene", op="bwd", tokens=6_000_000, vocab=65536, width=48, row=59, type="f32", grad="f32",
             index="i32", scale=1.0, spread="codes", masked=0.0, padding=-1),
        # the five groups of the smallest scene (2000 Gaussians, degree 0)
        dict(name="clip_small", op="clip", layout="scene", count=2000, sh=1, rows=0, type="f32", limit=1.0),
        # the 16-bit gradients of 220 layers in one flat buffer, odd sizes without padding between them
        dict(name="clip_layers", op="clip", layout="layers", count=220, sh=0, rows=900_001, type="bf16", limit=1.0),
        # the five groups of a 6M-Gaussian scene, degree 3
        dict(name="clip_scene", op="clip", layout="scene", count=6_000_000, sh=16, rows=0, type="f32", limit=1.0),
        # a small scene whose SH come from a table of 256 rows: geometry gradients are columns of the view's rows
        dict(name="adam_small", op="adam", layout="coded", count=2000, sh=1, rows=256, type="f32", copy="none",
             limit=1.0, decay=0.0, step=7),
        # 220 layers: 16-bit gradients, 32-bit weights and moments, a 16-bit copy of the weights for the next pass
        dict(name="adam_layers", op="adam", layout="layers", count=220, sh=0, rows=900_001, type="bf16", copy="bf16",
             limit=1.0, decay=0.01, step=1000),
        # the five groups of a 6M-Gaussian scene, degree 3
        dict(name="adam_scene", op="adam", layout="scene", count=6_000_000, sh=16, rows=0, type="f32", copy="none",
             limit=1.0, decay=0.0, step=100),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "clip", "adam"])
    if op in ("fwd", "bwd"):
        width = rng.choice([_log(rng, 1, 8192), 3 * rng.randint(1, 16), 64 * _log(rng, 1, 128)])
        c = dict(op=op, tokens=_log(rng, 1, min(6_000_000, 200_000_000 // width)),
                 vocab=_log(rng, 2, min(200_000, 150_000_000 // width)), width=width,
                 type=rng.choice(["f32", "f16", "bf16"]), index=rng.choice(["i32", "i64"]),
                 scale=rng.choice([1.0, 0.125, 64.0, rng.uniform(0.5, 2.0)]),
                 spread=rng.choice(["uniform", "zipf", "codes"]), masked=rng.choice([0.0, 0.0, 0.2]))
        if op == "bwd":
            c.update(row=rng.choice([width, width, width + rng.randint(1, 64)]), grad=rng.choice(["f32", c["type"]]),
                     padding=rng.choice([-1, 0]))
        return c
    layout = rng.choice(["scene", "layers", "coded"])
    c = dict(op=op, layout=layout, count=0, sh=0, rows=0, type=rng.choice(["f32", "f32", "f16", "bf16"]),
             limit=rng.choice([0.5, 1.0, 1e4]))
    if layout == "layers":
        c.update(count=rng.randint(1, 300), rows=_log(rng, 1, 900_000))
    else:
        c.update(count=_log(rng, 100, 3_000_000), sh=rng.choice([1, 4, 9, 16]),
                 rows=_log(rng, 16, 65536) if layout == "coded" else 0)
    if op == "adam":
        c.update(copy=rng.choice(["none", "bf16", "f16"]), decay=rng.choice([0.0, 0.01]), step=_log(rng, 1, 30000))
    return c


# ---------------------------------------------------------------------------- inputs

def _sizes(c):
    """Values of each tensor of a "layers" list (fixed by the case)."""
    r = random.Random(c["count"] * 1000003 + c["rows"])
    return [_log(r, 1, c["rows"]) for _ in range(c["count"])]


def _list(c, dtype, gen, fill):
    """The tensors of a list and the whole buffers that hold them.  fill(tensor, k) writes tensor k's values."""
    n, k = c["count"], 3 * c["sh"]
    if c["layout"] == "layers":
        sizes = _sizes(c)
        flat = torch.empty(sum(sizes), dtype=dtype, device=DEV)
        fill(flat, 0)
        views, at = [], 0
        for s in sizes:
            views.append(flat[at:at + s])
            at += s
        return views, [flat]
    if c["layout"] == "scene":
        views = [torch.empty((n, w) if w > 1 else (n,), dtype=dtype, device=DEV) for w in (3, 3, 4, 1, k)]
    else:   # geometry, and the table's rows instead of SH
        views = [torch.empty((n, w), dtype=dtype, device=DEV) for w in (3, 3, 4, 1)]
        views.append(torch.empty((c["rows"], k), dtype=dtype, device=DEV))
    for q, t in enumerate(views):
        fill(t, q)
    return views, views


def _columns(c, dtype):
    """The gradients of a "coded" scene: geometry as columns of the view's gradient rows [N][11 + 3K], and the
    table's gradient."""
    rows = torch.zeros((c["count"], 11 + 3 * c["sh"]), dtype=dtype, device=DEV)
    table = torch.zeros((c["rows"], 3 * c["sh"]), dtype=dtype, device=DEV)
    return [rows[:, a:b] for a, b in ((0, 3), (3, 6), (6, 10), (10, 11))] + [table]


def _indices(c, gen):
    t, v = c["tokens"], c["vocab"]
    u = torch.rand(t, generator=gen, device=DEV, dtype=torch.float64)
    if c["spread"] == "uniform":
        i = (u * v).long()
    else:   # log-uniform ranks, scattered over the table
        i = torch.exp(u * math.log(v + 1.0)).long() - 1 if c["spread"] == "zipf" else (u * u * v).long()
        i = (i.clamp(0, v - 1) * 7919 + 13) % v
    if c["spread"] == "codes":
        i[torch.rand(t, generator=gen, device=DEV) < 0.25] = v // 3
    i = i.clamp(0, v - 1)
    if c["masked"]:
        i[torch.rand(t, generator=gen, device=DEV) < c["masked"]] = -1
    return i.to(torch.int32 if c["index"] == "i32" else torch.int64)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    dt = TYPES[c["type"]]
    s = {"case": c}

    def normal(t, scale):
        t.normal_(0.0, 1.0, generator=gen)
        t.mul_(scale)

    if c["op"] == "fwd":
        s["table"] = torch.empty((c["vocab"], c["width"]), dtype=dt, device=DEV)
        normal(s["table"], 0.2)
        s["index"] = _indices(c, gen)
        s["out"] = torch.empty((c["tokens"], c["width"]), dtype=dt, device=DEV)
    elif c["op"] == "bwd":
        rows = torch.empty((c["tokens"], c["row"]), dtype=dt, device=DEV)
        normal(rows, 0.01)
        s["dout"] = rows[:, c["row"] - c["width"]:]
        s["index"] = _indices(c, gen)
        s["dtable"] = torch.empty((c["vocab"], c["width"]), dtype=TYPES[c["grad"]], device=DEV)
    else:
        # gradients of different magnitude per tensor, a third of them exact zeros (Gaussians the view does not see)
        def gradient(t, q):
            x = torch.empty(t.shape, dtype=torch.float32, device=DEV)
            normal(x, 10.0 ** -(q % 4))
            x[torch.rand(t.shape[0], generator=gen, device=DEV) < 0.33] = 0.0
            t.copy_(x)

        if c["layout"] == "coded":
            s["grads"] = s["grads_whole"] = _columns(c, dt)
            for q, t in enumerate(s["grads"]):
                gradient(t, q)
        else:
            s["grads"], s["grads_whole"] = _list(c, dt, gen, gradient)
        if c["op"] == "clip":
            if c["layout"] == "coded":
                s["out"] = s["whole"] = _columns(c, dt)
            else:
                s["out"], s["whole"] = _list(c, dt, gen, lambda t, q: t.zero_())
        else:
            f32 = torch.float32
            s["params"], p = _list(c, f32, gen, lambda t, q: normal(t, 1.0))
            s["m"], m = _list(c, f32, gen, lambda t, q: normal(t, 0.01))
            s["v"], v = _list(c, f32, gen, lambda t, q: (normal(t, 0.01), t.square_()))
            s["copies"], k = (None, []) if c["copy"] == "none" else \
                _list(c, TYPES[c["copy"]], gen, lambda t, q: t.zero_())
            s["whole"] = p + m + v + k
            s["groups"] = list(zip(p, m, v, s["grads_whole"], k or [None] * len(p)))
        s["norm"] = torch.zeros(2, dtype=torch.float32, device=DEV)   # the norm and the factor
    return s


# ---------------------------------------------------------------------------- one pass

_context = []


def _ctx():
    import differentiable_gaussian_splatting_amd as dgs
    if not _context:
        _context.append(dgs.Context())
    return dgs, _context[0]


def _norm(s):
    total = torch.zeros((), dtype=torch.float32, device=DEV)
    for g in s["grads_whole"]:
        x = g.float()
        total = total + (x * x).sum()
    norm = torch.sqrt(total)
    return norm, torch.clamp(s["case"]["limit"] / (norm + 1e-6), max=1.0)


def run(s):
    c = s["case"]
    if own:
        dgs, ctx = _ctx()
        if c["op"] == "fwd":
            return dgs.gs_embed_fwd(ctx, s["table"], s["index"], s["out"], scale=c["scale"])
        if c["op"] == "bwd":
            return dgs.gs_embed_bwd(ctx, s["index"], s["dout"], s["dtable"], scale=c["scale"], padding=c["padding"])
        if "lists" not in s:   # a training program describes its buffers once
            L = {k: dgs.TensorList(s[k]) for k in ("grads", "out", "params", "m", "v", "copies") if s.get(k)}
            s["lists"] = L
        L = s["lists"]
        if c["op"] == "clip":
            dgs.gs_clip_grads(ctx, L["grads"], c["limit"], s["norm"], out=L["out"])
        else:
            dgs.gs_grad_norm(ctx, L["grads"], c["limit"], s["norm"])
            dgs.gs_adam_tensors(ctx, L["params"], L["m"], L["v"], L["grads"], step=c["step"], lr=LR, beta1=BETA1,
                                beta2=BETA2, eps=EPS, weight_decay=c["decay"], norm=s["norm"],
                                copies=L.get("copies"))
        return [s["norm"][0]] + s["whole"]

    if c["op"] == "fwd":
        i, v = s["index"].long(), c["vocab"]
        inside = (i >= 0) & (i < v)
        x = s["table"][i.clamp(0, v - 1)].float() * c["scale"]
        return torch.where(inside[:, None], x, torch.zeros((), device=DEV)).to(s["table"].dtype)
    if c["op"] == "bwd":
        i, v = s["index"].long(), c["vocab"]
        inside = (i >= 0) & (i < v) & (i != c["padding"])
        x = torch.where(inside[:, None], s["dout"].float(), torch.zeros((), device=DEV))
        sums = torch.zeros((v, c["width"]), dtype=torch.float32, device=DEV)
        sums.index_add_(0, i.clamp(0, v - 1), x)
        return (sums * c["scale"]).to(s["dtable"].dtype)
    norm, factor = _norm(s)
    if c["op"] == "clip":
        for g, o in zip(s["grads_whole"], s["whole"]):
            o.copy_(g.float() * factor)
        return [norm] + s["whole"]
    t = c["step"]
    for p, m, v, g, low in s["groups"]:   # whole buffers: the layers of a flat buffer are updated together
        x = g.float().reshape(p.shape) * factor
        m.mul_(BETA1).add_(x * (1.0 - BETA1))
        v.mul_(BETA2).add_(x * x * (1.0 - BETA2))
        step = (m / (1.0 - BETA1 ** t)) / (torch.sqrt(v / (1.0 - BETA2 ** t)) + EPS)
        p.mul_(1.0 - LR * c["decay"]).sub_(step * LR)
        if low is not None:
            low.copy_(p)
    return [norm] + s["whole"]


def _values(c):
    if c["layout"] == "layers":
        return sum(_sizes(c))
    if c["layout"] == "scene":
        return c["count"] * (11 + 3 * c["sh"])
    return c["count"] * 11 + c["rows"] * 3 * c["sh"]


def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2, "none": 0, "i32": 4, "i64": 8}
    if c["op"] == "fwd":
        n = c["tokens"] * c["width"]
        rows = min(c["tokens"], c["vocab"]) * c["width"]   # at most that many distinct rows are read
        return {"bytes": c["tokens"] * size[c["index"]] + (rows + n) * size[c["type"]], "flops": n}
    if c["op"] == "bwd":
        n = c["tokens"] * c["width"]
        return {"bytes": c["tokens"] * size[c["index"]] + n * size[c["type"]] +
                c["vocab"] * c["width"] * size[c["grad"]], "flops": n}
    n = _values(c)
    if c["op"] == "clip":
        return {"bytes": 2 * n * size[c["type"]], "flops": 3 * n}
    return {"bytes": n * (size[c["type"]] + 24 + size[c["copy"]]), "flops": 16 * n}


# ---------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, f64 = s["case"], torch.float64
    if c["op"] == "fwd":
        wide = torch.cat([s["table"].double() * c["scale"], torch.zeros((1, c["width"]), dtype=f64, device=DEV)])
        i = s["index"].long()
        return wide.index_select(0, torch.where((i < 0) | (i >= c["vocab"]), torch.full_like(i, c["vocab"]), i))
    if c["op"] == "bwd":
        i = s["index"].long()
        keep = torch.nonzero((i >= 0) & (i < c["vocab"]) & (i != c["padding"]))[:, 0]
        out = torch.zeros((c["vocab"], c["width"]), dtype=f64, device=DEV)
        for a in range(0, keep.numel(), 1 << 20):
            k = keep[a:a + (1 << 20)]
            out.scatter_add_(0, i[k][:, None].expand(-1, c["width"]), s["dout"].index_select(0, k).double())
        return out * c["scale"]
    squares = sum(float(g.double().pow(2).sum()) for g in s["grads"])
    norm = math.sqrt(squares)
    factor = min(1.0, c["limit"] / (norm + 1e-6))
    if c["op"] == "clip":
        if c["layout"] == "layers":
            return [norm, torch.cat(s["grads"]).double() * factor]
        return [norm] + [g.double() * factor for g in s["grads"]]
    flat = c["layout"] == "layers"
    join = (lambda ts: [torch.cat(ts)]) if flat else (lambda ts: list(ts))
    t, ps, ms, vs = c["step"], [], [], []
    for p, m, v, g in zip(join(s["params"]), join(s["m"]), join(s["v"]), join(s["grads"])):
        x = g.double().view(p.shape) * factor if g.is_contiguous() else g.double().reshape(p.shape) * factor
        m1 = BETA1 * m.double() + (1.0 - BETA1) * x
        v1 = BETA2 * v.double() + (1.0 - BETA2) * x ** 2
        root = (v1 / (1.0 - BETA2 ** t)).sqrt() + EPS
        ps.append(p.double() - LR * c["decay"] * p.double() - LR * (m1 / (1.0 - BETA1 ** t)) / root)
        ms.append(m1)
        vs.append(v1)
    return [norm] + ps + ms + vs + (ps if c["copy"] != "none" else [])
