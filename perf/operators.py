"""The training and serving operators next to the all-reduce, as measured cases.

A linear layer (forward, input gradient, weight gradient), the Muon step with
its Newton-Schulz orthogonalisation, and the AdamW step of what Muon leaves.
Every case can be run in its plain form (elementary torch operations in 32
bits) and, with `own` set, through the library's entry points.
"""
import math

import torch

own = False

# Newton-Schulz: X <- a X + (b A + c A A) X with A = X X^T, five times
NS_A, NS_B, NS_C, NS_STEPS, NS_EPS = 3.4445, -4.7750, 2.0315, 5, 1e-7
# the optimizers' settings of every case
LR, MU, DECAY = 2e-3, 0.95, 0.1
BETA1, BETA2, ADAM_EPS, ADAM_STEP = 0.9, 0.95, 1e-8, 7

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")

# ResNet-50's stages: (blocks, width, input channels)
_STAGES = ((3, 64, 64), (4, 128, 256), (6, 256, 512), (3, 512, 1024))


def _block(width, cin, first):
    """(rows, cols) of a bottleneck block's convolutions as matrices."""
    return ([(width, cin), (width, 9 * width), (4 * width, width)]
            + ([(4 * width, cin)] if first else []))


def _resnet50():
    """ResNet-50's matrices (each convolution as out x in*k*k, the classifier)
    and the lengths of its vectors (two per batch norm, the classifier's bias)."""
    convs = [(64, 147)] + [s for blocks, width, cin in _STAGES for b in range(blocks)
                           for s in _block(width, cin if b == 0 else 4 * width, b == 0)]
    return convs + [(1000, 2048)], [r for r, _ in convs for _ in (0, 1)] + [1000]


def listed():
    return [
        # decoding: one token through a square projection
        dict(name="forward, one token", op="forward", m=1, n=4096, k=4096, dtype="bf16",
             act="silu", bias=True, residual=False, keep=False),
        # odd sizes throughout: rows of 2047 elements start off 16-byte boundaries
        dict(name="forward, odd sizes", op="forward", m=333, n=1000, k=2047, dtype="f16",
             act="relu", bias=True, residual=True, keep=True),
        # the widening layer of a transformer's MLP over 8192 tokens, as trained
        dict(name="forward, wide", op="forward", m=8192, n=16384, k=4096, dtype="bf16",
             act="gelu_tanh", bias=True, residual=False, keep=True),
        # the narrowing layer's input gradient, through the activation before it
        dict(name="input gradient, wide", op="dgrad", m=8192, n=4096, k=16384, dtype="bf16",
             act="gelu_tanh", residual=False),
        # ResNet-50's classifier on a ragged batch, with a skip connection's gradient
        dict(name="input gradient, classifier", op="dgrad", m=999, n=1000, k=2048, dtype="f16",
             act="relu", residual=True),
        # one micro-batch more on binary32 gradients of a square projection
        dict(name="weight gradient, accumulated", op="wgrad", m=16384, n=4096, k=4096,
             dtype="bf16", out="f32", add=True),
        # ResNet-50's classifier into a binary16 bucket
        dict(name="weight gradient, classifier", op="wgrad", m=512, n=1000, k=2048,
             dtype="f16", out="f16", add=False),
        # one tall gradient matrix, orthogonalised by itself
        dict(name="orthogonalise, tall", op="orthogonalise", count=1, rows=4096, cols=1024,
             dtype="bf16"),
        # every matrix of ResNet-50 in one step, binary16 gradients
        dict(name="muon, ResNet-50", op="muon", count=0, rows=0, cols=0, dtype="f16",
             copy="none"),
        # a few large square layers with bfloat16 working copies
        dict(name="muon, large", op="muon", count=3, rows=4096, cols=4096, dtype="f32",
             copy="bf16"),
        # the vectors of ResNet-50, which Muon leaves: 107 short spans
        dict(name="adamw, ResNet-50 vectors", op="adamw", count=0, n=0, dtype="f32",
             copy="none"),
        # ResNet-50's whole parameter buffer with binary16 gradients and copies
        dict(name="adamw, whole buffer", op="adamw", count=1, n=25557032, dtype="f16",
             copy="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("forward", "forward", "dgrad", "wgrad", "orthogonalise", "muon", "adamw"))
    if op in ("forward", "dgrad", "wgrad"):
        c = dict(op=op, m=_log(rng, 1, 16384), n=_log(rng, 8, 16384), k=_log(rng, 8, 16384),
                 dtype=rng.choice(("bf16", "f16")))
        if rng.random() < 0.5:  # most layers' widths are multiples of 64
            c["n"], c["k"] = -(-c["n"] // 64) * 64, -(-c["k"] // 64) * 64
        while c["m"] * c["n"] * c["k"] > 8192 * 16384 * 4096:
            c["m"] = c["m"] // 2 + 1
        if op == "wgrad":
            c.update(out=rng.choice(("f32", "f16" if c["dtype"] == "f16" else "bf16")))
            c.update(add=c["out"] == "f32" and rng.random() < 0.5)
        else:
            c.update(act=rng.choice(ACTS), residual=rng.random() < 0.5)
        if op == "forward":
            c.update(bias=rng.random() < 0.7, keep=rng.random() < 0.5)
        return c
    if op == "adamw":
        return dict(op=op, count=_log(rng, 1, 100), n=_log(rng, 1, 250000),
                    dtype=rng.choice(("f32", "f16")), copy=rng.choice(("none", "f16", "bf16")))
    c = dict(op=op, count=_log(rng, 1, 16), rows=_log(rng, 16, 4096), cols=_log(rng, 16, 4096))
    while c["count"] * _ns_flops(c["rows"], c["cols"]) > 3 * _ns_flops(4096, 4096):
        c["count"] = max(1, c["count"] // 2)
    if op == "muon":
        return dict(c, dtype=rng.choice(("f32", "f16")), copy=rng.choice(("none", "bf16")))
    return dict(c, dtype=rng.choice(("f32", "f16", "bf16")))


def _ns_flops(r, c):
    """A X X^T and an A A are symmetric: half of each has to be computed."""
    s, l = min(r, c), max(r, c)
    return NS_STEPS * (3 * s * s * l + s * s * s)


def _size(name):
    return 0 if name == "none" else 4 if name == "f32" else 2


def _matrices(case):
    """[(offset, rows, cols)] of the case's matrices in one flat buffer."""
    shapes = [(case["rows"], case["cols"])] * case["count"] if case["count"] else _resnet50()[0]
    at = [sum(r * c for r, c in shapes[:i]) for i in range(len(shapes))]
    return [(o, r, c) for o, (r, c) in zip(at, shapes)]


def _spans(case):
    """[(offset, count)] of the case's vectors; they lie 16 elements apart at
    least, as after the matrices that they belong to."""
    sizes = [case["n"]] * case["count"] if case["count"] else _resnet50()[1]
    step = [-(-s // 16) * 16 + 16 for s in sizes]
    return [(sum(step[:i]), s) for i, s in enumerate(sizes)]


def work(case):
    op, e = case["op"], _size(case["dtype"])
    if op in ("forward", "dgrad", "wgrad"):
        m, n, k = case["m"], case["n"], case["k"]
        flops = 2 * m * n * k
        if op == "forward":
            b = e * (m * k + n * k + m * n * (1 + case["residual"] + case["keep"]) + n * case["bias"])
        elif op == "dgrad":
            acts = case["act"] != "none"
            b = e * (m * n + n * k + m * k * (1 + case["residual"] + 2 * acts))
        else:
            b = e * (m * n + m * k) + _size(case["out"]) * (n * k + n) * (1 + case["add"])
        return {"bytes": b, "flops": flops}
    if op == "adamw":
        n = sum(c for _, c in _spans(case))
        return {"bytes": n * (e + 24 + _size(case["copy"])), "flops": 15 * n}
    n = sum(r * c for _, r, c in _matrices(case))
    flops = sum(_ns_flops(r, c) for _, r, c in _matrices(case))
    b = 2 * e * n if op == "orthogonalise" else n * (e + 16 + _size(case["copy"]))
    return {"bytes": b, "flops": flops}


def _scale(r, c):
    """Muon's factor that gives an orthogonal r x c update AdamW's usual size."""
    return 0.2 * math.sqrt(max(r, c))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype="f32"):
        return (torch.randn(*shape, generator=gen, device="cuda") * sigma).to(TYPES[dtype])

    op, t = case["op"], case["dtype"]
    s = {"case": case}
    if op in ("forward", "dgrad", "wgrad"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "forward":
            s["x"], s["w"] = normal(m, k, dtype=t), normal(n, k, sigma=k ** -0.5, dtype=t)
            s["bias"] = normal(n, sigma=0.1, dtype=t) if case["bias"] else None
            s["residual"] = normal(m, n, dtype=t) if case["residual"] else None
        elif op == "dgrad":
            s["dz"], s["w"] = normal(m, n, dtype=t), normal(n, k, sigma=n ** -0.5, dtype=t)
            s["residual"] = normal(m, k, dtype=t) if case["residual"] else None
            s["z"] = normal(m, k, dtype=t) if case["act"] != "none" else None
        else:
            s["dz"], s["x"] = normal(m, n, sigma=m ** -0.5, dtype=t), normal(m, k, dtype=t)
            s["dw"] = normal(n, k, dtype=case["out"])
            s["db"] = normal(n, dtype=case["out"])
    elif op == "adamw":
        s["spans"] = _spans(case)
        n = s["spans"][-1][0] + s["spans"][-1][1]
        s["grad"] = normal(n, sigma=1e-2, dtype=t)
        s["m"], s["v"] = normal(n, sigma=1e-2), normal(n, sigma=1e-2).square()
        s["weights"] = normal(n, sigma=0.02)
    else:
        s["matrices"] = _matrices(case)
        n = s["matrices"][-1][0] + s["matrices"][-1][1] * s["matrices"][-1][2]
        s["grad"] = normal(n, sigma=1e-2, dtype=t)
        if op == "muon":
            s["momentum"], s["weights"] = normal(n, sigma=3e-2), normal(n, sigma=0.02)
        else:
            s["out"] = torch.empty_like(s["grad"])
    if case.get("copy", "none") != "none":
        s["copy"] = torch.zeros(n, device="cuda", dtype=TYPES[case["copy"]])
    if own:  # what a program keeps from call to call: output buffers, workspaces, handles
        import sgd_gradient_all_amd as ddl
        if op == "forward":
            s["y"] = torch.empty(m, n, device="cuda", dtype=TYPES[t])
            s["keep"] = torch.empty_like(s["y"]) if case["keep"] else None
        if op == "dgrad":
            s["dx"] = torch.empty(m, k, device="cuda", dtype=TYPES[t])
            s["dz_prev"] = torch.empty_like(s["dx"]) if case["act"] != "none" else None
        if op in ("forward", "dgrad", "wgrad"):
            s["workspace"] = torch.empty(ddl.linear_workspace(op, m, n, k), device="cuda",
                                         dtype=torch.uint8)
        elif op == "adamw":
            s["handle"] = ddl.AdamW(s["spans"])
        else:
            s["handle"] = ddl.Muon([(o, r, c, _scale(r, c)) for o, r, c in s["matrices"]])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return torch.clamp_min(z, 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return (0.5 * (1 + t)
                + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z))
    g = 1 / (1 + torch.exp(-z))  # silu
    return g * (1 + z * (1 - g))


def _orthogonal(u):
    """Newton-Schulz on u[..., r, c], in u's type; the norm in 64 bits."""
    tall = u.shape[-2] > u.shape[-1]
    x = u.transpose(-2, -1).contiguous() if tall else u
    norm = x.double().square().sum((-2, -1), keepdim=True).sqrt() + NS_EPS
    x = (x.double() / norm).to(u.dtype)
    for _ in range(NS_STEPS):
        a = x @ x.transpose(-2, -1).contiguous()
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x.transpose(-2, -1) if tall else x


def _by_shape(matrices, flat, then):
    """Calls then(offsets, stack of the matrices) for each shape there is."""
    shapes = {}
    for o, r, c in matrices:
        shapes.setdefault((r, c), []).append(o)
    for (r, c), offs in shapes.items():
        then(offs, torch.stack([flat[o:o + r * c].view(r, c) for o in offs]))


def _plain_forward(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    t = s["x"].dtype
    return {"y": y.to(t), "z": z.to(t)} if c["keep"] else {"y": y.to(t)}


def _plain_dgrad(s):
    c, t = s["case"], s["dz"].dtype
    dx = s["dz"].float() @ s["w"].float()
    if c["residual"]:
        dx = dx + s["residual"].float()
    if c["act"] == "none":
        return {"dx": dx.to(t)}
    return {"dx": dx.to(t), "dz": (dx * _act_slope(s["z"].float(), c["act"])).to(t)}


def _plain_wgrad(s):
    dz = s["dz"].float()
    dw, db = dz.t() @ s["x"].float(), dz.sum(0)
    if s["case"]["add"]:
        s["dw"] += dw
        s["db"] += db
    else:
        s["dw"].copy_(dw)
        s["db"].copy_(db)
    return {"dw": s["dw"], "db": s["db"]}


def _plain_orthogonalise(s):
    # binary32 results take 64-bit products: 32 bits leave the five rounds of a
    # few thousand columns over 1e-5 off
    wide = torch.float64 if s["case"]["dtype"] == "f32" else torch.float32

    def then(offs, u):
        for o, x in zip(offs, _orthogonal(u.to(wide))):
            s["out"][o:o + x.numel()].view(x.shape).copy_(x)
    _by_shape(s["matrices"], s["grad"], then)
    return s["out"]


def _plain_muon(s):
    g, w = s["grad"].float(), s["weights"]
    s["momentum"].mul_(MU).add_(g)

    def then(offs, u):
        for o, x in zip(offs, _orthogonal(u)):
            part = w[o:o + x.numel()].view(x.shape)
            part.mul_(1 - LR * DECAY).sub_(x, alpha=LR * _scale(*x.shape))
    _by_shape(s["matrices"], g + MU * s["momentum"], then)
    if "copy" in s:
        s["copy"].copy_(w)
    return [w, s["momentum"]] + ([s["copy"]] if "copy" in s else [])


def _plain_adamw(s):
    # over the whole buffer at once; what lies between the spans keeps its values
    if "inside" not in s:
        s["inside"] = torch.zeros_like(s["weights"], dtype=torch.bool)
        for o, c in s["spans"]:
            s["inside"][o:o + c] = True
    g, at = s["grad"].float(), s["inside"]
    m = BETA1 * s["m"] + (1 - BETA1) * g
    v = BETA2 * s["v"] + (1 - BETA2) * g * g
    step = (m / (1 - BETA1 ** ADAM_STEP)) / (torch.sqrt(v / (1 - BETA2 ** ADAM_STEP)) + ADAM_EPS)
    w = s["weights"] * (1 - LR * DECAY) - LR * step
    for name, x in (("m", m), ("v", v), ("weights", w)) + ((("copy", w),) if "copy" in s else ()):
        s[name].copy_(torch.where(at, x, s[name]))
    return [s["weights"], s["m"], s["v"]] + ([s["copy"]] if "copy" in s else [])


_PLAIN = {"forward": _plain_forward, "dgrad": _plain_dgrad, "wgrad": _plain_wgrad,
          "orthogonalise": _plain_orthogonalise, "muon": _plain_muon, "adamw": _plain_adamw}


def run(state):
    s = state
    if not own:
        return _PLAIN[s["case"]["op"]](s)
    import sgd_gradient_all_amd as ddl
    c = s["case"]
    op = c["op"]
    if op == "forward":
        ddl.linear(s["x"], s["w"], s["y"], bias=s["bias"], act=c["act"], residual=s["residual"],
                   z=s["keep"], workspace=s["workspace"])
        return {"y": s["y"], "z": s["keep"]} if c["keep"] else {"y": s["y"]}
    if op == "dgrad":
        ddl.linear_dgrad(s["dz"], s["w"], dx=s["dx"], residual=s["residual"], act=c["act"],
                         z_prev=s["z"], dz_prev=s["dz_prev"], workspace=s["workspace"])
        return {"dx": s["dx"]} if c["act"] == "none" else {"dx": s["dx"], "dz": s["dz_prev"]}
    if op == "wgrad":
        ddl.linear_wgrad(s["dz"], s["x"], s["dw"], db=s["db"], accumulate=c["add"],
                         workspace=s["workspace"])
        return {"dw": s["dw"], "db": s["db"]}
    if op == "orthogonalise":
        s["handle"].orthogonalise(s["grad"], s["out"])
        return s["out"]
    if op == "muon":
        s["handle"].step(s["grad"], s["momentum"], [s["weights"]], lr=LR, momentum_decay=MU,
                         nesterov=True, weight_decay=DECAY, copy=s.get("copy"))
        return [s["weights"], s["momentum"]] + ([s["copy"]] if "copy" in s else [])
    s["handle"].step(s["grad"], s["m"], s["v"], [s["weights"]], lr=LR, beta1=BETA1, beta2=BETA2,
                     eps=ADAM_EPS, weight_decay=DECAY, step=ADAM_STEP, copy=s.get("copy"))
    return [s["weights"], s["m"], s["v"]] + ([s["copy"]] if "copy" in s else [])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s, op, d = prepare(case, seed), case["op"], torch.float64
    if op == "forward":
        z = torch.mm(s["x"].to(d), s["w"].to(d).t().contiguous())
        z = z if s["bias"] is None else z.add_(s["bias"].to(d))
        cdf = torch.special.ndtr
        y = {"none": lambda t: t.clone(), "relu": lambda t: t.clamp(min=0.0),
             "gelu": lambda t: t * cdf(t),
             "gelu_tanh": lambda t: t * torch.sigmoid(1.5957691216057308 * (t + 0.044715 * t ** 3)),
             "silu": lambda t: t * torch.sigmoid(t)}[case["act"]](z)
        y = y if s["residual"] is None else y.add_(s["residual"].to(d))
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    if op == "dgrad":
        dx = torch.mm(s["dz"].to(d), s["w"].to(d))
        dx = dx if s["residual"] is None else dx.add_(s["residual"].to(d))
        if s["z"] is None:
            return {"dx": dx}
        z = s["z"].to(d)
        if case["act"] == "relu":
            return {"dx": dx, "dz": dx.masked_fill(z <= 0, 0.0)}
        if case["act"] == "gelu":
            slope = torch.special.ndtr(z) + z * torch.exp(-z * z / 2) * 0.3989422804014327
        else:  # t sigmoid(u): slope sigmoid(u) (1 + z u' (1 - sigmoid(u)))
            k = 1.5957691216057308
            u, du = ((z, 1.0) if case["act"] == "silu"
                     else (k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z * z)))
            sg = torch.sigmoid(u)
            slope = sg + z * du * sg * torch.sigmoid(-u)
        return {"dx": dx, "dz": dx * slope}
    if op == "wgrad":
        dw = torch.mm(s["dz"].to(d).t().contiguous(), s["x"].to(d))
        db = s["dz"].to(d).sum(0)
        if case["add"]:
            dw, db = dw + s["dw"], db + s["db"]
        return {"dw": dw, "db": db}
    if op == "adamw":
        g, m, v, w = (s[k].to(d) for k in ("grad", "m", "v", "weights"))
        cp = s["copy"].to(d) if "copy" in s else None
        for o, n in s["spans"]:
            at = slice(o, o + n)
            m[at] += (1 - BETA1) * (g[at] - m[at])
            v[at] += (1 - BETA2) * (g[at] ** 2 - v[at])
            hat = (v[at] / (1 - BETA2 ** ADAM_STEP)).sqrt() + ADAM_EPS
            w[at] -= LR * (m[at] / (1 - BETA1 ** ADAM_STEP) / hat + DECAY * w[at])
            if cp is not None:
                cp[at] = w[at]
        return [w, m, v] + ([cp] if cp is not None else [])
    g = s["grad"].to(d)
    if op == "muon":
        mom = s["momentum"].to(d) * MU + g
        src, w = g + mom * MU, s["weights"].to(d)
    else:
        src, w = g, torch.empty_like(g)
    for o, r, c in s["matrices"]:
        x = src[o:o + r * c].reshape(r, c)
        x = x / (torch.linalg.matrix_norm(x) + NS_EPS)
        for _ in range(NS_STEPS):
            if r <= c:
                p = torch.mm(x, x.t().contiguous())
                x = NS_A * x + torch.mm(NS_B * p + NS_C * torch.mm(p, p), x)
            else:
                p = torch.mm(x.t().contiguous(), x)
                x = NS_A * x + torch.mm(x, NS_B * p + NS_C * torch.mm(p, p))
        part = w[o:o + r * c].view(r, c)
        if op == "muon":
            part.copy_(part - LR * (DECAY * part + _scale(r, c) * x))
        else:
            part.copy_(x)
    if op == "orthogonalise":
        return w
    return [w, mom] + ([w.clone()] if "copy" in s else [])
