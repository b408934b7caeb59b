"""Both ends of a training step next to the all-reduce, as measured cases.

The softmax cross entropy of a projection onto many classes, with its
gradient, in pieces of the classes and without its logits in memory; and the
AdamW step with both states in 8 bits.  Every case can be run in its plain
form (elementary torch operations in 32 bits, in 64 next to the borders between
8-bit values) and, with `own` set, through the library's entry points.
"""
import math

import torch

own = False

# the optimizer's settings of every case
LR, DECAY, BETA1, BETA2, EPS, STEP = 2e-3, 0.1, 0.9, 0.95, 1e-8, 7
# elements that share the scales of their 8-bit states
BLOCK = 256

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# ResNet-50's batch norms (two vectors each) and its classifier's bias
_STAGES = ((3, 64), (4, 128), (6, 256), (3, 512))
_RESNET50 = [n for n in [64] + [w * f for blocks, w in _STAGES for b in range(blocks)
                                for f in ((1, 1, 4, 4) if b == 0 else (1, 1, 4))]
             for _ in (0, 1)] + [1000]


def listed():
    return [
        # scoring one next token against a large vocabulary
        dict(name="loss, one token", op="loss", m=1, n=131072, k=4096, dtype="bf16", bias=False,
             smoothing=0.0, ignored=0.0),
        # ResNet-50's classifier on a worker's batch of 32 with smoothed labels
        dict(name="loss, classifier", op="loss", m=32, n=1000, k=2048, dtype="f16", bias=True,
             smoothing=0.1, ignored=0.0),
        # odd sizes throughout, and a third of the rows without a target (prompts)
        dict(name="loss, odd sizes", op="loss", m=1999, n=50001, k=1023, dtype="f16", bias=True,
             smoothing=0.0, ignored=0.33),
        # a language model's validation loss over 8192 tokens
        dict(name="loss, large", op="loss", m=8192, n=131072, k=4096, dtype="bf16", bias=False,
             smoothing=0.0, ignored=0.0),
        # ResNet-50's classifier, gradients into a binary16 bucket
        dict(name="gradient, classifier", op="gradient", m=512, n=1000, k=2048, dtype="f16",
             bias=True, smoothing=0.1, ignored=0.0, out="f16", add=False),
        # a padded batch (half of its rows) of odd sizes into 16-bit gradients
        dict(name="gradient, odd sizes", op="gradient", m=1023, n=32003, k=1111, dtype="bf16",
             bias=True, smoothing=0.0, ignored=0.5, out="bf16", add=False),
        # one micro-batch more on binary32 gradients, as the all-reduce takes them
        dict(name="gradient, accumulated", op="gradient", m=4096, n=65536, k=2048, dtype="bf16",
             bias=False, smoothing=0.0, ignored=0.1, out="f32", add=True),
        # a language model's last layer over 8192 tokens
        dict(name="gradient, large", op="gradient", m=8192, n=131072, k=4096, dtype="bf16",
             bias=False, smoothing=0.0, ignored=0.0, out="bf16", add=False),
        # ResNet-50's batch norms and bias: 107 short vectors
        dict(name="adamw8, ResNet-50 vectors", op="adamw8", count=0, n=0, dtype="f32",
             copy="none"),
        # ResNet-50's whole parameter buffer with binary16 gradients and copies
        dict(name="adamw8, whole buffer", op="adamw8", count=1, n=25557032, dtype="f16",
             copy="f16"),
        # the 300M-parameter buffer, binary32 gradients and bfloat16 copies
        dict(name="adamw8, 300M", op="adamw8", count=1, n=300000000, dtype="f32", copy="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("loss", "loss", "gradient", "gradient", "adamw8"))
    if op == "adamw8":
        c = dict(op=op, count=_log(rng, 1, 100), n=_log(rng, 1, 30000000),
                 dtype=rng.choice(("f32", "f16", "bf16")),
                 copy=rng.choice(("none", "f16", "bf16")))
        while c["count"] * c["n"] > 100000000:
            c["count"] = max(1, c["count"] // 2)
        return c
    c = dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 1000, 131072), k=_log(rng, 64, 4096),
             dtype=rng.choice(("bf16", "f16")), bias=rng.random() < 0.5,
             smoothing=rng.choice((0.0, 0.0, 0.1)), ignored=rng.choice((0.0, 0.1, 0.5)))
    if rng.random() < 0.5:  # most layers' widths are multiples of 64
        c["n"], c["k"] = -(-c["n"] // 64) * 64, -(-c["k"] // 64) * 64
    if op == "gradient":
        c["out"] = rng.choice(("f32", c["dtype"]))
        c["add"] = c["out"] == "f32" and rng.random() < 0.5
    return c


def _size(name):
    return 0 if name == "none" else 4 if name == "f32" else 2


def _spans(case):
    """[(offset, count)] of the case's vectors; they lie 16 elements apart at
    least, as between the matrices that they belong to."""
    sizes = [case["n"]] * case["count"] if case["count"] else _RESNET50
    step = [-(-s // 16) * 16 + 16 for s in sizes]
    return [(sum(step[:i]), s) for i, s in enumerate(sizes)]


def _blocks(case):
    return sum(-(-c // BLOCK) for _, c in _spans(case))


def work(case):
    """Rows without a target need nothing but their zeros."""
    if case["op"] == "adamw8":
        n = sum(c for _, c in _spans(case))
        # codes and scales read and written, their values written
        return {"bytes": n * (_size(case["dtype"]) + 8 + 4 + 8 + _size(case["copy"]))
                + 16 * _blocks(case), "flops": 40 * n}
    m, n, k = case["m"], case["n"], case["k"]
    rows = max(1, round(m * (1 - case["ignored"])))
    b = 2 * (rows * k + n * k + n * case["bias"]) + 16 * m
    if case["op"] == "loss":
        return {"bytes": b, "flops": 2 * rows * n * k}
    b += 2 * m * k + _size(case["out"]) * (n * k + n) * (1 + case["add"])
    return {"bytes": b, "flops": 6 * rows * n * k}


# ---------------------------------------------------------------------------
# 8-bit states: m is scale (k / 127)^2 with k's sign, k = -127 .. 127; v is
# scale (k / 255)^4, k = 0 .. 255; the scale is the block's largest magnitude
# in binary32, and k the nearest to the value's own root
# ---------------------------------------------------------------------------

def _decode(m, v, m_scale, v_scale):
    """64-bit values of codes[blocks, BLOCK]."""
    a, b = m.double() / 127, v.double() / 255
    return a * a.abs() * m_scale.double()[:, None], b.square().square() * v_scale.double()[:, None]


def _encode(m, v):
    """(codes of m, of v, scales of m, of v) of 64-bit values[blocks, BLOCK]."""
    sm, sv = m.abs().amax(1).float(), v.amax(1).float()
    one = torch.ones((), device=m.device, dtype=torch.float64)
    a = m.abs() / torch.where(sm > 0, sm.double(), one)[:, None]
    b = v / torch.where(sv > 0, sv.double(), one)[:, None]
    a = torch.round(127 * torch.sqrt(a)).clamp(max=127) * torch.sign(m)
    b = torch.round(255 * torch.sqrt(torch.sqrt(b))).clamp(max=255)
    return a.to(torch.int8), b.to(torch.uint8), sm, sv


def _in_blocks(s, flat):
    """The spans' elements of a flat buffer as [blocks, BLOCK], zeros behind a
    span's end."""
    if len(s["spans"]) == 1:
        n, rows = s["spans"][0][1], s["rows"]
        return torch.nn.functional.pad(flat[:n], (0, rows * BLOCK - n)).view(rows, BLOCK)
    return torch.where(s["inside"], flat[s["index"]], torch.zeros((), device=flat.device,
                                                                  dtype=flat.dtype))


def _from_blocks(s, x, flat):
    """The inverse, into the flat buffer."""
    if len(s["spans"]) == 1:
        n = s["spans"][0][1]
        flat[:n].copy_(x.reshape(-1)[:n])
    else:
        flat[s["index"][s["inside"]]] = x[s["inside"]].to(flat.dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype="f32"):
        return (torch.randn(*shape, generator=gen, device="cuda") * sigma).to(TYPES[dtype])

    t, s = case["dtype"], {"case": case}
    if case["op"] == "adamw8":
        s["spans"] = _spans(case)
        n, s["rows"] = sum(s["spans"][-1]), _blocks(case)
        if len(s["spans"]) > 1:  # where each block's elements lie
            starts = torch.tensor([(o + b, c - b) for o, c in s["spans"]
                                   for b in range(0, c, BLOCK)], device="cuda")
            lane = torch.arange(BLOCK, device="cuda")
            s["inside"] = lane < starts[:, 1:]
            s["index"] = torch.where(s["inside"], starts[:, :1] + lane, starts[:, :1])
        s["grad"], s["weights"] = normal(n, sigma=1e-2, dtype=t), normal(n, sigma=0.02)
        # moments after a few steps: neighbours' gradients differ a few times
        spread = torch.exp(normal(s["rows"], BLOCK))
        m, v = (normal(s["rows"], BLOCK, sigma=3e-3) * spread,
                (1e-2 * spread * (1 + 0.2 * normal(s["rows"], BLOCK))).square())
        if len(s["spans"]) == 1:
            m.view(-1)[case["n"]:], v.view(-1)[case["n"]:] = 0, 0
        else:
            m, v = m * s["inside"], v * s["inside"]
        m, v, s["m_scale"], s["v_scale"] = _encode(m.double(), v.double())
        s["m"] = torch.zeros(n, device="cuda", dtype=torch.int8)
        s["v"] = torch.zeros(n, device="cuda", dtype=torch.uint8)
        _from_blocks(s, m, s["m"])
        _from_blocks(s, v, s["v"])
        s["m_value"], s["v_value"] = (torch.zeros(n, device="cuda") for _ in range(2))
        if case["copy"] != "none":
            s["copy"] = torch.zeros(n, device="cuda", dtype=TYPES[case["copy"]])
        if own:  # what a program keeps from step to step
            import sgd_gradient_all_amd as ddl
            s["handle"] = ddl.AdamW8(s["spans"])
        return s
    m, n, k = case["m"], case["n"], case["k"]
    target = torch.randint(n, (m,), generator=gen, device="cuda")
    s["w"] = normal(n, k, sigma=2 * k ** -0.5, dtype=t)
    # hidden states that know something of their target
    s["x"] = (normal(m, k) + 1.5 * s["w"][target].float()).to(TYPES[t])
    s["bias"] = normal(n, sigma=0.5, dtype=t) if case["bias"] else None
    s["target"] = torch.where(torch.rand(m, generator=gen, device="cuda") < case["ignored"],
                              torch.full_like(target, -100), target)
    if case["op"] == "gradient":
        s["lse"] = _plain_loss(s)["lse"]  # from the forward pass
        s["dloss"] = torch.full((m,), 1 / m, device="cuda")  # of a mean
        # gradients of the size of one row's share, as an earlier micro-batch leaves them
        s["dw"] = normal(n, k, sigma=1 / m, dtype=case["out"])
        s["db"] = normal(n, sigma=1 / m, dtype=case["out"]) if case["bias"] else None
    if own:  # output buffers and the workspace
        import sgd_gradient_all_amd as ddl
        if case["op"] == "loss":
            s["loss"], s["lse"] = (torch.empty(m, device="cuda") for _ in range(2))
        else:
            s["dx"] = torch.empty_like(s["x"])
        op = "forward" if case["op"] == "loss" else "grad"
        s["workspace"] = torch.empty(ddl.cross_entropy_workspace(op, m, n, k), device="cuda",
                                     dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _logits(s):
    z = s["x"].float() @ s["w"].float().t()
    return z if s["bias"] is None else z + s["bias"].float()


def _plain_loss(s):
    a, t = s["case"]["smoothing"], s["target"]
    z = _logits(s)
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    at = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    loss = lse - (1 - a) * at - a * z.mean(1)
    zero = torch.zeros((), device=z.device)
    return {"loss": torch.where(t >= 0, loss, zero), "lse": torch.where(t >= 0, lse, zero)}


def _plain_gradient(s):
    c, t = s["case"], s["target"]
    a, n = c["smoothing"], c["n"]
    dz = torch.exp(_logits(s) - s["lse"][:, None]) - a / n
    dz.scatter_add_(1, t.clamp(min=0)[:, None], torch.full_like(dz[:, :1], a - 1))
    dz = torch.where(t >= 0, s["dloss"], torch.zeros_like(s["dloss"]))[:, None] * dz
    dx = (dz @ s["w"].float()).to(s["x"].dtype)
    dw, db = dz.t() @ s["x"].float(), dz.sum(0)
    if c["add"]:
        s["dw"] += dw
    else:
        s["dw"].copy_(dw)
    out = {"dx": dx, "dw": s["dw"]}
    if s["db"] is not None:
        s["db"].copy_(s["db"] + db if c["add"] else db)
        out["db"] = s["db"]
    return out


def _plain_adamw8(s):
    g, w = _in_blocks(s, s["grad"]).double(), _in_blocks(s, s["weights"])
    m, v = _decode(_in_blocks(s, s["m"]), _in_blocks(s, s["v"]), s["m_scale"], s["v_scale"])
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    step = ((m.float() / (1 - BETA1 ** STEP))
            / (torch.sqrt(v.float() / (1 - BETA2 ** STEP)) + EPS))
    w = w * (1 - LR * DECAY) - LR * step
    m, v, sm, sv = _encode(m, v)
    s["m_scale"].copy_(sm)
    s["v_scale"].copy_(sv)
    values = _decode(m, v, sm, sv)
    _from_blocks(s, m, s["m"])
    _from_blocks(s, v, s["v"])
    _from_blocks(s, values[0], s["m_value"])
    _from_blocks(s, values[1], s["v_value"])
    _from_blocks(s, w, s["weights"])
    if "copy" in s:
        _from_blocks(s, w, s["copy"])
    return [s["weights"], s["m_value"], s["v_value"]] + ([s["copy"]] if "copy" in s else [])


_PLAIN = {"loss": _plain_loss, "gradient": _plain_gradient, "adamw8": _plain_adamw8}


def run(state):
    s = state
    c = s["case"]
    if not own:
        return _PLAIN[c["op"]](s)
    import sgd_gradient_all_amd as ddl
    if c["op"] == "loss":
        ddl.cross_entropy(s["x"], s["w"], s["target"], s["loss"], s["lse"], bias=s["bias"],
                          smoothing=c["smoothing"], workspace=s["workspace"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if c["op"] == "gradient":
        ddl.cross_entropy_grad(s["x"], s["w"], s["target"], s["lse"], dloss=s["dloss"],
                               dx=s["dx"], dw=s["dw"], db=s["db"], bias=s["bias"],
                               smoothing=c["smoothing"], accumulate=c["add"],
                               workspace=s["workspace"])
        out = {"dx": s["dx"], "dw": s["dw"]}
        return out if s["db"] is None else dict(out, db=s["db"])
    states = s["m"], s["v"], s["m_scale"], s["v_scale"]
    s["handle"].step(s["grad"], *states, [s["weights"]], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                     weight_decay=DECAY, step=STEP, copy=s.get("copy"))
    # the states as the values that they stand for, as a checkpoint takes them
    s["handle"].values(*states, s["m_value"], s["v_value"])
    return [s["weights"], s["m_value"], s["v_value"]] + ([s["copy"]] if "copy" in s else [])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s, d = prepare(case, seed), torch.float64
    if case["op"] == "adamw8":
        return _exact_adamw8(case, s)
    a, n = case["smoothing"], case["n"]
    x, w, have = s["x"].to(d), s["w"].to(d), s["target"] >= 0
    z = torch.mm(x, w.t().contiguous())
    if s["bias"] is not None:
        z += s["bias"].to(d)
    # what the loss wants: the target's class, mixed with all of them evenly
    rows = torch.nonzero(have)[:, 0]
    cols = s["target"][rows]
    if case["op"] == "loss":
        lse = torch.logsumexp(z, 1)
        loss = lse - a * z.mean(1)
        loss[rows] -= (1 - a) * z[rows, cols]
        return {"loss": loss.masked_fill(~have, 0.0), "lse": lse.masked_fill(~have, 0.0)}
    z = z.sub_(s["lse"].to(d)[:, None]).exp_().sub_(a / n)
    z[rows, cols] -= 1 - a
    z = z.mul_(s["dloss"].to(d)[:, None]).masked_fill_(~have[:, None], 0.0)
    out = {"dx": torch.mm(z, w), "dw": torch.mm(z.t().contiguous(), x)}
    if s["db"] is not None:
        out["db"] = z.sum(0)
    if case["add"]:
        out["dw"] += s["dw"]
        if s["db"] is not None:
            out["db"] += s["db"]
    return out


def _exact_adamw8(case, s):
    # the borders between neighbouring codes, as parts of the scale
    m_border = ((2 * torch.arange(127, device="cuda", dtype=torch.float64) + 1) / 254) ** 2
    v_border = ((2 * torch.arange(255, device="cuda", dtype=torch.float64) + 1) / 510) ** 4
    g, w = s["grad"].double(), s["weights"].double()
    mv, vv = s["m_value"].double(), s["v_value"].double()
    copy = [s["copy"].double()] if "copy" in s else []
    first = 0
    for o, c in s["spans"]:
        at, rows = slice(o, o + c), -(-c // BLOCK)
        block = torch.arange(c, device="cuda") // BLOCK
        ms, vs = (s[q][first:first + rows] for q in ("m_scale", "v_scale"))
        first += rows
        k, h = s["m"][at].double(), s["v"][at].double()
        m = BETA1 * (k * k.abs() / 16129 * ms.double()[block]) + (1 - BETA1) * g[at]
        v = BETA2 * ((h / 255) ** 4 * vs.double()[block]) + (1 - BETA2) * g[at] ** 2
        hat = (v / (1 - BETA2 ** STEP)).sqrt() + EPS
        w[at] -= LR * (m / (1 - BETA1 ** STEP) / hat + DECAY * w[at])
        top = torch.zeros(2, rows, device="cuda", dtype=torch.float64)
        top[0].scatter_reduce_(0, block, m.abs(), "amax")
        top[1].scatter_reduce_(0, block, v, "amax")
        top = top.float().double()
        safe = torch.where(top > 0, top, torch.ones_like(top))
        k = torch.bucketize(m.abs() / safe[0][block], m_border).double()
        h = torch.bucketize(v / safe[1][block], v_border).double()
        mv[at] = torch.sign(m) * (k / 127) ** 2 * top[0][block]
        vv[at] = (h / 255) ** 4 * top[1][block]
        for cp in copy:
            cp[at] = w[at]
    return [w, mv, vv] + copy
