"""The linear layer, Muon and AdamW on the GPU against plain forms in 64 bits.

Tolerances.  u(t) = finfo(t).eps / 2 is a type's rounding.  A product's sums
are binary32: k terms of magnitude |x||w| leave at most k u(f32) sum|x||w|,
and each output is rounded once; activations are within 8 u(f32) of their
value and their slopes at most 1.13.
"""
import ctypes
import math

import pytest
import torch

import sgd_gradient_all_amd as ddl

pytestmark = pytest.mark.gpu

F32 = torch.finfo(torch.float32).eps / 2
T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def u(t):
    return torch.finfo(t).eps / 2


def normal(gen, *shape, sigma=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * sigma).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def workspace(op, m, n, k):
    return torch.empty(ddl.linear_workspace(op, m, n, k), device="cuda", dtype=torch.uint8)


def strided(t, pad, first=0):
    """t with `pad` more elements between its rows, starting `first` elements in."""
    r, c = t.shape
    flat = torch.full((first + r * (c + pad),), float("nan"), device=t.device, dtype=t.dtype)
    view = flat[first:].view(r, c + pad)[:, :c]
    view.copy_(t)
    return view


def act64(z, act):
    return {"none": lambda: z.clone(), "relu": lambda: z.clamp(min=0),
            "gelu": lambda: z * torch.special.ndtr(z),
            "gelu_tanh": lambda: z * torch.sigmoid(
                2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def near(got, want, slack):
    """|got - want| <= slack + one rounding to got's type."""
    t = got.dtype
    tiny = torch.finfo(t).tiny * u(t)
    limit = slack + (want.abs() + slack) * u(t) + tiny
    d = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    bad = d > limit
    assert not bad.any(), f"{int(bad.sum())} off, most {float((d - limit).max())}"


SIZES = [(1, 1, 1), (1, 64, 64), (2, 8, 2047), (5, 9, 7), (17, 130, 72), (64, 64, 64),
         (65, 63, 65), (129, 257, 130), (256, 256, 320), (300, 520, 2056), (1, 1000, 4096),
         (16, 4096, 512), (33, 1000, 2048), (2049, 2056, 64),
         (3, 2050, 264), (1, 2048, 2056)]
LAYOUTS = {"dense": (0, 0), "odd rows": (3, 0), "padded": (8, 0), "off by one": (0, 1)}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear(m, n, k, dtype):
    t, g = T[dtype], gen(m + 3 * n + 7 * k)
    x, w = normal(g, m, k, dtype=t), normal(g, n, k, sigma=k ** -0.5, dtype=t)
    b, r = normal(g, n, sigma=0.1, dtype=t), normal(g, m, n, dtype=t)
    zw = x.double() @ w.double().t().contiguous() + b.double()
    slack = (k + 4) * F32 * (x.double().abs() @ w.double().abs().t().contiguous()
                             + b.double().abs())
    for i, (act, layout) in enumerate([("none", "dense"), ("relu", "odd rows"),
                                       ("gelu", "padded"), ("gelu_tanh", "off by one"),
                                       ("silu", "dense")]):
        pad, first = LAYOUTS[layout]
        print(f"linear {m} {n} {k} {dtype} {act} {layout}", flush=True)
        y = strided(torch.zeros(m, n, device="cuda", dtype=t), pad, first)
        z = strided(torch.zeros(m, n, device="cuda", dtype=t), pad, first)
        ddl.linear(strided(x, pad, first), strided(w, pad, first), y, bias=b, act=act,
                   residual=strided(r, pad, first), z=z,
                   workspace=workspace("forward", m, n, k))
        near(z, zw, slack)
        a = act64(zw, act)
        near(y, a + r.double(), 1.13 * slack + 8 * F32 * (a.abs() + r.double().abs()))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_input_gradient(m, n, k, dtype):
    t, g = T[dtype], gen(m + 5 * n + 11 * k)
    dz, w = normal(g, m, n, dtype=t), normal(g, n, k, sigma=n ** -0.5, dtype=t)
    r, z = normal(g, m, k, dtype=t), normal(g, m, k, dtype=t)
    want = dz.double() @ w.double() + r.double()
    slack = (n + 4) * F32 * (dz.double().abs() @ w.double().abs() + r.double().abs())
    for act, layout in [("none", "odd rows"), ("relu", "dense"), ("gelu", "off by one"),
                        ("gelu_tanh", "padded"), ("silu", "dense")]:
        pad, first = LAYOUTS[layout]
        print(f"dgrad {m} {n} {k} {dtype} {act} {layout}", flush=True)
        dx = strided(torch.zeros(m, k, device="cuda", dtype=t), pad, first)
        dp = strided(torch.zeros(m, k, device="cuda", dtype=t), pad, first)
        ddl.linear_dgrad(strided(dz, pad, first), strided(w, pad, first), dx,
                         residual=strided(r, pad, first), act=act, z_prev=strided(z, pad, first),
                         dz_prev=dp, workspace=workspace("dgrad", m, n, k))
        near(dx, want, slack)
        zz = z.double().requires_grad_()
        slope, = torch.autograd.grad(act64(zz, act).sum(), zz)
        near(dp, want * slope, slack * 1.13 + 16 * F32 * want.abs() * (1 + z.double().abs()))


@pytest.mark.parametrize("dtype,out", [("f16", "f32"), ("bf16", "f32"), ("f16", "f16"),
                                       ("bf16", "bf16")])
@pytest.mark.parametrize("m,n,k", SIZES + [(4096, 64, 72), (0, 5, 6)])
def test_weight_gradient(m, n, k, dtype, out):
    t, g = T[dtype], gen(m + 13 * n + 17 * k)
    dz, x = normal(g, m, n, dtype=t), normal(g, m, k, dtype=t)
    dw0, db0 = normal(g, n, k, dtype=T[out]), normal(g, n, dtype=T[out])
    want = dz.double().t().contiguous() @ x.double()
    slack = (m + 2) * F32 * (dz.double().abs().t().contiguous() @ x.double().abs())
    bwant, bslack = dz.double().sum(0), (m + 2) * F32 * dz.double().abs().sum(0)
    for add, (pad, first) in ((False, (0, 0)), (True, (0, 0)), (True, (3, 1)), (False, (8, 0))):
        print(f"wgrad {m} {n} {k} {dtype} {out} {add} {pad} {first}", flush=True)
        dw, db = strided(dw0, pad, first), db0.clone()
        ddl.linear_wgrad(strided(dz, pad, first), strided(x, pad, first), dw, db=db,
                         accumulate=add, workspace=workspace("wgrad", m, n, k))
        old, bold = (dw0.double(), db0.double()) if add else (0 * dw0.double(), 0 * db0.double())
        near(dw, want + old, slack + F32 * (want + old).abs() * 2)
        near(db, bwant + bold, bslack + F32 * (bwant + bold).abs() * 2)


def test_empty_sums_and_extents():
    t = torch.bfloat16
    e = lambda *s: torch.empty(*s, device="cuda", dtype=t)  # noqa: E731
    b, y = normal(gen(1), 6, dtype=t), normal(gen(2), 4, 6, dtype=t)
    ddl.linear(e(4, 0), e(6, 0), y, bias=b, act="relu")
    assert torch.equal(y, b.clamp(min=0).expand(4, 6))
    ddl.linear(e(0, 3), e(6, 3), e(0, 6))
    dx = normal(gen(3), 4, 5, dtype=t)
    ddl.linear_dgrad(e(4, 0), e(0, 5), dx)
    assert (dx == 0).all()


def test_nan_stays_in_its_row_and_tail():
    """NaN of one row reaches that row alone; NaN beside a row reaches none."""
    t, g = torch.float16, gen(4)
    x, w = normal(g, 70, 100, dtype=t), normal(g, 66, 100, sigma=0.1, dtype=t)
    x[3, 99] = float("nan")
    for pad in (4, 1):  # direct and staged copies; the padding itself is NaN
        y = torch.empty(70, 66, device="cuda", dtype=t)
        ddl.linear(strided(x, pad), strided(w, pad), y, workspace=workspace("forward", 70, 66, 100))
        assert torch.isnan(y[3]).all()
        assert torch.isfinite(torch.cat([y[:3], y[4:]])).all()


def test_residual_in_place():
    t, g = torch.float16, gen(5)
    for m, n, k in ((40, 48, 4096), (300, 264, 128)):
        x, w, r = normal(g, m, k, dtype=t), normal(g, n, k, sigma=k ** -0.5, dtype=t), \
            normal(g, m, n, dtype=t)
        ws = workspace("forward", m, n, k)
        y = torch.empty_like(r)
        ddl.linear(x, w, y, residual=r, workspace=ws)
        ddl.linear(x, w, r, residual=r, workspace=ws)
        assert torch.equal(r, y)


def test_gradients_against_differences():
    """A two-layer loss: the three calls' gradients against central differences."""
    g, t = gen(6), torch.bfloat16
    m, k, h = 24, 40, 56
    x, w1, b1 = normal(g, m, k, dtype=t), normal(g, h, k, sigma=0.2, dtype=t), \
        normal(g, h, sigma=0.1, dtype=t)
    w2, c = normal(g, 8, h, sigma=0.2, dtype=t), normal(g, m, 8, dtype=t)

    def loss(w1, b1):
        return (act64(x.double() @ w1.t().contiguous() + b1, "silu")
                @ w2.double().t().contiguous() * c.double()).sum()

    z1 = torch.empty(m, h, device="cuda", dtype=t)
    a1, da, dz = torch.empty_like(z1), torch.empty_like(z1), torch.empty_like(z1)
    ddl.linear(x, w1, a1, bias=b1, act="silu", z=z1, workspace=workspace("forward", m, h, k))
    ddl.linear_dgrad(c, w2, da, act="silu", z_prev=z1, dz_prev=dz,
                     workspace=workspace("dgrad", m, 8, h))
    dw, db = torch.empty(h, k, device="cuda"), torch.empty(h, device="cuda")
    ddl.linear_wgrad(dz, x, dw, db=db, workspace=workspace("wgrad", m, h, k))
    p, q = w1.double(), b1.double()
    # z1 and dz are rounded once each to bfloat16: SiLU's slope changes by at
    # most half of a change of its argument
    scale = (c.double().abs() @ w2.double().abs()) * (1.1 + 0.5 * z1.double().abs()) * u(t)
    for i, j in ((0, 0), (7, 11), (55, 39)):
        d = torch.zeros_like(p)
        d[i, j] = 1e-4
        want = (loss(p + d, q) - loss(p - d, q)) / 2e-4
        limit = float((scale[:, i] * x[:, j].double().abs()).sum()) + 1e-5
        assert abs(float(want) - float(dw[i, j])) <= limit
        e = torch.zeros_like(q)
        e[i] = 1e-4
        want = (loss(p, q + e) - loss(p, q - e)) / 2e-4
        assert abs(float(want) - float(db[i])) <= float(scale[:, i].sum()) + 1e-5


def test_other_stream_and_repeats():
    """The same bits on another stream, and from call to call."""
    t, g = torch.bfloat16, gen(7)
    m, n, k = 96, 200, 4096  # cut along k
    x, w = normal(g, m, k, dtype=t), normal(g, n, k, dtype=t)
    ws = workspace("forward", m, n, k)
    y = torch.empty(m, n, device="cuda", dtype=t)
    ddl.linear(x, w, y, workspace=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    z = torch.empty_like(y)
    for _ in range(5):
        z.zero_()
        torch.cuda.synchronize()
        ddl.linear(x, w, z, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(y, z)


# ---------------------------------------------------------------------------
# Muon
# ---------------------------------------------------------------------------

def orthogonal64(x):
    tall = x.shape[0] > x.shape[1]
    x = (x.t() if tall else x).double()
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        a = x @ x.t().contiguous()
        x = 3.4445 * x + (-4.7750 * a + 2.0315 * (a @ a)) @ x
    return x.t() if tall else x


def pack(gap, shapes):
    at, out = 0, []
    for r, c in shapes:
        out.append((at, r, c))
        at += r * c + gap
    return out, at


SHAPES = [[(1, 1)], [(1, 7), (7, 1)], [(16, 17)], [(64, 64), (64, 147), (33, 300)],
          [(300, 33), (65, 64)], [(128, 640)], [(1000, 129)], [(520, 520), (0, 4), (4, 4)]]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shapes", SHAPES, ids=str)
@pytest.mark.parametrize("gap", [0, 3])
def test_orthogonalise(shapes, dtype, gap):
    t = T[dtype]
    mats, size = pack(gap, shapes)
    h = ddl.Muon([(o, r, c, 1.0) for o, r, c in mats])
    u_ = normal(gen(size), size + 1, sigma=1e-2, dtype=t)
    out = torch.full_like(u_, 7.0)
    print(f"orthogonalise {shapes} {dtype} {gap}", flush=True)
    h.orthogonalise(u_, out)
    inside = torch.zeros_like(u_, dtype=torch.bool)
    # relative to the result: pairs hold 2^-22, and five rounds multiply a
    # rounding of X by up to 3.4445^5 = 485 where its singular values are tiny
    # and by tens on the whole: 64 * 2^-22.  bfloat16's passes keep 2^-12 of
    # some factors: 16 * 2^-12.
    limit = 16 * 2.0 ** -12 if dtype == "bf16" else 64 * 2.0 ** -22
    for o, r, c in mats:
        inside[o:o + r * c] = True
        if r * c:
            want = orthogonal64(u_[o:o + r * c].view(r, c))
            got = out[o:o + r * c].view(r, c).double()
            assert float((got - want).norm() / want.norm()) <= limit + u(t)
    assert (out[~inside] == 7.0).all()
    again = torch.full_like(u_, 7.0)
    h.orthogonalise(u_, again)
    assert torch.equal(out, again)
    h.orthogonalise(u_, u_)  # in place
    assert torch.equal(out[inside], u_[inside])


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("grad,copy,nesterov,replicas", [
    ("f32", None, True, 1), ("f16", "f16", False, 3), ("bf16", "bf16", True, 2)])
def test_muon_step(grad, copy, nesterov, replicas, offset):
    mats, size = pack(5, [(100, 40), (24, 72), (200, 200)])
    scales = [0.2 * math.sqrt(max(r, c)) for _, r, c in mats]
    h = ddl.Muon([(o, r, c, s) for (o, r, c), s in zip(mats, scales)])
    g_ = gen(9)
    mk = lambda t, sigma: normal(g_, size + offset, sigma=sigma, dtype=t)[offset:]  # noqa: E731
    grad_, mom, w = mk(T[grad], 1e-2), mk(torch.float32, 3e-2), mk(torch.float32, 0.02)
    ws = [w.clone() for _ in range(replicas)]
    cp = torch.full((size,), 5.0, device="cuda", dtype=T[copy]) if copy else None
    lr, mu, wd = 0.02, 0.95, 0.1
    m64, w64 = mom.double(), w.double()
    mom = mom.clone()
    for step in range(2):
        print(f"muon {grad} {copy} {nesterov} {replicas} {offset} step {step}", flush=True)
        before = mom.clone()
        h.step(grad_, mom, ws, lr=lr, momentum_decay=mu, nesterov=nesterov, weight_decay=wd,
               copy=cp)
        inside = torch.zeros(size, device="cuda", dtype=torch.bool)
        for (o, r, c), s in zip(mats, scales):
            at = slice(o, o + r * c)
            inside[at] = True
            gg = grad_[at].double()
            m64[at] = mu * m64[at] + gg
            # three roundings a step
            assert ((mom[at].double() - m64[at]).abs()
                    <= 4 * (step + 1) * F32 * (m64[at].abs() + gg.abs() + 0.1)).all()
            x = orthogonal64((gg + mu * m64[at] if nesterov else m64[at]).view(r, c))
            w64[at] = (1 - lr * wd) * w64[at] - lr * s * x.reshape(-1)
            err = (ws[0][at].double() - w64[at]).norm()
            assert float(err) <= (step + 1) * (64 * 2.0 ** -22 * lr * s * float(x.norm())
                                               + 4 * F32 * float(w64[at].norm()))
        assert torch.equal(mom[~inside], before[~inside])
        for k in ws[1:]:
            assert torch.equal(k[inside], ws[0][inside])
        assert torch.equal(ws[0][~inside], w[~inside])
        if copy:
            assert torch.equal(cp[inside], ws[0][inside].to(T[copy]))
            assert (cp[~inside] == 5.0).all()


def test_muon_zero_and_nan_matrices():
    """A zero matrix stays zero; NaN and infinities spoil their own matrix alone."""
    mats, size = pack(0, [(40, 40), (70, 20), (20, 70), (30, 30)])
    h = ddl.Muon([(o, r, c, 1.0) for o, r, c in mats])
    u_ = normal(gen(10), size)
    o, r, c = mats[0]
    u_[o:o + r * c] = 0
    u_[mats[1][0] + 5] = float("nan")
    u_[mats[2][0] + 5] = float("inf")
    out = torch.empty_like(u_)
    h.orthogonalise(u_, out)
    part = lambda i: out[mats[i][0]:mats[i][0] + mats[i][1] * mats[i][2]]  # noqa: E731
    assert (part(0) == 0).all()
    assert torch.isnan(part(1)).all() and torch.isnan(part(2)).all()
    assert torch.isfinite(part(3)).all()


def test_muon_scales_and_rank():
    """Huge and tiny matrices give the same as ordinary ones (a power of two
    passes through exactly), and a matrix of rank 1 keeps its direction."""
    x = normal(gen(11), 48 * 80)
    h = ddl.Muon([(0, 48, 80, 1.0)])
    outs = []
    for e in (0, 60, 100):
        out = torch.empty_like(x)
        h.orthogonalise(x * 2.0 ** e, out)
        outs.append(out)
    # the norm's eps is 1e-7 of numbers near 60: below binary32's rounding
    assert float((outs[0] - outs[1]).norm()) <= 64 * 2.0 ** -22 * float(outs[0].norm())
    assert torch.equal(outs[1], outs[2])
    a, b = normal(gen(12), 48, 1), normal(gen(13), 1, 80)
    one, out = (a @ b).contiguous().view(-1), torch.empty(48 * 80, device="cuda")
    h.orthogonalise(one, out)
    want = orthogonal64(one.view(48, 80))
    assert float((out.view(48, 80).double() - want).norm() / want.norm()) <= 512 * 2.0 ** -22


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("grad,copy,replicas", [("f32", None, 1), ("f16", "f16", 1),
                                                ("bf16", "bf16", 3), ("f32", "bf16", 2)])
@pytest.mark.parametrize("offset", [0, 1])
def test_adamw(grad, copy, replicas, offset):
    spans = [(0, 1), (3, 5), (16, 4096), (5000, 2047), (9001, 1), (9010, 0), (9016, 3)]
    size = 9100
    h = ddl.AdamW(spans)
    g_ = gen(14)
    mk = lambda t, sigma: normal(g_, size + offset, sigma=sigma, dtype=t)[offset:]  # noqa: E731
    gr, m, v, w = mk(T[grad], 1e-2), mk(torch.float32, 1e-2), mk(torch.float32, 1e-2).square(), \
        mk(torch.float32, 0.02)
    m, v = m.clone() if not offset else m, v if not offset else v.clone()
    ws = [w.clone() for _ in range(replicas)]
    cp = torch.full((size,), 5.0, device="cuda", dtype=T[copy]) if copy else None
    inside = torch.zeros(size, device="cuda", dtype=torch.bool)
    for o, c in spans:
        inside[o:o + c] = True
    m0, v0, w0 = m.clone(), v.clone(), w.clone()
    lr, b1, b2, eps, wd, step = 2e-3, 0.9, 0.95, 1e-8, 0.1, 3
    h.step(gr, m, v, ws, lr=lr, beta1=b1, beta2=b2, eps=eps, weight_decay=wd, step=step, copy=cp)
    gd = gr.double()
    md, vd = b1 * m0.double() + (1 - b1) * gd, b2 * v0.double() + (1 - b2) * gd * gd
    up = (md / (1 - b1 ** step)) / ((vd / (1 - b2 ** step)).sqrt() + eps)
    wd_ = w0.double() * (1 - lr * wd) - lr * up
    ins = lambda t: t[inside]  # noqa: E731
    mag = b1 * m0.double().abs() + (1 - b1) * gd.abs()
    # each coefficient, product and sum rounded: 4 a term
    assert (ins((m.double() - md).abs()) <= ins(4 * F32 * mag)).all()
    assert (ins((v.double() - vd).abs()) <= ins(6 * F32 * vd)).all()
    big = lr * (mag / (1 - b1 ** step)) / ((vd / (1 - b2 ** step)).sqrt() + eps)
    assert (ins((ws[0].double() - wd_).abs()) <= ins(16 * F32 * big + 4 * F32 * w0.abs())).all()
    for t, t0 in ((m, m0), (v, v0), (ws[0], w0)):
        assert torch.equal(t[~inside], t0[~inside])
    for k in ws[1:]:
        assert torch.equal(k[inside], ws[0][inside]) and torch.equal(k[~inside], w0[~inside])
    if copy:
        assert torch.equal(cp[inside], ws[0][inside].to(T[copy]))
        assert (cp[~inside] == 5.0).all()


def test_a_whole_step_in_a_graph():
    """Forward, both gradients, Muon and AdamW captured; replays with eager
    work between them give the eager bits."""
    t, m, n, k = torch.bfloat16, 80, 96, 136
    g_ = gen(15)
    x, dz = normal(g_, m, k, dtype=t), normal(g_, m, n, dtype=t)
    z, y, dx = torch.empty(m, n, device="cuda", dtype=t), torch.empty(
        m, n, device="cuda", dtype=t), torch.empty(m, k, device="cuda", dtype=t)
    grad = torch.empty(n * k + n, device="cuda")
    wcopy = normal(g_, n * k + n, sigma=0.1, dtype=t)
    start = dict(w=wcopy.float(), mom=torch.zeros(n * k + n, device="cuda"),
                 m=torch.zeros(n * k + n, device="cuda"), v=torch.zeros(n * k + n, device="cuda"))
    muon, adam = ddl.Muon([(0, n, k, 0.2)]), ddl.AdamW([(n * k, n)])
    size = max(ddl.linear_workspace(op, m, n, k) for op in ("forward", "dgrad", "wgrad"))
    ws = torch.empty(size, device="cuda", dtype=torch.uint8)

    def step(s, st):
        w16, b16 = wcopy[:n * k].view(n, k), wcopy[n * k:]
        ddl.linear(x, w16, y, bias=b16, act="silu", z=z, workspace=ws, stream=st)
        ddl.linear_dgrad(dz, w16, dx, workspace=ws, stream=st)
        ddl.linear_wgrad(dz, x, grad[:n * k].view(n, k), db=grad[n * k:], workspace=ws, stream=st)
        muon.step(grad, s["mom"], [s["w"]], lr=1e-2, copy=wcopy, stream=st)
        adam.step(grad, s["m"], s["v"], [s["w"]], lr=1e-2, step=1, copy=wcopy, stream=st)

    kept = wcopy.clone()
    eager = {q: v.clone() for q, v in start.items()}
    want = []
    for _ in range(3):
        step(eager, None)
        torch.cuda.synchronize()
        want.append([v.clone() for v in eager.values()] + [y.clone(), dx.clone(), wcopy.clone()])
    state = {q: v.clone() for q, v in start.items()}
    wcopy.copy_(kept)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        step(state, s)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got = list(state.values()) + [y, dx, wcopy]
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), f"replay {i}"
        (torch.randn(64, 64, device="cuda") @ torch.randn(64, 64, device="cuda")).sum().item()


def test_first_call_in_a_capture_is_refused():
    h = ddl.AdamW([(0, 8)])
    v = [torch.zeros(8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        v[0].add_(1)
        with pytest.raises(ddl.DDLError) as e:
            h.step(v[0], v[1], v[2], [v[3]], lr=1e-3, stream=s)
    assert e.value.code == -9


def test_training_example():
    """The example's loss falls, and two runs give the same numbers."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_mlp.py")
    spec = importlib.util.spec_from_file_location("train_mlp", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(steps=12)
    assert losses == mod.train(steps=12)
    assert losses[-1] < 0.5 * losses[0]


@pytest.mark.parametrize("r,c", [(1, 3), (40, 40), (200, 70), (130, 513)])
def test_binary32_orthogonalise_is_rounded_once(r, c):
    """Computed in binary64: what is left is the result's own rounding (five
    rounds of binary64 products leave below 485 * 1e3 * 2^-53 = 6e-11)."""
    x, out = normal(gen(r * c), r * c), torch.empty(r * c, device="cuda")
    ddl.Muon([(0, r, c, 1.0)]).orthogonalise(x, out)
    want = orthogonal64(x.view(r, c))
    near(out.view(r, c), want, 1e-10 * float(want.norm()))


def test_offsets_past_32_bits():
    """The last rows of arrays of more than 2^32 elements."""
    t, g = torch.bfloat16, gen(21)
    m, n, k = (1 << 21) + 5, 16, 2056
    x = torch.empty(m, k, device="cuda", dtype=t).normal_(generator=g)
    w = normal(g, n, k, sigma=k ** -0.5, dtype=t)
    y = torch.empty(m, n, device="cuda", dtype=t)
    print("forward past 32 bits", flush=True)
    ddl.linear(x, w, y, workspace=workspace("forward", m, n, k))
    tail = slice(m - 300, m)
    xd, wd = x[tail].double(), w.double()
    near(y[tail], xd @ wd.t().contiguous(),
         (k + 4) * F32 * (xd.abs() @ wd.abs().t().contiguous()))
    print("dgrad past 32 bits", flush=True)
    ddl.linear_dgrad(y, w, x, workspace=workspace("dgrad", m, n, k))
    yd = y[tail].double()
    near(x[tail], yd @ wd, (n + 4) * F32 * (yd.abs() @ wd.abs()))
    print("wgrad past 32 bits", flush=True)
    # one row in the far end of dz alone: dw is that row's outer product
    y.zero_()
    y[m - 2] = normal(g, 16, dtype=t)
    dw, db = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    ddl.linear_wgrad(y, x, dw, db=db, workspace=workspace("wgrad", m, n, k))
    assert torch.equal(db, y[m - 2].float())
    near(dw, y[m - 2].double()[:, None] * x[m - 2].double()[None, :],
         torch.zeros((), device="cuda", dtype=torch.float64))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_result_does_not_depend_on_the_other_matrices(dtype):
    """The same bits alone and beside a larger matrix: both handles take 64 x 64
    tiles, and none of the sums is long enough to be cut."""
    t, (r, c) = T[dtype], (100, 120)
    x = normal(gen(31), r * c + 200 * 200, sigma=1e-2, dtype=t)
    alone, beside = torch.empty_like(x), torch.empty_like(x)
    ddl.Muon([(0, r, c, 1.0)]).orthogonalise(x, alone)
    ddl.Muon([(0, r, c, 1.0), (r * c, 200, 200, 1.0)]).orthogonalise(x, beside)
    assert torch.equal(alone[:r * c], beside[:r * c])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("r,c", [(300, 640), (640, 300), (256, 256)])
def test_orthogonalise_is_rounded_once(r, c, dtype):
    """Pairs of binary16 values leave e with |e| <= 64 * 2^-22 of the result in
    norm, so a 16-bit result is the exact one's rounding but where e crosses
    the border between two: in |e| / step of the places on the average.  Steps
    are u to 2 u of the value, so with values over a quarter of their mean
    square root, e / step is at most 4 * 64 * 2^-22 / u."""
    t = T[dtype]
    x = normal(gen(r + c), r * c, sigma=1e-2, dtype=t)
    out = torch.empty_like(x)
    ddl.Muon([(0, r, c, 1.0)]).orthogonalise(x, out)
    want = orthogonal64(x.view(r, c)).reshape(-1)
    ref = want.to(t)
    big = want.abs() >= want.square().mean().sqrt() / 4
    crossed = (out != ref) & big
    assert ((out.double() - ref.double()).abs()[big] <= 2 * u(t) * ref.double().abs()[big]).all()
    assert float(crossed.sum()) <= 4 * 64 * 2.0 ** -22 / u(t) * float(big.sum())


SMOOTH = ["gelu", "gelu_tanh", "silu"]


def slopes(values, act, t):
    """dz_prev at z_prev = values where dx is 1."""
    m, k = values.numel(), 8
    dz, w = torch.zeros(m, 8, device="cuda", dtype=t), torch.zeros(8, k, device="cuda", dtype=t)
    dz[:, 0], w[0] = 1, 1
    z = values[:, None].expand(m, k).contiguous()
    dx, dp = torch.empty_like(z), torch.empty_like(z)
    ddl.linear_dgrad(dz, w, dx, act=act, z_prev=z, dz_prev=dp,
                     workspace=workspace("dgrad", m, 8, k))
    assert (dx == 1).all()
    return dp


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_slopes_far_out(act, dtype):
    """The slope is 1 far to the right, 0 far to the left, and NaN at NaN."""
    t = T[dtype]
    far = [200.0, 1e4, 6e4, float("inf")] + ([1e12, 2e13, 1e19, 3e19, 1e30, 3e38]
                                             if dtype == "bf16" else [])
    v = torch.tensor(far, device="cuda").to(t)
    assert (slopes(v, act, t) == 1).all()
    assert (slopes(-v, act, t) == 0).all()
    assert torch.isnan(slopes(torch.full_like(v, float("nan")), act, t)).all()


def cdf64(z):
    """Phi(z) without the cancellation that torch.special.ndtr has on the left."""
    return 0.5 * torch.special.erfc(z * -math.sqrt(0.5))


def grid(t):
    """Arguments of the activations, and the size of the exponent that each
    form takes at them (the rounding of the exponent is that much of the
    result's relative error)."""
    v = torch.cat([torch.linspace(-12, 12, 769, device="cuda"),
                   torch.linspace(-1e-3, 1e-3, 21, device="cuda")]).to(t)
    a = v.double().abs()
    return v, {"gelu": a * a / 2, "gelu_tanh": 1.6 * a + 0.0714 * a ** 3, "silu": a}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_activations_in_their_tails(act, dtype):
    """Every value to its own relative error, the small ones of the left tail
    too: 8 roundings and 4 of the exponent.  Results under 2^-125 |v| may be 0
    (2^x leaves binary32's range)."""
    t = T[dtype]
    v, a = grid(t)
    m, n, k = v.numel(), 8, 8
    x, w = torch.zeros(m, k, device="cuda", dtype=t), torch.zeros(n, k, device="cuda", dtype=t)
    x[:, 0], w[:, 0] = v, 1
    y = torch.empty(m, n, device="cuda", dtype=t)
    ddl.linear(x, w, y, act=act, workspace=workspace("forward", m, n, k))
    z = v.double()
    want = z * cdf64(z) if act == "gelu" else act64(z, act)
    slack = (4 * a[act] + 8) * F32 * want.abs() + 2.0 ** -125 * z.abs()
    near(y, want[:, None].expand(m, n), slack[:, None])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_slopes_in_their_tails(act, dtype):
    """Slopes are a sum of two terms, each to its own relative error."""
    t = T[dtype]
    v, a = grid(t)
    z = v.double()
    if act == "gelu":
        p, q = cdf64(z), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        k = 2 * math.sqrt(2 / math.pi)
        arg, d = (z, 1.0) if act == "silu" else (k * (z + 0.044715 * z ** 3),
                                                 k * (1 + 0.134145 * z * z))
        p = torch.sigmoid(arg)
        q = z * d * p * torch.sigmoid(-arg)
    slack = (4 * a[act] + 8) * F32 * (p + q.abs()) + 2.0 ** -125 * (1 + z.abs() ** 3)
    got = slopes(v, act, t)
    near(got, (p + q)[:, None].expand(got.shape), slack[:, None])


def test_an_older_error_is_not_the_calls():
    """An error that an earlier call of the HIP runtime left behind (here an
    allocation of 2^60 bytes) is not reported by calls that succeed."""
    hip, p = ddl.lib(), ctypes.c_void_p()
    t, g_ = torch.bfloat16, gen(33)
    x, w, dz = (normal(g_, 64, 64, dtype=t) for _ in range(3))
    y, dw = torch.empty_like(x), torch.empty(64, 64, device="cuda")
    db = torch.empty(64, device="cuda")
    flat = [torch.zeros(4096, device="cuda") for _ in range(4)]
    muon, adam = ddl.Muon([(0, 64, 64, 1.0)]), ddl.AdamW([(0, 4096)])
    ws = workspace("wgrad", 64, 64, 64)
    torch.cuda.synchronize()
    calls = [lambda: ddl.linear(x, w, y, workspace=ws),
             lambda: ddl.linear_dgrad(dz, w, y, workspace=ws),
             lambda: ddl.linear_wgrad(dz, x, dw, db=db, workspace=ws),
             lambda: muon.step(flat[0], flat[1], [flat[2]], lr=0.1),
             lambda: muon.orthogonalise(flat[0], flat[1]),
             lambda: adam.step(flat[0], flat[1], flat[2], [flat[3]], lr=0.1)]
    try:
        for call in calls:
            assert hip.hipMalloc(ctypes.byref(p), ctypes.c_size_t(1 << 60)) != 0
            call()
    finally:
        hip.hipGetLastError()
        torch.cuda.synchronize()


def test_empty_sums_over_many_rows():
    """An empty sum's outputs (the bias alone) over more than 2^32 pieces of 8."""
    m, n, t = 1 << 30, 25, torch.bfloat16
    b = normal(gen(34), n, dtype=t)
    y = torch.zeros(m, n, device="cuda", dtype=t)
    e = torch.empty(m, 0, device="cuda", dtype=t)
    ddl.linear(e, torch.empty(n, 0, device="cuda", dtype=t), y, bias=b)
    for at in (0, m // 2, m - 1000):
        assert torch.equal(y[at:at + 1000], b.expand(1000, n))
    assert int((y[:, n - 1] != b[n - 1]).sum()) == 0


# ---------------------------------------------------------------------------
# the tiles of large products
# ---------------------------------------------------------------------------

def tiles(m, n, t):
    return -(-m // t) * -(-n // t)


def linear_tile(m, n, k):
    """(side of the tile, parts of k) by the library's rule for an m x n output."""
    t = 256 if tiles(m, n, 256) >= 192 else 128 if tiles(m, n, 128) >= 192 else 64
    have, kt = tiles(m, n, t), -(-k // 64)
    return t, max(1, min(512 // have, kt // 8, 64)) if have < 256 and kt >= 16 else 1


def muon_tile(shapes):
    def up(n, t):
        return -(-n // t) * t

    def lower(t):
        return sum(up(min(s), t) // t * (up(min(s), t) // t + 1) // 2 for s in shapes)

    def issued(t):
        both = [(up(min(s), t), up(max(s), t)) for s in shapes]
        return sum(s * (s + t) / 2 * (n + s) + s * s * n for s, n in both)
    if lower(128) < 128 or issued(128) > 1.45 * issued(64):
        return 64
    return 256 if lower(256) >= 256 and issued(256) <= 1.03 * issued(128) else 128


# (side, parts, rows and columns of the output, length of the sums)
LARGE = [(128, 1, 1496, 2104, 200), (128, 2, 1496, 2104, 1096), (256, 1, 3600, 3400, 264),
         (256, 2, 3600, 3400, 1096), (128, 2, 1501, 2099, 1097), (256, 1, 3601, 3403, 203),
         (256, 2, 3601, 3403, 1097)]
LARGE_IDS = [f"{s[0]}x{s[1]}-{s[2]}x{s[3]}x{s[4]}" for s in LARGE]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("side,parts,m,n,k", LARGE, ids=LARGE_IDS)
def test_linear_large_tiles(side, parts, m, n, k, dtype):
    assert linear_tile(m, n, k) == (side, parts)
    t, g_ = T[dtype], gen(m + n + k)
    x, w = normal(g_, m, k, dtype=t), normal(g_, n, k, sigma=k ** -0.5, dtype=t)
    b, r = normal(g_, n, sigma=0.1, dtype=t), normal(g_, m, n, dtype=t)
    zw = x.double() @ w.double().t().contiguous() + b.double()
    slack = (k + 4) * F32 * (x.double().abs() @ w.double().abs().t().contiguous()
                             + b.double().abs())
    y, z = (torch.empty(m, n, device="cuda", dtype=t) for _ in range(2))
    ws = workspace("forward", m, n, k)
    for act in ("none", "gelu", "gelu_tanh"):
        print(f"linear {m} {n} {k} {dtype} {act}", flush=True)
        ddl.linear(x, w, y, bias=b, act=act, residual=r, z=z, workspace=ws)
        a = act64(zw, act)
        near(z, zw, slack)
        near(y, a + r.double(), 1.13 * slack + 8 * F32 * (a.abs() + r.double().abs()))
    print(f"linear {m} {n} {k} {dtype} alone", flush=True)
    ddl.linear(x, w, y, workspace=ws)
    near(y, zw - b.double(), slack)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("side,parts,m,k,n", LARGE, ids=LARGE_IDS)
def test_input_gradient_large_tiles(side, parts, m, k, n, dtype):
    assert linear_tile(m, k, n) == (side, parts)
    t, g_ = T[dtype], gen(m + n + k)
    dz, w = normal(g_, m, n, dtype=t), normal(g_, n, k, sigma=n ** -0.5, dtype=t)
    r, z = normal(g_, m, k, dtype=t), normal(g_, m, k, dtype=t)
    want = dz.double() @ w.double() + r.double()
    slack = (n + 4) * F32 * (dz.double().abs() @ w.double().abs() + r.double().abs())
    dx, dp = (torch.empty(m, k, device="cuda", dtype=t) for _ in range(2))
    for act in ("relu", "gelu", "silu"):
        print(f"dgrad {m} {n} {k} {dtype} {act}", flush=True)
        ddl.linear_dgrad(dz, w, dx, residual=r, act=act, z_prev=z, dz_prev=dp,
                         workspace=workspace("dgrad", m, n, k))
        near(dx, want, slack)
        zz = z.double().requires_grad_()
        slope, = torch.autograd.grad(act64(zz, act).sum(), zz)
        if act == "relu":  # at 0, which the inputs hold here and there, the slope is 0
            slope = (zz > 0).double()
        near(dp, want * slope, slack * 1.13 + 16 * F32 * want.abs() * (1 + z.double().abs()))


@pytest.mark.parametrize("dtype,out", [("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("side,parts,n,k,m", LARGE, ids=LARGE_IDS)
def test_weight_gradient_large_tiles(side, parts, n, k, m, dtype, out):
    assert linear_tile(n, k, m) == (side, parts)
    t, g_ = T[dtype], gen(m + n + k)
    dz, x = normal(g_, m, n, dtype=t), normal(g_, m, k, dtype=t)
    dw0, db0 = normal(g_, n, k, dtype=T[out]), normal(g_, n, dtype=T[out])
    want = dz.double().t().contiguous() @ x.double()
    slack = (m + 2) * F32 * (dz.double().abs().t().contiguous() @ x.double().abs())
    bwant, bslack = dz.double().sum(0), (m + 2) * F32 * dz.double().abs().sum(0)
    for add in (False, True):
        print(f"wgrad {m} {n} {k} {dtype} {out} {add}", flush=True)
        dw, db = dw0.clone(), db0.clone()
        ddl.linear_wgrad(dz, x, dw, db=db, accumulate=add, workspace=workspace("wgrad", m, n, k))
        old, bold = (dw0.double(), db0.double()) if add else (0 * dw0.double(), 0 * db0.double())
        near(dw, want + old, slack + F32 * (want + old).abs() * 2)
        near(db, bwant + bold, bslack + F32 * (bwant + bold).abs() * 2)


# 128: sums in three parts; 256: whole sums, and sums of one long matrix in parts
MUON_LARGE = [(128, [(2000, 2300)]), (128, [(2300, 2000)]),
              (128, [(2100, 2300)] * 3 + [(2300, 2100)] * 3),
              (256, [(2300, 2304)] * 4 + [(2304, 2300)] * 4),
              (256, [(2300, 2304)] * 8 + [(2290, 40000)]),
              (256, [(2304, 2300)] * 8 + [(40000, 2290)])]
MUON_IDS = [f"{side}-{len(s)}x{s[-1][0]}x{s[-1][1]}" for side, s in MUON_LARGE]


@pytest.mark.parametrize("side,shapes", MUON_LARGE, ids=MUON_IDS)
def test_muon_large_tiles(side, shapes):
    """A step, and orthogonalise in both 16-bit types.  The bound is four times
    2^-20, the binary32 products' error that the entry point documents as 2e-6."""
    assert muon_tile(shapes) == side
    mats, size = pack(1, shapes)
    h = ddl.Muon([(o, r, c, 0.5) for o, r, c in mats])
    g_ = gen(size)
    lr, mu = 0.5, 0.9
    grad, mom = normal(g_, size, sigma=1e-2), normal(g_, size, sigma=3e-2)
    w = normal(g_, size, sigma=0.02)
    m64, w0 = mom.double(), w.double()
    print(f"muon {side} {shapes[-1]}", flush=True)
    h.step(grad, mom, [w], lr=lr, momentum_decay=mu, weight_decay=0.1)
    outs = {}
    for t in (torch.float16, torch.bfloat16):
        outs[t] = (grad.to(t), torch.empty(size, device="cuda", dtype=t))
        h.orthogonalise(*outs[t])
    for i in {0, len(mats) // 2, len(mats) - 1}:
        o, r, c = mats[i]
        at = slice(o, o + r * c)
        m = mu * m64[at] + grad[at].double()
        x = orthogonal64((grad[at].double() + mu * m).view(r, c))
        want = (1 - lr * 0.1) * w0[at] - lr * 0.5 * x.reshape(-1)
        err = float((w[at].double() - want).norm())
        assert err <= 4 * 2.0 ** -20 * lr * 0.5 * float(x.norm()) + 4 * F32 * float(want.norm())
        for t, (g16, out) in outs.items():
            want = orthogonal64(g16[at].view(r, c))
            err = float((out[at].view(r, c).double() - want).norm() / want.norm())
            assert err <= 4 * 2.0 ** -20 + u(t)
