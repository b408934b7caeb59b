"""The cross entropy and its gradient on the GPU against plain forms in 64 bits.

Tolerances.  u(t) = finfo(t).eps / 2 is a type's rounding, F32 binary32's.
Logits are binary32 sums of k products: k F32 sum|x||w| off at most (`slack`).
An exponential under a largest logit t is off by its argument's rounding (the
value (t - v) e^(v - t) F32 is under F32) and 4 F32 of its own; sums of them go
through a tile (16 terms in a lane, 2 exchanges, 4 waves), then at most 64 parts
in a lane and 8 exchanges, with up to 6 F32 more where the largest logit changes:
under 600 F32 of the sum, which is what the log-sum-exp is off by.

dz is off by p (slack + (4 + 3 |z - lse|) F32) + 4 F32 of its terms, and rounded
to 16 bits: u(t), and in binary16, whose subnormal numbers end at 2^-25 where
the largest factor is at least 2^14, 2^-39 of that factor.  As a pair: u(t)^2.
"""
import math

import pytest
import torch

import sgd_gradient_all_amd as ddl

pytestmark = pytest.mark.gpu

F32 = torch.finfo(torch.float32).eps / 2
T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def u(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, sigma=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(dtype)


def strided(t, pad, first=0):
    """t with `pad` more elements between its rows, starting `first` elements in."""
    r, c = t.shape
    flat = torch.full((first + r * (c + pad),), float("nan"), device=t.device, dtype=t.dtype)
    view = flat[first:].view(r, c + pad)[:, :c]
    view.copy_(t)
    return view


def workspace(op, m, n, k):
    # all ones: NaN as binary32 and as either 16-bit type, so that nothing left
    # over from before is taken for a value
    return torch.full((ddl.cross_entropy_workspace(op, m, n, k),), 255, device="cuda",
                      dtype=torch.uint8)


def inputs(m, n, k, dtype, ignored=0.3, bias=True, seed=0):
    g, t = gen(seed + m + 3 * n + 7 * k), T[dtype]
    w = normal(g, n, k, sigma=2 * max(k, 1) ** -0.5, dtype=t)
    target = torch.randint(n, (m,), generator=g, device="cuda")
    x = (normal(g, m, k) + 1.5 * w[target].float()).to(t)
    b = normal(g, n, sigma=0.5, dtype=t) if bias else None
    gone = torch.rand(m, generator=g, device="cuda") < ignored
    target = torch.where(gone, torch.where(target % 2 == 0, -100, -1), target)
    return x, w, b, target


def logits(x, w, b):
    """(logits in 64 bits, how far binary32 sums may be off)."""
    xd, wd = x.double(), w.double().t().contiguous()
    z, s = xd @ wd, xd.abs() @ wd.abs()
    if b is not None:
        z, s = z + b.double(), s + b.double().abs()
    return z, (x.shape[1] + 4) * F32 * s


def check_loss(x, w, b, target, a, loss, lse):
    z, slack = logits(x, w, b)
    want = torch.logsumexp(z, 1)
    off = slack.amax(1) + 600 * F32 + 2 * F32 * want.abs()
    have = target >= 0
    assert (loss[~have] == 0).all() and (lse[~have] == 0).all()
    assert ((lse.double() - want).abs() <= off)[have].all()
    at = z.gather(1, target.clamp(min=0)[:, None])[:, 0]
    mean, most = (z.mean(1), z.abs().mean(1)) if a else (0 * at, 0 * at)
    value = want - (1 - a) * at - a * mean
    off = 2 * off + slack.amax(1) + 4 * F32 * (want.abs() + at.abs()) + 100 * a * F32 * most
    assert ((loss.double() - value).abs() <= off)[have].all()


def run_loss(x, w, b, target, a=0.0, stream=None):
    m, k = x.shape
    loss, lse = (torch.full((m,), float("nan"), device="cuda") for _ in range(2))
    ddl.cross_entropy(x, w, target, loss, lse, bias=b, smoothing=a,
                      workspace=workspace("forward", m, w.shape[0], k), stream=stream)
    return loss, lse


SIZES = [(1, 1, 1), (1, 2, 0), (3, 5, 7), (1, 64, 64), (17, 130, 72), (64, 64, 64), (65, 63, 65),
         (129, 257, 130), (256, 256, 320), (300, 520, 2056), (2049, 1000, 64), (5000, 70, 40),
         (1, 2048, 256), (16, 4100, 264), (7, 33000, 2056), (15, 20001, 1000), (33, 2048, 512),
         (1, 4096, 4095), (40, 32768, 128)]
LAYOUTS = [(0, 0), (3, 0), (8, 0), (0, 1)]  # elements between rows, before the first


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_loss(m, n, k, dtype):
    for i, (a, bias, ignored) in enumerate([(0.0, False, 0.0), (0.1, True, 0.3),
                                            (1.0, False, 0.5), (0.0, True, 0.9)]):
        x, w, b, target = inputs(m, n, k, dtype, ignored, bias, i)
        pad, first = LAYOUTS[i]
        print(f"loss {m} {n} {k} {dtype} {a} {bias} {ignored} {pad} {first}", flush=True)
        loss, lse = run_loss(strided(x, pad, first), strided(w, pad, first), b, target, a)
        check_loss(x, w, b, target, a, loss, lse)


def check_grad(x, w, b, target, lse, dloss, scale, a, dx, dw, db, dw0=None, db0=None):
    """Every output against the formula; what a sum of terms may be off by is the
    same product of the terms' own slacks."""
    m, n, t = x.shape[0], w.shape[0], x.dtype
    z, slack = logits(x, w, b)
    g = torch.full((m,), scale, device="cuda", dtype=torch.float64)
    if dloss is not None:
        g = g * dloss.double()
    # a product of two binary32 numbers
    gslack = F32 * g.abs()
    have = (target >= 0) & (g != 0)
    p = torch.exp(z - lse.double()[:, None])
    hot = torch.zeros_like(z)
    hot.scatter_(1, target.clamp(min=0)[:, None], 1.0)
    raw = p - (1 - a) * hot - a / n
    off = p * (slack + (4 + 3 * (z - lse.double()[:, None]).abs()) * F32) \
        + 4 * F32 * (p + hot + a / n)
    row = torch.where(have, g, 0.0)[:, None]
    dz = torch.where(have[:, None], raw * row, 0.0)
    doff = torch.where(have[:, None], off * row.abs() + raw.abs() * gslack[:, None], 0.0)
    top = float(row.abs().max()) if m else 0.0
    floor = torch.where(have[:, None], 2.0 ** -39 * top, 0.0)
    one = doff + u(t) * (dz.abs() + doff) + floor
    pair = doff + u(t) ** 2 * (dz.abs() + doff) + floor
    xd, wd = x.double(), w.double()
    xd = torch.where(have[:, None], xd, 0.0)

    def near(got, want, slack):
        v = got.dtype
        limit = slack + (want.abs() + slack) * u(v) * (1.01) + torch.finfo(v).tiny * u(v)
        d = (got.double() - want).abs()
        assert torch.isfinite(got).all()
        assert (d <= limit).all(), f"{int((d > limit).sum())} off, {float((d - limit).max())}"
    if dx is not None:
        near(dx, dz @ wd, one @ wd.abs() + (n + 8) * F32 * (dz.abs() @ wd.abs()))
        assert (dx[~have] == 0).all()
    if dw is not None:
        part = pair if dw.dtype == torch.float32 else one
        want, s = dz.t().contiguous() @ xd, dz.abs().t().contiguous() @ xd.abs()
        limit = part.t().contiguous() @ xd.abs() + (2 * m + 8) * F32 * s
        if dw0 is not None:
            want = want + dw0.double()
            limit = limit + F32 * want.abs() * 2
        near(dw, want, limit)
    if db is not None:
        want, limit = dz.sum(0), doff.sum(0) + (m + 8) * F32 * dz.abs().sum(0)
        if db0 is not None:
            want = want + db0.double()
            limit = limit + F32 * want.abs() * 2
        near(db, want, limit)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gradient(m, n, k, dtype):
    t = T[dtype]
    for i, (a, bias, ignored, out, add, weighted) in enumerate([
            (0.0, False, 0.0, "f32", False, False), (0.1, True, 0.3, dtype, False, True),
            (0.0, True, 0.5, "f32", True, True), (0.3, True, 0.9, dtype, True, False)]):
        x, w, b, target = inputs(m, n, k, dtype, ignored, bias, i)
        z, _ = logits(x, w, b)
        lse = torch.logsumexp(z, 1).float()
        g_ = gen(i)
        dloss = (torch.rand(m, generator=g_, device="cuda") / max(m, 1)) if weighted else None
        scale = 1.0 if weighted else 1 / 512
        pad, first = LAYOUTS[(i + 1) % 4]
        dx = strided(torch.zeros(m, k, device="cuda", dtype=t), pad, first)
        dw0 = normal(g_, n, k, sigma=1e-3, dtype=T[out])
        db0 = normal(g_, n, sigma=1e-3, dtype=T[out]) if bias else None
        dw, db = strided(dw0, pad, first), db0.clone() if bias else None
        print(f"gradient {m} {n} {k} {dtype} {a} {bias} {ignored} {out} {add} {pad} {first}",
              flush=True)
        ddl.cross_entropy_grad(strided(x, pad, first), strided(w, pad, first), target, lse,
                               dloss=dloss, scale=scale, dx=dx, dw=dw, db=db, bias=b, smoothing=a,
                               accumulate=add, workspace=workspace("grad", m, n, k))
        check_grad(x, w, b, target, lse, dloss, scale, a, dx, dw, db, dw0 if add else None,
                   db0 if add else None)
