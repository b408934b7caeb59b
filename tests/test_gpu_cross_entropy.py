"""The cross entropy and its gradient on the GPU against plain forms in 64 bits.

Tolerances.  u(t) = finfo(t).eps / 2 is a type's rounding, F32 binary32's.
Logits are binary32 sums of k products: k F32 sum|x||w| off at most (`slack`).
An exponential under a largest logit t is off by its argument's rounding (the
value (t - v) e^(v - t) F32 is under F32) and 4 F32 of its own; sums of them go
through a tile (16 terms in a lane, 2 exchanges, 4 waves), then at most 64 parts
in a lane and 8 exchanges, with up to 6 F32 more where the largest logit changes:
under 600 F32 of the sum, which is what the log-sum-exp is off by.

dz is off by p (slack + (4 + 3 |z - lse|) F32) + 4 F32 of its terms, by 2^-126 more
where p is below binary32's normal numbers (2^x is 0 there), and rounded to 16 bits: u(t), and in binary16, whose subnormal numbers end at 2^-25 where
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
        + 4 * F32 * (p + hot + a / n) + 2.0 ** -126
    row = torch.where(have, g, 0.0)[:, None]
    dz = torch.where(have[:, None], raw * row, 0.0)
    doff = torch.where(have[:, None], off * row.abs() + raw.abs() * gslack[:, None], 0.0)
    top = float(row.abs().max()) if m else 0.0
    floor = torch.where(have[:, None], 2.0 ** -39 * top, 0.0)
    one = doff + 2.0 ** -11 * (dz.abs() + doff) + floor
    pair = doff + 2.0 ** -22 * (dz.abs() + doff) + floor
    xd, wd = x.double(), w.double()
    xd = torch.where(have[:, None], xd, 0.0)
    # binary16 takes the largest to 2^14 or more, and is off by at most 2^-25
    xoff, woff = (2.0 ** -39 * float(v.abs().max()) if v.numel() else 0.0 for v in (xd, wd))

    def near(got, want, slack):
        v = got.dtype
        limit = slack + (want.abs() + slack) * u(v) * (1.01) + torch.finfo(v).tiny * u(v)
        d = (got.double() - want).abs()
        assert torch.isfinite(got).all()
        assert (d <= limit).all(), f"{int((d > limit).sum())} off, {float((d - limit).max())}"
    if dx is not None:
        near(dx, dz @ wd, one @ wd.abs() + (n + 8) * F32 * (dz.abs() @ wd.abs())
             + woff * one.sum(1)[:, None] + woff * dz.abs().sum(1)[:, None])
        assert (dx[~have] == 0).all()
    if dw is not None:
        part = pair if dw.dtype == torch.float32 else one
        want, s = dz.t().contiguous() @ xd, dz.abs().t().contiguous() @ xd.abs()
        limit = part.t().contiguous() @ xd.abs() + (2 * m + 8) * F32 * s \
            + xoff * (part + dz.abs()).sum(0)[:, None]
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


# bfloat16 operands in pairs, and, from 1.2e9 products on, as binary16: both
# outputs' types and an odd k, which is packed
ONCE = [(65, 63, 65), (300, 520, 2056), (512, 9800, 2056), (1030, 8200, 2400), (1100, 9001, 2051),
        (700, 1000, 2048), (1100, 1000, 1201)]


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("m,n,k", ONCE)
def test_gradient_is_rounded_once(m, n, k, dtype, out):
    """What dz loses is small beside the result's own rounding.  Rounding to nearest
    leaves a result of p bits an error of about 2^-p / sqrt(3) of its binade; dz's 11
    bits against bfloat16's 8 add an eighth of it, whose square is 1 / 64, and a root
    of 1 + 3 / 64 covers sums whose terms cancel by a factor of sqrt(3)."""
    x, w, b, target = inputs(m, n, k, dtype, 0.2)
    z, _ = logits(x, w, b)
    lse = torch.logsumexp(z, 1).float()
    dx = torch.empty(m, k, device="cuda", dtype=T[dtype])
    dw, db = torch.empty(n, k, device="cuda", dtype=T[out]), None
    ddl.cross_entropy_grad(x, w, target, lse, scale=1 / m, dx=dx, dw=dw, bias=b,
                           workspace=workspace("grad", m, n, k))
    check_grad(x, w, b, target, lse, None, 1 / m, 0.0, dx, dw, db)
    dz = torch.exp(z - lse.double()[:, None])
    dz[torch.arange(m), target.clamp(min=0)] -= 1
    dz = torch.where((target >= 0)[:, None], dz / m, 0.0)
    for got, want in ((dx, dz @ w.double()), (dw, dz.t().contiguous() @ x.double())):
        if got.dtype == torch.float32:
            continue  # by check_grad alone
        off, own = ((v.double() - want).norm().item() for v in (got, want.to(got.dtype)))
        print(f"{m} {n} {k} {dtype} {off / own}")
        assert off <= own * (1 + 3 / 64) ** 0.5


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("m,n,k", [(1100, 4801, 1000), (600, 9000, 1001), (130, 700, 264)])
def test_gradients_alone_and_of_few_of_the_rows(m, n, k, dtype, out):
    """Each output without the others, and none, one, or half of the rows with a
    target, whatever the others hold."""
    x, w, b, target = inputs(m, n, k, dtype, 0.0)
    z, _ = logits(x, w, b)
    lse = torch.logsumexp(z, 1).float()
    ws = workspace("grad", m, n, k)
    for rows in (0, 1, m // 2, m):
        have = target.clone()
        have[rows:] = -1
        bad = x.clone()
        bad[rows:] = float("nan")
        for which in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1)):
            print(f"alone {m} {n} {k} {dtype} {out} {rows} {which}", flush=True)
            dx = torch.full((m, k), 7.0, device="cuda", dtype=T[dtype]) if which[0] else None
            dw = torch.full((n, k), 7.0, device="cuda", dtype=T[out]) if which[1] else None
            db = torch.full((n,), 7.0, device="cuda", dtype=T[out]) if which[2] else None
            ws.fill_(255)
            ddl.cross_entropy_grad(bad, w, have, lse, scale=1 / m, dx=dx, dw=dw, db=db, bias=b,
                                   workspace=ws)
            check_grad(x, w, b, have, lse, None, 1 / m, 0.0, dx, dw, db)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("large", [0, 90, -90])
def test_gradient_of_a_wide_range(large, out):
    """bfloat16 values past binary16's range, and far apart."""
    m, n, k = 1030, 8200, 2400
    x, w, b, target = inputs(m, n, k, "bf16", 0.2)
    g = gen(9)
    far = torch.exp2(-torch.randint(0, 30, (k,), generator=g, device="cuda").float())
    x = (x.float() * far * 2.0 ** large).to(torch.bfloat16)
    w = (w.float() * torch.exp2(-torch.randint(0, 30, (n, 1), generator=g, device="cuda").float())
         * 2.0 ** -large).to(torch.bfloat16)
    x[target < 0] = float("inf")
    clean = torch.where((target >= 0)[:, None], x, 0)
    z, _ = logits(clean, w, b)
    lse = torch.logsumexp(z, 1).float()
    dx = torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
    dw = torch.empty(n, k, device="cuda", dtype=T[out])
    ddl.cross_entropy_grad(x, w, target, lse, scale=1 / m, dx=dx, dw=dw, bias=b,
                           workspace=workspace("grad", m, n, k))
    check_grad(clean, w, b, target, lse, None, 1 / m, 0.0, dx, dw, None)


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


def run_grad(x, w, b, target, lse, dloss=None, scale=1.0, a=0.0, out=torch.float32, stream=None):
    (m, k), n = x.shape, w.shape[0]
    dx = torch.full_like(x, 9.0)
    dw = torch.full((n, k), 9.0, device="cuda", dtype=out)
    db = torch.full((n,), 9.0, device="cuda", dtype=out)
    ddl.cross_entropy_grad(x, w, target, lse, dloss=dloss, scale=scale, dx=dx, dw=dw, db=db, bias=b,
                           smoothing=a, workspace=workspace("grad", m, n, k), stream=stream)
    return dx, dw, db


# (m, n, k) that take every tile of the loss and of the three products of the
# gradient, sums in parts and whole, short last k tiles, odd rows packed, and
# several pieces; which is which is checked on the host
LARGE = [(3000, 6000, 136), (4096, 4096, 256), (1500, 2100, 200), (700, 500, 1096),
         (520, 264, 4104), (2047, 9001, 1023), (1023, 12003, 111), (300, 30000, 72),
         (8199, 20001, 72), (8192, 33000, 63), (70, 3000, 640), (5000, 40, 130),
         (4000, 3000, 4096), (4090, 2001, 4000)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", LARGE)
def test_large(m, n, k, dtype):
    t = T[dtype]
    for a, bias, ignored, out, first in ((0.1, True, 0.1, "f32", 0), (0.0, False, 0.5, dtype, 1)):
        print(f"large {m} {n} {k} {dtype} {a} {bias} {ignored} {out} {first}", flush=True)
        x, w, b, target = inputs(m, n, k, dtype, ignored, bias)
        off = strided(w, 0, first)  # off 16 bytes: rows go through registers
        loss, lse = run_loss(x, off, b, target, a)
        check_loss(x, w, b, target, a, loss, lse)
        dx, dw, db = run_grad(x, off, b, target, lse, scale=1 / m, a=a, out=T[out])
        lse = torch.where(target >= 0, lse, torch.zeros_like(lse))
        check_grad(x, w, b, target, lse, None, 1 / m, a, dx, dw, db)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 16, 17, 33, 64])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_few_rows(m, dtype):
    """Every kernel for few rows, whole batches of loads and what is left of them."""
    for n, k in ((37, 8), (5000, 2048), (3001, 2056), (2050, 4616), (100, 16392)):
        print(f"few {m} {n} {k} {dtype}", flush=True)
        x, w, b, target = inputs(m, n, k, dtype, 0.3, True)
        target[0] = n - 1
        check_loss(x, w, b, target, 0.1, *run_loss(x, w, b, target, 0.1))
        check_loss(x, w, None, target, 0.0, *run_loss(x, w, None, target, 0.0))


@pytest.mark.parametrize("m,n,k", [(40, 300, 72), (700, 1000, 264), (2000, 3000, 100)])
def test_rows_without_a_target_reach_nothing(m, n, k):
    """NaN and infinities in them, and in the factors and log-sum-exps of theirs."""
    t = torch.bfloat16
    x, w, b, target = inputs(m, n, k, "bf16", 0.4)
    gone = target < 0
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda")
    dirty = x.clone()
    dirty[gone] = bad[torch.arange(int(gone.sum()), device="cuda") % 3].to(t)[:, None]
    loss, lse = run_loss(dirty, w, b, target)
    check_loss(x, w, b, target, 0.0, loss, lse)
    dloss = torch.rand(m, generator=gen(3), device="cuda") + 0.5
    dirty_lse, dirty_dloss = lse.clone(), dloss.clone()
    dirty_lse[gone], dirty_dloss[gone] = float("nan"), float("nan")
    got = run_grad(dirty, w, b, target, dirty_lse, dloss=dirty_dloss, scale=1 / m)
    check_grad(x, w, b, target, lse, dloss, 1 / m, 0.0, *got)
    # a factor of 0 is no target either
    kept = torch.where(gone, torch.ones_like(target), target)
    zero = torch.where(gone, torch.zeros_like(dloss), dloss)
    again = run_grad(dirty, w, b, kept, dirty_lse, dloss=zero, scale=1 / m)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("m", [5, 100, 2000])
def test_no_row_has_a_target(m):
    x, w, b, target = inputs(m, 70, 40, "f16", 2.0)
    loss, lse = run_loss(x, w, b, target)
    assert (loss == 0).all() and (lse == 0).all()
    dx, dw, db = run_grad(x, w, b, target, lse)
    assert (dx == 0).all() and (dw == 0).all() and (db == 0).all()
    dw.fill_(3.0)
    ddl.cross_entropy_grad(x, w, target, lse, dw=dw, accumulate=True,
                           workspace=workspace("grad", m, 70, 40))
    assert (dw == 3).all()


def test_no_rows():
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    w, b = normal(gen(1), 6, 8, dtype=torch.float16), normal(gen(2), 6, dtype=torch.float16)
    x, target = e(0, 8).half(), e(0).long()
    ddl.cross_entropy(x, w, target, e(0), e(0), bias=b)
    for out in (torch.float32, torch.float16):
        dw, db = torch.ones(6, 8, device="cuda", dtype=out), torch.ones(6, device="cuda", dtype=out)
        ddl.cross_entropy_grad(x, w, target, e(0), dw=dw, db=db, bias=b, accumulate=True)
        assert (dw == 1).all() and (db == 1).all()
        ddl.cross_entropy_grad(x, w, target, e(0), dw=dw, db=db, bias=b)
        assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("m,n,k", [(3, 90, 64), (30, 90, 64), (300, 700, 72)])
def test_masked_classes(m, n, k):
    """A bias of -inf: no share of the sum, no gradient; and rows of nothing else."""
    x, w, b, target = inputs(m, n, k, "bf16", 0.0)
    b[n // 2:] = -float("inf")
    target %= n // 2
    loss, lse = run_loss(x, w, b, target)
    check_loss(x, w[:n // 2], b[:n // 2], target, 0.0, loss, lse)
    dx, dw, db = run_grad(x, w, b, target, lse, scale=1 / m)
    assert (dw[n // 2:] == 0).all() and (db[n // 2:] == 0).all()
    check_grad(x, w[:n // 2], b[:n // 2], target, lse, None, 1 / m, 0.0, dx, dw[:n // 2],
               db[:n // 2])
    loss, lse = run_loss(x, w, torch.full_like(b, -float("inf")), target)
    assert (lse == -float("inf")).all() and torch.isnan(loss).all()
    target.fill_(n - 1)  # a masked class is wanted
    loss, lse = run_loss(x, w, b, target)
    assert (loss == float("inf")).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("m", [4, 50, 500])
def test_targets_out_of_range_are_loud(m):
    n, k = 130, 72
    x, w, b, target = inputs(m, n, k, "f16", 0.0)
    target[1], target[2] = n, 1 << 40
    loss, lse = run_loss(x, w, b, target)
    fine = torch.ones(m, device="cuda", dtype=torch.bool)
    fine[1:3] = False
    assert torch.isnan(loss[~fine]).all() and torch.isfinite(lse).all()
    assert torch.isfinite(loss[fine]).all()
    dx, dw, db = run_grad(x, w, b, target, lse)
    assert torch.isnan(dx[~fine]).all() and torch.isfinite(dx[fine]).all()
    assert torch.isnan(dw).all() and torch.isnan(db).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_row_with_an_infinite_factor_spoils_no_other_dx(dtype):
    m, n, k = 60, 200, 72
    x, w, b, target = inputs(m, n, k, dtype, 0.0)
    _, lse = run_loss(x, w, b, target)
    dloss = torch.full((m,), 0.25, device="cuda")
    clean = run_grad(x, w, b, target, lse, dloss=dloss)[0]
    dloss[7] = float("inf")
    dx = run_grad(x, w, b, target, lse, dloss=dloss)[0]
    fine = torch.arange(m, device="cuda") != 7
    assert torch.equal(dx[fine], clean[fine]) and not torch.isfinite(dx[7]).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scales_of_the_loss(dtype):
    """A power of two in the loss is the same power in binary32 gradients, bit for
    bit, up to scales whose 16-bit values would not be numbers."""
    m, n, k = 100, 3000, 136
    x, w, b, target = inputs(m, n, k, dtype, 0.2)
    _, lse = run_loss(x, w, b, target)
    _, dw, db = run_grad(x, w, b, target, lse, scale=1 / 64)
    for e in (-60, -20, 10, 40):
        _, dw2, db2 = run_grad(x, w, b, target, lse, scale=2.0 ** e / 64)
        assert torch.equal(dw2, dw * 2.0 ** e) and torch.equal(db2, db * 2.0 ** e)
    check_grad(x, w, b, target, torch.where(target >= 0, lse, torch.zeros_like(lse)), None, 1 / 64,
               0.0, None, dw, db)


def test_large_logits():
    """Logits of thousands, of both signs, as sums of exponentials meet them."""
    for m in (2, 20, 200):
        x, w, b, target = inputs(m, 500, 64, "bf16", 0.0)
        x = x * 400
        loss, lse = run_loss(x, w, b, target)
        check_loss(x, w, b, target, 0.0, loss, lse)
        dx, dw, db = run_grad(x, w, b, target, lse, scale=1 / m)
        check_grad(x, w, b, target, lse, None, 1 / m, 0.0, dx, dw, db)


@pytest.mark.parametrize("a", [0.0, 0.2])
def test_gradient_against_differences(a):
    """The three gradients against central differences of the loss in 64 bits."""
    m, n, k, t = 24, 50, 40, torch.bfloat16
    x, w, b, target = inputs(m, n, k, "bf16", 0.2)
    dloss = torch.rand(m, generator=gen(5), device="cuda") + 0.1
    have = target >= 0
    _, lse = run_loss(x, w, b, target, a)
    dx, dw, db = run_grad(x, w, b, target, lse, dloss=dloss, a=a)

    def total(x, w, b):
        z = x @ w.t().contiguous() + b
        at = z.gather(1, target.clamp(min=0)[:, None])[:, 0]
        loss = torch.logsumexp(z, 1) - (1 - a) * at - a * z.mean(1)
        return float((loss * dloss.double())[have].sum())

    args = [v.double() for v in (x, w, b)]
    h = 1e-4
    z = args[0] @ args[1].t().contiguous() + args[2]
    p = torch.exp(z - lse.double()[:, None])
    p.scatter_add_(1, target.clamp(min=0)[:, None], torch.ones_like(p[:, :1]))
    # of dz: a rounding to bfloat16 (dx alone; pairs and db keep 2^-16), log-sum-exps
    # that are 600 F32 off, and differences' h^2 and 1e-16 / h of sums of 24 losses
    size = torch.where(have, dloss, torch.zeros_like(dloss)).double()[:, None] * (p + a / n)
    for which, got, at in ((0, dx, (3, 7)), (0, dx, (20, 39)), (1, dw, (0, 0)), (1, dw, (49, 11)),
                           (2, db, (0,)), (2, db, (33,))):
        ends = []
        for s in (h, -h):
            moved = [v.clone() for v in args]
            moved[which][at] += s
            ends.append(total(*moved))
        want = (ends[0] - ends[1]) / (2 * h)
        terms = (float((size[at[0]] * args[1][:, at[1]].abs()).sum()) if which == 0 else
                 float((size[:, at[0]] * args[0][:, at[1]].abs()).sum()) if which == 1 else
                 float(size[:, at[0]].sum()))
        rounding = u(t) * (terms + abs(want)) if which == 0 else 2.0 ** -15 * terms
        assert abs(float(got[at]) - want) <= rounding + 1000 * F32 * terms + 1e-7 * (1 + terms)


def test_outputs_stay_inside_their_rows():
    m, n, k, t = 300, 270, 100, torch.float16
    x, w, b, target = inputs(m, n, k, "f16", 0.3)
    _, lse = run_loss(x, w, b, target)
    for out in (torch.float32, t):
        dx = strided(torch.zeros(m, k, device="cuda", dtype=t), 5, 1)
        dw = strided(torch.zeros(n, k, device="cuda", dtype=out), 3, 1)
        db = torch.full((n + 2,), 5.0, device="cuda", dtype=out)
        ddl.cross_entropy_grad(x, w, target, lse, dx=dx, dw=dw, db=db[1:-1], bias=b,
                               workspace=workspace("grad", m, n, k))
        for v, pad in ((dx, 5), (dw, 3)):
            flat = v.as_strided((v.shape[0], k + pad), (k + pad, 1), v.storage_offset())
            assert torch.isnan(flat[:, k:]).all() and torch.isfinite(v).all()
        assert float(db[0]) == 5 and float(db[-1]) == 5


@pytest.mark.parametrize("m,n,k", [(60, 700, 264), (1500, 3000, 200), (1500, 4001, 1001)])
def test_same_bits_on_another_stream_and_in_a_graph(m, n, k):
    """The loss, then the gradient from its log-sum-exps: eagerly, on another stream,
    and captured and replayed with eager work between."""
    x, w, b, target = inputs(m, n, k, "bf16", 0.3)
    ws = torch.empty(max(ddl.cross_entropy_workspace(o, m, n, k) for o in ("forward", "grad")),
                     device="cuda", dtype=torch.uint8)

    def fresh():
        return [torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda"),
                torch.zeros_like(x), torch.zeros(n, k, device="cuda"),
                torch.zeros(n, device="cuda")]

    def step(o, stream):
        ddl.cross_entropy(x, w, target, o[0], o[1], bias=b, smoothing=0.1, workspace=ws,
                          stream=stream)
        ddl.cross_entropy_grad(x, w, target, o[1], scale=1 / m, dx=o[2], dw=o[3], db=o[4], bias=b,
                               smoothing=0.1, accumulate=True, workspace=ws, stream=stream)

    eager, want = fresh(), []
    for _ in range(3):
        step(eager, None)
        torch.cuda.synchronize()
        want.append([v.clone() for v in eager])
    side, s = fresh(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(3):
        step(side, s)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(side, want[i]))
    held, graph = fresh(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        step(held, s)
    for i in range(3):
        target2 = target.clone()  # eager work between
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want[i])), f"replay {i}"
        assert torch.equal(target2, target)
        (torch.randn(64, 64, device="cuda") @ torch.randn(64, 64, device="cuda")).sum().item()


def test_classes_past_32_bits():
    """w, dw of more than 2^32 elements: the classes at the far end."""
    m, n, k, t = 3, (1 << 21) + 300, 2056, torch.bfloat16
    w = torch.empty(n, k, device="cuda", dtype=t).normal_(generator=gen(8)).mul_(k ** -0.5)
    x = normal(gen(9), m, k, dtype=t)
    target = torch.tensor([n - 1, 5, n - 300], device="cuda")
    print("classes past 32 bits", flush=True)
    loss, lse = run_loss(x, w, None, target)
    z = torch.cat([x.double() @ part.double().t().contiguous() for part in w.split(1 << 18)], 1)
    slack = (k + 4) * F32 * float((x.double().abs().amax() * w.double().abs().amax()) * k)
    want = torch.logsumexp(z, 1)
    assert ((lse.double() - want).abs() <= slack + 600 * F32 + 2 * F32 * want).all()
    at = z[torch.arange(m, device="cuda"), target]
    assert ((loss.double() - (want - at)).abs() <= 2 * slack + 1300 * F32 + 6 * F32 * want).all()
    dx, dw, _ = torch.empty_like(x), torch.empty(n, k, device="cuda", dtype=t), None
    ddl.cross_entropy_grad(x, w, target, lse, dx=dx, dw=dw, workspace=workspace("grad", m, n, k))
    p = torch.exp(z - lse.double()[:, None])
    p[torch.arange(m, device="cuda"), target] -= 1
    for rows in (slice(n - 300, n), slice(0, 10), slice(n // 2, n // 2 + 10)):
        want = p[:, rows].t().contiguous() @ x.double()
        off = p[:, rows].abs().t().contiguous() @ x.double().abs()
        assert ((dw[rows].double() - want).abs() <= (2 * u(t) + 2 * slack + 64 * F32) * off
                + u(t) * want.abs() + 1e-30).all()
    want = sum(p[:, i:i + (1 << 18)] @ w[i:i + (1 << 18)].double() for i in range(0, n, 1 << 18))
    off = sum(p[:, i:i + (1 << 18)].abs() @ w[i:i + (1 << 18)].double().abs()
              for i in range(0, n, 1 << 18))
    assert ((dx.double() - want).abs() <= (u(t) + 2 * slack + n * F32) * off
            + 2 * u(t) * want.abs()).all()


def test_rows_past_32_bits():
    """x and dx of more than 2^32 elements: the rows at the far end."""
    m, n, k, t = (1 << 21) + 100, 64, 2056, torch.bfloat16
    x = torch.empty(m, k, device="cuda", dtype=t).normal_(generator=gen(10))
    w = normal(gen(11), n, k, sigma=k ** -0.5, dtype=t)
    target = torch.full((m,), -1, device="cuda")
    some = torch.cat([torch.arange(50, device="cuda"), torch.arange(m - 300, m, device="cuda")])
    target[some] = some % n
    print("rows past 32 bits", flush=True)
    loss, lse = run_loss(x, w, None, target)
    check_loss(x[some], w, None, target[some], 0.0, loss[some], lse[some])
    assert int((loss != 0).sum()) == some.numel()
    dx = torch.full_like(x, 9.0)
    dw = torch.empty(n, k, device="cuda")
    ddl.cross_entropy_grad(x, w, target, lse, scale=1 / 64, dx=dx, dw=dw,
                           workspace=workspace("grad", m, n, k))
    check_grad(x[some], w, None, target[some], lse[some], None, 1 / 64, 0.0, dx[some], dw, None)
    assert int((dx != 0).any(1).sum()) <= some.numel()


def test_an_older_error_is_not_the_calls():
    import ctypes
    hip, p = ddl.lib(), ctypes.c_void_p()
    x, w, b, target = inputs(20, 40, 64, "f16")
    lse = torch.zeros(20, device="cuda")
    h = ddl.AdamW8([(0, 64)])
    st = [torch.zeros(64, device="cuda", dtype=t) for t in (torch.int8, torch.uint8)] \
        + [torch.zeros(1, device="cuda") for _ in range(2)]
    v = [torch.zeros(64, device="cuda") for _ in range(2)]
    loss, dx, dw = torch.zeros(20, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    fw, gw = workspace("forward", 20, 40, 64), workspace("grad", 20, 40, 64)
    torch.cuda.synchronize()
    calls = [lambda: ddl.cross_entropy(x, w, target, loss, lse, bias=b, workspace=fw),
             lambda: ddl.cross_entropy_grad(x, w, target, lse, dx=dx, dw=dw, bias=b, workspace=gw),
             lambda: h.step(v[0], *st, [v[1]], lr=0.1), lambda: h.values(*st, *v)]
    try:
        for call in calls:
            assert hip.hipMalloc(ctypes.byref(p), ctypes.c_size_t(1 << 60)) != 0
            call()
    finally:
        hip.hipGetLastError()
        torch.cuda.synchronize()
