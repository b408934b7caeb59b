"""The cross entropy's gradient at the edges of its tiles and of its operands'
ranges, with the tolerances of test_gpu_cross_entropy.py."""
import pytest
import torch

import sgd_gradient_all_amd as ddl
import test_gpu_cross_entropy as ce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1024, 1050, 2048), (1024, 1056, 1152), (512, 992, 4096),
                                   (1100, 1049, 1201), (549, 2321, 1608)])
def test_columns_past_the_last_class(m, n, k, out):
    """64 x 32 tiles of dz whose last k tile of 64 is half past the classes: in a
    workspace full of NaN, and again in one that holds the call before."""
    x, w, b, target = ce.inputs(m, n, k, "bf16", 0.2)
    z, _ = ce.logits(x, w, b)
    lse = torch.logsumexp(z, 1).float()
    ws = ce.workspace("grad", m, n, k)
    first = None
    for _ in range(2):
        dx = torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
        dw = torch.empty(n, k, device="cuda", dtype=ce.T[out])
        db = torch.empty(n, device="cuda", dtype=ce.T[out])
        print(f"past the last class {m} {n} {k} {out}", flush=True)
        ddl.cross_entropy_grad(x, w, target, lse, scale=1 / m, dx=dx, dw=dw, db=db, bias=b,
                               workspace=ws)
        ce.check_grad(x, w, b, target, lse, None, 1 / m, 0.0, dx, dw, db)
        if first is not None:
            assert all(torch.equal(p, q) for p, q in zip(first, (dx, dw, db)))
        first = dx, dw, db


def terms(x, w, b, target, lse, scale):
    """dz in 64 bits and what it is off by, held in 11 and in 22 bits, as check_grad
    has it (without smoothing)."""
    z, slack = ce.logits(x, w, b)
    have = (target >= 0)[:, None]
    hot = torch.zeros_like(z)
    hot.scatter_(1, target.clamp(min=0)[:, None], 1.0)
    far = (z - lse.double()[:, None]).abs()
    p = torch.exp(z - lse.double()[:, None])
    dz = torch.where(have, (p - hot) * scale, 0.0)
    off = p * (slack + (4 + 3 * far) * ce.F32) + 4 * ce.F32 * (p + hot) + 2.0 ** -126
    off = torch.where(have, off * scale, 0.0) + ce.F32 * dz.abs()
    floor = torch.where(have, 2.0 ** -39 * scale, 0.0)
    return dz, off + 2.0 ** -11 * (dz.abs() + off) + floor, \
        off + 2.0 ** -22 * (dz.abs() + off) + floor


def near(got, want, slack):
    limit = slack + (want.abs() + slack) * ce.u(got.dtype) * 1.01
    assert torch.isfinite(got).all()
    d = (got.double() - want).abs()
    assert (d <= limit).all(), f"{int((d > limit).sum())} off, {float((d - limit).max())}"


def check_columns(x, w, b, target, lse, scale, dx, dw):
    """As check_grad, but what x and w are off by goes by their columns: 2^-39 of a
    column's largest value."""
    (m, n), (xd, wd) = (x.shape[0], w.shape[0]), (x.double(), w.double())
    dz, one, pair = terms(x, w, b, target, lse, scale)
    part = pair if dw.dtype == torch.float32 else one
    xoff, woff = (2.0 ** -39 * v.abs().amax(0)[None, :] for v in (xd, wd))
    near(dx, dz @ wd, one @ wd.abs() + (n + 8) * ce.F32 * (dz.abs() @ wd.abs())
         + (one + dz.abs()).sum(1)[:, None] * woff)
    dzt, part = dz.t().contiguous(), part.t().contiguous()
    near(dw, dzt @ xd, part @ xd.abs() + (2 * m + 8) * ce.F32 * (dzt.abs() @ xd.abs())
         + (part + dzt.abs()).sum(1)[:, None] * xoff)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1030, 8200, 2400), (1100, 9001, 2051), (600, 9000, 1001),
                                   (300, 520, 2056), (8192, 33000, 72)])
def test_a_column_that_is_small_throughout(m, n, k, out):
    """Columns of x and w 2^-60 and 2^-45 of the others keep their digits, with few
    rows and with many, in one piece of the classes and in several."""
    x, w, b, target = ce.inputs(m, n, k, "bf16", 0.0)
    w[:, 5::7] = (w[:, 5::7].float() * 2.0 ** -60).bfloat16()
    x[:, 3::5] = (x[:, 3::5].float() * 2.0 ** -45).bfloat16()
    w[n // 2:, 1] = 0  # of one that is 0 in a half of the classes
    w[:, 2], x[:, 4] = 0, 0
    z, _ = ce.logits(x, w, b)
    lse = torch.logsumexp(z, 1).float()
    dx = torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
    dw = torch.empty(n, k, device="cuda", dtype=ce.T[out])
    print(f"small columns {m} {n} {k} {out}", flush=True)
    ddl.cross_entropy_grad(x, w, target, lse, scale=1 / m, dx=dx, dw=dw, bias=b,
                           workspace=ce.workspace("grad", m, n, k))
    check_columns(x, w, b, target, lse, 1 / m, dx, dw)
    assert (dx[:, 2] == 0).all() and (dw[:, 4] == 0).all()


@pytest.mark.parametrize("huge", [1.0, 2.0 ** 40, 2.0 ** 66, 2.0 ** 100])
@pytest.mark.parametrize("m,n,k", [(1030, 8200, 2400), (1100, 9001, 2051), (300, 520, 2056),
                                   (8192, 33000, 72)])
def test_never_wanted_classes_may_hold_anything(m, n, k, huge):
    """Padding of a vocabulary, with a bias of -inf and large weights, changes no
    other class's share of dx, wherever it lies."""
    x, w, b, target = ce.inputs(m, n, k, "bf16", 0.2)
    pad = torch.arange(n, device="cuda") % 97 == 5
    pad[-100:] = True
    target = torch.where((target >= 0) & pad[target.clamp(min=0)], 0, target)
    b[pad] = -float("inf")
    z, _ = ce.logits(x, w, b)
    lse = torch.logsumexp(z, 1).float()
    w[pad] = (w[pad].float() * huge).bfloat16()
    for out in (torch.bfloat16, torch.float32):
        dx = torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
        dw, db = (torch.empty(*s, device="cuda", dtype=out) for s in ((n, k), (n,)))
        print(f"never wanted {m} {n} {k} {huge} {out}", flush=True)
        ddl.cross_entropy_grad(x, w, target, lse, scale=1 / m, dx=dx, dw=dw, db=db, bias=b,
                               workspace=ce.workspace("grad", m, n, k))
        assert (dw[pad] == 0).all() and (db[pad] == 0).all()
        place = torch.cumsum(~pad, 0) - 1
        kept = torch.where(target >= 0, place[target.clamp(min=0)], target)
        check_columns(x, w[~pad], b[~pad], kept, lse, 1 / m, dx, dw[~pad])


def test_a_never_wanted_class_that_is_wanted():
    """Its loss is infinite; with weights like the others' its gradient is exact."""
    m, n, k = 1030, 8200, 2400
    x, w, b, target = ce.inputs(m, n, k, "bf16", 0.0)
    b[7] = -float("inf")
    target[::50] = 7
    z, _ = ce.logits(x, w, b)
    lse = torch.logsumexp(z, 1).float()
    dx = torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
    dw = torch.empty(n, k, device="cuda")
    ddl.cross_entropy_grad(x, w, target, lse, scale=1 / m, dx=dx, dw=dw, bias=b,
                           workspace=ce.workspace("grad", m, n, k))
    far = b.clone()
    far[7] = -1e4  # the same shares, in numbers
    check_columns(x, w, far, target, lse, 1 / m, dx, dw)


@pytest.mark.parametrize("m,n,k,dtype", [(100, 3000, 136, "f16"), (100, 3000, 136, "bf16"),
                                         (1030, 8200, 2400, "bf16")])
def test_scales_to_the_ends_of_binary32(m, n, k, dtype):
    """A power of two in the loss is the same power in the gradients, bit for bit,
    from the smallest factors to the largest; subnormal results are rounded once."""
    x, w, b, target = ce.inputs(m, n, k, dtype, 0.2)
    z, _ = ce.logits(x, w, b)
    lse = torch.logsumexp(z, 1).float()
    want = ce.run_grad(x, w, b, target, lse, scale=1 / 64)
    assert all(torch.isfinite(v).all() and (v != 0).any() for v in want)

    def same(got, e, which):
        for i in which:
            assert torch.equal(got[i], (want[i].double() * 2.0 ** e).to(want[i].dtype)), (e, i)

    for e in (-140, -120, -110, -90, 100, 115, 123):
        print(f"scale {m} {n} {k} {dtype} {e}", flush=True)
        got = ce.run_grad(x, w, b, target, lse, scale=2.0 ** e / 64)
        # binary16's range is its own, and subnormal bfloat16 is rounded from binary32's
        same(got, e, (0, 1, 2) if dtype == "bf16" and e > -100 else (1, 2))
    for p, q in ((100, -160), (-120, 140), (20, -80)):  # of the two factors
        dloss = torch.full((m,), 2.0 ** p, device="cuda")
        got = ce.run_grad(x, w, b, target, lse, dloss=dloss, scale=2.0 ** q / 64)
        same(got, p + q, (1, 2))


# (m, n, k, elements that w starts past a 16-byte boundary): with test_large's sizes, every
# tile of bfloat16's products with rows of w through registers; which is which is
# checked on the host
THROUGH_REGISTERS = [(7621, 130, 552, 1), (990, 8469, 1496, 0), (151, 7761, 7456, 1),
                     (1970, 605, 1024, 1), (800, 662, 2432, 1)]


@pytest.mark.parametrize("m,n,k,first", THROUGH_REGISTERS)
def test_rows_through_registers(m, n, k, first):
    x, w, b, target = ce.inputs(m, n, k, "bf16", 0.1)
    off = ce.strided(w, 0, first)
    for out in (torch.bfloat16, torch.float32):
        print(f"through registers {m} {n} {k} {first} {out}", flush=True)
        loss, lse = ce.run_loss(x, off, b, target, 0.1)
        ce.check_loss(x, w, b, target, 0.1, loss, lse)
        dx, dw, db = ce.run_grad(x, off, b, target, lse, scale=1 / m, a=0.1, out=out)
        ce.check_grad(x, w, b, target, lse, None, 1 / m, 0.1, dx, dw, db)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 131072, 512), (2, 50001, 1000), (3, 40000, 1023)])
def test_gradient_of_a_token_or_a_few(m, n, k, dtype):
    """Large vocabularies: every class of every output."""
    x, w, b, target = ce.inputs(m, n, k, dtype, 0.0)
    loss, lse = ce.run_loss(x, w, b, target)
    ce.check_loss(x, w, b, target, 0.0, loss, lse)
    for out in (ce.T[dtype], torch.float32):
        print(f"a few {m} {n} {k} {out}", flush=True)
        dx, dw, db = ce.run_grad(x, w, b, target, lse, scale=1 / m, out=out)
        ce.check_grad(x, w, b, target, lse, None, 1 / m, 0.0, dx, dw, db)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [
    (1, 300, 24576), (2, 300, 12288), (1, 300, 24584), (2, 300, 12296), (4, 300, 4096),
    (3, 300, 4104), (2, 700, 2040), (16, 12288, 72), (16, 12289, 72), (32, 8192, 40),
    (32, 8193, 40), (64, 4096, 72), (64, 4097, 72), (17, 8192, 8), (33, 4096, 264)])
def test_few_rows_on_both_sides_of_the_rules(m, n, k, dtype):
    """By vectors, by groups of 16 columns and by tiles."""
    for a, bias, ignored in ((0.0, True, 0.0), (0.2, False, 0.4)):
        x, w, b, target = ce.inputs(m, n, k, dtype, ignored, bias)
        target[0] = n - 1
        print(f"both sides {m} {n} {k} {dtype} {a}", flush=True)
        ce.check_loss(x, w, b, target, a, *ce.run_loss(x, w, b, target, a))
