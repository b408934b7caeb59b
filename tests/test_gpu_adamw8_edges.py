"""The AdamW8 step where its numbers are subnormal, with the tolerances of
test_gpu_adamw8.py."""
import pytest
import torch

import sgd_gradient_all_amd as ddl
from test_gpu_adamw8 import B, F32, gen, normal

pytestmark = pytest.mark.gpu


def zeros(n, blocks):
    return [torch.zeros(n, device="cuda", dtype=t) for t in (torch.int8, torch.uint8)] \
        + [torch.zeros(blocks, device="cuda") for _ in range(2)]


@pytest.mark.parametrize("eps", [1e-11, 1e-13, 1e-8, 1e-3, 1e-20])
@pytest.mark.parametrize("b2", [0.95, 0.9999, 0.999999])
def test_a_second_moment_under_the_normal_numbers(b2, eps):
    """Gradients around the size whose v is subnormal, a factor of 1.5 apart: the root
    of v beside eps."""
    n = 4 * B
    h, st = ddl.AdamW8([(0, n)]), zeros(n, 4)
    top = (2.0 ** -126 / (1 - b2)) ** 0.5
    gr = (top * 1.5 ** (torch.arange(n, device="cuda") % 8 - 5.0)).float()
    w = torch.zeros(n, device="cuda")
    print(f"subnormal v {b2} {eps}", flush=True)
    h.step(gr, *st, [w], lr=1e-2, beta1=0.9, beta2=b2, eps=eps)
    g = gr.double()
    # v is rounded once, to 2^-150 at most where it is subnormal, its root by half as much
    v = (1 - b2) * g * g
    want = -1e-2 * g / (g + eps)
    slack = (2.0 ** -150 / v) * 0.5 * g / (g + eps) * want.abs()
    assert ((w.double() - want).abs() <= 16 * F32 * want.abs() + slack).all()


@pytest.mark.parametrize("eps", [1e-40, 1e-50, 1e-300, 2.0 ** -126, 1e-38])
def test_weights_without_a_gradient_stay_under_a_tiny_eps(eps):
    n = 3 * B + 5
    h, g_ = ddl.AdamW8([(0, n)]), gen(1)
    st, w = zeros(n, h.blocks), normal(g_, n, 0.02)
    gr, w0 = normal(g_, n, 1e-2), w.clone()
    gr[::3] = 0.0
    gr[B:2 * B] = 0.0
    print(f"tiny eps {eps}", flush=True)
    h.step(gr, *st, [w], lr=1e-2, eps=eps, weight_decay=0.0)
    assert torch.equal(w[gr == 0], w0[gr == 0])
    want = w0.double() - 1e-2 * torch.sign(gr.double())
    assert ((w.double() - want).abs() <= 16 * F32 * 1e-2 + 4 * F32 * w0.double().abs()).all()


def test_a_huge_eps():
    """Its reciprocal is subnormal; the product with a large gradient is not."""
    n = B
    h, st = ddl.AdamW8([(0, n)]), zeros(n, 1)
    gr, w = normal(gen(2), n, 1e17), torch.zeros(n, device="cuda")
    h.step(gr, *st, [w], lr=1e10, eps=2.0 ** 127)
    want = -1e10 * gr.double() / (gr.double().abs() + 2.0 ** 127)
    assert ((w.double() - want).abs() <= 16 * F32 * want.abs()).all()
