"""The loss, its gradient, the all-reduce and the optimizers together, as the
classifier example uses them."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_classifier.py")
    spec = importlib.util.spec_from_file_location("train_classifier", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_runs_the_same_twice():
    mod = example()
    losses = mod.train(steps=6)
    assert len(losses) == 6 and all(math.isfinite(x) for x in losses)
    assert losses == mod.train(steps=6)


def test_example_gradients():
    """A rank's gradient against autograd's of the same loss in 64 bits, on the
    bfloat16 working weights.  On the way a1, h2, dh2, da1 and dz1 are rounded to
    bfloat16, dz3 for dh2 once more: six roundings of 2^-8 at most, each of which a
    product passes on to the gradient's norm as it passes on its input's, but for
    what cancels; 4 is allowed for that."""
    model = example().Classifier()
    loss = model.gradient(1)
    w = {n: model.part(model.work, n).double().requires_grad_() for n in model.at}
    t = model.targets[1]
    a1 = torch.nn.functional.silu(model.xs[1].double() @ w["w1"].t() + w["b1"])
    z = (a1 @ w["w2"].t() + w["b2"]) @ w["w3"].t() + w["b3"]
    have = t >= 0
    at = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    each = torch.logsumexp(z, 1) - 0.9 * at - 0.1 * z.mean(1)
    total = each[have].mean()
    grads = dict(zip(w, torch.autograd.grad(total, list(w.values()))))
    # logits of a few units, of values rounded to bfloat16 twice
    assert abs(float(loss) - float(total.detach())) <= 2 * 2.0 ** -8 * float(z.detach().abs().mean()) * 2
    for name, want in grads.items():
        got = model.part(model.grads[1], name).double()
        assert float((got - want).norm()) <= 4 * 6 * 2.0 ** -8 * float(want.norm()), name
    model.destroy()


def test_example_step_is_the_parts_in_order():
    """The weights that a step leaves: the mean gradient by the all-reduce, AdamW on
    it with zero states (m / sqrt(v) is the gradient's sign, nearly), decay."""
    model = example().Classifier()
    for r in range(4):
        model.gradient(r)
    mean = sum(g.double() for g in model.grads) / 4
    before = model.weights.clone()
    model.step(1)
    for name in ("b1", "b2", "w3", "b3"):
        first, *shape = model.at[name]
        at = slice(first, first + math.prod(shape))
        g, w0 = mean[at], before[at].double()
        want = w0 * (1 - 0.01 * 0.01) - 0.01 * g / (g.abs() + 1e-8)
        # the mean is rounded to binary32 four times, and sign(g) turns over eps
        slack = 0.01 * 8 * 2.0 ** -24 * g.abs().max() / (g.abs() + 1e-8) + 2.0 ** -20 * w0.abs() \
            + 1e-2 * 2.0 ** -18
        assert ((model.weights[at].double() - want).abs() <= slack).all(), name
        assert torch.equal(model.work[at], model.weights[at].bfloat16())
    model.destroy()
