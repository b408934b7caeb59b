"""A two-layer perceptron trained data-parallel with the library's own kernels.

P virtual ranks each run forward and backward on their part of the batch in
bfloat16 (linear, linear_dgrad, linear_wgrad), the binary32 gradients are
averaged by the ring all-reduce, and the shared binary32 weights take a Muon
step (the matrices) and an AdamW step (the biases), which also write the
bfloat16 working copy of the next pass.  Synthetic data: a fixed random
teacher network.

    python examples/train_mlp.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sgd_gradient_all_amd as ddl  # noqa: E402


def train(steps=30, ranks=4, batch=256, sizes=(64, 256, 32), seed=0, device="cuda"):
    """The mean squared error before each step."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=gen, device=device) * sigma

    k, h, n = sizes
    # one flat buffer: W1, b1, W2, b2
    at = {"w1": (0, h, k), "b1": (h * k, h), "w2": (h * k + h, n, h)}
    at["b2"] = (at["w2"][0] + n * h, n)
    total = at["b2"][0] + n

    def part(flat, name):
        off, *shape = at[name]
        return flat[off:off + math.prod(shape)].view(*shape)

    weights = torch.zeros(total, device=device)
    part(weights, "w1").copy_(normal(h, k, sigma=k ** -0.5))
    part(weights, "w2").copy_(normal(n, h, sigma=h ** -0.5))
    work = weights.bfloat16()
    momentum, m, v = (torch.zeros_like(weights) for _ in range(3))
    teacher = normal(n, k, sigma=k ** -0.5)
    xs = [normal(batch, k).bfloat16() for _ in range(ranks)]
    ts = [torch.tanh(x.float() @ teacher.t()) for x in xs]

    grads = [torch.zeros_like(weights) for _ in range(ranks)]
    plan = ddl.Plan(ranks, total, "f32", "mean", ddl.topo("ring"),
                    [(at["w2"][0], total - at["w2"][0]), (0, at["w2"][0])])
    muon = ddl.Muon([(*at[w], 0.2 * math.sqrt(max(at[w][1:]))) for w in ("w1", "w2")])
    adam = ddl.AdamW([at["b1"], at["b2"]])
    space = torch.empty(max(ddl.linear_workspace(op, batch, *s) for s in ((h, k), (n, h))
                            for op in ("forward", "dgrad", "wgrad")),
                        device=device, dtype=torch.uint8)
    half = dict(device=device, dtype=torch.bfloat16)
    z1, a1, dz1, da1 = (torch.empty(batch, h, **half) for _ in range(4))
    y = torch.empty(batch, n, **half)

    losses = []
    for step in range(1, steps + 1):
        loss = 0.0
        for x, t, g in zip(xs, ts, grads):
            ddl.linear(x, part(work, "w1"), a1, bias=part(work, "b1"), act="silu", z=z1,
                       workspace=space)
            ddl.linear(a1, part(work, "w2"), y, bias=part(work, "b2"), workspace=space)
            d = y.float() - t
            loss = loss + d.square().mean() / ranks
            dy = (d * (2 / batch)).bfloat16()
            ddl.linear_wgrad(dy, a1, part(g, "w2"), db=part(g, "b2"), workspace=space)
            ddl.linear_dgrad(dy, part(work, "w2"), da1, act="silu", z_prev=z1, dz_prev=dz1,
                             workspace=space)
            ddl.linear_wgrad(dz1, x, part(g, "w1"), db=part(g, "b1"), workspace=space)
        plan.execute(grads)
        muon.step(grads[0], momentum, [weights], lr=0.02, weight_decay=0.01, copy=work)
        adam.step(grads[0], m, v, [weights], lr=0.01, weight_decay=0.01, step=step, copy=work)
        losses.append(loss)
    torch.cuda.synchronize()
    plan.destroy()
    muon.destroy()
    adam.destroy()
    return [float(x) for x in losses]


if __name__ == "__main__":
    for i, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)):
        print(f"step {i:3d}  loss {loss:.5f}")
