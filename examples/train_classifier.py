"""A classifier trained data-parallel, from the loss to 8-bit optimizer states.

P virtual ranks each run a perceptron with two hidden layers in bfloat16 on their
part of the batch; the last layer's logits are never in memory (cross_entropy,
and cross_entropy_grad from its log-sum-exps).  The binary32 gradients are
averaged by the ring all-reduce; the hidden layers' matrices take a Muon step, the
last layer and the biases an AdamW step with both states in 8 bits, which also
write the bfloat16 working copy of the next pass.  Synthetic data: a fixed random
teacher's classes, some rows without one.

    python examples/train_classifier.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sgd_gradient_all_amd as ddl  # noqa: E402


class Classifier:
    """x -> silu(x w1^T + b1) -> w2, b2 -> classes by w3, b3; one flat buffer."""

    def __init__(self, ranks=4, batch=256, sizes=(64, 128, 96, 1000), seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, sigma=1.0):
            return torch.randn(*shape, generator=gen, device=device) * sigma

        k, h, g, n = sizes
        self.sizes, self.batch, self.at, total = sizes, batch, {}, 0
        # parts start 16 elements apart at least, where vectors of any type may
        for name, shape in (("w1", (h, k)), ("b1", (h,)), ("w2", (g, h)), ("b2", (g,)),
                            ("w3", (n, g)), ("b3", (n,))):
            self.at[name] = (total, *shape)
            total += -(-math.prod(shape) // 16) * 16
        self.weights = torch.zeros(total, device=device)
        for name in ("w1", "w2", "w3"):
            w = self.part(self.weights, name)
            w.copy_(normal(*w.shape, sigma=w.shape[1] ** -0.5))
        self.work = self.weights.bfloat16()
        self.grads = [torch.zeros_like(self.weights) for _ in range(ranks)]
        teacher = normal(n, k, sigma=k ** -0.5)
        self.xs = [normal(batch, k).bfloat16() for _ in range(ranks)]
        self.targets = [(x.float() @ teacher.t()).argmax(1) for x in self.xs]
        for t in self.targets:
            t[::7] = -1  # no target

        half = dict(device=device, dtype=torch.bfloat16)
        self.z1, self.a1, self.dz1, self.da1 = (torch.empty(batch, h, **half) for _ in range(4))
        self.h2, self.dh2 = (torch.empty(batch, g, **half) for _ in range(2))
        self.loss, self.lse = (torch.empty(batch, device=device) for _ in range(2))
        self.space = torch.empty(
            max([ddl.linear_workspace(op, batch, *s) for s in ((h, k), (g, h))
                 for op in ("forward", "dgrad", "wgrad")]
                + [ddl.cross_entropy_workspace(op, batch, n, g) for op in ("forward", "grad")]),
            device=device, dtype=torch.uint8)

        self.plan = ddl.Plan(ranks, total, "f32", "mean", ddl.topo("ring"),
                             [(self.at["w3"][0], total - self.at["w3"][0]),
                              (0, self.at["w3"][0])])
        self.muon = ddl.Muon([(*self.at[w], 0.2 * math.sqrt(max(self.at[w][1:])))
                              for w in ("w1", "w2")])
        self.adam = ddl.AdamW8([(self.at[p][0], math.prod(self.at[p][1:]))
                                for p in ("b1", "b2", "w3", "b3")])
        self.momentum = torch.zeros_like(self.weights)
        self.m = torch.zeros(total, device=device, dtype=torch.int8)
        self.v = torch.zeros(total, device=device, dtype=torch.uint8)
        self.scales = [torch.zeros(self.adam.blocks, device=device) for _ in range(2)]

    def part(self, flat, name):
        first, *shape = self.at[name]
        return flat[first:first + math.prod(shape)].view(*shape)

    def gradient(self, rank):
        """The rank's loss, a mean over its rows with a target; its gradient into
        self.grads[rank]."""
        x, t, g, w, s = (self.xs[rank], self.targets[rank], self.grads[rank],
                         lambda name: self.part(self.work, name), self.space)
        ddl.linear(x, w("w1"), self.a1, bias=w("b1"), act="silu", z=self.z1, workspace=s)
        ddl.linear(self.a1, w("w2"), self.h2, bias=w("b2"), workspace=s)
        ddl.cross_entropy(self.h2, w("w3"), t, self.loss, self.lse, bias=w("b3"), smoothing=0.1,
                          workspace=s)
        rows = self.batch - len(range(0, self.batch, 7))
        ddl.cross_entropy_grad(self.h2, w("w3"), t, self.lse, scale=1 / rows, dx=self.dh2,
                               dw=self.part(g, "w3"), db=self.part(g, "b3"), bias=w("b3"),
                               smoothing=0.1, workspace=s)
        ddl.linear_wgrad(self.dh2, self.a1, self.part(g, "w2"), db=self.part(g, "b2"),
                         workspace=s)
        ddl.linear_dgrad(self.dh2, w("w2"), self.da1, act="silu", z_prev=self.z1,
                         dz_prev=self.dz1, workspace=s)
        ddl.linear_wgrad(self.dz1, x, self.part(g, "w1"), db=self.part(g, "b1"), workspace=s)
        return self.loss.sum() / rows

    def step(self, number):
        """One training step (counted from 1); the mean loss before it."""
        losses = [self.gradient(r) for r in range(len(self.xs))]
        self.plan.execute(self.grads)
        self.muon.step(self.grads[0], self.momentum, [self.weights], lr=0.02, weight_decay=0.01,
                       copy=self.work)
        self.adam.step(self.grads[0], self.m, self.v, *self.scales, [self.weights], lr=0.01,
                       weight_decay=0.01, step=number, copy=self.work)
        return sum(losses) / len(losses)

    def destroy(self):
        torch.cuda.synchronize()
        for handle in (self.plan, self.muon, self.adam):
            handle.destroy()


def train(steps=30, **kw):
    """The mean loss before each step."""
    model = Classifier(**kw)
    losses = [model.step(i) for i in range(1, steps + 1)]
    model.destroy()
    return [float(x) for x in losses]


if __name__ == "__main__":
    for i, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)):
        print(f"step {i:3d}  loss {loss:.5f}")
