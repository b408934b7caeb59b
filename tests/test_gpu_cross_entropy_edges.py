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
