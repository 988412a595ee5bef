"""GPU parity of the linear layer, continued: whole numbers, so every result is exact in fp32 and must equal the
64-bit one rounded once."""

import pytest
import torch

import zero_partition_plan_amd as Z
from gpu_util import DEV, banner
from test_gpu_linear import DT, Placed, gen, ints, same, ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,k,n", [(5, 40, 24), (300, 264, 136)])
def test_backward_without_what_it_does_not_read(m, k, n):
    """dx without x, dweight without the weight, dbias and dz without either: as with them."""
    banner(f"linear backward without operands m={m} k={k} n={n}")
    dt, g = torch.bfloat16, gen(m)
    x, w, dy, pre = (ints(g, *s).to(dt) for s in ((m, k), (n, k), (m, n), (m, n)))
    dx, dw, db, dz = torch.empty_like(x), torch.empty(n, k, device=DEV), torch.empty(n, device=DEV), torch.empty_like(dy)
    w0 = ws(m, k, n, True)
    Z.zero_linear_backward(dy, None, w, dx=dx, workspace=w0)
    Z.zero_linear_backward(dy, x, None, dweight=dw, workspace=w0)
    Z.zero_linear_backward(dy, None, None, dbias=db, workspace=w0)
    D = dy.double().cpu()
    same(dx, (D @ w.double().cpu()).to(DEV), "dx")
    same(dw, (D.t() @ x.double().cpu()).to(DEV), "dweight")
    same(db, D.sum(0).to(DEV), "dbias")
    D = D * (pre.double().cpu() > 0)
    Z.zero_linear_backward(dy, None, None, act="relu", pre=pre, dz=dz, dbias=db, workspace=w0)
    same(dz, D.to(DEV), "dz")
    same(db, D.sum(0).to(DEV), "dbias behind relu")
    with pytest.raises(Z.ZeroError):
        Z.zero_linear_backward(dy, None, w, dweight=dw, workspace=w0)
    with pytest.raises(Z.ZeroError):
        Z.zero_linear_backward(dy, x, None, dx=dx, workspace=w0)
    with pytest.raises(ValueError):
        Z.zero_linear_backward(dy, x, None, dx=torch.empty(m, k + 1, dtype=dt, device=DEV), workspace=w0)
