"""GPU parity of the linear layer, continued: whole numbers, so every result is exact in fp32 and must equal the
64-bit one rounded once."""

import pytest
import torch

import zero_partition_plan_amd as Z
from gpu_util import DEV, banner
from linear_shapes import TILES, TOO_MANY_TILES
from test_gpu_linear import DT, SHARED, SIZES, Placed, gen, ints, same, ws

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


def _exact(a, b):
    """a b^T of whole numbers, exact in fp32 (sums below 2^24)."""
    return torch.mm(a.float().contiguous(), b.float().contiguous().t())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("order,shape,split", TILES)
def test_every_tile_with_all_that_it_writes(order, shape, split, held, dtype):
    """Each tile of each product, joined over k or not, from operands loaded directly and from ones an element
    off: forward with bias, activation, residual and the kept pre-activation, and over the residual itself;
    weight gradients written and added to, 16-bit and fp32. Edges odd (or even, beside them), NaN around every operand."""
    m, k, n = TILES[order, shape, split]
    n += held
    off, pad = (1, 0) if held else (8, "to 8")
    banner(f"linear tile {order} {shape} split={split} held={held} {dtype} m={m} k={k} n={n}")
    dt, g, nan = DT[dtype], gen(m + k + n), float("nan")
    x = Placed(m, k, dt, off, pad, nan).set(ints(g, m, k))
    w = Placed(n, k, dt, off, 0, nan).set(ints(g, n, k))
    if order == "fwd":
        b = Placed(1, n, dt, off, 0, nan).set(ints(g, 1, n))
        r = Placed(m, n, dt, off, pad).set(ints(g, m, n, 50))
        y, pre = Placed(m, n, dt, off, pad), Placed(m, n, dt, off, pad)
        z = _exact(x.t, w.t)
        Z.zero_linear_forward(x.t, w.t, y.t, workspace=ws(m, k, n))
        same(y.t, z, "y")
        z = z + b.t.float()
        Z.zero_linear_forward(x.t, w.t, y.t, bias=b.t[0], residual=r.t, act="relu", pre=pre.t, workspace=ws(m, k, n))
        same(y.t, z.clamp_min(0) + r.t.float(), "y of everything")
        same(pre.t, z, "pre")
        z = z + r.t.float()
        Z.zero_linear_forward(x.t, w.t, r.t, bias=b.t[0], residual=r.t, workspace=ws(m, k, n))
        same(r.t, z, "y in place of the residual")
        for p, what in ((y, "y"), (pre, "pre"), (r, "residual")):
            p.check_canary(what)
        return
    dy = Placed(m, n, dt, off, pad, nan).set(ints(g, m, n))
    if order == "dx":
        dx = Placed(m, k, dt, off, pad)
        Z.zero_linear_backward(dy.t, None, w.t, dx=dx.t, workspace=ws(m, k, n, True))
        same(dx.t, _exact(dy.t, w.t.t()), "dx")
        dx.check_canary("dx")
        return
    want = _exact(dy.t.t(), x.t.t())
    for gdt in (dt, torch.float32):
        dw, old = Placed(n, k, gdt, off), ints(g, n, k, 40).float()
        Z.zero_linear_backward(dy.t, x.t, None, dweight=dw.t, workspace=ws(m, k, n, True))
        same(dw.t, want, "dweight")
        dw.t.copy_(old)
        Z.zero_linear_backward(dy.t, x.t, None, dweight=dw.t, accumulate=True, workspace=ws(m, k, n, True))
        same(dw.t, want + old, "dweight added to")
        dw.check_canary("dweight")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,k,n", SIZES + SHARED)
def test_residual_in_place_at_every_size(m, k, n, dtype):
    banner(f"linear residual in place m={m} k={k} n={n} {dtype}")
    dt, g = DT[dtype], gen(m + n)
    x, w = ints(g, m, k).to(dt), ints(g, n, k).to(dt)
    r = Placed(m, n, dt, 3, 5).set(ints(g, m, n, 50))
    want = _exact(x, w) + r.t.float()
    Z.zero_linear_forward(x, w, r.t, residual=r.t, workspace=ws(m, k, n))
    same(r.t, want, "y in place of the residual")
    r.check_canary("y")


def test_more_tiles_than_a_grid_holds():
    """A long and narrow result whose 64 x 64 tiles, the planned ones, are past 2^23: it takes larger ones."""
    m, k, n = TOO_MANY_TILES
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GiB")
    banner(f"linear more tiles than a grid holds m={m} k={k} n={n}")
    g = gen(9)
    x = torch.randint(-3, 4, (m, k), generator=g, device=DEV, dtype=torch.int8).bfloat16()
    w = ints(g, n, k).bfloat16()
    y = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    Z.zero_linear_forward(x, w, y, workspace=ws(m, k, n))
    wt = w.float().t().contiguous()
    for r in range(0, m, 1 << 22):                 # whole numbers of at most 72: exact in bf16
        assert torch.equal(y[r:r + (1 << 22)], (x[r:r + (1 << 22)].float() @ wt).bfloat16()), r
    del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,unit", [("f16", 2.0 ** -24), ("bf16", 2.0 ** -133)])
@pytest.mark.parametrize("m,k,n", [(3, 72, 40), (100, 200, 136), (700, 264, 520)])
def test_subnormal_operands(m, k, n, dtype, unit):
    """Whole multiples of the type's smallest number: what gradients below a loss scale come to. Exact as the
    whole numbers are, in the products, the sums, the 16-bit results and the bias gradient."""
    banner(f"linear subnormal {dtype} m={m} k={k} n={n}")
    dt, g = DT[dtype], gen(m)
    x, dy = (ints(g, *s, 9) * unit for s in ((m, k), (m, n)))
    w = ints(g, n, k)
    xt, dt_, wt = x.to(dt), dy.to(dt), w.to(dt)
    assert torch.equal(xt.double(), x) and torch.equal(dt_.double(), dy)
    y, dx, dw, db = (torch.empty(s, dtype=dt, device=DEV) for s in ((m, n), (m, k), (n, k), (n,)))
    Z.zero_linear_forward(xt, wt, y, workspace=ws(m, k, n))
    one = torch.ones(m, k, dtype=dt, device=DEV)
    Z.zero_linear_backward(dt_, one, wt, dx=dx, dweight=dw, dbias=db, workspace=ws(m, k, n, True))
    same(y, (x.cpu() @ w.cpu().t()).to(DEV), "y")
    same(dx, (dy.cpu() @ w.cpu()).to(DEV), "dx")
    same(db, dy.sum(0), "dbias")
    same(dw, dy.sum(0)[:, None].expand(n, k), "dweight")


_FIRST = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import zero_partition_plan_amd as Z
dev = "cuda:0"
m, k, n = 2048, 2048, 8192          # tiles of more LDS than a kernel has without asking
x, w, dy = (torch.randint(-3, 4, s, device=dev).bfloat16() for s in ((m, k), (n, k), (m, n)))
y, dx, dw = torch.empty(m, n, dtype=torch.bfloat16, device=dev), torch.empty_like(x), torch.empty(n, k, device=dev)
z = torch.randn(64, 5000, device=dev)
idx, top, loss, grad = torch.randint(5000, (64, 4), device=dev), torch.randn(64, 4, device=dev), torch.empty(64, device=dev), torch.empty_like(z)
ws = torch.empty(max(16, *(Z.zero_linear_workspace_bytes(m, k, n, b) for b in (False, True))), dtype=torch.uint8, device=dev)
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    Z.zero_linear_forward(x, w, y, workspace=ws)
    Z.zero_linear_backward(dy, x, w, dx=dx, dweight=dw, workspace=ws)
    Z.zero_distill_step(z, idx, top, 1.0, loss, grad)
for _ in range(3):
    for t in (y, dx, dw, loss, grad):
        t.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, dx, dw, loss, grad)]
    Z.zero_linear_forward(x, w, y, workspace=ws)
    Z.zero_linear_backward(dy, x, w, dx=dx, dweight=dw, workspace=ws)
    Z.zero_distill_step(z, idx, top, 1.0, loss, grad)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw, loss, grad)))
    assert torch.equal(y.float(), (x.float() @ w.float().t()).bfloat16().float())
print("captured first")
"""


def test_the_first_call_of_a_process_may_be_captured():
    """Nothing of the library's kernels loaded or allowed before the capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", _FIRST, root], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and "captured first" in run.stdout, (run.stdout + run.stderr)[-3000:]
