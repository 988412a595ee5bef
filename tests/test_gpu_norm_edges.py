"""GPU parity of the block boundaries where single entries are infinite or NaN, and of statistics off 16 bytes.
Bounds: those of test_gpu_norm."""

import numpy as np
import pytest
import torch

import test_gpu_norm as G
import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _memory_given_back():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("gate,per", [(None, 1), ("channel", 6), ("token", 1), ("sequence", 4)])
@pytest.mark.parametrize("dtype,stream,n", [("bf16", "bf16", 64), ("f16", "f32", 779), ("bf16", "f32", 4100), ("bf16", "bf16", 8208)])
def test_a_branch_without_a_norm_has_no_part_in_its_own_gradient(dtype, stream, n, gate, per):
    """dbranch = branch_scale*gate*dy, whatever the branch holds: an inf or a NaN of it stays where it is."""
    banner(f"norm branch of no norm {dtype} {stream} n={n} {gate}")
    c = G.Case(n, 6, n, dtype, stream, "none", "none", gate, per)
    for r, col, x in ((0, 0, "inf"), (2, n - 1, "-inf"), (3, n // 2, "nan"), (5, 5, "inf")):
        c.branch[r, col] = float(x)
    y, _ = c.forward()
    bad = ~torch.isfinite(c.branch)
    assert torch.equal(~torch.isfinite(y), bad)
    c.backward()
    g = 1.0 if c.gate is None else G.N.spread(G.host(c.gate), 6, per)
    want = c.c * g * G.host(c.dy)
    G.close(G.host(c.grads["dbranch"]), want, (G.K + G.HALF[dtype]) * np.abs(want) + G.LEAST[dtype], "dbranch")
    want = c.a * G.host(c.dy)
    G.close(G.host(c.grads["dx"]), want, (G.K + G.HALF[stream]) * np.abs(want), "dx")
    if gate is not None:
        each = c.c * G.host(c.dy) * G.host(c.branch)
        want = np.zeros((len(c.gate), n))
        np.add.at(want, np.arange(6) // per, each)
        size = np.zeros((len(c.gate), n))
        np.add.at(size, np.arange(6) // per, np.abs(each))
        G.close(G.host(c.grads["dgate"]), want, (G.K + 6 * G.U) * size, "dgate")


@pytest.mark.parametrize("n", [96, 4096, 8208])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_statistics_at_any_float(off, n):
    """stats is an array of float: every multiple of 4 bytes is a place for it."""
    c = G.Case(off, 9, n, "bf16", "bf16", "layer", "rms", "channel", 9)
    y, h = (t.clone() for t in c.forward())
    first = c.backward()
    buf = torch.full((4 * 9 + 8,), -7.0, device=DEV)
    stats = buf[off:off + 36].view(9, 4)
    y2, h2 = torch.empty_like(y), torch.empty_like(h)
    Z.zero_norm_forward(c.x, h=h2, y=y2, stats=stats, **c.kw())
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(stats, c.stats)
    assert bool((buf[:off] == -7.0).all()) and bool((buf[off + 36:] == -7.0).all())
    grads = {k: torch.empty_like(t) for k, t in c.grads.items()}
    ws = torch.empty(Z.zero_norm_workspace_bytes(9, n, gate_rows=9), dtype=torch.uint8, device=DEV)
    Z.zero_norm_backward(c.y, stats, dy=c.dy, dh=c.dh, workspace=ws, **grads, **c.kw())
    torch.cuda.synchronize()
    for k, t in grads.items():
        assert np.array_equal(G.host(t), first[k]), k
