"""GPU parity of the block boundaries where single entries are infinite or NaN.
Bounds: those of test_gpu_norm."""

import numpy as np
import pytest
import torch

import test_gpu_norm as G
from gpu_util import banner

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
