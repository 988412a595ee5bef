"""The distillation loss on batches: rows that a weight of 0 masks."""

import pytest
import torch

import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu


def test_masked_rows_are_not_read():
    """A row of weight 0 costs the write of its zeros and no read: a batch of nothing else moves half the bytes
    of an ordinary one (524 MB of each, past the caches). Both times are the least of 20; between 1/2 and 1 lies the bound."""
    R, V, K = 8192, 32000, 16
    banner("distill masked rows")
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    z = torch.randn(R, V, generator=g, device=DEV).bfloat16()
    idx = torch.randint(V, (R, K), generator=g, device=DEV)
    top = torch.randn(R, K, generator=g, device=DEV)
    loss, grad = torch.empty(R, device=DEV), torch.empty_like(z)

    def least(weight):
        best = 1e9
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            Z.zero_distill_step(z, idx, top, 1.0, loss, grad, weight=weight)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    full = least(torch.ones(R, device=DEV))
    assert bool(grad.any()) and bool((loss > 0).all())
    masked = least(torch.zeros(R, device=DEV))
    assert not bool(grad.any()) and not bool(loss.any())
    print(f"[gpu] all rows {full * 1e3:.0f} us, all masked {masked * 1e3:.0f} us", flush=True)
    assert masked <= 0.75 * full
