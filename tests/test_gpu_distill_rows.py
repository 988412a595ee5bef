"""The distillation loss on batches: every kernel that 512 rows and more take, the largest sizes, and rows that a weight
of 0 masks. Against the definition in 64 bits on the device, with test_gpu_distill's bounds: q and p are off by
rel = (V/256 + 64 + 4 span) 2^-24 relative, a gradient by g (2 q + 2 |grad|/g) rel and its rounding, a loss by rel and 8 roundings
of its logarithms."""

import numpy as np
import pytest
import torch

import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
U = 2.0 ** -24


def definition(z, idx, top, T, tail, weight):
    """(loss, gradient, q) in fp64, of rows that have a softmax or no weight."""
    lq = torch.log_softmax(z.double() / T, 1)
    valid = (idx >= 0) & (idx < z.shape[1])
    cols = torch.where(valid, idx, 0).long()
    lp = (top.double() / T).masked_fill(~valid, -torch.inf)
    if tail is not None:
        lp = torch.cat([lp, tail.double()[:, None]], 1)
    none = lp.max(1).values == -torch.inf
    lp = torch.log_softmax(lp, 1)
    K = idx.shape[1]
    p = torch.where(none[:, None], 0.0, lp.exp())
    terms = torch.where(p[:, :K] > 0, p[:, :K] * (lp[:, :K] - lq.gather(1, cols)), 0.0)
    loss, q = terms.sum(1), lq.exp()
    grad = q.clone().scatter_add_(1, cols, -p[:, :K])
    if tail is not None:
        listed = torch.zeros(z.shape, dtype=torch.int8, device=z.device).scatter_add_(1, cols, valid.to(torch.int8)) > 0
        log_rest = torch.logsumexp(lq.masked_fill(listed, -torch.inf), 1)
        loss += torch.where(p[:, K] > 0, p[:, K] * (lp[:, K] - log_rest), 0.0)
        grad -= (p[:, K:] * (lq - log_rest[:, None]).exp()).masked_fill(listed, 0.0)
    off = none | (weight == 0)
    grad = torch.where(off[:, None], 0.0, grad * (weight.double() / T)[:, None])
    return torch.where(off, 0.0, loss * weight.double()), grad, torch.nan_to_num(q)


def batch(R, V, K, dtype, tail, seed):
    """Rows with distinct entries whose logits the student shares up to noise; some short, some with an entry outside or twice,
    one without any, every seventh masked and one of those not even a number."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = torch.randn(R, V, generator=g, device=DEV) * 2
    idx = (torch.randint(V, (R, 1), generator=g, device=DEV) + torch.arange(K, device=DEV) * 7) % V
    top = torch.randn(R, K, generator=g, device=DEV) * 2 + 6
    z.scatter_(1, idx, top + torch.randn(R, K, generator=g, device=DEV))
    weight = torch.rand(R, generator=g, device=DEV) + 0.25
    weight[3::7] = 0.0
    idx[1, K // 2:] = -1
    idx[4, 0] = V
    if K > 2:
        idx[2, 2] = idx[2, 0]
    idx[5] = -1
    z = z.to(DT[dtype])
    z[3] = float("nan")
    z[6, : V // 3] = float("-inf")                      # masked logits
    z[6].scatter_(0, idx[6].clamp(min=0), 1.0)
    return z, idx.int(), top, (torch.randn(R, generator=g, device=DEV) + 4 if tail else None), weight


def agree(R, V, K, dtype, tail, kind, T, scale):
    banner(f"distill batch R={R} V={V} K={K} {dtype} tail={tail} {kind}")
    z, idx, top, t, weight = batch(R, V, K, dtype, tail, R + V)
    up = torch.rand(R, device=DEV) + 0.5
    loss, grad = torch.full((R,), -9.0, device=DEV), torch.full_like(z, -9.0)
    kw = dict(tail=t, weight=weight)
    if kind == "step":
        Z.zero_distill_step(z, idx, top, T, loss, grad, upstream=up, scale=scale, **kw)
    else:
        stats = torch.empty(R, 2, device=DEV)
        Z.zero_distill_forward(z, idx, top, T, loss, stats, **kw)
        Z.zero_distill_backward(z, idx, top, T, stats, grad, upstream=up, scale=scale, **kw)
    torch.cuda.synchronize()
    most = max(1, (1 << 26) // V)                         # 64-bit copies of half a gigabyte
    for lo in range(0, R, most):
        at = slice(lo, min(R, lo + most))
        want, wg, q = definition(z[at], idx[at], top[at], T, None if t is None else t[at], weight[at])
        w = weight[at].double()
        real = torch.where(torch.isfinite(z[at].float()), z[at].float(), 0.0)
        span = (1.4427 / T * (real.max(1).values - real.min(1).values)).clamp(max=60).double()
        rel = (V / 256 + 64 + 4 * span) * U
        err = (loss[at].double() - want).abs()
        ok = err <= w * (rel + 8 * U * (span + np.log2(V) + 40))
        assert bool(ok.all()), ("loss", lo + int((~ok).nonzero()[0]), float(err.max()))
        f = (scale * up[at].double())[:, None]
        wg = wg * f
        g = (f[:, 0] * w / T)[:, None]
        tol = 2 * (g * q + wg.abs()) * rel[:, None] + HALF_STEP[dtype] * wg.abs() + g * 2.0 ** -40
        if dtype == "f16":
            tol += 2.0 ** -25
        bad = ~((grad[at].double() - wg).abs() <= tol)
        if bool(bad.any()):
            r, c = (int(v) for v in bad.nonzero()[0])
            raise AssertionError(("gradient", int(bad.sum()), lo + r, c, float(grad[lo + r, c]), float(wg[r, c]), float(tol[r, c])))


# columns (16-bit; fp32 rows are half as long) up to each amount of a row that a thread holds: 4, 8, 16 and 28 vectors in 256
# threads, 28 in 512, 16 in 1024, and longer ones, which are read twice
WIDTHS = [8191, 16384, 32000, 50257, 100001, 131072, 140003]


@pytest.mark.parametrize("kind", ["step", "calls"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("width", WIDTHS)
def test_batches(width, large, dtype, tail, kind):
    """512 rows and a few, and as many as make a gradient of 128 MiB, which goes past the caches."""
    V = (width + 1) // 2 if dtype == "f32" else width
    R = (1 << 27) // (V * (4 if dtype == "f32" else 2)) + 3 if large else 513
    if large and R < 512:
        R = 700
    agree(R, V, 33, dtype, tail, kind, 2.0, 64.0)


@pytest.mark.parametrize("kind", ["step", "calls"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R", [8, 520])
def test_the_largest_row_and_teacher(R, dtype, kind):
    agree(R, Z.ZERO_DISTILL_MAX_VOCAB, Z.ZERO_DISTILL_MAX_TOPK, dtype, True, kind, 1.0, 1.0)


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


@pytest.mark.parametrize("kind", ["step", "calls"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", [(3, 140003), (520, 140003), (520, 50257), (40, 16001)])
def test_over_the_logits_themselves(R, V, dtype, kind):
    """The gradient in place of the logits, rows longer and shorter than the registers hold: bit for bit as apart."""
    banner(f"distill in place R={R} V={V} {dtype} {kind}")
    z, idx, top, t, weight = batch(max(R, 8), V, 33, dtype, True, R)
    z, idx, top, t, weight = (a[:R].contiguous() for a in (z, idx, top, t, weight))
    out = []
    for apart in (True, False):
        logits = z.clone()
        loss, grad = torch.empty(R, device=DEV), torch.empty_like(z) if apart else logits
        kw = dict(tail=t, weight=weight)
        if kind == "step":
            Z.zero_distill_step(logits, idx, top, 2.0, loss, grad, scale=8.0, **kw)
        else:
            stats = torch.empty(R, 2, device=DEV)
            Z.zero_distill_forward(logits, idx, top, 2.0, loss, stats, **kw)
            Z.zero_distill_backward(logits, idx, top, 2.0, stats, grad, scale=8.0, **kw)
        torch.cuda.synchronize()
        out.append((loss, grad))
    bits = torch.int32 if dtype == "f32" else torch.int16
    assert torch.equal(out[0][0].view(torch.int32), out[1][0].view(torch.int32))
    assert torch.equal(out[0][1].view(bits), out[1][1].view(bits))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("kind", ["step", "calls"])
def test_a_teacher_without_a_softmax(kind, tail):
    """A NaN or +inf among the teacher's logits, or a NaN for the tail: the loss and the listed entries' gradients
    are NaN, so that the overflow flag sees the row; other rows are as without it."""
    z, idx, top, t, weight = batch(9, 3001, 20, "f32", tail, 2)
    weight.fill_(1.0)
    z[3], z[6] = z[0], z[1]
    clean = None
    for spoil in (False, True):
        if spoil:
            top[0, 7], top[7, 3] = float("nan"), float("inf")
            if tail:
                t[8] = float("nan")
        loss, grad, stats = torch.empty(9, device=DEV), torch.empty_like(z), torch.empty(9, 2, device=DEV)
        if kind == "step":
            Z.zero_distill_step(z, idx, top, 1.5, loss, grad, tail=t, weight=weight)
        else:
            Z.zero_distill_forward(z, idx, top, 1.5, loss, stats, tail=t, weight=weight)
            Z.zero_distill_backward(z, idx, top, 1.5, stats, grad, tail=t, weight=weight)
        torch.cuda.synchronize()
        if not spoil:
            clean = loss, grad
            assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad).all())
    bad = [0, 7] + ([8] if tail else [])
    good = [r for r in range(9) if r not in bad]
    assert bool(torch.isnan(loss[bad]).all())
    for r in bad:
        assert bool(torch.isnan(grad[r, idx[r][idx[r] >= 0].long()]).all())
    assert torch.equal(loss[good], clean[0][good]) and torch.equal(grad[good], clean[1][good])
