"""The linear layer's activations and their slopes over every 16-bit value of a range, relative to the
value itself: where a gate is small the result still has all the digits its type holds.

A product with one feature and a weight of 1 hands the kernel z itself, and a gradient of 1 gives the slope
as dz. Bounds, with r = 2^-24 and v the argument of the gate's sigmoid: the argument of erfc is off by two
roundings and erfc(a) changes by 2a^2 + 1 times its argument's relative change, a^2 = z^2/2; erfc itself is
off by at most 16 units of 2^-23 and the products by a few r: (2 z^2 + 40) r. An exponential of v is off by
|v| times its argument's relative error, at most 8 roundings for gelu_tanh's cubic and 3 for silu's
product with log2(e), and a few units of exp2, the sum and the reciprocal: (8 |v| + 40) r. The slopes add
a term z s (1 - s) u': its factors off by as much, and 1 - s by 8 r absolute near s = 1. A gate
below the smallest normal fp32 number may be 0. Then half a step of the type, and half its smallest number."""

import numpy as np
import pytest
import torch

import oracle as O
import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu
L = O.layer
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
R = 2.0 ** -24
FLUSH = 2.0 ** -126
C, A = np.sqrt(2 / np.pi), 0.044715


def values(dtype, most):
    """Every value of the type with 2^-8 <= |z| <= most, and 0."""
    z = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    z = z[torch.isfinite(z.float()) & (z.float().abs() <= most) & (z.float().abs() >= 2.0 ** -8)]
    return torch.cat([z, torch.zeros(1, dtype=z.dtype)])


def _gate_error(z, kind):
    """(relative error of the gate, the gate) in fp64."""
    if kind == "gelu":
        return (2 * z * z + 40) * R, L._erfc(-z / np.sqrt(2)) / 2
    v = 2 * C * (z + A * z ** 3) if kind == "gelu_tanh" else z
    return (8 * np.abs(v) + 40) * R, L._sigmoid(v)


def act_bound(z, kind):
    y = L.act(z, kind)
    if kind in ("none", "relu"):
        return y, 0 * z
    return y, _gate_error(z, kind)[0] * np.abs(y) + np.abs(z) * FLUSH


def slope_bound(z, kind):
    s = L.act_slope(z, kind)
    if kind == "relu":
        return s, 0 * z
    rel, gate = _gate_error(z, kind)
    if kind == "gelu":
        second = np.abs(z) * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        return s, rel * (gate + second) + (1 + np.abs(z)) * FLUSH
    du = 2 * C * (1 + 3 * A * z * z) if kind == "gelu_tanh" else 1.0
    v = 2 * C * (z + A * z ** 3) if kind == "gelu_tanh" else z
    second = np.abs(z) * gate * L._sigmoid(-v) * du
    return s, rel * (gate + 2 * second) + 8 * R * np.abs(z) * gate ** 2 * du + (1 + np.abs(z) * du) * FLUSH


def hold(got, want, err, dtype, what, z):
    half, tiny = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}[dtype]
    off = np.abs(got - want[:, None])
    ok = off <= (err + half * (np.abs(want) + err) + tiny)[:, None]
    at = np.argwhere(~ok)
    assert ok.all(), (what, len(at), [(z[i], got[i, j], want[i]) for i, j in at[:4]])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", L.ACTS)
def test_every_value_relative_to_itself(kind, dtype):
    banner(f"activation {kind} {dtype}")
    zt = values(dtype, 12.0).to(DEV)
    z, m, n = zt.double().cpu().numpy(), zt.numel(), 24
    one = torch.ones(n, 1, dtype=zt.dtype, device=DEV)
    ws = torch.empty(max(16, *(Z.zero_linear_workspace_bytes(m, 1, n, b) for b in (False, True))), dtype=torch.uint8, device=DEV)
    y, pre, dz = (torch.empty(m, n, dtype=zt.dtype, device=DEV) for _ in range(3))
    Z.zero_linear_forward(zt[:, None], one, y, act=kind, pre=pre, workspace=ws)           # the tile kernel
    few = torch.empty(1, m, dtype=zt.dtype, device=DEV)
    Z.zero_linear_forward(one[:1], zt[:, None], few, act=kind)                            # the kernel for few rows
    torch.cuda.synchronize()
    assert torch.equal(pre, zt[:, None].expand(m, n))
    want, err = act_bound(z, kind)
    hold(y.double().cpu().numpy(), want, err, dtype, "y", z)
    hold(few.double().cpu().numpy().T, want, err, dtype, "y of one row", z)
    if kind == "none":
        return
    Z.zero_linear_backward(torch.ones_like(pre), zt[:, None], one, act=kind, pre=pre, dz=dz, workspace=ws)
    torch.cuda.synchronize()
    want, err = slope_bound(z, kind)
    hold(dz.double().cpu().numpy(), want, err, dtype, "dz", z)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", [k for k in L.ACTS if k != "none"])
def test_slopes_of_far_values(kind, dtype):
    """Every value beyond 12, up to the type's largest, and the infinities that an overflow of the
    pre-activation's type leaves: the slope goes to 1 and 0, and is no NaN. A NaN stays one."""
    banner(f"far slopes {kind} {dtype}")
    z = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    zt = z[~torch.isnan(z.float()) & (z.float().abs() > 12.0)].to(DEV)
    assert int(torch.isinf(zt).sum()) == 2
    z, m, n = zt.double().cpu().numpy(), zt.numel(), 8
    pre = zt[:, None].expand(m, n).contiguous()
    dz, dx = torch.empty_like(pre), torch.empty(m, 1, dtype=zt.dtype, device=DEV)
    x, w = torch.ones(m, 1, dtype=zt.dtype, device=DEV), torch.ones(n, 1, dtype=zt.dtype, device=DEV)
    ws = torch.empty(max(16, Z.zero_linear_workspace_bytes(m, 1, n, True)), dtype=torch.uint8, device=DEV)
    Z.zero_linear_backward(torch.ones_like(pre), x, w, act=kind, pre=pre, dz=dz, dx=dx, workspace=ws)
    torch.cuda.synchronize()
    near = np.clip(z, -1e18, 1e18)                    # the bounds' own terms stay finite
    want, err = slope_bound(near, kind)
    assert np.array_equal(want, np.clip(L.act_slope(z, kind), -9, 9))
    got = dz.double().cpu().numpy()
    far = np.abs(z) > 200                             # where even silu's slope is a whole number
    assert (got[far] == (z[far] > 0)[:, None]).all()
    hold(got, want, np.where(far, 0.0, err), dtype, "dz", z)
    assert bool(torch.isfinite(dx).all())
    pre.fill_(float("nan"))
    Z.zero_linear_backward(torch.ones_like(pre), x, w, act=kind, pre=pre, dz=dz, workspace=ws)
    torch.cuda.synchronize()
    assert bool(torch.isnan(dz).all())
