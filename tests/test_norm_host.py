"""The argument checks of the block boundaries, on the CPU: every call here is refused (or is empty) before any
device work."""

import ctypes

import pytest
import torch

import zero_partition_plan_amd as Z

INVAL, OVERFLOW, UNSUPPORTED = 1, 2, 3
A = 1 << 40                                            # fake addresses, never dereferenced
STEP = 1 << 28


def _addr(k):
    return A + k * STEP


BLOCK = dict(rows=8, features=32, gate_rows=4, dtype=Z.ZERO_BF16, stream_dtype=Z.ZERO_F32, post=1, pre=2, eps=1e-5,
             residual_scale=1.0, branch_scale=1.0, branch=_addr(1), ld_branch=32, gate=_addr(2), ld_gate=32,
             post_weight=_addr(3), post_bias=_addr(4), pre_weight=_addr(5), pre_bias=_addr(6))


def _block(**kw):
    return Z.ZeroNormBlock(**{**BLOCK, **kw})


def _fwd(b=None, x=_addr(10), ldx=32, y=_addr(11), ldy=32, h=_addr(12), ldh=32, stats=_addr(13)):
    b = b or _block()
    return Z.lib().zero_norm_forward(ctypes.byref(b), x, ldx, y, ldy, h, ldh, stats, None)


def _bwd(b=None, stats=_addr(13), y=_addr(11), ldy=32, dy=_addr(14), lddy=32, dh=_addr(15), lddh=32, dx=_addr(16), lddx=32,
         db=_addr(17), lddb=32, dg=_addr(18), lddg=32, dpw=_addr(19), dpb=_addr(20), dnw=_addr(21), dnb=_addr(22),
         gdt=Z.ZERO_F32, acc=0, ws=_addr(23), wsb=STEP):
    b = b or _block()
    return Z.lib().zero_norm_backward(ctypes.byref(b), stats, y, ldy, dy, lddy, dh, lddh, dx, lddx, db, lddb, dg, lddg, dpw,
                                      dpb, dnw, dnb, gdt, acc, ws, wsb, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_refusals_of_the_block(call):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(dtype=9), dict(post=3), dict(pre=-1), dict(gate_rows=0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
               dict(residual_scale=nan), dict(branch_scale=inf), dict(post=0), dict(pre=0), dict(branch=None),
               dict(branch=None, gate=None), dict(ld_branch=31), dict(ld_gate=31), dict(branch=_addr(1) + 1),
               dict(gate=_addr(2) + 1), dict(post_weight=_addr(3) + 1), dict(pre_bias=_addr(6) + 1),
               dict(branch=None, gate=None, post=0, post_weight=None, post_bias=None, pre=0, pre_weight=None, pre_bias=None)):
        assert call(_block(**kw)) == INVAL, kw
    assert call(_block(dtype=Z.ZERO_F32)) == UNSUPPORTED and call(_block(stream_dtype=Z.ZERO_F16)) == UNSUPPORTED
    assert call(_block(features=16385)) == UNSUPPORTED and call(_block(rows=(1 << 27) + 1)) == OVERFLOW
    assert call(_block(ld_branch=1 << 60)) == OVERFLOW
    L = Z.lib()
    assert L.zero_norm_forward(None, A, 1, A, 1, A, 1, None, None) == INVAL


def test_forward_refusals():
    for kw in (dict(x=None), dict(y=None), dict(h=None), dict(ldx=31), dict(ldy=31), dict(ldh=31), dict(x=_addr(10) + 2),
               dict(y=_addr(11) + 2), dict(h=_addr(12) + 1), dict(stats=_addr(13) + 2)):
        assert _fwd(**kw) == INVAL, kw
    for kw in (dict(y=_addr(10) + 4), dict(y=_addr(10), ldy=33), dict(y=_addr(1)), dict(h=_addr(10)), dict(h=_addr(5) + 10),
               dict(stats=_addr(11) + 64), dict(h=_addr(11) + 1000), dict(y=_addr(2)), dict(stats=_addr(1))):
        assert _fwd(**kw) == INVAL and "overlap" in Z.zero_last_error(), kw


def test_backward_refusals():
    for kw in (dict(stats=None), dict(y=None), dict(dh=None), dict(ldy=31), dict(lddy=31), dict(lddh=31), dict(lddx=31),
               dict(lddb=31), dict(lddg=31), dict(dx=_addr(16) + 2), dict(db=_addr(17) + 1), dict(dg=_addr(18) + 2),
               dict(dpw=_addr(19) + 2), dict(gdt=7), dict(ws=None), dict(ws=_addr(23) + 8), dict(wsb=16),
               dict(dx=None, db=None, dg=None, dpw=None, dpb=None, dnw=None, dnb=None)):
        assert _bwd(**kw) == INVAL, kw
    assert _bwd(gdt=Z.ZERO_F16) == UNSUPPORTED
    for kw in (dict(b=_block(post_bias=None)), dict(b=_block(pre_weight=None)), dict(b=_block(gate=None))):
        assert _bwd(**kw) == INVAL and "not there" in Z.zero_last_error(), kw
    for kw in (dict(dx=_addr(14) + 4), dict(dx=_addr(14), lddx=33), dict(dx=_addr(11)), dict(db=_addr(1)), dict(db=_addr(15)),
               dict(dg=_addr(2)), dict(dpw=_addr(3)), dict(dpb=_addr(19) + 64), dict(ws=_addr(16)), dict(dnb=_addr(13) + 16)):
        assert _bwd(**kw) == INVAL and "overlap" in Z.zero_last_error(), kw


def test_empty_calls_and_workspace():
    none = dict(branch=None, gate=None)
    assert _fwd(_block(rows=0, **none), x=None, y=None, h=None, stats=None) == 0
    assert _fwd(_block(features=0), x=None, y=None, h=None) == 0
    assert _bwd(_block(features=0)) == 0
    assert _bwd(_block(rows=0, **none), acc=1, stats=None, y=None, dy=None, dh=None, dx=None, db=None, dg=None) == 0
    w = Z.zero_norm_workspace_bytes
    for size in ((0, 5), (5, 0), (1 << 28, 64), (8, 20000)):
        assert w(*size) == 0
    for rows in (1, 2, 7, 255, 1001, 8192, 100_003):
        for d in (1, 64, 513, 4096, 16384):
            need = [w(rows, d, g) for g in (0, 1, 2, 3, 64, 1000, rows)]
            # five sums of one row a block: blocks of one row at least, a few for each of 256 compute units
            assert all(5 * 4 * d <= n <= 5 * 4 * (d + 4) * min(2 * rows, 700) for n in need), (rows, d, need)


def test_binding_refuses():
    x, w = torch.zeros(3, 5), torch.zeros(5)
    h = x.to(torch.bfloat16)
    for kw in (dict(h=h), dict(h=h, pre="best"), dict(h=x), dict(h=h, branch=h, gate=h, gate_rows=0)):
        with pytest.raises((TypeError, ValueError)):
            Z.zero_norm_forward(x, **kw)
    with pytest.raises((TypeError, ValueError)):
        Z.zero_norm_backward(x, w, dh=h)
    assert ctypes.sizeof(Z.ZeroNormBlock) == 120
