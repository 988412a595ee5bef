"""The linear layer's and the distillation loss's argument checks, on the CPU: every call here is
refused (or is empty) before any device work."""

import ctypes

import pytest
import torch

import zero_partition_plan_amd as Z

INVAL, OVERFLOW, UNSUPPORTED = 1, 2, 3
A = 1 << 40                                            # a fake address, never dereferenced
STEP = 1 << 28


def _addr(k):
    return A + k * STEP


def _shape(rows=8, k=32, n=16, dtype=Z.ZERO_BF16, act=0):
    return Z.ZeroLinearShape(rows, k, n, dtype, act)


def _fwd(s=None, x=_addr(1), ldx=32, w=_addr(2), b=None, r=None, ldr=16, pre=None, ldp=16, y=_addr(3),
         ldy=16, ws=_addr(20), wsb=STEP):
    s = s or _shape()
    return Z.lib().zero_linear_forward(ctypes.byref(s), x, ldx, w, b, r, ldr, pre, ldp, y, ldy, ws, wsb, None)


def _bwd(s=None, dy=_addr(1), lddy=16, x=_addr(2), ldx=32, w=_addr(3), pre=_addr(4), ldp=16, dz=_addr(5),
         lddz=16, dx=_addr(6), lddx=32, dw=_addr(7), db=_addr(8), gdt=Z.ZERO_BF16, acc=0, ws=_addr(20),
         wsb=STEP):
    s = s or _shape(act=4)
    return Z.lib().zero_linear_backward(ctypes.byref(s), dy, lddy, x, ldx, w, pre, ldp, dz, lddz, dx, lddx,
                                        dw, db, gdt, acc, ws, wsb, None)


def test_linear_forward_refusals():
    assert Z.lib().zero_linear_forward(None, A, 1, A, None, None, 0, None, 0, A, 1, None, 0, None) == INVAL
    assert _fwd(_shape(dtype=7)) == INVAL and _fwd(_shape(dtype=Z.ZERO_F32)) == UNSUPPORTED
    assert _fwd(_shape(act=5)) == INVAL and _fwd(_shape(act=-1)) == INVAL
    assert _fwd(_shape(rows=1 << 31)) == OVERFLOW and _fwd(_shape(k=1 << 40)) == OVERFLOW
    assert _fwd(x=None) == INVAL and _fwd(w=None) == INVAL and _fwd(y=None) == INVAL
    for kw in (dict(ldx=31), dict(ldy=15), dict(r=_addr(5), ldr=15), dict(pre=_addr(5), ldp=3)):
        assert _fwd(**kw) == INVAL and "leading dimension" in Z.zero_last_error(), kw
    for kw in (dict(x=_addr(1) + 1), dict(w=_addr(2) + 1), dict(b=_addr(4) + 1), dict(y=_addr(3) + 3)):
        assert _fwd(**kw) == INVAL and "not aligned" in Z.zero_last_error(), kw
    assert _fwd(ldx=1 << 61) == OVERFLOW


def test_linear_forward_overlaps():
    y = _addr(3)
    for kw in (dict(x=y + 2), dict(w=y + 40), dict(b=y + 14), dict(pre=y), dict(pre=y + 8 * 32 - 2),
               dict(r=y + 2), dict(r=y, ldr=17), dict(y=_addr(1) - 2)):
        assert _fwd(**kw) == INVAL and "overlap" in Z.zero_last_error(), kw
    # slices of one buffer of 64 columns: y in columns 16..31 meets x in columns 0..31, and a
    # residual whose columns wrap into the next row's
    assert _fwd(x=y - 32, ldx=64, y=y, ldy=64) == INVAL
    assert _fwd(r=y + 2 * 50, ldr=64, ldy=64) == INVAL


def test_linear_backward_refusals():
    assert _bwd(_shape(act=9)) == INVAL and _bwd(_shape(dtype=Z.ZERO_F32, act=1)) == UNSUPPORTED
    assert _bwd(gdt=Z.ZERO_F16) == UNSUPPORTED and _bwd(gdt=8) == INVAL
    assert _bwd(dy=None) == INVAL and _bwd(x=None) == INVAL and _bwd(w=None) == INVAL
    assert _bwd(pre=None) == INVAL and _bwd(dz=None) == INVAL
    assert _bwd(_shape(), dx=None, dw=None, db=None) == INVAL and "no output" in Z.zero_last_error()
    for kw in (dict(lddy=15), dict(ldx=31), dict(ldp=15), dict(lddz=15), dict(lddx=31)):
        assert _bwd(**kw) == INVAL and "leading dimension" in Z.zero_last_error(), kw
    for kw in (dict(dw=_addr(7) + 1), dict(db=_addr(8) + 2, gdt=Z.ZERO_F32, dw=_addr(7)),
               dict(dw=_addr(7) + 2, gdt=Z.ZERO_F32)):
        assert _bwd(**kw) == INVAL and "not aligned" in Z.zero_last_error(), kw
    for kw in (dict(dx=_addr(2)), dict(dx=_addr(1)), dict(dw=_addr(3)), dict(db=_addr(7) + 30), dict(dz=_addr(2) + 4),
               dict(dz=_addr(1), lddz=17), dict(dz=_addr(4) + 2), dict(dw=_addr(6) + 64)):
        assert _bwd(**kw) == INVAL and "overlap" in Z.zero_last_error(), kw


def test_linear_workspace_is_checked():
    """A size that needs a workspace refuses a missing, short, misaligned or overlapping one."""
    m, k, n = 512, 8192, 64
    for back, call in ((False, _fwd), (True, _bwd)):
        need = Z.zero_linear_workspace_bytes(m, k, n, back)
        s = _shape(m, k, n, act=4 if back else 0)
        ld = dict(ldx=k, lddy=n, ldp=n, lddz=n, lddx=k) if back else dict(ldx=k, ldy=n)
        if need:
            for kw in (dict(ws=None), dict(wsb=need - 1), dict(ws=_addr(20) + 8), dict(ws=_addr(2))):
                assert call(s, wsb=kw.pop("wsb", need), **ld, **kw) == INVAL, kw
    for m, k, n in ((0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0), (1, 1, 1)):
        assert Z.zero_linear_workspace_bytes(m, k, n) < 1 << 20 and Z.zero_linear_workspace_bytes(m, k, n, True) < 1 << 20
    for big in ((1 << 31, 1, 1), (1, 1 << 33, 1), (1, 1, 1 << 63)):
        assert Z.zero_linear_workspace_bytes(*big) == 0 == Z.zero_linear_workspace_bytes(*big, True)


def test_linear_empty_calls():
    assert _fwd(_shape(rows=0), x=None, w=None, y=None) == 0
    assert _fwd(_shape(n=0), x=None, w=None, y=None) == 0
    assert _bwd(_shape(rows=0, n=0), dy=None, x=None, w=None, pre=None, dz=None) == 0
    assert _bwd(_shape(rows=0), acc=1, dy=None, x=None, w=None, pre=None, dz=None) == 0


def _distill(kind="step", loss=_addr(8), stats=_addr(9), dlogits=_addr(10), ldg=100, scale=1.0, upstream=None, **kw):
    f = dict(rows=4, vocab=100, topk=5, logit_dtype=Z.ZERO_BF16, teacher_dtype=Z.ZERO_F32, index_bytes=4,
             temperature=1.0, logits=_addr(1), ld_logits=100, top_index=_addr(2), top_logits=_addr(3), ld_top=5,
             tail=None, weight=None)
    f.update(kw)
    a = Z.ZeroDistillIn(**f)
    L = Z.lib()
    if kind == "forward":
        return L.zero_distill_forward(ctypes.byref(a), loss, stats, None)
    if kind == "backward":
        return L.zero_distill_backward(ctypes.byref(a), stats, upstream, scale, dlogits, ldg, None)
    return L.zero_distill_step(ctypes.byref(a), upstream, scale, loss, dlogits, ldg, None)


@pytest.mark.parametrize("kind", ["forward", "backward", "step"])
def test_distill_refusals(kind):
    for kw in (dict(logits=None), dict(top_index=None), dict(top_logits=None), dict(vocab=0, ld_logits=0),
               dict(topk=0), dict(index_bytes=2), dict(temperature=0.0), dict(temperature=float("nan")),
               dict(temperature=-1.0), dict(temperature=1e30), dict(ld_logits=99), dict(ld_top=4),
               dict(logits=_addr(1) + 1), dict(top_logits=_addr(3) + 2), dict(top_index=_addr(2) + 4, index_bytes=8),
               dict(tail=_addr(4) + 2), dict(weight=_addr(4) + 1)):
        assert _distill(kind, **kw) == INVAL, kw
    for kw in (dict(logit_dtype=3), dict(teacher_dtype=-1), dict(topk=1025, ld_top=1025),
               dict(vocab=Z.ZERO_DISTILL_MAX_VOCAB + 1, ld_logits=1 << 20, ldg=1 << 20)):
        assert _distill(kind, **kw) == UNSUPPORTED, kw
    assert _distill(kind, rows=1 << 31) == OVERFLOW and _distill(kind, ld_logits=1 << 62) == OVERFLOW
    assert _distill(kind, rows=0, logits=None, top_index=None, top_logits=None) == 0


def test_distill_outputs_checked():
    assert _distill("forward", loss=None) == INVAL and _distill("forward", stats=None) == INVAL
    assert _distill("backward", stats=None) == INVAL and _distill("backward", dlogits=None) == INVAL
    assert _distill("step", loss=None) == INVAL and _distill("step", dlogits=None) == INVAL
    for kind in ("backward", "step"):
        assert _distill(kind, ldg=99) == INVAL and _distill(kind, scale=float("inf")) == INVAL
        assert _distill(kind, dlogits=_addr(10) + 1) == INVAL
        for kw in (dict(dlogits=_addr(1) + 2), dict(dlogits=_addr(1), ldg=101), dict(dlogits=_addr(2) + 8),
                   dict(upstream=_addr(10) + 4), dict(weight=_addr(10) + 20)):
            assert _distill(kind, **kw) == INVAL and "overlap" in Z.zero_last_error(), kw
    assert _distill("forward", stats=_addr(8) + 4) == INVAL and _distill("step", loss=_addr(10)) == INVAL
    assert _distill("step", loss=_addr(1) + 8) == INVAL and _distill("backward", stats=_addr(10) + 8) == INVAL


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    y = torch.zeros(4, 6, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        Z.zero_linear_forward(x, w, y)                              # host memory
    with pytest.raises(TypeError):
        Z.zero_linear_forward(x, w.float(), y)
    with pytest.raises(ValueError):
        Z.zero_linear_forward(x, w, y, act="tanh")
    with pytest.raises(TypeError):
        Z.zero_linear_forward(x[0], w, y)
    with pytest.raises(ValueError):
        Z.zero_linear_backward(y[:, :5], x, w, dx=x)
    z = torch.zeros(4, 100)
    idx, top = torch.zeros(4, 5, dtype=torch.int32), torch.zeros(4, 5)
    with pytest.raises(TypeError):
        Z.zero_distill_step(z, idx, top, 1.0, torch.zeros(4), z)
    with pytest.raises(TypeError):
        Z.zero_distill_step(z, idx.short(), top, 1.0, torch.zeros(4), z)
    with pytest.raises(ValueError):
        Z.zero_distill_step(z, idx, top[:, :4], 1.0, torch.zeros(4), z)


def test_header_constants_match_binding():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "zero_shard.h")).read()
    for name in ("ZERO_DISTILL_MAX_TOPK", "ZERO_DISTILL_MAX_VOCAB"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(Z, name)
    for name in ("NONE", "RELU", "GELU", "GELU_TANH", "SILU"):
        assert int(re.search(rf"ZERO_ACT_{name} = (\d)", text).group(1)) == getattr(Z, f"ZERO_ACT_{name}")
    assert ctypes.sizeof(Z.ZeroLinearShape) == 32 and ctypes.sizeof(Z.ZeroDistillIn) == 96


def test_sizes_past_the_launch_limit_are_refused():
    """A grid dimension holds fewer than 2^32 threads: the layer refuses what would need more."""
    assert _fwd(_shape(rows=(1 << 27) + 1)) == OVERFLOW
    assert _fwd(_shape(n=(1 << 27) + 1)) == OVERFLOW and _fwd(_shape(k=(1 << 27) + 1)) == OVERFLOW
    assert Z.zero_linear_workspace_bytes((1 << 27) + 1, 8, 8) == 0


def test_binding_takes_none_for_what_a_backward_does_not_read():
    """None passes the binding's own checks of x and weight: what refuses these calls is the host memory
    of dy, and a tensor of another shape or kind is still refused for itself."""
    dy = torch.zeros(4, 6, dtype=torch.bfloat16)
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    for kw in (dict(x=x, weight=None, dweight=w), dict(x=None, weight=w, dx=x), dict(x=None, weight=None, dbias=dy[0]),
               dict(x=None, weight=None, act="silu", pre=dy, dz=dy)):
        with pytest.raises(TypeError, match="dy must be a device tensor"):
            Z.zero_linear_backward(dy, **kw)
    for kw in (dict(x=x[0], weight=None, dweight=w), dict(x=None, weight=w[0], dx=x), dict(x=None, weight=None, dx=[1])):
        with pytest.raises(TypeError, match="2-D"):
            Z.zero_linear_backward(dy, **kw)
    with pytest.raises(TypeError, match="dy must be a 2-D"):
        Z.zero_linear_backward(None, x, w)
