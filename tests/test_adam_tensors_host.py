"""The argument checks of the update of many tensors and of the 8-bit moments' conversions, on the CPU: every
call here is refused (or is empty) before any device work."""

import ctypes

import pytest
import torch

import zero_partition_plan_amd as Z

INVAL, OVERFLOW, UNSUPPORTED = 1, 2, 3
A = 1 << 40                                            # fake addresses, never dereferenced
STEP = 1 << 24


def _addr(k):
    return A + k * STEP


def _tensor(k=0, n=1000, bits=32, **kw):
    f = dict(n=n, param=_addr(10 * k + 1), grad=_addr(10 * k + 2), out_param=_addr(10 * k + 3), m=_addr(10 * k + 4),
             v=_addr(10 * k + 5), m_scale=None, v_scale=None, group=0, state_bits=bits)
    if bits == 8:
        f.update(m_scale=_addr(10 * k + 6), v_scale=_addr(10 * k + 7))
    f.update(kw)
    return Z.ZeroAdamTensor(**f)


def _step(*tensors, gdt=Z.ZERO_BF16, odt=Z.ZERO_BF16, groups=None, ngroups=None, gs=1.0, d_gs=None, skip=None, count=None):
    arr = (Z.ZeroAdamTensor * max(1, len(tensors)))(*tensors)
    hp = [Z.adam_hparams()] if groups is None else groups
    harr = (Z.ZeroAdamHParams * max(1, len(hp)))(*hp)
    return Z.lib().zero_adam_tensors_step(arr, len(tensors) if count is None else count, gdt, odt, harr,
                                          len(hp) if ngroups is None else ngroups, gs, d_gs, skip, None)


def _dev_t(*tensors, gs=_addr(900), table=_addr(901), ngroups=1, length=100, step=_addr(902), status=_addr(903), mode=0,
           skip=None):
    arr = (Z.ZeroAdamTensor * max(1, len(tensors)))(*tensors)
    return Z.lib().zero_adam_tensors_step_dev_t(arr, len(tensors), Z.ZERO_F32, Z.ZERO_BF16, gs, table, ngroups, length,
                                                step, status, mode, skip, None)


@pytest.mark.parametrize("bits", [8, 32])
def test_refusals(bits):
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(group=1), dict(state_bits=16),
               dict(state_bits=0), dict(param=_addr(1) + 2), dict(grad=_addr(2) + 1), dict(out_param=_addr(3) + 1)):
        assert _step(_tensor(1, bits=bits), _tensor(2, bits=bits, **kw)) == INVAL, kw
    assert _step(_tensor(n=1 << 61, bits=bits)) == OVERFLOW
    assert _step(_tensor(bits=bits), gdt=7) == INVAL and _step(_tensor(bits=bits), gdt=-1) == INVAL
    assert _step(_tensor(bits=bits), odt=Z.ZERO_F32) == UNSUPPORTED and _step(_tensor(bits=bits), odt=9) == INVAL
    assert _step(_tensor(grad=_addr(2) + 2, bits=bits), gdt=Z.ZERO_F32) == INVAL
    assert _step(_tensor(bits=bits), ngroups=0) == INVAL and _step(_tensor(bits=bits), ngroups=17) == INVAL
    assert _step(_tensor(bits=bits), groups=[Z.adam_hparams(beta1=1.0)]) == INVAL
    assert _step(_tensor(bits=bits), groups=[Z.adam_hparams(), Z.adam_hparams(lr=-1)]) == INVAL
    assert _step(_tensor(bits=bits), groups=[Z.adam_hparams(), Z.adam_hparams(wd_mode="l2")]) == INVAL
    assert _step(_tensor(bits=bits), d_gs=_addr(900) + 2) == INVAL and _step(_tensor(bits=bits), skip=_addr(900) + 1) == INVAL
    if bits == 8:
        assert _step(_tensor(bits=8, m_scale=None)) == INVAL and _step(_tensor(bits=8, v_scale=_addr(7) + 2)) == INVAL
    else:
        assert _step(_tensor(m_scale=_addr(6))) == INVAL and "32-bit" in Z.zero_last_error()
        assert _step(_tensor(m=_addr(4) + 2)) == INVAL
    arr = (Z.ZeroAdamTensor * 1)(_tensor(bits=bits))
    hp = Z.adam_hparams()
    L = Z.lib()
    assert L.zero_adam_tensors_step(None, 1, 0, 0, ctypes.byref(hp), 1, 1.0, None, None, None) == INVAL
    assert L.zero_adam_tensors_step(arr, 1, 2, 2, None, 1, 1.0, None, None, None) == INVAL
    assert L.zero_adam_tensors_step(arr, Z.ZERO_ADAM_MAX_TENSORS + 1, 2, 2, ctypes.byref(hp), 1, 1.0, None, None, None) \
        == UNSUPPORTED


@pytest.mark.parametrize("bits", [8, 32])
def test_overlaps(bits):
    """Within a tensor, between tensors in any order, the same tensor twice, and with the words of a call."""
    width = bits // 8 * 1000
    for kw in (dict(grad=_addr(1)), dict(out_param=_addr(1) + 3998), dict(m=_addr(5)), dict(v=_addr(4) + width - 4),
               dict(v=_addr(1) + 400)):
        assert _step(_tensor(bits=bits, **kw)) == INVAL and "overlap" in Z.zero_last_error(), kw
    one, two = _tensor(1, bits=bits), _tensor(2, bits=bits)
    assert _step(one, one) == INVAL and _step(two, one, _tensor(3, bits=bits), two) == INVAL
    for kw in (dict(param=_addr(11) + 3996), dict(m=_addr(14) + 100), dict(out_param=_addr(12)), dict(v=_addr(11)),
               dict(param=_addr(12) + 1996)):
        for pair in ((one, _tensor(2, bits=bits, **kw)), (_tensor(2, bits=bits, **kw), one), (two, _tensor(0, n=0), one, _tensor(3, bits=bits, **kw))):
            assert _step(*pair) == INVAL and "overlap" in Z.zero_last_error(), kw
    assert _step(_tensor(bits=bits), d_gs=_addr(1) + 8) == INVAL and _step(_tensor(bits=bits), skip=_addr(4)) == INVAL
    if bits == 8:
        assert _step(_tensor(bits=8, m_scale=_addr(7) + 12)) == INVAL
        assert _step(one, _tensor(2, bits=8, v_scale=_addr(16))) == INVAL


def test_empty_calls():
    assert _step() == 0 and _step(count=0) == 0
    assert _step(_tensor(n=0, param=None, grad=None, m=None, v=None, out_param=None), _tensor(n=0, bits=8)) == 0
    assert _step(ngroups=0) == INVAL and _step(groups=[Z.adam_hparams(lr=float("nan"))]) == INVAL


def test_device_step_refusals():
    for kw in (dict(gs=None), dict(table=None), dict(step=None), dict(status=None), dict(length=0), dict(ngroups=0),
               dict(ngroups=17), dict(mode=2), dict(step=_addr(902) + 4), dict(status=_addr(903) + 2), dict(table=_addr(901) + 2),
               dict(step=_addr(901) + 8), dict(status=_addr(1)), dict(step=_addr(2)), dict(status=_addr(902) + 4),
               dict(table=_addr(4)), dict(skip=_addr(903)), dict(gs=_addr(902))):
        assert _dev_t(_tensor(), **kw) == INVAL, kw


def test_state_conversions_refuse():
    L = Z.lib()
    ok = dict(codes=_addr(1), scale=_addr(2), n=1000, moment=1, values=_addr(3))
    for kw in (dict(codes=None), dict(scale=None), dict(values=None), dict(moment=0), dict(moment=3), dict(scale=_addr(2) + 1),
               dict(values=_addr(3) + 2), dict(codes=_addr(3) + 3999), dict(scale=_addr(1) + 996), dict(values=_addr(2) + 12)):
        f = {**ok, **kw}
        assert L.zero_adam_state_values(f["codes"], f["scale"], f["n"], f["moment"], f["values"], None) == INVAL, kw
        assert L.zero_adam_state_codes(f["values"], f["n"], f["moment"], f["codes"], f["scale"], None) == INVAL, kw
    assert L.zero_adam_state_values(_addr(1), _addr(2), 1 << 61, 1, _addr(3), None) == OVERFLOW
    assert L.zero_adam_state_values(None, None, 0, 2, None, None) == 0
    assert L.zero_adam_state_codes(None, 0, 1, None, None, None) == 0


def test_binding_refuses_what_is_no_device_tensor():
    x = torch.zeros(8)
    with pytest.raises((TypeError, ValueError)):
        Z.adam_tensor(x, x, x, x)
    with pytest.raises(TypeError):
        Z.adam_tensor(x, x, x.to(torch.int8), x.to(torch.uint8))
    with pytest.raises(TypeError):
        Z.adam_tensor(x, x, x, x, m_scale=x)
    with pytest.raises(ValueError):
        Z.adam_state(x, 16)
    with pytest.raises(TypeError):
        Z.zero_adam_state_values(x, x, x)
    s = Z.adam_state(torch.zeros(3, 200), 8)
    assert s["m"].shape == (3, 200) and s["m_scale"].shape == (3,) and s["v"].dtype is torch.uint8
    assert ctypes.sizeof(Z.ZeroAdamTensor) == 72
