"""The argument checks of the losses over tokens, on the CPU: every call here is refused (or is empty) before any
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


def _call(kind, loss=_addr(8), logp=_addr(9), stats=_addr(10), dlogits=_addr(11), ldg=100, scale=1.0, upstream=None,
          n_up=4, seq_logp=_addr(13), no_in=False, no_p=False, **kw):
    f = dict(rows=4, vocab=100, logit_dtype=Z.ZERO_BF16, label_bytes=8, temperature=1.0, logits=_addr(1), ld_logits=100,
             label=_addr(2))
    pol = dict(old_logp=_addr(3), advantage=_addr(4), ref_logp=_addr(5), weight=_addr(6), clip_low=0.2, clip_high=0.2,
               kl_coef=0.1)
    pref = dict(pairs=2, seq_start=_addr(3), start_bytes=8, average=0, ref_logp=_addr(5), weight=_addr(6), beta=0.1,
                label_smoothing=0.0, margin=0.0)
    use = pref if kind == "preference" else pol
    f.update({k: v for k, v in kw.items() if k in f})
    use.update({k: v for k, v in kw.items() if k in use})
    assert all(k in f or k in use for k in kw), kw
    a = None if no_in else ctypes.byref(Z.ZeroTokenIn(**f))
    p = None if no_p else ctypes.byref(Z.ZeroPreference(**pref) if kind == "preference" else Z.ZeroPolicy(**pol))
    L = Z.lib()
    if kind == "logp":
        return L.zero_token_logp(a, logp, stats, None)
    if kind == "forward":
        return L.zero_policy_forward(a, p, loss, logp, stats, None)
    if kind == "step":
        return L.zero_policy_step(a, p, upstream, scale, loss, logp, dlogits, ldg, None)
    if kind == "preference":
        return L.zero_preference_forward(a, p, loss, logp, seq_logp, stats, None)
    return L.zero_token_backward(a, stats, upstream, n_up, scale, dlogits, ldg, None)


KINDS = ["logp", "forward", "step", "preference", "backward"]


@pytest.mark.parametrize("kind", KINDS)
def test_refusals(kind):
    nan, inf = float("nan"), float("inf")
    assert _call(kind, no_in=True) == INVAL
    for kw in (dict(logits=None), dict(label=None), dict(vocab=0), dict(label_bytes=2), dict(temperature=0.0),
               dict(temperature=nan), dict(temperature=-1.0), dict(temperature=1e30), dict(ld_logits=99),
               dict(logits=_addr(1) + 1), dict(label=_addr(2) + 4)):
        assert _call(kind, **kw) == INVAL, kw
    assert _call(kind, logit_dtype=5) == UNSUPPORTED and _call(kind, logit_dtype=-1) == UNSUPPORTED
    assert _call(kind, rows=1 << 31) == OVERFLOW and _call(kind, vocab=1 << 31, ld_logits=1 << 31) == OVERFLOW
    assert _call(kind, ld_logits=1 << 60) == OVERFLOW
    if kind in ("step", "backward"):
        for kw in (dict(dlogits=None), dict(ldg=99), dict(scale=nan), dict(scale=inf), dict(dlogits=_addr(11) + 1),
                   dict(dlogits=_addr(1) + 2), dict(dlogits=_addr(1), ldg=101), dict(dlogits=_addr(2)),
                   dict(upstream=_addr(11)), dict(upstream=_addr(12) + 2)):
            assert _call(kind, **kw) == INVAL, kw
        assert _call(kind, ldg=1 << 60) == OVERFLOW
    if kind in ("forward", "step"):
        assert _call(kind, no_p=True) == INVAL
        for kw in (dict(old_logp=None), dict(advantage=None), dict(loss=None), dict(clip_low=-0.1), dict(clip_low=1.5),
                   dict(clip_low=nan), dict(clip_high=-1.0), dict(clip_high=inf), dict(kl_coef=-1.0), dict(kl_coef=inf),
                   dict(old_logp=_addr(3) + 2), dict(weight=_addr(6) + 1), dict(loss=_addr(3)), dict(loss=_addr(1) + 4),
                   dict(logp=_addr(8)), dict(logp=_addr(5) + 4)):
            assert _call(kind, **kw) == INVAL, kw
    if kind in ("forward", "preference", "logp"):
        for kw in (dict(stats=_addr(10) + 2), dict(stats=_addr(1)), dict(stats=_addr(9) - 64)):
            assert _call(kind, **kw) == INVAL, kw
    if kind in ("forward", "preference", "backward"):
        assert _call(kind, stats=None) == INVAL
    if kind == "logp":
        assert _call(kind, logp=None) == INVAL and _call(kind, logp=_addr(2) + 8) == INVAL
    if kind == "backward":
        assert _call(kind, n_up=1 << 31) == OVERFLOW and _call(kind, stats=_addr(11)) == INVAL
    if kind == "preference":
        assert _call(kind, no_p=True) == INVAL
        for kw in (dict(seq_start=None), dict(start_bytes=2), dict(loss=None), dict(beta=nan), dict(margin=inf),
                   dict(label_smoothing=-0.1), dict(label_smoothing=1.1), dict(seq_start=_addr(3) + 4),
                   dict(loss=_addr(5) + 12), dict(seq_logp=_addr(5)), dict(seq_logp=_addr(8) + 4), dict(seq_logp=_addr(13) + 2)):
            assert _call(kind, **kw) == INVAL, kw
        assert _call(kind, pairs=(1 << 23) + 1) == OVERFLOW


def test_empty_calls():
    for kind in KINDS:
        kw = dict(pairs=0, seq_start=None, loss=None) if kind == "preference" else {}
        assert _call(kind, rows=0, logits=None, label=None, **kw) == 0, kind
    assert _call("preference", rows=0, logits=None, label=None, seq_start=None) == INVAL


def test_binding_refuses():
    x, y = torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64)
    f = torch.zeros(3)
    for call in (lambda: Z.zero_token_logp(x, y, f), lambda: Z.zero_token_logp(f, y, f),
                 lambda: Z.zero_token_logp(x.double(), y, f), lambda: Z.zero_token_logp(x, f, f),
                 lambda: Z.zero_policy_forward(x, y, f, f, f, f), lambda: Z.zero_preference_forward(x, y, f, f, f)):
        with pytest.raises((TypeError, ValueError)):
            call()
    assert ctypes.sizeof(Z.ZeroTokenIn) == 56 and ctypes.sizeof(Z.ZeroPolicy) == 48 and ctypes.sizeof(Z.ZeroPreference) == 56
