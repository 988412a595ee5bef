"""Pins of the oracle's linear layer and distillation loss: torch's own operations and automatic
gradients in fp64, and central differences."""

import numpy as np
import pytest
import torch

import oracle as O

L = O.layer


def _t(a):
    return torch.from_numpy(np.asarray(a)).double()


@pytest.mark.parametrize("kind", L.ACTS)
def test_activations_match_torch_and_differences(kind):
    z = np.concatenate([np.linspace(-9, 9, 241), [-40.0, 40.0, -0.5, 0.5]]) + 1e-3
    f = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
         "silu": torch.nn.functional.silu}[kind]
    t = _t(z).requires_grad_()
    y = f(t)
    y.sum().backward()
    assert np.allclose(L.act(z, kind), y.detach().numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(L.act_slope(z, kind), t.grad.numpy(), rtol=1e-10, atol=1e-13)
    h = 1e-5
    diff = (L.act(z + h, kind) - L.act(z - h, kind)) / (2 * h)
    assert np.allclose(L.act_slope(z, kind), diff, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("kind", L.ACTS)
def test_linear_matches_autograd(kind):
    rng = np.random.default_rng(3)
    x, w, b, r, dy = (rng.standard_normal(s) for s in ((5, 7), (4, 7), (4,), (5, 4), (5, 4)))
    tx, tw, tb, tr = (_t(a).requires_grad_() for a in (x, w, b, r))
    z = torch.nn.functional.linear(tx, tw, tb)
    f = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
         "silu": torch.nn.functional.silu}[kind]
    y = f(z) + tr
    y.backward(_t(dy))
    got_y, got_z = L.linear_forward(x, w, b, r, kind)
    assert np.allclose(got_y, y.detach().numpy(), rtol=1e-12) and np.allclose(got_z, z.detach().numpy())
    dx, dw, db = L.linear_backward(dy * L.act_slope(got_z, kind), x, w)
    for got, want in ((dx, tx.grad), (dw, tw.grad), (db, tb.grad), (dy, tr.grad)):
        assert np.allclose(got, want.numpy(), rtol=1e-11, atol=1e-13)


def _case(seed, R=6, V=23, K=5):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((R, V)) * 2
    idx = np.stack([rng.permutation(V)[:K] for _ in range(R)])
    return rng, z, idx, rng.standard_normal((R, K)) * 2


@pytest.mark.parametrize("T", [1.0, 2.5])
@pytest.mark.parametrize("with_tail", [False, True])
def test_distill_matches_kl_div_of_the_whole_teacher(T, with_tail):
    """The teacher written out as a distribution: without a tail p is the softmax of the listed
    entries; with one, torch's kl_div over the listed entries and one bucket of the rest."""
    rng, z, idx, top = _case(1)
    R, V = z.shape
    w = rng.uniform(0.2, 2.0, R)
    tail = rng.standard_normal(R) if with_tail else None
    tz = _t(z).requires_grad_()
    lq = torch.log_softmax(tz / T, 1)
    cols = torch.from_numpy(idx)
    parts = _t(top) / T
    listed = lq.gather(1, cols)
    if with_tail:
        parts = torch.cat([parts, _t(tail)[:, None]], 1)
        inside = torch.zeros(R, V, dtype=torch.bool).scatter_(1, cols, True)
        listed = torch.cat([listed, torch.logsumexp(lq.masked_fill(inside, -np.inf), 1)[:, None]], 1)
    kl = torch.nn.functional.kl_div(listed, torch.log_softmax(parts, 1), log_target=True,
                                    reduction="none").sum(1) * _t(w)
    kl.sum().backward()
    loss, grad = L.distill(z, idx, top, T, tail, w)
    assert np.allclose(loss, kl.detach().numpy(), rtol=1e-11)
    assert np.allclose(grad, tz.grad.numpy(), rtol=1e-9, atol=1e-13)


@pytest.mark.parametrize("with_tail", [False, True])
def test_distill_gradient_by_differences(with_tail):
    rng, z, idx, top = _case(2)
    idx[0, 3] = idx[0, 1]                              # one index twice
    idx[1, 2:] = -1                                    # a short row
    top[2, 0] = -np.inf
    tail = rng.standard_normal(len(z)) if with_tail else None
    _, grad = L.distill(z, idx, top, 1.7, tail)
    h = 1e-6
    for v in range(z.shape[1]):
        e = np.zeros_like(z)
        e[:, v] = h
        diff = (L.distill(z + e, idx, top, 1.7, tail)[0] - L.distill(z - e, idx, top, 1.7, tail)[0]) / (2 * h)
        assert np.allclose(grad[:, v], diff, rtol=1e-6, atol=1e-8), v


def test_one_entry_is_the_cross_entropy_of_a_label():
    rng, z, _, _ = _case(4)
    label = rng.integers(0, z.shape[1], len(z))
    loss, grad = L.distill(z, label[:, None], np.full((len(z), 1), 3.0), 1.0)
    t = _t(z).requires_grad_()
    ce = torch.nn.functional.cross_entropy(t, torch.from_numpy(label), reduction="none")
    ce.sum().backward()
    assert np.allclose(loss, ce.detach().numpy(), rtol=1e-12) and np.allclose(grad, t.grad.numpy(), rtol=1e-10)


def test_rows_without_teacher_or_weight_are_zero():
    _, z, idx, top = _case(5)
    w = np.ones(len(z))
    w[0], idx[1] = 0.0, -1
    top[2] = -np.inf
    z[0, 3] = np.nan                                    # not read
    loss, grad = L.distill(z, idx, top, 1.0, None, w)
    assert (loss[:3] == 0).all() and (grad[:3] == 0).all() and (loss[3:] > 0).all()


@pytest.mark.parametrize("kind", [k for k in L.ACTS if k != "none"])
def test_activations_keep_their_digits_far_out(kind):
    """Relative accuracy where a gate is small: scipy's normal distribution and logistic function, and the
    slopes by the formula in their terms (an exponential of e is off by |e| roundings, at most 300 here)."""
    from scipy import special
    z = np.concatenate([np.linspace(-12, 12, 481), [-30.0, 30.0]]) + 1e-3
    c, a = np.sqrt(2 / np.pi), 0.044715
    u = 2 * c * (z + a * z ** 3)
    phi = np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    y, first, second = {
        "relu": (np.maximum(z, 0), (z > 0) * 1.0, 0 * z),
        "gelu": (z * special.ndtr(z), special.ndtr(z), z * phi),
        "gelu_tanh": (z * special.expit(u), special.expit(u),
                      z * special.expit(u) * special.expit(-u) * 2 * c * (1 + 3 * a * z * z)),
        "silu": (z * special.expit(z), special.expit(z), z * special.expit(z) * special.expit(-z)),
    }[kind]
    assert (np.abs(L.act(z, kind) - y) <= 1e-12 * np.abs(y)).all()
    assert (np.abs(L.act_slope(z, kind) - (first + second)) <= 1e-12 * (first + np.abs(second))).all()


@pytest.mark.parametrize("kind", [k for k in L.ACTS if k != "none"])
def test_slopes_far_out_are_their_limits(kind):
    z = np.array([-np.inf, -3e38, -1e20, -1e4, 1e4, 1e20, 3e38, np.inf, np.nan])
    got = L.act_slope(z, kind)
    assert np.array_equal(got[:8], [0, 0, 0, 0, 1, 1, 1, 1]) and (kind == "relu" or np.isnan(got[8]))
