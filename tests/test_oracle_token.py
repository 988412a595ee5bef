"""The oracle of the losses over tokens against torch's automatic gradients and central differences."""

import numpy as np
import pytest
import torch

import oracle as O

K = O.token


def _rows(seed, R=7, V=11):
    rng = np.random.default_rng(seed)
    label = rng.integers(0, V, R)
    label[2] = -1
    return rng, rng.standard_normal((R, V)) * 2, label


@pytest.mark.parametrize("T", [1.0, 0.5, 3.0])
def test_log_probability(T):
    rng, z, label = _rows(1)
    l, g = K.softmax(z, label, T)
    t = torch.tensor(z, requires_grad=True)
    on = label >= 0
    want = torch.log_softmax(t / T, 1)[torch.arange(7), torch.tensor(label).clamp(min=0)] * torch.tensor(on)
    want.sum().backward()
    assert np.abs(l - want.detach().numpy()).max() <= 1e-13 and np.abs(g - t.grad.numpy()).max() <= 1e-13


@pytest.mark.parametrize("kl", [0.0, 0.3])
@pytest.mark.parametrize("clip", [(0.2, 0.2), (0.1, 0.4), (1.0, 0.0)])
def test_policy(clip, kl):
    rng, z, label = _rows(2, 40)
    l0, _ = K.softmax(z, label)
    old, ref = l0 + rng.normal(0, 0.3, 40), l0 + rng.normal(0, 0.3, 40)
    adv, w = rng.standard_normal(40), rng.uniform(0.5, 2, 40)
    adv[5], w[6] = 0.0, 0.0
    loss, l, g = K.policy_rows(z, label, old, adv, clip, ref, kl, w, 1.3)
    t = torch.tensor(z, requires_grad=True)
    on = torch.tensor((label >= 0) & (w != 0))
    lt = torch.log_softmax(t / 1.3, 1)[torch.arange(40), torch.tensor(label).clamp(min=0)]
    ratio, a = (lt - torch.tensor(old)).exp(), torch.tensor(adv)
    d = torch.tensor(ref) - lt
    want = -torch.minimum(ratio * a, ratio.clamp(1 - clip[0], 1 + clip[1]) * a) + kl * (d.exp() - 1 - d)
    want = torch.where(on, want * torch.tensor(w), torch.zeros_like(want))
    want.sum().backward()
    assert np.abs(loss - want.detach().numpy()).max() <= 1e-12
    assert np.abs(l - np.where(on, lt.detach().numpy(), 0)).max() <= 1e-12
    assert np.abs(g - t.grad.numpy()).max() <= 1e-12
    assert (g[6] == 0).all() and (g[2] == 0).all()


def test_the_kl_term_keeps_its_digits():
    from fractions import Fraction
    for d in (1e-9, -1e-6, 1e-3, -0.3, 0.49, 0.51, -2.0):
        x, total, term = Fraction(d), Fraction(0), Fraction(1)
        for k in range(1, 40):
            term = term * x / k
            total += term if k >= 2 else 0
        assert abs(K._expm1_less(d) - float(total)) <= 4e-16 * max(float(total), abs(d) if abs(d) > 0.5 else 0.0)


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("smoothing", [0.0, 0.2, 1.0])
def test_preference(smoothing, average):
    rng = np.random.default_rng(3)
    start = np.array([0, 4, 9, 9, 15, 18, 20])
    on = rng.random(22) < 0.8
    l = np.where(on, -rng.random(22) * 3, 0.0)
    ref, w = rng.standard_normal(6), np.array([1.0, 0.5, 0.0])
    loss, seq, slope = K.preference(l, on, start, 0.7, ref, w, smoothing, 0.1, average)
    t = torch.tensor(l, requires_grad=True)
    n = [max(1, int(on[a:b].sum())) if average else 1 for a, b in zip(start[:-1], start[1:])]
    s = torch.stack([t[a:b].sum() / k for (a, b), k in zip(zip(start[:-1], start[1:]), n)])
    gap = s - torch.tensor(ref)
    x = 0.7 * (gap[0::2] - gap[1::2]) - 0.1
    sp = torch.nn.functional.softplus
    want = torch.tensor(w) * ((1 - smoothing) * sp(-x) + smoothing * sp(x))
    want.sum().backward()
    assert np.abs(loss - want.detach().numpy()).max() <= 1e-13 and np.abs(seq - s.detach().numpy()).max() <= 1e-13
    assert np.abs(slope - np.where(on, t.grad.numpy(), 0)).max() <= 1e-13 and (slope[20:] == 0).all()


def test_differences():
    """Central differences of the whole preference loss in the logits."""
    rng, z, label = _rows(4, 9, 5)
    start = np.array([0, 3, 6, 7, 9])

    def value(z):
        l, _ = K.softmax(z, label)
        return K.preference(l, label >= 0, start, 0.5, None, None, 0.1)[0].sum()

    l, g = K.softmax(z, label)
    slope = K.preference(l, label >= 0, start, 0.5, None, None, 0.1)[2]
    h = 1e-5
    for r in range(9):
        for v in range(5):
            up, down = z.copy(), z.copy()
            up[r, v] += h
            down[r, v] -= h
            assert abs((value(up) - value(down)) / (2 * h) - slope[r] * g[r, v]) <= 1e-9


def test_rows_without_a_softmax():
    z = np.zeros((5, 4))
    z[0, 1], z[1, 2], z[2] = np.nan, np.inf, -np.inf
    z[3, :3] = -np.inf
    l, g = K.softmax(z, [0, 0, 0, 3, 0])
    assert np.isnan(l[:3]).all() and np.isnan(g[:3]).all() and l[3] == 0 and (g[3] == 0).all() and l[4] == -np.log(4)
