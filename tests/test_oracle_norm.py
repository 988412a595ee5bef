"""The oracle of the block boundaries against torch's layers, its automatic gradients and central differences."""

import numpy as np
import pytest
import torch

import oracle as O

N = O.norm


def _torch_norm(v, kind, w, b, eps):
    if kind == "none":
        return v
    if kind == "layer":
        return torch.nn.functional.layer_norm(v, v.shape[1:], w, b, eps)
    x = v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + eps)
    x = x if w is None else x * w
    return x if b is None else x + b


def _case(seed, R, n, gate_rows, post, pre, gated):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.tensor(rng.standard_normal(s), requires_grad=True)  # noqa: E731
    c = {"x": t(R, n), "branch": t(R, n)}
    c["gate"] = t(-(-R // gate_rows), n) if gated else None
    for k, kind in (("post", post), ("pre", pre)):
        c[k + "_w"], c[k + "_b"] = (t(n), t(n)) if kind != "none" else (None, None)
    return rng, c


@pytest.mark.parametrize("gate_rows", [1, 3, 8])
@pytest.mark.parametrize("pre", N.KINDS)
@pytest.mark.parametrize("post", N.KINDS)
def test_against_automatic_gradients(post, pre, gate_rows):
    R, n, eps, a, s = 8, 13, 1e-3, 0.7, 1.3
    rng, c = _case(1, R, n, gate_rows, post, pre, True)
    g = c["gate"][torch.arange(R) // gate_rows]
    y = a * c["x"] + s * g * _torch_norm(c["branch"], post, c["post_w"], c["post_b"], eps)
    y.retain_grad()
    h = _torch_norm(y, pre, c["pre_w"], c["pre_b"], eps)
    dy, dh = torch.tensor(rng.standard_normal((R, n))), torch.tensor(rng.standard_normal((R, n)))
    ((y * dy).sum() + ((h * dh).sum() if pre != "none" else 0.0)).backward()
    v = {k: None if t is None else t.detach().numpy() for k, t in c.items()}
    got_y = N.forward_sum(v["x"], v["branch"], v["gate"], gate_rows, post, v["post_w"], v["post_b"], eps, a, s)
    assert np.abs(got_y - y.detach().numpy()).max() <= 1e-12
    assert np.abs(N.forward_next(got_y, pre, v["pre_w"], v["pre_b"], eps) - h.detach().numpy()).max() <= 1e-12
    got = N.backward(got_y, dy.numpy(), dh.numpy(), v["branch"], v["gate"], gate_rows, post, v["post_w"], v["post_b"], pre,
                     v["pre_w"], eps, a, s)
    for k, t in (("dx", "x"), ("dbranch", "branch"), ("dgate", "gate"), ("dpost_weight", "post_w"), ("dpost_bias", "post_b"),
                 ("dpre_weight", "pre_w"), ("dpre_bias", "pre_b")):
        if c[t] is not None:
            assert np.abs(got[k] - c[t].grad.numpy()).max() <= 1e-11, k


def test_differences():
    rng, c = _case(2, 3, 5, 2, "layer", "rms", True)
    v = {k: t.detach().numpy().copy() for k, t in c.items()}
    dy, dh = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def value(v):
        y = N.forward_sum(v["x"], v["branch"], v["gate"], 2, "layer", v["post_w"], v["post_b"], 1e-2, 0.9, 1.1)
        return (y * dy).sum() + (N.forward_next(y, "rms", v["pre_w"], v["pre_b"], 1e-2) * dh).sum()

    y = N.forward_sum(v["x"], v["branch"], v["gate"], 2, "layer", v["post_w"], v["post_b"], 1e-2, 0.9, 1.1)
    got = N.backward(y, dy, dh, v["branch"], v["gate"], 2, "layer", v["post_w"], v["post_b"], "rms", v["pre_w"], 1e-2, 0.9, 1.1)
    for k, t in (("dx", "x"), ("dbranch", "branch"), ("dgate", "gate"), ("dpost_weight", "post_w"), ("dpre_bias", "pre_b")):
        for i in range(v[t].size):
            was = v[t].flat[i]
            v[t].flat[i] = was + 1e-5
            up = value(v)
            v[t].flat[i] = was - 1e-5
            down = value(v)
            v[t].flat[i] = was
            assert abs((up - down) / 2e-5 - got[k].flat[i]) <= 1e-8, (k, i)


def test_without_a_branch_or_a_stream_gradient():
    rng = np.random.default_rng(3)
    x, dh, w = rng.standard_normal((4, 6)), rng.standard_normal((4, 6)), rng.standard_normal(6)
    t = torch.tensor(x, requires_grad=True)
    (_torch_norm(t, "rms", torch.tensor(w), None, 1e-4) * torch.tensor(dh)).sum().backward()
    assert (N.forward_sum(x, None, None, 1, "none", None, None, 1e-4, 0.5, 2.0) == x).all()
    got = N.backward(x, None, dh, None, None, 1, "none", None, None, "rms", w, 1e-4, 0.5, 2.0)
    assert np.abs(got["dx"] - t.grad.numpy()).max() <= 1e-13 and "dbranch" not in got
