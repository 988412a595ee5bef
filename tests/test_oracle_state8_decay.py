"""What 8-bit moments keep over many steps. Rounding to the nearest index undoes a change of less than half an index, and
a moment whose gradient stops shrinks by a factor f a step (m by beta1, the root of v by sqrt(beta2)): index q has left for
q - 1 only if f*q^2 < (q - 1/2)^2, that is 1 - f > 1/q - 1/(4 q^2). So a share of its block's largest above (q/T)^2 with
q = 1/(1 - f) is forgotten, and one below it is kept for as long as another element keeps the largest up."""

import numpy as np
import pytest

import oracle as O

S = O.state8
F32 = np.float32


def _one_kept_up(top, f, steps):
    """A block whose largest element is kept up by its gradient and whose others, one of each index 1 to top - 1, have none:
    their indices after `steps` steps of factor f in fp32."""
    codes = np.zeros(256, np.int8 if top == 127 else np.uint8)
    codes[:top] = [top, *range(1, top)]
    state = (codes, np.ones(1, F32))
    for _ in range(steps):
        x = S.decode(*state, top)
        x[1:] *= F32(f)
        x[0] = 1.0
        state = S.encode(x, top)
    return state[0][1:top].astype(int)


@pytest.mark.parametrize("top,f", [(127, 0.9), (127, 0.5), (255, 0.95 ** 0.5), (255, 0.99 ** 0.5), (255, 0.999 ** 0.5)])
def test_indices_under_the_limit_stay_and_those_above_fall_to_it(top, f):
    q = np.arange(1, top)
    limit = int(q[f * q ** 2 > (q - 0.5) ** 2].max())
    assert limit == q[-1] or -0.25 - 1e-9 <= 1.0 / (1.0 - f) - limit <= 1.25 + 1e-9   # q = 1/(1 - f) - 1/4 or a little over
    assert np.array_equal(_one_kept_up(top, f, 2000), np.minimum(q, limit))


def _gradients(rng, n, steps, kind, at):
    half = rng.random(n) < 0.5
    for t in range(1, steps + 1):
        g = rng.standard_normal(n).astype(F32) * F32(1e-3)
        yield np.where(half & (t > at), g * F32({"steady": 1.0, "fall": 0.1, "stop": 0.0}[kind]), g), half


@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("kind", ["steady", "fall", "stop"])
def test_against_moments_in_32_bits_over_thousands_of_steps(kind, beta2):
    """Gradients of one size, half of which fall tenfold or stop after 500 steps, with the root's and m's ratio to those in
    32 bits 2000 steps later: steady ones stay near, fallen ones only where beta2 forgets in an index, stopped ones not."""
    rng, nb, steps = np.random.default_rng(3), 4, 2500
    n = 256 * nb
    m8, v8 = (np.zeros(n, np.int8), np.zeros(nb, F32)), (np.zeros(n, np.uint8), np.zeros(nb, F32))
    v = np.zeros(n)
    b1, b2 = F32(0.9), F32(beta2)
    for g, half in _gradients(rng, n, steps, kind, 500):
        w = S.decode(*v8, 255)
        v8 = S.encode(S.roots(b2 * (w * w) + F32(1 - beta2) * (g * g)), 255)
        m8 = S.encode(b1 * S.decode(*m8, 127) + F32(0.1) * g, 127)
        v = beta2 * v + (1 - beta2) * g.astype(np.float64) ** 2
    root = S.decode(*v8, 255)
    with np.errstate(divide="ignore"):
        ratio = root / np.sqrt(v)
    assert 0.8 < np.median(ratio[~half]) < 1.25
    if kind == "steady":
        assert 0.8 < np.median(ratio[half]) < 1.25
    if kind == "fall":
        # in 32 bits the root falls to a tenth; at 0.999 here it goes with the block's largest alone
        assert (0.8 < np.median(ratio[half]) < 1.25) if beta2 == 0.95 else (np.median(ratio[half]) > 2)
    if kind == "stop":
        # in 32 bits m is 0.9^2000 of what it was and the root beta2^1000. Here an index of m remains, and with it a step; the
        # root keeps its share of a largest that moves by less than 30% (0.999), or one index at least (0.95)
        kept = np.abs(S.decode(*m8, 127))[half]
        assert np.count_nonzero(kept) > 0.9 * half.sum() and np.abs(m8[0][half]).max() <= 9
        assert (ratio[half] > (0.7 if beta2 == 0.999 else 0.5 / 255 ** 2) * beta2 ** -1000).all()
