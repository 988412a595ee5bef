"""The oracle's 8-bit moments against a search over all indices and against the spacing's error bounds."""

import numpy as np
import pytest

import oracle as O

S = O.state8


def _numbers(kind, n, rng):
    x = rng.standard_normal(n).astype(np.float32)
    if kind == "wide":
        x *= np.exp(rng.uniform(-30, 0, n)).astype(np.float32)
    if kind == "tiny":
        x *= np.float32(2.0 ** -120)
    if kind == "few":
        x[rng.random(n) < 0.9] = 0.0
    return x


@pytest.mark.parametrize("top", [127, 255])
@pytest.mark.parametrize("kind", ["plain", "wide", "tiny", "few"])
@pytest.mark.parametrize("n", [1, 255, 256, 257, 1000])
def test_the_index_is_the_nearest_in_square_root(top, kind, n):
    rng = np.random.default_rng(n)
    x = _numbers(kind, n, rng)
    x = np.abs(x) if top == 255 else x
    codes, scale = S.encode(x, top)
    values = np.arange(top + 1, dtype=np.float64) ** 2 / top ** 2
    for i in range(n):
        s = float(scale[i // 256])
        block = x[i // 256 * 256:(i // 256 + 1) * 256]
        assert s == (np.abs(block).max() if np.abs(block).max() >= 2.0 ** -126 else 0.0)
        q = abs(int(codes[i]))
        if s == 0.0 or x[i] == 0.0:
            assert q == 0
            continue
        far = np.abs(np.sqrt(values) - np.sqrt(abs(float(x[i])) / s))
        # two roundings to 2^-24 relative lie between |x|/s and t: half of that in the root, over at most 1
        assert far[q] <= far.min() + 2.0 ** -23 or (top == 255 and q == 1)
        assert (int(codes[i]) < 0) <= (x[i] < 0)
        if top == 255:
            assert q >= 1


@pytest.mark.parametrize("top", [127, 255])
def test_values_are_within_half_a_step(top):
    """Half an index in the root is (q + 1/4)/top^2 of the largest in the value (from 0 to 2.25/top^2 for the least
    index of 255, which takes all that is not 0); 4 roundings beside it."""
    rng = np.random.default_rng(top)
    x = _numbers("wide", 4096, rng)
    x = np.abs(x) if top == 255 else x
    codes, scale = S.encode(x, top)
    got = S.decode(codes, scale, top).astype(np.float64)
    s = np.repeat(scale, 256).astype(np.float64)
    q = np.abs(codes.astype(np.float64))
    step = (q + 0.25) / top ** 2
    assert (np.abs(got - x) <= s * step + 4 * 2.0 ** -24 * np.abs(x)).all()
    again, scale2 = S.encode(got.astype(np.float32), top)
    assert np.array_equal(again, codes) and np.abs(scale2 / scale - 1).max() <= 2.0 ** -22


def test_blocks_that_hold_no_numbers():
    for bad in (np.nan, np.inf, -np.inf):
        x = np.linspace(-1, 1, 600).astype(np.float32)
        x[300] = bad
        codes, scale = S.encode(x, 127)
        assert np.isnan(scale[1]) and not codes[256:512].any() and np.isfinite(scale[[0, 2]]).all()
        assert np.isnan(S.decode(codes, scale, 127)[256:512]).all()
    codes, scale = S.encode(np.full(300, 1e-39, np.float32), 255)
    assert not codes.any() and not scale.any() and not S.decode(codes, scale, 255).any()


def test_halves_go_down_and_the_largest_is_the_last_index():
    x = np.zeros(256, np.float32)
    x[0] = 65025.0                                        # scale 255^2: t = x up to one rounding each
    for q in (0, 1, 7, 100, 254):
        x[1] = (q + 0.5) ** 2
        inv = np.float32(1.0) / x[0]
        t = np.float32(np.float32(x[1] * inv) * np.float32(65025.0))
        want = q if t <= x[1] else q + 1
        codes, _ = S.encode(x, 255)
        assert codes[0] == 255 and codes[1] == max(want, 1)
    x[0], x[1] = 1.0, 1.0
    assert S.encode(-x, 127)[0][:2].tolist() == [-127, -127]


def test_a_step_is_the_full_width_step_on_the_values():
    rng = np.random.default_rng(5)
    n = 700
    m = S.encode(rng.standard_normal(n).astype(np.float32), 127)
    v = S.encode(np.abs(rng.standard_normal(n)).astype(np.float32), 255)
    p, g = (rng.standard_normal(n).astype(np.float32) for _ in range(2))
    hp = O.AdamHParams(lr=1e-2, weight_decay=0.1, step=3)
    p1, m1, v1, out = S.step(g, "f32", 0.5, p, m, v, hp, "bf16")
    m64, w64 = S.decode(*m, 127).astype(np.float64), S.decode(*v, 255).astype(np.float64)
    g64 = 0.5 * g
    m64, v64 = 0.9 * m64 + 0.1 * g64, 0.999 * w64 ** 2 + 0.001 * g64 ** 2
    want = p * (1 - 1e-3) - 1e-2 / (1 - 0.9 ** 3) * m64 / (np.sqrt(v64) / np.sqrt(1 - 0.999 ** 3) + 1e-8)
    assert np.abs(p1 - want).max() <= 1e-5 and out.dtype == np.uint16
    assert np.abs(S.decode(*m1, 127) - m64).max() <= 1.01 * np.abs(m64).max() / 127
    assert np.abs(S.decode(*v1, 255) - np.sqrt(v64)).max() <= 1.01 * np.sqrt(v64).max() / 255
