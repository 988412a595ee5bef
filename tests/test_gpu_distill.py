"""GPU parity of the distillation loss against the fp64 oracle.

Bounds, with u = 2^-24. A sum of V exponentials in fp32 over 256 threads or more is off by at most
(V/256 + 24) u relative; an exponential of a base-2 exponent e by (|e| + 4) u, and exponents stay
under 2 max|z - m| log2(e)/T. So q and p are off by rel = (V/256 + 64 + 4 span) u relative, with span
the row's spread of base-2 exponents over the entries that matter (those further than 2^-40 down are
under the absolute floor 2^-40). The gradient is scale*w/T times (q + p) times rel, plus its
rounding; the loss is a sum over k of p_k times logarithms that are each off by rel + 4u |log|."""

import numpy as np
import pytest
import torch

import oracle as O
import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
U = 2.0 ** -24


def case(seed, R, V, K, dtype, teacher="f32", index="i32", tail=False, off=0, pad=0, std=2.0):
    """Device tensors (each matrix `off` elements into a buffer, rows `pad` longer) of one problem."""
    rng = np.random.default_rng(seed)

    def place(a, dt, filler):
        buf = torch.full((off + a.shape[0] * (a.shape[1] + pad) + 3,), filler, dtype=dt, device=DEV)
        t = buf[off:off + a.shape[0] * (a.shape[1] + pad)].view(a.shape[0], a.shape[1] + pad)[:, :a.shape[1]]
        t.copy_(torch.from_numpy(a).to(dt))
        return t

    z = rng.standard_normal((R, V)) * std
    idx = np.stack([rng.permutation(V)[:K] if K <= V else rng.integers(0, V, K) for _ in range(R)])
    top = -np.sort(-rng.standard_normal((R, K)) * 2, axis=1) + 6
    np.put_along_axis(z, idx, top + rng.standard_normal((R, K)), 1)
    s = dict(logits=place(z, DT[dtype], float("nan")), top=place(top, DT[teacher], float("nan")),
             idx=place(idx, torch.int64 if index == "i64" else torch.int32, 1 << 30),
             weight=torch.from_numpy(rng.uniform(0.25, 2.0, R)).float().to(DEV),
             upstream=torch.from_numpy(rng.uniform(-2.0, 2.0, R)).float().to(DEV),
             tail=torch.from_numpy(rng.standard_normal(R) + 5).float().to(DEV) if tail else None)
    return s


def run(s, T, scale, kind, in_place=False):
    """(loss, gradient) by one fused call or by two."""
    R, V = s["logits"].shape
    loss = torch.full((R,), -9.0, device=DEV)
    logits = s["logits"]
    if in_place:
        buf = torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype, device=DEV)
        buf.copy_(logits)
        logits = grad = buf
    else:
        grad = torch.full((R, V + 3), -9.0, dtype=logits.dtype, device=DEV)[:, :V]
    kw = dict(tail=s["tail"], weight=s["weight"])
    if kind == "step":
        Z.zero_distill_step(logits, s["idx"], s["top"], T, loss, grad, upstream=s["upstream"], scale=scale, **kw)
    else:
        stats = torch.empty(R, 2, device=DEV)
        Z.zero_distill_forward(logits, s["idx"], s["top"], T, loss, stats, **kw)
        Z.zero_distill_backward(logits, s["idx"], s["top"], T, stats, grad, upstream=s["upstream"], scale=scale, **kw)
    torch.cuda.synchronize()
    if not in_place:
        assert bool((grad.as_strided((R, 3), (V + 3, 1), V) == -9.0).all()), "write past a row"
    return loss.double().cpu().numpy(), grad.double().cpu().numpy()


def check(s, T, scale, got, dtype):
    h = {k: (None if v is None else v.double().cpu().numpy()) for k, v in s.items()}
    V, K = h["logits"].shape[1], h["idx"].shape[1]
    loss, grad = O.layer.distill(h["logits"], h["idx"], h["top"], T, h["tail"], h["weight"])
    grad = grad * (scale * h["upstream"])[:, None]
    spread = np.nan_to_num(np.where(np.isfinite(h["logits"]), h["logits"], 0.0))
    span = np.minimum(1.4427 / T * (spread.max(1) - spread.min(1)), 60.0)
    rel = (V / 256 + 64 + 4 * span) * U
    g = np.abs(scale * h["upstream"] * h["weight"] / T)
    logs = span + np.log2(V) + 40
    with np.errstate(invalid="ignore"):
        err = np.abs(got[0] - loss)
        ok = (err <= h["weight"] * (rel + 8 * U * logs)) | (np.isnan(loss) & np.isnan(got[0])) | (loss == got[0])
        assert ok.all(), ("loss", np.flatnonzero(~ok)[:5], got[0][~ok][:5], loss[~ok][:5])
        # q and p are at most |grad|/g plus twice the smaller of the two; 2 is the bound of both
        y = h["logits"] / T
        q = np.exp(y - np.nanmax(y, 1, keepdims=True))
        q = np.nan_to_num(q / np.nansum(q, 1, keepdims=True))   # a NaN logit gives no bound: its row must be NaN, or 0 unread
        big = g[:, None] * (q + np.abs(np.nan_to_num(grad)) / np.maximum(g[:, None], 1e-30)) * 2
        tol = big * rel[:, None] + HALF_STEP[dtype] * np.abs(grad) + g[:, None] * 2.0 ** -40 \
            + {"f16": 2.0 ** -25}.get(dtype, 0.0)
        err = np.abs(got[1] - grad)
        ok = (err <= tol) | (np.isnan(grad) & np.isnan(got[1]))
    at = np.argwhere(~ok)
    assert ok.all(), ("gradient", len(at), at[:3], got[1][~ok][:3], grad[~ok][:3], tol[~ok][:3])


@pytest.mark.parametrize("kind", ["step", "calls"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,V,K", [(1, 1, 1), (2, 2, 1), (3, 7, 3), (5, 257, 16), (4, 1000, 130), (3, 4099, 64),
                                   (2, 50257, 16), (3, 32000, 32), (2, 9000, 1024), (1, 131072, 100)])
def test_against_the_oracle(R, V, K, dtype, tail, kind):
    if tail and K == V:
        pytest.skip("nothing is left for a tail: its own test")
    banner(f"distill R={R} V={V} K={K} {dtype} tail={tail} {kind}")
    for T, scale in ((1.0, 1.0), (2.5, 64.0)):
        s = case(R + V + K, R, V, K, dtype, tail=tail)
        check(s, T, scale, run(s, T, scale, kind), dtype)


@pytest.mark.parametrize("teacher,index", [("bf16", "i64"), ("f16", "i32"), ("f32", "i64")])
@pytest.mark.parametrize("off,pad", [(1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_types_offsets_and_strides(teacher, index, off, pad, dtype):
    banner(f"distill {dtype} {teacher} {index} off={off} pad={pad}")
    s = case(off + pad, 5, 1003, 20, dtype, teacher, index, True, off, pad)
    for kind in ("step", "calls"):
        got = run(s, 1.5, 3.0, kind)
        check(s, 1.5, 3.0, got, dtype)
        same = run(s, 1.5, 3.0, kind, in_place=True)
        assert np.array_equal(got[0], same[0]) and np.array_equal(got[1], same[1]), "in place"


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("kind", ["step", "calls"])
def test_short_rows_duplicates_and_masks(tail, kind):
    banner(f"distill masks tail={tail} {kind}")
    s = case(77, 12, 3001, 40, "f32", tail=tail)
    s["idx"][0, 5:] = -1                                        # a short row
    s["idx"][1, 7], s["idx"][1, 30], s["idx"][1, 39] = (s["idx"][1, 2].clone() for _ in range(3))   # listed four times
    s["idx"][2] = s["idx"][2, 0].clone()                        # one index forty times
    s["idx"][3, 3] = 3001                                       # just outside
    s["idx"][4] = -1                                            # no entry at all
    s["top"][5, 10:] = float("-inf")                            # listed, without mass
    s["top"][6] = float("-inf")                                 # no listed mass
    s["logits"][7, 100:2000] = float("-inf")                    # masked logits, some listed
    s["logits"][8, :1500] = torch.finfo(torch.float32).min      # masked with the lowest number
    s["logits"][9] = torch.finfo(torch.float32).min             # every logit the lowest
    s["weight"][10] = 0.0
    s["logits"][10, 5] = float("nan")                           # a row of weight 0 is not read
    s["top"][11] += 3e38                                        # far off, no overflow in the softmax
    got = run(s, 1.3, 2.0, kind)
    finite = [r for r in range(12) if r not in (7, 8)]
    sub = {k: (None if v is None else v[finite]) for k, v in s.items()}
    check(sub, 1.3, 2.0, (got[0][finite], got[1][finite]), "f32")
    h = {k: (None if v is None else v[7:9].double().cpu().numpy()) for k, v in s.items()}
    loss, grad = O.layer.distill(h["logits"], h["idx"], h["top"], 1.3, h["tail"], h["weight"])
    assert np.isposinf(got[0][7]) and loss[0] == np.inf          # p where q has none
    assert abs(got[0][8] / loss[1] - 1) < 1e-5 or (np.isinf(got[0][8]) and loss[1] > 3e38)
    g = 2.0 * h["upstream"][:, None]
    assert np.allclose(got[1][7:9], grad * g, rtol=1e-5, atol=1e-9)
    if not tail:
        assert got[0][4] == 0 and not got[1][4].any() and got[0][6] == 0 and not got[1][6].any()
    assert got[0][10] == 0 and not got[1][10].any()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_without_a_softmax_are_nan_and_leave_others_alone(dtype, tail):
    s = case(5, 6, 700, 9, dtype, tail=tail)
    s["logits"][1, 300] = float("nan")
    s["logits"][2, 699] = float("inf")
    s["logits"][3] = float("-inf")
    s["logits"][4, int(s["idx"][4, 2])] = float("nan")           # in a listed entry
    for kind in ("step", "calls"):
        got = run(s, 1.0, 1.0, kind)
        assert np.isnan(got[0][1:5]).all() and np.isnan(got[1][1:5]).all()
        keep = [0, 5]
        sub = {k: (None if v is None else v[keep]) for k, v in s.items()}
        check(sub, 1.0, 1.0, (got[0][keep], got[1][keep]), dtype)


def test_tail_with_nothing_left_of_the_vocabulary():
    s = case(3, 2, 8, 8, "f32", tail=True)
    got = run(s, 1.0, 1.0, "step")
    assert np.isposinf(got[0]).all() and np.isfinite(got[1]).all()
    s["tail"].fill_(float("-inf"))                               # no remaining mass: an ordinary loss
    got = run(s, 1.0, 1.0, "step")
    s["tail"] = None
    check(s, 1.0, 1.0, got, "f32")


def test_far_tail_mass_keeps_its_digits():
    """The student's remaining mass is 2^-60 of the whole: formed as a sum of its own, its logarithm
    is as exact as any other."""
    V, K = 5000, 4
    s = case(8, 3, V, K, "f32", tail=True, std=0.5)
    s["logits"].sub_(45.0)
    for r in range(3):
        s["logits"][r, s["idx"][r].long()] += 45.0
    check(s, 1.0, 1.0, run(s, 1.0, 1.0, "step"), "f32")
    check(s, 1.0, 1.0, run(s, 1.0, 1.0, "calls"), "f32")


def test_fused_equals_two_calls_and_repeats():
    for dtype in ("bf16", "f32"):
        s = case(21, 40, 12345, 50, dtype, tail=True)
        a, b, c = run(s, 2.0, 8.0, "step"), run(s, 2.0, 8.0, "calls"), run(s, 2.0, 8.0, "step")
        assert np.array_equal(a[0], c[0]) and np.array_equal(a[1], c[1])
        assert np.allclose(a[0], b[0], rtol=1e-5) and np.allclose(a[1], b[1], rtol=2 * HALF_STEP[dtype] + 1e-4, atol=1e-6)


def test_gradient_by_differences_of_the_loss():
    """The kernel's gradient against central differences of the kernel's own loss (fp32, so steps of
    2^-4 and a bound of the third derivative's h^2/6 <= 2^-4*2^-4/6 plus the losses' rounding)."""
    V, K, T = 64, 6, 1.0
    s = case(31, 1, V, K, "f32", tail=True, std=1.0)
    s["weight"].fill_(1.0)
    s["upstream"].fill_(1.0)
    _, grad = run(s, T, 1.0, "step")
    h = 2.0 ** -4
    base = s["logits"][0].clone()
    batch = base.repeat(2 * V, 1)
    batch[torch.arange(V), torch.arange(V)] += h
    batch[V + torch.arange(V), torch.arange(V)] -= h
    t = dict(logits=batch, idx=s["idx"].repeat(2 * V, 1), top=s["top"].repeat(2 * V, 1), weight=None,
             upstream=None, tail=s["tail"].repeat(2 * V))
    loss, _ = run(t, T, 1.0, "step")
    diff = (loss[:V] - loss[V:]) / (2 * h)
    assert np.abs(diff - grad[0]).max() <= h * h / 6 + 64 * U * 60 / h


def test_large_batch_on_the_device():
    """Enough rows to fill the card, checked against the definition in fp64 on the device."""
    R, V, K, T = 1500, 20011, 32, 2.0
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    z = (torch.randn(R, V, generator=g, device=DEV) * 2).bfloat16()
    idx = (torch.randint(V, (R, 1), generator=g, device=DEV) + torch.arange(K, device=DEV) * 7) % V
    top = torch.randn(R, K, generator=g, device=DEV) * 2
    loss, grad = torch.empty(R, device=DEV), torch.empty_like(z)
    Z.zero_distill_step(z, idx, top, T, loss, grad, scale=T * T)
    lq = torch.log_softmax(z.double() / T, 1)
    lp = torch.log_softmax(top.double() / T, 1)
    want = (lp.exp() * (lp - lq.gather(1, idx))).sum(1)
    q = lq.exp()
    w = (q.scatter_add(1, idx, -lp.exp())) * T
    torch.cuda.synchronize()
    assert float((loss.double() - want).abs().max()) <= 400 * U
    assert bool(((grad.double() - w).abs() <= w.abs() * 2.0 ** -8 + T * (q + 1.0 * (w < 0)) * 400 * U + 2.0 ** -40).all())


def test_device_refusals():
    s = case(1, 4, 50, 3, "f32")
    loss = torch.empty(4, device=DEV)
    with pytest.raises(ValueError):
        Z.zero_distill_step(s["logits"].t().contiguous().t(), s["idx"], s["top"], 1.0, loss, torch.empty(4, 50, device=DEV))
    with pytest.raises(Z.ZeroError):
        Z.zero_distill_step(s["logits"], s["idx"], s["top"], 0.0, loss, torch.empty(4, 50, device=DEV))
    with pytest.raises(TypeError):
        Z.zero_distill_step(s["logits"], s["idx"], s["top"], 1.0, loss, torch.empty(4, 50, device=DEV).half())


@pytest.mark.parametrize("kind", ["step", "calls"])
def test_more_rows_than_one_grid_dimension_holds(kind):
    """2^24 rows of 256 threads are 2^32. One listed entry at T = 1 is the cross entropy of a label.
    fp32 with 3 logits of at most 4: loss and gradient within a few dozen roundings of numbers up to 12."""
    R, V = (1 << 24) + 5, 3
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    z = torch.rand(R, V, generator=g, device=DEV) * 8 - 4
    idx = torch.randint(V, (R, 1), generator=g, device=DEV)
    top = torch.zeros(R, 1, device=DEV)
    loss, grad = torch.full((R,), -1.0, device=DEV), torch.full((R, V), -9.0, device=DEV)
    if kind == "step":
        Z.zero_distill_step(z, idx, top, 1.0, loss, grad)
    else:
        stats = torch.empty(R, 2, device=DEV)
        Z.zero_distill_forward(z, idx, top, 1.0, loss, stats)
        Z.zero_distill_backward(z, idx, top, 1.0, stats, grad)
    lq = torch.log_softmax(z.double(), 1)
    want = lq.exp().scatter_add(1, idx, torch.full((R, 1), -1.0, dtype=torch.double, device=DEV))
    torch.cuda.synchronize()
    assert float((loss.double() + lq.gather(1, idx)[:, 0]).abs().max()) <= 400 * U
    assert float((grad.double() - want).abs().max()) <= 400 * U
