"""GPU parity of the losses over tokens against the fp64 oracle.

Bounds, with u = 2^-24. A lane's fp32 sum of V/256 exponentials (the least number of threads is 256) is off by
at most V/256 u relative, an exponential of a base-2 exponent e by (|e| + 4) u, and a row's exponents stay under
its spread (those further than 2^-40 down are under the absolute floor 2^-40). So the sum, q and 1 - q are
off by rel = (V/256 + 16 + 4 span) u relative, and l by rel and its rounding. A ratio exp(x) is off by x's error
and (|x| + 4) u relative; the KL term by its derivative times l's error and 8 u of itself; the loss and the slope
by the sums of these and 4 u of themselves. The gradient is slope * q (or 1 - q), times scale * upstream / T,
with 4 more roundings, and its own."""

import numpy as np
import pytest
import torch

import oracle as O
import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _memory_given_back():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
LEAST = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 2.0 ** -150}   # half of the least subnormal
U = 2.0 ** -24
# fp32 has nothing between 0 and 2^-149: a ratio of exp(-200) and a loss of 1e-87 are 0 in it, and relative bounds
# on them say nothing. One such step for the exponential and one for the product.
TINY = 2.0 ** -149


def host(t):
    return None if t is None else t.double().cpu().numpy()


def place(a, dt, off=0, pad=0, filler=float("nan")):
    """A matrix `off` elements into a buffer, its rows `pad` longer."""
    buf = torch.full((off + a.shape[0] * (a.shape[1] + pad) + 3,), filler, dtype=dt, device=DEV)
    t = buf[off:off + a.shape[0] * (a.shape[1] + pad)].view(a.shape[0], a.shape[1] + pad)[:, :a.shape[1]]
    t.copy_(torch.from_numpy(a).to(dt))
    return t


def case(seed, R, V, dtype, index="i64", off=0, pad=0, std=2.0, lift=4.0, masked=True):
    rng = np.random.default_rng(seed)
    z, y = rng.standard_normal((R, V)) * std, rng.integers(0, V, R)
    z[np.arange(R), y] += rng.standard_normal(R) * 2 + lift
    logits = place(z, DT[dtype], off, pad)
    l = O.token.softmax(host(logits), y, 1.0)[0]
    w = rng.uniform(0.25, 2.0, R)
    if masked and R > 2:
        y[1], w[2] = -1, 0.0
        y[R - 1] = V + 5 if R > 4 else y[R - 1]
        logits[1].fill_(float("nan"))                 # rows without a token or weight are not read
        logits[2].fill_(float("inf"))
    f = lambda a: torch.from_numpy(a).float().to(DEV)  # noqa: E731
    return dict(logits=logits, label=torch.from_numpy(y).to(DEV, torch.int64 if index == "i64" else torch.int32),
                old=f(l + rng.normal(0, 0.2, R)), ref=f(l + rng.normal(0, 0.3, R)), adv=f(rng.standard_normal(R)),
                weight=f(w), upstream=f(rng.uniform(-2, 2, R)))


def run(s, kind, T=1.0, clip=(0.2, 0.3), kl=0.1, scale=3.0, in_place=False, weight=True, upstream=True):
    """(loss, logp, gradient) by one fused call or two."""
    R, V = s["logits"].shape
    loss, logp = (torch.full((R,), -9.0, device=DEV) for _ in range(2))
    logits = s["logits"]
    if in_place:
        logits = grad = torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype, device=DEV).copy_(logits)
    else:
        grad = torch.full((R, V + 3), -9.0, dtype=logits.dtype, device=DEV)[:, :V]
    kw = dict(ref_logp=s["ref"], weight=s["weight"] if weight else None, clip=clip, kl_coef=kl, temperature=T, logp=logp)
    up = s["upstream"] if upstream else None
    if kind == "step":
        Z.zero_policy_step(logits, s["label"], s["old"], s["adv"], loss, grad, upstream=up, scale=scale, **kw)
    else:
        stats = torch.empty(R, Z.ZERO_TOKEN_STATS, device=DEV)
        Z.zero_policy_forward(logits, s["label"], s["old"], s["adv"], loss, stats, **kw)
        Z.zero_token_backward(logits, s["label"], stats, grad, upstream=up, scale=scale, temperature=T)
    torch.cuda.synchronize()
    if not in_place:
        assert bool((grad.as_strided((R, 3), (V + 3, 1), V) == -9.0).all()), "a write past a row"
    return host(loss), host(logp), host(grad)


def bounds(z, label, T):
    """(rel of the row's sum, l's bound)."""
    V = z.shape[1]
    fin = np.where(np.isfinite(z), z, 0.0)
    span = np.minimum(1.4427 / T * (fin.max(1) - fin.min(1)), 60.0)
    return (V / 256 + 16 + 4 * span) * U


def close(got, want, tol, what):
    with np.errstate(invalid="ignore"):
        ok = (np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)) | (got == want)
    at = np.argwhere(~ok)
    assert ok.all(), (what, len(at), at[:3].tolist(), got[~ok][:3], want[~ok][:3], np.broadcast_to(tol, got.shape)[~ok][:3])


def check_gradient(got, z, label, T, coef, coef_err, rel, dtype):
    """got against coef * dl/dz; coef: scale * upstream * slope of each row, coef_err its error."""
    _, g = O.token.softmax(z, label, T)
    want = np.where(coef[:, None] == 0, 0.0, coef[:, None] * g)
    tol = np.abs(g) * coef_err[:, None] + np.abs(want) * (rel[:, None] + 8 * U + HALF[dtype]) \
        + np.abs(coef[:, None]) / T * 2.0 ** -40 + LEAST[dtype]
    close(got, want, np.where(np.isnan(tol), np.inf, tol), "gradient")


def check(s, got, T=1.0, clip=(0.2, 0.3), kl=0.1, scale=3.0, dtype="f32", weight=True, upstream=True):
    h = {k: host(v) for k, v in s.items()}
    label = h["label"].astype(int)
    R, V = h["logits"].shape
    w = h["weight"] if weight else np.ones(R)
    loss, l, _ = O.token.policy_rows(h["logits"], label, h["old"], h["adv"], clip, h["ref"], kl, w, T)
    rel = bounds(h["logits"], label, T)
    near = rel + 2 * U * np.abs(l)
    on = (label >= 0) & (label < V) & (w != 0)
    x, d = np.where(on, l - h["old"], 0), np.where(on, h["ref"] - l, 0)
    with np.errstate(over="ignore", invalid="ignore"):
        ratio = np.exp(x)
        ratio_err = ratio * (near + (np.abs(x) + 4) * U) + TINY
        kl_err = kl * (np.abs(np.expm1(d)) * near + 8 * U * np.abs(np.expm1(d)))
        loss_err = w * (np.abs(h["adv"]) * ratio_err + kl_err) + 8 * U * (np.abs(loss) + w * np.abs(h["adv"]) * ratio) + TINY
        slope = np.array([O.token.policy(l[r], h["old"][r], h["adv"][r], clip, h["ref"][r], kl)[1] if on[r] else 0.0
                          for r in range(R)])
        slope_err = np.abs(h["adv"]) * ratio_err + kl * (np.exp(d) * near + 8 * U * np.abs(np.expm1(d))) + 8 * U * np.abs(slope)
        # the derivative jumps by A*r at the range's ends, and l is known to `near`: there either side is right
        with np.errstate(divide="ignore"):
            ends = np.log([1.0 - clip[0], 1.0 + clip[1]])
        at_end = np.minimum(np.abs(x - ends[0]), np.abs(x - ends[1])) <= near
        slope_err = slope_err + np.where(at_end, np.abs(h["adv"]) * ratio, 0.0)
        close(got[1], l, near, "logp")
        close(got[0], loss, loss_err, "loss")
        k = scale * (h["upstream"] if upstream else 1.0) * np.where(on, w, 0.0)
        check_gradient(got[2], h["logits"], np.where(on, label, -1), T, k * slope, np.abs(k) * slope_err, rel, dtype)


SIZES = [(1, 1), (2, 2), (3, 7), (5, 257), (4, 1000), (3, 4099), (6, 50257), (3, 32000), (1, 131072), (600, 1500)]


@pytest.mark.parametrize("kind", ["step", "calls"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,V", SIZES)
def test_policy_against_the_oracle(R, V, dtype, kind):
    banner(f"policy R={R} V={V} {dtype} {kind}")
    for T, kl in ((1.0, 0.1), (2.5, 0.0)):
        s = case(R + V, R, V, dtype)
        check(s, run(s, kind, T, kl=kl), T, kl=kl, dtype=dtype)


# every number of vectors a thread holds, with many rows and with few, and rows past what is held
HELD = [(512, v) for v in (1024, 2047, 2049, 4096, 6000, 8193, 16384, 28673, 40000, 57345, 131071, 140000)] + \
       [(3, v) for v in (4095, 8193, 16384, 30000, 65537, 131073, 300000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", HELD)
def test_rows_held_and_read_again(R, V, dtype):
    """The first and last rows of a batch against the oracle, every row against the two calls: a row's result
    does not depend on how many there are but through the sum's order."""
    banner(f"policy held R={R} V={V} {dtype}")
    g = torch.Generator(device=DEV)
    g.manual_seed(V)
    few = case(V, 3, V, dtype, masked=False)
    s = {k: (v if v.dim() == 0 else v.repeat(*([-(-R // 3)] + [1] * (v.dim() - 1)))[:R].contiguous()) for k, v in few.items()}
    one, two = run(s, "step"), run(s, "calls")
    check({k: v[:3] for k, v in s.items()}, tuple(x[:3] for x in one), dtype=dtype)
    check({k: v[:3] for k, v in s.items()}, tuple(x[:3] for x in two), dtype=dtype)
    for x, y in zip(one, two):
        assert all(np.array_equal(x[i::3], np.broadcast_to(x[i], x[i::3].shape)) for i in range(min(3, R)))
        assert all(np.array_equal(y[i::3], np.broadcast_to(y[i], y[i::3].shape)) for i in range(min(3, R)))


@pytest.mark.parametrize("index", ["i32", "i64"])
@pytest.mark.parametrize("off,pad", [(1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_offsets_strides_and_in_place(dtype, off, pad, index):
    banner(f"policy {dtype} off={off} pad={pad} {index}")
    s = case(off + pad, 5, 1003, dtype, index, off, pad)
    for kind in ("step", "calls"):
        got = run(s, kind)
        check(s, got, dtype=dtype)
        same = run(s, kind, in_place=True)
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got, same))
    check(s, run(s, "step", upstream=False, scale=0.5), dtype=dtype, upstream=False, scale=0.5)


@pytest.mark.parametrize("T", [2.0 ** -20, 0.01, 0.7, 100.0, 2.0 ** 20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_temperatures(dtype, T):
    s = case(3, 6, 300, dtype)
    l = O.token.softmax(np.nan_to_num(host(s["logits"]), posinf=0.0), np.clip(host(s["label"]).astype(int), 0, 299), T)[0]
    s["old"], s["ref"] = (torch.from_numpy(l + d).float().to(DEV) for d in (0.1, -0.2))
    for kind in ("step", "calls"):
        check(s, run(s, kind, T), T, dtype=dtype)


def test_clips_signs_and_zero_advantages():
    """Ratios on both sides of both ends of the range with advantages of both signs and 0; ranges open to 0 and closed
    on one; overflowing ratios."""
    rng = np.random.default_rng(5)
    xs = np.array([-200.0, -1.0, -0.30, -0.2232, -0.2231, -0.1, 0.0, 0.1, 0.1823, 0.1824, 0.3, 1.0, 60.0])
    adv = np.array([1.5, -1.5, 0.0, 1e-20, -1e-20])
    R, V = xs.size * adv.size, 37
    s = case(6, R, V, "f32", masked=False)
    l = O.token.softmax(host(s["logits"]), host(s["label"]).astype(int), 1.0)[0]
    s["old"] = torch.from_numpy(l - np.repeat(xs, adv.size)).float().to(DEV)
    s["adv"] = torch.from_numpy(np.tile(adv, xs.size)).float().to(DEV)
    for clip in ((0.2, 0.2), (1.0, 0.0), (0.0, 0.0), (0.5, 1e30)):
        for kl in (0.0, 0.5):
            for kind in ("step", "calls"):
                check(s, run(s, kind, clip=clip, kl=kl), clip=clip, kl=kl)
    s["old"] = torch.full((R,), -300.0, device=DEV)             # exp(300) leaves fp32
    loss, _, grad = run(s, "step", clip=(0.2, 0.2), kl=0.0)
    w = host(s["weight"])
    pos, neg, nul = (np.tile(adv, xs.size) == a for a in (1.5, -1.5, 0.0))
    assert np.allclose(loss[pos], -1.2 * 1.5 * w[pos], rtol=1e-6) and (grad[pos] == 0).all()
    assert (loss[neg] == np.inf).all() and (loss[nul] == 0).all() and (grad[nul] == 0).all()


def test_sure_tokens_keep_the_digits_of_what_is_left():
    """A token that has nearly all the mass: l and 1 - q are those of the other entries' sum, to their own precision."""
    R, V = 6, 500
    z = np.zeros((R, V))
    y = np.arange(R) * 70
    z[np.arange(R), y] = [10.0, 20.0, 30.0, 40.0, 60.0, 80.0]
    logits, label = place(z, torch.float32), torch.from_numpy(y).to(DEV)
    logp, stats = torch.empty(R, device=DEV), torch.empty(R, Z.ZERO_TOKEN_STATS, device=DEV)
    grad = torch.empty(R, V, device=DEV)
    Z.zero_token_logp(logits, label, logp, stats=stats)
    Z.zero_token_backward(logits, label, stats, grad)
    torch.cuda.synchronize()
    left = (V - 1) * np.exp(-z[np.arange(R), y])
    rel = (V / 256 + 16 + 4 * 60) * U
    assert np.abs(host(logp) / -np.log1p(left) - 1).max() <= rel + 2 * U
    assert np.abs(host(grad)[np.arange(R), y] / (left / (1 + left)) - 1).max() <= rel + 4 * U


def test_rows_without_a_softmax_and_entries_without_mass():
    V = 700
    for kind in ("step", "calls"):
        for dtype in ("bf16", "f32"):
            s = case(9, 9, V, dtype, masked=False)
            z = s["logits"]
            z[0, 5], z[1, 699], z[2, 0] = float("nan"), float("inf"), float("nan")
            z[3] = float("-inf")
            z[4, ::2] = float("-inf")
            z[4, s["label"][4]] = 1.0
            z[5] = float("-inf")
            z[5, s["label"][5]] = 2.0                       # alone: l = 0
            z[6, s["label"][6]] = float("inf")
            z[7] = torch.finfo(z.dtype).min
            z[8, s["label"][8]] = float("nan")
            s["adv"][0] = 0.0                               # no softmax, whatever the advantage
            s["old"][4:8] = -3.0
            s["ref"][4:8] = -3.5
            got = run(s, kind)
            check(s, got, dtype=dtype)
            for r in (0, 1, 2, 3, 6, 8):
                assert np.isnan(got[0][r]) and np.isnan(got[1][r]) and np.isnan(got[2][r]).all(), r
            assert got[1][5] == 0 and (got[2][5] == 0).all()
    # a token of no mass beside others that have some: l = -inf, ratio 0
    z = torch.zeros(2, 9, device=DEV)
    z[:, 3] = float("-inf")
    label = torch.full((2,), 3, device=DEV)
    old, adv = torch.zeros(2, device=DEV), torch.tensor([1.0, -1.0], device=DEV)
    loss, logp, grad = torch.empty(2, device=DEV), torch.empty(2, device=DEV), torch.empty(2, 9, device=DEV)
    Z.zero_policy_step(z, label, old, adv, loss, grad, clip=0.2, logp=logp)
    torch.cuda.synchronize()
    assert host(logp).tolist() == [-np.inf, -np.inf] and np.allclose(host(loss), [0.0, 0.8]) and (host(grad) == 0).all()


def test_logp_alone_and_its_gradient():
    for dtype in ("bf16", "f16", "f32"):
        s = case(21, 7, 2000, dtype)
        h = {k: host(v) for k, v in s.items()}
        label = h["label"].astype(int)
        h["logits"][2], s["logits"][2] = 0.5, 0.5             # no weight here: the row counts
        logp, stats = torch.empty(7, device=DEV), torch.empty(7, Z.ZERO_TOKEN_STATS, device=DEV)
        grad = torch.empty_like(s["logits"])
        Z.zero_token_logp(s["logits"], s["label"], logp, temperature=1.5, stats=stats)
        Z.zero_token_backward(s["logits"], s["label"], stats, grad, upstream=s["upstream"], scale=-1.0, temperature=1.5)
        torch.cuda.synchronize()
        rel = bounds(h["logits"], label, 1.5)
        l, _ = O.token.softmax(h["logits"], label, 1.5)
        close(host(logp), l, rel + 2 * U * np.abs(l), "logp")
        on = (label >= 0) & (label < 2000)
        coef = -h["upstream"] * on
        check_gradient(host(grad), h["logits"], np.where(on, label, -1), 1.5, coef, 0 * coef, rel, dtype)
        bare = torch.empty(7, device=DEV)
        Z.zero_token_logp(s["logits"], s["label"], bare, temperature=1.5)
        torch.cuda.synchronize()
        assert torch.equal(bare, logp)


def prefer(s, start, pairs, dtype, beta=0.3, smoothing=0.1, margin=0.2, average=False, ref=True, weight=True, upstream=True,
           start_dtype=torch.int64, T=1.0):
    R, V = s["logits"].shape
    beta, smoothing, margin = (float(np.float32(x)) for x in (beta, smoothing, margin))   # as the call takes them
    rng = np.random.default_rng(R + pairs)
    f = lambda a: torch.from_numpy(a).float().to(DEV)  # noqa: E731
    refs, ws, ups = f(rng.standard_normal(2 * pairs) * 3), f(rng.uniform(0.5, 2, pairs)), f(rng.uniform(-2, 2, pairs))
    if pairs > 2:
        ws[1] = 0.0
    loss, logp, seq = (torch.full((n,), -9.0, device=DEV) for n in (pairs, R, 2 * pairs))
    stats = torch.full((R, Z.ZERO_TOKEN_STATS), float("nan"), device=DEV)
    grad = torch.full((R, V), -9.0, dtype=s["logits"].dtype, device=DEV)
    at = torch.from_numpy(np.asarray(start)).to(DEV, start_dtype)
    Z.zero_preference_forward(s["logits"], s["label"], at, loss, stats, ref_logp=refs if ref else None,
                              weight=ws if weight else None, beta=beta, label_smoothing=smoothing, margin=margin,
                              average=average, logp=logp, seq_logp=seq, temperature=T)
    Z.zero_token_backward(s["logits"], s["label"], stats, grad, upstream=ups if upstream else None, scale=2.0, temperature=T)
    torch.cuda.synchronize()
    z, label = host(s["logits"]), host(s["label"]).astype(int)
    on = (label >= 0) & (label < V)
    l, _ = O.token.softmax(z, np.where(on, label, -1), T)
    clamped = np.clip(start, 0, R)
    want, seqs, slope = O.token.preference(l, on, clamped, beta, host(refs) if ref else None, host(ws) if weight else None,
                                           smoothing, margin, average)
    rel = bounds(z, label, T)
    # l reaches the sums in two fp32 parts: rel alone
    err = np.where(on, rel, 0.0)
    sums = np.array([err[a:max(a, b)].sum() / (max(1, on[a:b].sum()) if average else 1) for a, b in zip(clamped[:-1], clamped[1:])])
    close(host(logp), l, err + 2 * U * np.abs(l), "logp")
    close(host(seq), seqs, sums + 2 * U * np.abs(seqs), "sequences")
    gap = abs(beta) * (sums[0::2] + sums[1::2])
    w = host(ws) if weight else np.ones(pairs)
    close(host(loss), want, w * gap + 4 * U * np.abs(want), "loss")
    of = np.searchsorted(clamped[1:], np.arange(R), side="right")
    pair = np.minimum(of // 2, pairs - 1)
    up = host(ups)[pair] if upstream else np.ones(R)
    coef = 2.0 * up * np.where(of < 2 * pairs, slope, 0.0)
    # the logistic function's slope is at most 1/4
    each = np.abs(2.0 * up * beta) * w[pair] * gap[pair] / 4 + 8 * U * np.abs(coef)
    check_gradient(host(grad), z, np.where(on, label, -1), T, coef, np.where(coef == 0, 0, each), rel, dtype)
    return host(loss), host(grad)


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,V,start", [
    (2, 5, [0, 1, 2]), (9, 257, [0, 3, 3, 5, 8]), (40, 1003, [0, 7, 11, 20, 21, 30, 36]), (700, 900, [0, 300, 650, 660, 690]),
    (12, 50257, [2, 5, 9]), (6, 64, [0, 0, 0, 3, 6])])
def test_preference_against_the_oracle(R, V, start, dtype, average):
    """Sequences of no row, of rows without a token, rows before the first and behind the last sequence."""
    banner(f"preference R={R} V={V} {dtype} {average}")
    s = case(R + V, R, V, dtype)
    s["logits"][2].fill_(0.25) if R > 2 else None
    pairs = len(start) // 2
    prefer(s, start, pairs, dtype, average=average)
    prefer(s, start, pairs, dtype, average=average, ref=False, weight=False, upstream=False, smoothing=0.0, margin=0.0,
           start_dtype=torch.int32, T=1.7)


def test_preferences_far_apart_and_starts_out_of_range():
    s = case(31, 10, 100, "f32", masked=False)
    for beta in (1e4, -1e4, 0.0):
        for smoothing in (0.0, 0.5, 1.0):
            prefer(s, [0, 2, 5, 7, 10], 2, "f32", beta=beta, smoothing=smoothing)
    prefer(s, [-5, 2, 5, 7, 90], 2, "f32")
    # starts that descend leave empty sequences; nothing is read or written out of the batch
    loss, grad = [t for t in prefer(s, [0, 5, 3, 3, 10], 2, "f32", upstream=False)]
    assert np.isfinite(loss).all() and np.isfinite(grad).all()


def test_a_row_without_a_softmax_spoils_its_pair_alone():
    s = case(33, 8, 50, "f32", masked=False)
    s["logits"][1, 3] = float("nan")
    start = torch.tensor([0, 2, 4, 6, 8], device=DEV)
    loss, stats = torch.empty(2, device=DEV), torch.empty(8, Z.ZERO_TOKEN_STATS, device=DEV)
    grad = torch.empty(8, 50, device=DEV)
    Z.zero_preference_forward(s["logits"], s["label"], start, loss, stats)
    Z.zero_token_backward(s["logits"], s["label"], stats, grad)
    torch.cuda.synchronize()
    assert torch.isnan(loss[0]) and torch.isfinite(loss[1])
    assert torch.isnan(grad[:4]).all() and torch.isfinite(grad[4:]).all()


def test_an_upstream_that_is_too_short_gives_nan_and_reads_nothing_else():
    s = case(35, 6, 40, "f32", masked=False)
    logp, stats = torch.empty(6, device=DEV), torch.empty(6, Z.ZERO_TOKEN_STATS, device=DEV)
    grad = torch.empty(6, 40, device=DEV)
    Z.zero_token_logp(s["logits"], s["label"], logp, stats=stats)
    Z.zero_token_backward(s["logits"], s["label"], stats, grad, upstream=torch.ones(4, device=DEV))
    torch.cuda.synchronize()
    assert torch.isfinite(grad[:4]).all() and torch.isnan(grad[4:]).all()


def test_empty_batches():
    z, y = torch.empty(0, 7, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    e = torch.empty(0, device=DEV)
    Z.zero_token_logp(z, y, e)
    Z.zero_policy_step(z, y, e, e, e, z)
    loss, seq = torch.empty(2, device=DEV), torch.empty(4, device=DEV)
    Z.zero_preference_forward(z, y, torch.zeros(5, dtype=torch.int64, device=DEV), loss, torch.empty(0, 8, device=DEV),
                              seq_logp=seq, margin=0.5)
    torch.cuda.synchronize()
    assert torch.allclose(loss, torch.full_like(loss, float(np.logaddexp(0, 0.5)))) and bool((seq == 0).all())


def test_captured_replayed_and_on_two_streams():
    s = case(41, 520, 3000, "bf16")
    start = torch.tensor([0, 100, 260, 400, 520], device=DEV)
    outs = [dict(loss=torch.empty(520, device=DEV), pl=torch.empty(2, device=DEV), grad=torch.empty_like(s["logits"]),
                 pg=torch.empty_like(s["logits"]), stats=torch.empty(520, 8, device=DEV)) for _ in range(3)]

    def both(o):
        Z.zero_policy_step(s["logits"], s["label"], s["old"], s["adv"], o["loss"], o["grad"], ref_logp=s["ref"],
                           weight=s["weight"], kl_coef=0.1)
        Z.zero_preference_forward(s["logits"], s["label"], start, o["pl"], o["stats"])
        Z.zero_token_backward(s["logits"], s["label"], o["stats"], o["pg"])

    both(outs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(outs[1])
    keep = s["old"].clone()
    for k in range(3):
        s["old"].copy_(keep + 0.1 * k)
        both(outs[0])
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both(outs[2])
        both(outs[0])
        torch.cuda.synchronize()
        for o in outs[1:]:
            for name in ("loss", "pl", "grad", "pg"):
                assert torch.equal(torch.nan_to_num(o[name]), torch.nan_to_num(outs[0][name])), (k, name)


def test_logits_past_32_bits():
    """More than 2^32 bytes of logits: the last rows as a small call gives them."""
    R, V = 9000, 131073
    z = torch.empty(R, V, device=DEV, dtype=torch.float32)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    z.normal_(0, 2, generator=g)
    label = torch.randint(V, (R,), generator=g, device=DEV)
    old, adv = torch.randn(R, device=DEV), torch.randn(R, device=DEV)
    loss, grad = torch.empty(R, device=DEV), torch.empty_like(z)
    Z.zero_policy_step(z, label, old, adv, loss, grad)
    tail = slice(R - 600, R)
    loss2, grad2 = torch.empty(600, device=DEV), torch.empty(600, V, device=DEV)
    Z.zero_policy_step(z[tail], label[tail], old[tail], adv[tail], loss2, grad2)
    torch.cuda.synchronize()
    assert torch.equal(loss[tail], loss2) and torch.equal(grad[tail], grad2)


def test_more_rows_than_one_grid_dimension_holds():
    R, V = (1 << 21) + 5, 9
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    z = torch.empty(R, V, device=DEV).normal_(generator=g)
    label = torch.randint(-1, V, (R,), generator=g, device=DEV, dtype=torch.int32)
    old, adv = torch.empty(R, device=DEV).normal_(-2, 0.3, generator=g), torch.empty(R, device=DEV).normal_(generator=g)
    loss, logp, grad = torch.empty(R, device=DEV), torch.empty(R, device=DEV), torch.empty_like(z)
    Z.zero_policy_step(z, label, old, adv, loss, grad, logp=logp)
    stats, grad2 = torch.empty(R, Z.ZERO_TOKEN_STATS, device=DEV), torch.empty_like(z)
    start = torch.tensor([0, R // 2, R], device=DEV)
    pair = torch.empty(1, device=DEV)
    Z.zero_preference_forward(z, label, start, pair, stats, average=True)
    Z.zero_token_backward(z, label, stats, grad2)
    torch.cuda.synchronize()
    l = torch.log_softmax(z.double(), 1)
    on = label >= 0
    want = torch.where(on, l.gather(1, label.long().clamp(min=0)[:, None])[:, 0], torch.zeros(R, dtype=torch.float64, device=DEV))
    rel = (V / 256 + 16 + 4 * 30) * U
    assert float((logp.double() - want).abs().max()) <= rel + 2 * U * float(want.abs().max())
    assert bool((grad[~on] == 0).all()) and bool((loss[~on] == 0).all())
    means = [float(want[a:b].sum() / max(1, int(on[a:b].sum()))) for a, b in ((0, R // 2), (R // 2, R))]
    x = 0.1 * (means[0] - means[1])
    assert abs(float(pair) - np.logaddexp(0, -x)) <= 0.2 * rel + 4 * U
    s = -0.1 / (1 + np.exp(x)) / int(on[:R // 2].sum())
    first = int(torch.nonzero(on)[0])
    q = l[first].exp()
    q[int(label[first])] -= 1
    assert float((grad2[first].double() + s * q).abs().max()) <= abs(s) * (rel + 0.2 * rel + 16 * U)
