"""GPU parity of the losses over tokens on rows with masks by large finite numbers, rows far from 0, and tokens that
are alone: every such row has a softmax. Bounds: those of test_gpu_token, whose exponent's span is at its limit here."""

import numpy as np
import pytest
import torch

import oracle as O
import test_gpu_token as G
import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu

MASKS = [-1e9, -1e10, -1e12, -1e20, -1e30, None]          # None: the type's lowest number
KINDS = 7


def masked_rows(dtype, mask, V, T, seed, repeat=1):
    """A row of each pattern, `repeat` times: the first half masked, every other 16 bytes, all but the token, all but
    the token and three others, all but the last columns and the token, one value throughout, and a whole row so far
    from 0."""
    rng = np.random.default_rng(seed)
    top = torch.finfo(G.DT[dtype]).min if mask is None else mask
    z, y = rng.standard_normal((KINDS, V)) * 2, rng.integers(0, V, KINDS)
    keep, per = np.zeros((KINDS, V), bool), 4 if dtype == "f32" else 8
    keep[0, V // 2:] = True
    keep[1] = np.arange(V) // per % 2 == 0
    keep[3, rng.integers(0, V, 3)] = True
    keep[4, V - 5:] = True
    keep[np.arange(KINDS), y] = True
    keep[5:] = True
    z = np.where(keep, z, top)
    z[5] = top
    z[6] = top if mask is None else top + z[6]
    logits = G.place(z, G.DT[dtype]).repeat(repeat, 1)
    y = np.tile(y, repeat)
    l = np.tile(O.token.softmax(G.host(logits[:KINDS]), y[:KINDS], T)[0], repeat)
    f = lambda a: torch.from_numpy(a).float().to(DEV)  # noqa: E731
    R = len(y)
    tile = lambda a: np.tile(a, repeat)  # noqa: E731
    return dict(logits=logits, label=torch.from_numpy(y).to(DEV), old=f(l + tile(rng.normal(0, 0.1, KINDS))),
                ref=f(l + tile(rng.normal(0, 0.2, KINDS))), adv=f(tile(rng.standard_normal(KINDS))),
                weight=f(tile(rng.uniform(0.5, 2, KINDS))), upstream=torch.ones(R, device=DEV))


@pytest.mark.parametrize("kind", ["step", "calls"])
@pytest.mark.parametrize("T", [0.1, 0.5, 0.7, 1.0, 64.0])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_masked_by_large_numbers(dtype, mask, T, kind):
    banner(f"masks {dtype} {mask} T={T} {kind}")
    T = float(np.float32(T))                              # as the call takes it
    s = masked_rows(dtype, mask, 1601, T, 3)
    got = G.run(s, kind, T)
    assert all(np.isfinite(x).all() for x in got)
    G.check(s, got, T, dtype=dtype)


@pytest.mark.parametrize("dtype,V,repeat", [("bf16", 1601, 75), ("f32", 1601, 75), ("f32", 70001, 1), ("bf16", 140003, 1)])
def test_masked_rows_of_batches_and_of_rows_read_again(dtype, V, repeat):
    for mask in (-1e10, -1e30):
        s = masked_rows(dtype, mask, V, 1.0, V, repeat)
        for kind in ("step", "calls"):
            got = G.run(s, kind)
            assert all(np.array_equal(x[i::KINDS], np.broadcast_to(x[i], x[i::KINDS].shape)) for x in got for i in range(KINDS))
            G.check({k: v[:KINDS] for k, v in s.items()}, tuple(x[:KINDS] for x in got), dtype=dtype)


@pytest.mark.parametrize("T", [1.0, 0.5, 0.7])
def test_masked_tokens_of_sequences(T):
    """A token that is masked itself has l of the mask's size, and the preference loss of its pair is linear in it."""
    V, T = 1000, float(np.float32(T))
    rng = np.random.default_rng(4)
    z = rng.standard_normal((6, V))
    z[:, :V // 2] = -1e10
    y = np.array([10, 900, 499, 500, 999, 0])
    logits, label = G.place(z, torch.float32), torch.from_numpy(y).to(DEV)
    start = torch.tensor([0, 3, 6], device=DEV)
    loss, logp, seq, stats = (torch.empty(n, device=DEV) for n in (1, 6, 2, 6 * Z.ZERO_TOKEN_STATS))
    Z.zero_preference_forward(logits, label, start, loss, stats.view(6, -1), logp=logp, seq_logp=seq, temperature=T)
    torch.cuda.synchronize()
    l = O.token.softmax(G.host(logits), y, T)[0]
    rel = G.bounds(G.host(logits), y, T)
    G.close(G.host(logp), l, rel + 2 * G.U * np.abs(l), "logp")
    sums = np.array([l[:3].sum(), l[3:].sum()])
    G.close(G.host(seq), sums, 3 * rel[0] + 2 * G.U * np.abs(sums), "seq")
    x = float(np.float32(0.1)) * (sums[0] - sums[1])
    want = np.logaddexp(0.0, -x)
    G.close(G.host(loss), np.array([want]), 6 * rel[0] + 4 * G.U * np.abs(want), "loss")


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("kind", ["step", "calls"])
def test_rows_about_the_ends_of_the_fused_exponent(kind, sign):
    """Whole numbers about 2^24 and 2^25 log 2, each lane's in an order of its own: places on both sides of the range in
    which an exponent is one fused operation are joined."""
    rng = np.random.default_rng(5)
    R, V = 8, 1500
    about = np.rint(np.array([2.0 ** 24, 2.0 ** 24, 2.0 ** 25, 2.0 ** 23]) * np.log(2.0))
    z = sign * (np.tile(about, 2)[:, None] + np.floor(rng.uniform(-14, 14, (R, V)) / 2) * 2)
    y = rng.integers(0, V, R)
    z[np.arange(R), y] = z.max(1)
    s = dict(logits=G.place(z, torch.float32), label=torch.from_numpy(y).to(DEV))
    l = O.token.softmax(G.host(s["logits"]), y, 1.0)[0]
    f = lambda a: torch.from_numpy(a).float().to(DEV)  # noqa: E731
    s.update(old=f(l + 0.1), ref=f(l - 0.2), adv=f(rng.standard_normal(R)), weight=torch.ones(R, device=DEV),
             upstream=torch.ones(R, device=DEV))
    G.check(s, G.run(s, kind))


@pytest.mark.parametrize("T", [1.0, 50.0, 64.0, 100.0, 2.0 ** 20])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 9, 700])
def test_a_token_alone_is_certain_at_any_temperature(V, dtype, T):
    z = torch.full((3, V), float("-inf"), dtype=G.DT[dtype], device=DEV)
    label = torch.tensor([0, V // 2, V - 1], device=DEV)
    z[torch.arange(3), label] = torch.tensor([2.0, -300.0, 1000.0], dtype=z.dtype, device=DEV)
    logp, stats, grad = torch.empty(3, device=DEV), torch.empty(3, Z.ZERO_TOKEN_STATS, device=DEV), torch.empty_like(z)
    Z.zero_token_logp(z, label, logp, temperature=T, stats=stats)
    Z.zero_token_backward(z, label, stats, grad, temperature=T)
    torch.cuda.synchronize()
    assert bool((logp == 0).all()) and bool((grad == 0).all())
    loss, adv = torch.empty(3, device=DEV), torch.tensor([1.0, -1.0, 0.5], device=DEV)
    Z.zero_policy_step(z, label, torch.zeros(3, device=DEV), adv, loss, grad, temperature=T, logp=logp)
    torch.cuda.synchronize()
    assert bool((logp == 0).all()) and bool((grad == 0).all()) and torch.equal(loss, -adv)


@pytest.mark.parametrize("kind", ["step", "calls"])
def test_a_token_without_mass_is_infinitely_far_from_a_reference(kind):
    """l = -inf with a finite reference: the KL term is inf, the derivative in l -inf; the reference's -inf with a finite l
    gives inf too, and the derivative kl."""
    V, kl = 9, 0.25
    z = torch.zeros(6, V, device=DEV)
    z[:3, 3] = float("-inf")
    s = dict(logits=z, label=torch.full((6,), 3, device=DEV), old=torch.full((6,), -2.0, device=DEV),
             ref=torch.tensor([0.0, -1.0, -60.0] + [float("-inf")] * 3, device=DEV),
             adv=torch.tensor([1.0, -1.0, 0.0] * 2, device=DEV), weight=torch.ones(6, device=DEV),
             upstream=torch.ones(6, device=DEV))
    loss, logp, grad = G.run(s, kind, clip=(0.2, 0.2), kl=kl, scale=1.0)
    assert (loss == np.inf).all()
    assert (logp[:3] == -np.inf).all() and np.abs(logp[3:] + np.log(V)).max() <= 32 * G.U
    token = np.arange(V) == 3
    assert (grad[:3, token] == -np.inf).all() and (grad[:3, ~token] == np.inf).all()
    l = -np.log(V)
    slope = np.array([O.token.policy(l, -2.0, a, (0.2, 0.2))[1] for a in (1.0, -1.0, 0.0)]) + kl
    want = slope[:, None] * (token - 1.0 / V)
    assert np.abs(grad[3:] - want).max() <= 64 * G.U


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_gradient_beside_its_logits(dtype):
    """Columns of one buffer do not overlap: the gradient may lie in other columns of the logits' rows."""
    s = G.case(31, 6, 300, dtype)
    buf = torch.full((7, 2 * 300 + 7), -9.0, dtype=G.DT[dtype], device=DEV)
    z, d = buf[:6, :300], buf[:6, 304:604]
    z.copy_(s["logits"])
    want = G.run(s, "step")
    loss, logp, stats = torch.empty(6, device=DEV), torch.empty(6, device=DEV), torch.empty(6, Z.ZERO_TOKEN_STATS, device=DEV)
    kw = dict(ref_logp=s["ref"], weight=s["weight"], clip=(0.2, 0.3), kl_coef=0.1, logp=logp)
    Z.zero_policy_step(z, s["label"], s["old"], s["adv"], loss, d, upstream=s["upstream"], scale=3.0, **kw)
    torch.cuda.synchronize()
    assert all(np.array_equal(G.host(a), b) for a, b in zip((loss, logp, d), want))
    d.fill_(-9.0)
    Z.zero_policy_forward(z, s["label"], s["old"], s["adv"], loss, stats, **kw)
    Z.zero_token_backward(z, s["label"], stats, d, upstream=s["upstream"], scale=3.0)
    torch.cuda.synchronize()
    assert np.array_equal(G.host(d), G.run(s, "calls")[2])
    assert bool((buf[:, 300:304] == -9.0).all()) and bool((buf[:, 604:] == -9.0).all())
    for bad in (buf[:6, 299:599], buf[:6, 1:301], buf[1:, 299:599], buf.as_strided((6, 300), (607, 1), 308)):
        with pytest.raises(Z.ZeroError):
            Z.zero_token_backward(z, s["label"], stats, bad)
