"""GPU parity of the update of many tensors and of the 8-bit moments, bit for bit against the oracle. Every
operation of both is one fp32 rounding in a stated order, so there is no tolerance."""

import numpy as np
import pytest
import torch

import oracle as O
import zero_partition_plan_amd as Z
from gpu_util import DEV, assert_bits_equal, assert_bits_equal_nan, banner

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _memory_given_back():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


T16 = {"bf16": torch.bfloat16, "f16": torch.float16}
DT = {**T16, "f32": torch.float32}
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=5)
BLOCK = 256


def _bits16(a, dtype):
    return O.cast_bf16_rne(a) if dtype == "bf16" else O.cast_fp16_rne(a)


def _host_tensor(rng, n, bits, gdt, scale=1e-3):
    """One tensor's host arrays; 8-bit moments as (codes, scale)."""
    size = np.exp(rng.normal(0, 1, -(-n // BLOCK) or 1)).astype(np.float32).repeat(BLOCK)[:n] * np.float32(scale)
    g = rng.standard_normal(n).astype(np.float32) * size
    t = {"p": rng.standard_normal(n).astype(np.float32) * np.float32(0.02), "g": g if gdt == "f32" else _bits16(g, gdt)}
    m = rng.standard_normal(n).astype(np.float32) * size * np.float32(0.3)
    v = (rng.random(n).astype(np.float32) * size * size * np.float32(0.01))
    t["m"], t["v"] = (O.state8.encode(m, 127), O.state8.encode(O.state8.roots(v), 255)) if bits == 8 else (m, v)
    return t


class Placed:
    """A host array on the device `off` elements into a buffer whose other bytes are watched."""

    def __init__(self, a, off, view=None):
        raw = np.ascontiguousarray(a)
        self.item, self.n, self.off = raw.itemsize, raw.size, off
        self.buf = torch.full(((off + raw.size + 9) * raw.itemsize,), 0x5A, dtype=torch.uint8, device=DEV)
        lo, hi = off * raw.itemsize, (off + raw.size) * raw.itemsize
        if raw.size:
            self.buf[lo:hi] = torch.from_numpy(raw.view(np.uint8).reshape(-1).copy()).to(DEV)
        self.t = self.buf[lo:hi].view(view) if raw.size else torch.empty(0, dtype=view, device=DEV)

    def get(self, dtype):
        all_ = self.buf.cpu().numpy()
        lo, hi = self.off * self.item, (self.off + self.n) * self.item
        assert (all_[:lo] == 0x5A).all() and (all_[hi:] == 0x5A).all(), "a write outside the array"
        return all_[lo:hi].copy().view(dtype)


def _place(t, bits, gdt, out, off):
    d = {"p": Placed(t["p"], off, torch.float32), "g": Placed(t["g"], off, DT[gdt])}
    if bits == 8:
        for k, dt in (("m", torch.int8), ("v", torch.uint8)):
            d[k], d[k + "s"] = Placed(t[k][0], off, dt), Placed(t[k][1], off, torch.float32)
    else:
        d["m"], d["v"] = Placed(t["m"], off, torch.float32), Placed(t["v"], off, torch.float32)
    d["out"] = Placed(np.zeros(t["p"].size, np.uint16), off, T16[out]) if out else None
    return d


def _entry(d, group=0):
    ms, vs = d.get("ms"), d.get("vs")
    return Z.adam_tensor(d["p"].t, d["g"].t, d["m"].t, d["v"].t, out=d["out"].t if d["out"] else None,
                         m_scale=ms.t if ms else None, v_scale=vs.t if vs else None, group=group)


def _want(t, bits, gdt, gs, hp, out):
    if bits == 8:
        return O.state8.step(t["g"], gdt, gs, t["p"], t["m"], t["v"], hp, out)
    return O.sharded_step([t["g"]], gdt, gs, t["p"], t["m"], t["v"], hp, out)


def _check(d, want, bits, out, what, nan=False):
    p, m, v, o = want

    def same(got, ref, name, kind=32):
        u = np.uint32 if kind == 32 else np.uint16
        if nan:
            assert_bits_equal_nan(got.view(u), ref.view(u), f"{what} {name}", kind)
        else:
            assert_bits_equal(got.view(u), ref.view(u), f"{what} {name}")

    same(d["p"].get(np.float32), p, "param")
    if bits == 8:
        for k, (codes, scale), dt in (("m", m, np.int8), ("v", v, np.uint8)):
            same(d[k + "s"].get(np.float32), scale, k + " scale")
            assert np.array_equal(d[k].get(dt), codes), f"{what} {k} codes"
    else:
        same(d["m"].get(np.float32), m, "m")
        same(d["v"].get(np.float32), v, "v")
    if out:
        same(d["out"].get(np.uint16), o, "out", out)


@pytest.mark.parametrize("wd_mode", ["adamw", "l2"])
@pytest.mark.parametrize("out", ["bf16", "f16", None])
@pytest.mark.parametrize("gdt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bits", [8, 32])
def test_against_the_oracle(bits, gdt, out, wd_mode):
    """Sizes about a block's and a lane's ends, at offsets that put arrays off every wider boundary."""
    banner(f"tensors {bits} {gdt} {out} {wd_mode}")
    rng = np.random.default_rng(bits + len(gdt))
    sizes = [1, 2, 3, 4, 5, 63, 255, 256, 257, 511, 512, 1000, 4099, 0, 70001]
    host = [_host_tensor(rng, n, bits, gdt) for n in sizes]
    dev = [_place(t, bits, gdt, out, k % 5) for k, t in enumerate(host)]
    Z.zero_adam_tensors_step([_entry(d) for d in dev], Z.adam_hparams(wd_mode=wd_mode, **HP), 0.25)
    torch.cuda.synchronize()
    hp = O.AdamHParams(wd_mode=wd_mode, **HP)
    for n, t, d in zip(sizes, host, dev):
        if n:
            _check(d, _want(t, bits, gdt, 0.25, hp, out), bits, out, f"n={n}")


def test_many_tensors_of_both_kinds_and_three_groups():
    """More than one launch of each kind, empty entries among them, three steps in a row."""
    rng = np.random.default_rng(7)
    kinds = [(int(rng.integers(0, 1500)), 8 if rng.random() < 0.5 else 32, int(rng.integers(0, 3))) for _ in range(170)]
    hps = [dict(HP, weight_decay=w, lr=lr) for w, lr in ((0.0, 1e-3), (0.1, 1e-3), (0.01, 1e-2))]
    host = [_host_tensor(rng, n, b, "bf16") for n, b, _ in kinds]
    dev = [_place(t, b, "bf16", "bf16", k % 4) for k, (t, (_, b, _)) in enumerate(zip(host, kinds))]
    step = Z.AdamTensorsStep([_entry(d, g) for d, (_, _, g) in zip(dev, kinds)])
    for t in (5, 6, 7):
        step([Z.adam_hparams(**dict(h, step=t)) for h in hps])
    torch.cuda.synchronize()
    for t, d, (n, b, g) in zip(host, dev, kinds):
        if n == 0:
            continue
        for k in (5, 6, 7):
            p, m, v, o = _want(t, b, "bf16", 1.0, O.AdamHParams(**dict(hps[g], step=k)), "bf16")
            t.update(p=p, m=m, v=v)
        _check(d, (p, m, v, o), b, "bf16", f"n={n} bits={b} group={g}")


def test_full_width_states_end_as_the_flat_step_ends():
    rng = np.random.default_rng(11)
    t = _host_tensor(rng, 5003, 32, "bf16")
    d, e = _place(t, 32, "bf16", "f16", 1), _place(t, 32, "bf16", "f16", 0)
    hp = Z.adam_hparams(**HP)
    Z.zero_adam_tensors_step([_entry(d)], hp, 0.5)
    Z.zero_adam_shard_step([e["g"].t], 5003, 0.5, e["p"].t, e["m"].t, e["v"].t, hp, out=e["out"].t)
    torch.cuda.synchronize()
    for k, dt in (("p", np.uint32), ("m", np.uint32), ("v", np.uint32), ("out", np.uint16)):
        assert np.array_equal(d[k].get(dt), e[k].get(dt)), k


def _special(n, rng):
    x = rng.standard_normal(n).astype(np.float32)
    x[:40] = [0.0, -0.0, 1e-45, -1e-45, 1e-38, 3e38, -3e38, 1.0, 2.0 ** -126, 2.0 ** -127] * 4
    return x


@pytest.mark.parametrize("poison", [None, np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("bits", [8, 32])
def test_numbers_at_the_ends_of_fp32(bits, poison):
    """Subnormals, overflows and blocks of zeros; a gradient that is no number spoils its block of an 8-bit
    state and its element of a 32-bit one, as the oracle has it."""
    rng = np.random.default_rng(13)
    n = 2000
    t = {"p": _special(n, rng), "g": _special(n, rng)[::-1].copy()}
    t["g"][512:1024] = 0.0
    m, v = _special(n, rng) * np.float32(1e-3), np.abs(_special(n, rng)) * np.float32(1e-6)
    m[512:1024] = v[512:1024] = 0.0
    m[1024:1280], v[1024:1280], t["g"][1024:1280] = 1e-41, 1e-41, 1e-30
    if poison is not None:
        t["g"][1500] = poison
    with np.errstate(all="ignore"):
        t["m"], t["v"] = (O.state8.encode(m, 127), O.state8.encode(O.state8.roots(v), 255)) if bits == 8 else (m, v)
        d = _place(t, bits, "f32", "bf16", 2)
        Z.zero_adam_tensors_step([_entry(d)], Z.adam_hparams(**HP), 1.0)
        torch.cuda.synchronize()
        _check(d, _want(t, bits, "f32", 1.0, O.AdamHParams(**HP), "bf16"), bits, "bf16", f"{poison}", nan=True)


@pytest.mark.parametrize("bits", [8, 32])
def test_skip_and_device_scale(bits):
    rng = np.random.default_rng(17)
    t = _host_tensor(rng, 777, bits, "f16")
    d = _place(t, bits, "f16", "bf16", 3)
    flag = torch.ones(1, dtype=torch.int32, device=DEV)
    gs = torch.full((1,), 0.125, device=DEV)
    before = {k: x.buf.clone() for k, x in d.items() if x}
    Z.zero_adam_tensors_step([_entry(d)], Z.adam_hparams(**HP), gs, skip=flag)
    torch.cuda.synchronize()
    for k, x in before.items():
        assert torch.equal(x, d[k].buf), f"{k} changed on a skipped step"
    flag.zero_()
    Z.zero_adam_tensors_step([_entry(d)], Z.adam_hparams(**HP), gs, skip=flag)
    torch.cuda.synchronize()
    _check(d, _want(t, bits, "f16", 0.125, O.AdamHParams(**HP), "bf16"), bits, "bf16", "device scale")


def test_device_counter_captured_and_replayed():
    """Both kinds in one captured step whose counter, constants and scale are on the device: each replay is the
    next training step; a skipped one does not count, and one past the table writes nothing and says so."""
    rng = np.random.default_rng(19)
    kinds = [(4099, 32, 0), (700, 8, 1), (64, 8, 0), (300, 32, 1)]
    host = [_host_tensor(rng, n, b, "f32") for n, b, _ in kinds]
    dev = [_place(t, b, "f32", "bf16", 0) for t, (_, b, _) in zip(host, kinds)]
    hps = [dict(HP, weight_decay=0.1), dict(HP, weight_decay=0.0)]
    table = torch.stack([Z.adam_table(Z.adam_hparams(**h), 4, DEV) for h in hps]).contiguous()
    count = torch.ones(1, dtype=torch.int64, device=DEV)
    status, skip = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
    gs = torch.full((1,), 0.5, device=DEV)
    step = Z.AdamTensorsStep([_entry(d, g) for d, (_, _, g) in zip(dev, kinds)], skip=skip)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.dev_t(gs, table, count, status)
    noise = torch.randn(1 << 18, device=DEV)
    for t in (1, 2, 3, 4):
        if t == 3:
            skip.fill_(1)
            graph.replay()
            torch.cuda.synchronize()
            assert int(count) == 3
            skip.zero_()
        graph.replay()
        noise.mul_(0.5).add_(1.0)
        torch.cuda.synchronize()
        for h, d, (n, b, g) in zip(host, dev, kinds):
            p, m, v, o = _want(h, b, "f32", 0.5, O.AdamHParams(**dict(hps[g], step=t)), "bf16")
            h.update(p=p, m=m, v=v)
            _check(d, (p, m, v, o), b, "bf16", f"replay {t} n={n}")
        assert int(count) == t + 1 and int(status) == 0
    before = [{k: x.buf.clone() for k, x in d.items() if x} for d in dev]
    graph.replay()
    torch.cuda.synchronize()
    assert int(count) == 5 and int(status) == Z.ZERO_DEV_T_OUT_OF_TABLE
    for old, d in zip(before, dev):
        for k, x in old.items():
            assert torch.equal(x, d[k].buf), k
    Z.zero_adam_tensors_step_dev_t([], gs, table, count.fill_(2), status.zero_())       # the advance alone
    torch.cuda.synchronize()
    assert int(count) == 3 and int(status) == 0


@pytest.mark.parametrize("moment", [1, 2])
@pytest.mark.parametrize("n", [1, 3, 255, 256, 257, 5001])
def test_codes_and_values(n, moment):
    rng = np.random.default_rng(n + moment)
    x = rng.standard_normal(n).astype(np.float32) * np.exp(rng.uniform(-20, 0, n)).astype(np.float32)
    x = np.abs(x) if moment == 2 else x
    top, dt = (127, np.int8) if moment == 1 else (255, np.uint8)
    codes, scale = O.state8.encode(x if moment == 1 else O.state8.roots(x), top)
    dx, dc, ds = Placed(x, 3, torch.float32), Placed(np.zeros(n, dt), 3, getattr(torch, np.dtype(dt).name)), \
        Placed(np.zeros(scale.size, np.float32), 1, torch.float32)
    Z.zero_adam_state_codes(dx.t, dc.t, ds.t)
    torch.cuda.synchronize()
    assert np.array_equal(dc.get(dt), codes)
    assert_bits_equal(ds.get(np.uint32), scale.view(np.uint32), "scale")
    Z.zero_adam_state_values(dc.t, ds.t, dx.t)
    torch.cuda.synchronize()
    want = O.state8.decode(codes, scale, top)
    want = want * want if moment == 2 else want
    assert_bits_equal(dx.get(np.uint32), want.view(np.uint32), "values")
    Z.zero_adam_state_codes(dx.t, dc.t, ds.t)                     # what came back keeps its codes
    torch.cuda.synchronize()
    assert np.array_equal(dc.get(dt), codes)


def test_a_second_moment_below_zero_spoils_its_block():
    x = torch.ones(600, device=DEV)
    x[300] = -1.0
    codes, scale = torch.empty(600, dtype=torch.uint8, device=DEV), torch.empty(3, device=DEV)
    Z.zero_adam_state_codes(x, codes, scale)
    Z.zero_adam_state_values(codes, scale, x)
    torch.cuda.synchronize()
    assert torch.isnan(x[256:512]).all() and torch.isfinite(x[:256]).all() and torch.isfinite(x[512:]).all()


def test_a_tensor_past_one_grid_and_past_32_bits():
    """2^32 + 4099 elements of 8-bit state, whose last tiles take a second launch: every byte of the ends and of
    the place where the launches meet as a small call gives it."""
    n, cut = (1 << 32) + 4099, 1 << 32
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    p = torch.empty(n, device=DEV).normal_(0, 0.02, generator=g)
    grad = torch.empty(n, dtype=torch.bfloat16, device=DEV).normal_(0, 1e-3, generator=g)
    s = Z.adam_state(p, 8)
    parts = [slice(0, 4096), slice(cut - 4096, cut), slice(cut, n)]
    small = [(p[x].clone(), grad[x].clone(), Z.adam_state(p[x], 8)) for x in parts]
    hp = Z.adam_hparams(**HP)
    Z.zero_adam_tensors_step([Z.adam_tensor(p, grad, **s)], hp)
    Z.zero_adam_tensors_step([Z.adam_tensor(a, b, **c) for a, b, c in small], hp)
    torch.cuda.synchronize()
    for x, (a, _, c) in zip(parts, small):
        b = slice(x.start // BLOCK, -(-x.stop // BLOCK))
        for got, want in ((p[x], a), (s["m"][x], c["m"]), (s["v"][x], c["v"]), (s["m_scale"][b], c["m_scale"]),
                          (s["v_scale"][b], c["v_scale"])):
            assert torch.equal(got, want), x
    values = torch.empty(n, device=DEV)
    Z.zero_adam_state_values(s["m"], s["m_scale"], values)
    tail = torch.empty(n - cut, device=DEV)
    Z.zero_adam_state_values(s["m"][cut:], s["m_scale"][cut // BLOCK:], tail)
    torch.cuda.synchronize()
    assert torch.equal(values[cut:], tail) and bool((tail != 0).any())


def test_two_streams_and_another_device_refused():
    rng = np.random.default_rng(23)
    host = [_host_tensor(rng, 100_003, 8, "bf16") for _ in range(2)]
    dev = [_place(t, 8, "bf16", "bf16", 0) for t in host]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for d, s in zip(dev, streams):
        with torch.cuda.stream(s):
            Z.zero_adam_tensors_step([_entry(d)], Z.adam_hparams(**HP))
    torch.cuda.synchronize()
    for t, d in zip(host, dev):
        _check(d, _want(t, 8, "bf16", 1.0, O.AdamHParams(**HP), "bf16"), 8, "bf16", "streams")
    with pytest.raises((TypeError, ValueError)):
        Z.adam_tensor(torch.zeros(8), dev[0]["g"].t, dev[0]["m"].t, dev[0]["v"].t)
    with pytest.raises(TypeError):
        Z.zero_adam_tensors_step([_entry(dev[0]), Z.adam_tensor(*(torch.zeros(8, device=DEV) for _ in range(4)))],
                                 Z.adam_hparams())
    Z.zero_adam_tensors_step([], Z.adam_hparams())


def test_a_gradient_shared_by_tensors_and_a_stream_given():
    rng = np.random.default_rng(29)
    t = _host_tensor(rng, 3001, 8, "bf16")
    d, e = _place(t, 8, "bf16", "bf16", 0), _place(t, 8, "bf16", "f16", 1)
    e["out"] = _place(t, 8, "bf16", "bf16", 1)["out"]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    one = Z.adam_tensor(d["p"].t, d["g"].t, d["m"].t, d["v"].t, out=d["out"].t, m_scale=d["ms"].t, v_scale=d["vs"].t)
    two = Z.adam_tensor(e["p"].t, d["g"].t, e["m"].t, e["v"].t, out=e["out"].t, m_scale=e["ms"].t, v_scale=e["vs"].t)
    Z.zero_adam_tensors_step([one, two], Z.adam_hparams(**HP), stream=side)
    side.synchronize()
    want = _want(t, 8, "bf16", 1.0, O.AdamHParams(**HP), "bf16")
    _check(d, want, 8, "bf16", "first")
    _check(e, want, 8, "bf16", "second")
    with pytest.raises(Z.ZeroError):
        Z.zero_adam_tensors_step([one, one], Z.adam_hparams(**HP))
