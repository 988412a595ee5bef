"""GPU parity of the block boundaries against the fp64 oracle.

Bounds, with u = 2^-24: a row's sum is at most 38 additions deep (16 in a lane, 6 in a wave, 16 waves), so it is off
by 38 u of the sum of magnitudes; 1/deviation by 22 u; a normalised value by 24 u of itself, and where a mean is
taken off by 40 u of (the mean magnitude in units of the deviation) more. Following the products through the two
norms of the backward, its row coefficients are off by at most 180 u of sums of magnitudes, its results by
229 u. K = 256 stands for all of them, on the magnitudes that `sizes` forms term by term; a sum over rows adds one u
of its magnitudes for each row. Then each result's own rounding, half a step."""

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


N = O.norm
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
U = 2.0 ** -24
K = 256 * U


def host(t):
    return None if t is None else t.double().cpu().numpy()


def matrix(a, dt, off=0, pad=0):
    """A matrix `off` elements into a buffer, its rows `pad` longer; what lies between is NaN."""
    R, n = a.shape
    buf = torch.full((off + R * (n + pad) + 3,), float("nan"), dtype=dt, device=DEV)
    t = buf[off:off + R * (n + pad)].view(R, n + pad)[:, :n]
    t.copy_(torch.from_numpy(a).to(dt))
    return t


def out(R, n, dt, off, pad):
    """A matrix to write, and a check that nothing beside it changed."""
    buf = torch.full((off + R * (n + pad) + 3,), -7.0, dtype=dt, device=DEV)
    t = buf[off:off + R * (n + pad)].view(R, n + pad)[:, :n]

    def clean():
        rest = buf.clone()
        rest[off:off + R * (n + pad)].view(R, n + pad)[:, :n] = -7.0
        assert bool((rest == -7.0).all()), "a write outside the matrix"

    return t, clean


class Case:
    def __init__(self, seed, R, n, dtype="bf16", stream="bf16", post="rms", pre="rms", gate=None, gate_rows=1, bias=True,
                 weights=True, off=0, pad=0, eps=1e-5, a=0.9, c=1.1, shift=0.3):
        rng = np.random.default_rng(seed)
        self.rng, self.R, self.n, self.dtype, self.stream = rng, R, n, dtype, stream
        self.post, self.pre, self.gate_rows, self.eps = post, pre, gate_rows, float(np.float32(eps))
        self.a, self.c, self.off, self.pad = float(np.float32(a)), float(np.float32(c)), off, pad
        m = lambda s, dt: matrix(s, DT[dt], off, pad)  # noqa: E731
        v = lambda s: matrix(s[None], DT[dtype], off)[0]  # noqa: E731
        self.x = m(rng.standard_normal((R, n)) + shift, stream)
        self.branch = m(rng.standard_normal((R, n)) * 0.7 + shift, dtype)
        self.gate = m(rng.standard_normal((-(-R // gate_rows), n)) * 0.5 + 0.5, dtype) if gate else None
        self.vec = {}
        for k, kind in (("post", post), ("pre", pre)):
            on = kind != "none"
            self.vec[k + "_weight"] = v(rng.standard_normal(n) * 0.2 + 1) if on and weights else None
            self.vec[k + "_bias"] = v(rng.standard_normal(n) * 0.2) if on and bias else None

    def kw(self):
        return dict(branch=self.branch, gate=self.gate, gate_rows=self.gate_rows, post=self.post, pre=self.pre, eps=self.eps,
                    residual_scale=self.a, branch_scale=self.c, **self.vec)

    def forward(self, in_place=False):
        R, n = self.R, self.n
        y, clean_y = out(R, n, DT[self.stream], self.off, self.pad)
        h, clean_h = out(R, n, DT[self.dtype], self.off, self.pad)
        x = self.x
        if in_place:
            y.copy_(x)
            x = y
        self.stats = torch.full((R, 4), float("nan"), device=DEV)
        Z.zero_norm_forward(x, h=h if self.pre != "none" else None, y=y, stats=self.stats, **self.kw())
        torch.cuda.synchronize()
        clean_y(), clean_h()
        self.y, self.h = y, h if self.pre != "none" else None
        return self.y, self.h

    def check_forward(self):
        v = {k: host(t) for k, t in self.vec.items()}
        x, o, g = host(self.x), host(self.branch), host(self.gate)
        y = N.forward_sum(x, o, g, self.gate_rows, self.post, v["post_weight"], v["post_bias"], self.eps, self.a, self.c)
        oh, _, ro = N.normalised(o, self.post, self.eps)
        size = np.abs(oh) + (ro * np.abs(o).mean(1, keepdims=True) if self.post == "layer" else 0.0)
        w = 1.0 if v["post_weight"] is None else np.abs(v["post_weight"])
        b = 0.0 if v["post_bias"] is None else np.abs(v["post_bias"])
        gate = np.abs(N.spread(g, self.R, self.gate_rows))
        tol = K * (abs(self.a) * np.abs(x) + abs(self.c) * gate * (size * w + b)) + HALF[self.stream] * np.abs(y) + LEAST[self.stream]
        close(host(self.y), y, tol, "y")
        if self.h is None:
            return
        got_y = host(self.y)
        h = N.forward_next(got_y, self.pre, v["pre_weight"], v["pre_bias"], self.eps)
        xh, _, rp = N.normalised(got_y, self.pre, self.eps)
        size = np.abs(xh) + (rp * np.abs(got_y).mean(1, keepdims=True) if self.pre == "layer" else 0.0)
        w = 1.0 if v["pre_weight"] is None else np.abs(v["pre_weight"])
        b = 0.0 if v["pre_bias"] is None else np.abs(v["pre_bias"])
        close(host(self.h), h, K * (size * w + b) + HALF[self.dtype] * np.abs(h) + LEAST[self.dtype], "h")

    def backward(self, grad="f32", accumulate=False, dy=True, only=None, in_place=False, ws=None):
        """Runs it on random gradients; what it leaves is checked by check_backward."""
        R, n, rng = self.R, self.n, self.rng
        gdt = DT[grad]
        self.dy = matrix(rng.standard_normal((R, n)), DT[self.stream], self.off, self.pad) if dy else None
        self.dh = matrix(rng.standard_normal((R, n)), DT[self.dtype], self.off, self.pad) if self.pre != "none" else None
        dy_host = host(self.dy)
        grads, clean, was = {}, [], {}
        names = ["dx", "dbranch"] + (["dgate"] if self.gate is not None else []) + ["d" + k for k, t in self.vec.items() if t is not None]
        for k in names:
            if only is not None and k not in only:
                continue
            shape = (R, n) if k in ("dx", "dbranch") else tuple(self.gate.shape) if k == "dgate" else (1, n)
            dt = DT[self.stream] if k == "dx" else DT[self.dtype] if k == "dbranch" else gdt
            t, c = out(*shape, dt, self.off, self.pad if len(shape) == 2 and shape[0] > 1 else 0)
            clean.append(c)
            if k not in ("dx", "dbranch") and accumulate:
                t.copy_(torch.from_numpy(rng.standard_normal(shape)).to(dt))
                was[k] = host(t)
            grads[k] = t if k in ("dx", "dbranch", "dgate") else t[0]
        if in_place:
            grads["dx"].copy_(self.dy)
            self.dy = grads["dx"]
        need = Z.zero_norm_workspace_bytes(R, n, gate_rows=self.gate_rows)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws
        Z.zero_norm_backward(self.y if self.pre != "none" else None, self.stats, dy=self.dy, dh=self.dh, workspace=ws,
                             accumulate=accumulate, **grads, **self.kw())
        torch.cuda.synchronize()
        for c in clean:
            c()
        self.grads, self.was, self.grad, self.dy_host = grads, was, grad, dy_host
        return {k: host(t) for k, t in grads.items()}

    def check_backward(self):
        v = {k: host(t) for k, t in self.vec.items()}
        o, g, y, dh = host(self.branch), host(self.gate), host(self.y), host(self.dh)
        want = N.backward(y, self.dy_host, dh, o, g, self.gate_rows, self.post, v["post_weight"], v["post_bias"], self.pre,
                          v["pre_weight"], self.eps, self.a, self.c)
        size = self.sizes(v, o, g, y, dh)
        for k, t in self.grads.items():
            ref, tol, half = want[k], K * size[k], HALF[self.stream if k == "dx" else self.dtype if k == "dbranch" else self.grad]
            least = LEAST[self.stream if k == "dx" else self.dtype if k == "dbranch" else self.grad]
            if k not in ("dx", "dbranch"):
                tol = tol + U * self.R * size[k]
            if k in self.was:
                old = self.was[k].reshape(ref.shape)
                ref = ref + old
                tol = tol + U * np.abs(old)
            close(host(t), ref, tol + half * np.abs(ref) + least, k)

    def sizes(self, v, o, g, y, dh):
        """The magnitudes that each gradient is a sum of."""
        mag = lambda t: 1.0 if t is None else np.abs(t)  # noqa: E731
        mean = lambda t: np.broadcast_to(t, o.shape).mean(1, keepdims=True)  # noqa: E731
        D = np.zeros(o.shape) if self.dy_host is None else np.abs(self.dy_host)
        out = {}
        if self.pre != "none":
            xh, _, rp = N.normalised(y, self.pre, self.eps)
            xs = np.abs(xh) + (rp * np.abs(y).mean(1, keepdims=True) + 1 if self.pre == "layer" else 0.0)
            gh = np.abs(dh) * mag(v["pre_weight"])
            D = D + rp * (gh + (mean(gh) if self.pre == "layer" else 0.0) + xs * mean(gh * xs))
            out["dpre_weight"], out["dpre_bias"] = (np.abs(dh) * xs).sum(0), np.abs(dh).sum(0)
        out["dx"] = abs(self.a) * D
        oh, _, ro = N.normalised(o, self.post, self.eps)
        os_ = np.abs(oh) + (ro * np.abs(o).mean(1, keepdims=True) + 1 if self.post == "layer" else 0.0)
        bias = 0.0 if v["post_bias"] is None else np.abs(v["post_bias"])
        each = abs(self.c) * D * (os_ * mag(v["post_weight"]) + bias)
        if g is not None:
            out["dgate"] = np.zeros(g.shape)
            np.add.at(out["dgate"], np.arange(self.R) // self.gate_rows, each)
        e = abs(self.c) * np.abs(N.spread(g, self.R, self.gate_rows)) * D
        out["dpost_weight"], out["dpost_bias"] = (e * os_).sum(0), e.sum(0)
        e = e * mag(v["post_weight"])
        out["dbranch"] = e if self.post == "none" else ro * (e + (mean(e) if self.post == "layer" else 0.0) + os_ * mean(e * os_))
        return out


def close(got, want, tol, what):
    got = got.reshape(want.shape)
    with np.errstate(invalid="ignore"):
        ok = (np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)) | (got == want)
    at = np.argwhere(~ok)
    assert ok.all(), (what, len(at), at[:3].tolist(), got[~ok][:3], want[~ok][:3], np.broadcast_to(tol, got.shape)[~ok][:3])


SIZES = [(1, 1), (2, 7), (5, 8), (3, 64), (4, 513), (7, 768), (33, 1000), (3, 1025), (5, 2048), (3, 4096), (2, 5121), (2, 8192),
         (3, 8200), (2, 12288), (2, 16384), (2, 16383), (700, 96), (300, 2050)]


@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("rms", "none"), ("layer", "rms"), ("none", "layer")])
@pytest.mark.parametrize("R,n", SIZES)
def test_against_the_oracle(R, n, post, pre):
    banner(f"norm R={R} n={n} {post} {pre}")
    for dtype, stream, gate in (("bf16", "bf16", None), ("f16", "f32", "channel"), ("bf16", "f32", "token"), ("f16", "f16", "sequence")):
        per = {None: 1, "channel": R, "token": 1, "sequence": max(2, R // 3)}[gate]
        c = Case(R + n, R, n, dtype, stream, post, pre, gate, per, bias=gate != "token", weights=gate != "sequence")
        c.forward()
        c.check_forward()
        c.backward("f32" if stream == "f32" else dtype)
        c.check_backward()


@pytest.mark.parametrize("per", [1, 2, 3, 5, 16, 17, 64, 100, 299, 300, 1000])
@pytest.mark.parametrize("n", [40, 1100, 4100])
def test_gates_shared_by_any_number_of_rows(n, per):
    """Segments shorter and longer than what a block takes, the last one short."""
    banner(f"norm gates n={n} per={per}")
    c = Case(per, 1301 if n < 2000 else 601, n, "bf16", "bf16", "rms", "rms", "gate", per)
    c.forward()
    c.check_forward()
    for acc in (False, True):
        c.backward("bf16" if acc else "f32", accumulate=acc)
        c.check_backward()


@pytest.mark.parametrize("off,pad", [(1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("dtype,stream", [("bf16", "bf16"), ("f16", "f32")])
def test_offsets_strides_in_place_and_accumulated(dtype, stream, off, pad):
    for gate, per in ((None, 1), ("channel", 9), ("token", 1)):
        c = Case(off, 9, 779, dtype, stream, "layer", "rms", gate, per, off=off, pad=pad)
        y, h = (t.clone() for t in c.forward())
        c.check_forward()
        y2, h2 = c.forward(in_place=True)
        assert torch.equal(y, y2) and torch.equal(h, h2)
        c.backward("f32", accumulate=True)
        c.check_backward()
        c.backward(dtype, in_place=True)
        c.check_backward()


@pytest.mark.parametrize("gate,per", [(None, 1), ("channel", 60), ("token", 1), ("sequence", 7)])
@pytest.mark.parametrize("n", [8200, 12289])
def test_wide_rows_in_place_and_accumulated(n, gate, per):
    """Rows whose sums are formed apart read dy after the rows' own pass: dx may still be dy."""
    c = Case(n, 60, n, "bf16", "bf16", "layer", "rms", gate, per)
    c.forward()
    c.backward("f32", accumulate=True)
    c.check_backward()
    c.backward("bf16", in_place=True)
    c.check_backward()
    c.backward(only=["dx", "dpre_weight"], in_place=True)
    c.check_backward()


def test_any_subset_of_the_gradients():
    c = Case(5, 50, 300, "bf16", "f32", "layer", "layer", "channel", 50)
    c.forward()
    for only in (["dx"], ["dbranch"], ["dgate"], ["dpost_bias"], ["dpre_weight", "dpre_bias"], ["dx", "dpost_weight"]):
        c.backward(only=only)
        c.check_backward()
    c.backward(only=["dx", "dbranch"], ws=torch.empty(0, dtype=torch.uint8, device=DEV))   # needs no workspace
    c.check_backward()
    c.backward(dy=False)
    c.check_backward()


def test_a_pre_norm_alone():
    rng = np.random.default_rng(7)
    for kind, stream in (("rms", "bf16"), ("layer", "f32")):
        x = matrix(rng.standard_normal((6, 500)) + 0.2, DT[stream])
        w, b = (torch.from_numpy(rng.standard_normal(500)).to(DEV, torch.bfloat16) for _ in range(2))
        h, stats = torch.empty(6, 500, dtype=torch.bfloat16, device=DEV), torch.empty(6, 4, device=DEV)
        Z.zero_norm_forward(x, h=h, pre=kind, pre_weight=w, pre_bias=b, stats=stats, residual_scale=0.5)
        dh = matrix(rng.standard_normal((6, 500)), torch.bfloat16)
        dx, dw = torch.empty_like(x).contiguous(), torch.empty(500, device=DEV)
        ws = torch.empty(Z.zero_norm_workspace_bytes(6, 500), dtype=torch.uint8, device=DEV)
        Z.zero_norm_backward(x, stats, dh=dh, pre=kind, pre_weight=w, pre_bias=b, dx=dx, dpre_weight=dw, workspace=ws,
                             residual_scale=0.5)
        torch.cuda.synchronize()
        want = N.forward_next(host(x), kind, host(w), host(b), 1e-5)
        size = np.abs(want) + np.abs(host(b)) + np.abs(host(w)) * 2
        close(host(h), want, K * size + HALF["bf16"] * np.abs(want), "h")
        ref = N.backward(host(x), None, host(dh), None, None, 1, "none", None, None, kind, host(w), 1e-5, 0.5, 1.0)
        close(host(dx), ref["dx"], K * (np.abs(host(dh) * host(w)) + 30) + HALF[stream] * np.abs(ref["dx"]), "dx")
        close(host(dw), ref["dpre_weight"], (K + 6 * U) * (np.abs(host(dh)) * 5).sum(0) + U * np.abs(ref["dpre_weight"]), "dw")


def test_rows_of_zeros_of_one_value_and_far_numbers():
    n = 600
    for post, pre in (("rms", "rms"), ("layer", "layer")):
        c = Case(9, 8, n, "bf16", "f32", post, pre, "channel", 8, eps=1e-6)
        c.branch[0], c.x[0] = 0.0, 0.0
        c.branch[1], c.x[1] = 3.0, -2.0
        c.branch[2] *= 1e-18
        c.branch[3] *= 1e15
        c.x[4] *= 1e6
        c.x[5, 7] = 1e4
        c.forward()
        c.check_forward()
        c.backward()
        c.check_backward()
        c.x[6, 3] = float("nan")
        c.branch[7, 599] = float("inf")
        y, h = c.forward()
        torch.cuda.synchronize()
        assert torch.isnan(h[6]).all() and torch.isnan(y[6]).sum() == 1
        assert not torch.isfinite(y[7]).all() and torch.isfinite(y[:6]).all() and torch.isfinite(h[:6]).all()


def test_no_rows_zero_the_sums_and_leave_them_with_accumulate():
    e = torch.empty(0, 70, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(70, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((70,), 5.0, device=DEV)
    kw = dict(branch=e, post="rms", post_weight=w, pre="rms", pre_weight=w, dpre_weight=dw)
    Z.zero_norm_backward(e, torch.empty(0, 4, device=DEV), dh=e, accumulate=True, **kw)
    torch.cuda.synchronize()
    assert bool((dw == 5.0).all())
    Z.zero_norm_backward(e, torch.empty(0, 4, device=DEV), dh=e, **kw)
    torch.cuda.synchronize()
    assert bool((dw == 0.0).all())
    Z.zero_norm_forward(e, h=e, branch=e, y=e)


def test_captured_replayed_repeated_and_on_two_streams():
    c = Case(11, 900, 1100, "bf16", "bf16", "rms", "layer", "gate", 50)
    c.forward()
    first = c.backward()
    ws = [torch.empty(Z.zero_norm_workspace_bytes(900, 1100, gate_rows=50), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [dict(y=torch.empty_like(c.x), h=torch.empty_like(c.branch), st=torch.empty(900, 4, device=DEV),
                 g={k: torch.empty_like(t) for k, t in c.grads.items()}) for _ in range(3)]

    def both(o, w):
        Z.zero_norm_forward(c.x, h=o["h"], y=o["y"], stats=o["st"], **c.kw())
        Z.zero_norm_backward(o["y"], o["st"], dy=c.dy, dh=c.dh, workspace=w, **o["g"], **c.kw())

    both(outs[0], ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(outs[1], ws[0])
    keep = c.x.clone()
    for k in range(3):
        c.x.copy_(keep * (1 + k))
        both(outs[0], ws[0])
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both(outs[2], ws[1])
        torch.cuda.current_stream().wait_stream(side)
        both(outs[0], ws[0])
        torch.cuda.synchronize()
        for o in outs[1:]:
            for name in ("y", "h", "st"):
                assert torch.equal(o[name], outs[0][name]), (k, name)
            for name, t in o["g"].items():
                assert torch.equal(t, outs[0]["g"][name]), (k, name)
    for name, t in outs[0]["g"].items():
        assert torch.isfinite(t).all(), name
    assert set(first) == set(outs[0]["g"])


def test_streams_past_32_bits():
    """More than 2^32 bytes in each array: the last rows as a small call gives them."""
    R, n = 140_000, 16384
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.empty(R, n, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    o = torch.empty(R, n, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    y, h, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(R, 4, device=DEV)
    Z.zero_norm_forward(x, h=h, y=y, branch=o, post="rms", stats=stats)
    tail = slice(R - 5, R)
    y2, h2, s2 = torch.empty(5, n, dtype=torch.bfloat16, device=DEV), torch.empty(5, n, dtype=torch.bfloat16, device=DEV), \
        torch.empty(5, 4, device=DEV)
    Z.zero_norm_forward(x[tail], h=h2, y=y2, branch=o[tail], post="rms", stats=s2)
    torch.cuda.synchronize()
    assert torch.equal(y[tail], y2) and torch.equal(h[tail], h2) and torch.equal(stats[tail], s2)
    dx, do, dx2, do2 = torch.empty_like(x), h, torch.empty_like(y2), torch.empty_like(h2)
    dh = o.clone()
    Z.zero_norm_backward(y, stats, dy=x, dh=dh, branch=o, post="rms", dx=dx, dbranch=do)
    Z.zero_norm_backward(y2, s2, dy=x[tail], dh=dh[tail], branch=o[tail], post="rms", dx=dx2, dbranch=do2)
    torch.cuda.synchronize()
    assert torch.equal(dx[tail], dx2) and torch.equal(do[tail], do2)


def test_more_rows_than_one_grid_dimension_holds():
    R, n = (1 << 20) + 37, 40
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x, o, dy, dh = (torch.empty(R, n, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(4))
    gate = torch.empty(-(-R // 1000), n, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    kw = dict(branch=o, gate=gate, gate_rows=1000, post="rms", pre="layer")
    y, h, st = torch.empty_like(x), torch.empty_like(x), torch.empty(R, 4, device=DEV)
    Z.zero_norm_forward(x, h=h, y=y, stats=st, **kw)
    dx, do, dg = torch.empty_like(x), torch.empty_like(x), torch.empty(gate.shape, device=DEV)
    ws = torch.empty(Z.zero_norm_workspace_bytes(R, n, gate_rows=1000), dtype=torch.uint8, device=DEV)
    Z.zero_norm_backward(y, st, dy=dy, dh=dh, dx=dx, dbranch=do, dgate=dg, workspace=ws, **kw)
    first = R // 1000 * 1000                                # the last gate's rows, alone
    t = slice(first, R)
    kw.update(branch=o[t], gate=gate[first // 1000:])
    y2, h2, st2 = torch.empty_like(x[t]), torch.empty_like(x[t]), torch.empty(R - first, 4, device=DEV)
    Z.zero_norm_forward(x[t], h=h2, y=y2, stats=st2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y[t], y2) and torch.equal(h[t], h2) and torch.equal(st[t], st2)
    dx2, do2, dg2 = torch.empty_like(y2), torch.empty_like(y2), torch.empty(1, n, device=DEV)
    Z.zero_norm_backward(y2, st2, dy=dy[t], dh=dh[t], dx=dx2, dbranch=do2, dgate=dg2, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert torch.equal(dx[t], dx2) and torch.equal(do[t], do2)
    # sums of up to 48 rows in another order: 48 u of their magnitudes
    xh, _, _ = N.normalised(host(o[t]), "rms", 1e-5)
    size = (np.abs(host(dx2)) * (np.abs(xh) + 1)).sum(0)
    close(host(dg)[-1], host(dg2)[0], (K + 64 * U) * size, "dgate")


def test_columns_of_one_buffer_and_a_stream_given():
    """Slices of one buffer's columns do not overlap; work goes to the stream that is given."""
    c = Case(13, 30, 64, "bf16", "bf16", "rms", "rms")
    y, h = (t.clone() for t in c.forward())
    buf = torch.zeros(30, 4 * 64, dtype=torch.bfloat16, device=DEV)
    x, o, y2, h2 = buf.split(64, 1)
    x.copy_(c.x)
    o.copy_(c.branch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kw = {**c.kw(), "branch": o}
    Z.zero_norm_forward(x, h=h2, y=y2, stream=side, **kw)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2)
    with pytest.raises(Z.ZeroError):
        Z.zero_norm_forward(x, h=buf[:, 96:160], y=y2, **kw)     # half in the branch, half in y
