"""GPU parity of the linear layer (forward and backward).

Two kinds of check. With small whole numbers every product and sum is exact in fp32 whatever the
order, so the result must equal the 64-bit result rounded once, bit for bit, at every size, offset
and stride. With ordinary values the bound is worked out per element: (K + 8) * 2^-23 times the sum
of |terms| for an fp32 sum of K exact products in any order (each addition off by at most 2^-23
relative to a partial sum, truncation allowed), carried through the activation (slope at most 1.13),
plus 2^-20 of the activation's operands for its fp32 evaluation, plus the final half step."""

import numpy as np
import pytest
import torch

import oracle as O
import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu
L = O.layer

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


class Placed:
    """A (rows, cols) matrix inside a larger buffer: `off` elements in, leading dimension cols + pad,
    the rest filled with a canary that must survive."""

    def __init__(self, rows, cols, dtype, off=0, pad=0, fill=-77.0):
        pad = 16 - cols % 8 if pad == "to 8" else pad
        self.rows, self.cols, self.ld, self.off, self.fill = rows, cols, cols + pad, off, fill
        self.buf = torch.full((off + rows * self.ld + 9,), fill, dtype=dtype, device=DEV)
        self.t = self.buf[off:off + rows * self.ld].view(rows, self.ld)[:, :cols]

    def set(self, values):
        self.t.copy_(torch.as_tensor(values).to(self.buf.dtype))
        return self

    def check_canary(self, what):
        keep = torch.ones_like(self.buf, dtype=torch.bool)
        keep[self.off:self.off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = False
        assert bool((self.buf[keep] == self.fill).all()), f"{what}: write outside the matrix"


def ints(g, rows, cols, most=3):
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device=DEV).double()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def ws(m, k, n, back=False):
    need = Z.zero_linear_workspace_bytes(m, k, n, back)
    return torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV) if need else None


def same(got, want64, what):
    want = want64.float().to(got.dtype)          # exact in fp32, rounded once
    torch.cuda.synchronize()
    bad = (got != want).nonzero()
    assert bad.numel() == 0, f"{what}: {len(bad)} differ, first at {bad[0].tolist()}: " \
                             f"{got[tuple(bad[0])].item()} != {want[tuple(bad[0])].item()}"


SIZES = [(1, 1, 1), (1, 64, 64), (2, 8, 3), (7, 33, 5), (16, 128, 64), (17, 96, 130), (1, 4096, 257), (3, 1000, 1001),
         (33, 256, 255), (64, 64, 64), (65, 72, 136), (127, 129, 128), (128, 640, 384), (200, 333, 77),
         (256, 256, 256), (257, 520, 263), (300, 2048, 40), (1000, 88, 1003), (512, 768, 512), (1030, 1024, 776)]
# (element offset, padding of each row; "to 8": up to a multiple of 8 beyond the row)
PLACES = [(0, 0), (8, 8), (1, 0), (3, 5), (8, "to 8"), (2, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("m,k,n", SIZES)
def test_forward_whole_numbers(m, k, n, place, dtype):
    banner(f"linear forward m={m} k={k} n={n} place={place} {dtype}")
    off, pad = place
    dt, g = DT[dtype], gen(m * 7 + k * 3 + n)
    x = Placed(m, k, dt, off, pad, fill=float("nan")).set(ints(g, m, k))
    w = Placed(n, k, dt, off, 0, fill=float("nan")).set(ints(g, n, k))
    b = Placed(1, n, dt, off, 0, fill=float("nan")).set(ints(g, 1, n))
    r = Placed(m, n, dt, off, pad, fill=float("nan")).set(ints(g, m, n, 50))
    y, pre = Placed(m, n, dt, off, pad), Placed(m, n, dt, off, pad)
    z = x.t.double().cpu() @ w.t.double().cpu().t() + b.t.double().cpu()
    z = z.to(DEV)
    for kw, want in ((dict(), z - b.t.double()), (dict(bias=b.t[0]), z),
                     (dict(bias=b.t[0], residual=r.t, act="relu", pre=pre.t), z.clamp_min(0) + r.t.double())):
        Z.zero_linear_forward(x.t, w.t, y.t, workspace=ws(m, k, n), **kw)
        same(y.t, want, "y")
        y.check_canary("y")
    same(pre.t, z, "pre")
    pre.check_canary("pre")
    Z.zero_linear_forward(x.t, w.t, r.t, bias=b.t[0], residual=r.t, workspace=ws(m, k, n))   # in place
    if float((z.abs().max())) < 200:                   # a residual of at most 50 added exactly
        same(r.t, want - z.clamp_min(0) + z, "y in place of the residual")


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("m,k,n", SIZES)
def test_backward_whole_numbers(m, k, n, place, dtype, grad):
    banner(f"linear backward m={m} k={k} n={n} place={place} {dtype} grad {grad}")
    off, pad = place
    dt, gdt, g = DT[dtype], {"f32": torch.float32, **DT}[grad], gen(m + k + n)
    x = Placed(m, k, dt, off, pad, fill=float("nan")).set(ints(g, m, k))
    w = Placed(n, k, dt, off, 0, fill=float("nan")).set(ints(g, n, k))
    dy = Placed(m, n, dt, off, pad, fill=float("nan")).set(ints(g, m, n))
    dx = Placed(m, k, dt, off, pad)
    dw, db = Placed(n, k, gdt, off), Placed(1, n, gdt, off)
    d, xd, wd = dy.t.double().cpu(), x.t.double().cpu(), w.t.double().cpu()
    want_dx, want_dw, want_db = (d @ wd).to(DEV), (d.t() @ xd).to(DEV), d.sum(0).to(DEV)
    call = dict(dx=dx.t, dweight=dw.t, dbias=db.t[0], workspace=ws(m, k, n, True))
    Z.zero_linear_backward(dy.t, x.t, w.t, **call)
    same(dx.t, want_dx, "dx")
    same(dw.t, want_dw, "dweight")
    same(db.t[0], want_db, "dbias")
    dw.t.copy_(ints(g, n, k, 40))
    db.t.copy_(ints(g, 1, n, 40))
    want_dw, want_db = want_dw + dw.t.double(), want_db + db.t[0].double()
    Z.zero_linear_backward(dy.t, x.t, w.t, accumulate=True, **call)
    same(dw.t, want_dw, "accumulated dweight")
    same(db.t[0], want_db, "accumulated dbias")
    dz = Placed(m, n, dt, off, pad)
    pre = Placed(m, n, dt, off, pad, fill=float("nan")).set(ints(g, m, n))
    Z.zero_linear_backward(dy.t, x.t, w.t, act="relu", pre=pre.t, dz=dz.t, **call)
    d = d * (pre.t.double().cpu() > 0)
    same(dz.t, d.to(DEV), "dz")
    same(dx.t, (d @ wd).to(DEV), "dx behind relu")
    same(dw.t, (d.t() @ xd).to(DEV), "dweight behind relu")
    same(db.t[0], d.sum(0).to(DEV), "dbias behind relu")
    for p, what in ((dx, "dx"), (dw, "dweight"), (db, "dbias"), (dz, "dz")):
        p.check_canary(what)


@pytest.mark.parametrize("m,k,n", [(4100, 4097, 4099), (4100, 4104, 4099), (4100, 4097, 4096), (9000, 771, 5003)])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 1), (8, "to 8")])
def test_large_odd_sizes(m, k, n, off, pad):
    """Sizes at which rows off 16 bytes are copied before the products; whole numbers, exact in fp32."""
    banner(f"linear large odd m={m} k={k} n={n} off={off} pad={pad}")
    dt, g = torch.bfloat16, gen(m + k + n)
    nan = float("nan")
    x = Placed(m, k, dt, off, pad, nan).set(ints(g, m, k))
    w = Placed(n, k, dt, off, 0, nan).set(ints(g, n, k))
    dy = Placed(m, n, dt, off, pad, nan).set(ints(g, m, n))
    y, dx, dw, db = Placed(m, n, dt, off, pad), Placed(m, k, dt, off, pad), Placed(n, k, torch.float32, off), Placed(1, n, torch.float32, off)
    Z.zero_linear_forward(x.t, w.t, y.t, workspace=ws(m, k, n))
    Z.zero_linear_backward(dy.t, x.t, w.t, dx=dx.t, dweight=dw.t, dbias=db.t[0], workspace=ws(m, k, n, True))
    X, W, D = x.t.float().contiguous(), w.t.float().contiguous(), dy.t.float().contiguous()
    same(y.t, X @ W.t(), "y")
    same(dx.t, D @ W, "dx")
    same(dw.t, D.t() @ X, "dweight")
    same(db.t[0], D.sum(0), "dbias")
    for p, what in ((y, "y"), (dx, "dx"), (dw, "dweight"), (db, "dbias")):
        p.check_canary(what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", L.ACTS)
@pytest.mark.parametrize("m,k,n", [(5, 64, 48), (70, 200, 131), (257, 512, 264)])
def test_forward_and_dz_ordinary_values(m, k, n, kind, dtype):
    banner(f"linear values m={m} k={k} n={n} {kind} {dtype}")
    dt, rng = DT[dtype], np.random.default_rng(m + n)
    t = {name: torch.from_numpy(rng.standard_normal(s)).to(dt).to(DEV)
         for name, s in (("x", (m, k)), ("b", (n,)), ("r", (m, n)), ("dy", (m, n)))}
    t["w"] = torch.from_numpy(rng.standard_normal((n, k)) * 2 / np.sqrt(k)).to(dt).to(DEV)
    h = {name: a.double().cpu().numpy() for name, a in t.items()}
    y, pre, dz = (torch.empty(m, n, dtype=dt, device=DEV) for _ in range(3))
    Z.zero_linear_forward(t["x"], t["w"], y, bias=t["b"], residual=t["r"], act=kind, pre=pre, workspace=ws(m, k, n))
    torch.cuda.synchronize()
    want_y, want_z = L.linear_forward(h["x"], h["w"], h["b"], h["r"], kind)
    terms = np.abs(h["x"]) @ np.abs(h["w"]).T + np.abs(h["b"])
    ez = (k + 8) * 2.0 ** -23 * terms
    half = HALF_STEP[dt]
    err = np.abs(pre.double().cpu().numpy() - want_z)
    assert (err <= ez + half * (np.abs(want_z) + ez) + TINY[dt]).all(), "pre"
    ey = 1.13 * ez + 2.0 ** -20 * (np.abs(want_z) + np.abs(h["r"]))
    err = np.abs(y.double().cpu().numpy() - want_y)
    assert (err <= ey + half * (np.abs(want_y) + ey) + TINY[dt]).all(), "y"
    if kind == "none":
        return
    p64 = pre.double().cpu().numpy()
    want = h["dy"] * L.act_slope(p64, kind)
    e = 2.0 ** -20 * np.abs(h["dy"]) * (1 + np.abs(p64))
    for out, src in ((dz, t["dy"]), (None, None), (None, pre)):          # apart, over dy, over pre
        d_y = t["dy"].clone() if out is None and src is None else t["dy"]
        p = pre.clone() if src is pre else pre
        o = out if out is not None else (d_y if src is None else p)
        Z.zero_linear_backward(d_y, t["x"], t["w"], act=kind, pre=p, dz=o, workspace=ws(m, k, n, True))
        torch.cuda.synchronize()
        err = np.abs(o.double().cpu().numpy() - want)
        assert (err <= e + half * (np.abs(want) + e) + TINY[dt]).all(), "dz"


@pytest.mark.parametrize("kind", L.ACTS)
def test_gradients_against_differences(kind):
    """dx, dweight, dbias of sum(dy * y) against central differences of the oracle's forward on the
    kernel's own (16-bit) inputs, fp32 parameter gradients. dz is rounded to 16 bits (half a step of
    2^-11 each) and pre too, so a gradient is off by at most 2^-10 of its sum of |terms| (the slope's
    own slope is at most 1.1, times |pre| * 2^-11), besides the differences' own error."""
    m, k, n = 6, 24, 9
    rng = np.random.default_rng(11)
    x, w, b, dy = (torch.from_numpy(rng.uniform(0.2, 1.0, s) * rng.choice([-1, 1], s)).half().to(DEV)
                   for s in ((m, k), (n, k), (n,), (m, n)))
    y, pre, dz = (torch.empty(m, n, dtype=torch.float16, device=DEV) for _ in range(3))
    dx = torch.empty(m, k, dtype=torch.float16, device=DEV)
    dw, db = torch.empty(n, k, device=DEV), torch.empty(n, device=DEV)
    Z.zero_linear_forward(x, w, y, bias=b, act=kind, pre=pre, workspace=ws(m, k, n))
    Z.zero_linear_backward(dy, x, w, act=kind, pre=pre, dz=dz, dx=dx, dweight=dw, dbias=db, workspace=ws(m, k, n, True))
    torch.cuda.synchronize()
    X, W, B, D = (t.double().cpu().numpy() for t in (x, w, b, dy))

    def f(X, W, B):
        return (D * L.linear_forward(X, W, B, None, kind)[0]).sum()

    step = 1e-5
    zmax = np.abs(L.linear_forward(X, W, B)[1]).max()
    slack = 2.0 ** -10 * (1 + 1.1 * zmax) * 1.2
    for got, arr, terms in ((dx, X, np.abs(D) @ np.abs(W)), (dw, W, np.abs(D).T @ np.abs(X)), (db, B, np.abs(D).sum(0))):
        got = got.double().cpu().numpy()
        for at in np.ndindex(arr.shape):
            old = arr[at]
            arr[at] = old + step
            hi = f(X, W, B)
            arr[at] = old - step
            lo = f(X, W, B)
            arr[at] = old
            assert abs(got[at] - (hi - lo) / (2 * step)) <= slack * terms[at] + 1e-6, (at, kind)


def test_empty_sums_and_empty_sides():
    for dt in DT.values():
        x, w = torch.empty(5, 0, dtype=dt, device=DEV), torch.empty(7, 0, dtype=dt, device=DEV)
        b, r = (torch.arange(s, device=DEV).to(dt) for s in (7, 35))
        y = torch.empty(5, 7, dtype=dt, device=DEV)
        Z.zero_linear_forward(x, w, y, bias=b, residual=r.view(5, 7), workspace=ws(5, 0, 7))
        same(y, b.double() + r.view(5, 7).double(), "no features in")
        dw, db = torch.full((7, 6), 3.0, device=DEV), torch.full((7,), 3.0, device=DEV)
        e = torch.empty(0, 7, dtype=dt, device=DEV)
        x0, w6 = torch.empty(0, 6, dtype=dt, device=DEV), torch.ones(7, 6, dtype=dt, device=DEV)
        Z.zero_linear_backward(e, x0, w6, dweight=dw, dbias=db, accumulate=True, workspace=ws(0, 6, 7, True))
        torch.cuda.synchronize()
        assert bool((dw == 3).all()) and bool((db == 3).all())
        Z.zero_linear_backward(e, x0, w6, dweight=dw, dbias=db, workspace=ws(0, 6, 7, True))
        torch.cuda.synchronize()
        assert bool((dw == 0).all()) and bool((db == 0).all())
        dx = torch.full((4, 6), 3.0, dtype=dt, device=DEV)
        Z.zero_linear_backward(torch.empty(4, 0, dtype=dt, device=DEV), torch.ones(4, 6, dtype=dt, device=DEV),
                               torch.empty(0, 6, dtype=dt, device=DEV), dx=dx, workspace=ws(4, 6, 0, True))
        torch.cuda.synchronize()
        assert bool((dx == 0).all())


@pytest.mark.parametrize("m,k,n", [(3, 40, 20), (130, 200, 140), (260, 300, 270)])
def test_nan_and_inf_stay_in_their_rows_and_columns(m, k, n):
    """A NaN in one row of x and an infinity in one row of W reach that row and that column of the
    result and nothing else, though neighbouring rows lie in the same tiles."""
    x = torch.ones(m, k, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(n, k, dtype=torch.bfloat16, device=DEV)
    x[1, k - 1], w[n - 2, 0] = float("nan"), float("inf")
    y = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    Z.zero_linear_forward(x, w, y, workspace=ws(m, k, n))
    want = torch.full((m, n), float(k), device=DEV)
    want[:, n - 2], want[1] = float("inf"), float("nan")
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(y.float(), nan=-1.0, posinf=-2.0),
                       torch.nan_to_num(want.bfloat16().float(), nan=-1.0, posinf=-2.0))
    dw = torch.empty(n, k, device=DEV)
    Z.zero_linear_backward(torch.ones(m, n, dtype=torch.bfloat16, device=DEV), x, w, dweight=dw, workspace=ws(m, k, n, True))
    torch.cuda.synchronize()
    assert bool(torch.isnan(dw[:, k - 1]).all()) and bool((dw[:, :k - 1] == m).all())


def test_column_slices_of_one_buffer():
    """x, residual and y as column slices of one buffer, all with its leading dimension."""
    g = gen(5)
    buf = torch.zeros(50, 200, dtype=torch.bfloat16, device=DEV)
    buf[:, :80] = ints(g, 50, 80).bfloat16()
    buf[:, 96:160] = ints(g, 50, 64).bfloat16()
    w = ints(g, 64, 80).bfloat16()
    want = (buf[:, :80].double().cpu() @ w.double().cpu().t()).to(DEV) + buf[:, 96:160].double()
    keep = buf[:, 160:].clone()
    Z.zero_linear_forward(buf[:, :80], w, buf[:, 96:160], residual=buf[:, 96:160], workspace=ws(50, 80, 64))
    same(buf[:, 96:160], want, "slice")
    assert torch.equal(buf[:, 160:], keep)


def test_calls_repeat_bit_for_bit_and_run_on_other_streams():
    g = gen(9)
    m, k, n = 300, 2048, 520
    x, w, dy = (torch.randn(s, generator=g, device=DEV).bfloat16() for s in ((m, k), (n, k), (m, n)))
    outs = []
    for i in range(3):
        s = torch.cuda.Stream() if i else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        y, dx, dw, db = (torch.empty(sh, dtype=torch.bfloat16, device=DEV) for sh in ((m, n), (m, k), (n, k), (n,)))
        w1, w2 = ws(m, k, n), ws(m, k, n, True)
        torch.cuda.synchronize()
        Z.zero_linear_forward(x, w, y, workspace=w1, stream=s)
        Z.zero_linear_backward(dy, x, w, dx=dx, dweight=dw, dbias=db, workspace=w2, stream=s)
        s.synchronize()
        outs.append((y, dx, dw, db))
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_device_refusals():
    x, w = (torch.zeros(4, 8, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    y = torch.zeros(4, 4, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        Z.zero_linear_forward(x, w.t().contiguous().t(), y)                    # rows not adjacent
    with pytest.raises(ValueError):
        Z.zero_linear_forward(x, torch.zeros(4, 9, dtype=torch.bfloat16, device=DEV)[:, :8], y)   # not contiguous
    with pytest.raises(Z.ZeroError):
        Z.zero_linear_forward(x, w, x[:, :4])                                  # y inside x
    with pytest.raises(Z.ZeroError):
        Z.zero_linear_forward(x[:1].expand(4, 8), w, y)                        # row stride 0
    with pytest.raises(TypeError):
        Z.zero_linear_backward(y, x, w, dweight=torch.zeros(4, 8, dtype=torch.float64, device=DEV))


def test_more_small_tiles_than_a_grid_holds():
    """A result of more than 2^35 elements (69 GB) over a short k, where small tiles would be fastest."""
    m, k, n = 131077, 8, 262148
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB")
    g = gen(9)
    x, w = ints(g, m, k).bfloat16(), ints(g, n, k).bfloat16()
    y = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    Z.zero_linear_forward(x, w, y, workspace=ws(m, k, n))
    wt = w.float().t().contiguous()
    for r in range(0, m, 8192):                    # whole numbers of at most 72: exact in bf16
        assert torch.equal(y[r:r + 8192], (x[r:r + 8192].float() @ wt).bfloat16()), r
    del y
    torch.cuda.empty_cache()


# Few tiles and a long k: a tile's steps are shared by groups of waves, and by splits whose last has one,
# two or three steps, so that a group has none, or the k ends inside a chunk of one group
SHARED = [(200, 200, 2319), (200, 2319, 200), (200, 300, 1582), (200, 1582, 300), (1582, 300, 200), (333, 256, 2404),
          (333, 2404, 256), (2404, 256, 333), (70, 523, 200), (333, 767, 2303)]


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("place", [(0, 0), (1, 0), (3, 5), (8, "to 8")])
@pytest.mark.parametrize("m,k,n", SHARED)
def test_k_shared_by_groups_and_splits(m, k, n, place, dtype, grad):
    test_forward_whole_numbers(m, k, n, place, dtype)
    test_backward_whole_numbers(m, k, n, place, dtype, grad)


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("rows", [1, 2, 8, 31, 32, 33, 64, 190, 200, 800])
def test_bias_gradient_of_any_chunks(rows, dtype, grad):
    """The bias gradient alone, written and added to, for rows of one chunk, of a few and of many."""
    n, dt, g = 523, DT[dtype], gen(rows)
    dy = Placed(rows, n, dt, 1, 3, fill=float("nan")).set(ints(g, rows, n))
    x, w = torch.zeros(rows, 8, dtype=dt, device=DEV), torch.zeros(n, 8, dtype=dt, device=DEV)
    db = Placed(1, n, DT.get(grad, torch.float32), 1)
    want = dy.t.double().sum(0, keepdim=True)       # at most 2400: exact in fp32
    Z.zero_linear_backward(dy.t, x, w, dbias=db.t[0], workspace=ws(rows, 8, n, True))
    same(db.t, want, "dbias")
    before = db.t.double().clone()
    Z.zero_linear_backward(dy.t, x, w, dbias=db.t[0], accumulate=True, workspace=ws(rows, 8, n, True))
    same(db.t, before + want, "dbias added to")
    db.check_canary("dbias")
