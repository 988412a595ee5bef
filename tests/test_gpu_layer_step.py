"""The layer operators run together with the framework's step: gather, forward, loss, backward into
replica rows, reduction, norm, clip, update, slot."""

import numpy as np
import pytest
import torch

import oracle as O
import zero_partition_plan_amd as Z
from gpu_util import DEV, assert_bits_equal, banner, bits16, bits32
from layer_chain import Chain

pytestmark = pytest.mark.gpu
NAMES = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}


def _host(t):
    t = t.detach().cpu()
    return t.numpy() if t.dtype == torch.float32 else t.view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("dtype,gdtype", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                          (torch.bfloat16, torch.float32)])
def test_training_step_of_the_librarys_calls(dtype, gdtype):
    """Gradients against fp64 automatic gradients; the update bit for bit against the oracle on the
    gradients the rows hold. A gradient passes at most 9 tensors rounded to 16 bits (pre, h, y, logits,
    dlogits, dy, dh, dz, itself), each off by at most half a step relative to it; the logits' own
    error, half a step of values of size at most 8 over T = 2, enters the softmax as a relative error
    4 times that. 12 half steps in all, in the Frobenius norm."""
    banner(f"layer step {dtype} {gdtype}")
    c = Chain(dtype=dtype, gdtype=gdtype)
    scale, S, n = 1024.0, c.plan.shard_elems, c.plan.n
    c.gather()
    half = torch.finfo(dtype).eps / 2
    for k in range(c.nd):
        c.forward_backward(k, scale)
        torch.cuda.synchronize()
        want_loss, want = c.reference(k, scale)
        assert bool(((c.loss[k].double() - want_loss).abs() <= 12 * half * (1 + want_loss.abs())).all())
        got = c.rows_of[k][:n].double()
        pos = 0
        for name, shape in c.shapes.items():
            m = torch.Size(shape).numel()
            a, b = got[pos:pos + m], want[pos:pos + m]
            assert float((a - b).norm() / b.norm()) <= 12 * half, name
            pos += m
    hp = dict(lr=1e-2, weight_decay=0.01)
    for r in range(c.nd):
        lo = r * S
        rows = [c.rows_of[k][lo:lo + S] for k in range(c.nd)]
        master = c.master[lo:lo + S].clone()
        m, v = torch.zeros(S, device=DEV), torch.zeros(S, device=DEV)
        grad, sq, gs = torch.empty(S, device=DEV), torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(1, device=DEV)
        flag = torch.zeros(1, dtype=torch.int32, device=DEV)
        Z.zero_reduce_shard_static(rows, S, grad, flag, sq, 1.0 / scale)
        Z.zero_clip_scale(sq, 1e9, 1e-6, 1.0 / scale, gs)
        Z.zero_adam_shard_step_dev_scale([grad], S, gs, master, m, v, Z.adam_hparams(step=1, **hp),
                                         out=c.full[lo:lo + S], skip=flag)
        torch.cuda.synchronize()
        assert int(flag) == 0
        acc = O.replica_sum([_host(t) for t in rows], NAMES[gdtype])
        p, m2, v2, out = O.sharded_step([acc], "f32", 1.0 / scale, c.master[lo:lo + S].cpu().numpy(),
                                        np.zeros(S, np.float32), np.zeros(S, np.float32), O.AdamHParams(step=1, **hp),
                                        NAMES[dtype])
        assert_bits_equal(bits32(master), p.view(np.uint32), "master")
        assert_bits_equal(bits16(c.full[lo:lo + S]), out, "slot")


def test_an_overflow_in_the_loss_scale_skips_the_step():
    c = Chain(dtype=torch.float16)
    c.gather()
    for k in range(c.nd):
        c.forward_backward(k, 1e9)                       # dlogits past fp16
    S = c.plan.shard_elems
    rows = [c.rows_of[k][:S] for k in range(c.nd)]
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    grad, master, m, v = (torch.zeros(S, device=DEV) for _ in range(4))
    Z.zero_reduce_shard(rows, S, grad, flag)
    Z.zero_adam_shard_step([grad], S, 1e-9, master, m, v, Z.adam_hparams(), skip=flag)
    torch.cuda.synchronize()
    assert int(flag) == 1 and not bool(master.any()) and not bool(v.any())


def test_captured_step_replays_as_eager():
    """Forward, loss and backward of every micro-batch in one graph, replayed with eager work between."""
    c = Chain(dtype=torch.bfloat16, d=128, f=512, v=2048, rows=300, seed=3)
    c.gather()
    for k in range(c.nd):
        c.forward_backward(k, 8.0)
    torch.cuda.synchronize()
    want, loss = c.rows_of.clone(), c.loss.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for k in range(c.nd):
            c.forward_backward(k, 8.0)
    noise = torch.randn(1 << 20, device=DEV)
    for i in range(4):
        c.rows_of.fill_(-1)
        c.loss.fill_(-1)
        c.ws.fill_(0xFF)                                   # holds nothing between calls
        graph.replay()
        noise.mul_(1.01)
        torch.cuda.synchronize()
        n = c.plan.n
        assert torch.equal(c.rows_of[:, :n].view(torch.int16), want[:, :n].view(torch.int16)), i
        assert torch.equal(c.loss, loss), i
        for k in range(c.nd):
            c.forward_backward(k, 8.0)                     # eager calls between replays


def test_two_streams_at_once_with_a_workspace_each():
    a, b = (Chain(dtype=torch.bfloat16, d=256, f=1024, v=4096, rows=500, seed=s) for s in (1, 2))
    want = []
    for c in (a, b):
        c.gather()
        c.forward_backward(0, 4.0)
        torch.cuda.synchronize()
        want.append(c.rows_of[0].clone())
        c.rows_of.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.forward_backward(0, 4.0)
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        assert torch.equal(c.rows_of[0].view(torch.int16), w.view(torch.int16))


def _whole(g, rows, cols, dt):
    return torch.randint(-2, 3, (rows, cols), generator=g, device=DEV).to(dt)


def test_matrices_past_32_bits():
    """Outputs and operands of more than 2^32 bytes: whole numbers, so rows and columns anywhere are exact."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    M, K, N, dt = 70_003, 72, 32_768, torch.bfloat16
    x, w = _whole(g, M, K, dt), _whole(g, N, K, dt)
    y = torch.empty(M, N, dtype=dt, device=DEV)
    banner(f"layer past 32 bits: y {M}x{N}")
    ws = torch.empty(max(Z.zero_linear_workspace_bytes(M, K, N, b) for b in (False, True)) + 16, dtype=torch.uint8, device=DEV)
    Z.zero_linear_forward(x, w, y, workspace=ws)
    at = torch.tensor([0, 1, 32_767, 32_768, 65_535, 65_536, 70_001, 70_002], device=DEV)
    want = x[at].float() @ w.float().t()
    torch.cuda.synchronize()
    assert torch.equal(y[at].float(), want)
    del want
    dy = y                                                  # reuse: small whole numbers as the gradient
    for lo in range(0, M, 10_000):
        dy[lo:lo + 10_000] = torch.randint(-1, 2, (min(10_000, M - lo), N), generator=g, device=DEV).to(dt)
    dx, dw, db = torch.empty(M, K, dtype=dt, device=DEV), torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    Z.zero_linear_backward(dy, x, w, dx=dx, dweight=dw, dbias=db, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(dx[at].float(), (dy[at].float() @ w.float()).to(dt).float())
    cols = torch.tensor([0, 5, 16_384, 32_767], device=DEV)
    part = dy[:, cols].float()
    assert torch.equal(dw[cols], part.t() @ x.float()) and torch.equal(db[cols], part.sum(0))


def test_rows_far_apart():
    """Leading dimensions past what the direct loads take: rows 2^22 and more elements apart."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    ld, dt = (1 << 22) + 8, torch.float16
    buf = torch.zeros(40 * ld, dtype=dt, device=DEV)
    x = buf.view(40, ld)[:, :64]
    x.copy_(_whole(g, 40, 64, dt))
    w = _whole(g, 100, 64, dt)
    y = torch.empty(40, 100, dtype=dt, device=DEV)
    Z.zero_linear_forward(x, w, y, workspace=None)
    dw = torch.empty(100, 64, device=DEV)
    ws = torch.empty(Z.zero_linear_workspace_bytes(40, 64, 100, True) + 16, dtype=torch.uint8, device=DEV)
    Z.zero_linear_backward(y, x, w, dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(y.float(), x.float() @ w.float().t())
    assert torch.equal(dw, y.float().t() @ x.float())


def test_distillation_past_32_bits():
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    R, V, K, dt = 70_001, 32_000, 4, torch.bfloat16
    banner(f"distill past 32 bits: {R}x{V}")
    z = torch.empty(R, V, dtype=dt, device=DEV)
    for lo in range(0, R, 10_000):
        z[lo:lo + 10_000] = torch.randn((min(10_000, R - lo), V), generator=g, device=DEV).to(dt)
    idx = torch.randint(V, (R, 1), generator=g, device=DEV).add(torch.arange(K, device=DEV) * 101) % V
    top = torch.randn(R, K, generator=g, device=DEV)
    at = torch.tensor([0, 1, 33_554, 33_555, 67_108, 67_109, 70_000], device=DEV)
    rows = z[at].double()
    loss = torch.empty(R, device=DEV)
    Z.zero_distill_step(z, idx, top, 1.0, loss, z)
    torch.cuda.synchronize()
    want, grad = O.layer.distill(rows.cpu().numpy(), idx[at].cpu().numpy(), top[at].double().cpu().numpy(), 1.0)
    assert np.abs(loss[at].double().cpu().numpy() - want).max() <= 1e-5
    err = np.abs(z[at].double().cpu().numpy() - grad)
    assert (err <= 2.0 ** -8 * np.abs(grad) + 1e-6 * (np.abs(grad) > 1e-3) + 2.0 ** -30).all()
