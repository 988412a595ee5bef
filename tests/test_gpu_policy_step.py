"""The block boundaries, the policy loss and the update of many tensors run together with the framework's step:
gather, forward, loss, backward into replica rows, reduction, norm, clip, update of every tensor, gather again."""

import numpy as np
import pytest
import torch

import oracle as O
import zero_partition_plan_amd as Z
from block_chain import BlockChain
from gpu_util import DEV, assert_bits_equal, banner, bits16, bits32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _memory_given_back():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


NAMES = {torch.float16: "f16", torch.bfloat16: "bf16"}


def _update(c, state, scale, t, hps):
    """Reduction, clip and the update of every tensor; (the reduced gradient, the grad scale)."""
    P = c.plan.padded_n
    grad, flag = torch.empty(P, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    parts, sq = torch.empty(Z.zero_sq_partials_len(P), dtype=torch.float64, device=DEV), torch.empty(1, dtype=torch.float64, device=DEV)
    gs = torch.empty(1, device=DEV)
    Z.zero_reduce_shard(c.rows_of, P, grad, flag, parts, 1.0 / scale)
    Z.zero_shard_sqnorm(None, P, 1.0 / scale, parts, sq)
    Z.zero_clip_scale(sq, 1.0, 1e-6, 1.0 / scale, gs)
    g, p, out = c.views(grad), c.views(c.master), c.views(c.full)
    step = Z.AdamTensorsStep([Z.adam_tensor(p[k], g[k], out=out[k], group=int(k not in ("w1", "w2", "head")), **state[k])
                              for k in c.shapes], skip=flag)
    step([Z.adam_hparams(step=t, **h) for h in hps], gs)
    torch.cuda.synchronize()
    assert int(flag) == 0
    return grad, float(gs)


@pytest.mark.parametrize("dtype,stream", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                          (torch.bfloat16, torch.float32)])
def test_training_steps_of_the_librarys_calls(dtype, stream):
    """Gradients against fp64 automatic gradients, two steps; the update bit for bit against the oracle on the gradients
    the rows hold, matrices with 8-bit moments and vectors with 32. A gradient passes at most 14 tensors rounded to 16
    bits (h0, pre, act, branch, y, h1, logits, dlogits, dh1, dx, dbranch, dact, dz, dh0), each off by at most half a
    step relative to it; the logits' own error, half a step of values up to 8, enters the softmax and the ratio as a
    relative error 8 times that each. 30 half steps in all, in the Frobenius norm; a row's loss has the ratio's, on
    numbers up to 1 + |its advantage| * 2."""
    banner(f"block step {dtype} {stream}")
    c = BlockChain(dtype, stream)
    scale, half = 256.0, torch.finfo(dtype).eps / 2
    hps = [dict(lr=1e-3, weight_decay=0.1), dict(lr=1e-3, weight_decay=0.0)]
    state = {k: Z.adam_state(t, 8 if k in ("w1", "w2", "head") else 32) for k, t in c.views(c.master).items()}
    for t in (1, 2):
        c.gather()
        for k in range(c.nd):
            c.behind(k)
            c.forward_backward(k, scale)
            torch.cuda.synchronize()
            loss, want, dx = c.reference(k, scale)
            assert bool(((c.loss[k].double() - loss).abs() <= 30 * half * (1 + 2 * c.batches[k]["adv"].double().abs())).all())
            assert float((c.dx.double() - dx).norm() / dx.norm()) <= 30 * half
            got, pos = c.rows_of[k][:c.n].double(), 0
            for name, shape in c.shapes.items():
                m = torch.Size(shape).numel()
                a, b = got[pos:pos + m], want[pos:pos + m]
                assert float((a - b).norm() / b.norm()) <= 30 * half, name
                pos += m
        before = {k: v.clone() for k, v in c.views(c.master).items()}
        old = {k: {n: x.cpu().numpy().copy() for n, x in s.items()} for k, s in state.items()}
        grad, gs = _update(c, state, scale, t, hps)
        assert gs < 1.0 / scale                                        # clipped
        for k, p in c.views(c.master).items():
            hp = O.AdamHParams(step=t, **hps[int(k not in ("w1", "w2", "head"))])
            args = (c.views(grad)[k].cpu().numpy().ravel(), "f32", gs, before[k].cpu().numpy().ravel())
            s = {n: x.ravel() for n, x in old[k].items()}
            if "m_scale" in s:
                p2, m2, v2, out = O.state8.step(*args, (s["m"], s["m_scale"]), (s["v"], s["v_scale"]), hp, NAMES[dtype])
                assert np.array_equal(state[k]["m"].cpu().numpy().ravel(), m2[0])
                assert np.array_equal(state[k]["v"].cpu().numpy().ravel(), v2[0])
            else:
                p2, m2, v2, out = O.sharded_step([args[0]], *args[1:], s["m"], s["v"], hp, NAMES[dtype])
                assert_bits_equal(bits32(state[k]["v"]).ravel(), v2.view(np.uint32), k)
            assert_bits_equal(bits32(p).ravel(), p2.view(np.uint32), k)
            assert_bits_equal(bits16(c.views(c.full)[k]).ravel(), out, k)


def test_captured_step_replays_as_eager():
    c = BlockChain(torch.bfloat16, torch.float32, d=128, f=512, v=2048, rows=300, seed=3)
    c.gather()
    for k in range(c.nd):
        c.behind(k)
        c.forward_backward(k, 8.0)
    torch.cuda.synchronize()
    want, loss = c.rows_of.clone(), c.loss.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for k in range(c.nd):
            c.forward_backward(k, 8.0)
    noise = torch.randn(1 << 20, device=DEV)
    for i in range(4):
        c.rows_of[:, :c.n].fill_(-1)
        c.loss.fill_(-1)
        c.ws.fill_(0xFF)                                   # holds nothing between calls
        graph.replay()
        noise.mul_(1.01)
        torch.cuda.synchronize()
        assert torch.equal(c.rows_of[:, :c.n], want[:, :c.n]) and torch.equal(c.loss, loss), i
        for k in range(c.nd):
            c.forward_backward(k, 8.0)                     # eager calls between replays
