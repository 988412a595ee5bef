"""GPU parity of the update of many tensors over many steps, bit for bit against the oracle: what the 8-bit moments' rounding
keeps (gradients of half of the elements that fall tenfold, or stop) is the same on the device."""

import numpy as np
import pytest
import torch

import oracle as O
import test_gpu_tensor_list as G
import zero_partition_plan_amd as Z
from gpu_util import DEV, banner

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("factor", [0.1, 0.0])
def test_hundreds_of_steps_with_gradients_that_fall(factor, beta2):
    banner(f"tensor steps {factor} {beta2}")
    rng = np.random.default_rng(31)
    n, steps, at = 1500, 300, 100
    host = {bits: G._host_tensor(rng, n, bits, "f32") for bits in (8, 32)}
    dev = {bits: G._place(t, bits, "f32", "bf16", 1) for bits, t in host.items()}
    step = Z.AdamTensorsStep([G._entry(d) for d in dev.values()])
    half = rng.random(n) < 0.5
    hp = dict(G.HP, beta2=beta2)
    for t in range(1, steps + 1):
        g = rng.standard_normal(n).astype(np.float32) * np.float32(1e-3)
        g = np.where(half & (t > at), g * np.float32(factor), g)
        for bits, d in dev.items():
            d["g"].t.copy_(torch.from_numpy(g).to(DEV))
            p, m, v, out = G._want(dict(host[bits], g=g), bits, "f32", 1.0, O.AdamHParams(**dict(hp, step=t)), "bf16")
            host[bits].update(p=p, m=m, v=v)
        step(Z.adam_hparams(**dict(hp, step=t)))
        if t in (1, at, at + 1, steps):
            torch.cuda.synchronize()
            for bits, d in dev.items():
                G._check(d, (host[bits]["p"], host[bits]["m"], host[bits]["v"], out if bits == 32 else None), bits,
                         "bf16" if bits == 32 else None, f"step {t} bits={bits}")
