"""A training step of a policy made of the library's calls: gather, a pre norm, a two-layer MLP, the block boundary
(post norm, gate, residual scale, the head's norm), a head, the clipped policy loss, the backward into replica rows.
Used by the GPU test of the operators together."""

import torch

import zero_partition_plan_amd as Z

EPS, A, C, CLIP, KL = 1e-5, 0.9, 1.1, (0.2, 0.2), 0.05


class BlockChain:
    """Parameters of odd sizes, flat and split over nd shards; the matrices' and the vectors' tensors are views of
    the flat arrays."""

    def __init__(self, dtype, stream, d=97, f=200, v=331, rows=70, nd=2, seed=0, device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.dims, self.nd, self.dtype, self.stream, self.device = (d, f, v, rows), nd, dtype, stream, device
        self.shapes = {"n0": (d,), "w1": (f, d), "w2": (d, f), "post": (d,), "post_b": (d,), "gate": (1, d), "n1": (d,),
                       "head": (v, d)}
        self.n = sum(torch.Size(s).numel() for s in self.shapes.values())
        self.plan = Z.zero_partition_plan(self.n, nd)
        flat = torch.zeros(self.plan.padded_n, device=device)
        for name, t in self.views(flat).items():
            t.copy_(torch.randn(t.shape, generator=g, device=device) * (0.1 if len(t.shape) == 1 else t.shape[1] ** -0.5))
            if name in ("n0", "post", "n1"):
                t.add_(1.0)
            if name == "gate":
                t.mul_(5.0).add_(0.5)
        self.master, self.full = flat, flat.to(dtype)
        self.gathered = torch.empty(self.n, dtype=dtype, device=device)
        self.rows_of = torch.zeros(nd, self.plan.padded_n, device=device)

        def new(*shape, dt=dtype):
            return torch.empty(shape, dtype=dt, device=device)

        self.batches = []
        for _ in range(nd):
            self.batches.append({
                "x": torch.randn((rows, d), generator=g, device=device).to(stream),
                "label": torch.randint(v, (rows,), generator=g, device=device).masked_fill_(torch.arange(rows, device=device) % 7 == 0, -1),
                # far from the ends of the ratio's range, log 0.8 and log 1.2, for the logits' own rounding
                "step": torch.tensor([-0.6, -0.05, 0.05, 0.6], device=device)[torch.randint(4, (rows,), generator=g, device=device)],
                "adv": torch.randn((rows,), generator=g, device=device),
                "weight": (torch.arange(rows, device=device) % 5 != 0).float()})
        self.h0, self.pre, self.act, self.branch = new(rows, d), new(rows, f), new(rows, f), new(rows, d)
        self.y, self.h1, self.logits = new(rows, d, dt=stream), new(rows, d), new(rows, v)
        self.st0, self.st1 = (torch.empty(rows, 4, device=device) for _ in range(2))
        self.dh1, self.dx, self.dbranch, self.dact, self.dz, self.dh0 = new(rows, d), new(rows, d, dt=stream), new(rows, d), \
            new(rows, f), new(rows, f), new(rows, d)
        self.loss, self.logp = torch.empty(nd, rows, device=device), torch.empty(rows, device=device)
        need = max(max(Z.zero_linear_workspace_bytes(rows, k, o, b) for b in (False, True)) for k, o in ((d, f), (f, d), (d, v)))
        self.ws = torch.empty(max(need, Z.zero_norm_workspace_bytes(rows, d, rows), 16), dtype=torch.uint8, device=device)
        self.edge = dict(post="layer", pre="rms", gate_rows=rows, eps=EPS, residual_scale=A, branch_scale=C)

    def views(self, flat):
        out, pos = {}, 0
        for name, shape in self.shapes.items():
            n = torch.Size(shape).numel()
            out[name] = flat[pos:pos + n].view(shape)
            pos += n
        return out

    def gather(self):
        S = self.plan.shard_elems
        Z.zero_gather_params([self.full[r * S:(r + 1) * S] for r in range(self.nd)], 0, self.n, self.gathered)

    def forward(self, k):
        b, p, ws = self.batches[k], self.views(self.gathered), self.ws
        Z.zero_norm_forward(b["x"], h=self.h0, pre="rms", pre_weight=p["n0"], eps=EPS, stats=self.st0)
        Z.zero_linear_forward(self.h0, p["w1"], self.act, act="silu", pre=self.pre, workspace=ws)
        Z.zero_linear_forward(self.act, p["w2"], self.branch, workspace=ws)
        Z.zero_norm_forward(b["x"], h=self.h1, branch=self.branch, y=self.y, gate=p["gate"], post_weight=p["post"],
                            post_bias=p["post_b"], pre_weight=p["n1"], stats=self.st1, **self.edge)
        Z.zero_linear_forward(self.h1, p["head"], self.logits, workspace=ws)

    def behind(self, k):
        """The old and reference policies' log probabilities: this one's, a little off."""
        b = self.batches[k]
        self.forward(k)
        Z.zero_token_logp(self.logits, b["label"], self.logp)
        b["old"], b["ref"] = self.logp - b["step"], self.logp + 0.3 * b["step"]

    def forward_backward(self, k, scale):
        b, p, g, ws = self.batches[k], self.views(self.gathered), self.views(self.rows_of[k]), self.ws
        self.forward(k)
        Z.zero_policy_step(self.logits, b["label"], b["old"], b["adv"], self.loss[k], self.logits, ref_logp=b["ref"],
                           weight=b["weight"], clip=CLIP, kl_coef=KL, scale=scale)      # the gradient over the logits
        Z.zero_linear_backward(self.logits, self.h1, p["head"], dx=self.dh1, dweight=g["head"], workspace=ws)
        Z.zero_norm_backward(self.y, self.st1, dh=self.dh1, branch=self.branch, gate=p["gate"], post_weight=p["post"],
                             post_bias=p["post_b"], pre_weight=p["n1"], dx=self.dx, dbranch=self.dbranch, dgate=g["gate"],
                             dpost_weight=g["post"], dpost_bias=g["post_b"], dpre_weight=g["n1"], workspace=ws, **self.edge)
        Z.zero_linear_backward(self.dbranch, self.act, p["w2"], dx=self.dact, dweight=g["w2"], workspace=ws)
        Z.zero_linear_backward(self.dact, self.h0, p["w1"], act="silu", pre=self.pre, dz=self.dz, dx=self.dh0,
                               dweight=g["w1"], workspace=ws)
        Z.zero_norm_backward(b["x"], self.st0, dy=self.dx, dh=self.dh0, pre="rms", pre_weight=p["n0"], eps=EPS, dx=self.dx,
                             dpre_weight=g["n0"], workspace=ws)

    def reference(self, k, scale):
        """(loss rows, flat gradient, the stream's gradient) of micro-batch k in fp64 by automatic gradients."""
        b = self.batches[k]
        p = {n: t.double().requires_grad_() for n, t in self.views(self.gathered).items()}
        x = b["x"].double().requires_grad_()

        def rms(v, w):
            return v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * w

        act = torch.nn.functional.silu(rms(x, p["n0"]) @ p["w1"].t())
        o = act @ p["w2"].t()
        n = x.shape[1]
        y = A * x + C * p["gate"] * torch.nn.functional.layer_norm(o, (n,), p["post"], p["post_b"], EPS)
        z = rms(y, p["n1"]) @ p["head"].t()
        on = (b["label"] >= 0) & (b["weight"] != 0)
        l = torch.log_softmax(z, 1).gather(1, b["label"].clamp(min=0)[:, None])[:, 0]
        ratio, a, d = (l - b["old"].double()).exp(), b["adv"].double(), b["ref"].double() - l
        loss = -torch.minimum(ratio * a, ratio.clamp(1 - CLIP[0], 1 + CLIP[1]) * a) + KL * (d.exp() - 1 - d)
        loss = torch.where(on, loss * b["weight"].double(), torch.zeros_like(loss))
        (loss.sum() * scale).backward()
        return loss.detach(), torch.cat([p[n].grad.reshape(-1) for n in self.shapes]), x.grad
