"""A small ZeRO-3 training step made of the library's calls alone: gather, a two-layer MLP block on a
residual stream, a head, the distillation loss, the backward into replica rows. Used by the GPU
tests of the operators together."""

import torch

import zero_partition_plan_amd as Z


class Chain:
    """Parameters w1 [f, d], b1, w2 [d, f], b2, head [v, d], flat and split over nd shards; odd sizes put
    most of them off 16 bytes."""

    def __init__(self, d=97, f=200, v=1031, rows=70, topk=9, nd=2, dtype=torch.float16, seed=0, device="cuda:0",
                 temperature=2.0, gdtype=None):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.dims, self.nd, self.dtype, self.T, self.device = (d, f, v, rows), nd, dtype, temperature, device
        self.shapes = {"w1": (f, d), "b1": (f,), "w2": (d, f), "b2": (d,), "head": (v, d)}
        n = sum(torch.Size(s).numel() for s in self.shapes.values())
        self.plan = Z.zero_partition_plan(n, nd)
        S = self.plan.shard_elems
        flat = torch.zeros(self.plan.padded_n, device=device)
        for name, view in self.views(flat).items():
            std = 0.1 if view.dim() == 1 else view.shape[1] ** -0.5
            view.copy_(torch.randn(view.shape, generator=g, device=device) * std)
        self.master = flat.clone()
        self.full = flat.to(dtype)
        self.gathered = torch.empty(n, dtype=dtype, device=device)
        self.rows_of = torch.zeros(nd, self.plan.padded_n, dtype=gdtype or dtype, device=device)

        def new(*shape, dt=dtype):
            return torch.empty(shape, dtype=dt, device=device)

        self.batches = []
        for _ in range(nd):
            base = torch.randint(v, (rows, 1), generator=g, device=device)
            idx = (base + torch.arange(topk, device=device) * 17) % v
            idx[3, 2:] = -1
            self.batches.append({
                "x": torch.randn((rows, d), generator=g, device=device).to(dtype), "idx": idx.to(torch.int32),
                "top": torch.randn((rows, topk), generator=g, device=device) * 2,
                "tail": torch.randn((rows,), generator=g, device=device),
                "weight": (torch.arange(rows, device=device) % 5 != 0).float()})
        self.h, self.pre, self.y, self.logits = new(rows, f), new(rows, f), new(rows, d), new(rows, v)
        self.dy, self.dh, self.dz = new(rows, d), new(rows, f), new(rows, f)
        self.loss = torch.empty(nd, rows, device=device)
        need = max(max(Z.zero_linear_workspace_bytes(rows, k, o, b) for b in (False, True))
                   for k, o in ((d, f), (f, d), (d, v)))
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)

    def views(self, flat):
        out, pos = {}, 0
        for name, shape in self.shapes.items():
            n = torch.Size(shape).numel()
            out[name] = flat[pos:pos + n].view(shape)
            pos += n
        return out

    def gather(self):
        S = self.plan.shard_elems
        Z.zero_gather_params([self.full[r * S:(r + 1) * S] for r in range(self.nd)], 0, self.plan.n, self.gathered)

    def forward_backward(self, k, scale):
        """Micro-batch k, its parameter gradients (times scale) in replica row k."""
        b, p, g, ws = self.batches[k], self.views(self.gathered), self.views(self.rows_of[k]), self.ws
        Z.zero_linear_forward(b["x"], p["w1"], self.h, bias=p["b1"], act="gelu_tanh", pre=self.pre, workspace=ws)
        Z.zero_linear_forward(self.h, p["w2"], self.y, bias=p["b2"], residual=b["x"], workspace=ws)
        Z.zero_linear_forward(self.y, p["head"], self.logits, workspace=ws)
        Z.zero_distill_step(self.logits, b["idx"], b["top"], self.T, self.loss[k], self.logits, tail=b["tail"],
                            weight=b["weight"], scale=scale)            # the gradient over the logits
        Z.zero_linear_backward(self.logits, self.y, p["head"], dx=self.dy, dweight=g["head"], workspace=ws)
        Z.zero_linear_backward(self.dy, self.h, p["w2"], dx=self.dh, dweight=g["w2"], dbias=g["b2"], workspace=ws)
        Z.zero_linear_backward(self.dh, b["x"], p["w1"], act="gelu_tanh", pre=self.pre, dz=self.dz, dweight=g["w1"],
                               dbias=g["b1"], workspace=ws)

    def reference(self, k, scale):
        """(loss rows, flat gradient) of micro-batch k in fp64 by automatic gradients."""
        b = self.batches[k]
        p = {n: t.double().requires_grad_() for n, t in self.views(self.gathered).items()}
        x = b["x"].double()
        h = torch.nn.functional.gelu(x @ p["w1"].t() + p["b1"], approximate="tanh")
        y = h @ p["w2"].t() + p["b2"] + x
        lq = torch.log_softmax(y @ p["head"].t() / self.T, 1)
        valid = b["idx"] >= 0
        cols = b["idx"].long().clamp(min=0)
        t = torch.cat([(b["top"].double() / self.T).masked_fill(~valid, -torch.inf), b["tail"].double()[:, None]], 1)
        lp = torch.log_softmax(t, 1)
        inside = torch.zeros(lq.shape, device=lq.device).scatter_add_(1, cols, valid.float()) > 0
        rest = torch.logsumexp(lq.masked_fill(inside, -torch.inf), 1)
        terms = lp.exp()[:, :-1] * (lp[:, :-1] - lq.gather(1, cols))
        loss = torch.where(valid, terms, torch.zeros_like(terms)).sum(1) + lp.exp()[:, -1] * (lp[:, -1] - rest)
        loss = loss * b["weight"].double()
        (loss.sum() * scale).backward()
        return loss.detach(), torch.cat([p[n].grad.reshape(-1) for n in self.shapes])
