"""The layer operators that surround the sharded step, as measured: the linear layer (matrix product
with bias, activation and residual, and its backward products) and the distillation loss over a
teacher's top logits (forward, backward, and both in one pass).

`run` computes a case in plain torch operations, or, with `own`, by the calls a training program
makes of zero_partition_plan_amd. Sizes are those of the models the workloads name (GPT-2 small,
Llama 7B and 13B shapes) or generic ones.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_DEV = "cuda:0"


# ------------------------------------------------------------------------------------ the cases

def _linear(name, pas, m, k, n, dtype, act="none", bias=False, residual=False, grad="same"):
    return {"name": name, "op": "linear", "pass": pas, "m": m, "k": k, "n": n, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "grad": grad}


def _distill(name, pas, rows, vocab, topk, dtype, tail, temperature, index="i32", teacher="f32"):
    return {"name": name, "op": "distill", "pass": pas, "rows": rows, "vocab": vocab, "topk": topk,
            "dtype": dtype, "tail": tail, "temperature": temperature, "index": index, "teacher": teacher}


def listed():
    return [
        # one token through a Llama-7B attention output projection added to the residual stream:
        # latency and the weight's read
        _linear("linear_one_token", "forward", 1, 4096, 4096, "bf16", residual=True),
        # a ragged batch through GPT-2's fused q/k/v projection with its bias, fp16
        _linear("linear_gpt2_ragged", "forward", 1001, 768, 2304, "f16", bias=True),
        # a batch of 4096 tokens through Llama-7B's gate projection, pre-activation kept
        _linear("linear_7b_gate", "forward", 4096, 4096, 11008, "bf16", act="silu"),
        # the output head over GPT-2's odd vocabulary: rows of odd length
        _linear("linear_gpt2_head", "forward", 2048, 768, 50257, "bf16"),
        # backward of a small biased layer with an activation on a ragged batch, fp16
        _linear("linear_back_ragged", "backward", 333, 768, 2304, "f16", act="gelu_tanh", bias=True),
        # backward of Llama-7B's down projection added to the residual stream, 16-bit gradient rows
        _linear("linear_back_7b_down", "backward", 4096, 11008, 4096, "bf16"),
        # backward of a Llama-13B square projection into fp32 gradient rows
        _linear("linear_back_13b_f32", "backward", 2048, 5120, 5120, "bf16", grad="f32"),
        # the loss of one row over GPT-2's vocabulary: latency
        _distill("distill_one_row", "step", 1, 50257, 16, "bf16", False, 1.0),
        # loss and gradient in one pass over a Llama batch of 8192 tokens
        _distill("distill_7b_step", "step", 8192, 32000, 32, "bf16", False, 2.0),
        # the same as two calls, as under an autograd engine, with the teacher's remaining mass
        _distill("distill_7b_two_calls", "both", 4096, 32000, 64, "bf16", True, 2.0, "i64", "bf16"),
        # fp32 logits over an odd vocabulary with the teacher's remaining mass
        _distill("distill_odd_f32", "step", 1023, 50257, 128, "f32", True, 1.5, "i64"),
        # evaluation: the loss alone over a large vocabulary
        _distill("distill_eval", "forward", 2048, 131072, 100, "f16", False, 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature count: mostly multiples of 64 as models have them, sometimes of 8, sometimes odd."""
    n, kind = _log(rng, lo, hi), rng.random()
    if kind < 0.6:
        return max(64, n // 64 * 64)
    return max(8, n // 8 * 8) if kind < 0.8 else n | 1


def draw(rng):
    if rng.random() < 0.55:
        pas = rng.choice(["forward", "backward"])
        k, n = _width(rng, 64, 12288), _width(rng, 64, 12288)
        most = min(8192, int(4096 * 4096 * 11008 // (k * n)))
        m = _log(rng, 1, max(2, most))
        dtype = rng.choice(["bf16", "f16"])
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        case = _linear("", pas, m, k, n, dtype, act, rng.random() < 0.5,
                       pas == "forward" and rng.random() < 0.5,
                       "f32" if pas == "backward" and act == "none" and rng.random() < 0.5 else "same")
    else:
        vocab = _log(rng, 1000, 131072)
        rows = _log(rng, 1, max(2, min(8192, 8192 * 32000 // (2 * vocab))))
        case = _distill("", rng.choice(["step", "both", "forward"]), rows, vocab, min(_log(rng, 1, 512), vocab // 4),
                        rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.5,
                        rng.choice([1.0, 1.5, 2.0, 4.0]), rng.choice(["i32", "i64"]),
                        rng.choice(["bf16", "f16", "f32"]))
    del case["name"]
    return case


def work(case):
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        if case["pass"] == "forward":
            keep = case["act"] != "none"
            elems = m * k + n * k + m * n * (1 + keep + case["residual"]) + n * case["bias"]
            return {"bytes": 2 * elems, "flops": 2 * m * n * k}
        act = case["act"] != "none"
        wb = 4 if case["grad"] == "f32" else 2
        elems = m * n * (1 + 2 * act) + 2 * m * k + n * k
        return {"bytes": 2 * elems + wb * (n * k + n * case["bias"]), "flops": 4 * m * n * k}
    rows, vocab = case["rows"], case["vocab"]
    eb = 4 if case["dtype"] == "f32" else 2
    per_top = (8 if case["index"] == "i64" else 4) + (4 if case["teacher"] == "f32" else 2)
    grad = case["pass"] != "forward"
    return {"bytes": rows * (vocab * eb * (1 + grad) + case["topk"] * per_top + 4 * (2 + case["tail"])),
            "flops": rows * vocab * (4 + 3 * grad)}


# ----------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device=_DEV).mul_(std).to(dtype)


def _linear_inputs(case, seed):
    g, dt = _gen(seed), _DT[case["dtype"]]
    m, k, n = case["m"], case["k"], case["n"]
    s = {"case": case, "x": _normal(g, (m, k), 1.0, dt), "w": _normal(g, (n, k), 0.02, dt)}
    s["b"] = _normal(g, (n,), 0.1, dt) if case["bias"] else None
    if case["pass"] == "forward":
        s["r"] = _normal(g, (m, n), 1.0, dt) if case["residual"] else None
    else:
        s["dy"] = _normal(g, (m, n), 1.0, dt)
        s["pre"] = _normal(g, (m, n), 1.3, dt) if case["act"] != "none" else None
    return s


def _coprime_step(vocab, seed):
    step = 1 + (seed * 7919 + 104729) % (vocab - 1)
    while math.gcd(step, vocab) != 1:
        step = step % (vocab - 1) + 1
    return step


def _distill_inputs(case, seed):
    """Student logits whose top tokens are mostly the teacher's: the teacher's entries are distinct
    tokens of falling logits, the student's logits there are the teacher's plus noise. A tenth of
    the rows carry weight 0 (prompt and padding tokens) and some rows list fewer entries (index -1)."""
    g, dt = _gen(seed), _DT[case["dtype"]]
    rows, vocab, topk = case["rows"], case["vocab"], case["topk"]
    logits = torch.randn((rows, vocab), generator=g, device=_DEV).mul_(1.5)
    base = torch.randint(vocab, (rows, 1), generator=g, device=_DEV)
    idx = (base + torch.arange(topk, device=_DEV) * _coprime_step(vocab, seed)) % vocab
    top = torch.randn((rows, topk), generator=g, device=_DEV).mul_(2.0).add_(9.0)
    top = top.sort(dim=1, descending=True).values
    logits.scatter_(1, idx, top + torch.randn((rows, topk), generator=g, device=_DEV))
    short = torch.rand((rows, 1), generator=g, device=_DEV) < 0.1
    idx = torch.where(short & (torch.arange(topk, device=_DEV) >= (topk + 1) // 2), -1, idx)
    weight = (torch.rand((rows,), generator=g, device=_DEV) < 0.9).float()
    weight[0] = 1.0
    s = {"case": case, "logits": logits.to(dt), "top": top.to(_DT[case["teacher"]]), "weight": weight,
         "idx": idx.to(torch.int64 if case["index"] == "i64" else torch.int32), "tail": None}
    if case["tail"]:
        s["tail"] = torch.randn((rows,), generator=g, device=_DEV).add_(7.0)
    s["scale"] = case["temperature"] ** 2
    return s


def prepare(case, seed):
    linear = case["op"] == "linear"
    s = _linear_inputs(case, seed) if linear else _distill_inputs(case, seed)
    if not own:
        return s
    import zero_partition_plan_amd as Z
    s["Z"] = Z
    if linear:
        m, k, n = case["m"], case["k"], case["n"]
        dt = _DT[case["dtype"]]

        def buf(*shape, dtype=dt):
            return torch.empty(shape, dtype=dtype, device=_DEV)

        back = case["pass"] == "backward"
        s["ws"] = buf(Z.zero_linear_workspace_bytes(m, k, n, backward=back), dtype=torch.uint8)
        if back:
            gdt = torch.float32 if case["grad"] == "f32" else dt
            s["dz"] = buf(m, n) if case["act"] != "none" else None
            s["dx"], s["dw"] = buf(m, k), buf(n, k, dtype=gdt)
            s["db"] = buf(n, dtype=gdt) if case["bias"] else None
        else:
            s["y"] = buf(m, n)
            s["pre"] = buf(m, n) if case["act"] != "none" else None
    else:
        rows = case["rows"]
        s["loss"] = torch.empty((rows,), device=_DEV)
        s["stats"] = torch.empty((rows, 2), device=_DEV) if case["pass"] != "step" else None
        s["dlogits"] = torch.empty_like(s["logits"]) if case["pass"] != "forward" else None
    return s


# --------------------------------------------------------------------------------- the operators

def run(state):
    if own:
        return _run_own(state)
    return _linear_plain(state) if state["case"]["op"] == "linear" else _distill_plain(state)


def _run_own(s):
    case, Z = s["case"], s["Z"]
    if case["op"] == "linear":
        if case["pass"] == "forward":
            Z.zero_linear_forward(s["x"], s["w"], s["y"], bias=s["b"], residual=s["r"], act=case["act"],
                                  pre=s["pre"], workspace=s["ws"])
            return [t for t in (s["y"], s["pre"]) if t is not None]
        Z.zero_linear_backward(s["dy"], s["x"], s["w"], act=case["act"], pre=s["pre"], dz=s["dz"],
                               dx=s["dx"], dweight=s["dw"], dbias=s["db"], workspace=s["ws"])
        return [t for t in (s["dz"], s["dx"], s["dw"], s["db"]) if t is not None]
    args = (s["logits"], s["idx"], s["top"], case["temperature"])
    kw = {"tail": s["tail"], "weight": s["weight"]}
    if case["pass"] == "step":
        Z.zero_distill_step(*args, s["loss"], s["dlogits"], scale=s["scale"], **kw)
        return [s["loss"], s["dlogits"]]
    Z.zero_distill_forward(*args, s["loss"], s["stats"], **kw)
    if case["pass"] == "forward":
        return [s["loss"]]
    Z.zero_distill_backward(*args, s["stats"], s["dlogits"], scale=s["scale"], **kw)
    return [s["loss"], s["dlogits"]]


_TANH_C, _TANH_A = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, kind):
    if kind == "relu":
        return z.clamp_min(0)
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_TANH_C * (z + _TANH_A * z * z * z)))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        t = torch.tanh(_TANH_C * (z + _TANH_A * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _TANH_C * (1 + 3 * _TANH_A * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _linear_plain(s):
    case, dt = s["case"], _DT[s["case"]["dtype"]]
    if case["pass"] == "forward":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, case["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return [y.to(dt)] + ([z.to(dt)] if case["act"] != "none" else [])
    # dz is an output of the layer's type, and what follows is formed from it as it is stored
    gdt = torch.float32 if case["grad"] == "f32" else dt
    dz = s["dy"]
    if case["act"] != "none":
        dz = (s["dy"].float() * _act_slope(s["pre"].float(), case["act"])).to(dt)
    d = dz.float()
    out = [dz] if case["act"] != "none" else []
    out += [(d @ s["w"].float()).to(dt), (d.t() @ s["x"].float()).to(gdt)]
    return out + ([d.sum(0).to(gdt)] if case["bias"] else [])


def _distill_plain(s):
    case = s["case"]
    z = s["logits"].float() / case["temperature"]
    valid = s["idx"] >= 0
    idx = s["idx"].long().clamp_min(0)
    t = (s["top"].float() / case["temperature"]).masked_fill(~valid, float("-inf"))
    m = t.max(1, keepdim=True).values
    if s["tail"] is not None:
        m = torch.maximum(m, s["tail"][:, None])
    e = torch.exp(t - m)
    total = e.sum(1, keepdim=True)
    if s["tail"] is not None:
        e_tail = torch.exp(s["tail"][:, None] - m)
        total = total + e_tail
    p, log_p = e / total, t - m - torch.log(total)
    zm = z.max(1, keepdim=True).values
    ez = torch.exp(z - zm)
    sz = ez.sum(1, keepdim=True)
    log_q = z.gather(1, idx) - zm - torch.log(sz)
    kl = torch.where(valid, p * (log_p - log_q), torch.zeros_like(p)).sum(1)
    q = ez / sz
    dense = torch.zeros_like(z).scatter_add_(1, idx, torch.where(valid, p, torch.zeros_like(p)))
    if s["tail"] is not None:
        p_tail = e_tail / total
        listed_ = torch.zeros_like(z).scatter_add_(1, idx, valid.float()) > 0
        rest = ez.masked_fill(listed_, 0.0).sum(1, keepdim=True)
        kl = kl + (p_tail * (torch.log(p_tail) - torch.log(rest / sz)))[:, 0]
        dense = dense + p_tail * ez.masked_fill(listed_, 0.0) / rest
    out = [s["weight"] * kl]
    if case["pass"] != "forward":
        coef = s["weight"][:, None] * (s["scale"] / case["temperature"])
        out.append((coef * (q - dense)).to(s["logits"].dtype))
    return out


# ----------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "linear":
        return _linear_exact(case, _linear_inputs(case, seed))
    return _distill_exact(case, _distill_inputs(case, seed))


def _linear_exact(case, s):
    kind = case["act"]
    x, w = s["x"].double(), s["w"].double()
    if case["pass"] == "forward":
        pre = torch.mm(x, w.t().contiguous())
        if case["bias"]:
            pre += s["b"].double()
        gate = {"none": lambda v: 1.0, "relu": lambda v: (v > 0).double(),
                "gelu": lambda v: 0.5 * torch.special.erfc(-v / math.sqrt(2.0)),
                "gelu_tanh": lambda v: torch.sigmoid(2 * _TANH_C * v * (1 + _TANH_A * v ** 2)),
                "silu": torch.sigmoid}[kind](pre)
        y = pre * gate
        if case["residual"]:
            y += s["r"].double()
        return [y] + ([pre] if kind != "none" else [])
    d = s["dy"].double()
    out = []
    if kind != "none":
        v = s["pre"].double()
        if kind == "relu":
            slope = (v > 0).double()
        elif kind == "gelu":
            slope = 0.5 * torch.special.erfc(-v / math.sqrt(2.0)) + v * torch.exp(-v ** 2 / 2) / math.sqrt(2 * math.pi)
        elif kind == "gelu_tanh":
            sg = torch.sigmoid(2 * _TANH_C * v * (1 + _TANH_A * v ** 2))
            slope = sg + v * sg * (1 - sg) * 2 * _TANH_C * (1 + 3 * _TANH_A * v ** 2)
        else:
            sg = torch.sigmoid(v)
            slope = sg + v * sg * (1 - sg)
        d = d * slope
        out.append(d)
        d = d.to(_DT[case["dtype"]]).double()
    out.append(torch.mm(d, w))
    out.append(torch.mm(d.t().contiguous(), x))
    if case["bias"]:
        out.append(torch.sum(d, 0))
    return out


def _distill_exact(case, s):
    """Row blocks, so that the 64-bit copies of the largest case stay small."""
    T, rows = case["temperature"], case["rows"]
    losses, grads = [], []
    block = max(1, (1 << 27) // case["vocab"])
    for a in range(0, rows, block):
        b = min(rows, a + block)
        ls = torch.log_softmax(s["logits"][a:b].double() / T, 1)
        idx, t = s["idx"][a:b].long(), s["top"][a:b].double() / T
        t[idx < 0] = -math.inf
        cols = idx.clamp(min=0)
        parts = [t] + ([s["tail"][a:b, None].double()] if case["tail"] else [])
        lp = torch.log_softmax(torch.cat(parts, 1), 1)
        p = lp.exp()
        k = case["topk"]
        diff = torch.where(p[:, :k] > 0, lp[:, :k] - ls.gather(1, cols), torch.zeros_like(t))
        kl = (p[:, :k] * diff).sum(1)
        target = torch.zeros_like(ls)
        target.scatter_add_(1, cols, p[:, :k])
        if case["tail"]:
            rest = ls.clone()
            r = torch.arange(b - a, device=_DEV)[:, None].expand(-1, k)
            keep = idx >= 0
            rest[r[keep], cols[keep]] = -math.inf
            log_rest = torch.logsumexp(rest, 1)
            kl += p[:, k] * (lp[:, k] - log_rest)
            target += p[:, k:] * (rest - log_rest[:, None]).exp()
        w = s["weight"][a:b].double()
        losses.append(w * kl)
        if case["pass"] != "forward":
            grads.append((ls.exp() - target) * (w * s["scale"] / T)[:, None])
    return [torch.cat(losses)] + ([torch.cat(grads)] if grads else [])
