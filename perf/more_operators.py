"""More operators of a training step around the sharded update, as measured: the AdamW step over many
tensors at once (states in 32 bits or in 8), the norms before and after a block with the block's gate and
residual scale (forward and backward), and the losses over the tokens of a batch: the clipped policy loss
with a KL term and the preference loss of paired answers (forward and gradient over the logits).

`run` computes a case in plain torch operations, or, with `own`, by the calls a training program
makes of zero_partition_plan_amd. Sizes are those of the models the workloads name (GPT-2 small, Llama 7B)
or generic ones.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_DEV = "cuda:0"
_BLOCK = 256                  # elements of a tensor that share a scale in the 8-bit states


# ------------------------------------------------------------------------------------ the cases

def _adam(name, kind, width, ffn, layers, vocab, rank, bits, grad, out):
    return {"name": name, "op": "adam", "kind": kind, "width": width, "ffn": ffn, "layers": layers, "vocab": vocab,
            "rank": rank, "bits": bits, "grad": grad, "out": out}


def _norm(name, pas, rows, features, dtype, stream, post, pre, gate, gate_rows, bias, grad="f32",
          residual_scale=1.0, branch_scale=1.0):
    return {"name": name, "op": "norm", "pass": pas, "rows": rows, "features": features, "dtype": dtype,
            "stream": stream, "post": post, "pre": pre, "gate": gate, "gate_rows": gate_rows, "bias": bias,
            "grad": grad, "residual_scale": residual_scale, "branch_scale": branch_scale}


def _policy(name, pas, rows, vocab, dtype, kl, temperature, index="i64", active=0.9):
    return {"name": name, "op": "policy", "pass": pas, "rows": rows, "vocab": vocab, "dtype": dtype, "kl": kl,
            "temperature": temperature, "index": index, "active": active}


def _preference(name, pas, rows, pairs, vocab, dtype, average, smoothing, index="i64", active=0.8):
    return {"name": name, "op": "preference", "pass": pas, "rows": rows, "pairs": pairs, "vocab": vocab,
            "dtype": dtype, "average": average, "smoothing": smoothing, "index": index, "active": active}


def listed():
    return [
        # fine-tuning by low-rank adapters: many small tensors of odd sizes, states in 8 bits
        _adam("adam8_adapters", "adapters", 1001, 0, 6, 0, 7, 8, "f16", "f16"),
        # every tensor of GPT-2 small in one call, matrices decayed and vectors not, states in 32 bits
        _adam("adam_gpt2_tensors", "model", 768, 0, 12, 50257, 0, 32, "bf16", "bf16"),
        # one Llama-7B block's tensors, states in 8 bits, and the states written out as numbers
        _adam("adam8_7b_block", "block", 4096, 11008, 1, 0, 0, 8, "bf16", "bf16"),
        # one token of a Llama-7B block: the branch's norm, the sum, the next block's norm; latency
        _norm("norm_one_token", "forward", 1, 4096, "bf16", "bf16", "rms", "rms", "none", 1, False),
        # the same over a batch of 8192 tokens with a learned gate for each channel and an fp32 residual stream
        _norm("norm_7b_batch", "forward", 8192, 4096, "bf16", "f32", "rms", "rms", "channel", 1, False, "f32", 1.0, 0.5),
        # its backward on a 16-bit stream, parameter gradients into fp32 replica rows
        _norm("norm_7b_backward", "backward", 8192, 4096, "bf16", "bf16", "rms", "rms", "channel", 1, False),
        # backward of a GPT-2 block boundary on a ragged batch: layer norms with biases, a gate of each token, fp16
        _norm("norm_gpt2_backward", "backward", 1001, 768, "f16", "f16", "layer", "layer", "token", 1, True, "same", 0.8),
        # the policy loss of one token over GPT-2's vocabulary: latency
        _policy("policy_one_row", "step", 1, 50257, "bf16", 0.05, 1.0, "i64", 1.0),
        # loss and gradient in one pass over a Llama batch of 8192 tokens, a tenth of them prompt
        _policy("policy_7b_step", "step", 8192, 32000, "bf16", 0.02, 1.0),
        # as two calls over fp32 logits with an odd vocabulary
        _policy("policy_two_calls_f32", "both", 1023, 50257, "f32", 0.1, 0.7, "i32"),
        # 8 pairs of answers with their prompts over Llama's vocabulary
        _preference("preference_7b", "both", 8192, 8, 32000, "bf16", False, 0.0),
        # ragged pairs over GPT-2's vocabulary, mean over each answer's tokens, the loss alone
        _preference("preference_eval", "forward", 1533, 5, 50257, "f16", True, 0.1, "i32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_adam(rng):
    kind, bits = rng.choice(["vectors", "model", "block", "adapters"]), rng.choice([8, 32])
    width = _log(rng, 48, 2048)
    case = _adam("", kind, width, _log(rng, width, 4 * width), 1, _log(rng, 100, 50257), _log(rng, 1, 64), bits,
                 rng.choice(["bf16", "f16", "f32"]), rng.choice(["bf16", "f16", "none"]))
    each = sum(_sizes(case)) - sum(_sizes({**case, "layers": 0}))
    case["layers"] = _log(rng, 1, max(1.5, min(48, 6e7 / max(1, each))))
    return case


def _draw_norm(rng):
    features = _log(rng, 64, 12288)
    if rng.random() < 0.7:
        features = max(64, features // 64 * 64)
    dtype = rng.choice(["bf16", "f16"])
    rows = _log(rng, 1, min(16384, 8192 * 4096 // features))
    post, pre = rng.choice([("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("none", "layer"), ("rms", "none")])
    return _norm("", rng.choice(["forward", "backward"]), rows, features, dtype, rng.choice([dtype, "f32"]), post, pre,
                 rng.choice(["none", "channel", "sequence", "token"]), _log(rng, 2, 2048), rng.random() < 0.5,
                 rng.choice(["same", "f32"]), rng.choice([1.0, 0.8]), rng.choice([1.0, 0.5]))


def _draw_loss(rng):
    vocab = _log(rng, 1000, 131072)
    rows = _log(rng, 8, min(8192, 8192 * 32000 // (2 * vocab)))
    dtype, index = rng.choice(["bf16", "f16", "f32"]), rng.choice(["i32", "i64"])
    if rng.random() < 0.5:
        return _policy("", rng.choice(["step", "both", "forward"]), rows, vocab, dtype, rng.choice([0.0, 0.05]),
                       rng.choice([1.0, 0.7]), index)
    return _preference("", rng.choice(["both", "forward"]), rows, rng.randint(1, max(1, min(16, rows // 8))), vocab, dtype,
                       rng.random() < 0.5, rng.choice([0.0, 0.1]), index)


def draw(rng):
    case = rng.choice([_draw_adam, _draw_norm, _draw_loss])(rng)
    del case["name"]
    return case


def _sizes(case):
    """The tensors' element counts, in the order of the flat space."""
    w, f, n = case["width"], case["ffn"], case["layers"]
    if case["kind"] == "vectors":
        return [w] * (4 * n + 2)
    if case["kind"] == "model":
        return [case["vocab"] * w, 1024 * w] + [w, w, 3 * w * w, w * w, w, w, 4 * w * w, 4 * w * w] * n + [w, w]
    if case["kind"] == "block":
        return [w, w * w, w * w, w * w, w * w, w, w * f, w * f, w * f] * n
    return [case["rank"] * w] * (8 * n)


def _eb(name):
    return 4 if name == "f32" else 2


def work(case):
    if case["op"] == "adam":
        n, g = sum(_sizes(case)), _eb(case["grad"])
        out = 0 if case["out"] == "none" else 2
        if case["bits"] == 32:
            return {"bytes": n * (g + 24 + out), "flops": 18 * n}
        # parameter, codes and scales in and out, and both moments written out as fp32 numbers
        return {"bytes": n * (g + 8 + 4 + out + 8) + 16 * (n // _BLOCK), "flops": 40 * n}
    if case["op"] == "norm":
        r, d, s = case["rows"], case["features"], _eb(case["stream"])
        gates = _gate_shape(case)[0] * d if case["gate"] != "none" else 0
        vec = d * ((case["post"] != "none") + (case["pre"] != "none")) * (1 + case["bias"])
        if case["pass"] == "forward":
            return {"bytes": r * d * (2 * s + 2 + 2 * (case["pre"] != "none")) + 2 * (gates + vec),
                    "flops": 12 * r * d}
        gb = 2 if case["grad"] == "same" else 4
        # gradients of the stream and of h, the sum and the branch in; two gradients out; 4 statistics a row
        pre = case["pre"] != "none"
        return {"bytes": r * d * (2 * s + 2 * 2 + pre * (2 + s)) + 16 * r + (2 + gb) * (gates + vec), "flops": 30 * r * d}
    r, v, e = case["rows"], case["vocab"], _eb(case["dtype"])
    grad = case["pass"] != "forward"
    read = int(r * case["active"])
    return {"bytes": read * v * e + r * v * e * grad + 28 * r, "flops": read * v * (4 + 3 * grad)}


# ----------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=_DEV).mul_(std).to(dtype)


_LR, _B1, _B2, _EPS, _STEP = 1e-3, 0.9, 0.999, 1e-8, 11
_DECAY = (0.1, 0.0)           # of the two groups: matrices, and vectors of one channel


def _adam_inputs(case, seed):
    """Flat arrays in which every tensor starts a block of 256 (what lies behind a tensor's end is 0 and stays
    0), warm states, gradients whose size differs from block to block."""
    g, sizes = _gen(seed), _sizes(case)
    blocks = [-(-n // _BLOCK) for n in sizes]
    starts = [0]
    for b in blocks:
        starts.append(starts[-1] + b)
    nb = starts[-1]
    group = [1 if n == case["width"] else 0 for n in sizes]
    live = torch.ones((nb, _BLOCK), dtype=torch.bool, device=_DEV)
    for n, b, a in zip(sizes, blocks, starts):
        live.view(-1)[a * _BLOCK + n:(a + b) * _BLOCK] = False
    size = torch.exp(_normal(g, (nb, 1), 0.7)) * 1e-3
    s = {"case": case, "sizes": sizes, "starts": starts, "group": group,
         "p": _normal(g, (nb, _BLOCK), 0.02).masked_fill_(~live, 0.0),
         "g": (_normal(g, (nb, _BLOCK), 1.0) * size).masked_fill_(~live, 0.0).to(_DT[case["grad"]]),
         "of": torch.repeat_interleave(torch.tensor(group, device=_DEV), torch.tensor(blocks, device=_DEV))}
    m = (_normal(g, (nb, _BLOCK), 0.23) * size).masked_fill_(~live, 0.0)
    v = torch.rand((nb, _BLOCK), generator=g, device=_DEV).add_(0.5).mul_(0.01) * size * size
    v.masked_fill_(~live, 0.0)
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["ms"] = _encode(m, 127)
        s["v"], s["vs"] = _encode(torch.sqrt(v), 255)
    s["out"] = None if case["out"] == "none" else s["p"].to(_DT[case["out"]])
    return s


def _gate_shape(case):
    rows = case["rows"]
    per = {"none": 1, "channel": max(rows, 1), "sequence": case["gate_rows"], "token": 1}[case["gate"]]
    return -(-rows // per), per


def _norm_inputs(case, seed):
    """A residual stream of growing channels, a branch's output, and for the backward the gradients that
    reach the sum and the next block's input, with the statistics that the forward leaves."""
    g, dt, st = _gen(seed), _DT[case["dtype"]], _DT[case["stream"]]
    r, d = case["rows"], case["features"]
    channel = torch.exp(_normal(g, (1, d), 0.3))
    s = {"case": case, "branch": (_normal(g, (r, d), 0.5) * channel + 0.05).to(dt)}
    gates, per = _gate_shape(case)
    s["per"] = per
    s["gate"] = _normal(g, (gates, d), 0.3, dt) + 0.5 if case["gate"] != "none" else None
    for which in ("post", "pre"):
        on = case[which] != "none"
        s[which + "_w"] = (_normal(g, (d,), 0.1) + 1.0).to(dt) if on else None
        s[which + "_b"] = _normal(g, (d,), 0.1, dt) if on and case["bias"] else None
    if case["pass"] == "forward":
        s["x"] = (_normal(g, (r, d), 1.0) * channel).to(st)
        return s
    s["y"] = (_normal(g, (r, d), 1.2) * channel + 0.02).to(st)
    s["dy"], s["dh"] = _normal(g, (r, d), 1e-2, st), None
    if case["pre"] != "none":
        s["dh"] = _normal(g, (r, d), 1e-2, dt)
    stats = [_stats(s["branch"].float(), case["post"]), _stats(s["y"].float(), case["pre"])]
    s["stats"] = torch.cat([t for pair in stats for t in pair], 1).contiguous()
    return s


_NORM_EPS = 1e-5


def _stats(v, kind):
    """(mean, 1/deviation) of each row, 0 and 1 where there is no norm."""
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    if kind == "none":
        return mean, torch.ones_like(mean)
    c = v - mean
    return mean, 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + _NORM_EPS)


def _token_inputs(case, seed):
    """Logits in which each row's token stands out, as under a trained policy."""
    g, dt = _gen(seed), _DT[case["dtype"]]
    rows, vocab = case["rows"], case["vocab"]
    label = torch.randint(vocab, (rows, 1), generator=g, device=_DEV)
    logits = torch.randn((rows, vocab), generator=g, device=_DEV).mul_(1.5)
    logits.scatter_add_(1, label, _normal(g, (rows, 1), 2.0) + 9.0)
    active = torch.rand((rows,), generator=g, device=_DEV) < case["active"]
    active[0] = True
    return g, logits.to(dt), label[:, 0].to(torch.int64 if case["index"] == "i64" else torch.int32), active


def _token_logp(logits, label, temperature):
    z = logits.float() / temperature
    return z.gather(1, label.long()[:, None])[:, 0] - torch.logsumexp(z, 1)


def _policy_inputs(case, seed):
    """Answers sampled from a policy a few updates old, with advantages of mean 0; prompt tokens have weight 0."""
    g, logits, label, active = _token_inputs(case, seed)
    lp = _token_logp(logits, label, case["temperature"])
    rows = case["rows"]
    return {"case": case, "logits": logits, "label": label, "weight": active.float(),
            "old": lp + _normal(g, (rows,), 0.15), "ref": lp + _normal(g, (rows,), 0.25) if case["kl"] else None,
            "advantage": _normal(g, (rows,), 1.0), "scale": 1.0 / rows}


def _preference_inputs(case, seed):
    """Sequences of uneven length one after the other, the last rows padding; prompt tokens have label -1.
    The reference's sums are near the policy's own."""
    g, logits, label, active = _token_inputs(case, seed)
    rows, pairs = case["rows"], case["pairs"]
    share = torch.rand((2 * pairs,), generator=g, device=_DEV) + 0.5
    ends = (share.cumsum(0) / share.sum() * (rows - rows // 50)).long()
    start = torch.cat([torch.zeros_like(ends[:1]), ends])
    lp = torch.where(active, _token_logp(logits, label, 1.0), torch.zeros_like(ends[:1]).float())
    label = torch.where(active, label, torch.full_like(label, -1))
    seq = _segments(lp.double(), start)
    if case["average"]:
        seq = seq / _segments(active.double(), start).clamp(min=1)
    ref = seq.float() + _normal(g, (2 * pairs,), 0.1 if case["average"] else 4.0)
    return {"case": case, "logits": logits, "label": label, "start": start, "ref": ref,
            "weight": torch.ones((pairs,), device=_DEV), "beta": 2.0 if case["average"] else 0.1,
            "scale": 1.0 / pairs}


def _segments(v, start):
    """Sums of v between consecutive places of `start`."""
    c = torch.cat([torch.zeros_like(v[:1]), v.cumsum(0)])
    return c[start[1:]] - c[start[:-1]]


_INPUTS = {"adam": _adam_inputs, "norm": _norm_inputs, "policy": _policy_inputs, "preference": _preference_inputs}


def prepare(case, seed):
    s = _INPUTS[case["op"]](case, seed)
    if not own:
        return s
    import zero_partition_plan_amd as Z
    s["Z"] = Z

    def buf(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device=_DEV)

    if case["op"] == "adam":
        eight, tensors = case["bits"] == 8, []
        for i, n in enumerate(s["sizes"]):
            a, b = s["starts"][i], s["starts"][i + 1]
            part = {k: s[k].view(-1)[a * _BLOCK:a * _BLOCK + n] for k in ("p", "g", "m", "v")}
            tensors.append(Z.adam_tensor(
                part["p"], part["g"], part["m"], part["v"], group=s["group"][i],
                out=None if s["out"] is None else s["out"].view(-1)[a * _BLOCK:a * _BLOCK + n],
                m_scale=s["ms"].view(-1)[a:b] if eight else None, v_scale=s["vs"].view(-1)[a:b] if eight else None))
        s["step"] = Z.AdamTensorsStep(tensors)
        s["hp"] = [Z.adam_hparams(lr=_LR, beta1=_B1, beta2=_B2, eps=_EPS, weight_decay=w, step=_STEP) for w in _DECAY]
        if eight:
            s["mf"], s["vf"] = buf(s["p"].numel(), dtype=torch.float32), buf(s["p"].numel(), dtype=torch.float32)
    elif case["op"] == "norm":
        r, d, dt, st = case["rows"], case["features"], _DT[case["dtype"]], _DT[case["stream"]]
        s["kw"] = dict(branch=s["branch"], gate=s["gate"], gate_rows=s["per"], post=case["post"],
                       post_weight=s["post_w"], post_bias=s["post_b"], pre=case["pre"], pre_weight=s["pre_w"],
                       pre_bias=s["pre_b"], eps=_NORM_EPS, residual_scale=case["residual_scale"],
                       branch_scale=case["branch_scale"])
        if case["pass"] == "forward":
            s["y"], s["h"] = buf(r, d, dtype=st), buf(r, d, dtype=dt) if case["pre"] != "none" else None
        else:
            gdt = dt if case["grad"] == "same" else torch.float32
            s["grads"] = {"dx": buf(r, d, dtype=st), "dbranch": buf(r, d, dtype=dt),
                          "dgate": None if s["gate"] is None else buf(*s["gate"].shape, dtype=gdt)}
            for k in ("post_w", "post_b", "pre_w", "pre_b"):
                name = "d" + k.replace("_w", "_weight").replace("_b", "_bias")
                s["grads"][name] = None if s[k] is None else buf(d, dtype=gdt)
            s["ws"] = buf(Z.zero_norm_workspace_bytes(r, d, gate_rows=s["per"]), dtype=torch.uint8)
    else:
        rows = case["rows"]
        s["loss"] = buf(rows if case["op"] == "policy" else case["pairs"], dtype=torch.float32)
        s["logp"] = buf(rows, dtype=torch.float32)
        s["seq_logp"] = buf(2 * case["pairs"], dtype=torch.float32) if case["op"] == "preference" else None
        s["stats"] = buf(rows, Z.ZERO_TOKEN_STATS, dtype=torch.float32) if case["pass"] != "step" else None
        s["dlogits"] = torch.empty_like(s["logits"]) if case["pass"] != "forward" else None
    return s


# --------------------------------------------------------------------------------- the operators

def run(state):
    op = state["case"]["op"]
    if own:
        return {"adam": _adam_own, "norm": _norm_own, "policy": _policy_own, "preference": _preference_own}[op](state)
    return {"adam": _adam_plain, "norm": _norm_plain, "policy": _policy_plain, "preference": _preference_plain}[op](state)


def _adam_own(s):
    s["step"](s["hp"])
    outs = {"p": s["p"], "out": s["out"]}
    if s["case"]["bits"] == 32:
        return {**outs, "m": s["m"], "v": s["v"]}
    Z = s["Z"]
    Z.zero_adam_state_values(s["m"].view(-1), s["ms"].view(-1), s["mf"])
    Z.zero_adam_state_values(s["v"].view(-1), s["vs"].view(-1), s["vf"])
    return {**outs, "m_scale": s["ms"], "v_scale": s["vs"], "m": s["mf"], "v": s["vf"]}


def _norm_own(s):
    Z = s["Z"]
    if s["case"]["pass"] == "forward":
        Z.zero_norm_forward(s["x"], h=s["h"], y=s["y"], **s["kw"])
        return {"y": s["y"], "h": s["h"]}
    Z.zero_norm_backward(s["y"], s["stats"], dy=s["dy"], dh=s["dh"], workspace=s["ws"], **s["grads"], **s["kw"])
    return dict(s["grads"])


def _policy_own(s):
    case, Z = s["case"], s["Z"]
    args = (s["logits"], s["label"], s["old"], s["advantage"], s["loss"])
    kw = dict(ref_logp=s["ref"], weight=s["weight"], clip=(0.2, 0.28), kl_coef=case["kl"],
              temperature=case["temperature"], logp=s["logp"])
    if case["pass"] == "step":
        Z.zero_policy_step(*args, s["dlogits"], scale=s["scale"], **kw)
    else:
        Z.zero_policy_forward(*args, s["stats"], **kw)
        if case["pass"] == "both":
            Z.zero_token_backward(s["logits"], s["label"], s["stats"], s["dlogits"], scale=s["scale"],
                                  temperature=case["temperature"])
    return {"loss": s["loss"], "logp": s["logp"], "dlogits": s["dlogits"]}


def _preference_own(s):
    case, Z = s["case"], s["Z"]
    Z.zero_preference_forward(s["logits"], s["label"], s["start"], s["loss"], s["stats"], ref_logp=s["ref"],
                              weight=s["weight"], beta=s["beta"], label_smoothing=case["smoothing"],
                              average=case["average"], logp=s["logp"], seq_logp=s["seq_logp"])
    if case["pass"] == "both":
        Z.zero_token_backward(s["logits"], s["label"], s["stats"], s["dlogits"], scale=s["scale"])
    return {"loss": s["loss"], "logp": s["logp"], "seq_logp": s["seq_logp"], "dlogits": s["dlogits"]}


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float64).float())


def _constants(s):
    """The step's constants of each block, rounded once to 32 bits: divisors and factors as tensors, so that
    each is one operation of its own."""
    dev = [[_f32(_LR / (1 - _B1 ** _STEP)), _f32(math.sqrt(1 - _B2 ** _STEP)), _f32(1 - _LR * w)] for w in _DECAY]
    table = torch.tensor(dev, device=_DEV)[s["of"]]
    return table[:, 0:1], table[:, 1:2], table[:, 2:3]


def _code(x, scale, top):
    """The index, 0 to top, of the value nearest in square root: steps of (q/top)^2 below the block's
    largest, halves down; nothing but 0 becomes 0 in the unsigned form."""
    fine = (scale >= 2.0 ** -126) & (scale < math.inf)
    t = (x * (torch.ones_like(scale) / scale)) * float(top * top)
    q = torch.ceil(torch.sqrt(t.double()) - 0.5).clamp_(max=top)      # 64 bits: exact next to a half
    return torch.where(fine, q, torch.zeros_like(q)), fine


def _encode(x, top):
    """x [blocks, 256] as 8-bit indices and one scale for each block: 127 for signed values, 255 for square roots
    of second moments."""
    mag = x.abs()
    scale = mag.amax(1, keepdim=True)
    q, fine = _code(mag, scale, top)
    if top == 255:
        q = torch.where(fine & (x > 0), q.clamp(min=1), q)
        codes = q.to(torch.uint8)
    else:
        codes = torch.where(x < 0, -q, q).to(torch.int8)
    low = scale < 2.0 ** -126
    kept = torch.where(low, torch.zeros_like(scale), torch.full_like(scale, math.nan))
    return codes, torch.where(fine, scale, kept)


def _decode(codes, scale, top):
    q = codes.float()
    return (q * q.abs()) * (scale * _f32(1.0 / (top * top)))


def _adam_plain(s):
    eight = s["case"]["bits"] == 8
    ss, bc, dec = _constants(s)
    if eight:
        m, w = _decode(s["m"], s["ms"], 127), _decode(s["v"], s["vs"], 255)
        v = w * w
    else:
        m, v = s["m"], s["v"]
    g = s["g"].float()
    m = m * _f32(_B1) + g * _f32(1 - _B1)
    v = v * _f32(_B2) + (g * g) * _f32(1 - _B2)
    root = torch.sqrt(v)
    s["p"].copy_(s["p"] * dec - ss * (m / (root / bc + _f32(_EPS))))
    if s["out"] is not None:
        s["out"].copy_(s["p"])
    outs = {"p": s["p"], "out": s["out"]}
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {**outs, "m": s["m"], "v": s["v"]}
    for k, x, top in (("m", m, 127), ("v", root, 255)):
        codes, scale = _encode(x, top)
        s[k].copy_(codes)
        s[k + "s"].copy_(scale)
    w = _decode(s["v"], s["vs"], 255)
    return {**outs, "m_scale": s["ms"], "v_scale": s["vs"], "m": _decode(s["m"], s["ms"], 127).view(-1),
            "v": (w * w).view(-1)}


def _spread(s):
    """The gate of each row."""
    case = s["case"]
    if s["gate"] is None:
        return 1.0
    gate = s["gate"].float()
    return torch.repeat_interleave(gate, s["per"], 0)[:case["rows"]] if case["gate"] == "sequence" else gate


def _affine(v, w, b):
    if w is not None:
        v = v * w.float()
    return v if b is None else v + b.float()


def _norm_plain(s):
    case, dt, st = s["case"], _DT[s["case"]["dtype"]], _DT[s["case"]["stream"]]
    o = s["branch"].float()
    if case["pass"] == "forward":
        mean, rstd = _stats(o, case["post"])
        y = case["residual_scale"] * s["x"].float() + case["branch_scale"] * _spread(s) * _affine(
            (o - mean) * rstd, s["post_w"], s["post_b"])
        y = y.to(st)                       # the sum is an output of the stream's type; the norm is of it as it is stored
        if case["pre"] == "none":
            return {"y": y, "h": None}
        mean, rstd = _stats(y.float(), case["pre"])
        return {"y": y, "h": _affine((y.float() - mean) * rstd, s["pre_w"], s["pre_b"]).to(dt)}
    gdt = dt if case["grad"] == "same" else torch.float32
    out, d = {}, s["dy"].float()
    if case["pre"] != "none":
        dh = s["dh"].float()
        xh = (s["y"].float() - s["stats"][:, 2:3]) * s["stats"][:, 3:4]
        out["dpre_weight"] = (dh * xh).sum(0).to(gdt)
        out["dpre_bias"] = None if s["pre_b"] is None else dh.sum(0).to(gdt)
        d = d + _through(dh * s["pre_w"].float(), xh, s["stats"][:, 3:4], case["pre"])
    out["dx"] = (case["residual_scale"] * d).to(st)
    oh = (o - s["stats"][:, 0:1]) * s["stats"][:, 1:2]
    if s["gate"] is not None:
        each = case["branch_scale"] * d * _affine(oh, s["post_w"], s["post_b"])
        out["dgate"] = _by_gate(each, s["gate"].shape[0], s["per"]).to(gdt)
    e = case["branch_scale"] * _spread(s) * d
    if case["post"] != "none":
        out["dpost_weight"] = (e * oh).sum(0).to(gdt)
        out["dpost_bias"] = None if s["post_b"] is None else e.sum(0).to(gdt)
        e = _through(e * s["post_w"].float(), oh, s["stats"][:, 1:2], case["post"])
    out["dbranch"] = e.to(dt)
    return out


def _through(g, xh, rstd, kind):
    """The gradient through a norm from the gradient g of its normalised values xh."""
    g = g - xh * (g * xh).mean(1, keepdim=True) - (g.mean(1, keepdim=True) if kind == "layer" else 0.0)
    return g * rstd


def _by_gate(each, gates, per):
    if per == 1:
        return each
    if gates == 1:
        return each.sum(0, keepdim=True)
    pad = torch.zeros((gates * per - each.shape[0], each.shape[1]), dtype=each.dtype, device=each.device)
    return torch.cat([each, pad]).view(gates, per, -1).sum(1)


def _softmax_plain(s, temperature):
    """(exponentials, their sum, log probability of each row's token in 64 bits, the token's column)."""
    z = s["logits"].float() / temperature
    label = s["label"].long().clamp(min=0)[:, None]
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True, dtype=torch.float64)   # 64 bits: a policy's ratio is compared with its clip
    return e, total, ((z.gather(1, label) - top).double() - torch.log(total))[:, 0], label


def _gradient_plain(s, e, total, lp, label, slope, temperature):
    """slope * (1 at the token - probability), one rounding at the end."""
    coef = (slope * (s["scale"] / temperature))[:, None]
    grad = e * (-coef / total).float()
    grad.scatter_(1, label, (coef * -torch.expm1(lp)[:, None]).float())
    return torch.where(coef == 0, torch.zeros_like(grad), grad).to(s["logits"].dtype)


def _policy_plain(s):
    case = s["case"]
    e, total, lp, label = _softmax_plain(s, case["temperature"])
    a, on = s["advantage"].double(), s["weight"] != 0
    ratio = torch.exp(lp - s["old"].double())
    first, second = ratio * a, ratio.clamp(0.8, 1.28) * a
    loss, slope = -torch.minimum(first, second), torch.where(first <= second, -first, torch.zeros_like(first))
    if s["ref"] is not None:
        gap = s["ref"].double() - lp
        loss = loss + case["kl"] * (torch.expm1(gap) - gap)
        slope = slope - case["kl"] * torch.expm1(gap)
    w = s["weight"].double()
    out = {"loss": torch.where(on, w * loss, 0 * w).float(), "logp": torch.where(on, lp, 0 * w).float(), "dlogits": None}
    if case["pass"] != "forward":
        out["dlogits"] = _gradient_plain(s, e, total, lp, label, torch.where(on, w * slope, 0 * w), case["temperature"])
    return out


def _preference_plain(s):
    case = s["case"]
    e, total, lp, label = _softmax_plain(s, 1.0)
    on = s["label"] >= 0
    lp = torch.where(on, lp, torch.zeros_like(lp))
    seq = _segments(lp, s["start"])
    count = _segments(on.double(), s["start"]).clamp(min=1) if case["average"] else torch.ones_like(seq)
    gap = (seq / count - s["ref"].double()).view(-1, 2)
    x = s["beta"] * (gap[:, 0] - gap[:, 1])
    soft, w = case["smoothing"], s["weight"].double()
    loss = w * ((1 - soft) * torch.log1p(torch.exp(-x)) + soft * torch.log1p(torch.exp(x)))
    out = {"loss": loss.float(), "logp": lp.float(), "seq_logp": (seq / count).float(), "dlogits": None}
    if case["pass"] != "forward":
        slope = w * s["beta"] * (torch.sigmoid(x) - (1 - soft))
        each = torch.stack([slope, -slope], 1).view(-1) / count
        of = torch.searchsorted(s["start"][1:], torch.arange(case["rows"], device=_DEV), right=True)
        inside = on & (of < 2 * case["pairs"])
        each = torch.where(inside, each[of.clamp(max=2 * case["pairs"] - 1)], torch.zeros_like(lp))
        out["dlogits"] = _gradient_plain(s, e, total, lp, label, each, 1.0)
    return out


# ----------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = _INPUTS[case["op"]](case, seed)
    return {"adam": _adam_exact, "norm": _norm_exact, "policy": _policy_exact, "preference": _preference_exact}[case["op"]](s)


def _adam_exact(s):
    """The 8-bit indices are defined by the 32-bit moments, so they have no value in 64 bits; the scales do."""
    case = s["case"]
    p, g = s["p"].double(), s["g"].double()
    if case["bits"] == 8:
        k = s["m"].double()
        m = torch.sign(k) * (k / 127) ** 2 * s["ms"].double()
        v = ((s["v"].double() / 255) ** 2 * s["vs"].double()) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = _B1 * m + (1 - _B1) * g
    v = _B2 * v + (1 - _B2) * g ** 2
    m_hat, v_hat = m / (1 - _B1 ** _STEP), v / (1 - _B2 ** _STEP)
    decay = torch.tensor(_DECAY, dtype=torch.float64, device=_DEV)[s["of"]][:, None]
    p = p - _LR * decay * p - _LR * m_hat / (v_hat.sqrt() + _EPS)
    out = None if s["out"] is None else p
    if case["bits"] == 8:
        return {"p": p, "out": out, "m_scale": m.abs().max(1, keepdim=True).values,
                "v_scale": v.max(1, keepdim=True).values.sqrt(), "m": None, "v": None}
    return {"p": p, "out": out, "m": m, "v": v}


def _unit(v, kind):
    """A row in units of its own deviation, and that deviation."""
    if kind == "none":
        return v, torch.ones_like(v[:, :1])
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    dev = (c.square().mean(1, keepdim=True) + _NORM_EPS).sqrt()
    return c / dev, dev


def _norm_exact(s):
    case = s["case"]
    vec = {k: None if s[k] is None else s[k].double() for k in ("post_w", "post_b", "pre_w", "pre_b")}
    of = torch.arange(case["rows"], device=_DEV) // s["per"]
    gate = torch.ones((1, 1), dtype=torch.float64, device=_DEV) if s["gate"] is None else s["gate"].double()[of]
    gate = gate * case["branch_scale"]
    oh, odev = _unit(s["branch"].double(), case["post"])
    value = oh if vec["post_w"] is None else oh * vec["post_w"]
    value = value if vec["post_b"] is None else value + vec["post_b"]
    if case["pass"] == "forward":
        y = case["residual_scale"] * s["x"].double() + gate * value
        if case["pre"] == "none":
            return {"y": y, "h": None}
        h = _unit(y.to(_DT[case["stream"]]).double(), case["pre"])[0] * vec["pre_w"]
        return {"y": y, "h": h if vec["pre_b"] is None else h + vec["pre_b"]}
    n = case["features"]

    def back(g, unit, dev, kind):
        if kind == "none":
            return g
        dot = torch.sum(g * unit, 1, keepdim=True) / n
        rest = torch.sum(g, 1, keepdim=True) / n if kind == "layer" else 0.0
        return (g - rest - unit * dot) / dev

    out, d = {}, s["dy"].double()
    if case["pre"] != "none":
        dh = s["dh"].double()
        xh, xdev = _unit(s["y"].double(), case["pre"])
        out["dpre_weight"] = torch.sum(dh * xh, 0)
        out["dpre_bias"] = None if vec["pre_b"] is None else torch.sum(dh, 0)
        d = d + back(dh * vec["pre_w"], xh, xdev, case["pre"])
    out["dx"] = d * case["residual_scale"]
    if s["gate"] is not None:
        sums = torch.zeros(s["gate"].shape, dtype=torch.float64, device=_DEV)
        out["dgate"] = sums.index_add_(0, of, d * value * case["branch_scale"])
    e = d * gate
    if case["post"] != "none":
        out["dpost_weight"] = torch.sum(e * oh, 0)
        out["dpost_bias"] = None if vec["post_b"] is None else torch.sum(e, 0)
        e = e * vec["post_w"]
    out["dbranch"] = back(e, oh, odev, case["post"])
    return out


def _rows_exact(s, temperature, slopes):
    """(log probabilities, gradient) by blocks of rows, so that the 64-bit copies of the largest case stay small;
    `slopes` turns all rows' log probabilities into the loss's derivatives in them."""
    case = s["case"]
    step = max(1, (1 << 27) // case["vocab"])
    cols = s["label"].long().clamp(min=0)[:, None]
    blocks = list(zip(s["logits"].split(step), cols.split(step)))
    lp = torch.cat([torch.log_softmax(z.double() / temperature, 1).gather(1, c)[:, 0] for z, c in blocks])
    slope = slopes(lp)
    if case["pass"] == "forward":
        return lp, None
    grads = []
    for (z, c), k in zip(blocks, (slope * s["scale"] / temperature)[:, None].split(step)):
        q = torch.softmax(z.double() / temperature, 1)
        grads.append(torch.zeros_like(q).scatter_(1, c, 1.0).sub_(q).mul_(k))
    return lp, torch.cat(grads)


def _policy_exact(s):
    case, w = s["case"], s["weight"].double()
    a, kept = s["advantage"].double(), {}

    def slopes(lp):
        ratio = (lp - s["old"].double()).exp()
        stops = torch.where(a > 0, ratio > 1.28, (ratio < 0.8) & (a < 0))
        bound = torch.where(a > 0, torch.full_like(a, 1.28), torch.full_like(a, 0.8))
        kept["loss"] = -a * torch.where(stops, bound, ratio)
        slope = -a * ratio * (~stops)
        if s["ref"] is not None:
            gap = s["ref"].double() - lp
            kept["loss"] = kept["loss"] + case["kl"] * (gap.exp() - 1 - gap)
            slope = slope + case["kl"] * (1 - gap.exp())
        return w * slope

    lp, grad = _rows_exact(s, case["temperature"], slopes)
    return {"loss": w * kept["loss"], "logp": lp * (w != 0), "dlogits": grad}


def _preference_exact(s):
    case, pairs, kept = s["case"], s["case"]["pairs"], {}
    ends = s["start"].tolist()

    def slopes(lp):
        on = s["label"] >= 0
        kept["lp"] = lp = lp * on
        spans = list(zip(ends[:-1], ends[1:]))
        n = [max(1, int(on[a:b].sum())) if case["average"] else 1 for a, b in spans]
        kept["seq"] = seq = torch.stack([lp[a:b].sum() / k for (a, b), k in zip(spans, n)])
        gap = seq - s["ref"].double()
        x = s["beta"] * (gap[0::2] - gap[1::2])
        soft, w = case["smoothing"], s["weight"].double()
        log_sigmoid = torch.nn.functional.logsigmoid
        kept["loss"] = -w * ((1 - soft) * log_sigmoid(x) + soft * log_sigmoid(-x))
        each = w * s["beta"] * (soft * torch.sigmoid(x) - (1 - soft) * torch.sigmoid(-x))
        slope = torch.zeros_like(lp)
        for i, (a, b) in enumerate(spans):
            slope[a:b] = (each[i // 2] if i % 2 == 0 else -each[i // 2]) / n[i]
        return slope * on

    _, grad = _rows_exact(s, 1.0, slopes)
    return {"loss": kept["loss"], "logp": kept["lp"], "seq_logp": kept["seq"], "dlogits": grad}
