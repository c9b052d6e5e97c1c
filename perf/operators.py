"""The measured cases of the gated feed-forward block and of the top-logit distillation loss.

``own`` false: each operator in elementary torch operations, in float32 (float64 for the few terms
of the loss that cancel), rounded once at the end.  ``own`` true: the calls a user of the package
makes.  ``exact`` gives the same outputs from the definitions in float64.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ID = {"i32": torch.int32, "i64": torch.int64}
_ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


def _ffn(name, mode, dtype, n, d, f, act):
    return {"name": name, "op": "ffn", "mode": mode, "dtype": dtype, "n": n, "d": d, "f": f, "act": act}


def _distill(name, mode, dtype, n, vocab, k, ids, masked, absent, temperature):
    return {"name": name, "op": "distill", "mode": mode, "dtype": dtype, "n": n, "vocab": vocab, "k": k, "ids": ids,
            "masked": masked, "absent": absent, "temperature": temperature}


def listed():
    return [
        # one token through the block: serving the calibrated model, where latency counts
        _ffn("ffn_token", "forward", "bf16", 1, 4096, 11264, "silu"),
        # a few requests decoded together, the other 16-bit type and activation
        _ffn("ffn_tokens", "forward", "f16", 24, 2560, 9728, "gelu"),
        # one ragged calibration batch on its way to the Hessian of the next layer
        _ffn("ffn_calibration", "forward", "bf16", 1999, 2560, 9728, "silu"),
        # a long prompt, or a large calibration batch
        _ffn("ffn_long", "forward", "bf16", 16384, 4096, 11264, "silu"),
        # one training step of the block (forward, then all three gradients) at full size
        _ffn("ffn_train", "train", "bf16", 8192, 4096, 11264, "silu"),
        # the same at sizes that fit no tile and no 16-byte row
        _ffn("ffn_train_odd", "train", "f16", 777, 1001, 2731, "gelu_tanh"),
        # a small float32 block
        _ffn("ffn_train_f32", "train", "f32", 500, 1024, 2816, "silu"),
        # the last few tokens of one sample, loss and gradient in one call: latency
        _distill("distill_few", "step", "bf16", 4, 32000, 32, "i64", 0.0, 0.0, 1.0),
        # a padded batch over an odd vocabulary (rows not 16-byte aligned), teacher lists cut short
        _distill("distill_odd", "step", "bf16", 2047, 50001, 64, "i64", 0.25, 0.3, 2.0),
        # a full training batch over a large vocabulary
        _distill("distill_long", "step", "bf16", 8192, 131072, 128, "i32", 0.0, 0.0, 1.0),
        # judging a quantized model: the loss alone, float32 logits
        _distill("distill_eval", "forward", "f32", 1024, 65537, 20, "i32", 0.0, 0.0, 1.0),
        # forward now, backward later with a gradient for each row from the caller
        _distill("distill_parts", "parts", "f16", 1000, 100000, 256, "i64", 0.1, 0.0, 1.5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    if rng.random() < 0.5:
        mode = rng.choice(["forward", "forward", "train"])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        # single tokens to long batches; one in two widths is a multiple of 64, the others are any
        step_d, step_f = rng.choice([1, 64]), rng.choice([1, 64])
        d = max(step_d, _log_int(rng, 128, 4096) // step_d * step_d)
        f = max(step_f, _log_int(rng, 128, 11264) // step_f * step_f)
        n = _log_int(rng, 1, 16384) if mode == "forward" else _log_int(rng, 64, 8192)
        if dtype == "f32":
            n = min(n, 4096)
        return {"op": "ffn", "mode": mode, "dtype": dtype, "n": n, "d": d, "f": f,
                "act": rng.choice(["silu", "gelu", "gelu_tanh"])}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    vocab = _log_int(rng, 1000, 131072)
    n = _log_int(rng, 1, 8192)
    if dtype == "f32":
        n = min(n, 4096)
    return {"op": "distill", "mode": rng.choice(["step", "step", "forward", "parts"]), "dtype": dtype, "n": n,
            "vocab": vocab, "k": _log_int(rng, 1, 256), "ids": rng.choice(["i32", "i64"]),
            "masked": rng.choice([0.0, 0.1, 0.4]), "absent": rng.choice([0.0, 0.3]),
            "temperature": rng.choice([1.0, 1.5, 2.0])}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = _generator(seed)
    dtype = _DT[case["dtype"]]
    n = case["n"]
    if case["op"] == "ffn":
        d, f = case["d"], case["f"]
        # activations with the spread of column scales that calibration inputs have; weights that keep
        # the projections' scale near one
        x = (_normal(gen, n, d) * torch.exp(0.5 * _normal(gen, d))).to(dtype)
        packed = (_normal(gen, 2 * f, d) * (0.7 / math.sqrt(d))).to(dtype)
        state = {"case": case, "x": x, "w_gate": packed[:f], "w_up": packed[f:]}
        if case["mode"] == "train":
            state["dh"] = _normal(gen, n, f).to(dtype)
        return state
    vocab, k = case["vocab"], case["k"]
    # the teacher's entries: distinct ids, logits falling off with the rank
    gaps = torch.randint(1, vocab // k + 1, (n, k), generator=gen, device="cuda")
    ids = gaps.cumsum(1) - 1
    ids = ids.gather(1, torch.rand(n, k, generator=gen, device="cuda").argsort(1))
    rank = torch.arange(1, k + 1, device="cuda", dtype=torch.float32)
    values = 14.0 - 1.5 * torch.log(rank) + 0.3 * _normal(gen, n, k)
    # the student agrees with it up to noise
    logits = torch.empty(n, vocab, dtype=dtype, device="cuda")
    rows = max(1, (1 << 28) // vocab)
    for r in range(0, n, rows):
        part = 2.0 * _normal(gen, min(rows, n - r), vocab)
        part.scatter_(1, ids[r:r + rows], values[r:r + rows] - 3.0 + _normal(gen, part.shape[0], k))
        logits[r:r + rows] = part.to(dtype)
    if case["absent"] > 0.0:
        # lists cut short: rank r is absent where the row keeps fewer
        keep = (k * (1.0 - 2.0 * case["absent"] * torch.rand(n, 1, generator=gen, device="cuda"))).ceil()
        ids = torch.where(rank[None, :] <= keep, ids, torch.full_like(ids, -1))
    weight = torch.rand(n, generator=gen, device="cuda") + 0.5
    if dtype == torch.float16:
        weight *= 1024.0  # loss scaling, without which float16 gradients underflow
    off = int(n * case["masked"])
    if off:
        weight[torch.randperm(n, generator=gen, device="cuda")[:off]] = 0.0
    state = {"case": case, "logits": logits, "ids": ids.to(_ID[case["ids"]]), "values": values, "weight": weight}
    if case["mode"] == "parts":
        state["dloss"] = torch.rand(n, generator=gen, device="cuda") + 0.5
    return state


def _act(g, act):
    """The activation and its derivative, float32."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_ffn(state):
    case, dtype = state["case"], state["x"].dtype
    x, wg, wu = state["x"].float(), state["w_gate"].float(), state["w_up"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(g, case["act"])
    h = (a * u).to(dtype)
    if case["mode"] == "forward":
        return h
    dh = state["dh"].float()
    dg, du = dh * u * da, dh * a
    dx = dg @ wg + du @ wu
    return h, dx.to(dtype), (dg.t() @ x).to(dtype), (du.t() @ x).to(dtype)


def _plain_distill(state):
    case = state["case"]
    z = state["logits"].float() / case["temperature"]
    live = state["weight"] != 0.0
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total)).double()
    present = state["ids"] >= 0
    ids = torch.where(present, state["ids"], 0).long()
    v = torch.where(present, state["values"].double() / case["temperature"], -math.inf)
    top = v.amax(1, keepdim=True)
    ev = torch.exp(v - top)
    tot = ev.sum(1, keepdim=True)
    p = ev / tot
    term = p * ((v - top - torch.log(tot)) - (z.gather(1, ids).double() - lse))
    loss = torch.where(present & (p > 0.0), term, 0.0).sum(1) * state["weight"].double()
    loss = torch.where(live, loss, 0.0).float()
    if case["mode"] == "forward":
        return loss
    scale = state["weight"] / case["temperature"]
    if case["mode"] == "parts":
        scale = scale * state["dloss"]
    q = e / total
    q.scatter_add_(1, ids, torch.where(present, -p, 0.0).float())
    grad = torch.where(live[:, None], q * scale[:, None], 0.0)
    return loss, grad.to(state["logits"].dtype)


def run(state):
    case = state["case"]
    if not own:
        return _plain_ffn(state) if case["op"] == "ffn" else _plain_distill(state)
    import gptq_hessian_accumulation_amd as hs
    if case["op"] == "ffn":
        x, wg, wu = state["x"], state["w_gate"], state["w_up"]
        if case["mode"] == "forward":
            return hs.gated_ffn_forward(x, wg, wu, act=case["act"])
        h, preact = hs.gated_ffn_forward(x, wg, wu, act=case["act"], save=True)
        dx, dwg, dwu = hs.gated_ffn_backward(state["dh"], x, wg, wu, preact, act=case["act"])
        return h, dx, dwg, dwu
    z, ids, values, weight, t = (state["logits"], state["ids"], state["values"], state["weight"],
                                 case["temperature"])
    if case["mode"] == "forward":
        return hs.distill_topk_forward(z, ids, values, weight=weight, temperature=t)[0]
    if case["mode"] == "step":
        return hs.distill_topk_step(z, ids, values, weight=weight, temperature=t)
    loss, lse = hs.distill_topk_forward(z, ids, values, weight=weight, temperature=t)
    return loss, hs.distill_topk_backward(state["dloss"], z, ids, values, lse, weight=weight, temperature=t)


def work(case):
    e, n = _ESIZE[case["dtype"]], case["n"]
    if case["op"] == "ffn":
        d, f = case["d"], case["f"]
        if case["mode"] == "forward":
            return {"bytes": e * (n * d + 2 * f * d + n * f), "flops": 4 * n * d * f}
        return {"bytes": e * (2 * n * d + 4 * f * d + 2 * n * f), "flops": 12 * n * d * f}
    vocab, k = case["vocab"], case["k"]
    live = n - int(n * case["masked"])
    entries = live * k * (4 + (8 if case["ids"] == "i64" else 4))
    if case["mode"] == "forward":
        return {"bytes": e * live * vocab + entries + 8 * n, "flops": 4 * live * vocab}
    return {"bytes": e * (live + n) * vocab + entries + 8 * n, "flops": 7 * live * vocab}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "ffn":
        x, dh = state["x"].double(), state.get("dh")
        wg, wu = state["w_gate"].double(), state["w_up"].double()
        g = torch.mm(x, wg.t())
        u = torch.mm(x, wu.t())
        if case["act"] == "silu":
            sig = torch.sigmoid(g)
            a, slope = g * sig, sig + g * sig * torch.sigmoid(-g)
        elif case["act"] == "gelu":
            phi = 0.5 * torch.erfc(-g / math.sqrt(2.0))
            a, slope = g * phi, phi + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
        else:
            # (1 + tanh(s)) / 2 = sigmoid(2 s)
            two_s = 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
            sig = torch.sigmoid(two_s)
            a = g * sig
            slope = sig + g * sig * torch.sigmoid(-two_s) * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * g * g)
        h = a * u
        if case["mode"] == "forward":
            return h
        dh = dh.double()
        dg, du = dh * u * slope, dh * a
        return h, torch.mm(dg, wg) + torch.mm(du, wu), torch.mm(dg.t(), x), torch.mm(du.t(), x)
    n, vocab, t = case["n"], case["vocab"], case["temperature"]
    loss = torch.zeros(n, dtype=torch.float64, device="cuda")
    grad = None if case["mode"] == "forward" else torch.zeros(n, vocab, dtype=torch.float64, device="cuda")
    rows = max(1, (1 << 27) // vocab)
    for r in range(0, n, rows):
        logq = torch.log_softmax(state["logits"][r:r + rows].double() / t, 1)
        ids = state["ids"][r:r + rows].long()
        w = state["weight"][r:r + rows].double()
        v = (state["values"][r:r + rows].double() / t).masked_fill(ids < 0, -math.inf)
        logp = torch.log_softmax(v, 1)
        p = logp.exp()
        pick = ids.clamp(min=0)
        terms = torch.where(p > 0.0, p * (logp - logq.gather(1, pick)), torch.zeros_like(p))
        loss[r:r + rows] = terms.sum(1) * w
        if grad is not None:
            dz = logq.exp_().scatter_add_(1, pick, -p)
            c = w / t
            if case["mode"] == "parts":
                c = c * state["dloss"][r:r + rows].double()
            grad[r:r + rows] = dz.mul_(c[:, None])
    return loss if grad is None else (loss, grad)
