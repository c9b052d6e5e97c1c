"""The measured cases of the 8-bit integer product and of 8-bit activation checkpoints.

``own`` false: each operator in elementary torch operations, in float32 (float64 for the codes of given
values, which next to a border need it), rounded once at the end.  ``own`` true: the calls a user of the
package makes.  ``exact`` gives the same outputs from the definitions in float64.

Codes, whole numbers to nearest, ties to even.  A row with a scale of its own: with a its largest magnitude,
a value x is held as 127 x / a and stands for that times a / 127.  In blocks of 32 columns: x is held as x / s and
stands for that times s, s the power of two with 64 <= a / s < 128 for the block's largest magnitude a, and
none past 127 in magnitude.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


def _linear(name, dtype, n, d, f, bits):
    return {"name": name, "op": "linear", "dtype": dtype, "n": n, "d": d, "f": f, "bits": bits}


def _step(name, dtype, n, d, f):
    return {"name": name, "op": "step", "dtype": dtype, "n": n, "d": d, "f": f}


def _ffn(name, dtype, n, d, f, act):
    return {"name": name, "op": "ffn", "dtype": dtype, "n": n, "d": d, "f": f, "act": act}


def _store(name, dtype, n, d, block):
    return {"name": name, "op": "store", "dtype": dtype, "n": n, "d": d, "block": block}


def listed():
    return [
        # one token through a projection in 8-bit integers, its 4-bit codes a calibrated quantization's:
        # serving, where latency counts
        _linear("linear_token", "bf16", 1, 4096, 11264, 4),
        # a few requests decoded together, the other 16-bit type, codes of 8 bits
        _linear("linear_tokens", "f16", 24, 2560, 9728, 8),
        # one ragged batch of prompts
        _linear("linear_batch", "bf16", 1999, 2560, 9728, 4),
        # a long prompt
        _linear("linear_long", "bf16", 16384, 4096, 11264, 8),
        # float32 activations, sizes that fit no tile and no 16-byte row
        _linear("linear_odd", "f32", 777, 1001, 2731, 8),
        # one training step of a projection that computes in 8 bits (forward, both gradients) at full size
        _step("step", "bf16", 8192, 4096, 11264),
        # the same at odd sizes
        _step("step_odd", "f16", 777, 1001, 2731),
        # a small float32 projection
        _step("step_small", "f32", 300, 704, 1000),
        # one training step of the feed-forward block, what it keeps for the backward pass held in 8 bits
        _ffn("ffn_step", "bf16", 8192, 4096, 11264, "silu"),
        # the same at odd sizes
        _ffn("ffn_step_odd", "f16", 777, 1001, 2731, "gelu_tanh"),
        # activations of a long batch stored for later and restored, block by block
        _store("store_long", "bf16", 16384, 11264, 32),
        # a short batch of float32 rows, a scale a row
        _store("store_rows", "f32", 300, 2731, 0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "step", "ffn", "store"])
    # one in two widths is a multiple of 64, the others are any
    step_d, step_f = rng.choice([1, 64]), rng.choice([1, 64])
    d = max(step_d, _log_int(rng, 128, 4096) // step_d * step_d)
    f = max(step_f, _log_int(rng, 128, 11264) // step_f * step_f)
    if op == "linear":
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "n": _log_int(rng, 1, 16384), "d": d,
                "f": f, "bits": rng.choice([4, 8])}
    if op == "step":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        n = _log_int(rng, 64, 8192)
        return {"op": op, "dtype": dtype, "n": min(n, 4096) if dtype == "f32" else n, "d": d, "f": f}
    if op == "ffn":
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"]), "n": _log_int(rng, 256, 8192), "d": d, "f": f,
                "act": rng.choice(["silu", "gelu", "gelu_tanh"])}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    n = _log_int(rng, 1, 16384)
    return {"op": op, "dtype": dtype, "n": min(n, 8192) if dtype == "f32" else n, "d": f, "block": rng.choice([0, 32])}


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, n, d = _DT[case["dtype"]], case["n"], case["d"]
    # activations with the spread of column scales that calibration inputs have
    x = (_normal(gen, n, d) * torch.exp(0.5 * _normal(gen, d))).to(dtype)
    state = {"case": case, "x": x}
    if case["op"] == "store":
        return state
    f = case["f"]
    if case["op"] == "linear":
        # weights as a quantization left them: whole codes and a step for each output channel
        w = _normal(gen, f, d)
        top = 2 ** (case["bits"] - 1) - 1
        step = w.abs().amax(1) / top
        state["codes"] = (w / step[:, None]).round().clamp(-top, top).to(torch.int8)
        state["scale"] = step * (0.7 / math.sqrt(d))
        return state
    # weights that keep the outputs' scale near one
    if case["op"] == "step":
        state["w"] = (_normal(gen, f, d) * (0.7 / math.sqrt(d))).to(dtype)
    else:
        packed = (_normal(gen, 2 * f, d) * (0.7 / math.sqrt(d))).to(dtype)
        state["w_gate"], state["w_up"] = packed[:f], packed[f:]
    state["dout"] = _normal(gen, n, f).to(dtype)
    return state


def _hold(x, block):
    """The codes of x's rows, and the scale at each place (block 0: of each row), in x's type."""
    if block == 0:
        top = x.abs().amax(1, keepdim=True)
        return torch.round(x * 127.0 / torch.where(top > 0.0, top, 1.0)), top / 127.0
    n, d = x.shape
    groups = -(-d // block)
    xb = torch.nn.functional.pad(x, (0, groups * block - d)).view(n, groups, block)
    top = xb.abs().amax(2, keepdim=True)
    top = torch.where(top > 0.0, top, 1.0)
    part = torch.frexp(top)[0]  # top / part is a power of two, and the quotient exact
    step = top / part / 128.0
    q, step = torch.round(xb / step).clamp(-127.0, 127.0), step.expand(-1, -1, block)
    return q.view(n, groups * block)[:, :d], step.reshape(n, groups * block)[:, :d]


def _held(x, block):
    """What the codes of x stand for, float32 (the codes and scales formed in x's type)."""
    q, s = _hold(x, block)
    return (q * s).float()


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


def _plain(state):
    case, x = state["case"], state["x"]
    dtype = x.dtype
    if case["op"] == "store":
        q, s = _hold(x.double(), case["block"])
        return (q * s).to(dtype)
    if case["op"] == "linear":
        q, s = _hold(x.double(), 0)
        return ((q.float() @ state["codes"].float().t()) * s.float() * state["scale"]).to(dtype)
    dout = state["dout"].float()
    if case["op"] == "step":
        xh, wh = _held(x.double(), 0), _held(state["w"].double(), 0)
        return (xh @ wh.t()).to(dtype), (dout @ wh).to(dtype), (dout.t() @ xh).to(dtype)
    wg, wu = state["w_gate"].float(), state["w_up"].float()
    g, u = x.float() @ wg.t(), x.float() @ wu.t()
    h = (_act(g, case["act"])[0] * u).to(dtype)
    gh, uh, xh = _held(g, 32), _held(u, 32), _held(x.double(), 32)
    a, da = _act(gh, case["act"])
    dg, du = dout * uh * da, dout * a
    return h, (dg @ wg + du @ wu).to(dtype), (dg.t() @ xh).to(dtype), (du.t() @ xh).to(dtype)


def run(state):
    if not own:
        return _plain(state)
    import gptq_hessian_accumulation_amd as hs
    case, x = state["case"], state["x"]
    if case["op"] == "store":
        return hs.dequantize_int8(hs.quantize_int8(x, block=case["block"]), dtype=x.dtype)
    if case["op"] == "linear":
        return hs.int8_linear_forward(x, hs.Int8Rows(state["codes"], state["scale"]))
    if case["op"] == "step":
        w8 = hs.quantize_int8(state["w"])
        y, x8 = hs.int8_linear_forward(x, w8, save=True)
        dx, dw = hs.int8_linear_backward(state["dout"], x8, w8)
        return y, dx, dw
    wg, wu, act = state["w_gate"], state["w_up"], case["act"]
    x8 = hs.quantize_int8(x, block=32)
    h, pre = hs.gated_ffn_forward(x, wg, wu, act=act, save=torch.int8)
    dx, dwg, dwu = hs.gated_ffn_backward(state["dout"], x8, wg, wu, pre, act=act)
    return h, dx, dwg, dwu


def work(case):
    e, n, d = _ESIZE[case["dtype"]], case["n"], case["d"]
    if case["op"] == "store":
        scales = 4 * n if case["block"] == 0 else n * -(-d // case["block"])
        return {"bytes": 2 * e * n * d + 2 * (n * d + scales), "flops": 4 * n * d}
    f = case["f"]
    if case["op"] == "linear":
        return {"bytes": e * n * (d + f) + f * (d + 4), "flops": 2 * n * d * f}
    if case["op"] == "step":
        return {"bytes": 2 * e * (n * d + f * d + n * f), "flops": 6 * n * d * f}
    # what is held for the backward pass is written and read: 8 bits a value and for 32 of them
    return {"bytes": e * (2 * n * d + 4 * f * d + 2 * n * f) + 2 * (n * d + 2 * n * f) * 33 // 32,
            "flops": 12 * n * d * f}


def exact(case, seed):
    state = prepare(case, seed)
    x = state["x"].double()

    def rows(v):
        """(whole codes, what one of them stands for) of rows with a scale of their own."""
        big = torch.linalg.vector_norm(v, ord=math.inf, dim=1, keepdim=True)
        return torch.where(big > 0.0, (127.0 * v) / big, torch.zeros_like(v)).round(), big[:, 0] / 127.0

    def held(v):
        """What the codes of v's blocks of 32 columns stand for."""
        n, d = v.shape
        out = torch.zeros_like(v)
        whole = d // 32 * 32
        for lo, hi, width in ((0, whole, 32), (whole, d, d - whole)):
            if hi == lo:
                continue
            part = v[:, lo:hi].reshape(n, -1, width)
            big = torch.linalg.vector_norm(part, ord=math.inf, dim=2, keepdim=True)
            # the power of two in big's exponent bits, less 6
            unit = (((big.view(torch.int64) >> 52) - 6).clamp(min=1) << 52).view(torch.float64)
            out[:, lo:hi] = torch.where(big > 0.0, (part / unit).round().clamp(-127.0, 127.0) * unit, torch.zeros_like(part)).reshape(n, -1)
        return out

    if case["op"] == "store":
        if case["block"] == 32:
            return held(x)
        q, unit = rows(x)
        return q * unit[:, None]
    if case["op"] == "linear":
        q, unit = rows(x)
        # whole sums below 2^53: nothing is lost before the scales
        return torch.mm(q, state["codes"].double().t()) * torch.outer(unit, state["scale"].double())
    dout = state["dout"].double()
    if case["op"] == "step":
        q, unit = rows(x)
        p, each = rows(state["w"].double())
        y = torch.mm(q, p.t()) * torch.outer(unit, each)
        return y, torch.mm(dout * each, p), torch.mm((dout * unit[:, None]).t(), q)
    wg, wu, act = state["w_gate"].double(), state["w_up"].double(), case["act"]

    def phi(g):
        """The factor of g in the activation, and its derivative."""
        if act == "silu":
            s = torch.sigmoid(g)
            return s, s * torch.sigmoid(-g)
        if act == "gelu":
            return 0.5 * torch.erfc(-g / math.sqrt(2.0)), torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
        r = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(r * (g + 0.044715 * g ** 3))
        return s, s * (1.0 - s) * r * (1.0 + 0.134145 * g * g)

    g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    h = g * phi(g)[0] * u
    g, u, xh = held(g), held(u), held(x)
    p, dp = phi(g)
    dg, du = dout * u * (p + g * dp), dout * g * p
    return h, torch.mm(dg, wg) + torch.mm(du, wu), torch.mm(dg.t(), xh), torch.mm(du.t(), xh)
