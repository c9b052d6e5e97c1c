"""Float64 CPU oracle of the gated feed-forward block and the top-logit distillation loss.

Test infrastructure only.  Inputs are float64 arrays holding the exact values
of the operators' bf16, fp16 or float32 inputs; it shares no code with the HIP path.
"""

from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])
ACTS = ("silu", "gelu", "gelu_tanh")


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act_and_slope(g: np.ndarray, act: str):
    """act(g) and its derivative."""
    if act == "silu":
        s = _sigmoid(g)
        return g * s, s + g * s * _sigmoid(-g)
    if act == "gelu":
        cdf = 0.5 * _erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        r = 2.0 * math.sqrt(2.0 / math.pi)
        s = _sigmoid(r * (g + 0.044715 * g ** 3))
        return g * s, s + g * s * (1.0 - s) * r * (1.0 + 3.0 * 0.044715 * g * g)
    raise ValueError(act)


def gated_ffn(x, w_gate, w_up, act):
    """(h, g, u): the block's output and its pre-activations."""
    g, u = x @ w_gate.T, x @ w_up.T
    return act_and_slope(g, act)[0] * u, g, u


def gated_ffn_grads(dh, x, w_gate, w_up, g, u, act):
    """(dx, dw_gate, dw_up, dg, du) of sum(dh * h) at the pre-activations g, u."""
    a, slope = act_and_slope(g, act)
    dg, du = dh * u * slope, dh * a
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x, dg, du


def distill_topk(logits, ids, values, weight, temperature):
    """(loss, stats, grad): each row's weighted divergence, (max, sum exp(. - max)) of logits / T, its gradient.

    Entries with a negative id or a value of -infinity are absent; a row of weight 0 or without a
    present entry has loss 0, a zero gradient and zero statistics; an id past the vocabulary gives NaN,
    whatever its value.
    """
    n, vocab = logits.shape
    loss, stats, grad = np.zeros(n), np.zeros((n, 2)), np.zeros((n, vocab))
    for r in range(n):
        here = (ids[r] >= 0) & ~(values[r] == -np.inf)
        if weight[r] == 0.0:
            continue
        if (ids[r] >= vocab).any():
            loss[r], stats[r], grad[r] = np.nan, np.nan, np.nan
            continue
        if not here.any():
            continue
        with np.errstate(all="ignore"):
            z = logits[r] / temperature
            m = z.max()
            e = np.exp(z - m)
            s = e.sum()
            stats[r] = m, s
            v = values[r][here] / temperature
            t = v - v.max()
            logp = t - np.log(np.exp(t).sum())
            p = np.exp(logp)
            j = ids[r][here]
            # a student logit of -infinity where the teacher has mass: an infinite loss
            loss[r] = weight[r] * sum(pi * (li - (z[ji] - m - np.log(s))) for pi, li, ji in zip(p, logp, j) if pi != 0.0)
            q = e / s
            np.subtract.at(q, j, p)
            grad[r] = weight[r] / temperature * q
    return loss, stats, grad


def quantize_rows(x):
    """(codes, scales) of rows: rint(127 x / a) with a = max |x|, ties to even, and a / 127."""
    codes, scales = np.zeros(x.shape), np.zeros(x.shape[0])
    for r, v in enumerate(x):
        if not np.isfinite(v).all():
            scales[r] = np.nan
            continue
        a = np.abs(v).max()
        if a > 0.0:
            codes[r] = np.rint(127.0 * v / a)
        scales[r] = a / 127.0
    return codes, scales


def quantize_blocks(x, block=32):
    """(codes, steps) of blocks of 32 columns: s the power of two with 64 <= a / s < 128, at least 2^-126."""
    n, d = x.shape
    groups = -(-d // block)
    codes, steps = np.zeros((n, d)), np.zeros((n, groups))
    for r in range(n):
        for b in range(groups):
            v = x[r, b * block:(b + 1) * block]
            if not np.isfinite(v).all():
                steps[r, b] = np.nan
                continue
            s, a = 2.0 ** -126, np.abs(v).max()
            while a / s >= 128.0:
                s *= 2.0
            codes[r, b * block:(b + 1) * block] = np.clip(np.rint(v / s), -127, 127)
            steps[r, b] = s
    return codes, steps


def stand_for(codes, steps, block=32):
    """What the codes of blocks stand for."""
    return codes * np.repeat(steps, block, axis=1)[:, :codes.shape[1]]
