"""Every tile kernel of the feed-forward block: each type, product and edge, whole, split along K, and both at once.

Tolerances are those of test_gated_ffn_gpu.py, derived there.
"""

import numpy as np
import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from oracle import ops_oracle as R
from tests import test_gated_ffn_gpu as G

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X GPU")]


@pytest.fixture(autouse=True)
def automatic():
    yield
    hs.set_ffn_schedule(0)


def check_all(n, d, f, dt, act, save):
    """The three products at small sizes against the oracle."""
    x, xn = G.draw(91, dt, n, d)
    wg, gn = G.draw(92, dt, f, d, scale=1.5 / d ** 0.5)
    wu, un = G.draw(93, dt, f, d, scale=1.5 / d ** 0.5)
    dh, dn = G.draw(94, dt, n, f)
    h, pre = hs.gated_ffn_forward(x, wg, wu, act=act, save=save)
    want, g, u = R.gated_ffn(xn, gn, un, act)
    th, tg, tu = G.forward_tolerance(xn, gn, un, g, u, act, dt)
    G.check("h", h, want, th)
    fp = -(-f // 8) * 8
    G.check("g", pre[:, :f], g, tg)
    G.check("u", pre[:, fp:fp + f], u, tu)
    assert not pre[:, f:fp].any() and not pre[:, fp + f:].any()
    pair, g, u = G.exact_preact(g, u, dt, f)
    grads = hs.gated_ffn_backward(dh, x, wg, wu, pair, act=act)
    *want, dg, du = R.gated_ffn_grads(dn, xn, gn, un, g, u, act)
    tol = G.backward_tolerance(dn, xn, gn, un, dg, du, g, act, dt)
    for name, got, w, t in zip(("dx", "dw_gate", "dw_up"), grads, want, tol):
        G.check(name, got, w, t * (1 + G.half(dt)) + G.half(dt) * np.abs(w) + G.FLOOR[dt])


# K takes 15 or 29 stages forward, 2 x 5 or 2 x 10 for dx (a range of three passes from gate to up) and 10 or 19
# for dW: the ring of five goes round, and odd counts end on a stage of zeros
@pytest.mark.parametrize("dt", list(G.TYPES))
@pytest.mark.parametrize("edge", [64, 128, 256])
@pytest.mark.parametrize("whole,parts", [(0, 1), (0, 3), (2, 2), (1, 64)])
@pytest.mark.parametrize("n,d,f", [(300, 456, 152), (301, 457, 131)])
def test_products(n, d, f, whole, parts, edge, dt):
    G.say(f"schedule {dt} {n}x{d}x{f} edge {edge}, {whole} whole, {parts} parts")
    hs.set_ffn_schedule(edge, whole, parts)
    check_all(n, d, f, dt, R.ACTS[(edge // 64 + parts) % 3], (True, G.TYPES[dt])[whole % 2])


@pytest.mark.parametrize("dt", list(G.TYPES))
@pytest.mark.parametrize("edge", [64, 128, 256])
def test_one_tile_and_few_stages(edge, dt):
    """Less than one tile, and K shorter than the ring."""
    G.say(f"one tile {dt} edge {edge}")
    hs.set_ffn_schedule(edge, 0, 2)
    check_all(66, 8, 8, dt, "silu", True)
    check_all(65, 40, 1, dt, "gelu", True)


@pytest.mark.parametrize("dt,n,d,f", [("bf16", 1999, 2560, 9728), ("f16", 777, 1001, 2731), ("f32", 2000, 1280, 4000),
                                      ("bf16", 4096, 2048, 5632)])
def test_full_sizes(dt, n, d, f):
    """The estimate's own schedules at full sizes: sampled tokens of h and dx, sampled features of dW."""
    G.say(f"full size {dt} {n}x{d}x{f}")
    act = "silu"
    x, xn = G.draw(95, dt, n, d)
    wg, gn = G.draw(96, dt, f, d, scale=1.2 / d ** 0.5)
    wu, un = G.draw(97, dt, f, d, scale=1.2 / d ** 0.5)
    dh, dn = G.draw(98, dt, n, f)
    h, pre = hs.gated_ffn_forward(x, wg, wu, act=act, save=True)
    dx, dwg, dwu = hs.gated_ffn_backward(dh, x, wg, wu, pre, act=act)
    torch.cuda.synchronize()
    fp = -(-f // 8) * 8
    rng = np.random.default_rng(99)
    rows = np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, 30)]))
    cols = np.unique(np.concatenate([[0, f - 1], rng.integers(0, f, 30)]))
    want, g, u = R.gated_ffn(xn[rows], gn, un, act)
    G.check("h", h[rows], want, G.forward_tolerance(xn[rows], gn, un, g, u, act, dt)[0])
    # the backward pass at the pre-activations that it was given
    pn = pre.double().cpu().numpy()
    g, u = pn[:, :f], pn[:, fp:fp + f]
    wx, _, _, dg, du = R.gated_ffn_grads(dn[rows], xn[rows], gn, un, g[rows], u[rows], act)
    t = G.backward_tolerance(dn[rows], xn[rows], gn, un, dg, du, g[rows], act, dt)[0]
    G.check("dx", dx[rows], wx, t * (1 + G.half(dt)) + G.half(dt) * np.abs(wx) + G.FLOOR[dt])
    _, wwg, wwu, dg, du = R.gated_ffn_grads(dn[:, cols], xn, gn[cols], un[cols], g[:, cols], u[:, cols], act)
    _, tg, tu = G.backward_tolerance(dn[:, cols], xn, gn[cols], un[cols], dg, du, g[:, cols], act, dt)
    G.check("dw_gate", dwg[cols], wwg, tg * (1 + G.half(dt)) + G.half(dt) * np.abs(wwg) + G.FLOOR[dt])
    G.check("dw_up", dwu[cols], wwu, tu * (1 + G.half(dt)) + G.half(dt) * np.abs(wwu) + G.FLOOR[dt])
