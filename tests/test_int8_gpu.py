"""8-bit integers: rows as codes, their product, the linear layer, and 8-bit checkpoints of the feed-forward
block, against the float64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half = half a step of the output type, eps / 2):
 * codes of given values are the exact quotient's: equal;
 * scales a / 127: one rounding to float32, u;
 * a product's sum is exact; (float)sum * b_scale * a_scale has three roundings (3.01 u), the output one more;
 * gradients of the linear layer: the operand xq or wq = code * scale, a float32 product of a scale rounded once
   (2.01 u), is rounded to the type (half, relative, at least half the smallest subnormal); sums of K terms in
   float32 add (K + 8) u of the terms' magnitudes; the output is rounded once.
 * what blocks of 32 stand for is exact (16-bit types and float32).
"""

import numpy as np
import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from oracle import ops_oracle as R
from tests import test_gated_ffn_gpu as G

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X GPU")]

U = 2.0 ** -24
TYPES = G.TYPES
say, draw, check, half, FLOOR = G.say, G.draw, G.check, G.half, G.FLOOR


def f64(t):
    return t.double().cpu().numpy()


def steps(rows):
    return rows.scale.float().double().cpu().numpy()


def values_with_ties(seed, dt, n, d):
    """Rows whose largest magnitude makes many exact ties (254 odd multiples) among ordinary ones."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((n, d)) * np.exp(rng.standard_normal((n, 1)) * 3)
    for r in range(0, n, 2):
        v[r] = rng.integers(-254, 255, d) / 2.0 * 2.0 ** rng.integers(-6, 7)
        v[r, rng.integers(d)] = (127.0 if r % 4 else 127.5) * np.abs(v[r]).max()
        v[r, 0] = np.abs(v[r]).max()
    t = torch.from_numpy(v.astype(np.float32)).to(TYPES[dt]).cuda()
    return t, f64(t)


ROWS = [(1, 1), (1, 8), (3, 7), (5, 31), (4, 32), (4, 33), (17, 100), (64, 1000), (3, 4096), (2, 4100), (2, 9001),
        (3, 16384), (2, 40000), (1, 131072)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d", ROWS)
def test_quantize_rows(n, d, dt):
    say(f"quantize rows {dt} {n}x{d}")
    x, xn = values_with_ties(1, dt, n, d)
    q = hs.quantize_int8(x)
    codes, scales = R.quantize_rows(xn)
    assert q.codes.dtype == torch.int8 and q.codes.shape == x.shape and q.scale.dtype == torch.float32
    assert np.array_equal(f64(q.codes), codes)
    # (values of some rows pass fp16's range: they stand for NaN)
    live = np.isfinite(scales)
    assert np.array_equal(np.isnan(f64(q.scale)), ~live)
    check("scale", q.scale[torch.from_numpy(live).cuda()], scales[live], scales[live] * U)
    back = hs.dequantize_int8(q, dtype=x.dtype)
    assert torch.isnan(back[torch.from_numpy(~live).cuda()]).all()
    back, want = back[torch.from_numpy(live).cuda()], (codes * scales[:, None])[live]
    check("restored", back, want, np.abs(want) * (half(dt) + 2.01 * U) * (1 + half(dt)) + FLOOR[dt])


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d", ROWS)
def test_quantize_blocks(n, d, dt):
    say(f"quantize blocks {dt} {n}x{d}")
    x, xn = values_with_ties(2, dt, n, d)
    q = hs.quantize_int8(x, block=32)
    codes, st = R.quantize_blocks(xn)
    assert q.block == 32 and np.array_equal(f64(q.codes), codes) \
        and np.array_equal(steps(q), st, equal_nan=True)
    want = R.stand_for(codes, st)
    for out in (torch.float32, torch.bfloat16):
        assert np.array_equal(f64(hs.dequantize_int8(q, dtype=out)), want, equal_nan=True)
    if dt == "f16":
        assert np.array_equal(f64(hs.dequantize_int8(q, dtype=torch.float16)), want, equal_nan=True)


@pytest.mark.parametrize("block", [0, 32])
@pytest.mark.parametrize("dt", list(TYPES))
def test_quantize_strides_and_shapes(dt, block):
    say(f"quantize strides {dt} {block}")
    x, xn = draw(3, dt, 11, 77, cols=91)
    a, b = hs.quantize_int8(x, block=block), hs.quantize_int8(x.contiguous(), block=block)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scale.float(), b.scale.float())
    t = hs.quantize_int8(x.t(), block=block)  # columns as rows: copied first
    assert np.array_equal(f64(t.codes), (R.quantize_rows if block == 0 else R.quantize_blocks)(xn.T)[0])
    y = x.contiguous()[:10].reshape(2, 5, 77)
    c = hs.quantize_int8(y, block=block)
    assert c.codes.shape == y.shape and torch.equal(c.codes.reshape(10, 77), b.codes[:10])
    wide = torch.full((11, 80), 7.0, dtype=x.dtype, device="cuda")
    hs.dequantize_int8(b, dtype=x.dtype, out=wide[:, 1:78])
    assert (wide[:, 0] == 7).all() and (wide[:, 78:] == 7).all()
    assert torch.equal(wide[:, 1:78], hs.dequantize_int8(b, dtype=x.dtype))
    e = hs.quantize_int8(x[:0], block=block)
    assert e.codes.shape == (0, 77) and hs.dequantize_int8(e).shape == (0, 77)


@pytest.mark.parametrize("dt", list(TYPES))
def test_quantize_extremes(dt):
    """Rows of zeros, the smallest and largest numbers, and rows with an infinity or NaN."""
    say(f"quantize extremes {dt}")
    info = torch.finfo(TYPES[dt])
    sub = info.smallest_normal * info.eps
    x = torch.zeros((9, 64), dtype=TYPES[dt])
    x[1, 5] = sub
    x[2, ::2], x[2, 1] = sub, -3 * sub
    x[3, :40], x[3, 40:] = info.max, info.min
    x[4, 33], x[4, 3] = float("inf"), 1.0
    x[5, 2] = float("nan")
    x[6, 63] = -float("inf")
    x[7] = torch.linspace(-1, 1, 64) * info.smallest_normal
    x[8] = torch.linspace(-1, 1, 64)
    xd, xn = x.cuda(), x.double().numpy()
    q, (codes, scales) = hs.quantize_int8(xd), R.quantize_rows(xn)
    # a float32 scale of tiny rows is subnormal: half its unit
    got = f64(q.scale)
    assert np.array_equal(f64(q.codes), codes)
    assert np.array_equal(np.isnan(got), np.isnan(scales))
    assert (np.abs(got - scales)[~np.isnan(scales)] <= (scales * U + 2.0 ** -150)[~np.isnan(scales)]).all()
    b, (codes, st) = hs.quantize_int8(xd, block=32), R.quantize_blocks(xn)
    assert np.array_equal(f64(b.codes), codes) and np.array_equal(steps(b), st, equal_nan=True)
    back = hs.dequantize_int8(b, dtype=torch.float32)
    assert np.array_equal(f64(back), R.stand_for(codes, st), equal_nan=True)


PRODUCTS = [(1, 1, 1), (1, 16, 16), (2, 63, 5), (3, 64, 17), (5, 65, 33), (16, 128, 48), (17, 200, 100), (33, 1000, 77),
            (64, 512, 256), (65, 513, 129), (128, 1024, 300), (130, 100, 520), (300, 704, 1000), (513, 333, 260)]


def random_codes(seed, n, d, ld=None):
    gen = torch.Generator().manual_seed(seed)
    c = torch.randint(-128, 128, (n, ld or d), generator=gen, dtype=torch.int8).cuda()[:, :d]
    s = torch.rand(n, generator=gen) * 0.1 + 0.001
    return hs.Int8Rows(c, s.cuda())


def product(a, b):
    return (f64(a.codes) @ f64(b.codes).T) * np.outer(f64(a.scale), f64(b.scale))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d,f", PRODUCTS)
def test_matmul(n, d, f, dt):
    say(f"matmul {dt} {n}x{d}x{f}")
    a, b = random_codes(4, n, d), random_codes(5, f, d)
    y = hs.int8_matmul(a, b, dtype=TYPES[dt])
    want = product(a, b)
    check("y", y, want, np.abs(want) * (half(dt) + 3.01 * U) * (1 + half(dt)) + FLOOR[dt])
    far = random_codes(4, n, d, d + 5), random_codes(5, f, d, d + 16 - d % 16)
    wide = torch.full((n, f + 3), 7.0, dtype=TYPES[dt], device="cuda")
    hs.int8_matmul(*far, dtype=TYPES[dt], out=wide[:, 1:f + 1])
    want = product(*far)
    check("y", wide[:, 1:f + 1], want, np.abs(want) * (half(dt) + 3.01 * U) * (1 + half(dt)) + FLOOR[dt])
    assert (wide[:, 0] == 7).all() and (wide[:, f + 1:] == 7).all()


@pytest.mark.parametrize("n", [2, 70, 300])
def test_matmul_largest_sums(n):
    """All codes -128 over the longest row: sums of 2^31 - 2^14."""
    say(f"largest sums {n}")
    d, f = (1 << 17) - 1, 40
    a = hs.Int8Rows(torch.full((n, d), -128, dtype=torch.int8, device="cuda"), torch.ones(n, device="cuda"))
    b = hs.Int8Rows(torch.full((f, d), -128, dtype=torch.int8, device="cuda"), torch.ones(f, device="cuda"))
    b.codes[f // 2:] = 127
    y = f64(hs.int8_matmul(a, b, dtype=torch.float32))
    want = np.full((n, f), float(d << 14))
    want[:, f // 2:] = -128.0 * 127.0 * d
    assert (np.abs(y - want) <= np.abs(want) * U).all()
    a.scale[0] = float("nan")
    y = hs.int8_matmul(a, b, dtype=torch.bfloat16)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1:]).all()


LAYERS = [(1, 1, 1), (1, 64, 64), (2, 130, 37), (4, 100, 33), (5, 65, 40), (16, 256, 100), (24, 513, 250), (33, 96, 257),
          (70, 200, 130), (257, 136, 129), (300, 1000, 250), (129, 2600, 700)]


def layer_case(seed, n, d, f, dt):
    x, xn = draw(seed, dt, n, d)
    w, wn = draw(seed + 1, dt, f, d, scale=1.0 / d ** 0.5)
    qx, sx = R.quantize_rows(xn)
    qw, sw = R.quantize_rows(wn)
    return x, w, qx, sx, qw, sw


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d,f", LAYERS)
def test_linear_forward(n, d, f, dt):
    say(f"linear {dt} {n}x{d}x{f}")
    x, w, qx, sx, qw, sw = layer_case(6, n, d, f, dt)
    w8 = hs.quantize_int8(w)
    y, x8 = hs.int8_linear_forward(x, w8, save=True)
    want = (qx @ qw.T) * np.outer(sx, sw)
    # both scales are a / 127 rounded: two more roundings than the product alone
    check("y", y, want, np.abs(want) * (half(dt) + 5.01 * U) * (1 + half(dt)) + FLOOR[dt])
    assert np.array_equal(f64(x8.codes), qx)
    direct = hs.quantize_int8(x)
    assert torch.equal(x8.codes, direct.codes) and torch.equal(x8.scale, direct.scale)
    assert torch.equal(y, hs.int8_linear_forward(x, w8)), "saving changes y"
    assert torch.equal(y, hs.int8_matmul(direct, w8, dtype=x.dtype)), "the parts give another y"
    # weights whose rows lie one behind the other
    packed = hs.Int8Rows(w8.codes.contiguous(), w8.scale)
    assert torch.equal(y, hs.int8_linear_forward(x, packed))


def gradient_tolerance(dyn, xq, wq, dt):
    """(dx, dw): what the roundings of the operands and the float32 sums may leave, before the last rounding."""
    f, n = wq.shape[0], xq.shape[0]
    op = (0.0 if dt == "f32" else half(dt)) * (1 + 3 * U) + 2.01 * U
    floor = 0.0 if dt == "f32" else FLOOR[dt]
    aw, ax = np.abs(wq), np.abs(xq)
    ew, ex = aw * op + floor, ax * op + floor
    a = np.abs(dyn)
    return (a @ ew + (f + 8) * U * (a @ (aw + ew)), a.T @ ex + (n + 8) * U * (a.T @ (ax + ex)))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d,f", LAYERS)
def test_linear_backward(n, d, f, dt):
    say(f"linear backward {dt} {n}x{d}x{f}")
    x, w, qx, sx, qw, sw = layer_case(8, n, d, f, dt)
    dy, dyn = draw(10, dt, n, f)
    w8 = hs.quantize_int8(w)
    x8 = hs.quantize_int8(x)
    dx, dw = hs.int8_linear_backward(dy, x8, w8)
    xq, wq = qx * sx[:, None], qw * sw[:, None]
    tx, tw = gradient_tolerance(dyn, xq, wq, dt)
    wx, ww = dyn @ wq, dyn.T @ xq
    check("dx", dx, wx, tx * (1 + half(dt)) + half(dt) * np.abs(wx) + FLOOR[dt])
    check("dw", dw, ww, tw * (1 + half(dt)) + half(dt) * np.abs(ww) + FLOOR[dt])
    only = hs.int8_linear_backward(dy, None, w8, need_w=False)
    assert only[1] is None and torch.equal(only[0], dx)
    only = hs.int8_linear_backward(dy, x8, None, need_x=False)
    assert only[0] is None and torch.equal(only[1], dw)
    strided, _ = draw(10, dt, n, f, cols=f + 8)
    strided.copy_(dy)
    again = hs.int8_linear_backward(strided, x8, w8)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


# -- the feed-forward block's 8-bit checkpoint ----------------------------------------------------

def pair_of(pre, f):
    """What the pair's codes stand for: (g, u), float64, and its parts."""
    fq = -(-f // 32) * 32
    p = pre.cpu()
    assert pre.shape[1] == -(-(2 * fq + fq // 16) // 16) * 16
    exps = p[:, 2 * fq:2 * fq + fq // 16].contiguous().view(torch.float8_e8m0fnu).float().double().numpy()
    g, u = p[:, :fq].double().numpy(), p[:, fq:2 * fq].double().numpy()
    return (R.stand_for(g, exps[:, :fq // 32]), R.stand_for(u, exps[:, fq // 32:]), g, u, exps[:, :fq // 32],
            exps[:, fq // 32:])


FFN = [(1, 8, 16), (3, 40, 72), (17, 129, 65), (65, 96, 257), (70, 48, 32), (130, 520, 136), (257, 72, 129),
       (300, 1000, 250), (300, 704, 1000)]


def check_pair(pre, f, g, u, tg, tu):
    gh, uh, gc, uc, gs, us = pair_of(pre, f)
    assert not gc[:, f:].any() and not uc[:, f:].any()
    for v, t, vh, c, s in ((g, tg, gh, gc, gs), (u, tu, uh, uc, us)):
        wide = np.repeat(s, 32, axis=1)[:, :f]
        # the nearest code to a value t away from the exact one, none past 127
        assert (np.abs(vh[:, :f] - v) <= np.maximum(wide / 2, np.abs(v) - 127 * wide) + t).all() and (np.abs(c) <= 127).all()
        # the block's largest value is 64 to 128 steps
        for b in range(s.shape[1]):
            top = (np.abs(v[:, 32 * b:32 * b + 32]) + t[:, 32 * b:32 * b + 32]).max(1)
            low = (np.abs(v[:, 32 * b:32 * b + 32]) - t[:, 32 * b:32 * b + 32]).max(1)
            assert (low < 128 * s[:, b]).all() and (top >= 64 * s[:, b]).all()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d,f", FFN)
def test_ffn_checkpoint(n, d, f, dt):
    act = R.ACTS[(n + d + f) % 3]
    say(f"ffn in 8 bits {dt} {n}x{d}x{f} {act}")
    x, xn = draw(1, dt, n, d)
    wg, gn = draw(2, dt, f, d, scale=1.5 / d ** 0.5)
    wu, un = draw(3, dt, f, d, scale=1.5 / d ** 0.5)
    dh, dn = draw(4, dt, n, f)
    h, pre = hs.gated_ffn_forward(x, wg, wu, act=act, save=torch.int8)
    want, g, u = R.gated_ffn(xn, gn, un, act)
    th = G.forward_tolerance(xn, gn, un, g, u, act, dt)
    check("h", h, want, th[0])
    if n > 64:
        assert torch.equal(h, hs.gated_ffn_forward(x, wg, wu, act=act)), "saving changes h"
    k = (d + 8) * U
    check_pair(pre, f, g, u, k * (np.abs(xn) @ np.abs(gn).T), k * (np.abs(xn) @ np.abs(un).T))
    # the backward pass, at what the codes stand for
    x8 = hs.quantize_int8(x, block=32)
    gh, uh = (v[:, :f] for v in pair_of(pre, f)[:2])
    xh = f64(hs.dequantize_int8(x8, dtype=torch.float32))
    dx, dwg, dwu = hs.gated_ffn_backward(dh, x8, wg, wu, pre, act=act)
    wx, wwg, wwu, dg, du = R.gated_ffn_grads(dn, xh, gn, un, gh, uh, act)
    tol = G.backward_tolerance(dn, xh, gn, un, dg, du, gh, act, dt)
    for name, got, w_, t in (("dx", dx, wx, tol[0]), ("dw_gate", dwg, wwg, tol[1]), ("dw_up", dwu, wwu, tol[2])):
        check(name, got, w_, t * (1 + half(dt)) + half(dt) * np.abs(w_) + FLOOR[dt])
    only = hs.gated_ffn_backward(dh, None, wg, wu, pre, act=act, need_w=False)
    assert only[1] is None and torch.equal(only[0], dx)
    only = hs.gated_ffn_backward(dh, x8, wg, wu, pre, act=act, need_x=False)
    assert only[0] is None and torch.equal(only[1], dwg) and torch.equal(only[2], dwu)
    if dt != "f32":  # a pair in another type beside x in 8 bits
        mixed = hs.gated_ffn_forward(x, wg, wu, act=act, save=x.dtype)[1]
        one = hs.gated_ffn_backward(dh, x8, wg, wu, mixed, act=act)
        two = hs.gated_ffn_backward(dh, hs.dequantize_int8(x8, dtype=x.dtype), wg, wu, mixed, act=act)
        assert all(torch.equal(p, q) for p, q in zip(one, two))
    same = hs.gated_ffn_backward(dh, hs.dequantize_int8(x8, dtype=x.dtype), wg, wu, pre, act=act)
    assert all(torch.equal(p, q) for p, q in zip(same, (dx, dwg, dwu)))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("edge,whole,parts", [(64, 1 << 30, 1), (64, 0, 2), (64, 3, 3), (128, 1 << 30, 1), (128, 0, 3),
                                              (128, 2, 2), (256, 1 << 30, 1), (256, 0, 2), (256, 1, 3)])
def test_ffn_checkpoint_schedules(edge, whole, parts, dt):
    """Each tile, done whole, split, and both at once: the pair of one schedule is the pair of another up to sums."""
    n, d, f = 300, 520, 330
    say(f"ffn in 8 bits {dt} edge {edge} whole {whole} parts {parts}")
    x, xn = draw(1, dt, n, d)
    wg, gn = draw(2, dt, f, d, scale=1.5 / d ** 0.5)
    wu, un = draw(3, dt, f, d, scale=1.5 / d ** 0.5)
    _, g, u = R.gated_ffn(xn, gn, un, "silu")
    try:
        hs.set_ffn_schedule(edge, whole, parts)
        h, pre = hs.gated_ffn_forward(x, wg, wu, save=torch.int8)
        plain = hs.gated_ffn_forward(x, wg, wu)
    finally:
        hs.set_ffn_schedule()
    assert torch.equal(h, plain)
    k = (d + 8) * U
    check_pair(pre, f, g, u, k * (np.abs(xn) @ np.abs(gn).T), k * (np.abs(xn) @ np.abs(un).T))


def test_ffn_checkpoint_not_finite():
    """An infinity in one token's gate: its block stands for NaN, no other token or block is touched."""
    say("ffn in 8 bits, not finite")
    n, d, f = 70, 64, 96
    x, _ = draw(1, "bf16", n, d)
    wg, _ = draw(2, "bf16", f, d, scale=0.2)
    wu, _ = draw(3, "bf16", f, d, scale=0.2)
    clean = pair_of(hs.gated_ffn_forward(x, wg, wu, save=torch.int8)[1], f)
    x[5, 7] = float("inf")
    got = pair_of(hs.gated_ffn_forward(x, wg, wu, save=torch.int8)[1], f)
    for a, b in zip(got[:2], clean[:2]):
        assert np.isnan(a[5]).all() and np.array_equal(np.delete(a, 5, 0), np.delete(b, 5, 0))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("edge,whole,parts", [(64, 1 << 30, 1), (64, 0, 2), (64, 5, 3), (128, 1 << 30, 1), (128, 0, 3),
                                              (128, 2, 2), (256, 1 << 30, 1), (256, 0, 2), (256, 1, 3)])
@pytest.mark.parametrize("n,d,f", [(300, 1040, 330), (300, 1001, 513)])
def test_matmul_schedules(n, d, f, edge, whole, parts, dt):
    """Each tile, done whole, split, and both at once: the same bits, since the sums are exact."""
    say(f"matmul {dt} {n}x{d}x{f} edge {edge} whole {whole} parts {parts}")
    a, b = random_codes(11, n, d), random_codes(12, f, d)
    want = hs.int8_matmul(a, b, dtype=TYPES[dt])
    exact = product(a, b)
    check("y", want, exact, np.abs(exact) * (half(dt) + 3.01 * U) * (1 + half(dt)) + FLOOR[dt])
    try:
        hs.set_ffn_schedule(edge, whole, parts)
        got = hs.int8_matmul(a, b, dtype=TYPES[dt])
    finally:
        hs.set_ffn_schedule()
    assert torch.equal(got, want)


# one row has kernels of its own, by width and length; up to 64 rows others, by both
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d,f", [(1, 40, 70), (1, 1001, 2731), (1, 2048, 100), (1, 2049, 4096), (1, 2500, 4113),
                                   (1, 4096, 4113), (1, 5000, 4200), (1, 8192, 48), (1, 8192, 4100), (1, 8193, 33),
                                   (16, 260, 4100), (17, 260, 4096), (32, 333, 4097), (33, 64, 100), (20, 200, 8193),
                                   (64, 200, 8200), (33, 1030, 8210), (64, 130, 8192),
                                   (17, 70, 12288), (20, 64, 12300), (40, 72, 12289), (40, 130, 6144), (50, 130, 6145),
                                   (64, 130, 2048), (64, 65, 2049), (33, 70, 4097), (33, 8191, 50), (33, 8192, 50),
                                   (40, 8200, 70), (64, 8205, 33), (32, 8205, 33)])
def test_few_rows(n, d, f, dt):
    say(f"few rows {dt} {n}x{d}x{f}")
    x, w, qx, sx, qw, sw = layer_case(13, n, d, f, dt)
    w8 = hs.quantize_int8(w)
    want = (qx @ qw.T) * np.outer(sx, sw)
    y = hs.int8_linear_forward(x, w8)
    check("y", y, want, np.abs(want) * (half(dt) + 5.01 * U) * (1 + half(dt)) + FLOOR[dt])
    y2, x8 = hs.int8_linear_forward(x, w8, save=True)
    assert torch.equal(y, y2) and torch.equal(y, hs.int8_matmul(x8, w8, dtype=x.dtype))
    packed = hs.Int8Rows(w8.codes.contiguous(), w8.scale)
    assert torch.equal(y, hs.int8_linear_forward(x, packed))


def test_one_row_not_finite():
    say("one row, not finite")
    w8 = hs.quantize_int8(torch.randn(50, 300, device="cuda"))
    x = torch.randn(1, 300, device="cuda")
    assert (hs.int8_linear_forward(torch.zeros_like(x), w8) == 0).all()
    for bad in (float("inf"), float("nan")):
        x[0, 299] = bad
        assert torch.isnan(hs.int8_linear_forward(x, w8)).all()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("edge", [64, 128, 256])
@pytest.mark.parametrize("act", R.ACTS)
def test_ffn_checkpoint_activations(act, edge, dt):
    """Every activation in every tile, inside the matrix and at its end: the pair does not depend on either."""
    n, d, f = 300, 72, 300
    say(f"ffn in 8 bits {dt} {act} edge {edge}")
    x, xn = draw(1, dt, n, d)
    wg, gn = draw(2, dt, f, d, scale=1.5 / d ** 0.5)
    wu, un = draw(3, dt, f, d, scale=1.5 / d ** 0.5)
    want, g, u = R.gated_ffn(xn, gn, un, act)
    try:
        hs.set_ffn_schedule(edge, 1 << 30, 1)
        h, pre = hs.gated_ffn_forward(x, wg, wu, act=act, save=torch.int8)
    finally:
        hs.set_ffn_schedule()
    check("h", h, want, G.forward_tolerance(xn, gn, un, g, u, act, dt)[0])
    k = (d + 8) * U
    check_pair(pre, f, g, u, k * (np.abs(xn) @ np.abs(gn).T), k * (np.abs(xn) @ np.abs(un).T))
