"""8-bit integers as they are used: under autograd, on streams, in graphs, in odd places, and together with the
quantization pass.  Tolerances are those of test_int8_gpu.py and test_gated_ffn_gpu.py, derived there."""

import numpy as np
import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from oracle import ops_oracle as R
from tests import test_gated_ffn_gpu as G
from tests import test_int8_gpu as I

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X GPU")]

TYPES, say, draw, check, half, f64 = I.TYPES, I.say, I.draw, I.check, I.half, I.f64


@pytest.mark.parametrize("dt", list(TYPES))
def test_linear_autograd(dt):
    say(f"linear autograd {dt}")
    x, _ = draw(1, dt, 70, 136)
    w, _ = draw(2, dt, 90, 136, scale=0.1)
    dy, _ = draw(3, dt, 70, 90)
    x, dy = x.view(2, 35, 136), dy.view(2, 35, 90)
    w8, x8 = hs.quantize_int8(w), hs.quantize_int8(x)
    y = hs.int8_linear_forward(x, w8)
    dx, dw = hs.int8_linear_backward(dy, x8, w8)
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    out = hs.int8_linear(xg, wg)
    assert torch.equal(out, y) and all(t is None or t.dtype in (torch.int8, torch.float32) for t in out.grad_fn.saved_tensors)
    out.backward(dy)
    assert torch.equal(xg.grad, dx) and torch.equal(wg.grad, dw)
    # weights already quantized: a gradient for x alone, and nothing of x is kept
    xg.grad = None
    out = hs.int8_linear(xg, w8)
    assert out.grad_fn.saved_tensors[0] is None
    out.backward(dy)
    assert torch.equal(xg.grad, dx)
    # x a constant: no weights are kept
    wg.grad = None
    out = hs.int8_linear(x, wg)
    assert out.grad_fn.saved_tensors[2] is None
    out.backward(dy)
    assert torch.equal(wg.grad, dw)
    assert not hs.int8_linear(x, w).requires_grad
    with torch.no_grad():
        assert not hs.int8_linear(xg, wg).requires_grad
    xg.grad = None
    g, = torch.autograd.grad(hs.int8_linear(xg, wg).float().square().sum(), xg, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError):
            hs.int8_linear(dual, w8)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("need", ["all", "x", "w"])
def test_ffn_autograd(dt, need):
    say(f"ffn in 8 bits, autograd {dt} {need}")
    n, d, f = 66, 100, 72
    x, _ = draw(1, dt, n, d)
    wg, _ = draw(2, dt, f, d, scale=0.15)
    wu, _ = draw(3, dt, f, d, scale=0.15)
    dh, _ = draw(4, dt, n, f)
    h, pre = hs.gated_ffn_forward(x, wg, wu, act="gelu", save=torch.int8)
    want = hs.gated_ffn_backward(dh, hs.quantize_int8(x, block=32), wg, wu, pre, act="gelu")
    a, b, c = (t.clone().requires_grad_(need in ("all", k)) for t, k in ((x, "x"), (wg, "w"), (wu, "w")))
    out = hs.gated_ffn(a, b, c, act="gelu", save=torch.int8)
    assert torch.equal(out, h)
    kept = out.grad_fn.saved_tensors
    assert kept[3].dtype == torch.int8 and (kept[0] is None if need == "x" else kept[0].dtype == torch.int8)
    out.backward(dh)
    for t, g in ((a, want[0]), (b, want[1]), (c, want[2])):
        assert t.grad is None if not t.requires_grad else torch.equal(t.grad, g)


def test_gradients_against_differences():
    """Directional derivatives, in float64, of the function whose gradient each backward pass is."""
    say("differences")
    n, d, f = 67, 90, 50
    x, _ = draw(1, "f32", n, d)
    w, _ = draw(2, "f32", f, d, scale=0.1)
    wu, un = draw(3, "f32", f, d, scale=0.1)
    dy, dyn = draw(4, "f32", n, f)
    rng = np.random.default_rng(5)
    x8, w8 = hs.quantize_int8(x), hs.quantize_int8(w)
    xq, wq = (f64(q.codes) * f64(q.scale)[:, None] for q in (x8, w8))
    dx, dw = (f64(t) for t in hs.int8_linear_backward(dy, x8, w8))

    def slope(fn, v, eps=1e-4):
        return (fn(eps * v) - fn(-eps * v)) / (2 * eps)

    vx, vw = rng.standard_normal((n, d)), rng.standard_normal((f, d))
    for got, fn, v in ((dx, lambda e: np.sum(dyn * ((xq + e) @ wq.T)), vx), (dw, lambda e: np.sum(dyn * (xq @ (wq + e).T)), vw)):
        want = slope(fn, v)
        # float32 gradients (K + 12 roundings of magnitudes up to sqrt(K) times the sum's) along a random direction
        assert abs(np.sum(got * v) - want) <= 1e-4 * np.abs(got * v).sum()
    wn = f64(w)
    xb = hs.quantize_int8(x, block=32)
    xh = f64(hs.dequantize_int8(xb, dtype=torch.float32))
    for act in R.ACTS:
        _, pre = hs.gated_ffn_forward(x, w, wu, act=act, save=torch.int8)
        g, u = (t[:, :f] for t in I.pair_of(pre, f)[:2])
        dx, dwg, dwu = (f64(t) for t in hs.gated_ffn_backward(dy, xb, w, wu, pre, act=act))

        def block(gate, up):
            return np.sum(dyn * R.act_and_slope(gate, act)[0] * up)

        for got, fn, v in ((dx, lambda e: block(g + e @ wn.T, u + e @ un.T), vx), (dwg, lambda e: block(g + xh @ e.T, u), vw),
                           (dwu, lambda e: block(g, u + xh @ e.T), vw)):
            # (the differences' own error is of order eps^2)
            assert abs(np.sum(got * v) - slope(fn, v)) <= 1e-4 * np.abs(got * v).sum()


@pytest.mark.parametrize("n", [1, 20, 100])
def test_unaligned_codes(n):
    """Codes, values and outputs that start at odd places: the same bits as aligned copies."""
    say(f"odd places {n}")
    for d, f in ((64, 48), (77, 40)):
        w = hs.quantize_int8(torch.randn(f, d, device="cuda"))
        flat = torch.empty(f * d + 1, dtype=torch.int8, device="cuda")
        odd = flat[1:].view(f, d)
        odd.copy_(w.codes)
        xf = torch.randn(n * d + 1, device="cuda").bfloat16()
        x = xf[1:].view(n, d)
        want = hs.int8_linear_forward(x.clone(), w)
        w_odd = hs.Int8Rows(odd, w.scale)
        assert torch.equal(hs.int8_linear_forward(x, w_odd), want)
        x8 = hs.quantize_int8(x)
        af = torch.empty(n * d + 3, dtype=torch.int8, device="cuda")
        a = af[3:].view(n, d)
        a.copy_(x8.codes)
        assert torch.equal(hs.int8_matmul(hs.Int8Rows(a, x8.scale), w_odd), want)
        assert torch.equal(hs.dequantize_int8(hs.Int8Rows(a, x8.scale)), hs.dequantize_int8(x8))
        df = torch.randn(n * f + 1, device="cuda").bfloat16()
        dy = df[1:].view(n, f)
        one, two = hs.int8_linear_backward(dy, x8, w), hs.int8_linear_backward(dy.clone(), hs.Int8Rows(a, x8.scale), w_odd)
        assert all(torch.equal(p, q) for p, q in zip(one, two))
        # one row for all tokens, and columns as rows
        y = hs.int8_linear_forward(x[:1].expand(n, d), w)
        assert torch.equal(y, want[:1].expand(n, f))
        assert torch.equal(hs.int8_linear_forward(x.t().contiguous().t(), w), want)


def test_int8_rows_far_apart():
    """Row strides whose offsets pass 32 bits: the same bits as contiguous rows."""
    say("far rows of codes")
    n, d, f, ld = 4300, 80, 48, 1 << 20
    big = torch.empty(n * ld, dtype=torch.int8, device="cuda")
    far = big.as_strided((n, d), (ld, 1))
    x = torch.randn(n, d, device="cuda").bfloat16()
    x8, w8 = hs.quantize_int8(x), hs.quantize_int8(torch.randn(f, d, device="cuda").bfloat16())
    far.copy_(x8.codes)
    a = hs.Int8Rows(far, x8.scale)
    want = hs.int8_matmul(x8, w8)
    assert torch.equal(hs.int8_matmul(a, w8), want)
    assert torch.equal(hs.int8_matmul(hs.Int8Rows(w8.codes, w8.scale), a), hs.int8_matmul(w8, x8))  # as the right operand
    assert torch.equal(hs.dequantize_int8(a), hs.dequantize_int8(x8))
    dy = torch.randn(n, f, device="cuda").bfloat16()
    assert torch.equal(hs.int8_linear_backward(dy, a, None, need_x=False)[1], hs.int8_linear_backward(dy, x8, None, need_x=False)[1])
    out = big.view(torch.bfloat16).as_strided((n, f), (ld // 2, 1), 128)
    hs.int8_matmul(x8, w8, out=out)
    assert torch.equal(out, want)
    xs = big.view(torch.bfloat16).as_strided((n, d), (ld // 2, 1))
    xs.copy_(x)
    got = hs.quantize_int8(xs)
    assert torch.equal(got.codes, x8.codes) and torch.equal(got.scale, x8.scale)
    b, c = hs.quantize_int8(xs, block=32), hs.quantize_int8(x, block=32)
    assert torch.equal(b.codes, c.codes) and torch.equal(b.scale.float(), c.scale.float())
    assert torch.equal(hs.int8_linear_forward(xs, w8), want)


def test_empty_batches():
    say("empty")
    w = torch.randn(24, 40, device="cuda").bfloat16()
    w8 = hs.quantize_int8(w)
    x = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    y, x8 = hs.int8_linear_forward(x, w8, save=True)
    assert y.shape == (0, 24) and x8.codes.shape == (0, 40)
    dx, dw = hs.int8_linear_backward(y, x8, w8)
    assert dx.shape == (0, 40) and dw.shape == (24, 40) and not dw.any()
    assert hs.int8_matmul(x8, w8).shape == (0, 24)
    h, pre = hs.gated_ffn_forward(x, w, w, save=torch.int8)
    grads = hs.gated_ffn_backward(h, hs.quantize_int8(x, block=32), w, w, pre)
    assert grads[0].shape == (0, 40) and not grads[1].any() and not grads[2].any()


def test_refusals_on_the_gpu():
    say("refusals")
    x = torch.randn(3, 40, device="cuda").bfloat16()
    w8 = hs.quantize_int8(torch.randn(24, 40, device="cuda"))
    x8, xb = hs.quantize_int8(x), hs.quantize_int8(x, block=32)
    with pytest.raises(ValueError, match="scale a row"):
        hs.int8_matmul(xb, w8)
    with pytest.raises(ValueError, match="block"):
        hs.quantize_int8(x, block=16)
    with pytest.raises(ValueError, match="scale of"):
        hs.int8_matmul(hs.Int8Rows(x8.codes, x8.scale[:2]), w8)
    with pytest.raises(ValueError, match="scale of"):
        hs.dequantize_int8(hs.Int8Rows(xb.codes, xb.scale.float(), 32))
    with pytest.raises(TypeError, match="int8"):
        hs.int8_matmul(hs.Int8Rows(x8.codes.view(torch.uint8), x8.scale), w8)
    with pytest.raises(TypeError, match="dtype"):
        hs.quantize_int8(torch.zeros(2, 8, dtype=torch.float64, device="cuda"))
    with pytest.raises(TypeError, match="dtype"):
        hs.int8_matmul(x8, w8, dtype=torch.float64)
    with pytest.raises(ValueError, match="must hold"):
        hs.int8_matmul(x8, hs.Int8Rows(w8.codes[:, :39], w8.scale))
    with pytest.raises(ValueError, match="dx needs w"):
        hs.int8_linear_backward(x[:, :24], x8, None)
    with pytest.raises(ValueError, match="dtype"):
        hs.int8_linear(x, torch.zeros(24, 40, device="cuda"))
    with pytest.raises(ValueError, match="must hold"):
        hs.int8_linear_backward(torch.zeros(4, 24, device="cuda").bfloat16(), x8, w8)
    both = torch.randn(80, 40, device="cuda").bfloat16()
    with pytest.raises(hs.HessError, match="overlaps"):
        hs.int8_linear_forward(both, hs.quantize_int8(both[:40]), out=both)
    with pytest.raises(ValueError, match="blocks of 32"):
        hs.gated_ffn_backward(x[:, :24], x8, both[:24], both[:24], torch.empty(3, 80, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError, match="need x"):
        hs.gated_ffn_backward(x[:, :24], None, both[:24], both[:24], torch.empty(3, 80, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError, match="save"):
        hs.gated_ffn_forward(x, both[:24], both[:24], save=torch.uint8)


def work_of(n, dt=torch.bfloat16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, 200, generator=gen, device="cuda").to(dt)
    w = (torch.randn(120, 200, generator=gen, device="cuda") / 14).to(dt)
    dy = torch.randn(n, 120, generator=gen, device="cuda").to(dt)
    return x, w, dy


def all_calls(x, w, dy):
    w8 = hs.quantize_int8(w)
    y, x8 = hs.int8_linear_forward(x, w8, save=True)
    xb = hs.quantize_int8(x, block=32)
    h, pre = hs.gated_ffn_forward(x, w, w, save=torch.int8)
    return (y, hs.int8_linear_forward(x, w8), hs.int8_matmul(x8, w8, dtype=x.dtype), *hs.int8_linear_backward(dy, x8, w8), h,
            *hs.gated_ffn_backward(dy, xb, w, w, pre), hs.dequantize_int8(xb, dtype=x.dtype))


@pytest.mark.parametrize("n", [1, 24, 300])
def test_streams(n):
    """The same calls on two streams at once, and by their stream argument."""
    say(f"streams {n}")
    a, b = work_of(n, seed=1), work_of(n, seed=2)
    want_a, want_b = all_calls(*a), all_calls(*b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            got_a = all_calls(*a)
        with torch.cuda.stream(t):
            got_b = all_calls(*b)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got_a + got_b, want_a + want_b))
    x, w, dy = a
    w8 = hs.quantize_int8(w, stream=s)
    y, x8 = hs.int8_linear_forward(x, w8, save=True, stream=s)
    dx, dw = hs.int8_linear_backward(dy, x8, w8, stream=s)
    z = hs.int8_matmul(x8, w8, stream=s)
    back = hs.dequantize_int8(x8, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want_a[0]) and torch.equal(z, want_a[2]) and torch.equal(dx, want_a[3]) and torch.equal(dw, want_a[4])
    assert torch.equal(back, hs.dequantize_int8(hs.quantize_int8(x)))


@pytest.mark.parametrize("n", [1, 24, 300])
def test_graphs(n):
    """Captured, then replayed several times on changed inputs, with eager work between the replays."""
    say(f"graph {n}")
    x, w, dy = work_of(n, seed=3)
    all_calls(x, w, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_calls(x, w, dy)
    for seed in (4, 5, 6):
        for t, v in zip((x, w, dy), work_of(n, seed=seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        want = all_calls(x, w, dy)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, want))


def test_repeatable():
    say("repeatable")
    x, w, dy = work_of(700, seed=7)
    a, b = all_calls(x, w, dy), all_calls(x, w, dy)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_quantization_pass_to_8_bit_product():
    """Hessian, 4-bit codes of whole rows, the projection in 8-bit integers, and a training step of the block in
    front of it whose activations are held in 8 bits, on the distillation loss of what the projection says."""
    say("the pass together")
    n, d, f, vocab, top = 300, 96, 160, 700, 16
    gen = torch.Generator(device="cuda").manual_seed(11)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x = (normal(n, d) * torch.exp(0.5 * normal(d))).bfloat16()
    gate, up = (normal(f, d) / d ** 0.5).bfloat16(), (normal(f, d) / d ** 0.5).bfloat16()
    head = normal(vocab, f) / f ** 0.5
    h = hs.gated_ffn(x, gate, up)
    hessian = hs.Hessian(f, torch.bfloat16)
    hessian.add_batch(h)
    H, _, _ = hessian.materialize(0.01)
    hessian.close()
    Q, codes, scales, _ = hs.gptq_quantize(head, hs.chol_inverse_upper(H))
    w8 = hs.Int8Rows(codes.to(torch.int8) - 8, scales[:, 0].contiguous())
    # the codes stand for the dequantized weights
    assert (np.abs(f64(Q) - f64(w8.codes) * f64(w8.scale)[:, None]) <= np.abs(f64(Q)) * 2.0 ** -23).all()
    z = hs.int8_linear(h, w8)
    qx, sx = R.quantize_rows(f64(h))
    want = (qx @ f64(w8.codes).T) * np.outer(sx, f64(w8.scale))  # (whole sums first: they cancel exactly)
    check("logits", z, want, np.abs(want) * (half("bf16") + 5.01 * I.U) * (1 + half("bf16")) + I.FLOOR["bf16"])
    values, ids = (h.float() @ head.t()).topk(top, dim=-1)
    params = [t.float().requires_grad_() for t in (gate, up)]

    def step(save, project):
        for p in params:
            p.grad = None
        hidden = hs.gated_ffn(x, params[0].bfloat16(), params[1].bfloat16(), save=save)
        loss = hs.distill_topk(project(hidden), ids, values).sum()
        loss.backward()
        return loss.detach(), [p.grad.clone() for p in params]

    loss8, grads8 = step(torch.int8, lambda t: hs.int8_linear(t, w8))
    loss16, grads16 = step(True, lambda t: hs.int8_linear(t, w8))
    assert torch.equal(loss8, loss16) and torch.isfinite(loss8)
    # the checkpoints alone differ: each held value is at most 1 / 128 of its block's largest off, so the gradients
    # are, with errors of random sign, within a few percent as vectors
    for a, b in zip(grads8, grads16):
        assert torch.isfinite(a).all() and float((a - b).norm() / b.norm()) <= 0.05


@pytest.mark.parametrize("n", [5, 70])
def test_checkpoint_of_odd_places(n):
    """Inputs of the block that start off 16 bytes, strided checkpoints and gradients: the same bits."""
    say(f"checkpoint, odd places {n}")
    for d, f in ((64, 48), (77, 43)):
        xf, wf = torch.randn(n * d + 1, device="cuda").bfloat16(), (torch.randn(2 * f * d + 1, device="cuda") / 8).bfloat16()
        x, w = xf[1:].view(n, d), wf[1:].view(2 * f, d)
        h, pre = hs.gated_ffn_forward(x, w[:f], w[f:], save=torch.int8)
        h2, pre2 = hs.gated_ffn_forward(x.clone(), w[:f].clone(), w[f:].clone(), save=torch.int8)
        used = 2 * (-(-f // 32) * 33)
        assert torch.equal(h, h2) and torch.equal(pre[:, :used], pre2[:, :used])
        x8 = hs.quantize_int8(x, block=32)
        want = hs.gated_ffn_backward(h, x8, w[:f], w[f:], pre)
        codes = torch.zeros(n, d + 5, dtype=torch.int8, device="cuda")[:, 3:d + 3]
        codes.copy_(x8.codes)
        scale = torch.empty(n, 2 * x8.scale.shape[1], dtype=torch.uint8, device="cuda")[:, ::2]
        scale.copy_(x8.scale.view(torch.uint8))
        odd = hs.Int8Rows(codes, scale.view(torch.float8_e8m0fnu), 32)
        dh = torch.zeros(n, f + 3, dtype=torch.bfloat16, device="cuda")[:, 1:f + 1]
        dh.copy_(h)
        got = hs.gated_ffn_backward(dh, odd, w[:f].clone(), w[f:].clone(), pre2)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal(hs.dequantize_int8(odd), hs.dequantize_int8(x8))
