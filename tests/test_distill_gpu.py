"""The top-logit distillation loss against the float64 oracle.

Tolerances, from the arithmetic (u = 2^-24): 1 / T is rounded once and scales both softmaxes, an
exponent's argument and the hardware exponential are off by at most 4 u (|argument| + 2), a float32 sum
of up to S values by S u; so the sum of exponentials and each probability carry, relative,
    E = 8 u (max|z| / T + max|v| / T + 2) + (vocab / 256 + 64) u,
the loss at most 4 E w (as a difference of two logarithms) plus its float32 rounding, a gradient
c (q + p) E plus half a step of its type (fp16: no less than half its smallest subnormal).
"""

import sys

import numpy as np
import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from oracle import ops_oracle as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X GPU")]

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FLOOR = {"bf16": 2.0 ** -126, "f16": 2.0 ** -25, "f32": 2.0 ** -126}


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def make(seed, dt, n, vocab, k, absent=0.0, distinct=True, ids=torch.int64, vdt="f32", pad=0):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy((2 * rng.standard_normal((n, vocab + pad))).astype(np.float32)).to(TYPES[dt]).cuda()
    z = z[:, pad // 2:pad // 2 + vocab]
    if distinct:
        i = np.stack([rng.permutation(vocab)[:k] for _ in range(n)])
    else:
        i = rng.integers(0, max(1, min(vocab, k // 2)), (n, k))
    i = np.where(rng.random((n, k)) < absent, -1 - rng.integers(0, 5, (n, k)), i)
    v = torch.from_numpy((3 * rng.standard_normal((n, k))).astype(np.float32)).to(TYPES[vdt]).cuda()
    w = torch.from_numpy((0.5 + rng.random(n)).astype(np.float32)).cuda()
    return z, torch.from_numpy(i).to(ids).cuda(), v, w


def f64(t):
    return t.double().cpu().numpy()


def tolerances(z, i, v, w, t, vocab, loss, grad, dt, dl=None):
    zf = np.abs(np.where(np.isfinite(z), z, 0)).max(1)
    here = (i >= 0) & np.isfinite(v)
    vf = np.where(here, np.abs(np.where(here, v, 0)), 0).max(1)
    e = 8 * U * (zf / t + vf / t + 2) + (vocab / 256 + 64) * U
    c = w / t * (1.0 if dl is None else np.abs(dl))
    # c (q + p) <= |grad| + 2 c p: p from the definition
    p = np.zeros_like(grad)
    for r in range(i.shape[0]):
        if here[r].any():
            s = v[r][here[r]] / t
            pr = np.exp(s - s.max())
            np.add.at(p[r], np.where(i[r][here[r]] < vocab, i[r][here[r]], 0), pr / pr.sum())
    hh = torch.finfo(TYPES[dt]).eps / 2
    tg = (np.abs(grad) + 2 * c[:, None] * p) * e[:, None]
    return 4 * e * w + U * np.abs(loss), tg * (1 + hh) + hh * np.abs(grad) + FLOOR[dt]


def compare(got, want, tol, what):
    got = f64(got)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= tol))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[tuple(np.argwhere(bad)[0])]} for {want[tuple(np.argwhere(bad)[0])]}")


def run_all(z, i, v, w, t, dt, dl=None):
    """loss, step's gradient, backward's gradient, each against the oracle."""
    n, vocab = z.shape
    zn, inn, vn = f64(z), i.cpu().numpy(), f64(v)
    wn = np.ones(n) if w is None else f64(w)
    loss, stats, grad = R.distill_topk(zn, inn, vn, wn, t)
    tl, tg = tolerances(zn, inn, vn, wn, t, vocab, loss, grad, dt)
    got_loss, got_stats = hs.distill_topk_forward(z, i, v, weight=w, temperature=t)
    compare(got_loss, loss, tl, "loss")
    step_loss, step_grad = hs.distill_topk_step(z, i, v, weight=w, temperature=t)
    torch.cuda.synchronize()
    compare(step_loss, loss, tl, "step's loss")
    compare(step_grad, grad, tg, "step's gradient")
    rng = np.random.default_rng(99)
    dl = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    back = hs.distill_topk_backward(dl, z, i, v, got_stats, weight=w, temperature=t)
    torch.cuda.synchronize()
    dn = f64(dl)
    tg = tolerances(zn, inn, vn, wn, t, vocab, loss, dn[:, None] * grad, dt, dl=dn)[1]
    compare(back, dn[:, None] * grad, tg, "backward's gradient")
    return got_loss, got_stats, step_grad


CASES = [(1, 1, 1), (1, 2, 2), (3, 7, 4), (2, 64, 64), (5, 100, 9), (4, 1000, 32), (300, 513, 20), (2, 4099, 1000),
         (3, 8192, 65), (7, 30001, 100), (2, 70000, 1024), (1, 150001, 50), (2, 300007, 7)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,vocab,k", CASES)
def test_loss_and_gradients(n, vocab, k, dt):
    say(f"{dt} {n}x{vocab} top {k}")
    t = (1.0, 2.0, 0.7)[(n + k) % 3]
    z, i, v, w = make(n * 7 + k, dt, n, vocab, k, ids=(torch.int64, torch.int32)[k % 2])
    run_all(z, i, v, w if n % 2 else None, t, dt)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("pad", [1, 2, 6, 16])
@pytest.mark.parametrize("vocab", [50, 4001])
def test_row_strides_and_alignments(vocab, pad, dt):
    say(f"{dt} rows of {vocab + pad}")
    z, i, v, w = make(5, dt, 6, vocab, 12, pad=pad)
    grad = run_all(z, i, v, w, 1.3, dt)[2]
    # into a strided view: the same bits, nothing outside touched
    wide = torch.full((6, vocab + 3), 5.0, dtype=z.dtype, device="cuda")
    hs.distill_topk_step(z, i, v, weight=w, temperature=1.3, out=wide[:, 1:vocab + 1])
    assert torch.equal(wide[:, 1:vocab + 1], grad)
    assert (wide[:, 0] == 5).all() and (wide[:, vocab + 1:] == 5).all()


@pytest.mark.parametrize("vocab", [40, 9001, 140000])
@pytest.mark.parametrize("dt", list(TYPES))
def test_masked_absent_repeated(dt, vocab):
    say(f"masked {dt} {vocab}")
    z, i, v, w = make(6, dt, 9, vocab, 24, absent=0.4, distinct=False, vdt="bf16")
    w[2] = 0.0
    z[2] = float("nan")          # a row left out is not read
    i[3] = -1                    # nothing present
    z[3] = float("inf")
    v[4] = -float("inf")         # nothing present
    v[5, :10] = -float("inf")
    v[6] = torch.finfo(torch.bfloat16).min   # the type's lowest value in every entry: equal teachers
    i[7, 3] = vocab              # an id past the vocabulary
    v[7, 3] = 1.0
    loss, _, grad = run_all(z, i, v, w, 1.0, dt)
    for r in (2, 3, 4):
        assert loss[r] == 0 and not grad[r].any()
    assert torch.isnan(loss[7]) and torch.isnan(grad[7]).all()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("vocab", [33, 20000])
def test_infinities_and_nan(dt, vocab):
    say(f"infinities {dt} {vocab}")
    z, i, v, w = make(8, dt, 7, vocab, 8)
    z[0] = -float("inf")
    z[0, 5] = 1.0                               # one candidate left
    i[0] = torch.arange(5, 13, device="cuda")
    v[0, 1:] = -float("inf")                    # ... and it is the teacher's
    z[1, :20] = -float("inf")                   # words struck out
    i[1] = torch.arange(20, 28, device="cuda")
    z[2] = -float("inf")                        # nothing left: NaN
    z[3, 2] = float("nan")
    z[4, 2] = float("inf")
    z[5, 3] = -float("inf")                     # the teacher's mass where the student has none
    i[5, 0] = 3
    i[5, 1:] = torch.arange(10, 17, device="cuda")
    z[6] = torch.finfo(TYPES[dt]).min           # every logit the type's lowest value
    zn, inn, vn, wn = f64(z), i.cpu().numpy(), f64(v), f64(w)
    loss, _, grad = R.distill_topk(zn, inn, vn, wn, 1.0)
    got, g = hs.distill_topk_step(z, i, v, weight=w)
    torch.cuda.synchronize()
    got, g = f64(got), f64(g)
    # p = q = 1 exactly, up to the last bits of the exponential and the logarithm
    assert abs(got[0] - loss[0]) <= 8 * U * wn[0] and np.abs(g[0]).max() <= 8 * U * wn[0]
    e = 8 * U * (np.abs(zn[1, 20:]).max() + np.abs(vn[1]).max() + 2) + (vocab / 256 + 64) * U
    assert abs(got[1] - loss[1]) <= 4 * e * wn[1] + U * abs(loss[1]) and not g[1, :20].any()
    assert np.isnan(got[2]) and np.isnan(got[3]) and np.isnan(got[4])
    assert np.isnan(g[2]).any() and np.isnan(g[3]).all()
    assert got[5] == np.inf and np.isfinite(g[5]).all()
    # equal logits: z - max is exactly 0, so the scale of the logits does not enter the tolerance
    e = 8 * U * (np.abs(vn[6]).max() + 2) + (vocab / 256 + 64) * U
    assert abs(got[6] - loss[6]) <= 4 * e * wn[6] + U * abs(loss[6])


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("vocab", [777, 33000, 200000])
def test_gradient_in_place_and_repeatable(dt, vocab):
    say(f"in place {dt} {vocab}")
    z, i, v, w = make(12, dt, 5, vocab, 30, distinct=False)
    loss, grad = hs.distill_topk_step(z, i, v, weight=w)
    again = hs.distill_topk_step(z, i, v, weight=w)
    assert torch.equal(loss, again[0]) and torch.equal(grad, again[1])
    _, stats = hs.distill_topk_forward(z, i, v, weight=w)
    dl = torch.ones(5, device="cuda")
    back = hs.distill_topk_backward(dl, z, i, v, stats, weight=w)
    copy = z.clone()
    assert hs.distill_topk_backward(dl, copy, i, v, stats, weight=w, out=copy) is copy
    assert torch.equal(copy, back)
    copy = z.clone()
    loss2, _ = hs.distill_topk_step(copy, i, v, weight=w, out=copy)
    assert torch.equal(copy, grad) and torch.equal(loss2, loss)


def test_gradient_against_differences():
    say("differences")
    n, vocab, t = 4, 5000, 1.5
    z, i, v, w = make(13, "f32", n, vocab, 16)
    d = torch.from_numpy(np.random.default_rng(14).standard_normal((n, vocab)).astype(np.float32)).cuda()
    loss, grad = hs.distill_topk_step(z, i, v, weight=w, temperature=t)
    step, quot, exact, tol = 2.0 ** -5, np.zeros(n), np.zeros(n), np.zeros(n)
    inn, vn, wn = i.cpu().numpy(), f64(v), f64(w)
    for s in (step, -step):
        zs = z + s * d
        l, _, g = R.distill_topk(f64(zs), inn, vn, wn, t)
        quot += f64(hs.distill_topk_forward(zs, i, v, weight=w, temperature=t)[0]) / (2 * s)
        exact += l / (2 * s)
        tol += tolerances(f64(zs), inn, vn, wn, t, vocab, l, g, "f32")[0] / (2 * step)
    l, _, g = R.distill_topk(f64(z), inn, vn, wn, t)
    tg = tolerances(f64(z), inn, vn, wn, t, vocab, l, g, "f32")[1]
    dn = f64(d)
    bound = np.abs(exact - (g * dn).sum(1)) + tol + (tg * np.abs(dn)).sum(1)
    assert (np.abs(quot - (f64(grad) * dn).sum(1)) <= bound).all()


def test_autograd_leading_dimensions_and_broadcast_gradient():
    say("autograd")
    z, i, v, w = make(15, "bf16", 6, 900, 10)
    z3 = z.reshape(2, 3, 900).clone().requires_grad_()
    loss = hs.distill_topk(z3, i.reshape(2, 3, 10), v.reshape(2, 3, 10), weight=w.reshape(2, 3), temperature=2.0)
    assert loss.shape == (2, 3)
    loss.sum().backward()
    l, stats = hs.distill_topk_forward(z, i, v, weight=w, temperature=2.0)
    g = hs.distill_topk_backward(torch.ones(6, device="cuda"), z, i, v, stats, weight=w, temperature=2.0)
    assert torch.equal(loss.reshape(-1), l) and torch.equal(z3.grad.reshape(6, 900), g)
    # a weight and a gradient that are one broadcast value
    one = torch.full((1,), 0.5, device="cuda").expand(6)
    a = hs.distill_topk_step(z, i, v, weight=one)
    b = hs.distill_topk_step(z, i, v, weight=torch.full((6,), 0.5, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_rows_other_stream_and_graph_replays():
    say("stream and graph")
    e = hs.distill_topk_step(torch.empty((0, 9), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                             torch.empty((0, 2), device="cuda"))
    assert e[0].shape == (0,) and e[1].shape == (0, 9)
    z, i, v, w = make(16, "f16", 5, 40000, 33)
    ref = hs.distill_topk_step(z, i, v, weight=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hs.distill_topk_step(z, i, v, weight=w, stream=side)
    side.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])

    dl = torch.linspace(-1, 1, 5, device="cuda")

    def both():
        loss, stats = hs.distill_topk_forward(z, i, v, weight=w)
        return (loss, hs.distill_topk_backward(dl, z, i, v, stats, weight=w),
                *hs.distill_topk_step(z, i, v, weight=w))

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for k in range(4):
        z.copy_(make(20 + k, "f16", 5, 40000, 33)[0])
        eager = both()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b), f"replay {k}"


def test_shape_refusals():
    z, i, v, w = make(17, "f32", 4, 30, 5)
    for bad in (lambda: hs.distill_topk_forward(z, i[:3], v), lambda: hs.distill_topk_forward(z, i, v[:, :4]),
                lambda: hs.distill_topk_forward(z, i, v, weight=w[:3]),
                lambda: hs.distill_topk_forward(z, i, v, weight=w.double()),
                lambda: hs.distill_topk_step(z, i, v, out=torch.empty((4, 31), device="cuda")),
                lambda: hs.distill_topk_backward(w, z, i, v, w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        hs.distill_topk_forward(z, i.to(torch.int16), v)
    with pytest.raises(TypeError):
        hs.distill_topk_forward(z.double(), i, v)
    with pytest.raises(hs.HessError):
        hs.distill_topk_forward(z, i, v, temperature=0.0)
    with pytest.raises(hs.HessError):
        hs.distill_topk_forward(z, i[:, :0], v[:, :0])
