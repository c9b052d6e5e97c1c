"""The feed-forward block and the distillation loss at the sizes where their kernels change.

Tolerances are those of test_gated_ffn_gpu.py and test_distill_gpu.py, derived there.
"""

import numpy as np
import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from oracle import ops_oracle as R
from tests import test_distill_gpu as D
from tests import test_gated_ffn_gpu as G

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X GPU")]

TYPES = list(G.TYPES)


def forward_case(n, d, f, dt, act):
    x, xn = G.draw(61, dt, n, d)
    wg, gn = G.draw(62, dt, f, d, scale=1.2 / d ** 0.5)
    wu, un = G.draw(63, dt, f, d, scale=1.2 / d ** 0.5)
    h, pre = hs.gated_ffn_forward(x, wg, wu, act=act, save=True)
    torch.cuda.synchronize()
    want, g, u = R.gated_ffn(xn, gn, un, act)
    th, tg, tu = G.forward_tolerance(xn, gn, un, g, u, act, dt)
    G.check("h", h, want, th)
    fp = -(-f // 8) * 8
    G.check("g", pre[:, :f], g, tg)
    G.check("u", pre[:, fp:fp + f], u, tu)
    assert not pre[:, f:fp].any() and not pre[:, fp + f:].any()
    assert torch.equal(h, hs.gated_ffn_forward(x, wg, wu, act=act))


# up to 16, 32 and 64 tokens have a kernel each, which widens at 8192 features
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("d", [72, 73])
@pytest.mark.parametrize("n", [15, 16, 17, 32, 33, 64, 65])
def test_few_tokens_many_features(n, d, dt):
    G.say(f"few {dt} {n}x{d}x8203")
    forward_case(n, d, 8203, dt, R.ACTS[n % 3])


# more tiles than the card has places: whole rounds, and a last round whose tiles may be split along K
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("n,d,f", [(2100, 640, 4200), (1030, 1601, 1290), (129, 2600, 700), (2050, 96, 2176)])
def test_forward_rounds_of_tiles(n, d, f, dt):
    G.say(f"rounds {dt} {n}x{d}x{f}")
    forward_case(n, d, f, dt, "gelu_tanh")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("n,d,f", [(2100, 520, 1000), (1029, 1601, 1290), (1100, 2304, 333), (66, 4100, 2056)])
def test_backward_rounds_of_tiles(n, d, f, dt):
    act = "silu"
    G.say(f"backward rounds {dt} {n}x{d}x{f}")
    x, xn = G.draw(64, dt, n, d)
    wg, gn = G.draw(65, dt, f, d, scale=1.5 / d ** 0.5)
    wu, un = G.draw(66, dt, f, d, scale=1.5 / d ** 0.5)
    dh, dn = G.draw(67, dt, n, f)
    _, g, u = R.gated_ffn(xn, gn, un, act)
    pre, g, u = G.exact_preact(g, u, dt, f)
    dx, dwg, dwu = hs.gated_ffn_backward(dh, x, wg, wu, pre, act=act)
    torch.cuda.synchronize()
    wx, wwg, wwu, dg, du = R.gated_ffn_grads(dn, xn, gn, un, g, u, act)
    tol = G.backward_tolerance(dn, xn, gn, un, dg, du, g, act, dt)
    for name, got, want, t in (("dx", dx, wx, tol[0]), ("dw_gate", dwg, wwg, tol[1]), ("dw_up", dwu, wwu, tol[2])):
        G.check(name, got, want, t * (1 + G.half(dt)) + G.half(dt) * np.abs(want) + G.FLOOR[dt])


@pytest.mark.parametrize("act", R.ACTS)
def test_activation_tails(act):
    """One feature of one input with unit weights: h = act(x) x, in float32 over the activations' whole range."""
    G.say(f"tails {act}")
    g = np.concatenate([np.linspace(-13, 13, 4001), [0.0, -0.0, 1e-30, -1e-30, 60.0, -60.0]]).astype(np.float32)
    one = torch.ones((1, 1), device="cuda")
    h = hs.gated_ffn_forward(torch.from_numpy(g)[:, None].cuda(), one, one, act=act)[:, 0].double().cpu().numpy()
    g = g.astype(np.float64)
    a = R.act_and_slope(g, act)[0]
    # tanh's argument 0.8 (g + 0.045 g^3) is formed with 4 roundings, up to 160 at |g| = 13, in an exponent
    arg = 2 * 0.8 * (np.abs(g) + 0.045 * np.abs(g) ** 3) * 4 * G.U if act == "gelu_tanh" else 0.0
    want = a * g
    # float32's own floor: products below its normal range are flushed
    assert (np.abs(h - want) <= np.abs(want) * (G.ACT_REL + arg + 4 * G.U) + 2.0 ** -126).all()
    special = torch.tensor([[float("inf")], [float("nan")]], device="cuda")
    got = hs.gated_ffn_forward(special, one, one, act=act)
    assert got[0, 0] == float("inf") and torch.isnan(got[1, 0])


@pytest.mark.parametrize("n", [5, 200])
@pytest.mark.parametrize("dt", TYPES)
def test_operands_off_16_bytes(dt, n):
    """Rows of a multiple of 16 bytes that do not start at one: the same bits as aligned copies."""
    G.say(f"off 16 bytes {dt} {n}")
    d, f = 64, 48
    flat = torch.randn(n * d + 1, device="cuda").to(G.TYPES[dt])
    wflat = (torch.randn(2 * f * d + 1, device="cuda") / 8).to(G.TYPES[dt])
    x, w = flat[1:].view(n, d), wflat[1:].view(2 * f, d)
    h, pre = hs.gated_ffn_forward(x, w[:f], w[f:], save=True)
    h2, pre2 = hs.gated_ffn_forward(x.clone(), w[:f].clone(), w[f:].clone(), save=True)
    assert torch.equal(h, h2) and torch.equal(pre, pre2)
    a = hs.gated_ffn_backward(h, x, w[:f], w[f:], pre)
    b = hs.gated_ffn_backward(h, x.clone(), w[:f].clone(), w[f:].clone(), pre)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_far_apart():
    """Row strides whose offsets pass 32 bits: the same bits as contiguous rows."""
    G.say("far rows")
    n, d, f, ld = 2200, 72, 40, 1 << 20
    big = torch.empty(n * ld, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((n, d), (ld, 1))
    x.copy_(torch.randn(n, d, device="cuda"))
    wg, wu = (torch.randn(2 * f, d, device="cuda") / 8).bfloat16().split(f)
    h, pre = hs.gated_ffn_forward(x, wg, wu, save=True)
    xc = x.contiguous()
    assert torch.equal(h, hs.gated_ffn_forward(xc, wg, wu))
    out = big.as_strided((n, f), (ld, 1), 128)
    assert torch.equal(hs.gated_ffn_forward(xc, wg, wu, out=out), h)
    a, b = hs.gated_ffn_backward(h, x, wg, wu, pre), hs.gated_ffn_backward(h, xc, wg, wu, pre)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


# vectors of a row: 512, 1024, 4096, 8192 and 16384 are the limits of the kernels that hold a row in registers
SIZES = {"bf16": [(3, 4103, 5), (300, 4104, 70), (260, 8199, 9), (258, 8200, 33), (258, 32775, 20), (258, 32776, 64),
                  (257, 65543, 7), (257, 65544, 12), (2, 131079, 129), (2, 131080, 40)],
         "f32": [(300, 2051, 16), (258, 16387, 8), (257, 32772, 3), (2, 65539, 300), (2, 65540, 65)],
         "f16": [(258, 16000, 257), (257, 40001, 513), (3, 200000, 1024)]}


@pytest.mark.parametrize("dt,n,vocab,k", [(dt, *s) for dt in SIZES for s in SIZES[dt]])
def test_loss_at_the_kernels_limits(dt, n, vocab, k):
    D.say(f"limits {dt} {n}x{vocab} top {k}")
    z, i, v, w = D.make(n + k, dt, n, vocab, k, absent=0.2, distinct=n < 100)
    D.run_all(z, i, v, w, 1.5, dt)


def test_many_short_rows():
    D.say("many rows")
    z, i, v, w = D.make(71, "bf16", 70000, 9, 3)
    loss, grad = hs.distill_topk_step(z, i, v, weight=w)
    rows = [0, 1, 65535, 65536, 69999]
    zn, inn, vn, wn = D.f64(z[rows]), i[rows].cpu().numpy(), D.f64(v[rows]), D.f64(w[rows])
    l, _, g = R.distill_topk(zn, inn, vn, wn, 1.0)
    tl, tg = D.tolerances(zn, inn, vn, wn, 1.0, 9, l, g, "bf16")
    D.compare(loss[rows], l, tl, "loss")
    D.compare(grad[rows], g, tg, "gradient")


def test_logits_past_32_bit_offsets():
    D.say("far logits")
    n, vocab, k = 16500, 131072, 16
    z = torch.empty((n, vocab), dtype=torch.bfloat16, device="cuda")
    for r in range(0, n, 2048):
        z[r:r + 2048].normal_(generator=torch.Generator("cuda").manual_seed(r))
    i = torch.randint(0, vocab, (n, k), device="cuda")
    v = torch.randn(n, k, device="cuda")
    loss, grad = hs.distill_topk_step(z, i, v)
    l2, stats = hs.distill_topk_forward(z, i, v)
    rows = [0, 16383, 16384, n - 1]
    zn, inn, vn = D.f64(z[rows]), i[rows].cpu().numpy(), D.f64(v[rows])
    l, _, g = R.distill_topk(zn, inn, vn, np.ones(4), 1.0)
    tl, tg = D.tolerances(zn, inn, vn, np.ones(4), 1.0, vocab, l, g, "bf16")
    D.compare(loss[rows], l, tl, "loss")
    D.compare(l2[rows], l, tl, "forward's loss")
    D.compare(grad[rows], g, tg, "gradient")
    hs.distill_topk_backward(torch.ones(n, device="cuda"), z, i, v, stats, out=grad)
    D.compare(grad[rows], g, tg, "backward's gradient")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,d,f", [(20, 72, 65), (300, 200, 520), (2100, 96, 1160)])
def test_preactivations_kept_in_float32(n, d, f, dt):
    """The forward pass's float32 pair, and the backward pass at such a pair."""
    act = R.ACTS[n % 3]
    G.say(f"float32 pair {dt} {n}x{d}x{f} {act}")
    x, xn = G.draw(81, dt, n, d)
    wg, gn = G.draw(82, dt, f, d, scale=1.5 / d ** 0.5)
    wu, un = G.draw(83, dt, f, d, scale=1.5 / d ** 0.5)
    dh, dn = G.draw(84, dt, n, f)
    h, pre = hs.gated_ffn_forward(x, wg, wu, act=act, save=True)
    h16, pre16 = hs.gated_ffn_forward(x, wg, wu, act=act, save=G.TYPES[dt])
    assert pre.dtype == torch.float32 and pre16.dtype == G.TYPES[dt]
    assert torch.equal(h, h16) and torch.equal(pre.to(G.TYPES[dt]), pre16)
    _, g, u = R.gated_ffn(xn, gn, un, act)
    fp = -(-f // 8) * 8
    k = (d + 8) * G.U
    G.check("g", pre[:, :f], g, k * (np.abs(xn) @ np.abs(gn).T))
    G.check("u", pre[:, fp:fp + f], u, k * (np.abs(xn) @ np.abs(un).T))
    pair = torch.zeros((n, 2 * fp), dtype=torch.float32)
    pair[:, :f], pair[:, fp:fp + f] = torch.from_numpy(g), torch.from_numpy(u)
    g, u = pair[:, :f].double().numpy(), pair[:, fp:fp + f].double().numpy()
    grads = hs.gated_ffn_backward(dh, x, wg, wu, pair.cuda(), act=act)
    torch.cuda.synchronize()
    *want, dg, du = R.gated_ffn_grads(dn, xn, gn, un, g, u, act)
    tol = G.backward_tolerance(dn, xn, gn, un, dg, du, g, act, dt)
    for name, got, w, t in zip(("dx", "dw_gate", "dw_up"), grads, want, tol):
        G.check(name, got, w, t * (1 + G.half(dt)) + G.half(dt) * np.abs(w) + G.FLOOR[dt])
    other = torch.float16 if dt == "bf16" else torch.bfloat16
    with pytest.raises(ValueError):
        hs.gated_ffn_forward(x, wg, wu, save=other)
    with pytest.raises(ValueError):
        hs.gated_ffn_backward(dh, x, wg, wu, pre.to(other))


def test_slopes_far_out():
    """gelu_tanh's and silu's derivatives where their polynomial overflows: 1 far right, 0 far left."""
    G.say("slopes far out")
    g = torch.tensor([3e19, -3e19, 1e30, -1e30], device="cuda")
    one = torch.ones((1, 1), device="cuda")
    for act in ("gelu_tanh", "silu", "gelu"):
        pre = torch.zeros((4, 16), device="cuda")
        pre[:, 0], pre[:, 8] = g, 1.0
        # dx = dg + du with dh = 2^-100: dg = dh act'(g), du = dh act(g); only dg through w_up = 0
        dx = hs.gated_ffn_backward(torch.full((4, 1), 2.0 ** -100, device="cuda"), g[:, None], one, 0 * one, pre,
                                   act=act, need_w=False)[0][:, 0]
        assert torch.equal(dx, torch.tensor([2.0 ** -100, 0.0, 2.0 ** -100, 0.0], device="cuda")), (act, dx)
