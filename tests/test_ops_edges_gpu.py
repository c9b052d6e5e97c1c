"""Rows and operands at the ends of what the distillation loss and the feed-forward block promise.

Tolerances are those of test_distill_gpu.py and test_gated_ffn_gpu.py, derived there.
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


# rows held in registers by 128 and 1024 threads, and rows past them
@pytest.mark.parametrize("vocab", [50, 30001, 140000])
@pytest.mark.parametrize("k", [1, 5, 200])
@pytest.mark.parametrize("dt", list(D.TYPES))
def test_only_ids_past_the_vocabulary(dt, k, vocab):
    """A row whose ids are all past the vocabulary, or else absent, is NaN; one of absent ids alone is 0."""
    D.say(f"only bad ids {dt} top {k} of {vocab}")
    z, i, v, w = D.make(31, dt, 6, vocab, k, distinct=k <= vocab, ids=(torch.int64, torch.int32)[k % 2])
    i[1] = vocab
    i[2] = -1
    i[2, k - 1] = vocab + 7         # the others absent
    i[3], v[3] = vocab, -float("inf")   # whatever its value
    i[4] = -1
    i[5], w[5] = vocab, 0.0         # a row left out
    loss, _, grad = D.run_all(z, i, v, w, 1.0, dt)
    assert torch.isnan(loss[1:4]).all() and torch.isnan(grad[1:4]).all()
    assert not loss[4:].any() and not grad[4:].any()
    back = hs.distill_topk_backward(torch.ones(6, device="cuda"), z, i, v, hs.distill_topk_forward(z, i, v, weight=w)[1],
                                    weight=w)
    assert torch.isnan(back[1:4]).all() and not back[4:].any()


@pytest.mark.parametrize("vocab", [3000, 30001, 140000])
@pytest.mark.parametrize("dt", list(D.TYPES))
def test_nan_among_the_teachers_values(dt, vocab):
    """One NaN makes every teacher probability of its row NaN, wherever in the list it stands."""
    D.say(f"NaN teacher {dt} {vocab}")
    z, i, v, w = D.make(32, dt, 5, vocab, 200)
    v[0, 64:128] = float("nan")     # all entries of one wave
    v[1, 128:] = float("nan")
    v[2, 70] = float("nan")
    v[3] = float("nan")
    loss, _, grad = D.run_all(z, i, v, w, 1.0, dt)
    assert torch.isnan(loss[:4]).all() and torch.isfinite(loss[4])
    for r in range(4):
        assert torch.isnan(grad[r, i[r]]).all()
        assert int(torch.isnan(grad[r]).sum()) == 200


def test_more_rows_than_a_grid_takes():
    """2^24 rows of 256 threads are 2^32 threads: two launches, in the loss and in the gradient (137 GB)."""
    n, vocab = 1 << 24, 4104
    D.say(f"{n} rows of {vocab}")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GiB of free GPU memory")
    z = torch.zeros((n, vocab), dtype=torch.bfloat16, device="cuda")
    ids = (torch.arange(n, device="cuda", dtype=torch.int32) % vocab)[:, None].contiguous()
    v = torch.zeros((n, 1), device="cuda")
    rows = [0, 1, n - 3, n - 2, n - 1]
    z[rows] = torch.randn((5, vocab), generator=torch.Generator("cuda").manual_seed(33), device="cuda").bfloat16()
    zn, inn, vn = D.f64(z[rows]), ids[rows].cpu().numpy(), D.f64(v[rows])
    l, _, g = R.distill_topk(zn, inn, vn, np.ones(5), 1.0)
    tl, tg = D.tolerances(zn, inn, vn, np.ones(5), 1.0, vocab, l, g, "bf16")
    loss, stats = hs.distill_topk_forward(z, ids, v)
    D.compare(loss[rows], l, tl, "loss")
    assert stats[2, 0] == 0 and stats[n - 4, 0] == 0
    # every other row is the same one: equal logits
    lz, _, gz = R.distill_topk(np.zeros((1, vocab)), np.zeros((1, 1), dtype=np.int64), np.zeros((1, 1)), np.ones(1), 1.0)
    tz = D.tolerances(np.zeros((1, vocab)), np.zeros((1, 1), dtype=np.int64), np.zeros((1, 1)), np.ones(1), 1.0, vocab,
                      lz, gz, "bf16")[0][0]
    assert float((loss[2:n - 3].double() - lz[0]).abs().max()) <= tz
    loss2, _ = hs.distill_topk_step(z, ids, v, out=z)
    torch.cuda.synchronize()
    D.compare(loss2[rows], l, tl, "step's loss")
    D.compare(z[rows], g, tg, "gradient")
    at = z[2:n - 3].gather(1, ids[2:n - 3].long())
    assert (at == at[0]).all() and abs(float(at[0]) - gz[0, 0]) <= 2.0 ** -8
    del z, at
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [20, 70, 300])
@pytest.mark.parametrize("dt", list(D.TYPES))
def test_padding_of_the_saved_pair_is_zero(dt, n):
    """Columns f .. f' - 1 of the saved pair are zeros whatever x and the weights hold."""
    D.say(f"padding {dt} {n}")
    d, f = 72, 61
    gen = torch.Generator("cuda").manual_seed(34)
    x = torch.randn((n, d), generator=gen, device="cuda").to(D.TYPES[dt])
    wg, wu = (torch.randn((2 * f, d), generator=gen, device="cuda") / 8).to(D.TYPES[dt]).split(f)
    x[3, 5], x[7, 70], wg[f - 1, 2] = float("inf"), float("nan"), float("-inf")
    for save in (True, D.TYPES[dt]):
        pre = hs.gated_ffn_forward(x, wg, wu, save=save)[1]
        assert not pre[:, f:64].any() and not pre[:, 64 + f:].any()
        assert torch.isnan(pre[7, :f]).all() and not torch.isfinite(pre[3, 64:64 + f]).any()


def test_smallest_temperature():
    """At 2^-126 both softmaxes are one word each: the gradient is weight / T there, with either sign."""
    D.say("smallest temperature")
    z, i, v, w = D.make(35, "f32", 4, 500, 20)
    best = z.argmax(1)
    i[:2, 3], v[:2, 3] = best[:2], 50.0     # rows 0 and 1: the teacher agrees
    i[2:, 3], v[2:, 3] = (best[2:] + 1) % 500, 50.0
    w[:] = 1.0
    t = 2.0 ** -126
    loss, grad = hs.distill_topk_step(z, i, v, weight=w, temperature=t)
    assert not loss[:2].any() and not grad[:2].any()
    want = torch.zeros_like(z)
    for r in (2, 3):
        want[r, best[r]], want[r, i[r, 3]] = 1 / t, -1 / t
    assert torch.equal(grad, want)
    far = (z[2:].gather(1, best[2:, None]) - z[2:].gather(1, i[2:, 3:4]))[:, 0].double() / t
    assert torch.allclose(loss[2:].double(), far.float().double(), rtol=2.0 ** -21, atol=0.0)
    with pytest.raises(hs.HessError, match="temperature"):
        hs.distill_topk_step(z, i, v, weight=w, temperature=1e-40)


@pytest.mark.parametrize("dt", list(D.TYPES))
@pytest.mark.parametrize("n", [1, 24, 64])
def test_few_tokens_copy_no_weights(n, dt):
    """Up to 64 tokens the forward pass reads weights of any alignment where they are."""
    D.say(f"no copies {dt} {n}")
    d, f = 512, 2048
    gen = torch.Generator("cuda").manual_seed(36)
    flat = (torch.randn(2 * f * (d + 8) + 1, generator=gen, device="cuda") / 16).to(D.TYPES[dt])
    x = torch.randn((n, d), generator=gen, device="cuda").to(D.TYPES[dt])
    xn = D.f64(x)
    # rows off 16 bytes; rows at an odd stride
    for w in (flat[1:1 + 2 * f * d].view(2 * f, d), flat[:2 * f * (d + 1)].view(2 * f, d + 1)[:, :d]):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        h = hs.gated_ffn_forward(x, w[:f], w[f:])
        assert torch.cuda.max_memory_allocated() - before < w[:f].numel() * w.element_size() // 2
        want, g, u = R.gated_ffn(xn, D.f64(w[:f]), D.f64(w[f:]), "silu")
        tol = G.forward_tolerance(xn, D.f64(w[:f]), D.f64(w[f:]), g, u, "silu", dt)[0]
        G.check("h", h, want, tol)


@pytest.mark.parametrize("dt", list(D.TYPES))
@pytest.mark.parametrize("n,d,f", [(33, 1032, 4104), (64, 264, 8200), (48, 5128, 136), (64, 5120, 4096), (31, 10248, 40)])
def test_tokens_where_tiles_take_over(n, d, f, dt):
    """Up to 64 tokens through the tiles, and through the other kernel where the rows do not start at 16 bytes."""
    D.say(f"take over {dt} {n}x{d}x{f}")
    x, xn = G.draw(41, dt, n, d)
    w, wn = G.draw(42, dt, 2 * f, d, scale=1.5 / d ** 0.5)
    want, g, u = R.gated_ffn(xn, wn[:f], wn[f:], "gelu")
    tol = G.forward_tolerance(xn, wn[:f], wn[f:], g, u, "gelu", dt)[0]
    G.check("h", hs.gated_ffn_forward(x, w[:f], w[f:], act="gelu"), want, tol)
    off = torch.empty(2 * f * d + 1, dtype=w.dtype, device="cuda")[1:].view(2 * f, d)
    off.copy_(w)
    G.check("h, weights off 16 bytes", hs.gated_ffn_forward(x, off[:f], off[f:], act="gelu"), want, tol)
    far = torch.zeros((n, d + 1), dtype=x.dtype, device="cuda")[:, :d]
    far.copy_(x)
    G.check("h, x at an odd stride", hs.gated_ffn_forward(far, w[:f], w[f:], act="gelu"), want, tol)


def test_gelu_relative_accuracy():
    """float32 gelu over the whole range.  In units u = 2^-24, relative: the fit 1; the hardware exponential 2; t's
    argument 1 and reciprocal 2, times the slope of t q(t), 1 + t q' / q, which is largest at t = 1: 3.8, so 12; the
    polynomial's eight steps, damped by t < 1, 3; the exponent's low part 1; the products e t q 2; 1 - tail 1; g times
    it 1: 23 in all."""
    D.say("gelu accuracy")
    g = np.concatenate([np.linspace(-12.9, 12.9, 400001), -np.logspace(-30, 1.1, 100001), np.logspace(-30, 1.1, 100001)])
    g = g.astype(np.float32)
    x = torch.from_numpy(np.stack([g, np.ones_like(g)], 1)).cuda()
    gate, up = torch.tensor([[1.0, 0.0]], device="cuda"), torch.tensor([[0.0, 1.0]], device="cuda")
    h = hs.gated_ffn_forward(x, gate, up, act="gelu")[:, 0].double().cpu().numpy()
    want = R.act_and_slope(g.astype(np.float64), "gelu")[0]
    assert (np.abs(h - want) <= 23 * G.U * np.abs(want) + 2.0 ** -126).all()
