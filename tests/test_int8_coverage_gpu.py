"""8-bit kernels at the sizes that only large calls reach: tiles in more than one round of the card, a second turn
of a loop over the grid, a second launch, rows past a slice.  Tolerances are those of test_int8_gpu.py; products of
codes and codes of given values are exact."""

import numpy as np
import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from oracle import ops_oracle as R
from tests import test_gated_ffn_gpu as G
from tests import test_int8_gpu as I

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X GPU")]

TYPES, U, say, draw, check, half = I.TYPES, I.U, I.say, I.draw, I.check, I.half


def exact_product(a, b):
    """The product in float64 (its sums are whole numbers below 2^53), on the GPU."""
    return torch.mm(a.codes.double(), b.codes.double().t().contiguous()) * torch.outer(a.scale.double(), b.scale.double())


def check_product(y, want):
    # the sum to float32, two scales, the output's type
    dt = next(k for k, v in TYPES.items() if v == y.dtype)
    off = (y.double() - want).abs() - (want.abs() * ((half(dt) + 3.01 * U) * (1 + half(dt))) + I.FLOOR[dt])
    assert bool((off <= 0).all()), f"{int((off > 0).sum())} of {off.numel()} off, first at {off.argmax()}"


# tiles: 64 from 513 workgroups on and 128 from 257 on have stages of their own; 256 from 257 on a second round
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d,f,edge,whole,parts", [
    (2000, 1333, 2600, 64, 1 << 30, 1), (2000, 1333, 2600, 64, 0, 2), (2000, 1040, 2600, 64, 1 << 30, 1),
    (2000, 1333, 2600, 128, 1 << 30, 1), (2000, 1333, 2600, 128, 0, 3), (2000, 1040, 2600, 128, 100, 2),
    (4200, 1333, 4200, 256, 1 << 30, 1), (4200, 1040, 4200, 256, 3, 2), (2000, 100, 2600, 64, 1 << 30, 1),
    (2000, 200, 2600, 128, 1 << 30, 1)])
def test_matmul_of_many_tiles(n, d, f, edge, whole, parts, dt):
    say(f"matmul {dt} {n}x{d}x{f} edge {edge} whole {whole} parts {parts}")
    a, b = I.random_codes(21, n, d), I.random_codes(22, f, d)
    try:
        hs.set_ffn_schedule(edge, whole, parts)
        y = hs.int8_matmul(a, b, dtype=TYPES[dt])
    finally:
        hs.set_ffn_schedule()
    check_product(y, exact_product(a, b))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d,f", [(1999, 500, 9728), (777, 1001, 2731), (9000, 130, 4100), (5000, 64, 5000), (65, 300, 131072)])
def test_matmul_in_rounds(n, d, f, dt):
    """The library's own schedules at products of one round of the card and more."""
    say(f"matmul {dt} {n}x{d}x{f}")
    a, b = I.random_codes(23, n, d), I.random_codes(24, f, d)
    check_product(hs.int8_matmul(a, b, dtype=TYPES[dt]), exact_product(a, b))


def power(e):
    """2^e in float64."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def block_codes(x):
    """(codes, exponent bytes) of x's blocks of 32 columns, in float64 on the GPU."""
    n, d = x.shape
    groups = -(-d // 32)
    v = torch.nn.functional.pad(x.double(), (0, groups * 32 - d)).view(n, groups, 32)
    top = v.abs().amax(2)
    # top = m 2^e with 1/2 <= m < 1: 64 <= top / 2^(e - 7) < 128
    e = (torch.frexp(top)[1] - 7).clamp(min=-126)
    e = torch.where(top > 0, e, -126)
    q = torch.round(v * power(-e)[..., None]).clamp(-127, 127)
    return q.view(n, groups * 32)[:, :d].to(torch.int8), (e + 127).to(torch.uint8)


@pytest.mark.parametrize("dt", list(TYPES))
def test_blocks_of_a_long_batch(dt):
    """More values than the grid takes in one turn (16.8 million, restored 8.4 or 16.8), rows of odd lengths."""
    n, d = 4300, 4099
    say(f"blocks {dt} {n}x{d}")
    gen = torch.Generator(device="cuda").manual_seed(31)
    x = (torch.randn(n, d, generator=gen, device="cuda") * torch.exp(torch.randn(n, 1, generator=gen, device="cuda"))).to(TYPES[dt])
    q = hs.quantize_int8(x, block=32)
    codes, exps = block_codes(x)
    assert torch.equal(q.codes, codes) and torch.equal(q.scale.view(torch.uint8), exps)
    assert not torch.as_strided(q.codes, (n, q.codes.stride(0) - d), (q.codes.stride(0), 1), d).any(), "columns past d"
    want = codes.double() * power(exps.int() - 127).repeat_interleave(32, 1)[:, :d]
    for out in TYPES.values():
        assert torch.equal(hs.dequantize_int8(q, dtype=out), want.to(out))


@pytest.mark.parametrize("dt", list(TYPES))
def test_rows_of_a_second_launch(dt):
    """More rows than one launch takes (2^20), a scale a row, and the product of so many."""
    n, d = (1 << 20) + 77, 5
    say(f"rows {dt} {n}x{d}")
    gen = torch.Generator(device="cuda").manual_seed(32)
    x = torch.randn(n, d, generator=gen, device="cuda").to(TYPES[dt])
    q = hs.quantize_int8(x)
    top = x.double().abs().amax(1)
    assert torch.equal(q.codes, torch.round(127.0 * x.double() / top[:, None]).to(torch.int8))
    assert torch.equal(q.scale, x.float().abs().amax(1) / torch.full((n,), 127.0, device="cuda"))
    b = I.random_codes(33, 3, d)
    check_product(hs.int8_matmul(q, b, dtype=TYPES[dt]), exact_product(q, b))
    y, x8 = hs.int8_linear_forward(x, b, save=True)  # a copy of the weights goes with the first launch
    assert torch.equal(x8.codes, q.codes) and torch.equal(x8.scale, q.scale)
    assert torch.equal(y, hs.int8_matmul(q, b, dtype=TYPES[dt])) and torch.equal(y, hs.int8_linear_forward(x, b))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,d,f", [(32768 + 70, 16, 24), (32768, 20, 33), (70, 40, 2100), (1200, 64, 4100)])
def test_ffn_checkpoint_of_many_rows_and_features(n, d, f, dt):
    """The gate gradients in two slices of rows, or more workgroups a row than one, x restored beside them."""
    I.test_ffn_checkpoint(n, d, f, dt)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("edge,whole,parts", [(64, 0, 2), (128, 0, 3), (128, 2, 2), (256, 0, 2), (256, 1, 3)])
@pytest.mark.parametrize("act", R.ACTS)
def test_ffn_checkpoint_activations_of_split_tiles(act, edge, whole, parts, dt):
    """Every activation where the parts of a sum are joined: the pair does not depend on it."""
    n, d, f = 300, 520, 330
    say(f"ffn in 8 bits {dt} {act} edge {edge} whole {whole} parts {parts}")
    x, xn = draw(1, dt, n, d)
    wg, gn = draw(2, dt, f, d, scale=1.5 / d ** 0.5)
    wu, un = draw(3, dt, f, d, scale=1.5 / d ** 0.5)
    want, g, u = R.gated_ffn(xn, gn, un, act)
    try:
        hs.set_ffn_schedule(edge, whole, parts)
        h, pre = hs.gated_ffn_forward(x, wg, wu, act=act, save=torch.int8)
        plain = hs.gated_ffn_forward(x, wg, wu, act=act)
    finally:
        hs.set_ffn_schedule()
    assert torch.equal(h, plain)
    check("h", h, want, G.forward_tolerance(xn, gn, un, g, u, act, dt)[0])
    k = (d + 8) * U
    I.check_pair(pre, f, g, u, k * (np.abs(xn) @ np.abs(gn).T), k * (np.abs(xn) @ np.abs(un).T))
