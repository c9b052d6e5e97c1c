"""What the 8-bit calls promise at their limits: padding columns, bytes behind rows, no copies that are not needed."""

import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from tests import test_int8_gpu as I

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X GPU")]

TYPES, say = I.TYPES, I.say
FILL = 0x5A


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("block", [0, 32])
@pytest.mark.parametrize("n,d,pad,ldc", [(3, 32, 64, 64), (5, 40, 80, 96), (2, 33, 128, 130), (1, 1, 200, 200),
                                         (4, 64, 64, 70), (3, 40, 40, 48), (3, 40, 45, 48), (2, 40, 67, 67),
                                         (300, 700, 1501, 1503), (2, 31, 9000, 9001)])
def test_padding_columns(n, d, pad, ldc, block, dt):
    """quantize writes zeros from d to pad, whatever pad is, and nothing behind it or behind the scales."""
    say(f"padding columns {dt} block {block} {n}x{d} pad {pad}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, d, generator=gen, device="cuda").to(TYPES[dt])
    want = hs.quantize_int8(x, block=block)
    codes = torch.full((n + 1, ldc), FILL, dtype=torch.int8, device="cuda")
    used = n * 4 if block == 0 else n * -(-d // 32)
    scale = torch.full((used + 16,), FILL, dtype=torch.uint8, device="cuda")
    lib = hs._load()
    hs._check(lib.hess_int8_quantize(x.data_ptr(), d, hs._CODES[x.dtype], n, d, block, codes.data_ptr(), ldc, pad,
                                     scale.data_ptr(), stream()))
    assert torch.equal(codes[:n, :d], want.codes)
    assert not codes[:n, d:pad].any(), "columns d to pad are not zeros"
    assert (codes[:n, pad:] == FILL).all() and (codes[n] == FILL).all() and (scale[used:] == FILL).all()
    assert torch.equal(scale[:used].view(want.scale.dtype).flatten().view(torch.uint8), want.scale.contiguous().flatten().view(torch.uint8))


@pytest.mark.parametrize("n,d,f", [(70, 40, 24), (300, 333, 130), (70, 8201, 5)])
def test_weights_that_end_with_their_last_code(n, d, f, monkeypatch):
    """Rows that tiles could read in place, but for the end of the last one's storage: copied, the outputs the same."""
    say(f"weights that end with their last code {n}x{d}x{f}")
    lib = hs._load()
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(n, d, generator=gen, device="cuda").bfloat16()
    w = hs.quantize_int8(torch.randn(f, d, generator=gen, device="cuda").bfloat16())
    x8, want, ld = hs.quantize_int8(x), hs.int8_linear_forward(x, w), -(-d // 16) * 16
    seen = []
    for name, at in (("hess_int8_linear_forward", 3), ("hess_int8_matmul", 3)):
        call = getattr(lib, name)
        monkeypatch.setattr(lib, name, lambda *a, call=call, at=at: seen.append(a[at:at + 2]) or call(*a))
    whole = torch.empty((f, ld), dtype=torch.int8, device="cuda")[:, :d]
    short = torch.empty((f - 1) * ld + d, dtype=torch.int8, device="cuda").as_strided((f, d), (ld, 1))
    for codes, copied in ((whole, False), (short, True)):
        codes.copy_(w.codes)
        rows = hs.Int8Rows(codes, w.scale)
        for y in (hs.int8_linear_forward(x, rows), hs.int8_matmul(x8, rows)):
            pointer, stride = seen.pop()
            assert (pointer != codes.data_ptr() and stride < ld) if copied else (pointer, stride) == (codes.data_ptr(), ld)
            assert torch.equal(y, want)


@pytest.mark.parametrize("n,d", [(1, 4096), (1, 8192), (24, 4096), (64, 4096), (64, 8176), (32, 8192), (32, 16384)])
def test_few_rows_of_unaligned_weights_copy_nothing(n, d):
    """Up to 64 rows the kernels read weights of any alignment: a call takes no memory of the weights' size."""
    f = 1000
    say(f"no copies {n}x{d}")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(n, d, generator=gen, device="cuda").bfloat16()
    w = hs.quantize_int8(torch.randn(f, d, generator=gen, device="cuda").bfloat16())
    odd = torch.empty(f * d + 1, dtype=torch.int8, device="cuda")[1:].view(f, d)
    odd.copy_(w.codes)
    wide = torch.empty(f, d + 5, dtype=torch.int8, device="cuda")[:, :d]
    wide.copy_(w.codes)
    want, x8 = hs.int8_linear_forward(x, w), hs.quantize_int8(x)
    for codes in (odd, wide):
        w_odd = hs.Int8Rows(codes, w.scale)
        for call in (lambda: hs.int8_linear_forward(x, w_odd), lambda: hs.int8_linear_forward(x, w_odd, save=True)[0],
                     lambda: hs.int8_matmul(x8, w_odd), lambda: hs.int8_linear(x, w_odd)):
            torch.cuda.synchronize()
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            got = call()
            assert torch.cuda.max_memory_allocated() - before < f * d // 2, "the weights were copied"
            assert torch.equal(got, want)


@pytest.mark.parametrize("n,d", [(33, 8192), (65, 4096), (65, 8192), (33, 16384), (64, 8192)])
def test_tiles_of_unaligned_weights(n, d):
    """One row past where the kernels read any alignment: the rows are copied first, the outputs the same."""
    f = 300
    say(f"unaligned tiles {n}x{d}")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, d, generator=gen, device="cuda").bfloat16()
    w = hs.quantize_int8(torch.randn(f, d, generator=gen, device="cuda").bfloat16())
    odd = torch.empty(f * d + 1, dtype=torch.int8, device="cuda")[1:].view(f, d)
    odd.copy_(w.codes)
    x8 = hs.quantize_int8(x)
    ax = torch.empty(n, d + 3, dtype=torch.int8, device="cuda")[:, :d]
    ax.copy_(x8.codes)
    want = hs.int8_linear_forward(x, w)
    assert torch.equal(hs.int8_linear_forward(x, hs.Int8Rows(odd, w.scale)), want)
    assert torch.equal(hs.int8_matmul(hs.Int8Rows(ax, x8.scale), hs.Int8Rows(odd, w.scale)), want)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("n,f,edge,whole,parts", [(5, 1, 0, 0, 1), (70, 32, 0, 0, 1), (70, 33, 0, 0, 1), (300, 200, 0, 0, 1),
                                                  (300, 256, 256, 1 << 30, 1), (300, 330, 64, 0, 2), (300, 330, 128, 2, 2),
                                                  (300, 96, 128, 1 << 30, 1), (300, 330, 256, 0, 2)])
def test_saved_pair_is_written_whole(n, f, edge, whole, parts, dt):
    """Every byte of the pair in 8 bits is the call's: those behind the exponents are zeros, and equal calls leave
    equal tensors whatever the memory held."""
    d = 520
    say(f"pair written whole {dt} {n}x{d}x{f} edge {edge} whole {whole} parts {parts}")
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(n, d, generator=gen, device="cuda").to(TYPES[dt])
    wg, wu = ((torch.randn(f, d, generator=gen, device="cuda") / 20).to(TYPES[dt]) for _ in range(2))
    lib, code = hs._load(), hs._CODES[x.dtype]
    cols, fq = lib.hess_gated_ffn_preact_i8_cols(f), -(-f // 32) * 32
    made = []
    try:
        hs.set_ffn_schedule(edge, whole, parts)
        for fill in (FILL, 0x25):
            pre = torch.full((n + 1, cols), fill, dtype=torch.int8, device="cuda")
            h = torch.empty(n, f, dtype=x.dtype, device="cuda")
            work = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
            hs._check(lib.hess_gated_ffn_forward(x.data_ptr(), d, wg.data_ptr(), d, wu.data_ptr(), d, code, hs._PREACT_I8, n, d,
                                                 f, h.data_ptr(), f, pre.data_ptr(), work.data_ptr(), work.numel(), stream()))
            assert (pre[n] == fill).all(), "written behind the last row"
            made.append(pre[:n])
    finally:
        hs.set_ffn_schedule()
    assert not made[0][:, 2 * fq + fq // 16:].any(), "bytes behind the exponents are not zeros"
    assert torch.equal(made[0], made[1])
