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
