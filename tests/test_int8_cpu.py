"""8-bit integers without a GPU: the arithmetic of the codes, and the refusals of the C ABI and the binding."""

import ctypes
import os

import numpy as np
import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from oracle import ops_oracle as R

built = pytest.mark.skipif(not os.path.exists(hs.library_path()), reason="libhess.so not built")
EINVAL, EALIGN = -1, -5
GB = 1 << 30


def _ptr(i, off=0):
    return ctypes.c_void_p((1 << 40) + i * 64 * GB + off)


def _message():
    return hs._load().hess_last_error()


@pytest.mark.parametrize("bits", [8, 11])
def test_codes_of_16_bit_rows_are_exact(bits):
    """rint of 127 x / a formed in float32 and rounded to 2^-21 relative is the exact quotient's, for every pair
    of mantissas and every exponent that leaves a code of 1 or more."""
    lo, hi = 1 << (bits - 1), 1 << bits
    a = np.arange(lo, hi, dtype=np.int64)[:, None]
    for e in range(9):
        x = np.arange(lo, hi, dtype=np.int64)[None, :]
        inverse = (np.float32(127.0) / a.astype(np.float32)).astype(np.float32)
        t = (x.astype(np.float32) * np.float32(2.0 ** -e)) * inverse
        snapped = ((t.view(np.uint32) + np.uint32(4)) & np.uint32(0xfffffff8)).view(np.float32)
        got = np.rint(snapped).astype(np.int64)
        # the exact one: 2 * 127 x / (a 2^e) against odd whole numbers, ties to even
        num, den = 127 * x, a << e
        q, r = num // den, num % den
        want = q + ((2 * r > den) | ((2 * r == den) & (q % 2 == 1)))
        inside = (x <= den)  # |x| <= a
        assert (got == want)[np.broadcast_to(inside, got.shape)].all()


def test_codes_of_float32_rows_are_exact():
    """The same for float32: formed in float64 and rounded to 2^-40, at ties and next to them."""
    rng = np.random.default_rng(0)
    a = np.concatenate([rng.integers(1 << 23, 1 << 24, 4000), np.full(500, 127 << 17), np.full(500, 254 << 16)])
    odd = 2 * rng.integers(0, 127, a.size) + 1
    near = (a * odd // 254)  # 127 x / a is next to odd / 2
    for off in (-1, 0, 1):
        x = near + off
        t = x.astype(np.float64) * (127.0 / a.astype(np.float64))
        got = np.rint((t + 6144.0) - 6144.0).astype(np.int64)
        num = [127 * int(v) for v in x]
        want = []
        for n, d in zip(num, a.tolist()):
            q, r = divmod(n, d)
            want.append(q + (2 * r > d or (2 * r == d and q % 2 == 1)))
        assert (got == np.array(want)).all()


def test_oracle_blocks():
    x = np.zeros((1, 70))
    x[0, :3] = 127.0, -63.5, 0.5
    x[0, 32:34] = 127.5, 1.0
    x[0, 64] = 2.0 ** -140
    codes, steps = R.quantize_blocks(x)
    assert steps.tolist() == [[1.0, 1.0, 2.0 ** -126]]
    assert codes[0, :3].tolist() == [127.0, -64.0, 0.0] and codes[0, 32:34].tolist() == [127.0, 1.0]
    assert not codes[0, 64:].any() and np.array_equal(R.stand_for(codes, steps)[0, :3], [127.0, -64.0, 0.0])


def _quantize(x=_ptr(0), ldx=40, dtype=0, n=5, d=40, block=0, codes=_ptr(1), ldc=48, pad=48, scale=_ptr(2)):
    return hs._load().hess_int8_quantize(x, ldx, dtype, n, d, block, codes, ldc, pad, scale, None)


def _dequantize(codes=_ptr(1), ldc=48, scale=_ptr(2), n=5, d=40, block=32, x=_ptr(0), ldx=40, dtype=0):
    return hs._load().hess_int8_dequantize(codes, ldc, scale, n, d, block, x, ldx, dtype, None)


@built
def test_rows_refusals():
    assert _quantize(n=0) == 0 and _dequantize(n=0) == 0
    for kw, code, word in [
            (dict(dtype=3), EINVAL, b"dtype"), (dict(n=-1), EINVAL, b"n = "), (dict(d=0), EINVAL, b"d = "),
            (dict(n=(1 << 24) + 1), EINVAL, b"n = "), (dict(d=(1 << 17) + 1), EINVAL, b"d = "),
            (dict(block=16), EINVAL, b"block"), (dict(ldx=39), EINVAL, b"of x"), (dict(ldc=39), EINVAL, b"of codes"),
            (dict(ldx=(1 << 20) + 1), EINVAL, b"of x"), (dict(x=None), EINVAL, b"null x"),
            (dict(codes=None), EINVAL, b"null codes"), (dict(scale=None), EINVAL, b"null scale"),
            (dict(x=_ptr(0, 1)), EALIGN, b"x not aligned"), (dict(scale=_ptr(2, 2)), EALIGN, b"scale"),
            (dict(codes=_ptr(0, 100)), EINVAL, b"codes overlaps x"), (dict(scale=_ptr(1, 100)), EINVAL, b"overlaps")]:
        assert _quantize(**kw) == code and word in _message(), (kw, _message())
        if "x" not in kw and "ldx" not in kw and "scale" not in kw and "codes" not in kw:
            assert _dequantize(**kw) == code, kw
    for pad in (39, 49):
        assert _quantize(pad=pad) == EINVAL and b"pad" in _message()
    assert _dequantize(x=_ptr(1, 16)) == EINVAL and b"x overlaps codes" in _message()
    assert _dequantize(x=_ptr(2)) == EINVAL and b"x overlaps scale" in _message()
    assert _quantize(block=32, scale=None) == EINVAL and b"null scale" in _message()


def _matmul(n=5, d=40, f=24, a=_ptr(0), lda=48, sa=_ptr(1), b=_ptr(2), ldb=48, sb=_ptr(3), y=_ptr(4), ldy=24, dtype=0,
            work=_ptr(5), bytes_=GB):
    return hs._load().hess_int8_matmul(a, lda, sa, b, ldb, sb, n, d, f, y, ldy, dtype, work, bytes_, None)


@built
def test_matmul_refusals():
    assert _matmul(n=0) == 0
    for kw, code, word in [
            (dict(dtype=7), EINVAL, b"dtype"), (dict(n=-1), EINVAL, b"n = "), (dict(f=0), EINVAL, b"f = "),
            (dict(d=1 << 17, lda=1 << 17, ldb=1 << 17), EINVAL, b"32 bits"), (dict(lda=39), EINVAL, b"of a"),
            (dict(ldb=39), EINVAL, b"of b"), (dict(ldy=23), EINVAL, b"of y"), (dict(a=None), EINVAL, b"null a"),
            (dict(sb=None), EINVAL, b"null b_scale"), (dict(sa=_ptr(1, 1)), EALIGN, b"a_scale"),
            (dict(y=_ptr(4, 1)), EALIGN, b"y not aligned"), (dict(y=_ptr(2)), EINVAL, b"y overlaps b"),
            (dict(y=_ptr(1, 4)), EINVAL, b"y overlaps a_scale")]:
        assert _matmul(**kw) == code and word in _message(), (kw, _message())
    assert hs._load().hess_int8_matmul_workspace(-1, 4, 4) == -1
    assert hs._load().hess_int8_matmul_workspace(1, 1 << 17, 4) == -1


def _forward(n=5, d=40, f=24, x=_ptr(0), ldx=40, dtype=0, w=_ptr(1), ldw=40, sw=_ptr(2), y=_ptr(3), ldy=24, xc=_ptr(4),
             ldc=48, xs=_ptr(5), work=_ptr(6), bytes_=GB):
    return hs._load().hess_int8_linear_forward(x, ldx, dtype, w, ldw, sw, n, d, f, y, ldy, xc, ldc, xs, work, bytes_,
                                               None)


def _backward(n=5, d=40, f=24, dy=_ptr(0), lddy=24, dtype=0, xc=_ptr(1), ldc=48, xs=_ptr(2), w=_ptr(3), ldw=40,
              sw=_ptr(4), dx=_ptr(5), lddx=40, dw=_ptr(6), lddw=40, work=_ptr(7), bytes_=GB):
    return hs._load().hess_int8_linear_backward(dy, lddy, dtype, xc, ldc, xs, w, ldw, sw, n, d, f, dx, lddx, dw, lddw,
                                                work, bytes_, None)


@built
def test_linear_refusals():
    assert _forward(n=0) == 0 and _backward(n=0, dw=None) == 0 and _backward(dx=None, dw=None) == 0
    for kw, code, word in [
            (dict(dtype=-1), EINVAL, b"dtype"), (dict(n=(1 << 24) + 1), EINVAL, b"n = "),
            (dict(d=1 << 17, ldx=1 << 17, ldw=1 << 17), EINVAL, b"32 bits"), (dict(xs=None), EINVAL, b"both or neither"),
            (dict(xc=None), EINVAL, b"both or neither"), (dict(ldx=39), EINVAL, b"of x"), (dict(ldw=39), EINVAL, b"of w"),
            (dict(ldy=23), EINVAL, b"of y"), (dict(ldc=40), EINVAL, b"of x_codes"), (dict(ldc=56), EALIGN, b"x_codes"),
            (dict(xc=_ptr(4, 8)), EALIGN, b"x_codes"), (dict(xs=_ptr(5, 2)), EALIGN, b"x_scale"),
            (dict(x=None), EINVAL, b"null x"), (dict(w=None), EINVAL, b"null w"), (dict(y=None), EINVAL, b"null y"),
            (dict(x=_ptr(0, 1)), EALIGN, b"x not aligned"), (dict(y=_ptr(0)), EINVAL, b"y overlaps x"),
            (dict(xc=_ptr(1, 16)), EINVAL, b"x_codes overlaps w"), (dict(xs=_ptr(3, 4)), EINVAL, b"y overlaps x_scale"),
            (dict(bytes_=16), EINVAL, b"workspace"), (dict(work=None), EINVAL, b"workspace"),
            (dict(work=_ptr(6, 8)), EALIGN, b"workspace"), (dict(work=_ptr(0)), EINVAL, b"overlaps the workspace")]:
        if "bytes_" in kw or "work" in kw:
            kw = dict(kw, xc=None, xs=None, n=100)
        assert _forward(**kw) == code and word in _message(), (kw, _message())
    for kw, code, word in [
            (dict(dtype=4), EINVAL, b"dtype"), (dict(dy=None), EINVAL, b"null dy"), (dict(lddy=23), EINVAL, b"of dy"),
            (dict(lddy=25), EALIGN, b"dy"), (dict(dy=_ptr(0, 2)), EALIGN, b"dy"), (dict(xc=None), EINVAL, b"x_codes"),
            (dict(xs=None), EINVAL, b"x_scale"), (dict(w=None), EINVAL, b"null w"), (dict(sw=None), EINVAL, b"w_scale"),
            (dict(lddx=39), EINVAL, b"of dx"), (dict(lddw=39), EINVAL, b"of dw"), (dict(dx=_ptr(0)), EINVAL, b"dx overlaps dy"),
            (dict(dw=_ptr(5, 64)), EINVAL, b"dx overlaps dw"), (dict(dw=_ptr(1)), EINVAL, b"dw overlaps x_codes"),
            (dict(bytes_=16), EINVAL, b"workspace"), (dict(work=_ptr(3)), EINVAL, b"overlaps the workspace")]:
        assert _backward(**kw) == code and word in _message(), (kw, _message())
    for bad in (-1, 5):
        assert hs._load().hess_int8_linear_workspace(5, 8, 8, 0, bad) == -1
    assert hs._load().hess_int8_linear_workspace(0, 8, 8, 0, 3) == 0


@built
def test_ffn_pair_in_8_bits_refusals():
    lib = hs._load()
    assert [lib.hess_gated_ffn_preact_i8_cols(f) for f in (0, 1, 32, 33, 64, (1 << 17) + 1)] == [-1, 80, 80, 144, 144, -1]

    def forward(act=64, pre=_ptr(4), bytes_=GB, xoff=0):
        return lib.hess_gated_ffn_forward(_ptr(0, xoff), 24, _ptr(1), 24, _ptr(2), 24, 0, act, 5, 24, 40, _ptr(3), 40, pre,
                                          _ptr(5), bytes_, None)

    for kw, code, word in [(dict(act=64 + 3), EINVAL, b"activation"), (dict(act=64 + 16), EINVAL, b"activation"),
                           (dict(pre=_ptr(4, 8)), EALIGN, b"preact"), (dict(pre=_ptr(3, 16)), EINVAL, b"h overlaps preact"),
                           (dict(xoff=2), EALIGN, b"16-byte")]:
        assert forward(**kw) == code and word in _message(), (kw, _message())


@built
def test_ffn_backward_x8_refusals():
    lib = hs._load()

    def backward(xc=_ptr(1), ldc=24, xe=_ptr(9), pre=_ptr(4), act=64, dx=_ptr(5), dwg=_ptr(6), dwu=_ptr(7), bytes_=GB):
        return lib.hess_gated_ffn_backward_x8(_ptr(0), 40, xc, ldc, xe, _ptr(2), 24, _ptr(3), 24, pre, 0, act, 5, 24, 40,
                                              dx, 24, dwg, 24, dwu, 24, _ptr(8), bytes_, None)

    assert backward(dx=None, dwg=None, dwu=None) == 0
    for kw, code, word in [(dict(xc=None), EINVAL, b"null x"), (dict(xe=None), EINVAL, b"x_exponents"),
                           (dict(ldc=23), EINVAL, b"of x"), (dict(dx=_ptr(1, 8)), EINVAL, b"dx overlaps x"),
                           (dict(dwg=_ptr(9, 2)), EINVAL, b"dw_gate overlaps x_exponents"),
                           (dict(pre=_ptr(4, 4)), EALIGN, b"preact"), (dict(act=80), EINVAL, b"activation"),
                           (dict(bytes_=16), EINVAL, b"workspace")]:
        assert backward(**kw) == code and word in _message(), (kw, _message())
    room = lib.hess_gated_ffn_workspace(5, 24, 40, 0, 3) - lib.hess_gated_ffn_workspace(5, 24, 40, 0, 1)
    assert room >= 5 * 24 * 2


@built
def test_binding_refusals():
    x = torch.zeros(2, 8)
    rows = hs.Int8Rows(torch.zeros(2, 8, dtype=torch.int8), torch.zeros(2))
    for call in (lambda: hs.quantize_int8(x), lambda: hs.dequantize_int8(rows), lambda: hs.int8_matmul(rows, rows),
                 lambda: hs.int8_linear_forward(x, rows), lambda: hs.int8_linear(x, rows),
                 lambda: hs.int8_linear_backward(x, rows, rows)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match="constants"):
        hs.int8_linear(x, hs.Int8Rows(rows.codes, rows.scale.clone().requires_grad_()))
