"""Refusals of the feed-forward block and the distillation loss that need no GPU: the C ABI's argument
checks (fake addresses, never dereferenced) and the binding's."""

import ctypes
import os

import pytest
import torch

import gptq_hessian_accumulation_amd as hs

pytestmark = pytest.mark.skipif(not os.path.exists(hs.library_path()), reason="libhess.so not built")

EINVAL, EALIGN = -1, -5
GB = 1 << 30
BASE = 1 << 40


def _ptr(i, off=0):
    return ctypes.c_void_p(BASE + i * 64 * GB + off)


def _forward(n=5, d=24, f=40, dtype=0, act=0, ld=(24, 24, 24, 40), ptrs=None, pre=_ptr(4), work=_ptr(5), bytes_=GB):
    lib = hs._load()
    p = ptrs or [_ptr(i) for i in range(4)]
    return lib.hess_gated_ffn_forward(p[0], ld[0], p[1], ld[1], p[2], ld[2], dtype, act, n, d, f, p[3], ld[3], pre,
                                      work, bytes_, None)


def _message():
    return hs._load().hess_last_error()


def test_ffn_forward_refusals():
    assert _forward(n=0) == 0
    for kw, code, word in [
            (dict(dtype=3), EINVAL, b"dtype"), (dict(act=3), EINVAL, b"activation"), (dict(act=-1), EINVAL, b"act"),
            (dict(n=-1), EINVAL, b"n = "), (dict(n=(1 << 24) + 1), EINVAL, b"n = "), (dict(d=0), EINVAL, b"d = "),
            (dict(f=0), EINVAL, b"f = "), (dict(f=(1 << 17) + 1), EINVAL, b"f = "),
            (dict(ld=(23, 24, 24, 40)), EINVAL, b"of x"), (dict(ld=(24, 23, 24, 40)), EINVAL, b"of w_gate"),
            (dict(ld=(24, 24, 23, 40)), EINVAL, b"of w_up"), (dict(ld=(24, 24, 24, 39)), EINVAL, b"of h"),
            (dict(ld=((1 << 20) + 1, 24, 24, 40)), EINVAL, b"of x"),
            (dict(ptrs=[None, _ptr(1), _ptr(2), _ptr(3)]), EINVAL, b"null x"),
            (dict(ptrs=[_ptr(0), _ptr(1), _ptr(2), None]), EINVAL, b"null h"),
            (dict(ptrs=[_ptr(0, 1), _ptr(1), _ptr(2), _ptr(3)]), EALIGN, b"x not aligned"),
            (dict(ptrs=[_ptr(0, 2), _ptr(1), _ptr(2), _ptr(3)], dtype=1), EALIGN, b"x not aligned"),
            (dict(pre=_ptr(4, 8)), EALIGN, b"preact"),
            (dict(ptrs=[_ptr(0), _ptr(1), _ptr(2), _ptr(0, 64)]), EINVAL, b"h overlaps x"),
            (dict(pre=_ptr(3, 64)), EINVAL, b"h overlaps preact"), (dict(pre=_ptr(1)), EINVAL, b"preact overlaps")]:
        assert _forward(**kw) == code and word in _message(), (kw, _message())


def test_ffn_workspace_rule():
    lib = hs._load()
    assert lib.hess_gated_ffn_workspace(0, 8, 8, 0, 0) == 0 and lib.hess_gated_ffn_workspace(0, 8, 8, 0, 1) == 0
    assert lib.hess_gated_ffn_workspace(-1, 8, 8, 0, 0) == -1 and lib.hess_gated_ffn_workspace(1, 8, 8, 5, 0) == -1
    assert lib.hess_gated_ffn_preact_cols(0) == -1
    assert lib.hess_gated_ffn_preact_cols(1) == 16 and lib.hess_gated_ffn_preact_cols(16) == 32
    # a long K over few tiles is split: partial tiles need room
    need = lib.hess_gated_ffn_workspace(100, 8192, 64, 0, 0)
    assert need > 0
    kw = dict(n=100, d=8192, f=64, ld=(8192, 8192, 8192, 64))
    assert _forward(bytes_=need - 1, **kw) == EINVAL and b"workspace" in _message()
    assert _forward(work=None, **kw) == EINVAL and b"workspace" in _message()
    assert _forward(work=_ptr(5, 8), **kw) == EALIGN
    assert _forward(work=_ptr(0), **kw) == EINVAL and b"overlaps the workspace" in _message()


def _backward(n=5, dx=_ptr(5), dwg=_ptr(6), dwu=_ptr(7), ldw=24, pre=_ptr(4), dtype=0, act=0, bytes_=GB,
              work=_ptr(8), dh=_ptr(0), lddh=40):
    return hs._load().hess_gated_ffn_backward(dh, lddh, _ptr(1), 24, _ptr(2), 24, _ptr(3), 24, pre, dtype, act, n, 24,
                                              40, dx, 24, dwg, ldw, dwu, ldw, work, bytes_, None)


def test_ffn_backward_refusals():
    assert _backward(dx=None, dwg=None, dwu=None) == 0  # nothing wanted, nothing launched
    for kw, code, word in [
            (dict(dwg=None), EINVAL, b"both or neither"), (dict(dwu=None), EINVAL, b"both or neither"),
            (dict(pre=None), EINVAL, b"null preact"), (dict(pre=_ptr(4, 2)), EALIGN, b"preact"),
            (dict(ldw=23), EINVAL, b"dw_gate"), (dict(act=7), EINVAL, b"activation"), (dict(dtype=-1), EINVAL, b"dtype"),
            (dict(dh=None), EINVAL, b"null dh"), (dict(lddh=39), EINVAL, b"of dh"),
            (dict(dwu=_ptr(6, 64)), EINVAL, b"dw_gate overlaps dw_up"), (dict(dx=_ptr(1)), EINVAL, b"dx overlaps x"),
            (dict(dx=_ptr(0)), EINVAL, b"dx overlaps dh"), (dict(dwg=_ptr(2)), EINVAL, b"dw_gate overlaps w_gate"),
            (dict(bytes_=16), EINVAL, b"workspace"), (dict(work=_ptr(1)), EINVAL, b"overlaps the workspace")]:
        assert _backward(**kw) == code and word in _message(), (kw, _message())


def _distill(n=4, vocab=100, k=8, dtype=0, vdtype=1, t=1.0, ldz=100, ldi=8, ldv=8, lddz=100, z=_ptr(0), ids=_ptr(1),
             vals=_ptr(2), w=_ptr(3), loss=_ptr(4), stats=_ptr(5), dz=_ptr(6), work=_ptr(7), ids64=0):
    return hs._load().hess_distill_topk(z, ldz, dtype, n, vocab, ids, ids64, ldi, vals, vdtype, ldv, k, w, t, loss, stats,
                                        dz, lddz, work, GB, None)


def _distill_back(n=4, dloss=_ptr(4), stats=_ptr(5), dz=_ptr(6), lddz=100):
    return hs._load().hess_distill_topk_backward(dloss, _ptr(0), 100, 0, n, 100, _ptr(1), 0, 8, _ptr(2), 1, 8, 8,
                                                 _ptr(3), 1.0, stats, dz, lddz, None)


def test_distill_refusals():
    assert _distill(n=0) == 0 and _distill_back(n=0) == 0
    for kw, code, word in [
            (dict(dtype=9), EINVAL, b"dtype"), (dict(vdtype=9), EINVAL, b"dtype"), (dict(n=-2), EINVAL, b"n = "),
            (dict(vocab=0), EINVAL, b"vocab"), (dict(vocab=(1 << 28) + 1), EINVAL, b"vocab"), (dict(k=0), EINVAL, b"k = "),
            (dict(k=1025, ldi=1025, ldv=1025), EINVAL, b"k = "), (dict(t=0.0), EINVAL, b"temperature"),
            (dict(t=-1.0), EINVAL, b"temperature"), (dict(t=float("inf")), EINVAL, b"temperature"),
            (dict(t=float("nan")), EINVAL, b"temperature"), (dict(z=None), EINVAL, b"null"),
            (dict(ids=None), EINVAL, b"null"), (dict(vals=None), EINVAL, b"null"), (dict(loss=None), EINVAL, b"loss"),
            (dict(ldz=99), EINVAL, b"stride"), (dict(ldi=7), EINVAL, b"stride"), (dict(ldv=7), EINVAL, b"stride"),
            (dict(lddz=99), EINVAL, b"stride"), (dict(z=_ptr(0, 1)), EALIGN, b"aligned"),
            (dict(ids=_ptr(1, 4), ids64=1), EALIGN, b"aligned"), (dict(w=_ptr(3, 2)), EALIGN, b"weight"),
            (dict(stats=_ptr(5, 2)), EALIGN, b"stats"), (dict(dz=_ptr(6, 1)), EALIGN, b"dlogits"),
            (dict(dz=_ptr(0, 2)), EINVAL, b"dlogits overlaps logits"),
            (dict(dz=_ptr(0), lddz=101), EINVAL, b"dlogits overlaps logits"),
            (dict(dz=_ptr(1)), EINVAL, b"dlogits overlaps ids"), (dict(loss=_ptr(3)), EINVAL, b"loss overlaps weight"),
            (dict(stats=_ptr(6)), EINVAL, b"dlogits overlaps stats"), (dict(stats=_ptr(4)), EINVAL, b"overlaps loss")]:
        assert _distill(**kw) == code and word in _message(), (kw, _message())
    for kw, word in [(dict(dloss=None), b"null"), (dict(stats=None), b"null"), (dict(dz=None), b"null"),
                     (dict(dz=_ptr(5)), b"overlaps stats"), (dict(dz=_ptr(3)), b"overlaps weight"),
                     (dict(lddz=50), b"stride")]:
        assert _distill_back(**kw) == EINVAL and word in _message(), (kw, _message())
    assert hs._load().hess_distill_topk_workspace(-1, 5, 0) == -1
    assert hs._load().hess_distill_topk_workspace(1, 5, 4) == -1


def test_binding_refuses_host_tensors_and_unknown_names():
    x, w = torch.zeros(2, 8), torch.zeros(16, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        hs.gated_ffn_forward(x, w, w)
    with pytest.raises(ValueError, match="activation"):
        hs.gated_ffn_forward(x, w, w, act="relu")
    z, ids, v = torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="on the GPU"):
        hs.distill_topk_forward(z, ids, v)
    with pytest.raises(ValueError, match="constants"):
        hs.distill_topk(z, ids, v.requires_grad_())


def test_ffn_refuses_rows_off_16_bytes():
    """More tokens than the kernel that takes any alignment: the C entry refuses, the binding copies."""
    for dtype, off in ((0, 2), (1, 4), (2, 8)):
        for p in range(3):
            ptrs = [_ptr(i, off if i == p else 0) for i in range(4)]
            assert _forward(n=100, dtype=dtype, ptrs=ptrs) == EALIGN and b"16-byte" in _message()
    assert _forward(n=100, ld=(25, 24, 24, 40)) == EALIGN
    assert _forward(n=100, ld=(24, 28, 24, 40)) == EALIGN
    assert hs._load().hess_gated_ffn_workspace(5, 24, 40, 0, 0) == 0
    # rows that are copied need room for x and both weights
    room = hs._load().hess_gated_ffn_workspace(100, 25, 40, 0, 0) - hs._load().hess_gated_ffn_workspace(100, 32, 40, 0, 0)
    assert room >= 2 * 32 * (100 + 2 * 40)


def test_ffn_float32_pair_flag():
    """HESS_PREACT_F32 (16) doubles what the pair spans; activations past it stay unknown."""
    assert _forward(act=16 + 3) == EINVAL and b"activation" in _message()
    assert _forward(act=32) == EINVAL and b"activation" in _message()
    # bf16 pair of 5 rows of 80: 800 bytes; h right behind it meets the float32 one
    ptrs = [_ptr(0), _ptr(1), _ptr(2), _ptr(4, 800)]
    assert _forward(act=16, ptrs=ptrs) == EINVAL and b"h overlaps preact" in _message()
