"""Limits of the 8-bit calls without a GPU: what is refused before anything runs, workspaces, the import."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import gptq_hessian_accumulation_amd as hs

pytestmark = pytest.mark.skipif(not os.path.exists(hs.library_path()), reason="libhess.so not built")
EINVAL = -1
GB = 1 << 30


def _ptr(i, off=0):
    return ctypes.c_void_p((1 << 40) + i * 64 * GB + off)


def _message():
    return hs._load().hess_last_error()


# (weights of 24 rows of d codes, ld bytes apart, whose pieces of 16 bytes the tiles read whole)
@pytest.mark.parametrize("d,ld", [(40, 48), (33, 64)])
@pytest.mark.parametrize("where", ["first", "last"])
def test_outputs_behind_the_last_row_of_weights(d, ld, where):
    """The bytes between the last row's codes and the end of their 16-byte piece are read: no output may lie there."""
    lib, n, f = hs._load(), 100, 24
    end = (f - 1) * ld
    y = _ptr(2, end + (-(-d // 4) * 4 if where == "first" else -(-d // 16) * 16 - 4))
    assert lib.hess_int8_matmul(_ptr(0), 64, _ptr(1), _ptr(2), ld, _ptr(3), n, d, f, y, f, 0, _ptr(5), GB, None) == EINVAL
    assert b"y overlaps b" in _message()
    assert lib.hess_int8_linear_forward(_ptr(0), d, 0, _ptr(2), ld, _ptr(3), n, d, f, y, f, None, 0, None, _ptr(5), GB,
                                        None) == EINVAL
    assert b"y overlaps w" in _message()
    assert lib.hess_int8_linear_forward(_ptr(0), d, 0, _ptr(2), ld, _ptr(3), n, d, f, _ptr(4), f, _ptr(6), 64, y, _ptr(5),
                                        GB, None) == EINVAL
    assert b"x_scale overlaps w" in _message()


@pytest.mark.parametrize("n,d,f", [(1, 64, 64), (5, 25, 40), (70, 333, 1000), (300, 704, 1000), (8192, 4096, 11264)])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_ffn_workspace_for_any_backward(n, d, f, dtype):
    """Every value but 0 asks for the backward pass's room; what a forward call with the pair in 8 bits needs has a
    function of its own, and 2 gives enough for either."""
    lib = hs._load()
    need = lib.hess_gated_ffn_workspace(n, d, f, dtype, 1)
    assert need >= n * 2 * f * (4 if dtype == 1 else 2)
    forward = lib.hess_gated_ffn_i8_workspace(n, d, f, dtype)
    assert forward >= 0
    for backward in (-1, 2, 3, 4, 64, 255):
        assert lib.hess_gated_ffn_workspace(n, d, f, dtype, backward) >= need
    assert lib.hess_gated_ffn_workspace(n, d, f, dtype, 2) >= forward
    assert lib.hess_gated_ffn_i8_workspace(0, d, f, dtype) == 0
    assert lib.hess_gated_ffn_i8_workspace(-1, d, f, dtype) == -1 and lib.hess_gated_ffn_i8_workspace(n, d, f, 7) == -1


def test_import_without_the_type_of_exponents():
    """A torch without float8_e8m0fnu: the package imports, and only blocks of 32 columns are refused."""
    code = """
import torch
del torch.float8_e8m0fnu
import gptq_hessian_accumulation_amd as hs
x = torch.zeros(2, 32)
for call, error, word in ((lambda: hs.quantize_int8(x, block=32), RuntimeError, "float8_e8m0fnu"),
                          (lambda: hs.quantize_int8(x, block=16), ValueError, "0 or 32"),
                          (lambda: hs.quantize_int8(x), ValueError, "on the GPU"),
                          (lambda: hs.gated_ffn_forward(x, x, x), ValueError, "on the GPU")):
    try:
        call()
    except error as e:
        assert word in str(e), e
    else:
        raise AssertionError(word)
print("imported")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(hs.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr


@pytest.mark.parametrize("n,d,f", [(100, 33, 24), (777, 1001, 2731), (1999, 2561, 9728), (16384, 4097, 11264)])
def test_linear_workspace_has_no_room_for_copies_never_made(n, d, f):
    """Codes of x go to padded rows as they are: the layer's room is what the product of given codes needs less the
    copy of its left operand, plus the codes and scales where the caller keeps none."""
    lib = hs._load()
    pad = -(-d // 16) * 16

    def up(v):
        return -(-v // 256) * 256

    product = lib.hess_int8_matmul_workspace(n, d, f)
    kept = lib.hess_int8_linear_workspace(n, d, f, 0, 4)
    assert kept == product - up(n * pad) and kept >= f * pad
    assert lib.hess_int8_linear_workspace(n, d, f, 0, 0) == kept + up(n * pad) + up(4 * n)
