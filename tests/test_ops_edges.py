"""Refusals of the feed-forward block and the distillation loss at the ends of what they promise; no GPU."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch
import torch.autograd.forward_ad as fwd

import gptq_hessian_accumulation_amd as hs


@pytest.mark.parametrize("recording", [True, False])
def test_forward_mode_is_refused(recording):
    """A dual tensor carries its derivative without requiring a gradient: refused, never dropped."""
    x, w = torch.zeros(2, 8), torch.zeros(16, 8)
    z, ids, v, weight = torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3), torch.ones(2)

    def dual(t):
        return fwd.make_dual(t, torch.ones_like(t))

    with fwd.dual_level(), torch.set_grad_enabled(recording):
        for args in ((dual(x), w, w), (x, dual(w), w), (x, w, dual(w))):
            with pytest.raises(NotImplementedError, match="gated_ffn"):
                hs.gated_ffn(*args)
        for args in ((dual(z), ids, v, weight), (z, ids, dual(v), weight), (z, ids, v, dual(weight)),
                     (dual(z), ids, v)):
            with pytest.raises(NotImplementedError, match="distill_topk"):
                hs.distill_topk(*args)
        # inside a level, tensors that carry nothing pass on to the other checks
        with pytest.raises(ValueError, match="on the GPU"):
            hs.gated_ffn(x, w, w)
        with pytest.raises(ValueError, match="on the GPU"):
            hs.distill_topk(z, ids, v)


ROWS = r"""
#include <cstdio>
#include "distill_internal.hpp"
using namespace hess;
int main() {
  for (int threads : {128, 256, 512, 1024})
    for (int64_t parts : {1, 2, 3, 4097, 8193}) {
      const int64_t most = distill_rows_per_launch(threads, parts);
      if (most < 1 || most * parts * threads >= (int64_t)1 << 32) return 1;
      if ((most + 1) * parts * threads < (int64_t)1 << 32) return 2;
    }
  DistillParams P{};
  P.z = (void*)4096, P.ldz = 11, P.n = 10, P.ids = (void*)8192, P.ids64 = 1, P.ldi = 7;
  P.values = (void*)16384, P.values_dtype = 0, P.ldv = 5, P.loss = (float*)32768, P.stats = (float*)65536;
  const DistillParams Q = distill_rows(P, 2, 4, 4), T = distill_rows(P, 4, 8, 4);
  if (Q.n != 4 || T.n != 2 || Q.weight || Q.dz || Q.dloss) return 3;
  if (Q.z != (void*)(4096 + 4 * 11 * 2) || T.z != (void*)(4096 + 8 * 11 * 4)) return 4;
  if (Q.ids != (void*)(8192 + 4 * 7 * 8) || Q.values != (void*)(16384 + 4 * 5 * 2)) return 5;
  if (Q.loss != P.loss + 4 || Q.stats != P.stats + 8) return 6;
  P.ids64 = 0, P.values_dtype = 1;
  P.weight = (float*)1024, P.dloss = (float*)2048, P.dz = (void*)512, P.lddz = (int64_t)1 << 30;
  const DistillParams S = distill_rows(P, 4, 6, 100);
  if (S.n != 4 || S.ids != (void*)(8192 + 6 * 7 * 4) || S.values != (void*)(16384 + 6 * 5 * 4)) return 7;
  if (S.weight != P.weight + 6 || S.dloss != P.dloss + 6 || S.dz != (void*)(512 + ((int64_t)24 << 30))) return 8;
  return 0;
}
"""


host_compiler = pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include/hip"),
                                   reason="needs a host compiler and HIP's headers")


def run_host(tmp_path, source):
    """The exit code of a program over the library's internal headers, compiled for the host."""
    csrc = os.path.join(os.path.dirname(os.path.abspath(hs.__file__)), "csrc")
    (tmp_path / "host.cpp").write_text(source)
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", csrc,
                    str(tmp_path / "host.cpp"), "-o", str(tmp_path / "host")], check=True)
    return subprocess.run([str(tmp_path / "host")]).returncode


@host_compiler
def test_rows_of_a_launch(tmp_path):
    """A grid stays below 2^32 threads, and a range of rows moves every pointer by its own stride."""
    assert run_host(tmp_path, ROWS) == 0


@pytest.mark.parametrize("t", [1e-40, 1.4e-45, 2.0 ** -127, 0.0, -1.0, float("inf"), float("nan")])
def test_temperatures_without_a_reciprocal(t):
    """A subnormal temperature has no float32 reciprocal: refused, like those that are no temperature."""
    lib = hs._load()
    p = [ctypes.c_void_p((1 << 40) + (q << 36)) for q in range(8)]
    assert lib.hess_distill_topk(p[0], 100, 0, 4, 100, p[1], 0, 8, p[2], 1, 8, 8, p[3], t, p[4], p[5], p[6], 100, p[7],
                                 1 << 30, None) == -1
    assert b"temperature" in lib.hess_last_error()
    assert lib.hess_distill_topk_backward(p[4], p[0], 100, 0, 4, 100, p[1], 0, 8, p[2], 1, 8, 8, p[3], t, p[5], p[6],
                                          100, None) == -1
    assert b"temperature" in lib.hess_last_error()


# (element bytes, tokens, d, f, us of the few-token kernel, us of the tiles), weights in no cache
FEW_OR_TILES = [
    (2, 8, 1024, 2816, 5.8, 11.6), (2, 16, 2560, 2816, 11.0, 15.8), (2, 16, 4096, 11264, 40.7, 51.5),
    (2, 16, 8192, 4096, 34.8, 41.0), (2, 16, 8192, 16384, 116.3, 138.8), (2, 24, 2560, 2816, 14.5, 15.9),
    (2, 32, 2560, 2816, 15.2, 16.5), (2, 32, 2560, 5632, 19.3, 25.2), (2, 32, 2560, 9728, 34.6, 38.6),
    (2, 32, 4096, 5632, 25.9, 29.4), (2, 32, 4096, 11264, 50.2, 54.1), (2, 32, 5120, 13824, 70.1, 76.0),
    (2, 32, 8192, 2816, 40.3, 30.8), (2, 32, 8192, 1024, 37.7, 18.3), (2, 32, 8192, 11264, 105.7, 97.3),
    (2, 33, 1024, 2816, 7.9, 11.9), (2, 33, 2560, 2816, 14.8, 16.7), (2, 64, 1024, 2816, 9.1, 12.2),
    (2, 64, 2560, 4096, 18.9, 22.2), (2, 40, 2560, 4160, 26.2, 21.8), (2, 64, 2560, 5632, 32.3, 30.1),
    (2, 64, 4096, 5632, 47.4, 32.7), (2, 64, 4096, 2816, 25.6, 20.6), (2, 64, 8192, 1024, 45.7, 19.3),
    (2, 48, 4096, 11264, 62.7, 57.5), (2, 64, 4096, 11264, 69.9, 60.0), (2, 64, 1024, 8192, 15.0, 12.1),
    (4, 16, 2560, 2816, 19.1, 27.6), (4, 16, 4096, 11264, 86.2, 110.7), (4, 32, 1024, 2816, 12.7, 18.8),
    (4, 32, 2560, 2816, 25.0, 28.4), (4, 32, 4096, 11264, 117.7, 111.3), (4, 33, 2560, 2816, 39.8, 28.9),
    (4, 64, 2560, 4096, 43.0, 34.1), (4, 64, 4096, 2816, 64.2, 39.2), (4, 64, 4096, 11264, 151.6, 116.3)]


@host_compiler
def test_few_tokens_take_the_faster_kernel(tmp_path):
    """The rule's choice where one kernel was timed at least a twentieth ahead of the other."""
    cases = "".join(f"if (ffn_prefers_few({n}, {d}, {f}, {e}) != {int(few < tiles)}) return {i + 1};\n"
                    for i, (e, n, d, f, few, tiles) in enumerate(FEW_OR_TILES) if max(few, tiles) > 1.05 * min(few, tiles))
    assert run_host(tmp_path, '#include "ffn_internal.hpp"\nusing namespace hess;\nint main() {\n' + cases
                    + "return ffn_prefers_few(65, 8, 8, 2);\n}\n") == 0


def test_workspace_up_to_64_tokens():
    """Where tiles take the call, their partial sums need room; rows they would have to copy stay with the other kernel."""
    room = hs._load().hess_gated_ffn_workspace
    assert room(64, 1024, 2816, 0, 0) == 0 and room(16, 16384, 512, 0, 0) == 0
    assert room(64, 8192, 1024, 0, 0) > 0 and room(64, 8193, 1024, 0, 0) == 0


def test_forced_schedules():
    """The hook's checks, and the workspace of the schedule it sets."""
    lib = hs._load()
    for bad in ((32, 0, 1), (-64, 0, 1), (64, -1, 1), (64, 0, 0), (64, 0, 65)):
        assert lib.hess_set_ffn_schedule(*bad) == -1
    room = lib.hess_gated_ffn_workspace
    natural = [room(300, 456, 152, t, b) for t in range(3) for b in (0, 1)]
    try:
        # 300 x 152 features: 2 x 2 tiles of 256 x 128, 5 x 5 of 64 x 32; K of 456: 15 stages in 2 bytes, 29 in 4
        assert lib.hess_set_ffn_schedule(256, 0, 1) == 0 and room(300, 456, 152, 0, 0) == 0
        assert lib.hess_set_ffn_schedule(256, 0, 3) == 0 and room(300, 456, 152, 0, 0) == 4 * 3 * 256 * 256 * 4
        assert lib.hess_set_ffn_schedule(256, 1, 3) == 0 and room(300, 456, 152, 1, 0) == 3 * 3 * 256 * 256 * 4
        assert lib.hess_set_ffn_schedule(64, 20, 4) == 0 and room(300, 456, 152, 2, 0) == 5 * 4 * 64 * 64 * 4
        # no more parts than stages; every tile whole
        assert lib.hess_set_ffn_schedule(64, 0, 64) == 0 and room(300, 456, 152, 0, 0) == 25 * 15 * 64 * 64 * 4
        assert lib.hess_set_ffn_schedule(128, 99, 2) == 0 and room(300, 456, 152, 0, 0) == 0
    finally:
        assert lib.hess_set_ffn_schedule(0, 0, 1) == 0
    assert natural == [room(300, 456, 152, t, b) for t in range(3) for b in (0, 1)]
