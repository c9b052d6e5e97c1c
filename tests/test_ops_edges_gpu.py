"""Rows and operands at the ends of what the distillation loss and the feed-forward block promise.

Tolerances are those of test_distill_gpu.py and test_gated_ffn_gpu.py, derived there.
"""

import numpy as np
import pytest
import torch

import gptq_hessian_accumulation_amd as hs
from tests import test_distill_gpu as D

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
