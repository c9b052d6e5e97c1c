"""Refusals of the feed-forward block and the distillation loss at the ends of what they promise; no GPU."""

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
