"""Quantize a gated feed-forward block to 4 bits and repair it from a teacher's top logits.

The whole pass on one GPU, with synthetic activations and random weights:

 1. the unquantized block's Hessian is accumulated from the calibration batches;
 2. both projections are quantized with it (groups of 64, error propagated);
 3. the unquantized model's top logits are kept for every token, as a teacher run would store them;
 4. the dequantized weights are trained for a few steps on the distillation loss (masked tokens left out).

    python examples/repair_gated_block.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gptq_hessian_accumulation_amd as hs  # noqa: E402


def quantize(weight, batches):
    """4-bit weights (dequantized, float32) from the Hessian of the batches."""
    hessian = hs.Hessian(weight.shape[1], torch.bfloat16)
    for x in batches:
        hessian.add_batch(x)
    H, _, _ = hessian.materialize(0.01)
    hessian.close()
    return hs.gptq_quantize(weight, hs.chol_inverse_upper(H), group_size=64)[0]


def main(d=256, f=768, vocab=5000, top=32, tokens=1024, steps=60, lr=2e-3, seed=0):
    """Returns the mean loss of the quantized block before and after the repair."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    spread = torch.exp(0.5 * normal(d))
    batches = [(normal(n, d) * spread).bfloat16() for n in (tokens, tokens - 37, 211)]
    gate, up = normal(f, d) / d ** 0.5, normal(f, d) / d ** 0.5
    head = (normal(vocab, f) * 2 / f ** 0.5).bfloat16()

    def logits(x, w_gate, w_up):
        return hs.gated_ffn(x, w_gate, w_up, act="silu") @ head.t()

    # the teacher: top logits of the unquantized block, stored as a list of ids and values for each token
    x = batches[0]
    values, ids = logits(x, gate.bfloat16(), up.bfloat16()).float().topk(top, dim=-1)
    weight = (torch.rand(tokens, generator=gen, device="cuda") > 0.1).float() / tokens  # padding left out

    params = [quantize(w, batches).requires_grad_() for w in (gate, up)]
    optimizer = torch.optim.Adam(params, lr=lr)
    losses = []
    for _ in range(steps + 1):
        z = logits(x, params[0].bfloat16(), params[1].bfloat16())
        loss = hs.distill_topk(z, ids, values, weight=weight, temperature=2.0).sum()
        losses.append(loss.detach())
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
    before, after = float(losses[0]), float(losses[-1])
    print(f"distillation loss of the 4-bit block: {before:.5f}, after {steps} steps: {after:.5f}")
    return before, after


if __name__ == "__main__":
    main()
