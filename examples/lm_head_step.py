"""The operators around the LM head, together as a model uses them.

Training: the final norm (an RMS norm, or a layer norm) with its residual in front of
the fused cross-entropy, forward and backward.  Serving: the same head in 8 bits; each
decode step norms the last layer's output straight into 8 bits, multiplies it with
the 8-bit weight, applies the requests' penalties, biases and grammar masks, and samples
a token: the first request takes the most likely one, the others by temperature, top-k,
top-p and min-p.

    python examples/lm_head_step.py [--hidden 1024] [--vocab 32000] [--steps 8]
                                    [--layer-norm] [--temperature 0.8]

Needs a GB300 and the built library.  There is no model under the head here: the
hidden states are random, and a decode step's are made from the embedding of the
token that was picked.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import lm_head_linear_flce_gb300 as flce  # noqa: E402


def training_step(x, residual, norm_weight, head, labels, norm_bias=None):
    """Loss and gradients of norm -> LM head -> cross-entropy; a layer norm where there is
    a bias."""
    leaves = [t.detach().requires_grad_() for t in (x, residual, norm_weight, head)]
    if norm_bias is None:
        y, _ = flce.rms_norm(leaves[0], leaves[2], residual=leaves[1])
    else:
        leaves.append(norm_bias.detach().requires_grad_())
        y, _ = flce.layer_norm(leaves[0], leaves[2], leaves[4], residual=leaves[1])
    loss = flce.linear_cross_entropy(y, leaves[3], labels, shift=True)
    loss.backward()
    return loss.detach(), [t.grad for t in leaves]


class Head8bit:
    """The norm and LM head of a decode step, the weight quantised once."""

    def __init__(self, norm_weight, head, norm_bias=None):
        self.norm_weight, self.norm_bias = norm_weight, norm_bias
        self.weight, self.scale = flce.quantize_fp8(head)

    def logits(self, x, residual):
        """bf16 [B, V]; the residual stream is updated in place."""
        if self.norm_bias is None:
            q, s, _ = flce.rms_norm_fp8(x, self.norm_weight, residual=residual,
                                        residual_out=residual)
        else:
            q, s, _ = flce.layer_norm_fp8(x, self.norm_weight, self.norm_bias,
                                          residual=residual, residual_out=residual)
        return flce.matmul_fp8(q, s, self.weight, self.scale)


def decode(head8, embedding, tokens, lengths, prompt_lengths, allowed, steps, temperature):
    """Sampling with penalties; appends `steps` tokens to each row of `tokens` [B, L]
    (int64) and returns them [B, steps].  temperature: float32 [B], 0 for greedy."""
    B = tokens.shape[0]
    dev = tokens.device
    rep = torch.full((B,), 1.2, device=dev)
    freq = torch.full((B,), 0.1, device=dev)
    pres = torch.full((B,), 0.2, device=dev)
    limits = dict(temperature=temperature, top_p=torch.full((B,), 0.95, device=dev),
                  top_k=torch.full((B,), 50, dtype=torch.int32, device=dev),
                  min_p=torch.full((B,), 0.02, device=dev))
    g = torch.Generator(device=dev).manual_seed(1)
    rows = torch.arange(B, device=dev)
    residual = torch.zeros(B, embedding.shape[1], dtype=torch.bfloat16, device=dev)
    out = []
    for _ in range(steps):
        x = embedding[tokens[rows, lengths.long() - 1]]
        z = head8.logits(x, residual)
        z = flce.process_logits(z, tokens=tokens, lengths=lengths, prompt_lengths=prompt_lengths,
                                repetition_penalty=rep, frequency_penalty=freq,
                                presence_penalty=pres, allowed=allowed, out_dtype=torch.float32)
        picked = flce.sample_logits(z, torch.rand(B, generator=g, device=dev), **limits)
        tokens[rows, lengths.long()] = picked
        lengths += 1
        out.append(picked)
    return torch.stack(out, 1)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--vocab", type=int, default=32000)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--tokens", type=int, default=512, help="training tokens per sequence")
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--layer-norm", action="store_true", help="instead of an RMS norm")
    p.add_argument("--temperature", type=float, default=0.8, help="of all but the first request")
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    norm_weight = 1 + rand(a.hidden, std=0.1)
    norm_bias = rand(a.hidden, std=0.1) if a.layer_norm else None
    head, embedding = rand(a.vocab, a.hidden, std=0.02), rand(a.vocab, a.hidden)
    x, residual = rand(2, a.tokens, a.hidden), rand(2, a.tokens, a.hidden)
    labels = torch.randint(0, a.vocab, (2, a.tokens), generator=g, device="cuda")
    loss, grads = training_step(x, residual, norm_weight, head, labels, norm_bias)
    print(f"training: loss {loss.item():.4f}, gradient norms "
          + ", ".join(f"{n} {t.float().norm().item():.3e}"
                      for n, t in zip(("x", "residual", "norm", "head", "bias"), grads)))

    B, prompt = a.batch, 16
    tokens = torch.zeros(B, prompt + a.steps, dtype=torch.int64, device="cuda")
    tokens[:, :prompt] = torch.randint(0, a.vocab, (B, prompt), generator=g, device="cuda")
    lengths = torch.full((B,), prompt, dtype=torch.int32, device="cuda")
    allowed = torch.full((B, (a.vocab + 31) // 32), -1, dtype=torch.int32, device="cuda")
    allowed[0, 4:] = 0  # the first request's grammar: token ids below 128
    temperature = torch.full((B,), a.temperature, device="cuda")
    temperature[0] = 0
    picked = decode(Head8bit(norm_weight, head, norm_bias), embedding, tokens, lengths,
                    lengths.clone(), allowed, a.steps, temperature)
    print("decoded:")
    for row in picked.tolist():
        print("  ", row)
    assert (picked[0] < 128).all() and loss.isfinite()


if __name__ == "__main__":
    main()
