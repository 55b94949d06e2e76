"""The operators around the LM head, together as a model uses them.

Training: the final norm with its residual in front of the fused cross-entropy,
forward and backward.  Serving: the same head in 8 bits; each decode step norms
the last layer's output straight into 8 bits, multiplies it with the 8-bit
weight, applies the requests' penalties, biases and grammar masks, and takes the
most likely token.

    python examples/lm_head_step.py [--hidden 1024] [--vocab 32000] [--steps 8]

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


def training_step(x, residual, norm_weight, head, labels):
    """Loss and gradients of norm -> LM head -> cross-entropy."""
    leaves = [t.detach().requires_grad_() for t in (x, residual, norm_weight, head)]
    y, _ = flce.rms_norm(leaves[0], leaves[2], residual=leaves[1])
    loss = flce.linear_cross_entropy(y, leaves[3], labels, shift=True)
    loss.backward()
    return loss.detach(), [t.grad for t in leaves]


class Head8bit:
    """The norm and LM head of a decode step, the weight quantised once."""

    def __init__(self, norm_weight, head):
        self.norm_weight = norm_weight
        self.weight, self.scale = flce.quantize_fp8(head)

    def logits(self, x, residual):
        """bf16 [B, V]; the residual stream is updated in place."""
        q, s, _ = flce.rms_norm_fp8(x, self.norm_weight, residual=residual,
                                    residual_out=residual)
        return flce.matmul_fp8(q, s, self.weight, self.scale)


def decode(head8, embedding, tokens, lengths, prompt_lengths, allowed, steps):
    """Greedy decoding with penalties; appends `steps` tokens to each row of
    `tokens` [B, L] (int64) and returns them [B, steps]."""
    B = tokens.shape[0]
    dev = tokens.device
    rep = torch.full((B,), 1.2, device=dev)
    freq = torch.full((B,), 0.1, device=dev)
    pres = torch.full((B,), 0.2, device=dev)
    rows = torch.arange(B, device=dev)
    residual = torch.zeros(B, embedding.shape[1], dtype=torch.bfloat16, device=dev)
    out = []
    for _ in range(steps):
        x = embedding[tokens[rows, lengths.long() - 1]]
        z = head8.logits(x, residual)
        z = flce.process_logits(z, tokens=tokens, lengths=lengths, prompt_lengths=prompt_lengths,
                                repetition_penalty=rep, frequency_penalty=freq,
                                presence_penalty=pres, allowed=allowed, out_dtype=torch.float32)
        picked = z.argmax(1)
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
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    norm_weight = 1 + rand(a.hidden, std=0.1)
    head, embedding = rand(a.vocab, a.hidden, std=0.02), rand(a.vocab, a.hidden)
    x, residual = rand(2, a.tokens, a.hidden), rand(2, a.tokens, a.hidden)
    labels = torch.randint(0, a.vocab, (2, a.tokens), generator=g, device="cuda")
    loss, grads = training_step(x, residual, norm_weight, head, labels)
    print(f"training: loss {loss.item():.4f}, gradient norms "
          + ", ".join(f"{n} {t.float().norm().item():.3e}"
                      for n, t in zip(("x", "residual", "norm", "head"), grads)))

    B, prompt = a.batch, 16
    tokens = torch.zeros(B, prompt + a.steps, dtype=torch.int64, device="cuda")
    tokens[:, :prompt] = torch.randint(0, a.vocab, (B, prompt), generator=g, device="cuda")
    lengths = torch.full((B,), prompt, dtype=torch.int32, device="cuda")
    allowed = torch.full((B, (a.vocab + 31) // 32), -1, dtype=torch.int32, device="cuda")
    allowed[0, 4:] = 0  # the first request's grammar: token ids below 128
    picked = decode(Head8bit(norm_weight, head), embedding, tokens, lengths, lengths.clone(),
                    allowed, a.steps)
    print("decoded:")
    for row in picked.tolist():
        print("  ", row)
    assert (picked[0] < 128).all() and loss.isfinite()


if __name__ == "__main__":
    main()
