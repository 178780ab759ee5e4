"""Score, sample and fine-tune through an int8 language-model head (synthetic data).

The head W [vocab][hidden] is quantized once to int8 rows.  Then, as a program would:

* a prompt's hidden states are multiplied by it and its tokens scored: log probability,
  entropy, the five likeliest alternatives;
* one token is decoded at a time from the alternatives of the last row;
* a low-rank adapter in front of the frozen head is trained on -log p with an entropy term:
  the gradient runs through the scores, the int8 head and the adapter.

    python examples/score_tokens.py [--tokens 512] [--hidden 2048] [--vocab 128256] [--steps 5]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import gemv_int4_quantize_amd as w4  # noqa: E402


class Adapter(torch.nn.Module):
    """x + x A B with a small inner width, B = 0 at the start."""

    def __init__(self, hidden: int, rank: int):
        super().__init__()
        self.a = torch.nn.Parameter(torch.randn(hidden, rank) * hidden ** -0.5)
        self.b = torch.nn.Parameter(torch.zeros(rank, hidden))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return x + ((x.float() @ self.a) @ self.b).to(x.dtype)


def score_prompt(head, x, tokens, top=5):
    """Scores of tokens [M] under the head's logits of hidden states x [M][hidden]."""
    with torch.no_grad():
        return w4.token_logprobs(head(x), tokens, top=top)


def decode(head, embed, x, count):
    """`count` greedy tokens, one row at a time: the likeliest token's embedding is the next state."""
    out = []
    with torch.no_grad():
        for _ in range(count):
            s = w4.token_logprobs(head(x), torch.zeros(1, dtype=torch.int64, device=x.device), top=1)
            out.append((s.top_ids[0, 0], s.top_logprobs[0, 0]))
            x = embed[s.top_ids[:, 0]]
    return [(int(i), float(p)) for i, p in out]


def train(head, adapter, x, tokens, steps, lr=1e-2, entropy_weight=0.01):
    """Steps of Adam on -log p(token) - entropy_weight * entropy; the losses."""
    opt = torch.optim.Adam(adapter.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        s = w4.token_logprobs(head(adapter(x)), tokens)
        loss = -(s.logprobs.mean() + entropy_weight * s.entropy.mean())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


def build(tokens, hidden, vocab, seed=0, device="cuda"):
    """A head, an adapter, an embedding, hidden states and the tokens to score."""
    g = torch.Generator().manual_seed(seed)
    weight = (torch.randn(vocab, hidden, generator=g) * hidden ** -0.5).to(torch.bfloat16).to(device)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16).to(device)
    t = torch.randint(vocab, (tokens,), generator=g).to(device)
    head = w4.W8A8Linear.from_weight(weight, out_dtype=torch.bfloat16)
    torch.manual_seed(seed)
    return head, Adapter(hidden, 16).to(device), weight, x, t


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--vocab", type=int, default=128256)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args()
    head, adapter, embed, x, t = build(a.tokens, a.hidden, a.vocab)
    s = score_prompt(head, x, t)
    print(f"prompt of {a.tokens} tokens: mean log p {s.logprobs.mean().item():.4f}, "
          f"mean entropy {s.entropy.mean().item():.4f}")
    print("first row's alternatives:", [(i, round(v, 3)) for i, v in zip(s.top_ids[0].tolist(), s.top_logprobs[0].tolist())])
    print("decoded:", [i for i, _ in decode(head, embed, x[-1:], 8)])
    print("losses:", [round(v, 4) for v in train(head, adapter, x, t, a.steps)])


if __name__ == "__main__":
    main()
