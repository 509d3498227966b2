"""A small recurrent language model on libmsscan, trained and sampled.

    python examples/recurrent_lm.py [--steps 200]

Token embedding (`embed`), layers of a gated linear recurrence (`gated_scan`),
a head on the tied table, and the loss from `token_logprobs`, whose gradient
also takes the entropy (a small bonus on it keeps early predictions from
collapsing).  Documents are packed into rows and `reset` starts each anew.
Generation carries the recurrence's state token by token (`gated_step`) and
prints the model's alternatives at each place.

The data are made here: documents of the form "a+b=c" over two-digit numbers,
one byte a token.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_81_amd as ms  # noqa: E402

VOCAB, END = 128, 10  # bytes; a document ends with a line feed


class Block(torch.nn.Module):
    """x + out(recurrence(x, r, i, z)) with all four from one projection."""

    def __init__(self, width: int, inner: int):
        super().__init__()
        self.norm = torch.nn.RMSNorm(width)
        self.proj = torch.nn.Linear(width, 4 * inner)
        self.out = torch.nn.Linear(inner, width, bias=False)
        # decays of 0.9 to 0.999 at an open gate
        keep = torch.empty(inner).uniform_(0.9, 0.999)
        self.lam = torch.nn.Parameter(torch.log(torch.expm1(-torch.log(keep) / 8.0)))

    def parts(self, x):
        dt = torch.bfloat16
        return self.proj(self.norm(x)).to(dt).chunk(4, dim=-1)  # read where they are

    def forward(self, x, reset):
        u, r, i, z = self.parts(x)
        y = ms.gated_scan(u, r, i, self.lam, z, reset=reset)
        return x + self.out(y.to(x.dtype))

    def prefill(self, x):
        """The same for a prompt, with the state after it."""
        u, r, i, z = self.parts(x)
        y, h = ms.gated_scan(u, r, i, self.lam, z, return_last=True)
        return x + self.out(y.to(x.dtype)), h

    def step(self, x, h):
        """One token; h is updated in place."""
        u, r, i, z = self.parts(x)
        return x + self.out(ms.gated_step(h, u, r, i, self.lam, z).to(x.dtype))


class Model(torch.nn.Module):
    def __init__(self, width: int = 128, inner: int = 256, layers: int = 2):
        super().__init__()
        self.table = torch.nn.Parameter(torch.randn(VOCAB, width) / width ** 0.5)
        self.blocks = torch.nn.ModuleList(Block(width, inner) for _ in range(layers))
        self.norm = torch.nn.RMSNorm(width)

    def head(self, x):
        return (self.norm(x) @ self.table.t()).flatten(0, -2)  # [tokens, VOCAB]

    def forward(self, ids, reset=None):
        x = ms.embed(ids, self.table)  # scaled by sqrt(width)
        for b in self.blocks:
            x = b(x, reset)
        return self.head(x)

    @torch.no_grad()
    def generate(self, prompt, count: int, top: int = 3):
        """Greedy continuation of prompt [batch, length]: the tokens, their log
        probabilities, and the alternatives' tokens and log probabilities, each
        [batch, count(, top)]."""
        x, state = ms.embed(prompt, self.table), []
        for b in self.blocks:
            x, h = b.prefill(x)
            state.append(h)
        x = x[:, -1]
        out = []
        for _ in range(count):
            r = ms.token_logprobs_fwd(self.head(x), top=top)
            token = r["top_id"][:, 0].contiguous()
            out.append((token, r["top_logprob"][:, 0], r["top_id"], r["top_logprob"]))
            x = ms.embed(token, self.table)
            for b, h in zip(self.blocks, state):
                x = b.step(x, h)
        return [torch.stack(t, 1) for t in zip(*out)]


def documents(rng: torch.Generator, rows: int, length: int):
    """(tokens [rows, length + 1], reset [rows, length]) of packed documents."""
    tokens = torch.empty(rows, length + 1, dtype=torch.int64)
    for k in range(rows):
        text = ""
        while len(text) < length + 1:
            a, b = torch.randint(10, 100, (2,), generator=rng).tolist()
            text += f"{a}+{b}={a + b}\n"
        tokens[k] = torch.tensor(list(text[:length + 1].encode()))
    reset = torch.zeros(rows, length, dtype=torch.uint8)
    reset[:, 1:] = tokens[:, :length - 1] == END
    return tokens, reset


def loss_of(model: Model, tokens, reset, bonus: float = 0.0):
    """Mean negative log probability of the next token, less bonus * entropy."""
    logits = model(tokens[:, :-1].contiguous(), reset)
    logprob, entropy, _, _ = ms.token_logprobs(logits, tokens[:, 1:].reshape(-1))
    return -logprob.mean() - bonus * entropy.mean()


def train(model: Model, steps: int, rows: int = 64, length: int = 127, seed: int = 0, log=print):
    rng = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3, weight_decay=0.0)
    losses = []
    for k in range(steps):
        tokens, reset = (t.cuda() for t in documents(rng, rows, length))
        loss = loss_of(model, tokens, reset, bonus=0.01)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if log and (k % 50 == 0 or k == steps - 1):
            log(f"step {k:4d}  loss {loss.item():.3f}")
    return torch.stack(losses)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    torch.manual_seed(0)
    model = Model().cuda()
    train(model, args.steps)
    prompt = torch.tensor([list(b"21+34="), list(b"58+67=")], device="cuda")
    tokens, logp, ids, lps = (t.tolist() for t in model.generate(prompt, 4))
    for k, p in enumerate(prompt.tolist()):
        print(f"\n{bytes(p).decode()}{bytes(tokens[k]).decode().split(chr(END))[0]}"
              f"   log p {sum(logp[k]):.2f}")
        for at in range(len(tokens[k])):
            print("   ", "  ".join(f"{chr(i)!r} {v:6.2f}" for i, v in zip(ids[k][at], lps[k][at])))


if __name__ == "__main__":
    main()
