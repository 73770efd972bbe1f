"""A small recurrent language model on the library's model operators: tokens ->
embedding -> (short causal convolution -> selective scan) -> logits, trained
on a made-up sequence and then continued one token at a time.

    python examples/recurrent_lm.py

The matrix products are torch's; everything between is this library's, with
its own gradients where autograd asks for them. Training is bit-reproducible: the
operators sum in one fixed order, so two runs end with the same parameters.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scan_canonical_reduce_gb300 as cr  # noqa: E402


class RecurrentLM:
    """One layer; parameters in float32, as are the activations here."""

    def __init__(self, vocab, dim, dstate=16, width=4, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device)

        self.vocab, self.dim, self.dstate, self.width = vocab, dim, dstate, width
        self.scale = math.sqrt(dim)
        step = torch.exp(torch.rand(dim, generator=g) * math.log(100) + math.log(1e-3))
        n = torch.arange(1, dstate + 1, dtype=torch.float32)
        self.p = {
            "table": normal(vocab, dim, std=1 / self.scale),
            "in": normal(dim, 2 * dim, std=1 / math.sqrt(dim)),
            "conv_w": normal(dim, width, std=1 / math.sqrt(width)),
            "conv_b": torch.zeros(dim, device=device),
            "mix": normal(dim, dim + 2 * dstate, std=1 / math.sqrt(dim)),
            "log_A": torch.log(n).repeat(dim, 1).to(device),
            "D": torch.ones(dim, device=device),
            "dt_bias": (step + torch.log(-torch.expm1(-step))).to(device),
            "out": normal(dim, vocab, std=1 / math.sqrt(dim)),
        }
        for v in self.p.values():
            v.requires_grad_(True)

    def _mix(self, x):
        dt, B, C = (x @ self.p["mix"]).split([self.dim, self.dstate, self.dstate], -1)
        return dt, B, C

    def logits(self, tokens):
        """(batch, time) tokens to (batch, time, vocab) logits, with gradients."""
        p = self.p
        x = cr.embedding(tokens, p["table"], self.scale)
        x, z = (x @ p["in"]).chunk(2, -1)
        x = cr.causal_conv(x, p["conv_w"], p["conv_b"], "silu")
        dt, B, C = self._mix(x)
        y = cr.selective_scan(x, dt, -torch.exp(p["log_A"]), B, C, p["D"], z, p["dt_bias"])
        return y @ p["out"]

    @torch.no_grad()
    def prompt(self, tokens, lengths=None):
        """The logits of a prompt's positions and the state after it."""
        p = self.p
        x = cr.embedding(tokens, p["table"], self.scale)
        x, z = (x @ p["in"]).chunk(2, -1)
        x, conv = cr.causal_conv(x, p["conv_w"], p["conv_b"], "silu", lengths=lengths,
                                 return_state=True)
        dt, B, C = self._mix(x)
        y, scan = cr.selective_scan(x, dt, -torch.exp(p["log_A"]), B, C, p["D"], z, p["dt_bias"],
                                    lengths=lengths, return_state=True)
        return y @ p["out"], (conv, scan)

    @torch.no_grad()
    def step(self, tokens, state):
        """One token of each stream: (batch,) to (batch, vocab); updates state."""
        p, (conv, scan) = self.p, state
        x = cr.embedding(tokens, p["table"], self.scale)
        x, z = (x @ p["in"]).chunk(2, -1)
        x = cr.causal_conv_step(x, conv, p["conv_w"], p["conv_b"], "silu")
        dt, B, C = self._mix(x)
        y = cr.selective_scan_step(x, dt, -torch.exp(p["log_A"]), B, C, scan, p["D"], z,
                                   p["dt_bias"])
        return y @ p["out"]


def sequence(batch, length, vocab, seed, device="cuda"):
    """Tokens that follow from the two before them."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (batch, length), generator=g)
    for i in range(2, length):
        t[:, i] = (3 * t[:, i - 1] + 5 * t[:, i - 2] + 1) % vocab
    return t.to(device)


def train(model, steps, batch=16, length=64, rate=0.02, seed=1):
    """Adam by hand; returns the losses."""
    state = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in model.p.items()}
    losses = []
    for i in range(1, steps + 1):
        t = sequence(batch, length, model.vocab, seed + i)
        out = torch.log_softmax(model.logits(t[:, :-1]).float(), -1)
        loss = -out.gather(-1, t[:, 1:, None])[:, 2:].mean()
        loss.backward()
        with torch.no_grad():
            for k, v in model.p.items():
                m, s = state[k]
                m.lerp_(v.grad, 0.1)
                s.lerp_(v.grad.square(), 0.01)
                v -= rate * (m / (1 - 0.9 ** i)) / ((s / (1 - 0.99 ** i)).sqrt() + 1e-8)
                v.grad = None
        losses.append(loss.detach())
    return torch.stack(losses)


def generate(model, tokens, count):
    """Continues (batch, time) tokens greedily, one step at a time."""
    logits, state = model.prompt(tokens)
    out = [logits[:, -1].argmax(-1)]
    for _ in range(count - 1):
        out.append(model.step(out[-1], state).argmax(-1))
    return torch.stack(out, 1)


def main():
    torch.backends.cuda.matmul.allow_tf32 = False
    model = RecurrentLM(vocab=31, dim=128)
    losses = train(model, 150).tolist()
    print("loss: %.3f at the start, %.3f at the end" % (losses[0], losses[-1]))
    t = sequence(4, 40, model.vocab, 99)
    got = generate(model, t[:, :24], 16)
    right = (got == t[:, 24:]).float().mean().item()
    print("continued 4 sequences by 16 tokens: %.0f %% right" % (100 * right))
    return losses, right


if __name__ == "__main__":
    main()
