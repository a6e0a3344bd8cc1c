"""A small language model around the matrix-state scan, trained and then served:

    embed (rows of a table for the token, of another for its predecessor, scaled)
    blocks: x + mix(norm(x)),  x + down(gated_projection(norm(x)))
    linear_cross_entropy over the vocabulary, against the embedding's own table

    python examples/language_model.py [--steps 100]

trains it on packed sequences that repeat cycles of tokens, then reads packed
prompts into pools of states, one a layer, and generates token by token.  The
mixing layer is that of mixing_layer.py.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import gated_linear_recurrence_history_amd as gs  # noqa: E402
from mixing_layer import MixingLayer, pack, predecessors, recall_batch  # noqa: E402


class FeedForward(torch.nn.Module):
    """down(silu(gate(x)) * up(x)); both projections and their product in one kernel."""

    def __init__(self, width, inner, device="cuda"):
        super().__init__()
        self.gate = torch.nn.Parameter(torch.randn(inner, width, device=device) * width ** -0.5)
        self.up = torch.nn.Parameter(torch.randn(inner, width, device=device) * width ** -0.5)
        self.down = torch.nn.Linear(inner, width, bias=False, device=device)

    def forward(self, x):
        # (the parameters stay float32: their gradients come back through the casts)
        return self.down(gs.gated_projection(x, self.gate.to(x.dtype), self.up.to(x.dtype)))


class Block(torch.nn.Module):
    def __init__(self, width, inner, **kw):
        super().__init__()
        self.norms = torch.nn.ModuleList(torch.nn.RMSNorm(width, device="cuda") for _ in range(2))
        self.mix, self.feed = MixingLayer(width, **kw), FeedForward(width, inner)

    def forward(self, x, positions, seq_offsets, state=None):
        y, state = self.mix(self.norms[0](x.float()).to(x.dtype), positions, seq_offsets, state)
        x = x + y
        return x + self.feed(self.norms[1](x.float()).to(x.dtype)), state

    @torch.no_grad()
    def step(self, x, positions, pool, slots):
        x = x + self.mix.step(self.norms[0](x.float()).to(x.dtype), positions, pool, slots)
        return x + self.feed(self.norms[1](x.float()).to(x.dtype))


class LanguageModel(torch.nn.Module):
    """Activations in `dtype`, parameters float32; the output weights are the table."""

    def __init__(self, vocabulary=64, width=256, inner=512, layers=2, dtype=torch.bfloat16, **kw):
        super().__init__()
        self.table, self.before = (torch.nn.Parameter(torch.randn(vocabulary, width, device="cuda") * width ** -0.5)
                                   for _ in range(2))
        self.blocks = torch.nn.ModuleList(Block(width, inner, **kw) for _ in range(layers))
        self.norm = torch.nn.RMSNorm(width, device="cuda")
        self.dtype, self.scale = dtype, width ** 0.5

    def _embed(self, tokens, before):
        return gs.embed(self.table, tokens, scale=self.scale, dtype=self.dtype) + \
            gs.embed(self.before, before, scale=self.scale, dtype=self.dtype)

    def forward(self, tokens, positions, seq_offsets):
        """Packed tokens -> (last hidden states, every layer's states)."""
        x, states = self._embed(tokens, predecessors(tokens, positions)), []
        with torch.autocast("cuda", self.dtype, enabled=self.dtype == torch.bfloat16):
            for block in self.blocks:
                x, state = block(x, positions, seq_offsets)
                states.append(state)
        return self.norm(x.float()).to(self.dtype), states

    def loss(self, tokens, target, positions, seq_offsets):
        """Mean over the targets in the vocabulary, without the logits in memory."""
        h, _ = self(tokens, positions, seq_offsets)
        return gs.linear_cross_entropy(h, self.table.to(h.dtype), target)

    @torch.no_grad()
    def logits(self, h):
        return h.float() @ self.table.T

    @torch.no_grad()
    def step(self, tokens, before, positions, pools, slots):
        """One token of each request -> logits; the pools' states are updated."""
        x = self._embed(tokens, before)
        with torch.autocast("cuda", self.dtype, enabled=self.dtype == torch.bfloat16):
            for block, pool in zip(self.blocks, pools):
                x = block.step(x, positions, pool, slots)
        return self.logits(self.norm(x.float()).to(self.dtype))


def train(model, steps, gen, lengths=(96, 160, 64, 192, 130, 77) * 12, vocabulary=64, rate=2e-3):
    """Losses of the steps.  The first 16 tokens of a sequence (its cycle, which cannot be
    known) do not count."""
    offsets, positions = pack(lengths)
    last = (offsets[1:] - 1).long()
    optimizer = torch.optim.AdamW(model.parameters(), lr=rate)
    losses = []
    for _ in range(steps):
        tokens = recall_batch(gen, lengths, vocabulary)
        target = torch.roll(tokens, -1)
        target[last] = -100
        target[positions < 15] = -100
        loss = model.loss(tokens, target, positions, offsets)
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def generate(model, prompts, count, pool_size):
    """Greedy continuations [requests, count] of packed prompts."""
    lengths = [len(p) for p in prompts]
    offsets, positions = pack(lengths)
    h, states = model(torch.cat(prompts).cuda(), positions, offsets)
    slots = torch.randperm(pool_size)[:len(prompts)].to(torch.int32).cuda()
    pools = []
    for state in states:
        pools.append(state.new_zeros(pool_size, *state.shape[1:]))
        pools[-1][slots.long()] = state
    before = torch.stack([p[-1] for p in prompts]).cuda()
    token = model.logits(h[(offsets[1:] - 1).long()]).argmax(-1)
    position, made = torch.tensor(lengths).cuda(), [token]
    for _ in range(count - 1):
        before, token = token, model.step(token, before, position, pools, slots).argmax(-1)
        position = position + 1
        made.append(token)
    return torch.stack(made, 1)


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=100)
    args = parser.parse_args()
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(1)
    model = LanguageModel()
    start = time.time()
    losses = train(model, args.steps, gen)
    print(f"{args.steps} steps in {time.time() - start:.1f} s: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    prompts = [recall_batch(gen, [n], 64, "cpu") for n in (40, 33, 70, 51)]
    made = generate(model, prompts, 32, pool_size=16).cpu()
    want = torch.stack([p[:16].repeat(8)[len(p):len(p) + 32] for p in prompts])
    print(f"32 tokens of {len(prompts)} requests generated: {(made == want).float().mean():.3f} continue their cycle")


if __name__ == "__main__":
    main()
