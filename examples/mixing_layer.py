"""A sequence-mixing layer over the matrix-state scan, trained and then served:

    x -> one projection -> q, k, v, gate
    q, k -> qk_norm_rope (RMS norm per head, rotation by position)
    state_scan (training, prompts) or state_scan_step (one token per request)
    -> output projection

    python examples/mixing_layer.py [--steps 60]

trains one layer on a synthetic task (say again the token that followed this
one's last occurrence), then reads packed prompts of several requests into a
pool of states and generates token by token from them.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_linear_recurrence_history_amd as gs  # noqa: E402


class MixingLayer(torch.nn.Module):
    """heads states of key_width x value_width; queries and keys have key_heads
    heads, shared by groups of heads.  Under torch.autocast the projection's
    output, and with it the scan, is bfloat16; states stay float32."""

    def __init__(self, width, heads=8, key_heads=4, key_width=64, value_width=64, device="cuda",
                 dtype=torch.float32):
        super().__init__()
        self.shape = (heads, key_heads, key_width, value_width)
        self.parts = [key_heads * key_width, key_heads * key_width, heads * value_width, heads]
        self.proj = torch.nn.Linear(width, sum(self.parts), bias=False, device=device, dtype=dtype)
        self.out = torch.nn.Linear(heads * value_width, width, bias=False, device=device, dtype=dtype)
        self.q_weight = torch.nn.Parameter(torch.ones(key_width, device=device))
        self.k_weight = torch.nn.Parameter(torch.ones(key_width, device=device))
        freq, self.magnitude = gs.rotary_frequencies(key_width // 2, device=device)
        self.register_buffer("freq", freq)

    def _operands(self, x, positions):
        """x [tokens, width] -> q, k (normed, rotated), v, gate: the latter two
        are slices of the projection's output, read in place (copied where its
        rows, gates included, are no multiple of 16 bytes)."""
        heads, key_heads, dk, dv = self.shape
        q, k, v, gate = self.proj(x).split(self.parts, dim=-1)
        q, k = gs.qk_norm_rope(q.unflatten(-1, (key_heads, dk)), k.unflatten(-1, (key_heads, dk)),
                               self.q_weight, self.k_weight, positions, self.freq,
                               magnitude=self.magnitude)
        return q, k, v.unflatten(-1, (heads, dv)), gate

    def forward(self, x, positions, seq_offsets, state=None):
        """Packed sequences x [tokens, width] -> (y, final states)."""
        q, k, v, gate = self._operands(x, positions)
        o, state = gs.state_scan(q, k, v, gate, state, scale=self.shape[2] ** -0.5, gate_shift=4.0,
                                 seq_offsets=seq_offsets)
        return self.out(o.flatten(-2)), state

    @torch.no_grad()
    def step(self, x, positions, pool, slots):
        """One token of each request, x [requests, width]; their states,
        pool[slots], are updated in place."""
        q, k, v, gate = self._operands(x, positions)
        o = gs.state_scan_step(q, k, v, gate, pool, slots, scale=self.shape[2] ** -0.5, gate_shift=4.0)
        return self.out(o.flatten(-2))


class Model(torch.nn.Module):
    """Embedding of a token and its predecessor, one mixing layer, logits."""

    def __init__(self, vocabulary=64, width=256, **kw):
        super().__init__()
        dev, dt = kw.get("device", "cuda"), kw.get("dtype", torch.float32)
        self.embed = torch.nn.Embedding(vocabulary, width, device=dev, dtype=dt)
        self.before = torch.nn.Embedding(vocabulary, width, device=dev, dtype=dt)
        self.mix = MixingLayer(width, **kw)
        self.head = torch.nn.Linear(width, vocabulary, bias=False, device=dev, dtype=dt)
        for e in (self.embed, self.before):
            torch.nn.init.normal_(e.weight, std=0.5)

    def forward(self, tokens, before, positions, seq_offsets, state=None):
        x = self.embed(tokens) + self.before(before)
        y, state = self.mix(x, positions, seq_offsets, state)
        return self.head(x + y).float(), state

    @torch.no_grad()
    def step(self, tokens, before, positions, pool, slots):
        x = self.embed(tokens) + self.before(before)
        return self.head(x + self.mix.step(x, positions, pool, slots)).float()


def pack(lengths, device="cuda"):
    """(seq_offsets int32, positions int64) of packed sequences."""
    n = torch.tensor([0] + list(lengths)).cumsum(0)
    positions = torch.cat([torch.arange(x) for x in lengths]) if sum(lengths) else torch.empty(0, dtype=torch.long)
    return n.to(torch.int32).to(device), positions.to(device)


def predecessors(tokens, positions):
    before = torch.roll(tokens, 1)
    before[positions == 0] = 0
    return before


def recall_batch(gen, lengths, vocabulary, device="cuda"):
    """Sequences that repeat a random cycle of distinct tokens."""
    seqs = []
    for n in lengths:
        cycle = torch.randperm(vocabulary - 1, generator=gen)[:16] + 1
        seqs.append(cycle.repeat(n // 16 + 1)[:n])
    return torch.cat(seqs).to(device)


def train(model, steps, gen, lengths=(96, 160, 64, 192, 130, 77) * 12, vocabulary=64, rate=2e-3):
    """Mean losses of the steps."""
    offsets, positions = pack(lengths)
    last = (offsets[1:] - 1).long()
    optimizer = torch.optim.AdamW(model.parameters(), lr=rate)
    losses = []
    for _ in range(steps):
        tokens = recall_batch(gen, lengths, vocabulary)
        with torch.autocast("cuda", torch.bfloat16):
            logits, _ = model(tokens, predecessors(tokens, positions), positions, offsets)
        target = torch.roll(tokens, -1)
        target[last] = -100
        loss = torch.nn.functional.cross_entropy(logits, target)
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
@torch.autocast("cuda", torch.bfloat16)
def generate(model, prompts, count, pool_size):
    """Greedy continuations [requests, count] of packed prompts."""
    lengths = [len(p) for p in prompts]
    offsets, positions = pack(lengths)
    tokens = torch.cat(prompts).cuda()
    logits, states = model(tokens, predecessors(tokens, positions), positions, offsets)
    # the requests' states live in scattered slots of a pool
    pool = states.new_zeros(pool_size, *states.shape[1:])
    slots = torch.randperm(pool_size)[:len(prompts)].to(torch.int32).cuda()
    pool[slots.long()] = states
    ends = (offsets[1:] - 1).long()
    before, token = tokens[ends], logits[ends].argmax(-1)
    position = torch.tensor(lengths).cuda()
    made = [token]
    for _ in range(count - 1):
        logits = model.step(token, before, position, pool, slots)
        before, token, position = token, logits.argmax(-1), position + 1
        made.append(token)
    return torch.stack(made, 1)


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    args = parser.parse_args()
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(1)
    model = Model()
    start = time.time()
    losses = train(model, args.steps, gen)
    print(f"{args.steps} steps in {time.time() - start:.1f} s: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    prompts = [recall_batch(gen, [n], 64, "cpu") for n in (40, 33, 70, 51)]
    made = generate(model, prompts, 32, pool_size=16).cpu()
    want = torch.stack([p[:16].repeat(8)[len(p):len(p) + 32] for p in prompts])
    print(f"32 tokens of {len(prompts)} requests generated: {(made == want).float().mean():.3f} continue their cycle")


if __name__ == "__main__":
    main()
