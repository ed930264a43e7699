"""A feed-forward unit's training steps, from the gathered buffer to the shards.

N data-parallel ranks share one feed-forward block (gate, up and down
projections, fp32 shards of each on every rank).  One step is what an FSDP2
unit does, with every rank's compute run in turn on this GPU:

  pack      every rank's fp32 shards into the rank-major bf16 buffer
  place     the buffer into per-parameter storage
  forward   h = act(x Wg^T) * (x Wu^T), its activations kept in 8 bits, then
            y = h Wd^T from 8-bit blocks of h and Wd
  backward  dWd and dh from dy; dWg, dWu (and h again) from the 8-bit checkpoint
  reduce-scatter   the ranks' bf16 gradients into fp32 shards of their mean
  update    plain gradient descent on the shards

The block learns a fixed random map; the loss of each step is printed.

    python examples/feed_forward_unit.py [--steps 30] [--tokens 250] [--hidden 256] [--ffn 704]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layout_aware_collectives_gb300 as tide  # noqa: E402


class Unit:
    """One feed-forward unit's storage, sharded over `ranks`."""

    def __init__(self, ranks: int, hidden: int, ffn: int, seed: int = 0):
        self.shapes = [(ffn, hidden), (ffn, hidden), (hidden, ffn)]  # gate, up, down
        self.layout = tide.Layout(self.shapes, ranks)
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = dict(device="cuda", dtype=torch.bfloat16)
        self.ranks, self.hidden, self.ffn = ranks, hidden, ffn
        # every rank's fp32 shards: its rows of each parameter, zero-padded
        self.shards = [[] for _ in range(ranks)]
        for p, (rows, cols) in enumerate(self.shapes):
            chunk = self.layout.chunk_rows(p)
            whole = torch.zeros(ranks * chunk, cols, device="cuda")
            whole[:rows] = torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5
            for r in range(ranks):
                self.shards[r].append(whole[r * chunk:(r + 1) * chunk].clone())
        self.updates = [[torch.empty_like(s) for s in rank] for rank in self.shards]
        self.gathered = torch.empty(ranks * self.layout.block_numel, **new)
        self.params = [torch.empty(*s, **new) for s in self.shapes]
        self.grads = [[torch.empty(*s, **new) for s in self.shapes] for _ in range(ranks)]

    def flat(self, of):
        return [t for rank in of for t in rank]

    def gather(self):
        self.layout.pack(-1, self.flat(self.shards), self.gathered)
        self.layout.place(self.gathered, self.params)

    def reduce_and_update(self, rate: float):
        self.layout.reduce_scatter(self.flat(self.grads), self.flat(self.updates), 1.0 / self.ranks)
        for w, g in zip(self.flat(self.shards), self.flat(self.updates)):
            w.sub_(g, alpha=rate)


class Activations:
    """Buffers of one rank's pass over `tokens` tokens."""

    def __init__(self, tokens: int, hidden: int, ffn: int):
        def new(*s, dtype=torch.bfloat16):
            return torch.empty(*s, device="cuda", dtype=dtype)

        def blocks(rows, cols, block_rows=1):
            return (new(rows, cols, dtype=torch.float8_e4m3fn),
                    new(-(-rows // block_rows), -(-cols // 128), dtype=torch.float32))

        self.h, self.y = new(tokens, ffn), new(tokens, hidden)
        self.h8, self.down8 = blocks(tokens, ffn), blocks(hidden, ffn, 128)
        self.checkpoint = tide.GatedCheckpoint(*blocks(tokens, ffn), *blocks(tokens, ffn), *blocks(tokens, hidden))
        self.workspace = new(tide.gated_workspace_bytes(tokens, hidden, ffn), dtype=torch.uint8)


def step(unit: Unit, compute: tide.Compute, acts: Activations, inputs, targets, rate: float) -> float:
    m, k, f = inputs[0].shape[0], unit.hidden, unit.ffn
    unit.gather()
    gate, up, down = unit.params
    compute.fp8_store(k, f, down, *acts.down8, block_rows=128)
    loss = 0.0
    for r in range(unit.ranks):
        x, d_gate, d_up, d_down = inputs[r], *unit.grads[r]
        compute.gated_forward(m, k, f, x, gate, up, acts.h, checkpoint=acts.checkpoint)
        compute.fp8_store(m, f, acts.h, *acts.h8)
        compute.fp8_matmul(m, k, f, *acts.h8, *acts.down8, acts.y)
        # mean squared error; from here on h and x exist in 8 bits only
        off = acts.y.float() - targets[r]
        loss += float((off * off).mean()) / unit.ranks
        dy = (off * (2.0 / off.numel())).bfloat16()
        dh = dy @ down
        compute.gated_backward(m, k, f, dh, None, gate, up, None, d_gate, d_up, acts.workspace,
                               checkpoint=acts.checkpoint, h=acts.h)
        torch.mm(dy.T, acts.h, out=d_down)
    unit.reduce_and_update(rate)
    compute.check_device()
    return loss


def train(steps: int = 30, ranks: int = 4, tokens: int = 250, hidden: int = 256, ffn: int = 704, rate: float = 60.0,
          seed: int = 0):
    """The loss of each step."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    inputs = [torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16() for _ in range(ranks)]
    goal = torch.randn(hidden, hidden, generator=g, device="cuda") * hidden ** -0.5
    targets = [x.float() @ goal for x in inputs]
    unit = Unit(ranks, hidden, ffn, seed)
    acts = Activations(tokens, hidden, ffn)
    with tide.Compute() as compute:
        return [step(unit, compute, acts, inputs, targets, rate) for _ in range(steps)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("steps", 30), ("ranks", 4), ("tokens", 250), ("hidden", 256), ("ffn", 704)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--rate", type=float, default=60.0)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps, a.ranks, a.tokens, a.hidden, a.ffn, a.rate)):
        print(f"step {i:3d}  loss {loss:.5f}")
