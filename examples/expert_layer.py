"""An expert layer's training steps, from the gathered buffer to orthogonalised updates.

N data-parallel ranks share a router and E experts of gate, up and down
projections (fp32 shards of each on every rank).  One step, with every rank's
compute run in turn on this GPU:

  pack, place   every rank's fp32 shards into per-parameter bf16 storage
  route         each token's experts and weights from its logits
  dispatch      the tokens' rows in expert order
  experts       h = act(x Wg^T) * (x Wu^T) and z = h Wd^T, expert by expert
  combine       y = each token's results by its weights
  backward      the same way back: dz and dweights, dWd and dh, dWg, dWu and the
                logits' gradients
  reduce-scatter   the ranks' bf16 gradients into fp32 shards of their mean
  update        the mean gradients, packed and placed as the parameters are,
                orthogonalised matrix by matrix (the router's as it is)

The layer learns a fixed random map; the loss of each step is printed.

    python examples/expert_layer.py [--steps 20] [--tokens 300] [--experts 8] [--topk 2] [--hidden 256] [--ffn 192]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layout_aware_collectives_gb300 as tide  # noqa: E402


def new(*s, dtype=torch.bfloat16):
    return torch.empty(*s, device="cuda", dtype=dtype)


class Layer:
    """The layer's storage, sharded over `ranks`: router, then gate, up and down of each expert."""

    def __init__(self, ranks: int, experts: int, topk: int, hidden: int, ffn: int, seed: int = 0):
        self.shapes = [(experts, hidden)] + [(ffn, hidden), (ffn, hidden), (hidden, ffn)] * experts
        self.layout = tide.Layout(self.shapes, ranks)
        self.router = tide.Router(experts, topk)
        self.ranks, self.experts, self.topk, self.hidden, self.ffn = ranks, experts, topk, hidden, ffn
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.shards = [[] for _ in range(ranks)]  # every rank's rows of each parameter, zero-padded
        for p, (rows, cols) in enumerate(self.shapes):
            chunk = self.layout.chunk_rows(p)
            whole = torch.zeros(ranks * chunk, cols, device="cuda")
            whole[:rows] = torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5
            for r in range(ranks):
                self.shards[r].append(whole[r * chunk:(r + 1) * chunk].clone())
        self.means = [[torch.empty_like(s) for s in rank] for rank in self.shards]
        self.gathered = new(ranks * self.layout.block_numel)
        self.params = [new(*s) for s in self.shapes]
        self.grads = [[new(*s) for s in self.shapes] for _ in range(ranks)]
        self.whole = [new(*s) for s in self.shapes]  # mean gradients, then updates' sources
        self.updates = [new(*s) for s in self.shapes]
        wide, tall = (ffn, hidden), (hidden, ffn)
        self.workspace = new(max(tide.orthogonalize_workspace_bytes(2 * experts, *wide), tide.orthogonalize_workspace_bytes(experts, *tall)),
                             dtype=torch.uint8)

    def place(self, shards, params):
        self.layout.pack(-1, [t for rank in shards for t in rank], self.gathered)
        self.layout.place(self.gathered, params)

    def expert(self, tensors, e):
        return tensors[1 + 3 * e:4 + 3 * e]


class Pass:
    """Buffers of one rank's pass over `tokens` tokens."""

    def __init__(self, layer: Layer, tokens: int):
        k, e, pairs = layer.topk, layer.experts, tokens * layer.topk
        self.ids, self.slots = new(tokens, k, dtype=torch.int32), new(tokens, k, dtype=torch.int32)
        self.offsets = new(e + 1, dtype=torch.int32)
        self.weights, self.dweights = new(tokens, k, dtype=torch.float32), new(tokens, k, dtype=torch.float32)
        self.dlogits = new(tokens, e, dtype=torch.float32)
        self.x, self.z, self.dz = (new(pairs, layer.hidden) for _ in range(3))
        self.h = new(pairs, layer.ffn)
        self.y = new(tokens, layer.hidden)
        self.order = new(tide.expert_slots_workspace_bytes(tokens, k, e), dtype=torch.uint8)
        self.workspace = new(tide.gated_workspace_bytes(pairs, layer.hidden, layer.ffn), dtype=torch.uint8)


def forward_backward(layer: Layer, compute: tide.Compute, work: Pass, x, target, grads) -> float:
    """One rank's loss; its gradients in `grads`."""
    m, k, hidden, ffn = x.shape[0], layer.topk, layer.hidden, layer.ffn
    logits = x.float() @ layer.params[0].float().T
    compute.route(layer.router, m, logits, work.ids, work.weights)
    compute.expert_slots(m, k, layer.experts, work.ids, work.slots, work.offsets, work.order)
    compute.expert_gather(m, hidden, k, x, work.slots, work.x, m * k)
    at = work.offsets.tolist()
    mine = [slice(at[e], at[e + 1]) for e in range(layer.experts)]
    for e, rows in enumerate(mine):
        gate, up, down = layer.expert(layer.params, e)
        compute.gated_forward(rows.stop - rows.start, hidden, ffn, work.x[rows], gate, up, work.h[rows])
        torch.mm(work.h[rows], down.T, out=work.z[rows])
    compute.expert_combine(m, hidden, k, work.z, m * k, work.slots, work.weights, work.y)
    off = work.y.float() - target
    dy = (off * (2.0 / off.numel())).bfloat16()
    compute.expert_combine_backward(m, hidden, k, dy, work.z, m * k, work.slots, work.weights, work.dz, work.dweights)
    for e, rows in enumerate(mine):
        gate, up, down = layer.expert(layer.params, e)
        d_gate, d_up, d_down = layer.expert(grads, e)
        torch.mm(work.dz[rows].T, work.h[rows], out=d_down)
        dh = work.dz[rows] @ down
        compute.gated_backward(rows.stop - rows.start, hidden, ffn, dh, work.x[rows], gate, up, None, d_gate, d_up, work.workspace)
    compute.route_backward(layer.router, m, logits, work.ids, work.dweights, work.dlogits)
    grads[0].copy_(work.dlogits.T @ x.float())
    return float((off * off).mean())


def step(layer: Layer, compute: tide.Compute, work: Pass, inputs, targets, rate: float) -> float:
    layer.place(layer.shards, layer.params)
    loss = 0.0
    for r in range(layer.ranks):
        loss += forward_backward(layer, compute, work, inputs[r], targets[r], layer.grads[r]) / layer.ranks
    flat = [t for rank in layer.grads for t in rank]
    layer.layout.reduce_scatter(flat, [t for rank in layer.means for t in rank], 1.0 / layer.ranks)
    # a matrix's update needs all of its rows: the shards come together as the parameters do
    layer.place(layer.means, layer.whole)
    for rows, cols, of in ((layer.ffn, layer.hidden, (0, 1)), (layer.hidden, layer.ffn, (2,))):
        at = [1 + 3 * e + i for e in range(layer.experts) for i in of]
        compute.orthogonalize(rows, cols, [layer.whole[p] for p in at], [layer.updates[p] for p in at], layer.workspace, src_type="bf16")
    layer.updates[0].copy_(layer.whole[0])
    for p, update in enumerate(layer.updates):
        chunk = layer.layout.chunk_rows(p)
        for r in range(layer.ranks):
            rows = update[r * chunk:(r + 1) * chunk]
            layer.shards[r][p][:rows.shape[0]].sub_(rows, alpha=rate)
    compute.check_device()
    return loss


def problem(layer: Layer, tokens: int, seed: int):
    g = torch.Generator(device="cuda").manual_seed(seed)
    inputs = [torch.randn(tokens, layer.hidden, generator=g, device="cuda").bfloat16() for _ in range(layer.ranks)]
    goal = torch.randn(layer.hidden, layer.hidden, generator=g, device="cuda") * layer.hidden ** -0.5
    return inputs, [x.float() @ goal for x in inputs]


def train(steps: int = 20, ranks: int = 2, tokens: int = 300, experts: int = 8, topk: int = 2, hidden: int = 256, ffn: int = 192,
          rate: float = 0.02, seed: int = 0):
    """The loss of each step."""
    layer = Layer(ranks, experts, topk, hidden, ffn, seed)
    work = Pass(layer, tokens)
    inputs, targets = problem(layer, tokens, seed + 1)
    with tide.Compute() as compute:
        return [step(layer, compute, work, inputs, targets, rate) for _ in range(steps)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("steps", 20), ("ranks", 2), ("tokens", 300), ("experts", 8), ("topk", 2), ("hidden", 256), ("ffn", 192)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--rate", type=float, default=0.02)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps, a.ranks, a.tokens, a.experts, a.topk, a.hidden, a.ffn, a.rate)):
        print(f"step {i:3d}  loss {loss:.5f}")
