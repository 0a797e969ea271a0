"""A recurrent layer's steps in speculative decoding: a prompt, a tree of drafted tokens, their verification, and the accepted path's
way into the layer's states.

The layer's products are W12 (exact).  Every launch goes to the current stream.  Random weights of a small generic shape:

    python examples/recurrent_layer.py
"""
import os
import sys

import torch

sys.path[:0] = [os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__))]
import lossless_bit_weight_encode_amd as w12
from verify_layer import tree_of

HIDDEN, K_HEADS, V_HEADS, DIM, TAPS, VOCAB = 1024, 4, 8, 128, 4, 5000
QK, V = K_HEADS * DIM, V_HEADS * DIM


class RecurrentLayer:
    """Weights, and the states of a few requests: the convolution's last rows and the delta rule's matrices."""

    def __init__(self, requests: int = 2, seed: int = 0):
        gen = torch.Generator("cuda").manual_seed(seed)
        dev = dict(device="cuda", generator=gen)

        def weights(n, k):
            return (torch.randn(n, k, **dev) * k ** -0.5).bfloat16()

        self.norm = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")
        self.qkv = w12.encode(weights(2 * QK + V, HIDDEN))
        self.gates = w12.encode(weights(2 * V_HEADS, HIDDEN))
        self.o = w12.encode(weights(HIDDEN, V))
        self.head = w12.encode(weights(VOCAB, HIDDEN))
        self.conv = weights(2 * QK + V, TAPS)
        self.rate = torch.exp(torch.linspace(-5, 0, V_HEADS, device="cuda"))
        self.rows = torch.zeros(requests, TAPS - 1, 2 * QK + V, device="cuda")
        self.states = torch.zeros(requests, V_HEADS, DIM, DIM, device="cuda")

    def project(self, x):
        """What the layer's rows bring along: the convolution's input, decays and strengths."""
        y = w12.add_rmsnorm(x, self.norm)
        gates = w12.gemm(y, self.gates)
        g = -self.rate * torch.nn.functional.softplus(gates[:, :V_HEADS])
        return w12.gemm(y, self.qkv), g, torch.sigmoid(gates[:, V_HEADS:])

    def step(self, x, seq_ptr, slots, tree_mask=None):
        """x: FP32 [n, HIDDEN].  A prompt's rows, or single tokens, move the states of `slots`; a tree's leave them.
        Returns the residual stream after the layer, and what advance() needs."""
        u, g, beta = self.project(x)
        dst = None if tree_mask is not None else slots
        y = w12.short_conv(u, self.conv, self.rows, seq_ptr, slots, dst=dst, tree_mask=tree_mask)
        q, k, v = y.split((QK, QK, V), 1)
        a = w12.gated_delta(q, k, v, g, beta, self.states, seq_ptr, slots, dst=dst, tree_mask=tree_mask)
        return x + w12.gemm(a, self.o), (u, y, g, beta)

    def advance(self, kept, seq_ptr, slots, path, count):
        """Moves the states along each request's accepted path."""
        u, y, g, beta = kept
        move = dict(dst=slots, rows=path, lens=count, outputs=False)
        _, k, v = y.split((QK, QK, V), 1)
        w12.gated_delta(None, k, v, g, beta, self.states, seq_ptr, slots, **move)
        w12.short_conv(u, self.conv, self.rows, seq_ptr, slots, **move)

    def verify(self, x, tokens, u, seq_ptr, tree_mask):
        return w12.verify_draft(w12.gemm(w12.add_rmsnorm(x, self.norm), self.head), tokens, u, seq_ptr, tree_mask=tree_mask)


def main():
    layer = RecurrentLayer()
    gen = torch.Generator("cuda").manual_seed(1)
    ints = dict(dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1], **ints)
    prompts = torch.randn(300 + 45, HIDDEN, device="cuda", generator=gen)
    layer.step(prompts, torch.tensor([0, 300, 345], **ints), slots)
    before = layer.rows.clone(), layer.states.clone()
    trees = [[-1, 0, 0, 1, 1, 2, 3, 3, 5], [-1, 0, 1, 1, 2]]
    nodes, mask = sum(map(len, trees)), torch.cat([tree_of(t)[1] for t in trees])
    seq_ptr = torch.tensor([0, len(trees[0]), nodes], **ints)
    drafted = torch.randn(nodes, HIDDEN, device="cuda", generator=gen)
    out, kept = layer.step(drafted, seq_ptr, slots, mask)
    # tokens as a good drafter would have drawn them: of the first children, what the target says itself
    u = torch.rand(nodes, device="cuda", generator=gen)
    alone = torch.arange(nodes + 1, **ints)
    taken = layer.verify(out, torch.zeros(nodes, **ints), u, alone, None)[2]
    tokens = torch.full((nodes,), VOCAB - 1, **ints)
    at = 0
    for tree in trees:
        for i, p in enumerate(tree):
            if p >= 0 and i == tree.index(p):
                tokens[at + i] = taken[at + p]
        at += len(tree)
    path, count, following = layer.verify(out, tokens, u, seq_ptr, mask)
    layer.advance(kept, seq_ptr, slots, path, count)
    # the same tokens one after another, from the states before: the same up to how the products' sums fall (a value of BF16 here or
    # there is its neighbour)
    after = layer.rows.clone(), layer.states.clone()
    layer.rows.copy_(before[0])
    layer.states.copy_(before[1])
    at, off = [0, len(trees[0])], []

    def apart(a, b):
        off.append(((a - b).norm() / b.norm()).item())

    for b in range(2):
        for r in path[at[b]:at[b] + count[b]].long():
            chain, _ = layer.step(drafted[r:r + 1], torch.tensor([0, 1], **ints), slots[b:b + 1])
            apart(out[r:r + 1], chain)
    apart(after[0], layer.rows)
    apart(after[1], layer.states)
    print(f"accepted {count.tolist()} of {[len(t) for t in trees]} nodes, next {following.tolist()}; token by token: outputs off by"
          f" {max(off[:-2]):.1e}, the convolution's rows by {off[-2]:.1e}, the states by {off[-1]:.1e}")
    return count, off


if __name__ == "__main__":
    main()
