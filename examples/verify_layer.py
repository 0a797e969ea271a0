"""One layer's step of speculative decoding: a tree of drafted tokens through attention and MLP.

The target's products are W12 (exact); `drafter_mlp` takes the same rows through an MLP kept in 8 bits, as a
drafter's may be.  Every launch goes to the current stream.  Random weights of a small generic shape:

    python examples/verify_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lossless_bit_weight_encode_amd as w12

HIDDEN, Q_HEADS, KV_HEADS, DIM, FFN, PAGE = 1024, 8, 2, 128, 2816, 64


class Layer:
    """Weights, cache and page table of one layer and one request."""

    def __init__(self, pages: int = 16, seed: int = 0):
        gen = torch.Generator("cuda").manual_seed(seed)
        dev = dict(device="cuda", generator=gen)

        def weights(n, k):
            return (torch.randn(n, k, **dev) * k ** -0.5).bfloat16()

        self.norm1 = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")
        self.norm2 = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")
        up, down = weights(2 * FFN, HIDDEN), weights(HIDDEN, FFN)
        self.qkv = w12.encode(weights((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN))
        self.o = w12.encode(weights(HIDDEN, Q_HEADS * DIM))
        self.up, self.down = w12.encode(up), w12.encode(down)
        self.up8 = self.quantised(up)
        zeros = dict(dtype=torch.bfloat16, device="cuda")
        self.cache = w12.KVCache(torch.zeros(pages, PAGE, KV_HEADS, DIM, **zeros), torch.zeros(pages, PAGE, KV_HEADS, DIM, **zeros))
        self.page_table = torch.randperm(pages, **dev).int().view(1, pages)
        self.inv_freq = 10000.0 ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device="cuda") / DIM)

    @staticmethod
    def quantised(w):
        """E4M3 with a scale per 128 x 128 (the sizes here are whole blocks)."""
        n, k = w.shape
        blocks = w.float().view(n // 128, 128, k // 128, 128)
        scale = blocks.abs().amax((1, 3)) / 448
        return (blocks / scale[:, None, :, None]).reshape(n, k).to(torch.float8_e4m3fn), scale

    def slots(self, first: int, n: int):
        """Where tokens first .. first + n - 1 of the request are in the cache."""
        token = torch.arange(first, first + n, device="cuda")
        return self.page_table[0, token // PAGE].long() * PAGE + token % PAGE

    def step(self, x, ctx: int, depth=None, tree_mask=None):
        """x: FP32 [n, HIDDEN], the residual stream of n nodes behind ctx cached tokens; depth [n]: a node's
        depth in the tree (its position is ctx + depth); tree_mask: a chain without it.
        Returns the residual stream after the layer and the drafter's view of its MLP input."""
        n = x.shape[0]
        depth = torch.arange(n, device="cuda") if depth is None else depth
        x = x.clone()
        y = w12.add_rmsnorm(x, self.norm1, residual_out=x)
        qkv = w12.gemm(y, self.qkv)
        q = w12.rope_append(qkv, self.cache, (ctx + depth).int().view(1, n), self.slots(ctx, n), self.inv_freq, Q_HEADS)
        ints = dict(dtype=torch.int32, device="cuda")
        a = w12.tree_attention(q, self.cache, self.page_table, torch.tensor([ctx], **ints), torch.tensor([0, n], **ints),
                               tree_mask=tree_mask)
        y = torch.empty(n, HIDDEN, dtype=torch.bfloat16, device="cuda")
        yq = torch.empty(n, HIDDEN, dtype=torch.float8_e4m3fn, device="cuda")
        yq_scale = torch.empty(n, HIDDEN // 128, device="cuda")
        w12.add_rmsnorm(x, self.norm2, w12.gemm(a, self.o), residual_out=x, y=y, yq=yq, yq_scale=yq_scale)
        return x + w12.gemm(self.gated(w12.gemm(y, self.up)), self.down), (yq, yq_scale)

    @staticmethod
    def gated(u):
        return (torch.nn.functional.silu(u[:, :FFN]) * u[:, FFN:]).bfloat16()

    def drafter_mlp(self, yq, yq_scale):
        return w12.gemm(self.gated(w12.gemm_e4m3(yq, yq_scale, *self.up8)), self.down)


def tree_of(parents):
    """Depths and the mask (a node, its ancestors) of a tree given by parents (-1: behind the last cached token)."""
    depth, mask = [], []
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        mask.append((1 << i) | (0 if p < 0 else mask[p]))
    signed = [m - (1 << 64) if m >> 63 else m for m in mask]
    return torch.tensor(depth, device="cuda"), torch.tensor(signed, dtype=torch.int64, device="cuda").view(-1, 1)


def main():
    layer = Layer()
    gen = torch.Generator("cuda").manual_seed(1)
    prompt = torch.randn(300, HIDDEN, device="cuda", generator=gen)
    layer.step(prompt, 0)
    parents = [-1, 0, 0, 1, 1, 2, 3, 3, 5]
    drafted = torch.randn(len(parents), HIDDEN, device="cuda", generator=gen)
    depth, mask = tree_of(parents)
    out, mlp_in = layer.step(drafted, 300, depth, mask)
    draft = layer.drafter_mlp(*mlp_in)
    # what the tree says of the path to node 6 (0, 1, 3, 6) is what the path says as a chain of its own
    path = [0, 1, 3, 6]
    chain, _ = layer.step(drafted[path], 300)
    print(f"tree of {len(parents)} nodes: path against chain, largest difference {(out[path] - chain).abs().max():.2e}"
          f" of {chain.abs().max():.2f}; drafter's MLP {tuple(draft.shape)}")


if __name__ == "__main__":
    main()
