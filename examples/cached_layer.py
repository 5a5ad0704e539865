"""A served attention layer: prompts of several tenants, then decode steps, through the
multi-adapter projections, the rotation and the key/value cache in 8 or in 4 bits.

    python examples/cached_layer.py

Each step: the fused q|k|v projection with every row's adapter, norms and rotation of the
queries and keys by their positions, the new keys and values appended to the pages,
attention of the new rows over the cache, the output projection with every row's adapter.
Weights, adapters and inputs are random.  Prints the largest difference from the same layer
in plain fp64 operations over keys and values that were never quantised.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Layer:
    """Projections, adapters and cache of one layer."""

    def __init__(self, hidden=1024, q_heads=8, kv_heads=2, head_dim=128, tenants=3, rank=16, page_size=32,
                 max_seqs=4, max_len=512, max_tokens=1024, seed=0, bits=8):
        import torch
        from heterogeneous_lora_gemm_gb300 import Cache, Cache4, Pool, Rotary
        self.q_heads, self.kv_heads, self.head_dim, self.page_size = q_heads, kv_heads, head_dim, page_size
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(*shape, size=1.0):
            return (torch.randn(shape, device="cuda", generator=g) * size).bfloat16()

        heads = q_heads + 2 * kv_heads
        self.Wqkv = weight(heads * head_dim, hidden, size=hidden ** -0.5)
        self.Wo = weight(hidden, q_heads * head_dim, size=(q_heads * head_dim) ** -0.5)
        self.adapters = []
        self.qkv = Pool(tenants, tenants * rank, rank, hidden, heads * head_dim, "bf16", max_tokens)
        self.out = Pool(tenants, tenants * rank, rank, q_heads * head_dim, hidden, "bf16", max_tokens)
        for a in range(tenants):
            pair = []
            for pool, W in ((self.qkv, self.Wqkv), (self.out, self.Wo)):
                down, up = weight(rank, W.shape[1], size=W.shape[1] ** -0.5), weight(W.shape[0], rank, size=0.25)
                pool.load(a, down, up, 1.0)
                pair.append((down, up))
            self.adapters.append(pair)
        width = -(-max_len // page_size)
        shape = (max_seqs * width, kv_heads, page_size, head_dim)
        self.pages = torch.randperm(shape[0], device="cuda", generator=g).int().view(max_seqs, width)
        if bits == 4:
            blocks = (max_seqs * width, kv_heads, page_size // 16, 18 * head_dim)
            self.cache = Cache4(torch.empty(blocks, dtype=torch.uint8, device="cuda"), q_heads)
        else:
            codes, scale = dict(dtype=torch.int8, device="cuda"), dict(device="cuda")
            self.cache = Cache(torch.zeros(shape, **codes), torch.zeros(shape[:2], **scale), torch.zeros(shape, **codes),
                               torch.zeros(shape[:2], **scale), q_heads)
        self.rotary = Rotary(head_dim)
        self.q_norm, self.k_norm = (1 + 0.1 * torch.randn(head_dim, device="cuda", generator=g) for _ in range(2))

    def step(self, X, row_adapter, lengths, offsets=None, max_new=1):
        """One step of rows X [T, hidden]; lengths as they are after it."""
        import torch
        T, D = X.shape[0], self.head_dim
        Y = torch.empty((T, self.Wqkv.shape[0]), dtype=X.dtype, device=X.device)
        self.qkv.forward(X, self.Wqkv, row_adapter, Y)
        q, k, v = Y.unflatten(1, (-1, D)).split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        pages = self.pages[:lengths.shape[0]]
        self.rotary.apply(q, k, lengths, offsets=offsets, max_new=max_new, q_weight=self.q_norm, k_weight=self.k_norm)
        self.cache.append(k, v, lengths, pages, offsets=offsets, max_new=max_new)
        A = torch.empty((T, self.q_heads * D), dtype=X.dtype, device=X.device)
        self.cache.attend(q, A.unflatten(1, (-1, D)), lengths, pages, offsets=offsets, max_new=max_new)
        Z = torch.empty((T, self.Wo.shape[0]), dtype=X.dtype, device=X.device)
        self.out.forward(A, self.Wo, row_adapter, Z)
        return Z

    def plain(self, X, adapter, keep):
        """The same layer for one sequence's new rows in fp64; `keep` holds its keys and values."""
        import torch
        D, G = self.head_dim, self.q_heads // self.kv_heads

        def project(x, W, which):
            y = x @ W.double().T
            if adapter >= 0:
                down, up = (t.double() for t in self.adapters[adapter][which])
                y = y + (x @ down.T) @ up.T
            return y

        q, k, v = project(X.double(), self.Wqkv, 0).unflatten(1, (-1, D)).split(
            [self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        held = keep[0].shape[0] if keep else 0
        angle = torch.arange(held, held + X.shape[0], device=X.device).double()[:, None, None] * torch.tensor(
            [10000.0 ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64, device=X.device)

        def turn(y, weight):
            y = y * weight.double() / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            a, b = y.chunk(2, dim=-1)
            return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], dim=-1)

        q, k = turn(q, self.q_norm), turn(k, self.k_norm)
        keep[:] = [torch.cat([keep[0], k]), torch.cat([keep[1], v])] if keep else [k, v]
        k, v = (t.repeat_interleave(G, dim=1) for t in keep)
        n, L = X.shape[0], k.shape[0]
        w = torch.einsum("ihd,thd->hit", q, k) * D ** -0.5
        seen = torch.arange(L, device=X.device) <= torch.arange(L - n, L, device=X.device)[:, None]
        w = w.masked_fill(~seen, float("-inf")).softmax(dim=-1)
        return project(torch.einsum("hit,thd->ihd", w, v).flatten(1), self.Wo, 1)


def main(prompts=(200, 33, 1, 97), adapters=(0, -1, 2, 1), decode_steps=8, bits=8) -> float:
    """Prompts, then decode steps; returns the largest difference over the outputs' size."""
    import torch
    from heterogeneous_lora_gemm_gb300 import mlora
    layer = Layer(bits=bits)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    keep, held, worst = [[] for _ in prompts], list(prompts), 0.0
    for s in range(decode_steps + 1):
        rows = list(prompts) if s == 0 else [1] * len(prompts)
        held = held if s == 0 else [n + 1 for n in held]
        X = torch.randn((sum(rows), layer.Wqkv.shape[1]), device="cuda", generator=g).bfloat16()
        row_adapter = torch.tensor([a for a, n in zip(adapters, rows) for _ in range(n)], **i32)
        ends = torch.tensor([0] + rows, device="cuda").cumsum(0).int()
        Z = layer.step(X, row_adapter, torch.tensor(held, **i32), offsets=ends if s == 0 else None, max_new=max(rows))
        for b, a in enumerate(adapters):
            at = slice(sum(rows[:b]), sum(rows[:b + 1]))
            want = layer.plain(X[at], a, keep[b])
            worst = max(worst, float((Z[at] - want).norm() / want.norm()))
    assert layer.cache.status() == layer.rotary.status() == layer.qkv.status() == layer.out.status() == mlora.MLORA_OK
    return worst


if __name__ == "__main__":
    for bits in (8, 4):
        print(f"{bits} bits: largest relative difference from fp64 without quantisation: {main(bits=bits):.4f}")
