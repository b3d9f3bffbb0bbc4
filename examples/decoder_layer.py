"""One decoder layer serving several tenants from a shared base, on the GPU.

    python examples/decoder_layer.py [--bits 8]

Random weights of a small grouped-query layer and three variants of it.  The
requests' prompts are prefilled in chunks, each through its tenant's variant;
then all requests decode together, a token each, through the mixed-variant
linears.  Every step is the same five calls around the linears: the norm that
adds the residual, the cache's write, attention over the cache, and the norm
before the feed-forward part.  (Rotary positions are left out: they are applied
to q and k, as views of the fused projection's rows, before the write.)
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tenant_linear_layers_amd as T

EPS = 1e-5
DECODE = 64        # tokens that one mixed-variant linear takes


class PagedCache:
    """Keys and values of many sequences in pages taken from one pool."""

    def __init__(self, pages: int, page: int, kv_heads: int, dim: int, bits: int, device):
        shape = (pages, kv_heads, page, dim)
        kind = torch.bfloat16 if bits == 16 else torch.float8_e4m3fn
        self.k, self.v = (torch.zeros(shape, dtype=kind, device=device) for _ in range(2))
        self.k_scale = self.v_scale = None
        if bits == 8:
            self.k_scale, self.v_scale = (
                torch.zeros(shape[:3], dtype=torch.uint8, device=device)
                .view(torch.float8_e8m0fnu) for _ in range(2))
        self.page, self.device = page, device
        self.free = list(range(pages))
        self.pages, self.length = {}, {}

    def batch(self, requests):
        """What a step over [(sequence, new tokens)] needs on the device."""
        slots, cu, kv, rows = [], [0], [], []
        for seq, new in requests:
            mine, n = self.pages.setdefault(seq, []), self.length.get(seq, 0)
            while len(mine) * self.page < n + new:
                mine.append(self.free.pop())
            slots += [mine[j // self.page] * self.page + j % self.page for j in range(n, n + new)]
            self.length[seq] = n + new
            cu.append(cu[-1] + new)
            kv.append(n + new)
            rows.append(mine)
        width = max(map(len, rows))

        def ints(x):
            return torch.tensor(x, dtype=torch.int32, device=self.device)

        return dict(slots=ints(slots), cu_q=ints(cu), kv_len=ints(kv),
                    table=ints([r + [0] * (width - len(r)) for r in rows]),
                    max_q=max(n for _, n in requests))

    def release(self, seq):
        self.free += self.pages.pop(seq)
        del self.length[seq]


class DecoderLayer:
    def __init__(self, base: dict, norms: dict, variants, heads: int, kv_heads: int, dim: int):
        """base: bf16 weights "qkv", "o", "gate", "up", "down"; norms: bf16
        "attn" and "ffn"; variants: of each, {name: (packed signs, alpha)}."""
        self.base, self.norms, self.variants = base, norms, variants
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim

    def linear(self, name, x, ids, ids_dev):
        if len(set(ids)) == 1 and ids[0] >= 0:
            return T.linear(x, self.base[name], *self.variants[ids[0]][name], T.ALPHA_PER_ROW)
        packs, alphas = zip(*(v[name] for v in self.variants))
        y = [T.linear_multi(x[i:i + DECODE], ids_dev[i:i + DECODE], self.base[name], list(packs),
                            list(alphas), T.ALPHA_PER_ROW) for i in range(0, len(ids), DECODE)]
        return y[0] if len(y) == 1 else torch.cat(y)

    def forward(self, x, residual, ids, cache: PagedCache, batch):
        """(output, residual stream) of the tokens x, whose variants are ids; the
        next layer's first norm adds the two.  residual: None in the first."""
        ids_dev = torch.tensor(ids, dtype=torch.int32, device=x.device)
        y, h = T.rms_norm(x, self.norms["attn"], EPS, residual)
        h = x if h is None else h
        qkv = self.linear("qkv", y, ids, ids_dev)
        at = self.heads * self.dim, self.kv_heads * self.dim
        q, k, v = (t.unflatten(1, (-1, self.dim)) for t in qkv.split([at[0], at[1], at[1]], 1))
        T.kv_write(k, v, batch["slots"], cache.k, cache.v, cache.k_scale, cache.v_scale)
        o = T.paged_attention(q, cache.k, cache.v, batch["table"], batch["cu_q"],
                              batch["kv_len"], batch["max_q"], cache.k_scale, cache.v_scale)
        y, h = T.rms_norm(self.linear("o", o.flatten(1), ids, ids_dev), self.norms["ffn"], EPS, h)
        gate, up = (self.linear(n, y, ids, ids_dev) for n in ("gate", "up"))
        return self.linear("down", torch.nn.functional.silu(gate) * up, ids, ids_dev), h


def random_layer(device, hidden=1024, ffn=2816, heads=8, kv_heads=2, dim=128, n_variants=3,
                 seed=0) -> DecoderLayer:
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, std):
        return torch.randn(shape, generator=g, device=device).mul_(std)

    shapes = dict(qkv=((heads + 2 * kv_heads) * dim, hidden), o=(hidden, heads * dim),
                  gate=(ffn, hidden), up=(ffn, hidden), down=(hidden, ffn))
    base = {n: normal(*s, std=s[1] ** -0.5).bfloat16() for n, s in shapes.items()}
    variants = [{n: T.compress((w.float() + normal(*w.shape, std=1e-3)).bfloat16(), w,
                               T.ALPHA_PER_ROW) for n, w in base.items()}
                for _ in range(n_variants)]
    norms = {n: normal(hidden, std=0.1).add_(1.0).bfloat16() for n in ("attn", "ffn")}
    return DecoderLayer(base, norms, variants, heads, kv_heads, dim)


def serve(layer: DecoderLayer, cache: PagedCache, prompts, ids, steps, chunk=128):
    """prompts: bf16 [tokens, hidden] each; ids: their variants; steps: inputs
    [requests, hidden] of the decode steps.  The layer's outputs (with the
    residual stream added) of each request, prompt and decoded tokens."""
    out = [[] for _ in prompts]
    for r, p in enumerate(prompts):
        for i in range(0, len(p), chunk):
            x = p[i:i + chunk]
            y, h = layer.forward(x, None, [ids[r]] * len(x), cache, cache.batch([(r, len(x))]))
            out[r].append(y + h)
    for x in steps:
        y, h = layer.forward(x, None, ids, cache, cache.batch([(r, 1) for r in range(len(ids))]))
        for r, row in enumerate(y + h):
            out[r].append(row.unsqueeze(0))
    return [torch.cat(o) for o in out]


def main():
    args = argparse.ArgumentParser()
    args.add_argument("--bits", type=int, choices=(8, 16), default=16, help="of the cache")
    bits = args.parse_args().bits
    dev = torch.device("cuda:0")
    layer = random_layer(dev)
    cache = PagedCache(64, 16, layer.kv_heads, layer.dim, bits, dev)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    prompts = [torch.randn(n, 1024, generator=g, device=dev).bfloat16() for n in (300, 17, 130)]
    steps = [torch.randn(3, 1024, generator=g, device=dev).bfloat16() for _ in range(4)]
    for r, o in enumerate(serve(layer, cache, prompts, [0, 2, 1], steps)):
        print(f"request {r}: {len(o)} tokens, last output's rms "
              f"{o[-1].float().square().mean().sqrt().item():.4f}, "
              f"{len(cache.pages[r])} pages of {cache.page}")


if __name__ == "__main__":
    main()
