"""One adapted transformer layer for a mixed serving batch, run through the library: chats with a few new
rows each beside a decision prompt whose rows take the adapter.

    h += x;  y = norm(h)                          add_rms_norm
    q, k, v = y Wqkv^T (+ adapter)                LoraLinear
    q, k turned by position; k, v to the cache    kv_append
    o = attention of the new rows over the cache  PagedAttention
    h += o Wo^T (+ adapter);  y = norm(h)         LoraLinear, add_rms_norm
    x = (silu(y Wg^T) * y Wu^T) Wd^T (+ adapter)  LoraLinear

    python examples/adapted_layer.py [--steps 20] [--graph]

prints the time of one layer's step for six chats with eight draft rows each (48 rows) and of the same
batch with a 2,048-row prompt chunk. The backbone around it, and the product of the gate with the up
projection, stay with the caller (a torch expression here).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixed_lora_projection_gb300 import LoraLinear, PagedAttention, add_rms_norm, kv_append  # noqa: E402

BF16 = torch.bfloat16


class AdaptedLayer:
    """Weights of one layer and its handles. ``adapters``: {projection: (A, B, scale)} of adapter 1."""

    def __init__(self, hidden, heads, kv_heads, head_dim, mlp, rank, page_size, max_tokens, max_seqs, device, seed=0,
                 rot=64, positions=32768, window=0, sinks=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.mlp = hidden, heads, kv_heads, head_dim, mlp
        self.window, self.sinks = window, sinks
        shapes = {"qkv": (hidden, (heads + 2 * kv_heads) * head_dim), "o": (heads * head_dim, hidden),
                  "gate_up": (hidden, 2 * mlp), "down": (mlp, hidden)}
        self.W, self.adapters, self.linear = {}, {}, {}
        for name, (d_in, d_out) in shapes.items():
            def draw(*shape, var):
                return (torch.randn(shape, generator=g, device=device) * var ** 0.5).to(BF16)
            self.W[name] = draw(d_out, d_in, var=1 / d_in)
            self.adapters[name] = (draw(rank, d_in, var=1 / d_in), draw(d_out, rank, var=0.25 / rank), 1.0)
            self.linear[name] = LoraLinear(d_in, d_out, rank, max_tokens, max_seqs, device)
        self.norm_in = torch.rand(hidden, generator=g, device=device).to(BF16)          # weight - 1
        self.norm_mlp = torch.rand(hidden, generator=g, device=device).to(BF16)
        half = rot // 2
        freq = 1e6 ** (-torch.arange(half, device=device, dtype=torch.float64) / half)
        angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * freq
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.attention = PagedAttention(heads, kv_heads, head_dim, page_size, max_tokens, max_seqs, device)

    def close(self):
        for p in self.linear.values():
            p.close()
        self.attention.close()

    def project(self, name, x, offsets, ids):
        a, b, s = self.adapters[name]
        return self.linear[name].forward(x, offsets, ids, self.W[name], [a], [b], [s])

    def forward(self, x, h, offsets, ids, kv_lens, block_table, k_cache, v_cache):
        """(x, h) after the layer: x [T, hidden] is the layer's input not yet added to the residual h."""
        H, KV, D, T = self.heads, self.kv_heads, self.head_dim, x.shape[0]
        y, h = add_rms_norm(x, self.norm_in, h, weight_offset=1.0)
        qkv = self.project("qkv", y, offsets, ids).view(T, H + 2 * KV, D)
        q = kv_append(qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:], offsets, kv_lens, block_table, k_cache, v_cache,
                      self.cos, self.sin, q_out=qkv[:, :H])
        o = self.attention.forward(q, k_cache, v_cache, offsets, kv_lens, block_table, window=self.window,
                                   sinks=self.sinks, out=torch.empty(T, H, D, dtype=BF16, device=x.device))
        y, h = add_rms_norm(self.project("o", o.view(T, H * D), offsets, ids), self.norm_mlp, h, weight_offset=1.0)
        gate, up = self.project("gate_up", y, offsets, ids).split(self.mlp, -1)
        return self.project("down", torch.nn.functional.silu(gate) * up, offsets, ids), h


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--graph", action="store_true", help="replay the step from a CUDA graph")
    args = ap.parse_args()
    dev = torch.device("cuda", 0)
    chats, draft, context, page = 6, 8, 16384, 64
    layer = AdaptedLayer(5120, 24, 12, 256, 17408, 256, page, 48 + 2048, 16, dev)
    for name, chunk in (("48 decode rows", 0), ("48 decode rows and a 2,048-row prompt chunk", 2048)):
        rows = [draft] * chats + ([chunk] if chunk else [])
        offsets = [0]
        for n in rows:
            offsets.append(offsets[-1] + n)
        ids = [0] * chats + ([1] if chunk else [])
        lens = [context - 1000 * i for i in range(chats)] + ([8192] if chunk else [])
        per = -(-max(lens) // page)
        table = torch.randperm(per * len(rows), device=dev).to(torch.int32).view(len(rows), per)
        cache = [torch.randn(per * len(rows), page, 12, 256, device=dev, dtype=BF16) for _ in range(2)]
        kv = torch.tensor(lens, dtype=torch.int32, device=dev)
        x = torch.randn(offsets[-1], 5120, device=dev).to(BF16)
        h = torch.randn(offsets[-1], 5120, device=dev).to(BF16)

        def step():
            return layer.forward(x, h, offsets, ids, kv, table, *cache)

        for _ in range(3):
            step()
        run = step
        if args.graph:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            run = graph.replay
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(args.steps):
            run()
        b.record()
        b.synchronize()
        print(f"{name}: {a.elapsed_time(b) / args.steps * 1e3:.1f} us a layer")
    assert layer.attention.status() == 0
    layer.close()


if __name__ == "__main__":
    main()
