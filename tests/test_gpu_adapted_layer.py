"""The example's layer (examples/adapted_layer.py) on a GPU: the operators together, step after step, against
the same layer in 64 bits on the bf16 values that each operator hands to the next."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F64, BF16 = torch.float64, torch.bfloat16


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("adapted_layer", os.path.join(ROOT, "examples", "adapted_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Plain:
    """The layer by its formulas in 64 bits, each operator's output rounded to bf16 as the library's are."""

    def __init__(self, layer):
        self.l = layer
        self.k, self.v = {}, {}

    def project(self, name, x, ids):
        a, b, s = (t.to(F64) if torch.is_tensor(t) else t for t in self.l.adapters[name])
        y = x.to(F64) @ self.l.W[name].to(F64).T
        delta = s * (x.to(F64) @ a.T) @ b.T
        return (y + delta * torch.tensor(ids, device=x.device, dtype=F64)[:, None]).to(BF16)

    def norm(self, h, w):
        return (h / ((h * h).mean(-1, keepdim=True) + 1e-6).sqrt() * (w.to(F64) + 1)).to(BF16)

    def turn(self, x, pos):
        c, s = self.l.cos[pos].to(F64)[:, None], self.l.sin[pos].to(F64)[:, None]
        n = c.shape[-1]
        x = x.to(F64)
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * n:]], -1).to(BF16)

    def step(self, x, h, offsets, seg_ids, lens):
        L = self.l
        H, KV, D = L.heads, L.kv_heads, L.head_dim
        ids = [i for s, i in enumerate(seg_ids) for _ in range(offsets[s + 1] - offsets[s])]
        h = x.to(F64) + h.to(F64)
        qkv = self.project("qkv", self.norm(h, L.norm_in), ids).view(-1, H + 2 * KV, D)
        h = h.to(BF16)
        o = torch.zeros(x.shape[0], H, D, dtype=F64, device=x.device)
        for s, n in enumerate(lens):
            a, b = offsets[s], offsets[s + 1]
            pos = torch.arange(n - (b - a), n, device=x.device)
            q, k = self.turn(qkv[a:b, :H], pos), self.turn(qkv[a:b, H:H + KV], pos)
            self.k[s] = torch.cat([self.k[s], k]) if s in self.k else k
            self.v[s] = torch.cat([self.v[s], qkv[a:b, H + KV:]]) if s in self.v else qkv[a:b, H + KV:]
            sc = torch.einsum("qhgd,khd->hgqk", q.to(F64).view(b - a, KV, H // KV, D), self.k[s].to(F64)) * D ** -0.5
            j, p = torch.arange(n, device=x.device)[None], pos[:, None]
            seen = (j <= p) & ((j > p - L.window) | (j < L.sinks) if L.window else True)
            w = torch.softmax(sc.masked_fill(~seen, float("-inf")), -1)
            o[a:b] = torch.einsum("hgqk,khd->qhgd", w, self.v[s].to(F64)).reshape(b - a, H, D)
        h = self.project("o", o.to(BF16).view(-1, H * D), ids).to(F64) + h.to(F64)
        gu = self.project("gate_up", self.norm(h, L.norm_mlp), ids)
        gate, up = gu.split(L.mlp, -1)
        return self.project("down", torch.nn.functional.silu(gate) * up, ids), h.to(BF16)


@pytest.mark.parametrize("dim,window,sinks", [(64, 0, 0), (128, 100, 4), (256, 0, 0)])
def test_layer_steps(example, dim, window, sinks):
    # three prompts of odd lengths, then steps of one and of four new rows; the second sequence takes the adapter
    heads, kv_heads, page, hidden, mlp = 6, 2, 32, 512, 768
    dev = torch.device("cuda", torch.cuda.current_device())
    layer = example.AdaptedLayer(hidden, heads, kv_heads, dim, mlp, 32, page, 700, 4, dev, rot=32, positions=1000, window=window,
                                 sinks=sinks)
    plain = Plain(layer)
    g = torch.Generator(device=dev)
    g.manual_seed(dim)
    per = 20
    table = torch.randperm(3 * per, generator=g, device=dev).to(torch.int32).view(3, per)
    caches = [torch.full((3 * per, page, kv_heads, dim), float("nan"), dtype=BF16, device=dev) for _ in range(2)]
    lens = [0, 0, 0]
    for rows in ([130, 301, 5], [1, 1, 1], [4, 0, 4], [1, 60, 1]):
        offsets = [0]
        for n in rows:
            offsets.append(offsets[-1] + n)
        lens = [a + b for a, b in zip(lens, rows)]
        x = torch.randn(offsets[-1], hidden, generator=g, device=dev).to(BF16)
        h = torch.randn(offsets[-1], hidden, generator=g, device=dev).to(BF16)
        got_x, got_h = layer.forward(x, h, offsets, [0, 1, 0], torch.tensor(lens, dtype=torch.int32, device=dev), table, *caches)
        ref_x, ref_h = plain.step(x, h, offsets, [0, 1, 0], lens)
        # Each operator's output is bf16 (half a unit: 2^-8); a value that falls to the other side of a rounding
        # differs by one unit, 2^-7, and passes through the four projections that follow, where such errors add up
        # as independent ones: 2 * 2^-7 of the tensor's norm bounds six of them, sqrt(6) 2^-8 < 2^-6.6, with room.
        for got, ref in ((got_x, ref_x), (got_h, ref_h)):
            rel = (got.to(F64) - ref.to(F64)).norm() / ref.to(F64).norm()
            assert rel < 2.0 ** -6, rel
    assert layer.attention.status() == 0
    layer.close()
