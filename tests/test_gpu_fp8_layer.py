"""The example's layer (examples/adapted_layer.py) with activations and weights in 8 bits, and the log probabilities that it
reads from a head, against the same layer in 64 bits on the values that each operator hands to the next."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F64, BF16, FP8 = torch.float64, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("adapted_layer_fp8", os.path.join(ROOT, "examples", "adapted_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def blocks(q, s):
    """A weight of fp8_blocks in 64 bits."""
    w = s.to(F64).repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.to(F64) * w


def rows8(x):
    """x (64 bits) by rows and 128 features in 8 bits, as the operators round it."""
    out = torch.empty_like(x)
    for k in range(0, x.shape[1], 128):
        part = x[:, k:k + 128]
        s = (part.abs().amax(-1, keepdim=True) / 448).clamp_min(2.0 ** -100).float().to(F64)
        out[:, k:k + 128] = (part / s).float().to(FP8).to(F64) * s
    return out


class Plain:
    def __init__(self, layer):
        self.l = layer
        self.k, self.v = {}, {}

    def project(self, name, x, ids):
        a, b, s = (t.to(F64) if torch.is_tensor(t) else t for t in self.l.adapters[name])
        y = rows8(x) @ blocks(*self.l.W8[name]).T
        delta = s * (x.to(BF16).to(F64) @ a.T) @ b.T
        return (y + delta * torch.tensor(ids, device=x.device, dtype=F64)[:, None]).to(BF16).to(F64)

    def norm(self, h, w):
        return h / ((h * h).mean(-1, keepdim=True) + 1e-6).sqrt() * (w.to(F64) + 1)

    def turn(self, x, pos):
        c, s = self.l.cos[pos].to(F64)[:, None], self.l.sin[pos].to(F64)[:, None]
        n = c.shape[-1]
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * n:]], -1).to(BF16).to(F64)

    def step(self, x, h, offsets, seg_ids, lens):
        L = self.l
        H, KV, D = L.heads, L.kv_heads, L.head_dim
        ids = [i for s, i in enumerate(seg_ids) for _ in range(offsets[s + 1] - offsets[s])]
        h = x.to(F64) + h.to(F64)
        qkv = self.project("qkv", self.norm(h, L.norm_in), ids).view(-1, H + 2 * KV, D)
        h = h.to(BF16).to(F64)
        o = torch.zeros(x.shape[0], H, D, dtype=F64, device=x.device)
        for s, n in enumerate(lens):
            a, b = offsets[s], offsets[s + 1]
            pos = torch.arange(n - (b - a), n, device=x.device)
            q, k = self.turn(qkv[a:b, :H], pos), self.turn(qkv[a:b, H:H + KV], pos)
            self.k[s] = torch.cat([self.k[s], k]) if s in self.k else k
            self.v[s] = torch.cat([self.v[s], qkv[a:b, H + KV:]]) if s in self.v else qkv[a:b, H + KV:]
            sc = torch.einsum("qhgd,khd->hgqk", q.view(b - a, KV, H // KV, D), self.k[s]) * D ** -0.5
            w = torch.softmax(sc.masked_fill(torch.arange(n, device=x.device)[None] > pos[:, None], float("-inf")), -1)
            o[a:b] = torch.einsum("hgqk,khd->qhgd", w, self.v[s]).reshape(b - a, H, D)
        h = self.project("o", o.to(BF16).to(F64).view(-1, H * D), ids) + h
        gate, up = self.project("gate_up", self.norm(h, L.norm_mlp), ids).split(L.mlp, -1)
        return self.project("down", torch.nn.functional.silu(gate) * up, ids), h.to(BF16).to(F64)


def build(example, **more):
    dev = torch.device("cuda", torch.cuda.current_device())
    return example.AdaptedLayer(512, 6, 2, 64, 768, 32, 32, 700, 4, dev, rot=32, positions=1000, fp8=True, **more)


def test_layer_steps_in_8_bits(example):
    layer = build(example, vocab=1008)
    plain = Plain(layer)
    dev = layer.norm_in.device
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    table = torch.randperm(60, generator=g, device=dev).to(torch.int32).view(3, 20)
    caches = [torch.full((60, 32, 2, 64), float("nan"), dtype=BF16, device=dev) for _ in range(2)]
    lens = [0, 0, 0]
    for rows in ([130, 301, 5], [1, 1, 1], [4, 0, 4], [1, 60, 1]):
        offsets = [0]
        for n in rows:
            offsets.append(offsets[-1] + n)
        lens = [a + b for a, b in zip(lens, rows)]
        x = torch.randn(offsets[-1], 512, generator=g, device=dev).to(BF16)
        h = torch.randn(offsets[-1], 512, generator=g, device=dev).to(BF16)
        seg_ids = [0, 1, 0]
        got_x, got_h = layer.forward(x, h, offsets, seg_ids, torch.tensor(lens, dtype=torch.int32, device=dev), table, *caches)
        ref_x, ref_h = plain.step(x, h, offsets, seg_ids, lens)
        # Both sides round the same values to 8 bits, so that a result differs where a value's bf16 or fp32 error carries it
        # over a rounding: by one unit of e4m3, at most 2^-3 of it. An input whose bf16 differs by e of itself is carried over
        # with the chance 2 e / 2^-3 at most, so that the square of the change it makes in the sum is at most
        # (2 e / 2^-3) (2^-3)^2 = e 2^-2 of its share: relative to the norm sqrt(e) / 2, for e <= 2^-8 at most 2^-5 a
        # projection. Four projections follow one another, added as independent errors: 2 * 2^-5 = 2^-4; h holds two of them
        # and the layer's own input beside them.
        for got, ref in ((got_x, ref_x), (got_h, ref_h)):
            rel = (got.to(F64) - ref).norm() / ref.norm()
            assert rel < 2.0 ** -4, rel
        last = torch.tensor([offsets[s + 1] - 1 for s in range(3) if rows[s]], device=dev)
        tokens = torch.randint(1008, (len(last),), generator=g, device=dev)
        got = layer.score(got_x, got_h, last, tokens, top=5)
        y = plain.norm(got_x[last].to(F64) + got_h[last].to(F64), layer.norm_out)
        lp = torch.log_softmax(plain.project("head", y, [0] * len(last)), -1)
        # the same bound on the logits' norm: their error is 2^-5 of it for one projection, a row's sqrt(1008) times its mean
        bound = 2.0 ** -5 * lp.exp().new_tensor(1008.0).sqrt() * plain.project("head", y, [0] * len(last)).square().mean(-1).sqrt()
        assert ((got.logprobs.to(F64) - lp.gather(1, tokens[:, None])[:, 0]).abs() <= 2 * bound).all()
        assert got.top_tokens.shape == (len(last), 5) and (got.top_logprobs[:, :-1] >= got.top_logprobs[:, 1:]).all()
    assert layer.attention.status() == 0
    layer.close()


def test_captured_step_in_8_bits(example):
    # a captured step of eight rows reads new inputs and lengths at every replay, and equals the eager one bit for bit
    layer = build(example)
    dev = layer.norm_in.device
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    table = torch.randperm(40, generator=g, device=dev).to(torch.int32).view(2, 20)
    caches = [torch.randn(40, 32, 2, 64, generator=g, device=dev).to(BF16) for _ in range(2)]
    copies = [c.clone() for c in caches]
    x, h = (torch.randn(8, 512, generator=g, device=dev).to(BF16) for _ in range(2))
    kv = torch.tensor([9, 300], dtype=torch.int32, device=dev)
    step = lambda c: layer.forward(x, h, [0, 4, 8], [0, 1], kv, table, *c)  # noqa: E731
    step([c.clone() for c in caches])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches)
    for i in range(3):
        x.copy_(torch.randn(8, 512, generator=g, device=dev))
        kv.add_(4)
        graph.replay()
        want = step(copies)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    layer.close()
