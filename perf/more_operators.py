"""Cases of the 8-bit path of an adapted layer and of what reads its answer: projections of 8-bit
activations through an 8-bit base weight with a scale for each block of 128 (adapters beside it in
bf16), the product of the gate with the up projection (bf16 or 8-bit output), activations and weights
brought to 8 bits, and log probabilities of given tokens with entropy and top alternatives.

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or, where
``own`` is set, through this package's entry points. ``exact`` computes it in 64 bits.

Sizes: 5,120 hidden features, 6,144 attention outputs, 12,288 fused qkv outputs, 34,816 gate and up
outputs and 17,408 down inputs are the projections this library runs, with adapters of rank 256; 48
rows are six chats with eight draft rows each, 16,384 tokens a long prompt. Vocabularies are generic.
"""
import math
import random

import torch

own = False

FP8_MAX = 448.0             # largest e4m3 value
SCALE_FLOOR = 2.0 ** -100   # an all-zero group or block has this scale


# ------------------------------------------------------------------------------ cases

def _project(name, d_in, d_out, rank, rows, ids):
    """``rows``, ``ids``: the request segments' lengths and adapters, as texts."""
    c = {"kind": "project", "d_in": d_in, "d_out": d_out, "rank": rank, "rows": " ".join(map(str, rows)),
         "ids": " ".join(map(str, ids))}
    return dict(c, name=name) if name else c


def _gate(name, rows, width, out):
    c = {"kind": "gate", "rows": rows, "width": width, "out": out}
    return dict(c, name=name) if name else c


def _narrow(name, rows, width, by):
    c = {"kind": "narrow", "rows": rows, "width": width, "by": by}
    return dict(c, name=name) if name else c


def _score(name, rows, vocab, bits, top, temperature, masked):
    c = {"kind": "score", "rows": rows, "vocab": vocab, "bits": bits, "top": top, "temperature": temperature,
         "masked": masked}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one chat's next token through the attention's output projection: latency
        _project("project 1 row", 6144, 5120, 256, [1], [0]),
        # one decode step of six chats with eight draft rows each: the weight's bytes
        _project("project 48 rows", 5120, 34816, 256, [8] * 6, [0] * 6),
        # chats beside two short decision prompts on adapters of their own, odd lengths
        _project("project short prompts", 17408, 5120, 64, [8, 8, 301, 8, 1252], [0, 0, 1, 0, 2]),
        # a long decision prompt, all rows on one adapter
        _project("project 16k prompt", 5120, 5120, 256, [16384], [1]),
        # six chats beside a prompt chunk that takes the adapter
        _project("project mixed batch", 5120, 34816, 256, [8] * 6 + [4096], [0] * 6 + [1]),
        # the same decode step between gate_up and down
        _gate("gate 48 rows", 48, 17408, "group"),
        # a prompt chunk of odd length, for a down projection in bf16
        _gate("gate 4001 rows", 4001, 17408, "bf16"),
        # a prefix tail's attention outputs ahead of their projection
        _narrow("rows 1601 to 8 bits", 1601, 6144, "group"),
        # a weight as it is loaded
        _narrow("weight to 8 bits", 34816, 5120, "block"),
        # one chat's next token with its alternatives: latency
        _score("score 1 row", 1, 131072, 32, 20, 1.0, 0.0),
        # draft rows to verify, part of the vocabulary ruled out
        _score("score 48 rows", 48, 131072, 16, 5, 0.7, 0.5),
        # every token of a prompt chunk, an odd vocabulary
        _score("score 4096 rows", 4096, 100003, 16, 20, 1.0, 0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


SHAPES = [(5120, 12288), (6144, 5120), (5120, 34816), (17408, 5120), (5120, 5120)]


def draw(rng):
    kind = rng.choice(["project", "project", "project", "gate", "narrow", "score", "score"])
    if kind == "project":
        d_in, d_out = rng.choice(SHAPES + [(16 * _log(rng, 8, 1088), 8 * _log(rng, 16, 4352))] * 2)
        most = min(16384, max(1, 4144 * 5120 * 34816 // (d_in * d_out)))
        total = _log(rng, 1, most)
        n = rng.choice([1, 1, 2, 5, 9])
        cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
        rows = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        ids = [rng.choice([0, 0, 1, 1, 2]) for _ in rows]
        return _project(None, d_in, d_out, rng.choice([16, 64, 200, 256]), rows, ids)
    if kind == "gate":
        width = 8 * _log(rng, 16, 2176)
        return _gate(None, _log(rng, 1, max(1, 4001 * 17408 // max(width, 5120))), width,
                     rng.choice(["bf16", "row", "group"]))
    if kind == "narrow":
        by = rng.choice(["row", "group", "block"])
        width = 8 * _log(rng, 16, 2176)
        return _narrow(None, _log(rng, 1, max(1, 34816 * 5120 // max(width, 5120))), width, by)
    vocab = _log(rng, 512, 262144)
    rows = _log(rng, 1, max(1, min(8192, 4096 * 100003 // vocab)))
    return _score(None, rows, vocab, rng.choice([16, 16, 32]), rng.choice([0, 1, 5, 20, 32]),
                  rng.choice([1.0, 1.0, 0.7, 1.5]), rng.choice([0.0, 0.0, 0.5, 0.999]))


def _segments(case):
    rows, ids = [int(v) for v in case["rows"].split()], [int(v) for v in case["ids"].split()]
    offs = [0]
    for n in rows:
        offs.append(offs[-1] + n)
    return offs, ids


# ------------------------------------------------------------------------------ inputs

def _to_groups(x, group):
    """(e4m3 values, scales) of fp32 rows, one scale per ``group`` features."""
    rows, width = x.shape
    n = -(-width // group)
    p = torch.nn.functional.pad(x, (0, n * group - width)).view(rows, n, group)
    scales = (p.abs().amax(-1) * (1.0 / FP8_MAX)).clamp(min=SCALE_FLOOR)
    q = (p * (1.0 / scales)[..., None]).clamp(-FP8_MAX, FP8_MAX).view(rows, -1)[:, :width]
    return q.to(torch.float8_e4m3fn), scales


def _to_blocks(w):
    """(e4m3 values, scales) of an fp32 matrix, one scale per block of 128 x 128."""
    rows, cols = w.shape
    nr, nc = -(-rows // 128), -(-cols // 128)
    p = torch.nn.functional.pad(w, (0, nc * 128 - cols, 0, nr * 128 - rows)).view(nr, 128, nc, 128)
    scales = (p.abs().amax((1, 3)) * (1.0 / FP8_MAX)).clamp(min=SCALE_FLOOR)
    q = (p * (1.0 / scales)[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).view(nr * 128, -1)[:rows, :cols]
    return q.to(torch.float8_e4m3fn), scales


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(bf16)

    def activations(rows, width):
        # normal features, of which one in 64 is some ten times as large as the others
        loud = 1 + 9 * (torch.rand(width, generator=g, device=dev) < 1 / 64).float()
        return (torch.randn(rows, width, generator=g, device=dev) * loud).to(bf16)

    s = {"case": case}
    if case["kind"] == "project":
        d_in, d_out, rank = case["d_in"], case["d_out"], case["rank"]
        offs, ids = _segments(case)
        x = activations(offs[-1], d_in)
        s["offsets"], s["ids"] = offs, ids
        s["x8"], s["xs"] = _to_groups(x.float(), 128)
        s["x"] = x if any(ids) else None
        s["w8"], s["ws"] = _to_blocks(normal(d_out, d_in, std=d_in ** -0.5).float())
        s["a"] = [normal(rank, d_in, std=d_in ** -0.5) for _ in range(max(ids))]
        s["b"] = [normal(d_out, rank, std=0.5 * rank ** -0.5) for _ in range(max(ids))]
        s["scales"] = [1.0, 0.5][:max(ids)]
        if own:
            from mixed_lora_projection_gb300 import LoraLinear
            s["linear"] = LoraLinear(d_in, d_out, rank, max(offs[-1], 1), len(ids))
    elif case["kind"] == "gate":
        s["x"] = normal(case["rows"], 2 * case["width"], std=2.0)
    elif case["kind"] == "narrow":
        rows, width = case["rows"], case["width"]
        s["x"] = normal(rows, width, std=width ** -0.5) if case["by"] == "block" else activations(rows, width)
    else:
        rows, vocab = case["rows"], case["vocab"]
        # rows of a projection whose outputs are padded to a multiple of 8
        x = torch.empty(rows, -(-vocab // 8) * 8, device=dev, dtype=bf16 if case["bits"] == 16 else torch.float32)
        x = x[:, :vocab]
        x.copy_(torch.randn(rows, vocab, generator=g, device=dev) * 2.5)
        # four likely tokens a row, one in each quarter of the vocabulary
        top = torch.randint(vocab // 4, (rows, 4), generator=g, device=dev) + torch.arange(4, device=dev) * (vocab // 4)
        x.scatter_add_(1, top, (torch.rand(rows, 4, generator=g, device=dev) * 14).to(x.dtype))
        if case["masked"]:
            x.masked_fill_(torch.rand(vocab, generator=g, device=dev) < case["masked"], -math.inf)
            x[:, 0] = 1.0
        rest = torch.randint(vocab, (rows,), generator=g, device=dev)
        s["tokens"] = torch.where(torch.rand(rows, generator=g, device=dev) < 0.7, x.argmax(-1), rest)
        s["logits"] = x
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"project": _own_project, "gate": _own_gate, "narrow": _own_narrow, "score": _own_score}[kind](state)
    return {"project": _plain_project, "gate": _plain_gate, "narrow": _plain_narrow, "score": _plain_score}[kind](state)


def _own_project(s):
    return s["linear"].forward_fp8(s["x8"], s["xs"], s["offsets"], s["ids"], s["w8"], s["ws"], s["a"], s["b"],
                                   s["scales"], x=s["x"])


def _plain_project(s):
    width = s["x8"].shape[1]
    x = s["x8"].float() * s["xs"].repeat_interleave(128, 1)[:, :width]
    w = s["w8"].float() * s["ws"].repeat_interleave(128, 0)[:len(s["w8"])].repeat_interleave(128, 1)[:, :width]
    y = x @ w.T
    for lo, hi, a in zip(s["offsets"], s["offsets"][1:], s["ids"]):
        if a:
            u = s["x"][lo:hi].float() @ s["a"][a - 1].float().T * s["scales"][a - 1]
            y[lo:hi] += u @ s["b"][a - 1].float().T
    return y.to(torch.bfloat16)


def _own_gate(s):
    from mixed_lora_projection_gb300 import silu_mul, silu_mul_fp8
    out = s["case"]["out"]
    if out == "bf16":
        return silu_mul(s["x"])
    q, scales = silu_mul_fp8(s["x"], group=128 if out == "group" else 0)
    return {"y": q, "scales": scales}


def _plain_gate(s):
    c = s["case"]
    gate, up = s["x"][:, :c["width"]].float(), s["x"][:, c["width"]:].float()
    y = gate / (1 + torch.exp(-gate)) * up
    if c["out"] == "bf16":
        return y.to(torch.bfloat16)
    q, scales = _to_groups(y, 128 if c["out"] == "group" else c["width"])
    return {"y": q, "scales": scales}


def _own_narrow(s):
    from mixed_lora_projection_gb300 import fp8_blocks, fp8_rows
    by = s["case"]["by"]
    q, scales = fp8_blocks(s["x"]) if by == "block" else fp8_rows(s["x"], group=128 if by == "group" else 0)
    return {"q": q, "scales": scales}


def _plain_narrow(s):
    c = s["case"]
    x = s["x"].float()
    q, scales = _to_blocks(x) if c["by"] == "block" else _to_groups(x, 128 if c["by"] == "group" else c["width"])
    return {"q": q, "scales": scales}


def _own_score(s):
    from mixed_lora_projection_gb300 import token_logprobs
    c = s["case"]
    r = token_logprobs(s["logits"], s["tokens"], top=c["top"], temperature=c["temperature"])
    return {"logprobs": r.logprobs, "ranks": r.ranks, "entropy": r.entropy, "top_logprobs": r.top_logprobs,
            "top_tokens": r.top_tokens}


def _plain_score(s):
    c = s["case"]
    x, tokens = s["logits"].float(), s["tokens"][:, None]
    z = x * (1.0 / c["temperature"])
    z = z - z.amax(-1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    entropy = (total.log() - (e * z.clamp(min=-1e4)).sum(-1, keepdim=True) / total)[:, 0]
    z -= total.log()
    mine = x.gather(1, tokens)
    index = torch.arange(c["vocab"], device=x.device)
    ranks = ((x > mine) | ((x == mine) & (index < tokens))).sum(-1)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
    return {"logprobs": z.gather(1, tokens)[:, 0], "ranks": ranks.to(torch.int32), "entropy": entropy,
            "top_logprobs": z.gather(1, order), "top_tokens": order.to(torch.int32)}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["kind"] == "project":
        d_in = case["d_in"]
        x, w = s["x8"].to(f64), s["w8"].to(f64)
        block = torch.arange(len(w), device=w.device) // 128
        y = torch.zeros(len(x), len(w), dtype=f64, device=w.device)
        for i, k in enumerate(range(0, d_in, 128)):
            x[:, k:k + 128] *= s["xs"][:, i:i + 1].to(f64)
            w[:, k:k + 128] *= s["ws"][block, i:i + 1].to(f64)
        torch.matmul(x, w.T, out=y)
        for i, a in enumerate(s["ids"]):
            r = slice(s["offsets"][i], s["offsets"][i + 1])
            if a:
                y[r].addmm_(s["x"][r].to(f64) @ s["a"][a - 1].to(f64).T, s["b"][a - 1].to(f64).T, alpha=s["scales"][a - 1])
        return y
    if case["kind"] in ("gate", "narrow"):
        x, by = s["x"].to(f64), case.get("by", case.get("out"))
        if case["kind"] == "gate":
            gate, up = x.chunk(2, -1)
            x = gate * torch.sigmoid(gate) * up
            if by == "bf16":
                return x
        rows, width = x.shape
        if by == "block":
            scales = torch.stack([torch.stack([t.abs().amax() for t in r.split(128, 1)]) for r in x.split(128, 0)])
        else:
            scales = torch.stack([t.abs().amax(-1) for t in x.split(128 if by == "group" else width, 1)], -1)
        scales = scales.clamp(min=FP8_MAX * SCALE_FLOOR) / FP8_MAX
        r = torch.arange(rows, device=x.device) // (128 if by == "block" else 1)
        k = torch.arange(width, device=x.device) // (width if by == "row" else 128)
        return {"y" if case["kind"] == "gate" else "q": x / scales[r][:, k], "scales": scales}
    parts = []
    for lo in range(0, case["rows"], 512):
        x, t = s["logits"][lo:lo + 512].to(f64), s["tokens"][lo:lo + 512, None]
        lp = torch.log_softmax(x / case["temperature"], -1)
        mine = x.gather(1, t)
        before = (x == mine) & (torch.arange(case["vocab"], device=x.device) < t)
        value, order = torch.sort(-x, dim=-1, stable=True)
        order = order[:, :case["top"]]
        parts.append({"logprobs": lp.gather(1, t)[:, 0], "ranks": ((x > mine).sum(-1) + before.sum(-1)).to(torch.int32),
                      "entropy": torch.special.entr(lp.exp()).sum(-1), "top_logprobs": lp.gather(1, order),
                      "top_tokens": order.to(torch.int32)})
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


# ------------------------------------------------------------------------------ work

def work(case):
    if case["kind"] == "project":
        d_in, d_out, rank = case["d_in"], case["d_out"], case["rank"]
        offs, ids = _segments(case)
        rows = offs[-1]
        lens = [b - a for a, b in zip(offs, offs[1:])]
        with_adapter = sum(n for n, a in zip(lens, ids) if a)
        adapters = len({a for n, a in zip(lens, ids) if a and n})
        k = -(-d_in // 128)
        return {"bytes": rows * (d_in + 4 * k) + d_out * d_in + 4 * k * -(-d_out // 128) + 2 * rows * d_out
                + 2 * with_adapter * d_in + 2 * adapters * rank * (d_in + d_out),
                "flops": 2 * rows * d_in * d_out + 2 * with_adapter * rank * (d_in + d_out)}
    if case["kind"] in ("gate", "narrow"):
        rows, width = case["rows"], case["width"]
        by = case.get("by", case.get("out"))
        scales = {"bf16": 0, "row": rows, "group": rows * -(-width // 128), "block": -(-rows // 128) * -(-width // 128)}[by]
        out = rows * width * (2 if by == "bf16" else 1) + 4 * scales
        gate = case["kind"] == "gate"
        return {"bytes": rows * width * (4 if gate else 2) + out, "flops": rows * width * (6 if gate else 3)}
    rows, vocab = case["rows"], case["vocab"]
    return {"bytes": rows * (vocab * case["bits"] // 8 + 8 + 12 + 8 * case["top"]), "flops": rows * vocab * 6}
