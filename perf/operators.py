"""Cases of the operators that stand between an adapted layer's projections: the residual's
addition with the root-mean-square norm (bf16 or 8-bit output), the append of new keys and
values to a paged cache, attention of a few new tokens per request over that cache, and
attention of whole prompts with a sliding window and first tokens that stay visible.

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or, where
``own`` is set, through this package's entry points. ``exact`` computes it in 64 bits.

Sizes: 5,120 hidden features, 6,144 attention outputs and 12,288 fused qkv outputs are the
projections this library runs (24 query heads and 12 key/value heads of 256, or heads of 128);
48 rows are six chats with eight draft rows each; 16,384 tokens are a long prompt; 1,552 tokens
are the cache block of a hybrid backbone, 16 and 64 the usual page sizes.
"""
import math
import random

import torch

own = False

FP8_MAX = 448.0             # largest e4m3 value
SCALE_FLOOR = 2.0 ** -100   # an all-zero row or group has this scale


# ------------------------------------------------------------------------------ cases

def _norm(name, rows, width, out, offset=0.0):
    c = {"kind": "norm", "rows": rows, "width": width, "out": out, "offset": offset}
    return dict(c, name=name) if name else c


def _append(name, heads, kv_heads, dim, page, seqs, q, kv, ragged, rot):
    c = {"kind": "append", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "seqs": seqs,
         "q": q, "kv": kv, "ragged": ragged, "rot": rot}
    return dict(c, name=name) if name else c


def _attn(name, heads, kv_heads, dim, page, seqs, q, kv, ragged, window=0, sinks=0):
    c = {"kind": "attention", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "seqs": seqs,
         "q": q, "kv": kv, "ragged": ragged, "window": window, "sinks": sinks}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of six chats with eight draft rows each: latency
        _norm("norm 48 rows", 48, 5120, "bf16"),
        # a long decision prompt ahead of projections that take 8-bit activations
        _norm("norm 16k to 8 bits", 16384, 5120, "row", 1.0),
        # a prefix tail, one scale per 128 features, a width that is no multiple of 128
        _norm("norm 1601 groups of 8 bits", 1601, 5128, "group"),
        # the six chats' new keys and values go into cache blocks of 1,552 tokens
        _append("append 6 x 8 rows", 24, 12, 256, 1552, 6, 8, 20000, 3, 64),
        # a whole prompt goes into the cache
        _append("append 16k prompt", 24, 12, 256, 64, 1, 16384, 16384, 0, 64),
        # one chat that has just begun: latency
        _attn("decode 1 chat", 24, 12, 256, 16, 1, 1, 517, 0),
        # six chats of uneven length, cache blocks of 1,552 tokens
        _attn("decode 6 chats", 24, 12, 256, 1552, 6, 1, 32768, 5),
        # the same with eight draft rows to verify, six query heads to a key/value head
        _attn("verify 6 x 8 rows", 24, 4, 256, 64, 6, 8, 20000, 7),
        # a full batch of chats
        _attn("decode 64 chats", 48, 8, 128, 64, 64, 1, 16384, 9),
        # a long prompt in one pass, window and first tokens
        _attn("prompt 16k window", 24, 12, 256, 64, 1, 16384, 16384, 0, 4096, 4),
        # a chunk of a prompt whose beginning is in the cache already
        _attn("chunk 4096 of 16k", 48, 8, 128, 16, 1, 4096, 16384, 0),
        # several prompts of odd lengths, one key/value head per query head, a window no page divides
        _attn("prompts odd window", 16, 16, 64, 16, 5, 3001, 3501, 11, 1000, 5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(24, 12, 256), (24, 4, 256), (48, 8, 128), (48, 48, 128), (32, 1, 128), (16, 16, 64), (40, 5, 64)]


def draw(rng):
    kind = rng.choice(["norm", "append", "decode", "decode", "prompt", "prompt"])
    if kind == "norm":
        width = 8 * _log(rng, 8, 2176)                       # 64 .. 17,408
        rows = _log(rng, 1, max(1, 16384 * 5120 // max(width, 5120)))
        return _norm(None, rows, width, rng.choice(["bf16", "row", "group"]), rng.choice([0.0, 1.0]))
    heads, kv_heads, dim = rng.choice(HEADS)
    page = rng.choice([16, 48, 64, 128, 1552])
    if kind == "append":
        seqs = _log(rng, 1, 64)
        q = _log(rng, 1, 16384 // seqs)
        kv = q + _log(rng, 1, max(2, 32768 // seqs)) - 1
        return _append(None, heads, kv_heads, dim, page, seqs, q, kv, rng.randrange(1, 1000),
                       rng.choice([0, 32, dim // 2, dim]))
    window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 16, 8192), rng.choice([0, 1, 4, 130]))])
    if kind == "decode":
        seqs = _log(rng, 1, 64)
        q = rng.choice([1, 1, 1, 2, 5, 8])
        most = min(32768, 16384 * 64 * 8 * 128 // (seqs * kv_heads * dim))
        kv = _log(rng, max(8, q), max(16, most))
        return _attn(None, heads, kv_heads, dim, page, seqs, q, kv, rng.randrange(1, 1000), window, sinks)
    seqs = _log(rng, 1, 8)
    q = _log(rng, 9, 16384 // seqs)
    # the plain form holds every score: seqs x heads x q x kv values
    most = min(16384, 16384 * 16384 * 24 // (seqs * heads * q), 4096 * 16384 * 48 * 128 // (seqs * heads * q * dim))
    kv = min(max(q, _log(rng, q, max(q, most))), 16384)
    return _attn(None, heads, kv_heads, dim, page, seqs, min(q, kv), kv, rng.randrange(1, 1000), window, sinks)


def _lens(case):
    """(q_lens, kv_lens): equal ones, or uneven ones that the case's own number fixes."""
    n = case["seqs"]
    if not case["ragged"]:
        return [case["q"]] * n, [case["kv"]] * n
    r = random.Random(case["ragged"])
    q = [case["q"]] + [max(1, int(case["q"] * r.uniform(0.3, 1.0))) for _ in range(n - 1)]
    kv = [case["kv"]] + [max(a, int(case["kv"] * r.uniform(0.05, 1.0))) for a in q[1:]]
    if case["q"] <= 8:                                       # a decode step has one row count
        q = [case["q"]] * n
        kv = [max(a, b) for a, b in zip(q, kv)]
    return q, kv


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=bf16)

    s = {"case": case}
    if case["kind"] == "norm":
        rows, width = case["rows"], case["width"]
        s["x"], s["residual"] = normal(rows, width), normal(rows, width) * 4
        s["weight"] = (torch.rand(width, generator=g, device=dev) + 0.5 - case["offset"]).to(bf16)
        return s
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    q_lens, kv_lens = _lens(case)
    offs = [0]
    for n in q_lens:
        offs.append(offs[-1] + n)
    per = max(-(-n // page) for n in kv_lens)
    need = sum(-(-n // page) for n in kv_lens)
    order = torch.randperm(need, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(case["seqs"], per, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(kv_lens):
        m = -(-n // page)
        table[i, :m] = order[at:at + m]
        at += m
    s.update(q_offsets=offs, q_lens=q_lens, lens=kv_lens, block_table=table,
             kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=dev))
    T = offs[-1]
    if case["kind"] == "append":
        # q, k and v are slices of the fused qkv projection's rows
        y = normal(T, heads + 2 * kv_heads, dim)
        s["q"], s["k"], s["v"] = y[:, :heads], y[:, heads:heads + kv_heads], y[:, heads + kv_heads:]
        s["k_cache"] = torch.zeros(need, page, kv_heads, dim, dtype=bf16, device=dev)
        s["v_cache"] = torch.zeros(need, page, kv_heads, dim, dtype=bf16, device=dev)
        s["cos"] = s["sin"] = None
        if case["rot"]:
            half = case["rot"] // 2
            freq = 1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
            angle = torch.arange(max(kv_lens), device=dev, dtype=torch.float64)[:, None] * freq
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        return s
    s["q"] = normal(T, heads, dim)
    s["k_cache"], s["v_cache"] = normal(need, page, kv_heads, dim), normal(need, page, kv_heads, dim)
    if own:
        from mixed_lora_projection_gb300 import PagedAttention
        s["attn"] = PagedAttention(heads, kv_heads, dim, page, T, case["seqs"])
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"norm": _own_norm, "append": _own_append, "attention": _own_attention}[kind](state)
    return {"norm": _plain_norm, "append": _plain_append, "attention": _plain_attention}[kind](state)


def _own_norm(s):
    from mixed_lora_projection_gb300 import add_rms_norm, add_rms_norm_fp8
    c = s["case"]
    if c["out"] == "bf16":
        y, h = add_rms_norm(s["x"], s["weight"], s["residual"], eps=1e-6, weight_offset=c["offset"])
        return {"y": y, "h": h}
    y, scales, h = add_rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=1e-6, weight_offset=c["offset"],
                                    group=128 if c["out"] == "group" else 0)
    return {"y": y, "scales": scales, "h": h}


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * (s["weight"].float() + c["offset"])
    h = h.to(torch.bfloat16)
    if c["out"] == "bf16":
        return {"y": y.to(torch.bfloat16), "h": h}
    rows, width = y.shape
    group = 128 if c["out"] == "group" else width
    n = -(-width // group)
    padded = y if n * group == width else torch.nn.functional.pad(y, (0, n * group - width))
    padded = padded.view(rows, n, group)
    scales = (padded.abs().amax(-1) * (1.0 / FP8_MAX)).clamp(min=SCALE_FLOOR)
    q = (padded * (1.0 / scales)[..., None]).clamp(-FP8_MAX, FP8_MAX).view(rows, -1)[:, :width]
    return {"y": q.to(torch.float8_e4m3fn), "scales": scales, "h": h}


def _own_append(s):
    from mixed_lora_projection_gb300 import kv_append
    q = kv_append(s["q"], s["k"], s["v"], s["q_offsets"], s["kv_lens"], s["block_table"], s["k_cache"],
                  s["v_cache"], s["cos"], s["sin"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _row_index(s, device):
    """For every new row its sequence and its position in it."""
    q_lens = torch.tensor(s["q_lens"], device=device)
    seq = torch.repeat_interleave(torch.arange(len(s["q_lens"]), device=device), q_lens,
                                  output_size=s["q_offsets"][-1])
    start = torch.tensor(s["q_offsets"][:-1], device=device)
    pos = torch.arange(s["q_offsets"][-1], device=device) - start[seq] + (s["kv_lens"].long() - q_lens)[seq]
    return seq, pos


def _rotate(x, cos, sin):
    half = cos.shape[-1]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    cos, sin = cos[:, None], sin[:, None]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_append(s):
    page = s["case"]["page"]
    seq, pos = _row_index(s, s["q"].device)
    q, k = s["q"].float(), s["k"].float()
    if s["cos"] is not None:
        cos, sin = s["cos"][pos], s["sin"][pos]
        q, k = _rotate(q, cos, sin), _rotate(k, cos, sin)
    where = s["block_table"][seq, pos // page].long()
    s["k_cache"][where, pos % page] = k.to(torch.bfloat16)
    s["v_cache"][where, pos % page] = s["v"]
    return {"q": q.to(torch.bfloat16), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    c = s["case"]
    return s["attn"].forward(s["q"], s["k_cache"], s["v_cache"], s["q_offsets"], s["kv_lens"], s["block_table"],
                             window=c["window"], sinks=c["sinks"])


def _plain_attention(s):
    c = s["case"]
    heads, kv_heads, dim = c["heads"], c["kv_heads"], c["dim"]
    n, most_q, most_kv = c["seqs"], max(s["q_lens"]), max(s["lens"])
    dev = s["q"].device
    seq, pos = _row_index(s, dev)
    local = pos - (s["kv_lens"].long() - torch.tensor(s["q_lens"], device=dev))[seq]
    q = torch.zeros(n, most_q, heads, dim, device=dev)
    q[seq, local] = s["q"].float()
    q = q.view(n, most_q, kv_heads, heads // kv_heads, dim).permute(0, 2, 3, 1, 4).reshape(n, kv_heads, -1, dim)
    k = s["k_cache"][s["block_table"].long()].view(n, -1, kv_heads, dim)[:, :most_kv].permute(0, 2, 3, 1).float()
    p = torch.matmul(q, k)
    del k
    p *= 1.0 / math.sqrt(dim)
    at = torch.zeros(n, most_q, dtype=torch.long, device=dev)
    at[seq, local] = pos
    j, i = torch.arange(most_kv, device=dev), at[:, :, None]
    seen = j <= i
    if c["window"]:
        seen &= (j > i - c["window"]) | (j < c["sinks"])
    p = p.view(n, heads, most_q, most_kv).masked_fill_(~seen[:, None], -math.inf)
    p -= p.amax(-1, keepdim=True)
    p.exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][s["block_table"].long()].view(n, -1, kv_heads, dim)[:, :most_kv].permute(0, 2, 1, 3).float()
    o = torch.matmul(p.view(n, kv_heads, -1, most_kv), v).view(n, heads, most_q, dim) / total
    return o.permute(0, 2, 1, 3)[seq, local].to(torch.bfloat16)


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["kind"] == "norm":
        h = s["x"].to(f64) + s["residual"].to(f64)
        y = h / ((h * h).mean(-1, keepdim=True) + 1e-6).sqrt() * (s["weight"].to(f64) + case["offset"])
        if case["out"] == "bf16":
            return {"y": y, "h": h}
        group = 128 if case["out"] == "group" else case["width"]
        parts = y.split(group, -1)
        scales = torch.stack([t.abs().amax(-1).clamp(min=FP8_MAX * SCALE_FLOOR) / FP8_MAX for t in parts], -1)
        q = torch.cat([t / scales[:, i:i + 1] for i, t in enumerate(parts)], -1)
        return {"y": q, "scales": scales, "h": h}
    q_lens, kv_lens = _lens(case)
    page, dim = case["page"], case["dim"]
    if case["kind"] == "append":
        q, k, v = s["q"].to(f64), s["k"].to(f64), s["v"].to(f64)
        kc, vc = s["k_cache"].to(f64), s["v_cache"].to(f64)
        out, t0 = q.clone(), 0
        half = case["rot"] // 2
        for i, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
            pos = torch.arange(nk - nq, nk, device=q.device)
            kr = k[t0:t0 + nq].clone()
            if half:
                # the cos and sin that a caller hands over are 32-bit inputs
                turn = torch.complex(s["cos"][pos].to(f64), s["sin"][pos].to(f64))[:, None]
                for src in (out[t0:t0 + nq], kr):
                    z = torch.complex(src[..., :half].contiguous(), src[..., half:2 * half].contiguous()) * turn
                    src[..., :half], src[..., half:2 * half] = z.real, z.imag
            slots = s["block_table"][i].long()[pos // page] * page + pos % page
            kc.view(-1, *kc.shape[2:])[slots] = kr
            vc.view(-1, *vc.shape[2:])[slots] = v[t0:t0 + nq]
            t0 += nq
        return {"q": out, "k_cache": kc, "v_cache": vc}
    if sum(a * b for a, b in zip(q_lens, kv_lens)) * case["heads"] * dim > 2e12:
        return None
    out = torch.zeros(sum(q_lens), case["heads"], dim, dtype=f64, device=s["q"].device)
    shared, t0 = case["heads"] // case["kv_heads"], 0
    for i, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        where = torch.arange(nk, device=out.device)
        slots = s["block_table"][i].long()[where // page] * page + where % page
        for h in range(case["kv_heads"]):
            k = s["k_cache"][:, :, h].reshape(-1, dim)[slots].to(f64)
            v = s["v_cache"][:, :, h].reshape(-1, dim)[slots].to(f64)
            for r0 in range(0, nq, 1024):
                r1 = min(nq, r0 + 1024)
                first, last = nk - nq + r0, nk - nq + r1 - 1
                pos = torch.arange(first, last + 1, device=out.device)[:, None]
                # keys that some row of this block sees
                lo = max(0, first - case["window"] + 1) if case["window"] else 0
                cols = torch.cat([where[:min(case["sinks"], lo)], where[lo:last + 1]])
                seen = cols <= pos
                if case["window"]:
                    seen &= (cols > pos - case["window"]) | (cols < case["sinks"])
                qs = s["q"][t0 + r0:t0 + r1, h * shared:(h + 1) * shared].to(f64).transpose(0, 1)
                w = qs @ k[cols].T / math.sqrt(dim)
                w = torch.softmax(w.masked_fill(~seen, -math.inf), -1)
                out[t0 + r0:t0 + r1, h * shared:(h + 1) * shared] = (w @ v[cols]).transpose(0, 1)
        t0 += nq
    return out


# ------------------------------------------------------------------------------ work

def work(case):
    if case["kind"] == "norm":
        rows, width = case["rows"], case["width"]
        groups = {"bf16": 0, "row": 1, "group": -(-width // 128)}[case["out"]]
        out = rows * width * (2 if case["out"] == "bf16" else 1) + rows * groups * 4
        return {"bytes": rows * width * 6 + width * 2 + out, "flops": rows * width * 6}
    q_lens, kv_lens = _lens(case)
    heads, kv_heads, dim, T = case["heads"], case["kv_heads"], case["dim"], sum(q_lens)
    table = 4 * sum(-(-n // case["page"]) for n in kv_lens)
    if case["kind"] == "append":
        values = T * (heads + 2 * kv_heads) * dim
        turned = T * (heads + kv_heads) * case["rot"]
        return {"bytes": values * 4 + T * case["rot"] * 4 + T * 4, "flops": turned * 3}
    window, sinks = case["window"], case["sinks"]
    pairs = tokens = 0
    for nq, nk in zip(q_lens, kv_lens):
        first = nk - nq
        if not window:
            tokens += nk
            pairs += nq * first + nq * (nq + 1) // 2
            continue
        lo = max(0, first - window + 1)
        tokens += nk - lo + min(sinks, lo)
        for p in range(first, nk):
            a = max(0, p - window + 1)
            pairs += p - a + 1 + min(sinks, a)
    return {"bytes": T * heads * dim * 4 + tokens * kv_heads * dim * 4 + table, "flops": pairs * heads * dim * 4}
