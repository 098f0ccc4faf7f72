"""The operators between the projections (include/lora_layer.h) on a GPU, against their formulas in
64 bits. Tolerances follow from the roundings the header names:

- bf16 outputs of the norm and of the rotary turn are rounded once (8 significant bits: half a unit is
  at most 2^-8 of the value, as at 1 + 2^-8);
  the fp32 arithmetic before it adds less than 2^-17 (sums of at most 32,768 squares in blocks) or,
  for a cos - b sin, 3 * 2^-24 (|a| + |b|);
- e4m3: half a unit is 2^-4 of a normal value and 2^-10 (in units of the scale) of a subnormal one;
- attention: with c = sum_j p_j |v_j|, the weights' rounding to bf16 moves an output by at most
  2^-8 c and the output's own by 2^-8 |o|; fp32 scores (products of up to 256 terms, in
  magnitude under 32) and sums add less than 2^-11 c.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F64 = torch.float64
BF16 = torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF16)


def within(got, ref, most):
    got = got.to(F64)
    assert got.shape == ref.shape and not torch.isnan(got).any()
    worst = ((got - ref).abs() - most).max().item() if got.numel() else 0.0
    assert worst <= 0, f"beyond the bound by {worst:.3e}"


def bound(ref, c):
    return U * ref.abs() + ATTN * c + 2.0 ** -40


# --------------------------------------------------------------------------- norm

def norm_ref(x, r, w, off, eps):
    h = x.to(F64) + (r.to(F64) if r is not None else 0.0)
    return h, h / ((h * h).mean(-1, keepdim=True) + eps).sqrt() * (w.to(F64) + off)


U = 2.0 ** -8                                  # unit roundoff of bf16
BF16_TOL = U + 2.0 ** -17
ATTN = 2.0 ** -8 + 2.0 ** -11                  # of c, beside U |o|


@pytest.mark.parametrize("rows,width", [(1, 8), (3, 64), (7, 264), (5, 1000), (33, 1032), (48, 5120), (700, 5120),
                                        (2, 17408), (3, 32768), (0, 128)])
@pytest.mark.parametrize("residual", [False, True])
def test_add_rms_norm(rows, width, residual):
    from mixed_lora_projection_gb300 import add_rms_norm
    g = gen(rows * 7 + width)
    x, w = randn(g, rows, width), randn(g, width)
    r = randn(g, rows, width, scale=3) if residual else None
    y, h = add_rms_norm(x, w, r, eps=1e-5, weight_offset=1.0)
    hr, yr = norm_ref(x, r, w, 1.0, 1e-5)
    within(y, yr, yr.abs() * BF16_TOL)
    if residual:
        within(h, hr, hr.abs() * BF16_TOL)
    else:
        assert h is x


@pytest.mark.parametrize("rows,width,group", [(1, 8, 0), (5, 72, 32), (9, 264, 64), (48, 5120, 0), (48, 5120, 128),
                                              (400, 5128, 128), (3, 5128, 256), (2, 32768, 0), (2, 32760, 32)])
def test_add_rms_norm_8bit(rows, width, group):
    from mixed_lora_projection_gb300 import add_rms_norm_fp8
    g = gen(rows + width + group)
    x, r, w = randn(g, rows, width), randn(g, rows, width, scale=3), randn(g, width)
    x[0] = 0
    r[0] = 0                                                  # a row of zeros: q = 0, the smallest scale
    q, s, h = add_rms_norm_fp8(x, w, r, group=group)
    hr, yr = norm_ref(x, r, w, 0.0, 1e-6)
    n = group or width
    parts = yr.split(n, -1)
    ref_s = torch.stack([(t.abs().amax(-1) / 448).clamp(min=2.0 ** -100) for t in parts], -1)
    within(s, ref_s, ref_s * 2.0 ** -17)
    full = torch.repeat_interleave(s.to(F64), n, -1)[:, :width]
    within(q.to(torch.float32).to(F64) * full, yr, torch.maximum(yr.abs() * 2.0 ** -4, full * 2.0 ** -10) * (1 + 2.0 ** -12))
    assert (q[0].float() == 0).all() and (s[0] == 2.0 ** -100).all()
    within(h, hr, hr.abs() * BF16_TOL)


def test_add_rms_norm_strides_in_place_and_bad_rows():
    from mixed_lora_projection_gb300 import add_rms_norm
    g = gen(5)
    big = randn(g, 40, 3 * 520)
    x, r = big[:, 520:1040], big[:, 1040:]
    w = randn(g, 520)
    hr, yr = norm_ref(x, r, w, 0.0, 1e-6)
    keep = big[:, :520].clone()
    y, h = add_rms_norm(x, w, r, out=x, h_out=r)              # both outputs over their inputs
    assert y is x and h is r
    within(y, yr, yr.abs() * BF16_TOL)
    within(h, hr, hr.abs() * BF16_TOL)
    assert torch.equal(big[:, :520], keep)
    x = randn(g, 6, 1040)
    x[1, 7], x[3, 100], x[4, 1039] = math.nan, math.inf, -math.inf
    y, _ = add_rms_norm(x, randn(g, 1040))
    bad = torch.isnan(y).any(-1).tolist()
    assert bad == [False, True, False, True, True, False]


def test_add_rms_norm_8bit_nan_stays_in_its_row():
    from mixed_lora_projection_gb300 import add_rms_norm_fp8
    g = gen(6)
    x = randn(g, 4, 1032)
    x[2, 1031] = math.nan
    q, s, _ = add_rms_norm_fp8(x, randn(g, 1032))
    assert torch.isnan(s).flatten().tolist() == [False, False, True, False]
    assert not torch.isnan(q.float()[[0, 1, 3]]).any()


# --------------------------------------------------------------------------- cache

class Case:
    """Sequences with their new rows and a shuffled paged cache. layout: 'nhd' [page, token, head, dim],
    'hnd' [page, head, token, dim], 'kv' K and V interleaved in one buffer."""

    def __init__(self, q_lens, kv_lens, heads, kv_heads, dim, page, layout="nhd", seed=0, spare=3):
        g = gen(seed + 17)
        self.q_lens, self.kv_list = q_lens, kv_lens
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        self.off = [0]
        for n in q_lens:
            self.off.append(self.off[-1] + n)
        need = [-(-n // page) for n in kv_lens]
        total = sum(need) + spare
        self.n_pages = total
        perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        self.table = torch.full((len(q_lens), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = perm[at:at + n]
            at += n
        if layout == "hnd":
            self.k = randn(g, total, kv_heads, page, dim).transpose(1, 2)
            self.v = randn(g, total, kv_heads, page, dim).transpose(1, 2)
        elif layout == "kv":
            both = randn(g, total, 2, page, kv_heads, dim)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = randn(g, total, page, kv_heads, dim), randn(g, total, page, kv_heads, dim)
        self.q = randn(g, self.off[-1], heads, dim)
        self.kv = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)

    def slots(self, i, n):
        j = torch.arange(n, device=DEV)
        return self.table[i].long()[j // self.page], j % self.page

    def poison(self):
        """NaN in every place of the cache that no sequence's tokens are in."""
        used = torch.zeros(self.n_pages, self.page, dtype=torch.bool, device=DEV)
        for i, n in enumerate(self.kv_list):
            used[self.slots(i, n)] = True
        self.k[~used] = math.nan
        self.v[~used] = math.nan

    def ref(self, window=0, sinks=0, scale=None):
        """(o, c) in 64 bits: the output and sum_j p_j |v_j|."""
        scale = self.dim ** -0.5 if scale is None else scale
        o = torch.zeros(self.off[-1], self.heads, self.dim, dtype=F64, device=DEV)
        c = torch.zeros_like(o)
        shared = self.heads // self.kv_heads
        for i, (nq, nk) in enumerate(zip(self.q_lens, self.kv_list)):
            if nq == 0 or nk == 0:
                continue
            pg, sl = self.slots(i, nk)
            k, v = self.k[pg, sl].to(F64), self.v[pg, sl].to(F64)          # [nk, kv_heads, dim]
            q = self.q[self.off[i]:self.off[i + 1]].to(F64).view(nq, self.kv_heads, shared, self.dim)
            s = torch.einsum("qhgd,khd->hgqk", q, k) * scale
            pos = torch.arange(nk - nq, nk, device=DEV)[:, None]
            j = torch.arange(nk, device=DEV)[None]
            seen = j <= pos
            if window:
                seen &= (j > pos - window) | (j < sinks)
            s = s.masked_fill(~seen, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m.masked_fill(m == -math.inf, 0.0))
            p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
            o[self.off[i]:self.off[i + 1]] = torch.einsum("hgqk,khd->qhgd", p, v).reshape(nq, self.heads, self.dim)
            c[self.off[i]:self.off[i + 1]] = torch.einsum("hgqk,khd->qhgd", p, v.abs()).reshape(nq, self.heads, self.dim)
        return o, c

    def run(self, attn=None, **kw):
        from mixed_lora_projection_gb300 import PagedAttention
        own = attn is None
        if own:
            attn = PagedAttention(self.heads, self.kv_heads, self.dim, self.page, max(1, self.off[-1]), len(self.q_lens))
        o = attn.forward(self.q, self.k, self.v, self.off, self.kv, self.table, **kw)
        assert attn.status() == 0
        if own:
            attn.close()
        return o

    def check(self, window=0, sinks=0, **kw):
        ref, c = self.ref(window, sinks, kw.get("scale"))
        got = self.run(window=window, sinks=sinks, **kw)
        within(got, ref, bound(ref, c))
        return got


# decode: 1 to 8 new rows, every kind of length, pages that end inside a tile
DECODE = [
    ([1], [1], 2, 1, 64, 16), ([1, 1, 1], [64, 65, 63], 4, 4, 64, 16), ([1] * 5, [0, 1, 17, 300, 129], 6, 2, 128, 48),
    ([1, 1], [5000, 31], 24, 12, 256, 1552), ([8] * 3, [8, 100, 2000], 24, 12, 256, 64), ([8, 8], [700, 3], 24, 4, 256, 64),
    ([8, 0, 1, 5], [1000, 40, 0, 5], 12, 2, 128, 16), ([2], [4097], 32, 1, 128, 64), ([1], [20000], 8, 8, 128, 112),
    ([1] * 70, [1 + 37 * i for i in range(70)], 8, 2, 64, 32), ([4], [333], 128, 1, 64, 16), ([8], [1000], 8, 1, 256, 128),
    ([3, 8, 1], [500, 1300, 77], 10, 2, 128, 80), ([1], [517], 24, 12, 256, 16), ([7], [640], 40, 5, 64, 64),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{len(c[0])}x{c[0][0]}-{c[2]}-{c[3]}-{c[4]}-{c[5]}")
def test_decode(case):
    c = Case(*case, seed=len(case[0]) * 31 + case[4])
    c.poison()
    c.check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 4), (64, 64), (100, 200), (1000, 1), (10 ** 6, 5)])
def test_decode_window(window, sinks):
    c = Case([1, 8, 1, 2], [3000, 900, 50, 64], 12, 2, 128, 48, seed=window)
    c.poison()
    c.check(window, sinks)
    c = Case([4, 1], [1700, 400], 8, 4, 256, 64, seed=window + 1)
    c.check(window, sinks)


# prompts: more new rows than a decode step has; packed rows of 1 to 32 heads, ragged ends
PROMPTS = [
    ([65], [65], 1, 1, 64, 16), ([128, 130], [128, 130], 4, 4, 128, 64), ([300], [1300], 6, 1, 128, 48),
    ([257, 1, 90], [257, 800, 1000], 12, 2, 128, 16), ([500], [500], 4, 2, 256, 64), ([333, 70], [2000, 70], 12, 2, 256, 1552),
    ([200], [199], 8, 2, 64, 32), ([150], [20], 8, 8, 128, 16), ([129, 64, 512], [1000, 64, 513], 3, 3, 64, 80),
    ([40], [3000], 32, 1, 128, 64), ([7], [1000], 128, 1, 64, 16), ([1025], [1025], 2, 2, 128, 128), ([20], [5000], 24, 4, 256, 64),
    ([9, 300, 1, 0, 8], [777, 300, 5, 9, 2048], 10, 1, 256, 112),
]


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: f"{len(c[0])}x{c[0][0]}-{c[2]}-{c[3]}-{c[4]}-{c[5]}")
def test_prompt(case):
    c = Case(*case, seed=case[0][0])
    c.poison()
    c.check()


@pytest.mark.parametrize("heads,kv_heads,dim", [(64, 64, 64), (48, 48, 128), (32, 32, 256)])
def test_many_units_with_and_without_tokens(heads, kv_heads, dim):
    # several units a block; rows before the sequence's start see nothing, last tiles have few rows
    c = Case([400, 129, 300, 20, 257], [30, 129, 300, 3, 700], heads, kv_heads, dim, 32, seed=dim)
    c.poison()
    c.check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (63, 4), (128, 0), (129, 128), (300, 150), (10 ** 6, 5)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 64), (12, 2, 128), (6, 3, 256)])
def test_prompt_window(window, sinks, heads, kv_heads, dim):
    c = Case([700, 130, 1], [1400, 130, 900], heads, kv_heads, dim, 48, seed=window)
    c.poison()
    c.check(window, sinks)


@pytest.mark.parametrize("layout", ["hnd", "kv"])
@pytest.mark.parametrize("q", [1, 200])
def test_layouts_and_strides(layout, q):
    for dim, heads, kv_heads in ((128, 8, 2), (256, 6, 3), (64, 4, 1)):
        c = Case([q, q], [900, 333], heads, kv_heads, dim, 32, layout=layout, seed=q)
        c.poison()
        # queries inside a fused row, outputs with their heads outermost
        fused = torch.full((2 * q, heads + 4, dim), math.nan, dtype=BF16, device=DEV)
        fused[:, 2:2 + heads] = c.q
        c.q = fused[:, 2:2 + heads]
        out = torch.zeros(heads, 2 * q + 5, dim, dtype=BF16, device=DEV)
        c.check(out=out[:, 3:3 + 2 * q].transpose(0, 1))
        assert (out[:, :3] == 0).all() and (out[:, 3 + 2 * q:] == 0).all()


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 8, 2), (128, 12, 2), (256, 6, 3), (128, 96, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_queries_with_heads_outermost(dim, heads, kv_heads, window, sinks):
    # a head's rows lie together: the row stride is the smaller one
    for q_lens, kv_lens in (([1, 3], [700, 65]), ([130, 50, 1], [400, 50, 2000])):
        c = Case(q_lens, kv_lens, heads, kv_heads, dim, 48, seed=dim + heads)
        c.poison()
        c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
        assert c.q.stride(0) < c.q.stride(1)
        c.check(window, sinks)


def test_scale_and_large_scores():
    for q in (1, 150):
        c = Case([q], [600], 4, 2, 128, 16, seed=3)
        c.check(scale=0.7 * 128 ** -0.5)
        # growing scores: every tile raises the running maximum
        ramp = torch.linspace(0, 2.0, 600, device=DEV)
        pg, sl = c.slots(0, 600)
        direction = torch.ones(128, device=DEV) / math.sqrt(128)
        c.k[pg, sl] = (ramp[:, None, None] * direction * 10).to(BF16).expand(600, 2, 128)
        c.q = (direction * 12).to(BF16).expand(q, 4, 128).contiguous()
        c.check(scale=1.0)
        c.k[pg, sl] = c.k[pg.flip(0), sl.flip(0)]               # and falling ones
        c.check(scale=1.0)


def test_pages_outside_the_window_may_be_gone():
    for q in (1, 8, 200):
        c = Case([q], [2000], 6, 2, 128, 32, seed=q)
        window, sinks = 300, 5
        ref, w = c.ref(window, sinks)
        lo = 2000 - q - window + 1
        c.table[0, 1:lo // 32] = torch.tensor([-1, 2 ** 30], device=DEV, dtype=torch.int32).repeat(100)[:lo // 32 - 1]
        within(c.run(window=window, sinks=sinks), ref, bound(ref, w))


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 8, 4), (128, 6, 2), (256, 6, 3)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 70), (300, 5), (1000, 200)])
def test_bad_values_outside_the_window(dim, heads, kv_heads, window, sinks):
    """Tokens between the sinks and the first row's window hold NaN and infinities: no row sees them."""
    for q in (1, 5, 150, 333):
        c = Case([q, q], [1601, 1350], heads, kv_heads, dim, 32, seed=q)
        ref, w = c.ref(window, sinks)
        for i, n in enumerate(c.kv_list):
            pg, sl = (x[sinks:max(sinks, n - q - window + 1)] for x in c.slots(i, n))
            c.k[pg, sl], c.v[pg, sl] = math.nan, math.inf
            c.v[pg[::3], sl[::3]] = math.nan
        within(c.run(window=window, sinks=sinks), ref, bound(ref, w))


def test_same_bits_again_and_other_stream():
    for q, kv in ((1, 5000), (8, 3000), (260, 1500)):
        c = Case([q, q], [kv, kv // 3], 12, 4, 128, 64, seed=q)
        from mixed_lora_projection_gb300 import PagedAttention
        with PagedAttention(12, 4, 128, 64, 2 * q, 2) as attn:
            a = c.run(attn)
            for _ in range(5):
                assert torch.equal(c.run(attn), a)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            b = attn.forward(c.q, c.k, c.v, c.off, c.kv, c.table, stream=s)
            s.synchronize()
            assert torch.equal(a, b)


def test_cache_past_32_bits():
    # token places beyond 2^32 elements from the cache's start
    pages, page, kv_heads, dim = 4400, 64, 64, 256
    assert pages * page * kv_heads * dim > 2 ** 32
    k = torch.empty(pages, page, kv_heads, dim, dtype=BF16, device=DEV)
    g = gen(4)
    far = torch.tensor([pages - 1, pages - 3, pages - 2, 0], dtype=torch.int32, device=DEV)
    for q in (1, 70):
        c = Case([q], [200], 64, 64, dim, page, seed=9)
        c.v = c.k                                     # one buffer is K and V
        ref, w = c.ref()
        k[far.long()] = c.k[c.table[0, :4].long()]
        c.table, c.k, c.v = far[None].contiguous(), k, k
        within(c.run(), ref, bound(ref, w))
        # and the append writes there
        from mixed_lora_projection_gb300 import kv_append
        new = randn(g, 1, kv_heads, dim)
        kv_append(None, new, new, [0, 1], torch.tensor([130], dtype=torch.int32, device=DEV), c.table, k, k)
        assert torch.equal(k[pages - 2, 1], new[0])
    del k


def test_graph_replay_as_the_cache_grows():
    from mixed_lora_projection_gb300 import PagedAttention, kv_append
    heads, kv_heads, dim, page = 12, 2, 128, 16
    c = Case([1, 1], [90, 400], heads, kv_heads, dim, page, seed=11)
    g = gen(12)
    new = randn(g, 2, kv_heads, dim)
    with PagedAttention(heads, kv_heads, dim, page, 2, 2) as attn:
        out = torch.empty(2, heads, dim, dtype=BF16, device=DEV)

        def step():
            kv_append(None, new, new, c.off, c.kv, c.table, c.k, c.v)
            attn.forward(c.q, c.k, c.v, c.off, c.kv, c.table, out=out)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for lens in ([91, 3], [96, 385], [17, 400]):
            c.kv.copy_(torch.tensor(lens, dtype=torch.int32))
            new.copy_(randn(g, 2, kv_heads, dim))
            graph.replay()
            torch.cuda.synchronize()
            c.kv_list = lens
            for i in range(2):
                pg, sl = c.slots(i, lens[i])
                assert torch.equal(c.k[pg[-1], sl[-1]], new[i])
            ref, w = c.ref()
            within(out, ref, bound(ref, w))


# --------------------------------------------------------------------------- append

@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv"])
@pytest.mark.parametrize("rot", [0, 16, 64, 128])
def test_kv_append(layout, rot):
    from mixed_lora_projection_gb300 import kv_append
    q_lens, kv_lens = [1, 0, 8, 300, 20], [17, 5, 8, 1000, 12]     # the last one's first 8 rows have no place
    heads, kv_heads, dim = 6, 3, 128
    c = Case(q_lens, kv_lens, heads, kv_heads, dim, 48, layout=layout, seed=rot)
    g = gen(rot + 1)
    T = c.off[-1]
    y = randn(g, T, heads + 2 * kv_heads, dim)
    q, k, v = y[:, :heads], y[:, heads:heads + kv_heads], y[:, heads + kv_heads:]
    cos = sin = None
    if rot:
        angle = torch.rand(1001, rot // 2, generator=g, device=DEV, dtype=F64) * 6.28
        cos, sin = angle.cos().float(), angle.sin().float()
    kc, vc = c.k.clone(), c.v.clone()
    out = kv_append(q, k, v, c.off, c.kv, c.table, c.k, c.v, cos, sin, q_out=torch.empty(T, heads, dim, dtype=BF16, device=DEV))
    half = rot // 2
    for i, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        for r in range(nq):
            t, pos = c.off[i] + r, nk - nq + r
            for src, dst in ((q[t], out[t]), (k[t], None)):
                if dst is None:
                    if pos < 0:
                        continue
                    pg, sl = c.table[i, pos // 48].item(), pos % 48
                    dst = c.k[pg, sl]
                    assert torch.equal(c.v[pg, sl], v[t])
                    kc[pg, sl], vc[pg, sl] = dst, v[t]
                assert torch.equal(dst[:, rot:], src[:, rot:])
                if rot:
                    a, b = src[:, :half].to(F64), src[:, half:rot].to(F64)
                    cs, sn = cos[max(pos, 0)].to(F64), sin[max(pos, 0)].to(F64)
                    ref = torch.cat([a * cs - b * sn, b * cs + a * sn], -1)
                    mag = torch.cat([a.abs() + b.abs()] * 2, -1)
                    within(dst[:, :rot], ref, ref.abs() * U + mag * 2.0 ** -22)
    assert torch.equal(c.k, kc) and torch.equal(c.v, vc)          # nothing else was written


def test_kv_append_in_place_and_missing_pages():
    from mixed_lora_projection_gb300 import kv_append
    c = Case([4], [40], 2, 1, 64, 16, seed=1)
    g = gen(2)
    y = randn(g, 4, 4, 64)
    want = y[:, :2].clone()
    cos, sin = torch.ones(50, 32, device=DEV), torch.zeros(50, 32, device=DEV)
    c.table[0, 2] = -1                                            # tokens 32..47 have no page
    kc = c.k.clone()
    got = kv_append(y[:, :2], y[:, 2:3], y[:, 3:], c.off, c.kv, c.table, c.k, c.v, cos, sin, q_out=y[:, :2])
    assert torch.equal(got, want) and torch.equal(c.k, kc)
    c.table[0, 2] = c.n_pages                                     # past the last page
    kv_append(None, y[:, 2:3], y[:, 3:], c.off, c.kv, c.table, c.k, c.v)
    assert torch.equal(c.k, kc)


def test_binding_refusals_leave_outputs_untouched():
    from mixed_lora_projection_gb300 import LoraError, PagedAttention, add_rms_norm, add_rms_norm_fp8, kv_append
    x, w = torch.ones(4, 128, dtype=BF16, device=DEV), torch.ones(128, dtype=BF16, device=DEV)
    y = torch.full_like(x, 7.0)
    for bad, kw in ((TypeError, dict(weight=w.float())), (TypeError, dict(out=y.float())), (TypeError, dict(residual=1)),
                    (ValueError, dict(weight=w[:64])), (ValueError, dict(residual=x[:3])), (ValueError, dict(weight=w.cpu())),
                    (ValueError, dict(out=y.t().contiguous().t())), (LoraError, dict(eps=-1.0)), (LoraError, dict(h_out=y[:, :]))):
        kw = {"weight": w, "out": y, **kw}
        with pytest.raises(bad):
            add_rms_norm(x, **kw)
    with pytest.raises(ValueError):
        add_rms_norm_fp8(x, w, group=48)
    with pytest.raises(ValueError):
        add_rms_norm_fp8(x, w, scales=torch.ones(4, device=DEV))
    c = Case([2, 3], [20, 9], 4, 2, 64, 16)
    o = torch.full_like(c.q, 7.0)
    attn = PagedAttention(4, 2, 64, 16, 8, 4)
    good = dict(q=c.q, k_cache=c.k, v_cache=c.v, q_offsets=c.off, kv_lens=c.kv, block_table=c.table, out=o)
    for bad, kw in ((TypeError, dict(q=c.q.float())), (TypeError, dict(kv_lens=c.kv.long())), (TypeError, dict(q_offsets=3)),
                    (TypeError, dict(q_offsets=[0, 1.5, 5])), (ValueError, dict(q_offsets=[0, 2])), (ValueError, dict(q_offsets=[0, 2, 6])),
                    (ValueError, dict(q_offsets=[0, 2, 1 << 40])), (ValueError, dict(q=c.q[:, :2])), (ValueError, dict(out=o[:3])),
                    (ValueError, dict(v_cache=c.v[1:])), (ValueError, dict(kv_lens=c.kv[:1])), (ValueError, dict(block_table=c.table[0])),
                    (ValueError, dict(window=1 << 40)), (LoraError, dict(window=-1)), (LoraError, dict(scale=0.0)),
                    (LoraError, dict(q_offsets=[0, 6, 5]))):
        with pytest.raises(bad):
            attn.forward(**{**good, **kw})
    with pytest.raises(ValueError):
        kv_append(c.q, c.k[0, :5], c.v[0, :5], c.off, c.kv, c.table, c.k, c.v, torch.ones(30, 8, device=DEV))
    with pytest.raises(ValueError):
        kv_append(c.q[:4], c.k[0, :5], c.v[0, :5], c.off, c.kv, c.table, c.k, c.v)
    assert bool((o == 7).all()) and bool((y == 7).all())
    attn.close()
    with pytest.raises(LoraError):
        attn.forward(**good)


@pytest.mark.parametrize("q_lens,kv_lens", [([8] * 6, [500, 9, 1300, 77, 2000, 640]), ([1], [517]), ([700, 1, 40], [900, 3000, 40])])
def test_chained_kernels_wait_for_each_other(q_lens, kv_lens):
    """Each call reads what the one before wrote, in place: the same bits with and without a wait between calls."""
    from mixed_lora_projection_gb300 import PagedAttention, add_rms_norm, kv_append
    c = Case(q_lens, kv_lens, 8, 4, 128, 64)
    T, g = c.off[-1], gen(5)
    x0, w = randn(g, T, 2048), randn(g, 1024)
    cos, sin = torch.rand(3000, 32, generator=g, device=DEV), torch.rand(3000, 32, generator=g, device=DEV)
    attn = PagedAttention(8, 4, 128, 64, T, len(q_lens))
    k0, v0 = c.k.clone(), c.v.clone()

    def run(wait):
        c.k.copy_(k0), c.v.copy_(v0)
        y = x0.clone()
        h = torch.zeros(T, 1024, dtype=BF16, device=DEV)
        for _ in range(12):
            for step in (lambda: add_rms_norm(y[:, :1024], w, h, out=y[:, :1024], h_out=h),
                         lambda: kv_append(y[:, :1024].view(T, 8, 128), y[:, 1024:1536].view(T, 4, 128), y[:, 1536:].view(T, 4, 128), c.off,
                                           c.kv, c.table, c.k, c.v, cos, sin, q_out=y[:, :1024].view(T, 8, 128)),
                         lambda: attn.forward(y[:, :1024].view(T, 8, 128), c.k, c.v, c.off, c.kv, c.table, out=h.view(T, 8, 128))):
                step()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return y, h, c.k.clone(), c.v.clone()

    once = run(True)
    for _ in range(5):
        for a, b in zip(once, run(False)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert attn.status() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (12, 2), (10, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_calls_at_the_edge_of_one_tile_of_rows(dim, heads, kv_heads, window, sinks):
    """The longest sequence fills one tile of 128 rows, or needs one token more."""
    most = 128 // (heads // kv_heads)
    for longest in (most, most + 1):
        q = [longest, 1, most // 2 + 9, 0, longest - 1]
        Case(q, [longest, 300, 700, 40, 1285], heads, kv_heads, dim, 48, seed=longest).check(window, sinks)


def test_calls_without_rows_and_in_inference_mode():
    from mixed_lora_projection_gb300 import PagedAttention, add_rms_norm, add_rms_norm_fp8, kv_append
    x, w = torch.ones(0, 128, dtype=BF16, device=DEV), torch.ones(128, dtype=BF16, device=DEV)
    y, h = add_rms_norm(x, w, x.clone())
    q8, s, _ = add_rms_norm_fp8(x, w, group=32)
    assert y.shape == h.shape == q8.shape == (0, 128) and s.shape == (0, 4)
    c = Case([0, 0], [20, 0], 4, 2, 64, 16)
    k0 = c.k.clone()
    cos = torch.ones(32, 8, device=DEV)
    assert kv_append(c.q, c.k[0, :0], c.v[0, :0], c.off, c.kv, c.table, c.k, c.v, cos, cos).shape == (0, 4, 64)
    assert c.run().shape == (0, 4, 64) and torch.equal(c.k, k0)
    c = Case([3, 40], [20, 60], 4, 2, 64, 16)
    ref = c.run()
    with torch.inference_mode():
        with PagedAttention(4, 2, 64, 16, 64, 2) as attn:
            assert torch.equal(c.run(attn), ref)
        x = torch.ones(3, 128, dtype=BF16, device=DEV)
        y, h = add_rms_norm(x, torch.nn.Parameter(w), x)
        assert bool((h == 2).all()) and not y.requires_grad
