"""token_logprobs against 64 bits.

Bounds: whole numbers are equal. With z = x / temperature, t = (z - max z) log2(e): z - m is rounded twice (2^-24 each,
relative), an exponential to 2^-22, and a sum takes at most n = V / 256 + 64 additions of one term on its way (a thread
sums every 256th vector of 8, then come lanes, warps and parts). So the sum s is off by at most d = 2^-24 (n + 4 + 2 E|z - m|)
of itself, E the mean under the softmax; log s by d and one rounding of at most 2^-23 (1 + log s); a log probability by
that and 2^-22 |z - m|; the entropy's quotient by 2 d and the roundings of its terms, of E|z - m|."""
import math

import pytest
import torch

from mixed_lora_projection_gb300 import token_logprobs

pytestmark = pytest.mark.gpu

F64, BF16 = torch.float64, torch.bfloat16
INF, NAN = math.inf, math.nan


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def order(x):
    """Indices by falling x, ties by rising index, NaN last; -0 and 0 are equal."""
    key = torch.where(torch.isnan(x), INF, -x.to(F64))
    nan = torch.isnan(x)
    first = torch.sort(nan.to(torch.int8), dim=-1, stable=True).indices        # numbers, then NaN, each by index
    return first.gather(-1, torch.sort(key.gather(-1, first) + 0.0, dim=-1, stable=True).indices) if not nan.any() else \
        torch.stack([torch.cat([i[~nan[r][i]], i[nan[r][i]]]) for r, i in enumerate(torch.sort(key, dim=-1, stable=True).indices)])


def check(x, tokens, top, temperature=1.0):
    got = token_logprobs(x, tokens, top=top, temperature=temperature)
    rows, vocab = x.shape
    inv = torch.tensor(1.0 / temperature, dtype=torch.float32).double().item()
    z = x.to(F64) * inv
    odd = torch.isnan(z).any(-1) | (z == INF).any(-1)
    none = (z == -INF).all(-1)
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    e = torch.exp(z - m)
    s = e.sum(-1)
    p = e / s[:, None]
    mean = torch.where(p > 0, p * (z - m).abs(), 0.0).sum(-1)                   # E|z - m|
    H = s.log() + mean
    n = vocab / 256 + 64
    d = 2.0 ** -24 * (n + 4 + 2 * mean)
    log_tol = d + 2.0 ** -23 * (1 + s.log().abs())
    fine = ~odd & ~none
    assert got.entropy.shape == (rows,) and got.entropy.dtype == torch.float32
    assert torch.isnan(got.entropy[odd]).all() and (got.entropy[none] == 0).all()
    assert ((got.entropy.to(F64) - H).abs() <= log_tol + (2 * d + 2.0 ** -21) * mean)[fine].all()
    idx = order(x)[:, :top]
    assert torch.equal(got.top_tokens.long(), idx)
    lp = z - m - s.log()[:, None]

    def close(a, i):
        want, tol = lp.gather(1, i), log_tol[:, None] + 2.0 ** -22 * (z - m).gather(1, i).abs()
        zero = want == -INF
        assert torch.equal(torch.isnan(a), odd[:, None].expand_as(a))
        assert ((a == -INF) == (zero | none[:, None]))[~odd].all()
        ok = ((a.to(F64) - want).abs() <= tol) | zero
        assert ok[fine].all(), ((a.to(F64) - want).abs() / tol)[fine].max()

    close(got.top_logprobs, idx)
    if tokens is None:
        assert got.logprobs is None and got.ranks is None
        return got
    t = tokens.long()
    inside = (t >= 0) & (t < vocab)
    assert torch.isnan(got.logprobs[~inside]).all() and (got.ranks[~inside] == -1).all()
    tc = t.clamp(0, vocab - 1)[:, None]
    a = torch.where(inside, got.logprobs, lp.gather(1, tc)[:, 0].float())[:, None]
    if inside.all():
        close(a, tc)
    xt = x.gather(1, tc)
    i = torch.arange(vocab, device=x.device)
    number = ~torch.isnan(x)
    before = torch.where(torch.isnan(xt), number | (i < tc), number & ((x > xt) | ((x == xt) & (i < tc))))
    assert torch.equal(got.ranks.long()[inside], before.sum(-1)[inside])
    return got


SHAPES = [(1, 1, 1), (1, 5, 5), (2, 8, 3), (3, 33, 32), (5, 255, 20), (7, 1000, 1), (3, 4099, 32), (1, 131072, 20),
          (2, 100003, 20), (48, 8191, 5), (31, 50001, 0), (700, 2053, 7), (1300, 515, 32), (1, 262144, 32)]


@pytest.mark.parametrize("rows,vocab,top", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_against_64_bits(rows, vocab, top, dtype):
    g = gen(rows + vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(dtype)      # (odd rows begin off the 16-byte grid)
    tokens = torch.randint(vocab, (rows,), generator=g, device="cuda")
    got = check(x, tokens, top)
    again = token_logprobs(x, tokens, top=top)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    check(x, tokens.to(torch.int32), top, temperature=0.7)
    check(x, None, top, temperature=3.0)


PATTERNS = {
    "rising": lambda x: torch.arange(x.shape[1], device=x.device).expand_as(x).float() / 64,
    "falling": lambda x: -torch.arange(x.shape[1], device=x.device).expand_as(x).float() / 64,
    "equal": lambda x: torch.full_like(x, 1.5),
    "few values": lambda x: (x * 2).round(),
    "zeros of both signs": lambda x: torch.where(x > 0, 0.0, -0.0) * torch.ones_like(x),
    "nothing": lambda x: torch.full_like(x, -INF),
    "three left": lambda x: x.masked_fill(torch.arange(x.shape[1], device=x.device) % (x.shape[1] // 3 + 1) != 7, -INF),
    "half ruled out": lambda x: x.masked_fill(torch.arange(x.shape[1], device=x.device) % 2 == 0, -INF),
    "lowest values": lambda x: torch.where(x > 0, x, torch.finfo(BF16).min),
    "peaked": lambda x: torch.where(torch.arange(x.shape[1], device=x.device) == x.shape[1] // 2, 90.0, x),
    "large": lambda x: x * 1e30,
    "a NaN": lambda x: x.masked_fill(torch.arange(x.shape[1], device=x.device) == 11, NAN),
    "NaN alone": lambda x: torch.full_like(x, NAN),
    "NaN but two": lambda x: torch.where(torch.arange(x.shape[1], device=x.device) % (x.shape[1] // 2) == 5, x, NAN),
    "an infinity": lambda x: x.masked_fill(torch.arange(x.shape[1], device=x.device) == 13, INF),
}


@pytest.mark.parametrize("name", list(PATTERNS))
@pytest.mark.parametrize("rows,vocab", [(3, 40), (2, 5003), (2, 40000), (300, 6001)])
def test_patterns(name, rows, vocab):
    g = gen(vocab)
    for dtype in (BF16, torch.float32):
        x = PATTERNS[name](torch.randn(rows, vocab, generator=g, device="cuda")).to(dtype)
        for top in (1, 20, 32):
            check(x, torch.randint(vocab, (rows,), generator=g, device="cuda"), top)
        check(x, torch.full((rows,), 11, device="cuda"), 3)


def test_views_and_strides():
    g = gen(1)
    for dtype in (BF16, torch.float32):
        wide = torch.randn(9, 3 * 2001 + 5, generator=g, device="cuda").to(dtype)
        for lo in range(9):
            check(wide[:, lo:lo + 2001], torch.randint(2001, (9,), generator=g, device="cuda"), 20)
        check(wide[::3, 5:3000], torch.randint(2995, (3,), generator=g, device="cuda"), 20)


def test_tokens_outside_the_vocabulary():
    x = torch.randn(6, 777, generator=gen(2), device="cuda")
    check(x, torch.tensor([0, 776, -1, 777, -(2 ** 40), 2 ** 40], device="cuda"), 2)
    check(x, torch.tensor([0, 776, -1, 777, -(2 ** 31), 2 ** 31 - 1], dtype=torch.int32, device="cuda"), 2)


def test_no_rows():
    r = token_logprobs(torch.zeros(0, 10, device="cuda"), torch.zeros(0, dtype=torch.long, device="cuda"), top=3)
    assert [t.shape for t in r] == [(0,), (0,), (0,), (0, 3), (0, 3)]


def test_many_rows_and_few_entries():
    x = torch.randn(100000, 9, generator=gen(3), device="cuda").to(BF16)
    check(x, torch.randint(9, (100000,), generator=gen(4), device="cuda"), 9)


def test_graph_and_streams():
    g = gen(5)
    xs = [torch.randn(r, v, generator=g, device="cuda").to(BF16) for r, v in ((1, 131072), (48, 30001), (900, 4000))]
    ts = [torch.randint(x.shape[1], (x.shape[0],), generator=g, device="cuda") for x in xs]
    want = [token_logprobs(x, t, top=20) for x, t in zip(xs, ts)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [token_logprobs(x, t, top=20) for x, t in zip(xs, ts)]
    for _ in range(3):
        for o in outs:
            for a in o:
                a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [token_logprobs(x, t, top=20, stream=s) for _ in range(20) for x, t, s in zip(xs, ts, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i, o in enumerate(got) for a, b in zip(o, want[i % 3]))


# Blocks of four warps: a thread sums every 128th vector, V / 256 additions of pairs, so that the bounds above hold.
@pytest.mark.parametrize("name", list(PATTERNS))
@pytest.mark.parametrize("rows,vocab", [(611, 2003), (609, 20011)])
def test_patterns_of_many_rows(name, rows, vocab):
    g = gen(rows)
    for dtype in (BF16, torch.float32):
        x = PATTERNS[name](torch.randn(rows, vocab, generator=g, device="cuda")).to(dtype)
        for top in (1, 20, 32):
            check(x, torch.randint(vocab, (rows,), generator=g, device="cuda"), top)
        check(x, torch.full((rows,), 11, device="cuda"), 0)


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(2047, 33001), (2048, 33001), (609, 32768), (609, 32769), (2500, 1), (2500, 1023)])
def test_where_the_blocks_change(rows, vocab, dtype):
    g = gen(vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(dtype)
    for top in (min(32, vocab), 0):
        check(x, torch.randint(vocab, (rows,), generator=g, device="cuda"), top)
