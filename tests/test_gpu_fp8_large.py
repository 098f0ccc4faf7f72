"""Inputs and outputs of more than 2^31 elements: rows at both ends against 64 bits, or against the same rows alone where
every step is a row's own. A log probability of 131,075 entries is off by at most 2^-24 (V / 256 + 64 + 4 + 2 E|z - m|), with
E|z - m| under 10, its roundings 2^-23 (1 + 12) and 2^-22 12 (test_gpu_score.py): less than 2^-14."""
import pytest
import torch

from mixed_lora_projection_gb300 import LoraLinear, fp8_rows, silu_mul, silu_mul_fp8, token_logprobs

pytestmark = pytest.mark.gpu

F64, BF16, FP8 = torch.float64, torch.bfloat16, torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("ids", [[0], [1]])
def test_projection(ids):
    # (a head of 131,080 tokens behind a long prompt; the bound as test_gpu_fp8.py's)
    T, d_in, d_out, rank = 16400, 128, 131080, 16
    g = gen(1)
    x8 = (torch.randn(T, d_in, generator=g, device="cuda") * 60).to(FP8)
    w8 = (torch.randn(d_out, d_in, generator=g, device="cuda") * 60).to(FP8)
    xs = torch.rand(T, 1, generator=g, device="cuda") + 0.5
    ws = torch.rand(-(-d_out // 128), 1, generator=g, device="cuda") + 0.5
    x = torch.randn(T, d_in, generator=g, device="cuda").to(BF16)
    a, b = torch.randn(rank, d_in, generator=g, device="cuda").to(BF16), torch.randn(d_out, rank, generator=g, device="cuda").to(BF16)
    with LoraLinear(d_in, d_out, rank, T, 1) as ll:
        y = ll.forward_fp8(x8, xs, [0, T], ids, w8, ws, [a], [b], [1.0], x=x)
        torch.cuda.synchronize()
        assert ll.status() == 0
    assert y.numel() > 2 ** 31
    rows = torch.tensor([0, 1, 127, 128, T // 2, T - 129, T - 17, T - 16, T - 1], device="cuda")
    X = x8[rows].to(F64) * xs[rows].to(F64)
    W = w8.to(F64) * ws.to(F64).repeat_interleave(128, 0)[:d_out]
    ref, S, more = X @ W.T, X.abs() @ W.abs().T, 0.0
    if ids[0]:
        A, B, xr = a.to(F64), b.to(F64), x[rows].to(F64)
        u = xr @ A.T
        ref += u @ B.T
        S += u.abs() @ B.abs().T
        more = (2.0 ** -8 * u.abs() + 2.0 ** -13 * (xr.abs() @ A.abs().T)) @ B.abs().T
    assert ((y[rows].to(F64) - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * S + 1.01 * more).all()


def test_gated_activation_and_rows():
    rows, width = 62000, 17408
    x = torch.randn(rows, 2 * width, generator=gen(2), device="cuda", dtype=BF16)
    assert x.numel() > 2 ** 31
    ends = [0, 1, rows // 2, rows - 2, rows - 1]
    few = x[ends]
    assert torch.equal(silu_mul(x)[ends], silu_mul(few))
    for group in (0, 128):
        for f in (silu_mul_fp8, fp8_rows):
            if f is fp8_rows:
                big, small = x.view(2 * rows, width), x.view(2 * rows, width)[ends]
            else:
                big, small = x, few
            q, s = f(big, group=group)
            r, t = f(small, group=group)
            assert torch.equal(q[ends].view(torch.uint8), r.view(torch.uint8)) and torch.equal(s[ends], t)


@pytest.mark.parametrize("top", [0, 20])
def test_scores(top):
    rows, vocab = 17000, 131075
    x = torch.randn(rows, vocab, generator=gen(3), device="cuda", dtype=BF16)
    assert x.numel() > 2 ** 31
    tokens = torch.randint(vocab, (rows,), generator=gen(4), device="cuda")
    r = token_logprobs(x, tokens, top=top)
    for t in (0, rows // 2, rows - 1):
        z = x[t].to(F64)
        lp = torch.log_softmax(z, -1)
        assert abs(r.logprobs[t].item() - lp[tokens[t]].item()) <= 2.0 ** -14
        mine = z[tokens[t]]
        before = (z > mine).sum() + ((z == mine) & (torch.arange(vocab, device="cuda") < tokens[t])).sum()
        assert r.ranks[t].item() == before.item()
        order = torch.sort(-z, stable=True).indices[:top]
        assert torch.equal(r.top_tokens[t].long(), order)
