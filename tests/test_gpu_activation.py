"""silu_mul, silu_mul_fp8, fp8_rows and fp8_blocks against their formulas.

Rows and blocks in 8 bits are exact: a maximum, one rounding of the scale, of its reciprocal and of each product, so they
are compared bit for bit with the same steps in torch. The gated activation's exponential is off by at most
(2 + 1.16 |g|) units of 2^-23 and its quotient by two, less than 2^-15 in all for |g| <= 88, past which y is under 2^-120 |u|;
bf16 rounds by half a step, 2^-8 of the value; e4m3 by 2^-4 of it or half of the smallest step, 2^-10 of the scale."""
import pytest
import torch

from mixed_lora_projection_gb300 import LoraLinear, add_rms_norm, add_rms_norm_fp8, fp8_blocks, fp8_rows, silu_mul, silu_mul_fp8

pytestmark = pytest.mark.gpu

F64, BF16, FP8 = torch.float64, torch.bfloat16, torch.float8_e4m3fn


def rand(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def scale_of(amax):
    s = amax * torch.tensor(1 / 448, dtype=torch.float32)
    return torch.where(s < 2.0 ** -100, 2.0 ** -100, s)


def groups(x, group):
    """(q, scales) of fp32 rows, by torch."""
    rows, width = x.shape
    n = -(-width // group)
    p = torch.nn.functional.pad(x, (0, n * group - width)).view(rows, n, group)
    s = scale_of(p.abs().amax(-1))
    q = (p * (1.0 / s)[..., None]).view(rows, -1)[:, :width]
    return q.clamp(-448, 448).to(FP8), s


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8) if a.dtype == FP8 else a, b.view(torch.uint8) if b.dtype == FP8 else b)


WIDTHS = [8, 24, 128, 136, 256, 264, 1000, 5120, 8192, 8200, 17408, 32768]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
def test_rows(width, group):
    for rows in (1, 3, 49):
        x = rand(rows, width, seed=width + rows, std=3)
        x[0] = 0
        q, s = fp8_rows(x, group=group)
        rq, rs = groups(x.float(), group or width)
        assert same_bits(s, rs) and same_bits(q, rq)


@pytest.mark.parametrize("rows,cols", [(1, 8), (127, 136), (128, 128), (129, 264), (300, 1000), (5, 17408), (2049, 256)])
def test_blocks(rows, cols):
    w = rand(rows, cols + 24, seed=rows)[:, 8:8 + cols]               # rows of a wider matrix
    w[:100, :100] = 0
    q, s = fp8_blocks(w)
    nr, nc = -(-rows // 128), -(-cols // 128)
    p = torch.nn.functional.pad(w.float(), (0, nc * 128 - cols, 0, nr * 128 - rows)).view(nr, 128, nc, 128)
    rs = scale_of(p.abs().amax((1, 3)))
    rq = (p * (1.0 / rs)[:, None, :, None]).view(nr * 128, -1)[:rows, :cols].clamp(-448, 448).to(FP8)
    assert same_bits(s, rs) and same_bits(q, rq)


def silu64(x):
    gate, up = x.to(F64).chunk(2, -1)
    return gate * torch.sigmoid(gate) * up, up


@pytest.mark.parametrize("width", WIDTHS)
def test_silu_mul(width):
    for rows, std in ((1, 1), (49, 20)):
        x = rand(rows, 2 * width, seed=width, std=std)
        ref, up = silu64(x)
        y = silu_mul(x)
        assert y.dtype == BF16 and ((y.to(F64) - ref).abs() <= (2.0 ** -8 + 2.0 ** -15) * ref.abs() + 2.0 ** -110 * up.abs()).all()
        for group in (0, 32, 64, 128, 256):
            beside = torch.empty_like(y)
            q, s = silu_mul_fp8(x, group=group, y_out=beside)
            assert same_bits(beside, y)
            per = group or width
            n = -(-width // per)
            amax = torch.nn.functional.pad(ref.abs(), (0, n * per - width)).view(rows, n, per).amax(-1)
            assert ((s.to(F64) - (amax / 448).clamp(min=2.0 ** -100)).abs() <= 2.0 ** -14 * amax / 448).all()
            sv = s.to(F64).repeat_interleave(per, 1)[:, :width]
            assert ((q.to(F64) * sv - ref).abs() <= (2.0 ** -4 + 2.0 ** -14) * ref.abs() + 2.0 ** -10 * sv).all()


def test_a_nan_or_an_infinity_stays_in_its_group():
    for value in (float("nan"), float("inf")):
        x = rand(4, 2 * 512, seed=1)
        clean_q, clean_s = silu_mul_fp8(x, group=128)
        x[2, 200] = value
        q, s = silu_mul_fp8(x, group=128)
        keep = torch.ones(4, 512, dtype=torch.bool, device="cuda")
        keep[2, 128:256] = False
        assert torch.equal(q.view(torch.uint8)[keep], clean_q.view(torch.uint8)[keep]) and not torch.isfinite(s[2, 1])
        s[2, 1] = clean_s[2, 1]
        assert torch.equal(s, clean_s)
        w = rand(300, 300 // 8 * 8, seed=2)
        cq, cs = fp8_blocks(w)
        w[140, 150] = value
        q, s = fp8_blocks(w)
        assert not torch.isfinite(s[1, 1]) and torch.equal(s[0], cs[0]) and torch.equal(q[:128].view(torch.uint8), cq[:128].view(torch.uint8))


def test_outputs_streams_and_graph():
    x = rand(70, 2 * 640, seed=3)
    y, (q, s) = silu_mul(x), silu_mul_fp8(x, group=64)
    room = torch.zeros(72, 648, dtype=BF16, device="cuda")
    assert silu_mul(x, out=room[1:71, 8:]) .data_ptr() == room[1:71, 8:].data_ptr()
    assert torch.equal(room[1:71, 8:], y) and (room[0] == 0).all() and (room[71] == 0).all() and (room[:, :8] == 0).all()
    out, scales = torch.empty_like(q), torch.empty_like(s)
    version = out._version
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    silu_mul_fp8(x, group=64, out=out, scales=scales, stream=stream)
    torch.cuda.synchronize()
    assert same_bits(out, q) and torch.equal(scales, s) and out._version > version
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        silu_mul_fp8(x, group=64, out=out, scales=scales)
        w8, ws = fp8_blocks(x)
        r8, rs = fp8_rows(x)
    out.view(torch.uint8).zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(out, q) and same_bits(w8, fp8_blocks(x)[0]) and same_bits(r8, fp8_rows(x)[0])


def test_no_rows():
    assert silu_mul(torch.empty(0, 64, dtype=BF16, device="cuda")).shape == (0, 32)
    q, s = fp8_rows(torch.empty(0, 64, dtype=BF16, device="cuda"), group=32)
    assert q.shape == (0, 64) and s.shape == (0, 2)
    q, s = fp8_blocks(torch.empty(0, 64, dtype=BF16, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 1)


def test_norm_in_both_types():
    x, r, w = rand(33, 640, seed=4), rand(33, 640, seed=5), rand(640, seed=6)
    y, h = add_rms_norm(x, w, r)
    q, s, h8 = add_rms_norm_fp8(x, w, r, group=128)
    beside = torch.zeros_like(y)
    q2, s2, h2 = add_rms_norm_fp8(x, w, r, group=128, y_out=beside)
    assert torch.equal(beside, y) and same_bits(q2, q) and torch.equal(s2, s) and torch.equal(h2, h) and torch.equal(h8, h)


@pytest.mark.parametrize("rows", [[8] * 6, [1, 301, 40]])
def test_an_adapted_mlp_in_8_bits(rows):
    """norm, gate_up, the gated activation and down as a layer runs them, in both types; each step against 64 bits on what
    the step before wrote."""
    hidden, mlp, rank = 640, 896, 32
    ids = [0] * len(rows)
    ids[-1] = 1
    off = [0]
    for n in rows:
        off.append(off[-1] + n)
    T = off[-1]
    x, r, nw = rand(T, hidden, seed=7), rand(T, hidden, seed=8), rand(hidden, seed=9)
    y = torch.empty(T, hidden, dtype=BF16, device="cuda")
    q, s, h = add_rms_norm_fp8(x, nw, r, group=128, y_out=y)

    def project(q, s, x, d_in, d_out, seed):
        w = rand(d_out, d_in, seed=seed, std=d_in ** -0.5)
        a, b = rand(rank, d_in, seed=seed + 1, std=d_in ** -0.5), rand(d_out, rank, seed=seed + 2, std=rank ** -0.5)
        w8, ws = fp8_blocks(w)
        with LoraLinear(d_in, d_out, rank, T, len(rows)) as linear:
            out = linear.forward_fp8(q, s, off, ids, w8, ws, [a], [b], [0.5], x=x)
            torch.cuda.synchronize()
            assert linear.status() == 0
        xv = q.to(F64) * s.to(F64).repeat_interleave(128, 1)[:, :d_in]
        wv = w8.to(F64) * ws.to(F64).repeat_interleave(128, 0)[:d_out].repeat_interleave(128, 1)[:, :d_in]
        ref, S = xv @ wv.T, xv.abs() @ wv.abs().T
        t = off[-2]
        u = 0.5 * x[t:].to(F64) @ a.to(F64).T
        ref[t:] += u @ b.to(F64).T
        S[t:] += u.abs() @ b.to(F64).abs().T
        # (the bound of the projection's own tests; U's rounding and its sums: 2^-8 and less of |U| |B|^T)
        bound = 2.0 ** -8 * ref.abs() + 2.0 ** -13 * S
        bound[t:] += 1.1 * (2.0 ** -8 * u.abs() + 2.0 ** -13 * 0.5 * x[t:].to(F64).abs() @ a.to(F64).abs().T) @ b.to(F64).abs().T
        assert ((out.to(F64) - ref).abs() <= bound).all()
        # 8 bits of both operands are within 2^-4 of each, the products' errors independent: 4 % of the norm is far over them
        full = x.to(F64) @ w.to(F64).T
        full[t:] += u @ b.to(F64).T
        assert (ref - full).norm() <= 0.08 * full.norm()
        return out

    gu = project(q, s, y, hidden, 2 * mlp, 10)
    z = torch.empty(T, mlp, dtype=BF16, device="cuda")
    q2, s2 = silu_mul_fp8(gu, group=128, y_out=z)
    ref, up = silu64(gu)
    assert ((z.to(F64) - ref).abs() <= (2.0 ** -8 + 2.0 ** -15) * ref.abs() + 2.0 ** -110 * up.abs()).all()
    assert project(q2, s2, z, mlp, hidden, 20).shape == (T, hidden)
