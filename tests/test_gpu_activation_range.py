"""silu_mul where e^-g leaves fp32's range and the up projection is large: against 64 bits.

h = e^(-|g|/2) is off by at most (2 + 1.16 |g| / 2) units of 2^-23, its square by twice that; with the quotient's and the
products' roundings less than 2^-15 in all for |g| <= 206, past which y is under 2^-148 for any u of bf16. A subnormal h is off
by 2^-149 at most, y then by 2^-140. bf16 rounds by half a step, 2^-8 of the value or 2^-134 among its subnormals."""
import pytest
import torch

from mixed_lora_projection_gb300 import silu_mul, silu_mul_fp8

pytestmark = pytest.mark.gpu

F64, BF16 = torch.float64, torch.bfloat16


def reference(x):
    g, u = x.to(F64).chunk(2, -1)
    return g * torch.sigmoid(g) * u


@pytest.mark.parametrize("lo,hi", [(-90.0, -86.0), (-130.0, -88.0), (-206.0, -170.0), (-1.0, 1.0), (80.0, 90.0)])
@pytest.mark.parametrize("size", [1.0, 1e20, 1e37])
def test_large_up_projections(lo, hi, size):
    n = 4096
    g = torch.linspace(lo, hi, n, device="cuda").to(BF16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    u = (size * torch.randn(n, generator=gen, device="cuda")).to(BF16)
    x = torch.cat([g, u])[None]
    ref = reference(x)
    keep = ref.abs() < 3.3e38
    assert keep.all() or lo > 0
    y = silu_mul(x)
    assert ((y.to(F64) - ref).abs() <= (2.0 ** -8 + 2.0 ** -15) * ref.abs() + 2.0 ** -133)[keep].all()


def test_infinities_and_nan():
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([inf, inf, -inf, nan, 1.0, -300.0, 300.0, 0.0], dtype=BF16, device="cuda")
    u = torch.tensor([2.0, -2.0, 1.0, 1.0, nan, 3e38, 2.0, 5.0], dtype=BF16, device="cuda")
    y = silu_mul(torch.cat([g, u])[None])[0]
    assert y[0] == inf and y[1] == -inf and torch.isnan(y[2:5]).all() and y[5] == 0 and y[6] == 600 and y[7] == 0


def test_eight_bits_take_the_same_values():
    # one group whose values all stand where e^-g is past 2^126
    g = torch.full((1, 128), -88.0, dtype=BF16, device="cuda")
    u = torch.linspace(1e36, 1e38, 128, device="cuda").to(BF16)[None]
    x = torch.cat([g, u], -1)
    ref = reference(x)
    q, s = silu_mul_fp8(x, group=128)
    assert abs(s.item() * 448 / ref.abs().max().item() - 1) <= 2.0 ** -14
    assert ((q.to(F64) * s.to(F64) - ref).abs() <= (2.0 ** -4 + 2.0 ** -14) * ref.abs() + 2.0 ** -10 * s.to(F64)).all()


@pytest.mark.parametrize("rows", [5, 300, 700])
def test_a_row_takes_nothing_of_gates_beside_it(rows):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    x = (torch.randn(rows, 2 * 17408, generator=gen, device="cuda") * 2).to(BF16)
    y, (q, s) = silu_mul(x), silu_mul_fp8(x)
    far = x.clone()
    far[1::2, :17408:5] = -100.0
    z, (r, t) = silu_mul(far), silu_mul_fp8(far)
    assert torch.equal(y[::2], z[::2]) and torch.equal(q[::2].view(torch.uint8), r[::2].view(torch.uint8)) and torch.equal(s[::2], t[::2])
    rest = torch.arange(17408, device="cuda") % 5 != 0
    assert torch.equal(y[:, rest], z[:, rest])
