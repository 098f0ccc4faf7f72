"""What lora_linear_forward_fp8 launches (lora_linear_describe_fp8), and its forms that a batch's size alone selects, against
64 bits under the bound of test_gpu_fp8.py."""
import pytest
import torch

from mixed_lora_projection_gb300 import LoraLinear
from test_gpu_fp8 import BF16, Case

pytestmark = pytest.mark.gpu


def described(c):
    return c.linear.describe_fp8(c.T, c.off, c.ids)


# long prompts: the bf16 kernel's units run the shrink, on SM pairs, from an uploaded list; groups of an odd number of tiles
# are padded
@pytest.mark.parametrize("rows,ids", [([16384], [1]), ([5400, 5150, 30, 4400], [1, 2, 0, 3]), ([48, 16300], [0, 1])])
def test_shrink_of_a_long_prompt(rows, ids):
    c = Case(5120, 2056, 256, rows, ids, seed=len(rows))
    d = described(c)
    assert (d["shrink"], d["shrink_cluster"], d["uploaded"]) == (2, 2, 1), d
    y = c.run()
    c.check(y)
    assert torch.equal(c.run(), y)


def test_what_is_described():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ll = LoraLinear(5120, 12288, 256, 2048, 16)
    none = ll.describe_fp8(0, [0], [])
    assert not any(none.values())
    base = ll.describe_fp8(48, [0, 48], [0])
    assert base["shrink"] == base["shrink_grid"] == base["merged"] == base["uploaded"] == 0 and 1 <= base["grid"] <= sms
    one = ll.describe_fp8(48, [0, 48], [1])
    assert one["shrink"] == 1 and one["shrink_cluster"] >= 1 and 1 <= one["shrink_grid"] <= sms and one["merged"] == 0
    many = ll.describe_fp8(48, list(range(0, 49, 8)), [1, 2, 3, 4, 5, 6])
    assert many["merged"] == 1 and many["shrink"] == 1 and many["cluster"] == many["k_parts"]
    wide = ll.describe_fp8(2048, [0, 2048], [0])
    assert wide["cluster"] == 2 and wide["k_parts"] == 1 and wide["tile_n"] == 256 and wide["grid"] == sms // 2 * 2
    assert ll.describe_fp8(48, [0, 48], [2 ** 31 - 1])["shrink"] == 1
    for T, off, ids in ((2049, [0, 2049], [0]), (48, [0, 47], [0]), (48, [1, 48], [0]), (48, [0, 48], [-1]), (1, [0] + [1] * 17, [0] * 17)):
        with pytest.raises(Exception, match="invalid argument"):
            ll.describe_fp8(T, off, ids)
    ll.close()
    with pytest.raises(Exception):
        ll.describe_fp8(48, [0, 48], [0])
    odd = LoraLinear(264, 136, 16, 48, 4)                    # (d_in no multiple of 16: bf16 alone)
    with pytest.raises(Exception, match="invalid argument"):
        odd.describe_fp8(48, [0, 48], [0])


# five to eight adapters, of as many rows that no tile holds two and the bf16 kernel's units would run the shrink
@pytest.mark.parametrize("d_in,rows,ids", [(1024, [768] * 5, [1, 2, 3, 4, 5]), (1024, [512] * 8, [8, 7, 6, 5, 4, 3, 2, 1]), (256, [500] * 7, [1, 2, 3, 4, 5, 6, 7])])
def test_up_to_eight_adapters_are_captured(d_in, rows, ids):
    c = Case(d_in, 2056, 256, rows, ids, seed=len(rows))
    d = described(c)
    assert d["merged"] == 0 and d["shrink"] == 1 and d["uploaded"] == 0, d
    y = c.run()
    c.check(y)
    out = torch.zeros_like(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(y=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)


# rows without an adapter in tiles of their own, which share an SM pair with an adapter's tile, before and behind it
@pytest.mark.parametrize("rows,ids", [([128, 128], [0, 1]), ([128, 300, 84], [0, 1, 0]), ([256, 300], [0, 1]), ([384, 128, 640, 5], [0, 1, 0, 2]),
                                      ([128, 128], [1, 0]), ([128, 128, 128, 100], [2, 0, 1, 0])])
def test_an_adapter_with_a_nan_stays_off_tiles_without_one(rows, ids):
    c = Case(1024, 12288, 64, rows, ids, seed=len(rows))
    d = described(c)
    assert (d["cluster"], d["tile_n"], d["merged"]) == (2, 256, 0), d
    y = c.run()
    c.check(y)
    c.b[0][5, 3] = float("nan")
    c.b[0][4097] = float("inf")
    bad = c.run()
    named = {t // 128 for i, a in enumerate(ids) if a == 1 for t in range(c.off[i], c.off[i + 1])}
    i = ids.index(1)
    assert torch.isnan(bad[c.off[i]:c.off[i + 1], 5]).all()
    rest = [t for t in range(c.T) if t // 128 not in named]
    assert len(rest) >= 84 and torch.equal(bad[rest], y[rest])
    tile = [t for t in range(c.T) if t // 128 in named]
    assert torch.equal(bad[tile][:, 6:4097], y[tile][:, 6:4097])


# LORA_OPT_MAX_CTAS: neither launch has more CTAs; the shrink's take several units then
@pytest.mark.parametrize("d_in,d_out,rank,rows,ids", [
    (5120, 12288, 256, [48], [1]),
    (6144, 5120, 64, [1] * 8, [8, 7, 6, 5, 4, 3, 2, 1]),
    (1024, 1288, 40, [60] * 7, [1, 2, 1, 2, 1, 2, 1]),
    (1024, 2568, 256, [700, 5, 300], [1, 0, 2]),
    (5120, 5120, 256, [1500], [1]),
    (640, 264, 24, [4000], [1]),
])
@pytest.mark.parametrize("most", [2, 3, 9, 40, 151])
def test_fewer_sms(d_in, d_out, rank, rows, ids, most):
    from mixed_lora_projection_gb300 import _lib
    c = Case(d_in, d_out, rank, rows, ids, seed=d_in + rank)
    y = c.run()
    before = described(c)
    c.linear.set_option(_lib.OPT_MAX_CTAS, most)
    d = described(c)
    assert 1 <= d["grid"] <= most and 1 <= d["shrink_grid"] <= most, d
    z = c.run()
    c.check(z)
    assert all(torch.equal(c.run(), z) for _ in range(3))
    c.linear.set_option(_lib.OPT_MAX_CTAS, 0)
    assert described(c) == before and torch.equal(c.run(), y)


def test_more_units_of_the_shrink_than_sms():
    # (pairs of a tile and an adapter, by columns of the rank; and many tiles of few rows)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = Case(640, 136, 256, [1, 1] * 100, [1, 2] * 100, seed=1)
    c.check(c.run())
    d = described(c)
    assert d["grid"] <= sms and d["shrink_grid"] <= sms
    # a wait that runs out while CTAs have further units before them
    from mixed_lora_projection_gb300 import _lib
    e = Case(640, 264, 16, [30] * 8, [1, 2, 3, 4, 5, 6, 7, 8], seed=2)
    e.linear.set_option(_lib.OPT_MAX_CTAS, 3)
    y = e.run()
    e.check(y)
    e.linear.set_option(_lib.OPT_WAIT_LIMIT_US, 2000)
    e.linear.set_option(_lib.OPT_DEBUG_STALL, 1)
    e.run()
    assert e.linear.status() == _lib.LORA_ETIMEOUT
    e.linear.set_option(_lib.OPT_DEBUG_STALL, 0)
    assert e.linear.status(reset=True) == _lib.LORA_ETIMEOUT
    e.linear.set_option(_lib.OPT_WAIT_LIMIT_US, 4000000)
    assert torch.equal(e.run(), y) and e.linear.status() == 0


# the blocks of U of tiles that hold several adapters lie in the projection's own U where that is long enough
@pytest.mark.parametrize("most,segs", [(48, 6), (128, 2), (300, 16), (2047, 8), (2048, 8), (16384, 2)])
@pytest.mark.parametrize("d_in,d_out", [(640, 264), (6144, 5120)])
def test_several_adapters_on_handles_of_any_size(most, segs, d_in, d_out):
    rows = [max(1, min(most, 300) // segs)] * segs
    ids = [1 + i % 8 for i in range(segs)]
    c = Case(d_in, d_out, 64, rows, ids, seed=most)
    c.linear.close()
    c.linear = LoraLinear(d_in, d_out, 64, most, segs)
    y = c.run()
    # (tiles are merged where they would read much of the base several times)
    assert described(c)["merged"] == 1 or d_out == 264 or (most, segs) not in ((48, 6), (2047, 8), (2048, 8))
    c.check(y)
    # bf16 and 8-bit calls of one handle in turn, and one adapter's tiles beside none's: the zeros stay zeros
    w = torch.randn(d_out, d_in, device="cuda").to(BF16)
    base, z = c.x[:c.T], None
    for _ in range(3):
        b = c.linear.forward(base, c.off, c.ids, w, c.a, c.b, c.s)
        one = c.linear.forward_fp8(c.x8, c.xs, [0, c.T], [1], c.w8, c.ws, c.a, c.b, c.s, x=c.x)
        assert torch.equal(c.run(), y)
        if z is not None:
            assert torch.equal(b, z[0]) and torch.equal(one, z[1])
        z = b, one


def test_one_segment_or_odd_widths_keep_no_blocks():
    a = LoraLinear(640, 264, 64, 48, 1)
    assert a.describe_fp8(48, [0, 48], [1])["merged"] == 0
    b = LoraLinear(648, 264, 64, 48, 4)                      # (not for 8 bits)
    x, w = torch.randn(48, 648, device="cuda").to(BF16), torch.randn(264, 648, device="cuda").to(BF16)
    assert torch.isfinite(b.forward(x, [0, 48], [0], w, [], [], [])).all()
