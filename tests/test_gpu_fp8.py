"""The projection with 8-bit activations and base (lora_linear_forward_fp8) against 64 bits on the values that its
operands stand for.

Bound of an output: it is rounded to bf16 once, half a step, 2^-8 of the value; products of e4m3 values are exact in
fp32, and a sum of n fp32 terms in any order is off by at most n 2^-24 of the sum of their magnitudes, S: the 128 of a
group's products, the groups' scaled sums (each with the rounding of its scales' product and its own) and the expand
make at most n = 128 + 2 x 136 + 256 < 2^10 roundings on the way of one term, 2^-14 S. The tensor cores' own sums carry
fewer guard bits than an fp32 addition: 2^-13 S allows for two of them. U is rounded to bf16: 2^-8 of |U| |B|^T."""
import pytest
import torch

from mixed_lora_projection_gb300 import LoraLinear

pytestmark = pytest.mark.gpu

F64, BF16, FP8 = torch.float64, torch.bfloat16, torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Case:
    def __init__(self, d_in, d_out, rank, rows, ids, seed=0, spread=6):
        g = gen(seed)
        dev = torch.device("cuda")
        self.d_in, self.d_out, self.rank, self.ids = d_in, d_out, rank, list(ids)
        self.off = [0]
        for n in rows:
            self.off.append(self.off[-1] + n)
        self.T = T = self.off[-1]
        G, NB = -(-d_in // 128), -(-d_out // 128)
        # codes over the whole range of e4m3, scales over 2^spread
        def codes(r, c):
            return (torch.randn(r, c, generator=g, device=dev) * 60).clamp(-448, 448).to(FP8)
        def scales(*s):
            return torch.exp2(torch.rand(s, generator=g, device=dev) * spread - spread / 2)
        self.x8, self.xs = codes(T, d_in), scales(T, G) / 60
        self.w8, self.ws = codes(d_out, d_in), scales(NB, G) / 60 * d_in ** -0.5
        na = max(ids, default=0)
        self.x = torch.randn(T, d_in, generator=g, device=dev).to(BF16)
        self.a = [(torch.randn(rank, d_in, generator=g, device=dev) * d_in ** -0.5).to(BF16) for _ in range(na)]
        self.b = [(torch.randn(d_out, rank, generator=g, device=dev) * rank ** -0.5).to(BF16) for _ in range(na)]
        self.s = [1.0, -0.5, 2.0, 0.25, 1.5, 0.75][:na] + [1.0] * max(0, na - 6)
        self.linear = LoraLinear(d_in, d_out, rank, max(T, 1), max(1, len(ids)))

    def run(self, **kw):
        kw.setdefault("x", self.x)
        return self.linear.forward_fp8(self.x8, self.xs, self.off, self.ids, self.w8, self.ws, self.a, self.b, self.s, **kw)

    def reference(self):
        """(y, bound) in 64 bits."""
        x = self.x8.to(F64) * self.xs.to(F64).repeat_interleave(128, 1)[:, :self.d_in]
        w = self.w8.to(F64) * self.ws.to(F64).repeat_interleave(128, 0)[:self.d_out].repeat_interleave(128, 1)[:, :self.d_in]
        y, S, more = x @ w.T, x.abs() @ w.abs().T, torch.zeros(self.T, self.d_out, dtype=F64, device=x.device)
        for i, a in enumerate(self.ids):
            r = slice(self.off[i], self.off[i + 1])
            if a:
                A, B, xr = self.a[a - 1].to(F64), self.b[a - 1].to(F64), self.x[r].to(F64)
                u = xr @ A.T * self.s[a - 1]
                y[r] += u @ B.T
                S[r] += u.abs() @ B.abs().T
                more[r] = (2.0 ** -8 * u.abs() + 2.0 ** -13 * abs(self.s[a - 1]) * (xr.abs() @ A.abs().T)) @ B.abs().T
        return y, 2.0 ** -8 * y.abs() + 2.0 ** -13 * S + 1.01 * more

    def check(self, y):
        assert self.linear.status() == 0
        ref, bound = self.reference()
        assert y.shape == ref.shape and y.dtype == BF16
        worst = ((y.to(F64) - ref).abs() / (bound + 1e-300)).max().item()
        assert worst <= 1.0, worst


@pytest.mark.parametrize("d_in,d_out,rank,rows,ids", [
    (128, 128, 16, [1], [0]),
    (16, 8, 8, [1], [0]),
    (16, 8, 8, [1], [1]),
    (144, 136, 8, [3], [1]),
    (256, 512, 16, [32, 32], [0, 1]),
    (6144, 5120, 256, [1], [0]),
    (6144, 5120, 256, [1], [1]),
    (1040, 1288, 40, [127], [0]),
    (5120, 1288, 200, [48], [0]),
    (17408, 640, 256, [8, 0, 9], [1, 2, 0]),
    (1280, 2568, 256, [129], [1]),
    (640, 520, 64, [100, 100, 100], [0, 2, 1]),
    (256, 136, 16, [384], [0]),
    (2064, 1032, 72, [385], [1]),
    (640, 520, 256, [200, 1, 400, 33], [0, 1, 0, 2]),
    (512, 264, 24, [128, 128, 128, 128, 7], [0, 1, 0, 1, 2]),
    (1024, 8, 8, [700], [1]),
    (5120, 2056, 256, [2049], [1]),
    (384, 40, 16, [16384], [0]),
])
def test_against_64_bits(d_in, d_out, rank, rows, ids):
    c = Case(d_in, d_out, rank, rows, ids, seed=d_in + d_out + rank)
    y = c.run()
    c.check(y)
    assert torch.equal(c.run(), y)                          # the same call, the same bits


@pytest.mark.parametrize("T", list(range(1, 20)) + [31, 63, 64, 65, 96, 111, 128, 130, 255, 256, 257, 383, 511, 512, 513])
def test_row_counts(T):
    c = Case(384, 264, 16, [T], [T % 2], seed=T)
    c.check(c.run())


@pytest.mark.parametrize("d_out", [8, 24, 32, 40, 64, 96, 120, 128, 136, 160, 256, 264, 384, 1000, 4104])
def test_output_widths(d_out):
    for T in (5, 520):
        c = Case(1536, d_out, 32, [T], [1], seed=d_out)
        c.check(c.run())


@pytest.mark.parametrize("d_in", [16, 32, 112, 128, 144, 240, 256, 272, 384, 1000 // 16 * 16, 2048, 2064])
def test_input_widths(d_in):
    for T in (17, 600):
        c = Case(d_in, 200, 8, [T], [0], seed=d_in)
        c.check(c.run())


def test_many_segments_travel_in_an_uploaded_list():
    ids = [i % 6 for i in range(90)]
    c = Case(256, 136, 32, [1 + 7 * i % 50 for i in range(90)], ids, seed=3)
    y = c.run()
    c.check(y)
    # the host's lists are read before the call returns, and calls in a row keep their own
    ys = [c.run() for _ in range(12)]
    assert all(torch.equal(v, y) for v in ys)


def test_rows_around_the_output_stay():
    for T in (5, 700):
        c = Case(256, 264, 16, [T], [1], seed=T)
        room = torch.full((T + 2, 264), 7.0, dtype=BF16, device="cuda")
        c.check(c.run(y=room[1:T + 1]))
        assert (room[0] == 7).all() and (room[T + 1] == 7).all()


def test_a_row_with_nan_or_infinity_stays_alone():
    for T in (60, 600):
        c = Case(640, 264, 16, [T], [0], seed=9)
        c.x8.view(torch.uint8)[3, 200] = 0x7f                # NaN
        c.xs[5, 1] = float("inf")
        c.xs[7, 2] = float("nan")
        y = c.run()
        assert torch.isnan(y[3]).all() and torch.isnan(y[7]).all() and not torch.isfinite(y[5]).any()
        rest = [t for t in range(T) if t not in (3, 5, 7)]
        ref, bound = c.reference()
        assert ((y.to(F64) - ref).abs() <= bound)[rest].all()


def test_zero_scales_give_zeros():
    c = Case(256, 136, 16, [40], [0], seed=2)
    c.xs.zero_()
    assert (c.run() == 0).all()


def test_rows_without_adapters_need_no_bf16_input():
    c = Case(256, 136, 16, [3, 4], [0, 0], seed=2)
    c.check(c.run(x=None))
    # segments without rows name adapters in vain
    d = Case(256, 136, 16, [3, 0], [0, 1], seed=2)
    d.check(d.run(x=None))
    e = Case(256, 136, 16, [3, 4], [0, 1], seed=2)
    with pytest.raises(Exception, match="invalid argument"):
        e.run(x=None)


def test_no_rows():
    c = Case(256, 136, 16, [0], [0])
    assert c.run().shape == (0, 136)


def test_graph_and_streams():
    cases = [Case(1280, 520, 32, rows, ids, seed=i) for i, (rows, ids) in enumerate([([8] * 6, [0] * 6), ([8, 300], [0, 1]), ([700], [1])])]
    want = [c.run() for c in cases]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, o in zip(cases, outs):
            c.run(y=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    # each on a stream of its own, side by side, and through the stream argument
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in cases]
    for _ in range(20):
        for g, c, s in zip(got, cases, streams):
            g.append(c.run(stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for g, w in zip(got, want) for y in g)


def test_chained_calls_read_what_the_call_before_wrote():
    # the second projection's activations are brought to 8 bits by torch in between, on one stream, without a wait
    a = Case(512, 512, 16, [48], [0], seed=1)
    b = Case(512, 264, 16, [48], [0], seed=2)
    want = None
    for _ in range(50):
        y = a.run()
        b.x8.copy_(y.clamp(-448, 448).to(FP8))
        z = b.run()
        want = z if want is None else want
        assert torch.equal(z, want)
    b.check(want)


@pytest.mark.parametrize("T,ids", [(48, 0), (700, 1)])
def test_a_wait_that_runs_out_is_reported(T, ids):
    from mixed_lora_projection_gb300 import _lib
    c = Case(640, 264, 16, [T], [ids], seed=1)
    y = c.run()
    c.linear.set_option(_lib.OPT_WAIT_LIMIT_US, 2000)
    c.linear.set_option(_lib.OPT_DEBUG_STALL, 1)
    c.run()
    assert c.linear.status() == _lib.LORA_ETIMEOUT
    c.linear.set_option(_lib.OPT_DEBUG_STALL, 0)
    assert c.linear.status(reset=True) == _lib.LORA_ETIMEOUT
    c.linear.set_option(_lib.OPT_WAIT_LIMIT_US, 4000000)
    assert torch.equal(c.run(), y) and c.linear.status() == 0


# the shrink's rank in several tiles of columns, whole and not, one and more parts of K
@pytest.mark.parametrize("d_in,d_out,rank,rows,ids", [
    (5120, 264, 200, [48], [1]),
    (17408, 136, 256, [33], [1]),
    (6144, 264, 248, [130, 5], [1, 2]),
    (5120, 136, 40, [300], [1]),
    (4096, 136, 72, [16], [1]),
    (5120, 1032, 256, [8, 8, 8, 340, 8], [0, 1, 2, 3, 4]),
    (1024, 520, 136, [2, 1, 1, 600, 90], [1, 0, 2, 1, 3]),
])
def test_adapters_of_few_rows(d_in, d_out, rank, rows, ids):
    c = Case(d_in, d_out, rank, rows, ids, seed=d_in + rank)
    y = c.run()
    c.check(y)
    assert torch.equal(c.run(), y)


@pytest.mark.parametrize("rows,ids", [([48], [1]), ([5, 343], [0, 1]), ([700], [1]), ([2048], [1]), ([8] * 70, [0, 1] * 35)])
@pytest.mark.parametrize("captured", [False, True])
def test_operands_written_right_before(rows, ids, captured):
    # the base runs beside the shrink and waits for it alone: what the norm before both has written is what it reads
    from mixed_lora_projection_gb300 import add_rms_norm_fp8
    if captured and len(rows) > 60:
        pytest.skip("a work list of 70 segments is uploaded, which a capture refuses")
    c = Case(1024, 1288, 64, rows, ids, seed=len(rows))
    g = gen(5)
    n = 12
    hs = [torch.randn(c.T, c.d_in, generator=g, device="cuda").to(BF16) for _ in range(n)]
    w = torch.rand(c.d_in, generator=g, device="cuda").to(BF16)
    ys = [torch.empty(c.T, c.d_out, dtype=BF16, device="cuda") for _ in range(n)]

    def both():
        for h, y in zip(hs, ys):
            add_rms_norm_fp8(h, w, group=128, out=c.x8, scales=c.xs, y_out=c.x)
            c.run(y=y)

    both()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
        for y in ys:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
    for h, y in zip(hs, ys):
        add_rms_norm_fp8(h, w, group=128, out=c.x8, scales=c.xs, y_out=c.x)
        torch.cuda.synchronize()
        assert torch.equal(c.run(), y)
        torch.cuda.synchronize()
    c.check(ys[-1])


def test_fewer_sms_and_timing():
    from mixed_lora_projection_gb300 import _lib
    for rows, ids in (([48], [1]), ([300, 48], [1, 0]), ([1500], [1])):
        c = Case(2048, 1288, 64, rows, ids, seed=len(rows))
        for most in (2, 9, 40, 0):
            c.linear.set_option(_lib.OPT_MAX_CTAS, most)
            c.check(c.run())
        c.linear.set_option(_lib.OPT_TIMING, 1)
        c.check(c.run())


def test_refused_arguments():
    c = Case(256, 136, 16, [3, 4], [0, 1], seed=2)
    good = dict(x8=c.x8, x_scales=c.xs, seg_offsets=c.off, seg_ids=c.ids, W8=c.w8, W_scales=c.ws, A=c.a, B=c.b, scales=c.s, x=c.x, y=None)
    wide = torch.zeros(7, 512, device="cuda")

    def refused(error, **bad):
        with pytest.raises(error):
            c.linear.forward_fp8(**{**good, **bad})

    refused(TypeError, x8=c.x)
    refused(TypeError, x_scales=c.xs.to(BF16))
    refused(TypeError, W8=c.w8.view(torch.uint8))
    refused(TypeError, x=c.x.float())
    refused(TypeError, A=[c.a[0].float()])
    refused(TypeError, y=torch.zeros(7, 136, device="cuda"))
    refused(TypeError, seg_ids=None)
    refused(ValueError, x8=wide.to(FP8)[:, :256])
    refused(ValueError, x8=c.x8[0])
    refused(ValueError, x_scales=c.xs[:, :1])
    refused(ValueError, W_scales=c.ws[:1])
    refused(ValueError, W8=c.w8[:128])
    refused(ValueError, W8=c.w8.cpu())
    refused(ValueError, x=c.x.cpu())
    refused(ValueError, x=c.x[:6])
    refused(ValueError, B=[c.b[0].T])
    refused(ValueError, scales=[1.0, 2.0])
    refused(ValueError, seg_offsets=[0, 3])
    refused(ValueError, seg_offsets=[0, 3, 6])
    refused(ValueError, y=torch.zeros(6, 136, dtype=BF16, device="cuda"))
    refused(Exception, seg_ids=[0, 2])                       # no such adapter
    refused(Exception, seg_offsets=[0, 8, 7])
    refused(Exception, y=c.x8.view(BF16).view(-1)[:7 * 120].view(7, 120))
    c.check(c.run())
    c.linear.close()
    with pytest.raises(Exception):
        c.run()


# tiles that hold rows of several adapters: one expand each, over parts of K, single CTAs and pairs
@pytest.mark.parametrize("d_in,d_out,rank,rows,ids", [
    (256, 136, 16, [1, 1], [1, 2]),
    (5120, 1288, 256, [1, 0, 1, 1, 0], [1, 0, 0, 2, 2]),
    (6144, 5120, 256, [3, 1, 7, 2], [1, 2, 3, 4]),
    (6144, 5120, 64, [1] * 8, [8, 7, 6, 5, 4, 3, 2, 1]),
    (1024, 2568, 200, [0, 18, 5, 10, 3, 11, 6, 15, 26], [2, 2, 1, 0, 2, 2, 0, 1, 2]),
    (1024, 2568, 40, [11, 1, 44, 86, 81], [0, 1, 1, 0, 2]),
    (1024, 1288, 256, [100, 27, 1, 1, 126], [1, 2, 1, 2, 3]),
    (640, 264, 24, [60, 60, 60, 60, 60, 60, 60], [1, 2, 1, 2, 1, 2, 1]),
    (17408, 264, 256, [20, 20], [1, 2]),
    (2064, 5128, 72, [64, 64, 64, 64, 300], [1, 0, 2, 1, 0]),
    (1024, 34816, 64, [8, 8, 301, 8, 600], [0, 1, 2, 0, 1]),
    (1024, 5120, 64, [70] * 9, [1, 2, 3, 1, 2, 3, 1, 2, 3]),
    (384, 520, 16, [2] * 48, [1, 2] * 24),
    (384, 520, 16, [2] * 50, [1, 2] * 25),                  # (more segments than the parameters hold)
    (384, 520, 16, [4] * 9, list(range(1, 10))),            # (more adapters)
])
def test_tiles_of_several_adapters(d_in, d_out, rank, rows, ids):
    c = Case(d_in, d_out, rank, rows, ids, seed=d_out + rank)
    y = c.run()
    c.check(y)
    assert all(torch.equal(c.run(), y) for _ in range(3))


def test_several_adapters_captured_and_in_turn():
    # calls of one handle whose tiles are merged and not, in turn: the blocks of U are each call's own
    cases = [Case(1024, 1288, 64, rows, ids, seed=i) for i, (rows, ids) in enumerate([
        ([1] * 8, [1, 2, 3, 4, 5, 6, 7, 8]), ([128, 3], [1, 2]), ([300], [1]), ([9, 120, 30, 7], [2, 1, 0, 3])])]
    for c in cases[1:]:
        c.linear.close()
    shared = LoraLinear(1024, 1288, 64, 400, 16)
    for c in cases:
        c.linear = shared
    want = [c.run() for c in cases]
    for c, y in zip(cases, want):
        c.check(y)
    outs = [torch.zeros_like(y) for y in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            for c, o in zip(cases, outs):
                c.run(y=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, y) for o, y in zip(outs, want))


def test_a_wait_that_runs_out_with_several_adapters():
    from mixed_lora_projection_gb300 import _lib
    c = Case(640, 264, 16, [4, 5, 6], [1, 2, 3], seed=1)
    y = c.run()
    c.linear.set_option(_lib.OPT_WAIT_LIMIT_US, 2000)
    c.linear.set_option(_lib.OPT_DEBUG_STALL, 1)
    c.run()
    assert c.linear.status() == _lib.LORA_ETIMEOUT
    c.linear.set_option(_lib.OPT_DEBUG_STALL, 0)
    assert c.linear.status(reset=True) == _lib.LORA_ETIMEOUT
    c.linear.set_option(_lib.OPT_WAIT_LIMIT_US, 4000000)
    assert torch.equal(c.run(), y) and c.linear.status() == 0


# several stages an expand beside few of the base, many units a block: the ring is no shorter than the stages that pass
# between two uses of a buffer
@pytest.mark.parametrize("d_in,d_out,rank,rows,ids", [
    (128, 40960, 256, [48], [1]),
    (256, 40960, 256, [40, 60], [1, 2]),
    (128, 40960, 192, [20, 20, 8], [1, 2, 3]),
    (5120, 34816, 256, [8] * 6, [1, 2, 3, 4, 0, 0]),
    (384, 40960, 256, [100, 100, 100, 400], [1, 2, 1, 2]),
    (128, 20480, 256, [1500], [1]),
])
def test_more_expands_than_base_blocks(d_in, d_out, rank, rows, ids):
    c = Case(d_in, d_out, rank, rows, ids, seed=d_in + rank)
    y = c.run()
    c.check(y)
    assert all(torch.equal(c.run(), y) for _ in range(3))


@pytest.mark.parametrize("rows,d_out", [([5, 7, 4, 9], 1288), ([60, 100, 40, 80], 1288), ([90, 300, 100, 150, 90, 20], 20480)])
def test_an_adapter_with_a_nan_stays_off_other_adapters_rows(rows, d_out):
    # (rows without one may share a tile with it and add zero times its values, as in the bf16 projection)
    ids = [1, 2, 0, 3, 1, 0][:len(rows)]
    c = Case(1024, d_out, 64, rows, ids, seed=4)
    y = c.run()
    c.check(y)
    c.b[1][5, 3] = float("nan")
    c.b[1][9] = float("inf")
    c.a[1][2, 2] = float("inf")
    bad = c.run()
    mine = slice(c.off[1], c.off[2])
    assert torch.isnan(bad[mine, 5]).all()
    for i, a in enumerate(ids):
        if a not in (0, 2):
            r = slice(c.off[i], c.off[i + 1])
            assert torch.equal(bad[r], y[r])
