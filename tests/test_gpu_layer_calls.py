"""How the operators between the projections are called, on a GPU: streams, aliases, refusals, calls of many
sequences. Tolerances are those that test_gpu_layer.py derives."""
import pytest
import torch

from test_gpu_layer import BF16_TOL, DEV, F64, U, Case, bound, gen, norm_ref, randn, within

pytestmark = pytest.mark.gpu


def stream_of_block(t):
    """The stream whose pool a tensor's memory is from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no block of the allocator")


# name -> call(stream), its outputs; inputs are made once
def operators():
    from mixed_lora_projection_gb300 import PagedAttention, add_rms_norm, add_rms_norm_fp8, kv_append
    g = gen(1)
    c = Case([1, 40], [90, 400], 8, 2, 128, 16)
    x, r, w = randn(g, 256, 1024), randn(g, 256, 1024), randn(g, 1024)
    k, v = randn(g, 41, 2, 128), randn(g, 41, 2, 128)
    cos, sin = torch.rand(400, 32, generator=g, device=DEV), torch.rand(400, 32, generator=g, device=DEV)
    attn = PagedAttention(8, 2, 128, 16, 41, 2)
    return {
        "norm": lambda s: add_rms_norm(x, w, r, stream=s),
        "norm to 8 bits": lambda s: add_rms_norm_fp8(x, w, r, group=64, stream=s),
        "append": lambda s: (kv_append(c.q, k, v, c.off, c.kv, c.table, c.k, c.v, cos, sin, stream=s),),
        "attention": lambda s: (attn.forward(c.q, c.k, c.v, c.off, c.kv, c.table, stream=s),),
    }


def projections():
    from mixed_lora_projection_gb300 import LoraLinear, w4_repack
    g = gen(2)
    x, w = randn(g, 48, 256), randn(g, 512, 256)
    a, b = randn(g, 16, 256), randn(g, 512, 16)
    q = torch.randint(0, 256, (512, 128), generator=g, device=DEV, dtype=torch.uint8)
    scales = randn(g, 2, 512)
    ll = LoraLinear(256, 512, 16, 48)
    packed = w4_repack(q)
    return {
        "projection": lambda s: (ll.forward(x, [0, 20, 48], [0, 1], w, [a], [b], [1.0], stream=s),),
        "4-bit projection": lambda s: (ll.forward_w4(x, [0, 20, 48], [0, 1], packed, scales, [a], [b], [1.0], stream=s),),
        "4-bit layout": lambda s: (w4_repack(q, stream=s),),
    }


@pytest.mark.parametrize("name", ["norm", "norm to 8 bits", "append", "attention", "projection", "4-bit projection", "4-bit layout"])
def test_outputs_belong_to_the_stream_of_the_call(name):
    call = {**operators(), **projections()}[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    here = torch.cuda.current_stream().cuda_stream
    for out in call(None):
        assert stream_of_block(out) == here
    torch.cuda.synchronize()                                  # one handle's calls go one after another
    for out in call(s):
        assert stream_of_block(out) == s.cuda_stream
    assert torch.cuda.current_stream().cuda_stream == here
    # a buffer of this stream, freed with its reader still queued, is not the call's to write
    sizes = [(t.shape, t.dtype) for t in want]
    old = [torch.full(shape, 3.0, device=DEV).to(dtype) for shape, dtype in sizes]
    torch.cuda._sleep(20_000_000)
    kept = [t.clone() for t in old]
    del old
    got = call(s)
    torch.cuda.synchronize()
    for k, g, w in zip(kept, got, want):
        assert bool((k.float() == 3).all())
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
    # and outputs dropped before the call has run are not this stream's to write
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    del got
    call(s)
    new = [torch.full(shape, 5.0, device=DEV).to(dtype) for shape, dtype in sizes]
    torch.cuda.synchronize()
    assert all(bool((t.float() == 5).all()) for t in new)


@pytest.mark.parametrize("rows,width", [(1, 64), (5, 520), (300, 5120), (0, 64)])
def test_norm_over_its_input_returns_the_input_as_h(rows, width):
    from mixed_lora_projection_gb300 import add_rms_norm
    g = gen(rows)
    big, w = randn(g, rows, width + 64), randn(g, width)
    for x in (big[:, 64:], randn(g, rows, width)):
        before = x.clone()
        _, want = norm_ref(before, None, w, 0.0, 1e-6)
        y, h = add_rms_norm(x, w, out=x)
        assert y is x and torch.equal(h, before)
        within(y, want, want.abs() * BF16_TOL)


def give_up(c, stalls, **kw):
    """A call whose load warps stop after some tiles ends with LORA_ETIMEOUT; the handle then works as before."""
    from mixed_lora_projection_gb300 import PagedAttention, _lib as L
    with PagedAttention(c.heads, c.kv_heads, c.dim, c.page, c.off[-1], len(c.q_lens)) as attn:
        want = c.run(attn, **kw)
        attn.set_option(L.OPT_WAIT_LIMIT_US, 20000)
        for stall in stalls:
            attn.set_option(L.OPT_DEBUG_STALL, stall)
            attn.forward(c.q, c.k, c.v, c.off, c.kv, c.table, **kw)
            assert attn.status() == L.LORA_ETIMEOUT
            assert attn.status(reset=True) == L.LORA_ETIMEOUT
            assert attn.status() == L.LORA_OK
            attn.set_option(L.OPT_DEBUG_STALL, 0)
            assert torch.equal(c.run(attn, **kw), want)


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim", [
    ([1], [20000], 8, 8, 128), ([1] * 3, [9000, 0, 12000], 16, 16, 64), ([8] * 2, [7000, 16000], 24, 12, 256),
    ([1] * 70, [40 * i + 1 for i in range(70)], 8, 8, 128)])
def test_decode_gives_up_and_goes_on(q_lens, kv_lens, heads, kv_heads, dim):
    c = Case(q_lens, kv_lens, heads, kv_heads, dim, 64)
    give_up(c, (1, 2, 3, 5))
    give_up(c, (1, 2), window=3000, sinks=70)


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim", [
    ([300, 40, 700], [5000, 3000, 9000], 8, 8, 64), ([100, 90], [9000, 5000], 16, 16, 64),       # two tiles of rows, one
    ([300, 40, 700], [5000, 3000, 9000], 12, 2, 128), ([20, 21], [9000, 5000], 24, 4, 128),
    ([300, 40, 700], [5000, 3000, 9000], 6, 3, 256), ([260, 30, 1], [7000, 3000, 9000], 24, 12, 256)])
def test_prompt_gives_up_and_goes_on(q_lens, kv_lens, heads, kv_heads, dim):
    c = Case(q_lens, kv_lens, heads, kv_heads, dim, 64)
    give_up(c, (1, 2, 3))
    give_up(c, (1, 2), window=3000, sinks=70)                  # values to blank in the first tiles


def test_attention_handle_options():
    from mixed_lora_projection_gb300 import LoraError, PagedAttention, _lib as L
    with PagedAttention(4, 2, 64, 16, 8, 4) as attn:
        for option, value in ((L.OPT_WAIT_LIMIT_US, 999), (L.OPT_WAIT_LIMIT_US, 60000001), (L.OPT_DEBUG_STALL, -1),
                              (L.OPT_DEBUG_STALL, 1 << 31), (L.OPT_TILE_N, 0), (0, 0)):
            with pytest.raises(LoraError):
                attn.set_option(option, value)
        attn.set_option(L.OPT_WAIT_LIMIT_US, 1000)
        attn.set_option(L.OPT_DEBUG_STALL, 0)


@pytest.mark.parametrize("rows", [1, 3, 70])
def test_append_in_place_beside_keys_and_values(rows):
    """q, k and v of each head side by side in one buffer; the turned queries over themselves."""
    from mixed_lora_projection_gb300 import LoraError, kv_append
    c = Case([rows], [90], 4, 4, 64, 16)
    g = gen(rows)
    y = randn(g, rows, 4, 3, 64)
    q, k, v = y.clone().unbind(2)
    cos, sin = torch.ones(90, 32, device=DEV), torch.zeros(90, 32, device=DEV)
    out = kv_append(y[:, :, 0], y[:, :, 1], y[:, :, 2], c.off, c.kv, c.table, c.k, c.v, cos, sin, q_out=y[:, :, 0])
    pg, sl = c.slots(0, 90)
    assert torch.equal(out, q) and torch.equal(c.k[pg[-rows:], sl[-rows:]], k) and torch.equal(c.v[pg[-rows:], sl[-rows:]], v)
    assert torch.equal(y[:, :, 1], k) and torch.equal(y[:, :, 2], v)
    with pytest.raises(LoraError):                             # keys in the queries' place
        kv_append(y[:, :, 0], y[:, :, 0], y[:, :, 2], c.off, c.kv, c.table, c.k, c.v, cos, sin, q_out=y[:, :, 0])


@pytest.mark.parametrize("q_lens,kv_lens,positions", [([6], [40], 37), ([6, 20], [1000, 15], 1), ([1, 300], [600, 290], 200)])
def test_positions_past_the_rotary_tables_use_the_row_at_that_end(q_lens, kv_lens, positions):
    from mixed_lora_projection_gb300 import kv_append
    c = Case(q_lens, kv_lens, 2, 1, 64, 16)
    g = gen(positions)
    y = randn(g, c.off[-1], 4, 64)
    cos, sin = torch.rand(positions, 16, generator=g, device=DEV), torch.rand(positions, 16, generator=g, device=DEV)
    out = kv_append(y[:, :2], y[:, 2:3], y[:, 3:], c.off, c.kv, c.table, c.k, c.v, cos, sin)
    for i, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        pos = torch.arange(nk - nq, nk, device=DEV)
        at = pos.clamp(0, positions - 1)
        cs, sn = cos[at].to(F64)[:, None], sin[at].to(F64)[:, None]
        a, b = y[c.off[i]:c.off[i + 1], :3, :16].to(F64), y[c.off[i]:c.off[i + 1], :3, 16:32].to(F64)
        ref = torch.cat([a * cs - b * sn, b * cs + a * sn], -1)
        most = ref.abs() * U + torch.cat([a.abs() + b.abs()] * 2, -1) * 2.0 ** -22
        within(out[c.off[i]:c.off[i + 1], :, :32], ref[:, :2], most[:, :2])
        real = pos >= 0
        pg, sl = c.table[i].long()[pos[real] // 16], pos[real] % 16
        within(c.k[pg, sl][:, :, :32], ref[real][:, 2:], most[real][:, 2:])


# more sequences than the small parameter lists hold; near 1,024 the decode ring of heads of 256 has two slots
MANY = [65, 300, 1024]
SHAPES = [(4, 4, 64), (6, 1, 128), (4, 2, 256)]


@pytest.mark.parametrize("n", MANY)
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
def test_decode_of_many_sequences(n, heads, kv_heads, dim):
    c = Case([i % 3 for i in range(n)], [2 + (i * 37) % 200 for i in range(n)], heads, kv_heads, dim, 32, seed=n)
    c.poison()
    c.check()
    c.check(50, 2)


@pytest.mark.parametrize("n", MANY)
@pytest.mark.parametrize("most", [20, 150])                    # one tile of rows, two
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
def test_prompts_of_many_sequences(n, most, heads, kv_heads, dim):
    q = [17 + i % (most - 16) if i % 5 else 0 for i in range(n)]
    c = Case(q, [a + (i * 13) % 40 for i, a in enumerate(q)], heads, kv_heads, dim, 32, seed=n + most)
    c.poison()
    c.check()
    c.check(30, 2)


@pytest.mark.parametrize("n", MANY)
def test_decode_rows_beside_prompts_of_many_sequences(n):
    q = [(1, 0, 40, 3)[i % 4] for i in range(n)]
    c = Case(q, [a + (i * 29) % 300 for i, a in enumerate(q)], 6, 2, 128, 16, seed=n)
    c.poison()
    c.check()


@pytest.mark.parametrize("n", MANY)
def test_append_of_many_sequences(n):
    from mixed_lora_projection_gb300 import kv_append
    q = [i % 4 for i in range(n)]
    c = Case(q, [a + i % 30 for i, a in enumerate(q)], 2, 2, 64, 16, seed=n)
    new = randn(gen(n), c.off[-1], 2, 64)
    want = c.k.clone()
    kv_append(None, new, new, c.off, c.kv, c.table, c.k, c.v)
    for i, rows in enumerate(q):
        if rows:
            pg, sl = c.slots(i, c.kv_list[i])
            want[pg[-rows:], sl[-rows:]] = new[c.off[i]:c.off[i + 1]]
    assert torch.equal(c.k, want)


@pytest.mark.parametrize("q", [1, 40])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 2)])
def test_cache_of_one_page(q, heads, kv_heads):
    c = Case([q], [60], heads, kv_heads, 128, 64, seed=q, spare=0)
    assert c.k.shape[0] == 1
    c.check()
    c.check(20, 3)


@pytest.mark.parametrize("q", [1, 100])
@pytest.mark.parametrize("token_pad,page_pad", [(8, 0), (8, 24), (0, 8), (40, 64)])
def test_cache_with_gaps_between_tokens_and_pages(q, token_pad, page_pad):
    c = Case([q, q], [300, 129], 4, 2, 64, 16, seed=token_pad)
    n, page, kv_heads, dim = c.k.shape
    token = kv_heads * dim + token_pad
    per = page * token + page_pad
    for name in ("k", "v"):
        t = torch.zeros(n * per, dtype=c.k.dtype, device=DEV).as_strided((n, page, kv_heads, dim), (per, token, dim, 1))
        setattr(c, name, t.copy_(getattr(c, name)))
    c.check()


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim,times", [
    ([8, 8], [7000, 16000], 24, 12, 256, 2000), ([1], [20000], 8, 8, 128, 1000), ([1, 1], [9000, 12000], 16, 16, 64, 1000),
    ([300, 40], [5000, 9001], 6, 3, 256, 400), ([300, 40], [5000, 9001], 12, 2, 128, 400), ([300, 40], [5000, 9001], 8, 8, 64, 400),
    ([20, 21], [9001, 5000], 24, 4, 128, 400)])
def test_blanked_values_give_the_same_bits_every_time(q_lens, kv_lens, heads, kv_heads, dim, times):
    """Values that no row sees are blanked in the ring while it is refilled: a late write would show now and then."""
    from mixed_lora_projection_gb300 import PagedAttention
    window, sinks = 3000, 70
    c = Case(q_lens, kv_lens, heads, kv_heads, dim, 64, seed=dim)
    ref, w = c.ref(window, sinks)
    for i, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        pg, sl = (x[sinks:nk - nq - window + 1] for x in c.slots(i, nk))
        c.v[pg, sl] = float("nan")
    c.poison()
    with PagedAttention(heads, kv_heads, dim, 64, c.off[-1], len(q_lens)) as attn:
        first = c.run(attn, window=window, sinks=sinks)
        within(first, ref, bound(ref, w))
        other = torch.zeros((), dtype=torch.int64, device=DEV)
        for _ in range(times):
            o = attn.forward(c.q, c.k, c.v, c.off, c.kv, c.table, window=window, sinks=sinks)
            other += (o.view(torch.int16) != first.view(torch.int16)).any()
        assert attn.status() == 0 and other.item() == 0


def test_tensors_written_in_place_count_as_modified():
    from mixed_lora_projection_gb300 import PagedAttention, add_rms_norm, add_rms_norm_fp8, kv_append
    c = Case([2, 20], [20, 30], 4, 2, 64, 16)
    g = gen(8)
    x, w, new = randn(g, 4, 64), randn(g, 64), randn(g, 22, 2, 64)
    y, h = torch.empty_like(x), torch.empty_like(x)
    q8, s, o = torch.empty(4, 64, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(4, 2, device=DEV), torch.empty_like(c.q)

    def grew(tensors, call):
        before = [t._version for t in tensors]
        call()
        assert all(t._version > b for t, b in zip(tensors, before))

    grew([y, h], lambda: add_rms_norm(x, w, x, out=y, h_out=h))
    grew([q8, s, h], lambda: add_rms_norm_fp8(x, w, group=32, out=q8, scales=s, h_out=h))
    grew([c.k, c.v, o], lambda: kv_append(c.q, new, new, c.off, c.kv, c.table, c.k, c.v, q_out=o))
    with PagedAttention(4, 2, 64, 16, 22, 2) as attn:
        grew([o], lambda: attn.forward(c.q, c.k, c.v, c.off, c.kv, c.table, out=o))
    read = [t._version for t in (x, w, c.q, new, c.kv, c.table)]
    add_rms_norm(x, w, x)
    kv_append(c.q, new, new, c.off, c.kv, c.table, c.k, c.v)
    assert read == [t._version for t in (x, w, c.q, new, c.kv, c.table)]
    # a value that a gradient needs is not overwritten unnoticed
    a = torch.ones(4, 64, dtype=x.dtype, device=DEV, requires_grad=True) * 2
    loss = (a * a).sum()
    add_rms_norm(x, w, out=a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        add_rms_norm(x, w, out=torch.empty_like(x))


def test_projection_launched_early_reads_weights_written_before_the_norm():
    """W's writer, the norm, then a projection that may request W before it waits for the norm."""
    from mixed_lora_projection_gb300 import LoraLinear, _lib as L, add_rms_norm
    g = gen(3)
    x, w, weights = randn(g, 48, 1024), randn(g, 1024), randn(g, 4, 2048, 1024)
    a, b = randn(g, 16, 1024), randn(g, 2048, 16)
    W = torch.empty(2048, 1024, dtype=x.dtype, device=DEV)
    with LoraLinear(1024, 2048, 16, 48) as ll:
        ll.set_option(L.OPT_PDL, 1)

        def step(i):
            W.copy_(weights[i])
            y, _ = add_rms_norm(x, w)
            return ll.forward(y, [0, 48], [0], W, [a], [b], [1.0])

        want = []
        for i in range(4):
            want.append(step(i))
            torch.cuda.synchronize()
        for _ in range(50):
            got = [step(i) for i in range(4)]
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("n,heads,kv_heads,dim,page,window", [
    (70, 12, 12, 256, 128, 700), (2, 24, 12, 256, 64, 0), (70, 16, 4, 128, 48, 0), (20, 8, 8, 64, 16, 300)])
def test_decode_gives_the_same_bits_beside_other_work(n, heads, kv_heads, dim, page, window):
    """A slot of the ring is refilled only when its last reads are done, whatever keeps the block waiting."""
    from mixed_lora_projection_gb300 import PagedAttention
    c = Case([1 + i % 2 for i in range(n)], [2 + (i * 397) % (14000 // n + 300) for i in range(n)], heads, kv_heads, dim, page, seed=n)
    c.poison()
    first = c.check(window, 4)
    side, a = torch.cuda.Stream(), torch.randn(2048, 2048, device=DEV).to(torch.bfloat16)
    other = torch.zeros((), dtype=torch.int64, device=DEV)
    with PagedAttention(heads, kv_heads, dim, page, c.off[-1], n) as attn:
        for i in range(4000):
            if i % 40 == 0:
                with torch.cuda.stream(side):
                    for _ in range(40):
                        a @ a
            o = attn.forward(c.q, c.k, c.v, c.off, c.kv, c.table, window=window, sinks=4)
            other += (o.view(torch.int16) != first.view(torch.int16)).any()
        assert attn.status() == 0 and other.item() == 0
