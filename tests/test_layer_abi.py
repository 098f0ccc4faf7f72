"""The host side of the operators between the projections (include/lora_layer.h): argument checks on raw
pointers, without a GPU, and the binding's refusals."""
import ctypes as C

import pytest
import torch

EINVAL = -1
P = 1 << 20          # an aligned address that no check dereferences


@pytest.fixture
def norm(lib):
    good = dict(x=P, xs=128, r=2 * P, rs=128, w=3 * P, off=0.0, eps=1e-6, rows=4, width=128, h=4 * P, hs=128, y=5 * P, ys=128,
                q=None, qs=0, s=None, group=0)

    def call(**kw):
        a = dict(good, **kw)
        return lib.lora_linear_add_rms_norm(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["off"], a["eps"], a["rows"], a["width"],
                                            a["h"], a["hs"], a["y"], a["ys"], a["q"], a["qs"], a["s"], a["group"], None)
    return call


@pytest.mark.parametrize("bad", [
    dict(width=0), dict(width=4), dict(width=12), dict(width=32776), dict(rows=-1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(off=float("inf")), dict(x=None), dict(w=None), dict(x=P + 2), dict(w=3 * P + 8), dict(y=None), dict(xs=120), dict(xs=132),
    dict(rs=64), dict(hs=129), dict(y=P + 256), dict(h=3 * P), dict(y=4 * P), dict(r=5 * P),
    dict(q=6 * P, qs=128), dict(q=6 * P, qs=64, s=7 * P), dict(q=6 * P, qs=128, s=7 * P, group=48),
    dict(q=6 * P, qs=128, s=7 * P + 2), dict(q=5 * P, qs=128, s=7 * P), dict(q=6 * P, qs=128, s=6 * P + 256),
])
def test_norm_refuses(norm, bad):
    assert norm(**bad) == EINVAL


def test_norm_of_no_rows_is_nothing(norm):
    assert norm(rows=0, x=None, y=None) == 0


class Cache:
    """A lora_kv_cache that passes every check: 8 pages of 16 tokens, 2 heads of 64, 3 sequences."""

    def __init__(self, **kw):
        from mixed_lora_projection_gb300 import _lib
        self.off = (C.c_int32 * 4)(*kw.pop("off", [0, 1, 1, 5]))
        f = dict(k=P, v=2 * P, k_page_stride=2048, k_token_stride=128, k_head_stride=64, v_page_stride=2048,
                 v_token_stride=128, v_head_stride=64, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64,
                 block_table=3 * P, table_stride=4, pages_per_seq=4, n_seqs=3, kv_lens=4 * P)
        f.update(kw)
        self.c = _lib.KvCache(**f)
        self.c.q_offsets = C.cast(self.off, C.POINTER(C.c_int32)) if not kw.get("no_off") else None


BAD_CACHE = [dict(k=None), dict(v=2 * P + 8), dict(k_page_stride=2050), dict(v_token_stride=0), dict(k_head_stride=-64),
             dict(n_pages=0), dict(page_size=8), dict(page_size=24), dict(n_kv_heads=0), dict(head_dim=60), dict(block_table=None),
             dict(block_table=3 * P + 2), dict(table_stride=3), dict(pages_per_seq=0), dict(pages_per_seq=1 << 24, table_stride=1 << 24),
             dict(n_seqs=0), dict(n_seqs=1025), dict(kv_lens=None), dict(off=[1, 1, 1, 5]), dict(off=[0, 3, 2, 5]),
             dict(off=[0, 1, 1, (1 << 24) + 1])]


def attend(lib, cache=None, heads=4, kv=2, dim=64, page=16, tokens=8, seqs=4, q=5 * P, qs=256, qh=64, o=6 * P, os=256, oh=64, scale=0.125,
           window=0, sinks=0):
    c = cache or Cache()
    return lib.lora_linear_attn_validate(heads, kv, dim, page, tokens, seqs, C.byref(c.c), q, qs, qh, o, os, oh, scale, window, sinks)


@pytest.mark.parametrize("bad", BAD_CACHE)
def test_attention_refuses_caches(lib, bad):
    assert attend(lib) == 0
    assert attend(lib, Cache(**bad)) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(heads=3), dict(heads=0), dict(kv=0), dict(heads=258, kv=2), dict(dim=96), dict(dim=512), dict(page=32), dict(page=12), dict(tokens=4),
    dict(tokens=0), dict(seqs=2), dict(seqs=2000), dict(q=None), dict(o=None), dict(q=5 * P + 8), dict(qs=250), dict(qh=32),
    dict(oh=65), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
    dict(sinks=-1), dict(o=5 * P + 512), dict(o=P + 1024), dict(o=2 * P),
])
def test_attention_refuses(lib, bad):
    assert attend(lib, **bad) == EINVAL


def test_attention_of_no_rows_is_nothing(lib):
    assert attend(lib, Cache(off=[0, 0, 0, 0]), q=None, o=None) == 0


def append(lib, cache=None, q=5 * P, qs=512, qh=64, qo=6 * P, qos=256, qoh=64, heads=4, k=7 * P, ks=512, kh=64, v=8 * P, vs=512, vh=64,
           cos=9 * P, sin=10 * P, rot=32, npos=64):
    c = cache or Cache(off=[0, 0, 0, 0])
    return lib.lora_linear_kv_append(C.byref(c.c), q, qs, qh, qo, qos, qoh, heads, k, ks, kh, v, vs, vh, cos, sin, rot, npos, None)


@pytest.mark.parametrize("bad", BAD_CACHE[:-3])
def test_append_refuses_caches(lib, bad):
    assert append(lib) == 0                                 # no rows: checked, nothing launched
    assert append(lib, Cache(**bad)) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(rot=8), dict(rot=80), dict(rot=-16), dict(cos=None), dict(sin=10 * P + 4), dict(npos=0), dict(heads=-1), dict(q=None), dict(qo=None),
    dict(heads=0), dict(k=None), dict(v=8 * P + 4), dict(qs=60), dict(qoh=63), dict(ks=32), dict(vh=-64), dict(k=P), dict(q=2 * P),
    dict(qo=P + 64), dict(qo=7 * P),
])
def test_append_refuses(lib, bad):
    assert append(lib, Cache(), **bad) == EINVAL


def test_handle_refusals(lib):
    h = C.c_void_p(1)
    assert lib.lora_linear_attn_create(C.byref(h), 4, 3, 64, 16, 8, 4, 0) == EINVAL and not h.value
    assert lib.lora_linear_attn_create(None, 4, 2, 64, 16, 8, 4, 0) == EINVAL
    assert lib.lora_linear_attn_forward(None, None, None, 0, 0, None, 0, 0, 1.0, 0, 0, None) == EINVAL
    assert lib.lora_linear_attn_status(None, 0) == EINVAL
    assert lib.lora_linear_attn_destroy(None) == 0
    if not torch.cuda.is_available():
        assert lib.lora_linear_attn_create(C.byref(h), 4, 2, 64, 16, 8, 4, 0) == -6       # no device


def test_binding_refuses_host_tensors(lib):
    from mixed_lora_projection_gb300 import add_rms_norm, add_rms_norm_fp8, kv_append
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        add_rms_norm(x, x[0])
    with pytest.raises(ValueError):
        add_rms_norm_fp8(x, x[0], group=100)
    with pytest.raises(ValueError):
        kv_append(None, x.view(4, 2, 64), x.view(4, 2, 64), [0, 4], None, None, None, None)


def test_layer_signatures_match_the_header():
    import os
    import re
    from mixed_lora_projection_gb300 import _lib
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "lora_layer.h")).read(), flags=re.S)
    body = re.search(r"typedef struct lora_kv_cache \{(.*?)\}", src, flags=re.S).group(1)
    names = [n.strip(" *\n") for line in body.split(";") if line.strip()
             for n in line.replace("const int32_t", "").replace("long long", "").replace("int ", "").replace("void", "").split(",")]
    assert names == [f[0] for f in _lib.KvCache._fields_]
    for m in re.finditer(r"int (lora_linear_\w+)\((.*?)\);", src, flags=re.S):
        assert len(_lib.SIGNATURES[m.group(1)][1]) == len(m.group(2).split(",")), m.group(1)


def test_binding_refuses_what_is_no_tensor(lib):
    from mixed_lora_projection_gb300 import add_rms_norm, add_rms_norm_fp8, kv_append
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        add_rms_norm([[1.0]], x[0])
    with pytest.raises(ValueError):
        add_rms_norm_fp8(x, x[0], group=-1)
    with pytest.raises(TypeError):
        kv_append(None, None, None, [0, 4], None, None, None, None)


def test_handle_options_refuse_a_missing_handle(lib):
    for option, value in ((2, 20000), (3, 1), (99, 0)):
        assert lib.lora_linear_attn_set_option(None, option, value) == EINVAL


ECUDA = -3


def accepts(lib, **kw):
    """Whether an append passes the checks (on a machine without a GPU its launch fails; with one, these made-up
    addresses must not be launched)."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    rc = append(lib, Cache(), **kw)
    assert rc in (EINVAL, ECUDA)
    return rc == ECUDA


# queries over themselves, in rows of 4 + 2 + 2 heads of 64: q, k, v are slices, or share places they must not share
FUSED = dict(q=5 * P, qs=512, qh=64, qo=5 * P, qos=512, qoh=64, k=5 * P + 512, ks=512, kh=64, v=5 * P + 768, vs=512, vh=64)


@pytest.mark.parametrize("bad", [
    dict(k=5 * P), dict(v=5 * P), dict(k=5 * P + 384), dict(v=5 * P + 128), dict(k=5 * P + 1024), dict(v=5 * P + 512 - 128, vh=128),
    dict(k=5 * P + 4 * 1024 + 256), dict(k=5 * P, ks=256)])
def test_append_in_place_refuses_keys_and_values_in_the_queries(lib, bad):
    assert append(lib, Cache(), **{**FUSED, **bad}) == EINVAL


def test_append_in_place_takes_slices(lib):
    assert accepts(lib, **FUSED)
    # q, k and v of each head side by side: [rows, 2, 3, 64]
    row = dict(heads=2, q=5 * P, qo=5 * P, k=5 * P + 128, v=5 * P + 256, **{n: 384 for n in ("qs", "qos", "ks", "vs")},
               **{n: 192 for n in ("qh", "qoh", "kh", "vh")})
    assert accepts(lib, **row)
    assert not accepts(lib, **{**row, "k": 5 * P + 112})
    assert not accepts(lib, **{**row, "v": 5 * P + 336})
    # heads outermost, one after another
    assert accepts(lib, **{**FUSED, **{n: 64 for n in ("qs", "qos", "ks", "vs")}, **{n: 320 for n in ("qh", "qoh", "kh", "vh")},
                           "k": 5 * P + 4 * 640, "v": 5 * P + 6 * 640})


def test_append_of_one_row_goes_by_its_heads(lib):
    """A single row has no stride: q, k and v of each head side by side, whatever row strides are given."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    one = dict(heads=2, q=5 * P, qo=5 * P, k=5 * P + 128, v=5 * P + 256, qs=64, qos=64, ks=64, vs=64, qh=192, qoh=192, kh=192, vh=192)
    assert append(lib, Cache(off=[0, 0, 0, 1]), **one) == ECUDA
    assert append(lib, Cache(off=[0, 0, 0, 1]), **{**one, "k": 5 * P}) == EINVAL


def test_binding_refuses_an_output_for_no_queries(lib):
    from mixed_lora_projection_gb300 import kv_append
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q_out"):
        kv_append(None, x, x, [0, 4], None, None, None, None, q_out=x)
