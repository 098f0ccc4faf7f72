"""The host side of the 8-bit projection and of the operators around it (include/lora_linear.h, include/lora_layer.h):
argument checks on raw pointers, without a GPU, the bindings' refusals, and the order in which kernels let the next begin."""
import ctypes as C
import os
import re

import pytest
import torch

EINVAL = -1
P = 1 << 22          # addresses that no check dereferences
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_lora_projection_gb300", "csrc")


def project(lib, **kw):
    a = dict(d_in=256, d_out=136, rank=16, most=64, segs=4, x8=P, xs=2 * P, x=3 * P, T=10, off=[0, 4, 10], ids=[0, 1], w8=4 * P, ws=5 * P,
             A=[6 * P], B=[7 * P], s=[1.0], y=8 * P)
    a.update(kw)
    off, ids = (C.c_int32 * len(a["off"]))(*a["off"]), (C.c_int32 * len(a["ids"]))(*a["ids"])
    n = len(a["A"])
    A, B = (C.c_void_p * max(n, 1))(*a["A"]), (C.c_void_p * max(n, 1))(*a["B"])
    s = (C.c_float * max(n, 1))(*a["s"])
    return lib.lora_linear_validate_fp8(a["d_in"], a["d_out"], a["rank"], a["most"], a["segs"], a["x8"], a["xs"], a["x"], a["T"], off, ids,
                                        len(a["ids"]), a["w8"], a["ws"], A, B, s, n, a["y"])


def test_projection_accepts(lib):
    assert project(lib) == 0
    assert project(lib, x=None, ids=[0, 0]) == 0
    assert project(lib, x=None, off=[0, 10, 10]) == 0           # a segment without rows names an adapter in vain
    assert project(lib, T=0, off=[0, 0, 0], x8=None, xs=None, w8=None, ws=None, y=None) == 0
    assert project(lib, xs=2 * P + 4, ws=5 * P + 8) == 0


@pytest.mark.parametrize("bad", [
    dict(d_in=264), dict(d_in=8), dict(d_out=132), dict(rank=12), dict(T=65), dict(x8=None), dict(x8=P + 8), dict(xs=None), dict(xs=2 * P + 2),
    dict(x=None), dict(x=3 * P + 8), dict(w8=None), dict(w8=4 * P + 1), dict(ws=None), dict(ws=5 * P + 1), dict(y=None), dict(y=8 * P + 8),
    dict(y=P), dict(y=2 * P), dict(y=3 * P), dict(y=4 * P + 256), dict(y=5 * P), dict(y=6 * P), dict(y=7 * P),
    dict(A=[None]), dict(B=[7 * P + 2]), dict(s=[float("nan")]), dict(ids=[0, 2]), dict(ids=[0, -1]), dict(off=[0, 4, 9]), dict(off=[1, 4, 10]),
])
def test_projection_refuses(lib, bad):
    assert project(lib, **bad) == EINVAL


def test_projection_without_a_handle(lib):
    off, ids = (C.c_int32 * 2)(0, 1), (C.c_int32 * 1)(0)
    assert lib.lora_linear_forward_fp8(None, P, 2 * P, None, 1, off, ids, 1, 4 * P, 5 * P, None, None, None, 0, 8 * P, None) == EINVAL


def gate(lib, x=P, xs=512, rows=4, width=256, y=2 * P, ys=256, q=None, qs=0, s=None, group=0):
    return lib.lora_linear_silu_mul(x, xs, rows, width, y, ys, q, qs, s, group, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(width=0), dict(width=12), dict(width=32776), dict(x=None), dict(x=P + 8), dict(xs=504), dict(xs=516), dict(y=None),
    dict(ys=248), dict(ys=260), dict(y=2 * P + 2), dict(y=P), dict(y=P + 512), dict(q=3 * P), dict(q=3 * P, qs=256), dict(q=3 * P, qs=248, s=4 * P),
    dict(q=3 * P, qs=256, s=4 * P, group=16), dict(q=3 * P, qs=256, s=4 * P + 2), dict(q=2 * P, qs=256, s=4 * P), dict(q=3 * P, qs=256, s=3 * P),
    dict(y=None, q=P + 1024, qs=256, s=4 * P),
])
def test_gate_refuses(lib, bad):
    assert gate(lib, **bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(q=None), dict(x=None), dict(xs=248), dict(width=4), dict(rows=-2), dict(group=512), dict(s=None), dict(q=P)])
def test_rows_refuse(lib, bad):
    a = dict(dict(x=P, xs=256, rows=4, width=256, q=2 * P, qs=256, s=3 * P, group=128), **bad)
    assert lib.lora_linear_fp8_rows(a["x"], a["xs"], a["rows"], a["width"], a["q"], a["qs"], a["s"], a["group"], None) == EINVAL


@pytest.mark.parametrize("bad", [dict(w=None), dict(w=P + 8), dict(ws=248), dict(ws=260), dict(rows=-1), dict(cols=0), dict(cols=12), dict(q=None),
                                 dict(qs=128), dict(s=None), dict(s=3 * P + 1), dict(q=P), dict(s=2 * P), dict(rows=(1 << 20) + 1), dict(s=P + 512)])
def test_blocks_refuse(lib, bad):
    a = dict(dict(w=P, ws=256, rows=4, cols=256, q=2 * P, qs=256, s=3 * P), **bad)
    assert lib.lora_linear_fp8_blocks(a["w"], a["ws"], a["rows"], a["cols"], a["q"], a["qs"], a["s"], None) == EINVAL


def score(lib, **kw):
    a = dict(x=P, stride=1000, fp32=0, rows=4, vocab=1000, t=2 * P, t64=1, temp=1.0, top=3, lp=3 * P, rk=4 * P, en=5 * P, tl=6 * P, tt=7 * P)
    a.update(kw)
    return lib.lora_linear_token_logprobs(a["x"], a["stride"], a["fp32"], a["rows"], a["vocab"], a["t"], a["t64"], a["temp"], a["top"], a["lp"],
                                          a["rk"], a["en"], a["tl"], a["tt"], None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=(1 << 24) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1, stride=1 << 25), dict(stride=999), dict(x=None), dict(x=P + 1),
    dict(x=P + 2, fp32=1), dict(fp32=2), dict(t=None), dict(t=2 * P + 4), dict(t64=0, t=2 * P + 2), dict(temp=0.0), dict(temp=-1.0), dict(temp=float("nan")),
    dict(temp=float("inf")), dict(temp=1e-40), dict(top=-1), dict(top=33), dict(top=5, vocab=4), dict(tl=None), dict(tt=None), dict(lp=3 * P + 2),
    dict(lp=None, rk=None, en=None, top=0), dict(lp=P + 8), dict(rk=2 * P), dict(tt=6 * P + 8), dict(en=3 * P + 4),
])
def test_score_refuses(lib, bad):
    assert score(lib, **bad) == EINVAL


def test_nothing_to_do(lib):
    assert gate(lib, rows=0, x=None, y=None) == 0
    assert lib.lora_linear_fp8_rows(None, 256, 0, 256, None, 256, None, 128, None) == 0
    assert lib.lora_linear_fp8_blocks(None, 256, 0, 256, None, 256, None, None) == 0
    assert score(lib, rows=0, x=None) == 0


def test_binding_refuses(lib):
    from mixed_lora_projection_gb300 import fp8_blocks, fp8_rows, silu_mul, silu_mul_fp8, token_logprobs
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (silu_mul, silu_mul_fp8, fp8_rows, fp8_blocks, token_logprobs):
        with pytest.raises(ValueError, match="CUDA"):
            call(x)
        with pytest.raises(TypeError, match="tensor"):
            call([1.0])
    for call in (silu_mul_fp8, fp8_rows):
        with pytest.raises(ValueError, match="group"):
            call(x, group=-1)


@pytest.mark.parametrize("name", ["act_fp8.cu", "logprobs.cu", "kernels_fp8.cu"])
def test_kernels_wait_before_they_let_the_next_one_begin(name):
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    kernels = re.split(r"__global__", src)[1:]
    assert kernels
    for k in kernels:
        order = re.findall(r"griddep_(wait|launch_dependents)\(\)", k)
        assert order[:2] == ["wait", "launch_dependents"] and order.count("launch_dependents") == 1, name
        # the projection behind its own shrink, which has waited for all before both, waits for it ahead of U and at its end
        assert len(order) == (4 if "late_u" in k else 2), name
        assert k.count("if (!p.late_u) griddep_wait();") == ("late_u" in k), name
