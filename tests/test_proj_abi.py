"""C ABI of the operators around the halves of the layer without a GPU: the library exports what
include/moe_proj.h declares and refuses bad arguments before anything is enqueued (so fake device addresses are
safe)."""
import ctypes
import math
import os
import re

import pytest

from routed_expert_mlp_amd import capi
from routed_expert_mlp_amd import projection as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000
BIG = 1 << 40


def norm(x=FAKE, stride=256, res=FAKE, w=FAKE, eps=1e-6, T=4, H=256, h=FAKE + BIG, y=FAKE + 2 * BIG, q=FAKE, s=FAKE):
    return P._lib().moe_proj_norm(x, stride, res, w, eps, T, H, h, y, q, s, None)


def fp8(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, T=4, N=64, K=256, y=FAKE):
    return P._lib().moe_proj_fp8(x, xs, w, ws, T, N, K, y, None)


def adapters(**kw):
    base = dict(a=FAKE, b=FAKE, ranks=FAKE, scales=FAKE, n_adapters=3, max_rank=16, in_features=64, out_features=48)
    base.update(kw)
    return P.moe_proj_adapters(**base)


def size(d, T=4):
    n = ctypes.c_size_t(0)
    st = P._lib().moe_proj_lora_workspace_size(ctypes.byref(d) if d is not None else None, T, ctypes.byref(n))
    return st, n.value


def lora(d, x=FAKE, xs=64, T=4, ids=FAKE, base=FAKE, bs=48, out=FAKE + BIG, os=48, ws=FAKE, wsb=BIG):
    return P._lib().moe_proj_lora(ctypes.byref(d) if d is not None else None, x, xs, T, ids, base, bs, out, os, ws,
                                  wsb, None)


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "moe_proj.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(moe_\w+)\s*\(", text, flags=re.M))
    assert names == set(P.EXPORTED)
    for n in names:
        assert getattr(P._lib(), n) is not None
    for name, value in (("NORM_MAX_HIDDEN", P.NORM_MAX_HIDDEN), ("LORA_MAX_RANK", P.LORA_MAX_RANK)):
        assert re.search(rf"#define MOE_PROJ_{name}\s+{value}\b", text)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), capi.ERR_BAD_SHAPE), (dict(T=1 << 22), capi.ERR_BAD_SHAPE), (dict(H=0), capi.ERR_BAD_SHAPE),
    (dict(H=4), capi.ERR_BAD_SHAPE), (dict(H=252), capi.ERR_BAD_SHAPE), (dict(H=-8), capi.ERR_BAD_SHAPE),
    (dict(H=16392, stride=16392), capi.ERR_BAD_SHAPE), (dict(stride=248), capi.ERR_BAD_SHAPE),
    (dict(stride=260), capi.ERR_BAD_SHAPE), (dict(stride=1 << 31), capi.ERR_BAD_SHAPE),
    (dict(eps=-1e-9), capi.ERR_BAD_VALUE), (dict(eps=math.nan), capi.ERR_BAD_VALUE),
    (dict(eps=math.inf), capi.ERR_BAD_VALUE), (dict(x=None), capi.ERR_NULL_ARG),
    (dict(y=None, q=None, s=None), capi.ERR_NULL_ARG), (dict(q=None), capi.ERR_NULL_ARG),
    (dict(s=None), capi.ERR_NULL_ARG), (dict(x=FAKE + 8), capi.ERR_MISALIGNED),
    (dict(res=FAKE + 2), capi.ERR_MISALIGNED), (dict(w=FAKE + 4), capi.ERR_MISALIGNED),
    (dict(h=FAKE + 8), capi.ERR_MISALIGNED), (dict(y=FAKE + 2), capi.ERR_MISALIGNED),
    (dict(q=FAKE + 1), capi.ERR_MISALIGNED), (dict(s=FAKE + 4), capi.ERR_MISALIGNED),
    (dict(h=FAKE, stride=264), capi.ERR_BAD_VALUE), (dict(y=FAKE, stride=264), capi.ERR_BAD_VALUE),
    (dict(h=FAKE + BIG, y=FAKE + BIG), capi.ERR_BAD_VALUE),
    (dict(T=0), 0), (dict(T=0, x=None), 0),
])
def test_norm_refusals(kw, code):
    assert norm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), capi.ERR_BAD_SHAPE), (dict(T=1 << 22), capi.ERR_BAD_SHAPE), (dict(N=0), capi.ERR_BAD_SHAPE),
    (dict(N=8), capi.ERR_BAD_SHAPE), (dict(N=72), capi.ERR_BAD_SHAPE), (dict(N=1 << 20), capi.ERR_BAD_SHAPE),
    (dict(K=0), capi.ERR_BAD_SHAPE), (dict(K=64), capi.ERR_BAD_SHAPE), (dict(K=1 << 20), capi.ERR_BAD_SHAPE),
    (dict(T=1 << 20, N=1 << 12), capi.ERR_BAD_SHAPE), (dict(N=-16), capi.ERR_BAD_SHAPE), (dict(K=-128), capi.ERR_BAD_SHAPE),
    (dict(x=None), capi.ERR_NULL_ARG), (dict(xs=None), capi.ERR_NULL_ARG), (dict(w=None), capi.ERR_NULL_ARG),
    (dict(ws=None), capi.ERR_NULL_ARG), (dict(y=None), capi.ERR_NULL_ARG), (dict(x=FAKE + 8), capi.ERR_MISALIGNED),
    (dict(xs=FAKE + 4), capi.ERR_MISALIGNED), (dict(w=FAKE + 1), capi.ERR_MISALIGNED),
    (dict(ws=FAKE + 8), capi.ERR_MISALIGNED), (dict(y=FAKE + 2), capi.ERR_MISALIGNED), (dict(T=0), 0),
])
def test_fp8_refusals(kw, code):
    assert fp8(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_adapters=0), capi.ERR_BAD_SHAPE), (dict(n_adapters=-1), capi.ERR_BAD_SHAPE),
    (dict(n_adapters=(1 << 20) + 1), capi.ERR_BAD_SHAPE), (dict(max_rank=0), capi.ERR_BAD_SHAPE),
    (dict(max_rank=12), capi.ERR_BAD_SHAPE), (dict(max_rank=264), capi.ERR_BAD_SHAPE),
    (dict(max_rank=-8), capi.ERR_BAD_SHAPE), (dict(in_features=60), capi.ERR_BAD_SHAPE),
    (dict(in_features=0), capi.ERR_BAD_SHAPE), (dict(out_features=44), capi.ERR_BAD_SHAPE),
    (dict(out_features=1 << 20), capi.ERR_BAD_SHAPE),
])
def test_adapter_refusals(kw, code):
    assert lora(adapters(**kw)) == code
    assert size(adapters(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), capi.ERR_BAD_SHAPE), (dict(T=1 << 22), capi.ERR_BAD_SHAPE), (dict(xs=56), capi.ERR_BAD_SHAPE),
    (dict(xs=68), capi.ERR_BAD_SHAPE), (dict(bs=40), capi.ERR_BAD_SHAPE), (dict(os=52), capi.ERR_BAD_SHAPE),
    (dict(os=1 << 31), capi.ERR_BAD_SHAPE), (dict(x=None), capi.ERR_NULL_ARG), (dict(ids=None), capi.ERR_NULL_ARG),
    (dict(base=None), capi.ERR_NULL_ARG), (dict(out=None), capi.ERR_NULL_ARG), (dict(ws=None), capi.ERR_NULL_ARG),
    (dict(x=FAKE + 8), capi.ERR_MISALIGNED), (dict(ids=FAKE + 2), capi.ERR_MISALIGNED),
    (dict(base=FAKE + 8), capi.ERR_MISALIGNED), (dict(out=FAKE + 2), capi.ERR_MISALIGNED),
    (dict(ws=FAKE + 4), capi.ERR_MISALIGNED), (dict(wsb=0), capi.ERR_WORKSPACE_TOO_SMALL),
    (dict(out=FAKE, os=64), capi.ERR_BAD_VALUE), (dict(T=0), 0), (dict(T=0, x=None), 0),
])
def test_lora_refusals(kw, code):
    assert lora(adapters(), **kw) == code


def test_lora_null_descriptor_and_weights():
    assert lora(None) == capi.ERR_NULL_ARG and size(None)[0] == capi.ERR_NULL_ARG
    assert lora(adapters(a=None)) == capi.ERR_NULL_ARG
    assert lora(adapters(b=None)) == capi.ERR_NULL_ARG
    assert lora(adapters(a=FAKE + 8)) == capi.ERR_MISALIGNED
    assert lora(adapters(ranks=FAKE + 2)) == capi.ERR_MISALIGNED
    assert P._lib().moe_proj_lora_workspace_size(ctypes.byref(adapters()), 4, None) == capi.ERR_NULL_ARG


@pytest.mark.parametrize("kw", [{}, dict(in_features=4096, out_features=6144, max_rank=64, n_adapters=32),
                                dict(in_features=8, out_features=8, max_rank=8, n_adapters=1),
                                dict(in_features=(1 << 20) - 8, out_features=8, max_rank=256, n_adapters=1 << 20)])
def test_lora_workspace_serves_fewer_tokens(kw):
    d, last = adapters(**kw), 0
    for T in list(range(0, 200)) + [511, 512, 513, 4096, 32767, 32768, 32769, 40000, 1 << 20, (1 << 22) - 1]:
        st, n = size(d, T)
        assert st == 0 and n >= last, T
        last = n
    st, need = size(d, 64)
    assert lora(d, T=64, wsb=need - 1, xs=max(64, d.in_features), bs=d.out_features, os=d.out_features) == \
        capi.ERR_WORKSPACE_TOO_SMALL
