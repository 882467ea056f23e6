"""C ABI of the attention operators without a GPU: the library exports what
include/moe_attn.h declares and refuses bad arguments before anything is
enqueued (so fake device addresses are safe)."""
import ctypes
import math
import os
import random
import re

import pytest

from routed_expert_mlp_amd import attention as A
from routed_expert_mlp_amd import capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000
BIG = 1 << 40


def cfg(**kw):
    base = dict(n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, rotary_dim=64, rope_style=0, window=0, n_sinks=0,
                norm_eps=1e-6, scale=0.1)
    base.update(kw)
    return A.moe_attn_config(**base)


def cache(**kw):
    base = dict(k=FAKE, v=FAKE + 0x100000, n_pages=8)
    base.update(kw)
    return A.moe_attn_cache(**base)


def size(c, B=2, max_q=1, max_len=64, prefill=0, T=4):
    n = ctypes.c_size_t(0)
    st = A._lib().moe_attn_workspace_size(ctypes.byref(c) if c is not None else None, T, B, max_q, max_len, prefill,
                                          ctypes.byref(n))
    return st, n.value


def decode(c, cc, B=2, n_q=1, max_pages=4, max_len=64, q=FAKE, lens=FAKE, table=FAKE, out=FAKE, ws=FAKE, wsb=BIG):
    return A._lib().moe_attn_decode(ctypes.byref(c) if c is not None else None,
                                    ctypes.byref(cc) if cc is not None else None, q, B, n_q, lens, table, max_pages,
                                    max_len, out, ws, wsb, None)


def prefill(c, cc, T=4, B=2, max_q=4, max_pages=4, max_len=64, q=FAKE, cu=FAKE, lens=FAKE, table=FAKE, out=FAKE,
            ws=FAKE, wsb=BIG):
    return A._lib().moe_attn_prefill(ctypes.byref(c) if c is not None else None,
                                     ctypes.byref(cc) if cc is not None else None, q, T, cu, B, max_q, lens, table,
                                     max_pages, max_len, out, ws, wsb, None)


def prepare(c, cc, T=2, stride=12 * 128, qkv=FAKE, qw=FAKE, kw=FAKE, cs=FAKE, P=10, pos=FAKE, slots=FAKE, q=FAKE):
    return A._lib().moe_attn_prepare(ctypes.byref(c) if c is not None else None,
                                     ctypes.byref(cc) if cc is not None else None, qkv, stride, T, qw, kw, cs, P, pos,
                                     slots, q, None)


ALL = [decode, prefill, prepare]


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "moe_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(moe_\w+)\s*\(", text, flags=re.M))
    assert names == set(A.EXPORTED)
    for n in names:
        assert getattr(A._lib(), n) is not None


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("kw,code", [
    (dict(n_heads=0), capi.ERR_BAD_SHAPE), (dict(n_heads=7), capi.ERR_BAD_SHAPE),
    (dict(n_heads=2048), capi.ERR_BAD_SHAPE), (dict(n_kv_heads=0), capi.ERR_BAD_SHAPE),
    (dict(n_kv_heads=-2), capi.ERR_BAD_SHAPE), (dict(n_kv_heads=16), capi.ERR_BAD_SHAPE),
    (dict(head_dim=96), capi.ERR_BAD_SHAPE), (dict(head_dim=0), capi.ERR_BAD_SHAPE),
    (dict(page_size=8), capi.ERR_BAD_SHAPE), (dict(page_size=48), capi.ERR_BAD_SHAPE),
    (dict(page_size=512), capi.ERR_BAD_SHAPE), (dict(rotary_dim=-16), capi.ERR_BAD_SHAPE),
    (dict(rotary_dim=8), capi.ERR_BAD_SHAPE), (dict(rotary_dim=144), capi.ERR_BAD_SHAPE),
    (dict(rope_style=2), capi.ERR_BAD_VALUE), (dict(window=-1), capi.ERR_BAD_VALUE),
    (dict(n_sinks=-1), capi.ERR_BAD_VALUE), (dict(norm_eps=-1.0), capi.ERR_BAD_VALUE),
    (dict(norm_eps=math.nan), capi.ERR_BAD_VALUE), (dict(scale=0.0), capi.ERR_BAD_VALUE),
    (dict(scale=-1.0), capi.ERR_BAD_VALUE), (dict(scale=math.inf), capi.ERR_BAD_VALUE),
    (dict(scale=math.nan), capi.ERR_BAD_VALUE),
])
def test_config_validation(call, kw, code):
    assert call(cfg(**kw), cache()) == code
    assert size(cfg(**kw))[0] == code


@pytest.mark.parametrize("call", ALL)
def test_null_and_cache(call):
    assert call(None, cache()) == capi.ERR_NULL_ARG
    assert call(cfg(), None) == capi.ERR_NULL_ARG
    assert call(cfg(), cache(k=None)) == capi.ERR_NULL_ARG
    assert call(cfg(), cache(v=None)) == capi.ERR_NULL_ARG
    assert call(cfg(), cache(n_pages=0)) == capi.ERR_BAD_SHAPE
    assert call(cfg(), cache(n_pages=-1)) == capi.ERR_BAD_SHAPE
    assert call(cfg(), cache(n_pages=1 << 27)) == capi.ERR_BAD_SHAPE
    assert call(cfg(), cache(k=FAKE + 8)) == capi.ERR_MISALIGNED
    assert call(cfg(), cache(v=FAKE + 2)) == capi.ERR_MISALIGNED


@pytest.mark.parametrize("call,names", [(decode, ("q", "lens", "table", "out")),
                                        (prefill, ("q", "cu", "lens", "table", "out")),
                                        (prepare, ("qkv", "cs", "pos", "slots", "q"))])
def test_null_arguments(call, names):
    for n in names:
        assert call(cfg(), cache(), **{n: None}) == capi.ERR_NULL_ARG, n


@pytest.mark.parametrize("call,off", [(decode, dict(q=8, lens=2, table=1, out=4, ws=8)),
                                      (prefill, dict(q=8, cu=2, lens=2, table=3, out=4, ws=4)),
                                      (prepare, dict(qkv=8, qw=4, kw=8, cs=4, pos=2, slots=4, q=2))])
def test_misaligned_arguments(call, off):
    for n, d in off.items():
        assert call(cfg(), cache(), **{n: FAKE + d}) == capi.ERR_MISALIGNED, n


@pytest.mark.parametrize("kw", [dict(B=-1), dict(n_q=0), dict(n_q=9), dict(n_q=-1), dict(max_len=-1),
                                dict(max_len=65), dict(max_pages=-1), dict(max_pages=3), dict(B=1 << 60),
                                dict(B=1 << 62, n_q=8), dict(max_len=1 << 62, max_pages=1 << 62),
                                dict(max_len=1 << 30, max_pages=1 << 30), dict(B=1 << 24)])
def test_decode_sizes(kw):
    assert decode(cfg(), cache(), **kw) == capi.ERR_BAD_SHAPE


@pytest.mark.parametrize("kw", [dict(B=-1), dict(T=-1), dict(max_q=-1), dict(max_len=65), dict(max_pages=3),
                                dict(T=1 << 26), dict(T=1 << 62), dict(max_q=1 << 62), dict(B=1 << 62),
                                dict(B=1 << 20, max_q=1 << 10)])
def test_prefill_sizes(kw):
    assert prefill(cfg(), cache(), **kw) == capi.ERR_BAD_SHAPE


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=1 << 40), dict(stride=12 * 128 - 8), dict(stride=12 * 128 + 4),
                                dict(stride=1 << 40), dict(stride=-12 * 128), dict(P=0), dict(P=-5)])
def test_prepare_sizes(kw):
    assert prepare(cfg(), cache(), **kw) == capi.ERR_BAD_SHAPE


def test_calls_with_more_blocks_than_a_launch_takes():
    c = cfg(n_heads=8, n_kv_heads=8)
    big = dict(max_len=1 << 29, max_pages=1 << 25)
    assert decode(c, cache(), B=1 << 12, **big) == capi.ERR_BAD_SHAPE
    assert size(c, B=1 << 12, max_len=1 << 29, T=1 << 12)[0] == capi.ERR_BAD_SHAPE
    assert size(c, B=1, max_len=1 << 29, T=1)[0] == capi.OK
    # few blocks, and 32 Mi rows to join, four in a block
    assert size(cfg(n_heads=1024, n_kv_heads=1), B=1 << 15, max_len=4096, T=1)[0] == capi.OK
    wide = dict(B=4, max_len=1 << 20, T=(1 << 26) - 1, prefill=1)
    assert size(cfg(n_heads=1024, n_kv_heads=1024), max_q=(1 << 14) - 1, **wide) == (capi.OK, 0)
    assert size(cfg(n_heads=1024, n_kv_heads=1024, head_dim=64), B=(1 << 16) - 1, max_q=1, max_len=1 << 20,
                T=(1 << 26) - 1, prefill=1)[0] == capi.ERR_BAD_SHAPE


def test_nothing_to_do_is_ok():
    assert decode(cfg(), None, B=0, q=None, lens=None, table=None, out=None, ws=None, wsb=0) == capi.OK
    assert prefill(cfg(), None, T=0, q=None, cu=None, out=None, ws=None, wsb=0) == capi.OK
    assert prefill(cfg(), None, B=0, q=None, cu=None, lens=None, table=None, out=None, ws=None, wsb=0) == capi.OK
    assert prefill(cfg(), None, max_q=0, q=None, cu=None, out=None, ws=None, wsb=0) == capi.OK
    assert prepare(cfg(), None, T=0, qkv=None, cs=None, pos=None, slots=None, q=None) == capi.OK


def test_workspace_size_and_refusal():
    for pf, call in ((0, decode), (1, prefill)):
        assert size(cfg(), prefill=pf, max_len=1 << 62)[0] == capi.ERR_BAD_SHAPE
        assert size(cfg(), prefill=pf, T=-1)[0] == capi.ERR_BAD_SHAPE
        assert size(cfg(), prefill=pf, T=1 << 40)[0] == capi.ERR_BAD_SHAPE
        st, need = size(cfg(), B=2, max_q=4, max_len=64, prefill=pf)
        assert st == capi.OK
    # long caches of few rows are split and joined: that needs room
    long = dict(B=1, max_len=131072)
    st, need = size(cfg(), max_q=1, prefill=0, T=1, **long)
    assert st == capi.OK and need > 0
    assert decode(cfg(), cache(), max_pages=8192, wsb=need - 1, **long) == capi.ERR_WORKSPACE_TOO_SMALL
    assert decode(cfg(), cache(), max_pages=8192, ws=None, wsb=0, **long) == capi.ERR_NULL_ARG
    st, need = size(cfg(), max_q=100, prefill=1, T=100, **long)
    assert st == capi.OK and need > 0
    pre = dict(T=100, max_q=100, max_pages=8192, **long)
    assert prefill(cfg(), cache(), wsb=need - 1, **pre) == capi.ERR_WORKSPACE_TOO_SMALL
    assert prefill(cfg(), cache(), ws=None, wsb=0, **pre) == capi.ERR_NULL_ARG
    # short prompts are not, nor are long ones of many heads
    assert size(cfg(), B=1, max_q=512, max_len=512, T=512, prefill=1) == (capi.OK, 0)
    assert size(cfg(n_heads=32, n_kv_heads=8), B=1, max_q=4096, max_len=4096, T=4096, prefill=1) == (capi.OK, 0)
    n = ctypes.c_size_t(0)
    c = cfg()
    assert A._lib().moe_attn_workspace_size(ctypes.byref(c), 1, 1, 1, 16, 0, None) == capi.ERR_NULL_ARG
    assert n.value == 0


def test_ragged_prefill_is_limited_by_its_tokens():
    """Many sequences of which one has a long piece: what counts is the tokens, not sequences times the longest."""
    c = cfg(n_heads=32, n_kv_heads=8)
    assert size(c, B=256, max_q=8192, max_len=16384, prefill=1, T=8447)[0] == capi.OK
    assert size(c, B=64, max_q=32768, max_len=65536, prefill=1, T=32768 + 63)[0] == capi.OK
    assert size(c, B=(1 << 16) - 1, max_q=1 << 20, max_len=1 << 21, prefill=1, T=1 << 20)[0] == capi.OK
    assert size(c, B=1 << 16, max_q=64, max_len=64, prefill=1, T=1 << 16)[0] == capi.ERR_BAD_SHAPE
    # a bound above the tokens counts as the tokens
    assert size(c, B=1, max_q=(1 << 31) - 1, max_len=64, prefill=1, T=64) == (capi.OK, 0)
    for dim in (64, 128, 256):
        wide = cfg(n_heads=64, n_kv_heads=1, head_dim=dim)
        assert size(wide, B=1, max_q=(1 << 24) - 1, max_len=1 << 24, prefill=1, T=(1 << 24) - 1)[0] == capi.OK
        assert size(wide, B=1, max_q=1 << 24, max_len=1 << 24, prefill=1, T=1 << 24)[0] == capi.ERR_BAD_SHAPE
    wide = cfg(n_heads=1024, n_kv_heads=1024, head_dim=256)
    for B in (1, (1 << 16) - 1, (1 << 31) - 1):
        for max_q in (1, 1 << 10, (1 << 31) - 1):
            st = size(wide, B=B, max_q=max_q, max_len=(1 << 30) - 1, prefill=1, T=(1 << 26) - 1)[0]
            assert st == (capi.OK if B * max_q <= 1 << 10 else capi.ERR_BAD_SHAPE)
    assert prefill(c, cache(), B=256, max_q=1 << 20, T=8447, wsb=0, q=None) == capi.ERR_NULL_ARG


@pytest.mark.parametrize("kw", [dict(B=0), dict(max_q=0), dict(T=0)])
def test_nothing_to_do_needs_no_workspace(kw):
    c = cfg(n_heads=32, n_kv_heads=8)
    assert size(c, prefill=1, **{**dict(B=1, max_q=4096, max_len=1 << 20, T=4096), **kw}) == (capi.OK, 0)
    for dim in (64, 128, 256):
        c = cfg(n_heads=1024, n_kv_heads=1024, head_dim=dim)
        most = dict(B=1, max_q=1, max_len=(1 << 30) - 1, T=(1 << 26) - 1)
        assert size(c, prefill=1, **{**most, **kw}) == (capi.OK, 0)
    if "B" in kw:
        assert size(c, prefill=0, B=0, max_q=8, max_len=(1 << 30) - 1, T=0) == (capi.OK, 0)


def bound(c, B, max_q, max_len, prefill, T):
    n = ctypes.c_size_t(0)
    st = A._lib().moe_attn_workspace_bound(ctypes.byref(c) if c is not None else None, T, B, max_q, max_len, prefill,
                                           ctypes.byref(n))
    return st, n.value


GEOMETRIES = [dict(n_heads=h, n_kv_heads=k, head_dim=d, window=w, n_sinks=s)
              for h, k in ((32, 8), (64, 2), (8, 8), (71, 1)) for d in (64, 128, 256) for w, s in ((0, 0), (3000, 70))]


@pytest.mark.parametrize("pf", [0, 1])
@pytest.mark.parametrize("kw", GEOMETRIES, ids=lambda kw: "-".join(str(v) for v in kw.values()))
def test_workspace_bound_covers_every_smaller_call(kw, pf):
    """The bound of some largest sizes is at least the size, and the bound, of smaller ones, and no call within it
    is refused for its workspace."""
    rng, c = random.Random(f"{kw} {pf}"), cfg(**kw)

    def any_up_to(n):
        return rng.choice([n, rng.randint(1, n), max(1, int(math.exp(rng.uniform(0, math.log(n)))))])

    parts = 0
    for _ in range(12):
        B, max_q = any_up_to(200), any_up_to(8192 if pf else 8)
        max_len = any_up_to(200000)
        T = rng.choice([B * max_q, any_up_to(B * max_q), 3 * B * max_q]) if pf else B * max_q
        st, most = bound(c, B, max_q, max_len, pf, T)
        assert st == capi.OK
        for _ in range(300):
            b, q, n = any_up_to(B), any_up_to(max_q), any_up_to(max_len)
            t = any_up_to(T) if pf else b * q
            st, need = size(c, B=b, max_q=q, max_len=n, prefill=pf, T=t)
            st2, less = bound(c, b, q, n, pf, t)
            assert st == st2 == capi.OK and need <= less <= most, (B, max_q, max_len, T, b, q, n, t)
            parts += need > 0
    assert parts > 100


def test_workspace_of_parts_follows_the_gpu_and_not_the_rows():
    """Rows of q that belong to no sequence take no room, and the bound of prefill stays below 70 MB."""
    c = cfg(n_heads=32, n_kv_heads=8)
    small = size(c, B=1, max_q=1, max_len=65536, prefill=1, T=1)
    assert small[0] == capi.OK and 0 < small[1] < 2 << 20
    assert size(c, B=1, max_q=1, max_len=65536, prefill=1, T=100000) == small
    for kw in GEOMETRIES:
        assert 0 < bound(cfg(**kw), 1000, 100000, 1 << 20, 1, 1 << 20)[1] < 70 << 20
    # a call of a tile's length is one part whatever its batch
    assert bound(c, 1000, 8, 128, 0, 8000) == (capi.OK, 0)


def test_workspace_bound_refuses_what_the_size_does():
    assert bound(None, 1, 1, 64, 0, 1)[0] == capi.ERR_NULL_ARG
    assert bound(cfg(head_dim=96), 1, 1, 64, 1, 1)[0] == capi.ERR_BAD_SHAPE
    for pf in (0, 1):
        for kw in (dict(B=-1), dict(max_q=-1), dict(max_len=-1), dict(T=-1), dict(max_len=1 << 62), dict(B=1 << 62),
                   dict(T=1 << 62)):
            assert bound(cfg(), **{**dict(B=2, max_q=4, max_len=64, prefill=pf, T=8), **kw})[0] == capi.ERR_BAD_SHAPE
    assert bound(cfg(), 0, 8, 1 << 29, 1, 1000) == (capi.OK, 0)
    assert bound(cfg(), 0, 8, 1 << 29, 0, 0) == (capi.OK, 0)
    c = cfg()
    assert A._lib().moe_attn_workspace_bound(ctypes.byref(c), 1, 1, 1, 16, 0, None) == capi.ERR_NULL_ARG
