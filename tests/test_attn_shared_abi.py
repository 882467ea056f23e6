"""C ABI of decode behind a shared prefix without a GPU: bad arguments are refused before anything is enqueued (so
fake device addresses are safe)."""
import ctypes
import math
import random

import pytest

from routed_expert_mlp_amd import attention as A
from routed_expert_mlp_amd import capi
from test_attn_abi import BIG, FAKE, cache, cfg


def size(c, B=2, n_q=1, max_len=64, shared=20):
    n = ctypes.c_size_t(0)
    st = A._lib().moe_attn_shared_workspace_size(ctypes.byref(c) if c is not None else None, B, n_q, max_len, shared,
                                                 ctypes.byref(n))
    return st, n.value


def call(c, cc, B=2, n_q=1, max_pages=4, max_len=64, shared=20, q=FAKE, lens=FAKE, table=FAKE, pages=FAKE, out=FAKE,
         ws=FAKE, wsb=BIG):
    return A._lib().moe_attn_decode_shared(ctypes.byref(c) if c is not None else None,
                                           ctypes.byref(cc) if cc is not None else None, q, B, n_q, lens, table,
                                           max_pages, max_len, pages, shared, out, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_heads=0), capi.ERR_BAD_SHAPE), (dict(n_heads=7), capi.ERR_BAD_SHAPE), (dict(head_dim=96), capi.ERR_BAD_SHAPE),
    (dict(page_size=8), capi.ERR_BAD_SHAPE), (dict(window=-1), capi.ERR_BAD_VALUE), (dict(n_sinks=-1), capi.ERR_BAD_VALUE),
    (dict(scale=0.0), capi.ERR_BAD_VALUE), (dict(scale=math.nan), capi.ERR_BAD_VALUE),
])
def test_config(kw, code):
    assert call(cfg(**kw), cache()) == code and size(cfg(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    (dict(shared=-1), capi.ERR_BAD_SHAPE), (dict(shared=65), capi.ERR_BAD_SHAPE), (dict(B=-1), capi.ERR_BAD_SHAPE),
    (dict(n_q=0), capi.ERR_BAD_SHAPE), (dict(n_q=9), capi.ERR_BAD_SHAPE), (dict(max_len=-1), capi.ERR_BAD_SHAPE),
    (dict(max_len=65), capi.ERR_BAD_SHAPE), (dict(max_pages=-1), capi.ERR_BAD_SHAPE), (dict(max_pages=3), capi.ERR_BAD_SHAPE),
    (dict(B=1 << 25), capi.ERR_BAD_SHAPE), (dict(max_len=1 << 30, max_pages=1 << 27), capi.ERR_BAD_SHAPE),
    (dict(q=None), capi.ERR_NULL_ARG), (dict(lens=None), capi.ERR_NULL_ARG), (dict(table=None), capi.ERR_NULL_ARG),
    (dict(pages=None), capi.ERR_NULL_ARG), (dict(out=None), capi.ERR_NULL_ARG), (dict(ws=None), capi.ERR_NULL_ARG),
    (dict(q=FAKE + 8), capi.ERR_MISALIGNED), (dict(lens=FAKE + 2), capi.ERR_MISALIGNED),
    (dict(table=FAKE + 1), capi.ERR_MISALIGNED), (dict(pages=FAKE + 2), capi.ERR_MISALIGNED),
    (dict(out=FAKE + 4), capi.ERR_MISALIGNED), (dict(ws=FAKE + 8), capi.ERR_MISALIGNED),
    (dict(wsb=0), capi.ERR_WORKSPACE_TOO_SMALL), (dict(B=0), 0), (dict(B=0, q=None, ws=None), 0),
])
def test_arguments(kw, code):
    assert call(cfg(), cache(), **kw) == code


def test_cache_and_null():
    assert call(None, cache()) == capi.ERR_NULL_ARG and size(None)[0] == capi.ERR_NULL_ARG
    assert call(cfg(), None) == capi.ERR_NULL_ARG
    assert call(cfg(), cache(k=None)) == capi.ERR_NULL_ARG
    assert call(cfg(), cache(n_pages=0)) == capi.ERR_BAD_SHAPE
    assert call(cfg(), cache(v=FAKE + 2)) == capi.ERR_MISALIGNED
    assert A._lib().moe_attn_shared_workspace_size(ctypes.byref(cfg()), 2, 1, 64, 20, None) == capi.ERR_NULL_ARG


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv", [(1, 1), (32, 8), (128, 1), (24, 3)])
def test_sizes_of_many_calls(dim, heads, kv):
    """Every size that a call may have has a workspace, and a byte less than it asks for is refused."""
    for window, sinks in ((0, 0), (100, 5), (1 << 30, 1 << 30)):
        c = cfg(head_dim=dim, n_heads=heads, n_kv_heads=kv, window=window, n_sinks=sinks)
        for B in (1, 3, 64, 300):
            for n_q in (1, 4):
                for shared in (0, 1, 31, 32, 1000, 65536):
                    for own in (0, 1, 33, 5000):
                        st, need = size(c, B, n_q, shared + own, shared)
                        assert st == 0 and need > 0
                        assert call(c, cache(), B=B, n_q=n_q, max_pages=1 << 20, max_len=shared + own, shared=shared,
                                    wsb=need - 1) == capi.ERR_WORKSPACE_TOO_SMALL


def bound(c, B, n_q, max_len):
    n = ctypes.c_size_t(0)
    st = A._lib().moe_attn_shared_workspace_bound(ctypes.byref(c) if c is not None else None, B, n_q, max_len,
                                                  ctypes.byref(n))
    return st, n.value


def test_bound_refusals():
    assert bound(None, 2, 1, 64)[0] == capi.ERR_NULL_ARG
    assert bound(cfg(head_dim=96), 2, 1, 64)[0] == capi.ERR_BAD_SHAPE
    assert bound(cfg(), 2, 0, 64)[0] == capi.ERR_BAD_SHAPE
    assert bound(cfg(), -1, 1, 64)[0] == capi.ERR_BAD_SHAPE
    assert bound(cfg(), 0, 1, 64) == (0, 0)
    assert A._lib().moe_attn_shared_workspace_bound(ctypes.byref(cfg()), 2, 1, 64, None) == capi.ERR_NULL_ARG


def _spread(rng, high):
    """A size up to high, over its logarithm, the ends among them."""
    return rng.choice([high, max(1, int(round(math.exp(rng.uniform(0, math.log(high + 1)))))), rng.randint(1, high)])


@pytest.mark.parametrize("seed", range(12))
def test_bound_is_enough_for_smaller_calls(seed):
    rng = random.Random(seed)
    for _ in range(150):
        kv = rng.choice([1, 2, 3, 8])
        window = rng.choice([0, 0, 500, 1 << 20])
        c = cfg(head_dim=rng.choice([64, 128, 256]), n_kv_heads=kv, n_heads=kv * rng.choice([1, 3, 4, 16, 64]),
                window=window, n_sinks=rng.choice([0, 4, 3000]))
        B, n_q, max_len = _spread(rng, 512), rng.randint(1, 8), _spread(rng, 300000)
        st, most = bound(c, B, n_q, max_len)
        assert st == 0
        for _ in range(12):
            b, n, m = _spread(rng, B), rng.randint(1, n_q), _spread(rng, max_len)
            for shared in (0, m, m // 2, max(0, m - 100), rng.randint(0, m)):
                st, need = size(c, min(b, B), n, min(m, max_len), min(shared, m, max_len))
                assert st == 0 and need <= most, (B, n_q, max_len, b, n, m, shared)
