"""The helpers of the long attention tests, on the CPU: the fp64 torch definition against the oracle, and that
marked values show a lost tile where values of mean 0 do not."""
import numpy as np
import pytest

from attn_marks import TILE, attend_torch, mark_values
from attn_util import make_batch
from routed_expert_mlp_amd import attention as A


def config(heads, kv, dim, window=0, sinks=0):
    return A.AttnConfig(n_heads=heads, n_kv_heads=kv, head_dim=dim, page_size=16, rotary_dim=0, rope_style=A.ROPE_HALF,
                        norm_eps=1e-6, scale=dim ** -0.5, window=window, n_sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3), (1, 0), (40, 500)])
def test_torch_definition_is_the_oracle(window, sinks):
    cfg = config(6, 2, 64, window, sinks)
    b = mark_values(make_batch(cfg, [130, 5, 9, 0], [40, 5, 12, 3], seed=window))
    for (want, bound), q, k, v in zip(b.expected(), b.qs, b.keys, b.values):
        if not len(k):
            continue
        out, also = attend_torch(cfg, q, k, v, "cpu")
        np.testing.assert_allclose(out, want, rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(also, bound, rtol=1e-9, atol=1e-14)


@pytest.mark.parametrize("n,dim", [(30001, 128), (6700, 64), (20000, 64), (3500, 256)])
def test_marked_values_show_a_lost_tile(n, dim):
    cfg = config(1, 1, dim)
    b = mark_values(make_batch(cfg, [n], [1], seed=n, poison=False))
    (want, bound), = b.expected()
    q, k, v = b.qs[0], b.keys[0], b.values[0]
    tiles = -(-n // TILE)
    for tile in sorted({0, 1, 63, 64, tiles // 2, tiles - 2} & set(range(tiles))):
        keep = np.arange(n) // TILE != tile
        out, _ = attend_torch(cfg, q, k[keep], v[keep], "cpu")
        assert np.max(np.abs(out - want) / bound) > 2.0, f"tile {tile} of {tiles} lost unnoticed"
