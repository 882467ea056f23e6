"""GPU tests of what a call of the attention operators promises beside its
ordinary use: bounds below the lengths."""
import pytest
import torch

from attn_util import assert_within, make_batch
from routed_expert_mlp_amd import attention as A
from test_gpu_attn import DEV, cache_of, config

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,dim,new,lens,max_q,window,sinks", [
    (8, 2, 128, [70, 5, 90], [200, 40, 300], 33, 0, 0),
    (8, 2, 64, [70, 5, 90], [200, 40, 300], 33, 40, 3),
    (4, 1, 256, [9], [9], 1, 0, 0),
    (8, 2, 128, [40, 2], [3000, 2], 5, 0, 0),            # in parts
    (8, 2, 64, [40, 30], [4000, 20], 7, 900, 5),         # in parts; the second one's first positions are below zero
])
def test_prefill_of_more_new_tokens_than_max_q(heads, kv, dim, new, lens, max_q, window, sinks):
    """The first max_q new tokens keep their own positions; the others' rows are not written."""
    b = make_batch(config(heads, kv, dim, 16, window=window, sinks=sinks), lens, new, seed=dim + max_q)
    what = f"prefill of {new} new tokens, max_q {max_q}, window {window}+{sinks}"
    print(f"[case] {what}", flush=True)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    q = b.q.to(DEV)
    out = torch.full_like(q, 7.0)
    A.moe_attn_prefill(b.cfg, cache_of(b), q, torch.tensor(cu, dtype=torch.int32, device=DEV), max_q,
                       torch.tensor(lens, dtype=torch.int32, device=DEV), b.table.to(DEV), max(lens), out)
    got = out.double().cpu().numpy()
    for i, (want, bound) in enumerate(b.expected()):
        n = min(max_q, new[i])
        assert_within(got[cu[i]:cu[i] + n], want[:n], bound[:n], f"{what}, sequence {i}")
        assert (got[cu[i] + n:cu[i + 1]] == 7.0).all(), f"{what}, sequence {i}: a row past max_q was written"
