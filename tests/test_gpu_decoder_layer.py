"""The decoder-layer example: prompts in pieces, single-token steps and a
verify step give what whole prompts give.

Bound of the rows after the attention half: both runs round q, k, v, the
weights, the attention output and the projection to bf16 (u = 2^-8 each at
most) and differ in the order of their sums; the residual row is about as large
as the attention's, so 4 u = 1.6e-2 of a row is the most that six roundings
with random signs come to (2e-2 taken).  The MLP rounds four more times (5e-2)
and may route a token whose scores nearly tie to other experts."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [{}, {"window": 40, "n_sinks": 4}, {"prompts": (1, 300), "steps": 1, "verify": 8}])
def test_stepped_equals_whole(kw):
    import decoder_layer
    print(f"[case] decoder layer {kw}", flush=True)
    attention, layer, alike = decoder_layer.serve(**kw)
    torch.cuda.synchronize()
    print(f"[parity] decoder layer {kw}: attention {attention:.2e}, layer {layer:.2e}, alike {alike:.3f}", flush=True)
    assert attention <= 2e-2
    assert layer <= 5e-2
    assert alike >= 0.9
