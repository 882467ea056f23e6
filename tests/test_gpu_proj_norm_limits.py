"""GPU tests of the norm: any eps above 0, and every form within the roundings of its own sums."""
import numpy as np
import pytest
import torch

from oracle import proj_oracle as PO
from proj_util import E, U, assert_within, bf16
from routed_expert_mlp_amd import projection as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("H", [8, 640, 4104])
@pytest.mark.parametrize("eps", [2.0 ** -126, 2.0 ** -127, 1e-40, 2.0 ** -149])
def test_norm_of_zeros_with_the_least_eps(H, eps):
    """Any eps above 0 gives zeros for a row of zeros, and the norm beside it."""
    rng = np.random.default_rng(H)
    x, xd = bf16(rng.standard_normal((3, H)))
    x[1], xd[1] = 0, 0
    y, q = torch.empty((3, H), dtype=torch.bfloat16, device=DEV), torch.empty((3, H), dtype=torch.uint8, device=DEV)
    s = torch.empty((3, -(-H // 128)), dtype=torch.float32, device=DEV)
    P.moe_proj_norm(x.to(DEV), None, eps, None, None, y, q, s)
    want = PO.norm(xd, None, None, eps)[1]
    assert_within(y.double().cpu().numpy(), want, (U + 32 * E) * np.abs(want), f"norm {H}, eps {eps}")
    assert ((q[1] & 0x7F) == 0).all() and torch.isfinite(s).all()


@pytest.mark.parametrize("H", [8, 136, 512, 520, 1544, 4096, 8192, 8200, 16384])
def test_norm_within_the_roundings_of_its_own_form(H):
    """A lane adds at most 16 squares, 6 steps of a wavefront's tree and 16 wavefronts' sums behind them: 38 e of the sum
    and 2 of the mean and eps, half of that in the root; the root's instruction is off by 1 ulp, 2 e; the products with
    the weight and with h 2, the sum h itself 1: 25 e before the rounding.  A scale has one product and one division's
    rounding more."""
    rng = np.random.default_rng(H)
    (x, xd), (r, rd) = bf16(rng.standard_normal((5, H))), bf16(rng.standard_normal((5, H)))
    w = (1.0 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    y = torch.empty((5, H), dtype=torch.bfloat16, device=DEV)
    q, s = torch.empty((5, H), dtype=torch.uint8, device=DEV), torch.empty((5, -(-H // 128)), dtype=torch.float32,
                                                                         device=DEV)
    P.moe_proj_norm(x.to(DEV), torch.from_numpy(w).to(DEV), 1e-6, r.to(DEV), None, y, q, s)
    want = PO.norm(xd, rd, w, 1e-6)[1]
    assert_within(y.double().cpu().numpy(), want, (U + 25 * E) * np.abs(want), f"norm {H}, y")
    top = np.stack([np.max(np.abs(want[:, i:i + 128]), axis=1) for i in range(0, H, 128)], axis=1) / 448.0
    assert_within(s.double().cpu().numpy(), top, 28 * E * top, f"norm {H}, scale")
