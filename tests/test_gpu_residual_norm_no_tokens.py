"""The residual norms' gradient where there are no tokens."""
import pytest
import torch

from mixture_experts_layer_03_amd import abi
from tests.test_gpu_residual_norm import DEV, DT

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("want_w,want_g", [(True, True), (True, False), (False, True)])
def test_no_tokens_give_zero_whatever_the_factors(want_w, want_g, dtype):
    d, dt = 136, DT[dtype]
    z, r = torch.empty(0, d, dtype=dt, device=DEV), torch.empty(0, device=DEV)
    w, gate = (torch.ones(d, dtype=dt, device=DEV) for _ in range(2))
    w[3], w[70], gate[5], gate[100] = INF, NAN, -INF, NAN
    new = lambda want: torch.full((d,), 3.0, device=DEV) if want else None
    dwp, dwn, dg = new(want_w), new(True), new(want_g)
    abi.moe_residual_norm_bwd(z, z, z, z, None, None, None, w, w, gate, 1.0, r, r, dwp, dwn, dg)
    for t in (dwp, dwn, dg):
        assert t is None or (t == 0).all()
