"""Values that are not finite in the gradients of the residual norms and of the weighted combine."""
import pytest
import torch

from mixture_experts_layer_03_amd import abi
from tests.test_gpu_residual_norm import DEV, DT, _inputs, _rand

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


# a piece a lane; two; rows worked twice
@pytest.mark.parametrize("dtype,T,d", [("bf16", 9, 520), ("fp32", 9, 520), ("bf16", 5, 4104), ("fp32", 5, 4104), ("bf16", 3, 8200)])
@pytest.mark.parametrize("gate", ["channel", "token", "element"])
def test_an_infinite_output_without_its_norm(gate, dtype, T, d):
    """out = x + gate y: d_y = gate d_out does not have y in it, and d_gate is infinite where y is."""
    dt = DT[dtype]
    g, x, y, _, _, gt = _inputs(T, d, dt, False, False, gate, 7)
    go = _rand(g, T, d, dt=dt)
    go[go == 0] = 1.0
    y[1, 7], y[2, d - 1] = INF, -INF
    d_x, d_y = torch.empty_like(x), torch.empty_like(x)
    dg = torch.empty_like(gt, dtype=torch.float32 if gate == "channel" else gt.dtype)
    ws = torch.empty(abi.moe_residual_norm_bwd_workspace_size(T, d), dtype=torch.uint8, device=DEV)
    abi.moe_residual_norm_bwd(go, None, None, y, d_x, d_y, ws, gate=gt, d_gate=dg)
    assert torch.equal(d_x, go)
    assert torch.equal(d_y, (go.float() * gt.float()).to(dt))       # one product, rounded once more in bf16
    finite = torch.where(torch.isinf(y), torch.ones_like(y), y)
    dg0, keep = torch.empty_like(dg), torch.empty_like(d_y)
    abi.moe_residual_norm_bwd(go, None, None, finite, d_x, keep, ws, gate=gt, d_gate=dg0)
    at = {"channel": lambda r, c: (c,), "token": lambda r, c: (r, 0), "element": lambda r, c: (r, c)}[gate]
    for r, c in ((1, 7), (2, d - 1)):
        want = float(y[r, c]) * float(go[r, c])
        assert float(dg[at(r, c)]) == want
        dg0[at(r, c)] = want
    assert torch.equal(dg, dg0)
