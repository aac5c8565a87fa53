"""Each gradient of the residual norms is the same whichever others are asked for."""
import itertools

import pytest
import torch

from mixture_experts_layer_03_amd import abi
from oracle import around_block as O
from tests.test_gpu_residual_norm import DEV, DT, _inputs, _np, _rand

pytestmark = pytest.mark.gpu


# a piece a lane; two; rows worked twice
@pytest.mark.parametrize("dtype,T,d", [("bf16", 20, 520), ("fp32", 20, 520), ("bf16", 5, 4104), ("bf16", 3, 8200)])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_every_choice_of_outputs(gate, post, pre, dtype, T, d):
    dt = DT[dtype]
    g, o, y, wp, wn, gt = _inputs(T, d, dt, post, pre, gate, 17)
    d_out, d_n = _rand(g, T, d, dt=dt), _rand(g, T, d, dt=dt) if pre else None
    rp = torch.tensor(O.rstd(_np(y), 1e-5)[:, 0]).float().to(DEV) if post else None
    rn = torch.tensor(O.rstd(_np(o), 1e-5)[:, 0]).float().to(DEV) if pre else None
    ws = torch.empty(abi.moe_residual_norm_bwd_workspace_size(T, d), dtype=torch.uint8, device=DEV)
    new = {"d_x": lambda: torch.empty_like(o), "d_y": lambda: torch.empty_like(o)}
    if post:
        new["d_w_post"] = lambda: torch.empty(d, device=DEV)
    if pre:
        new["d_w_pre"] = lambda: torch.empty(d, device=DEV)
    if gt is not None:
        new["d_gate"] = lambda: torch.empty_like(gt, dtype=torch.float32 if gate == "channel" else dt if gate == "element" else None)

    def grads(names):
        b = {n: new[n]() for n in names}
        abi.moe_residual_norm_bwd(d_out, d_n, o, y, b.get("d_x"), b.get("d_y"), ws, wp, wn, gt, 0.75, rp, rn, b.get("d_w_post"),
                                  b.get("d_w_pre"), b.get("d_gate"))
        return b

    whole = grads(new)
    for count in range(1, len(new)):
        for names in itertools.combinations(new, count):
            for n, t in grads(names).items():
                assert torch.equal(t, whole[n]), (names, n)
