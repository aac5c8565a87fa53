"""Which operands the bindings of the residual norms and the weighted combine hand on (no GPU needed).

The library is a recorder here and the current device is the tensors' own, so that a well-formed call goes
through and a refusal is for the one thing that is wrong."""
import pytest
import torch

from mixture_experts_layer_03_amd import abi

T, D, K, R = 4, 64, 2, 8
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(abi, "lib", lambda: rec)
    monkeypatch.setattr(abi, "_types", lambda: (torch, F32, -1))       # get_device() of these tensors
    monkeypatch.setattr(abi, "_current_stream", lambda: 0)
    return rec


def _z(*s, dt=BF):
    return torch.zeros(*s, dtype=dt)


def _bwd_args():
    rows = lambda: _z(T, D)
    return dict(d_out=rows(), d_n=rows(), out=rows(), y=rows(), d_x=rows(), d_y=rows(), ws=torch.zeros(4096, dtype=torch.uint8),
                w_post=_z(D), w_pre=_z(D), gate=_z(D), rstd_post=_z(T, dt=F32), rstd_pre=_z(T, dt=F32), d_w_post=_z(D, dt=F32),
                d_w_pre=_z(D, dt=F32), d_gate=_z(D, dt=F32))


def test_the_workspace_of_the_norms_gradient(lib):
    abi.moe_residual_norm_bwd(**_bwd_args())
    assert lib.calls == ["moe_residual_norm_bwd"]
    with pytest.raises(ValueError, match="ws must be contiguous"):
        abi.moe_residual_norm_bwd(**dict(_bwd_args(), ws=torch.zeros(8192, dtype=torch.uint8)[::2]))
    assert len(lib.calls) == 1


def test_a_workspace_on_another_device(lib, monkeypatch):
    ws = torch.zeros(4096, dtype=torch.uint8)
    elsewhere = type("Elsewhere", (torch.Tensor,), {"get_device": lambda self: 0})
    with pytest.raises(ValueError, match="ws must be contiguous and on the current device"):
        abi.moe_residual_norm_bwd(**dict(_bwd_args(), ws=ws.as_subclass(elsewhere)))
    assert not lib.calls
