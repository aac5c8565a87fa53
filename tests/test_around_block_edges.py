"""The edges of the calls around the block that are decided on the host (no GPU needed)."""
import ctypes

import pytest

from mixture_experts_layer_03_amd import abi

P = ctypes.c_void_p(0x1000)      # never dereferenced
N = None
INVALID, UNSUPPORTED = -1, -2


def _bwd(T=4, d=64, gate=N, kind=0, dwp=P, dg=N):
    return abi.lib().moe_residual_norm_bwd(P, P, P, P, gate, kind, P, P, P, P, 1.0, 1, T, d, P, P, dwp, P, dg, P, 1 << 30, N)


@pytest.mark.parametrize("dwp,dg", [(P, P), (N, P), (P, N)])
def test_a_channels_gate_is_not_empty_without_tokens(dwp, dg):
    """[d] values, which the weights' gradients are formed with also where there are no rows."""
    assert _bwd(T=0, kind=1, gate=N, dwp=dwp, dg=dg) == INVALID
    assert b"gate" in abi.lib().moe_last_error()
    assert abi.lib().moe_residual_norm(P, P, N, 1, P, P, 1.0, 1e-6, 1, 0, 64, P, P, P, P, N) == INVALID


@pytest.mark.parametrize("T", [(1 << 26) - 1, (1 << 26) - 3])
def test_norms_of_as_many_tokens_as_a_launch_has_no_threads_for(T):
    """Four rows of a wave each to a block: (T + 3) / 4 blocks of 256 threads, below 2^32 of them."""
    f = abi.lib()
    assert f.moe_residual_norm(P, P, N, 0, P, P, 1.0, 1e-6, 1, T, 8, P, P, P, P, N) == UNSUPPORTED
    assert f.moe_combine_residual_norm(P, 8, P, P, 1, P, N, 0, P, P, 1.0, 1e-6, 1, T, 8, N, P, P, P, P, N) == UNSUPPORTED


@pytest.mark.parametrize("T,k", [((1 << 26) - 1, 1), ((1 << 26) - 3, 1), (22369621, 3)])
def test_a_combines_gradient_of_as_many_slots_as_a_launch_has_no_threads_for(T, k):
    assert T * k in range((1 << 26) - 3, 1 << 26)
    assert abi.lib().moe_combine_weighted_bwd(P, P, 8, P, P, 1, T, 8, k, P, P, N) == UNSUPPORTED


# (the last: 16 bytes short of 2^32, where a counter in steps of some KB never passes the end)
@pytest.mark.parametrize("dtype,d", [(0, 1 << 29), (0, 1 << 30), (1, 1 << 30), (0, (1 << 30) - 8), (1, (1 << 31) - 8)])
def test_rows_of_2_gb(dtype, d):
    """Places in a row are counted in 32 bits of bytes."""
    f, b = abi.lib().moe_combine_weighted, abi.lib().moe_combine_weighted_bwd
    assert f(P, 8, P, P, dtype, 1, d, 1, P, N) == UNSUPPORTED
    assert b(P, P, 8, P, P, dtype, 1, d, 1, P, P, N) == UNSUPPORTED
