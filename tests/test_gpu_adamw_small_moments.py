"""AdamW where second moments are below the smallest normal number, 2^-126, and eps is below their roots."""
import pytest
import torch

from mixture_experts_layer_03_amd.optim import AdamW
from tests.test_gpu_adamw import DEV, DT, _check_step, _params

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,master", [("fp32", False), ("bf16", False), ("bf16", True)])
def test_roots_of_small_second_moments(param, master, bits):
    """(1 - beta2) g^2 of gradients of 1e-20 to 3e-14 is 1e-42 to 1e-29: each size in a tensor of its own, so that
    8-bit blocks hold it alone, and all in one.  The bound is test_gpu_adamw's: it knows no smallest moment."""
    sizes = [200] * 6 + [3000]
    g, params = _params(sizes, DT[param], 12)
    decay = [0.0] * len(sizes)
    opt = AdamW(params, lr=1e-2, betas=(0.9, 0.99), eps=1e-30, weight_decay=decay, state_bits=bits,
                masters=True if master else None, seed=21)
    for step in range(3):
        grads = [torch.randn(n, generator=g) for n in sizes]
        grads = [t.sign() * t.abs().clamp(min=0.1) for t in grads]
        size = [torch.full((n,), 10.0 ** (i - 19)) for i, n in enumerate(sizes[:-1])]
        size.append(10.0 ** (torch.rand(sizes[-1], generator=g) * 5 - 19))
        _check_step(opt, [(t * s).to(DEV) for t, s in zip(grads, size)], 1e-2, decay)
    for p, q in zip(params, _params(sizes, DT[param], 12)[1]):
        # the corrected m is a mean of g with weights within 1.1 of those whose mean of g^2 the corrected v is, so a step
        # is below 1.1 lr (4 covers the few bits of v); three bf16 roundings of up to 2^-7
        if bits == 32:
            assert ((p - q).abs() <= 3 * 4 * 1e-2 + q.abs() * 2 ** -5).all()


def test_captured_form():
    g, params = _params([300], torch.float32, 13)
    grad = (torch.randn(300, generator=g).sign() * 3e-20).to(DEV)
    start = params[0].clone()
    opt = AdamW(params, lr=1e-2, betas=(0.9, 0.99), eps=1e-30, weight_decay=0.0, capturable=True)
    opt.step([grad])
    # the first step is lr sign(g): v = 9e-42 has 13 bits, its root is off by 2^-13, and so is lr's factor
    want = start - 1e-2 * grad.sign()
    assert ((params[0] - want).abs() <= 1e-2 * 2 ** -12 + 2 ** -23 * (want.abs() + 1)).all()
