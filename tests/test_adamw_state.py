"""The states of optim.AdamW stay those that its kernel steps (no GPU needed)."""
import copy
import io

import pytest
import torch

from mixture_experts_layer_03_amd.optim import AdamW

BF = torch.bfloat16


def _opt(bits=8, masters=True, **kw):
    return AdamW([torch.ones(300, dtype=BF), torch.ones(7, dtype=BF)], lr=1e-3, state_bits=bits, masters=masters or None, **kw)


def _pointers(opt):
    """What the kernel is given."""
    names = ["m", "v"] + (["m_scale", "v_scale"] if opt.state_bits == 8 else []) + (["master"] if opt.masters else [])
    return [getattr(t, n) for t in opt._table for n in names]


def _shown(opt):
    lists = [opt.state[n] for n in opt.state] + ([opt.masters] if opt.masters else [])
    return [t.data_ptr() for i in range(len(opt.params)) for t in (l[i] for l in lists)]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("masters", [True, False])
def test_no_other_tensors_in_their_place(bits, masters):
    opt = _opt(bits, masters)
    given = _pointers(opt)
    assert _shown(opt) == given
    with pytest.raises(TypeError):
        opt.state["m"][0] = torch.zeros_like(opt.state["m"][0])
    with pytest.raises(TypeError):
        opt.state["m"] = list(opt.state["v"])
    with pytest.raises(TypeError):
        opt.state.update(m=list(opt.state["v"]))
    with pytest.raises(AttributeError):
        opt.state = {"m": [], "v": []}
    with pytest.raises(AttributeError):
        opt.masters = None
    if masters:
        with pytest.raises(TypeError):
            opt.masters[0] = torch.zeros(300)
    # a tensor that was handed out and moved is not the optimizer's any more
    moved = opt.state["v"][0]
    moved.data = torch.zeros_like(moved)
    assert _shown(opt) == given == _pointers(opt)


def test_the_callers_tensors_are_stepped_and_kept():
    state = {"m": [torch.zeros(300), torch.zeros(7)], "v": [torch.zeros(300), torch.zeros(7)]}
    masters = [torch.ones(300), torch.ones(7)]
    opt = AdamW([torch.ones(300, dtype=BF), torch.ones(7, dtype=BF)], lr=1e-3, state=state, masters=masters)
    given = [state["m"][0].data_ptr(), state["v"][0].data_ptr(), masters[0].data_ptr(), state["m"][1].data_ptr(),
             state["v"][1].data_ptr(), masters[1].data_ptr()]
    assert _pointers(opt) == given
    state["m"][0].data = torch.full((300,), 5.0)     # the caller's tensor goes elsewhere; what the kernel has stays
    del state, masters
    assert _shown(opt) == given and (opt.state["m"][0] == 0).all()
    opt.state["m"][0].fill_(2.0)
    assert (opt.state["m"][0] == 2).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_saved_and_loaded(bits):
    opt, other = _opt(bits), _opt(bits)
    for ts in opt.state.values():
        for i, t in enumerate(ts):
            t.view(torch.uint8).fill_(3 + i)
    opt.masters[1].fill_(0.25)
    f = io.BytesIO()
    torch.save({"state": opt.state, "masters": opt.masters}, f)
    f.seek(0)
    kept = torch.load(f, weights_only=True)
    given = _pointers(other)
    other.load_state(kept["state"], step=12, masters=kept["masters"])
    assert _shown(other) == given == _pointers(other) and other.steps == 12
    for n in opt.state:
        for a, b in zip(opt.state[n], other.state[n]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert (other.masters[1] == 0.25).all() and (other.masters[0] == 1).all()
    again = AdamW(opt.params, lr=1e-3, state_bits=bits, state=copy.deepcopy(opt.state), masters=list(opt.masters))
    assert torch.equal(again.state["m"][0].view(torch.uint8), opt.state["m"][0].view(torch.uint8))


def test_what_load_state_refuses():
    opt = _opt(32)
    ok = {n: [t.clone() for t in ts] for n, ts in opt.state.items()}
    masters = [t.clone() for t in opt.masters]
    ok["m"][0].fill_(9.0)
    for state, ms in (({"m": ok["m"]}, masters), ({**ok, "v": ok["v"][:1]}, masters), ({**ok, "v": [ok["v"][1], ok["v"][0]]}, masters),
                      ({**ok, "v": [t.double() for t in ok["v"]]}, masters), (ok, None), (ok, masters[:1])):
        with pytest.raises(ValueError):
            opt.load_state(state, step=3, masters=ms)
        assert opt.steps == 0 and (opt.state["m"][0] == 0).all()       # nothing is copied of a state that does not fit
    with pytest.raises(ValueError):
        _opt(32, masters=False).load_state(ok, step=3, masters=masters)
