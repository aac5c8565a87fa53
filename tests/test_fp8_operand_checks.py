"""The 8-bit calls refuse operands that they would read or write past the end, before the library is called."""
import pytest
import torch

from mixture_experts_layer_03_amd import abi

E, N, K, R, F = 3, 272, 400, 10, 144      # N and K: 3 and 4 blocks of 128; 2 F: 3


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


@pytest.fixture
def calls(monkeypatch):
    done = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: done.append(name) or 0

    monkeypatch.setattr(abi, "lib", lambda: Library())
    return done


def _rows():
    return dict(x=torch.zeros(R, K), q=u8(R, K), scale=u8(R, 4))


def _weights():
    return dict(w=torch.zeros(E, N, K), q=u8(E, N, K), scale=u8(E, 3, 4), qt=u8(E, K, N), scale_t=u8(E, 4, 4))


def _product(gathered=False):
    rows = R // 2 if gathered else R
    out = dict(a=u8(rows, K), a_scale=u8(rows, 4), offsets=torch.zeros(E + 1, dtype=torch.int32), b=u8(E, N, K),
               b_scale=u8(E, 3, 4), row_scale=torch.zeros(R), c=torch.zeros(R, N, dtype=torch.bfloat16))
    if gathered:
        out.update(row_to_slot=torch.zeros(R, dtype=torch.int32), k=2)
    return out


def _ffn(gathered=False):
    rows = R // 2 if gathered else R
    out = dict(x=u8(rows, K), x_scale=u8(rows, 4), offsets=torch.zeros(E + 1, dtype=torch.int32), w_gu=u8(E, 2 * F, K),
               w_gu_scale=u8(E, 3, 4), w_down=u8(E, K, F), w_down_scale=u8(E, 4, 4), row_scale=torch.zeros(R),
               h=u8(R, F), h_scale=u8(R, 4), y_perm=torch.zeros(R, K, dtype=torch.bfloat16))
    if gathered:
        out.update(row_to_slot=torch.zeros(R, dtype=torch.int32), k=2)
    return out


def _call(fn, args):
    getattr(abi, fn)(**args, stream=0)


CALLS = [("moe_quant_rows_fp8", _rows), ("moe_quant_weights_fp8", _weights), ("moe_grouped_gemm_fp8", _product),
         ("moe_grouped_ffn_fwd_fp8", _ffn), ("moe_grouped_gemm_fp8", lambda: _product(True)),
         ("moe_grouped_ffn_fwd_fp8", lambda: _ffn(True))]


@pytest.mark.parametrize("fn,make", CALLS, ids=["rows", "weights", "product", "ffn", "product-gathered", "ffn-gathered"])
def test_operands_that_fit_are_passed_on(fn, make, calls):
    args = make()
    _call(fn, args)
    for name in args:                       # more rows than are needed, and flat scales, fit
        if name in ("x", "w", "b", "w_down", "c", "y_perm", "k"):
            continue
        _call(fn, dict(args, **{name: torch.cat([args[name], args[name]])}))
        if "scale" in name:
            _call(fn, dict(args, **{name: args[name].reshape(-1)}))
    for name in ("row_scale", "qt"):
        if name in args:
            _call(fn, dict(args, **({"qt": None, "scale_t": None} if name == "qt" else {name: None})))
    assert set(calls) == {fn} and len(calls) > 3


@pytest.mark.parametrize("fn,make", CALLS, ids=["rows", "weights", "product", "ffn", "product-gathered", "ffn-gathered"])
def test_operands_that_do_not_fit_are_refused(fn, make, calls):
    args = make()
    bad = []
    for name, t in args.items():
        if name in ("x", "w", "b", "w_down", "k", "y_perm", "c"):
            continue                        # these give the sizes
        bad.append((name, t.reshape(-1)[:-1]))
        if "scale" in name and t.dim() > 1:
            wide = u8(*t.shape[:-2], 2 * t.shape[-2], 5)
            bad += [(name, t[..., :3].contiguous()), (name, wide), (name, wide[..., :4])]
    if fn == "moe_grouped_ffn_fwd_fp8":
        bad += [("x", args["x"][1:]), ("w_gu", args["w_gu"][1:])]
    if fn == "moe_grouped_gemm_fp8":
        bad += [("a", args["a"][1:]), ("c", args["c"].to(torch.uint8))]
    for name in ("x", "w", "a", "b", "q", "h", "w_gu", "qt"):
        if name in args:
            bad.append((name, args[name].transpose(-1, -2).contiguous().transpose(-1, -2)))
    if "row_scale" in args:
        bad.append(("row_scale", args["row_scale"].bfloat16()))
    for name, t in bad:
        with pytest.raises(ValueError, match=name):
            _call(fn, dict(args, **{name: t}))
            print(fn, name, tuple(t.shape))
    assert not calls
