"""GPU parity of the 8-bit products at the sizes where each of their kernels runs.

The kernel of big tiles takes products of more than 32 rows an expert (gate/up: 20)
whose small tiles do not all run at once: here many output columns reach it with
few rows, so that the ragged ends of its tiles (rows, columns, K, experts) are
cheap to cover.  Bounds are those of tests/test_gpu_fp8.py.
"""
import numpy as np
import pytest

from mixture_experts_layer_03_amd import inputs as I
from oracle import scored_fp8 as S
from tests.gpu_util import down, need_gpu
from tests.test_gpu_fp8 import U, _check, _i32, _offsets, _rng, _spread, _u8

pytestmark = pytest.mark.gpu

# rows per expert, N, K: big tiles, but for the last two
BIG = [([300, 0, 2, 65], 16400, 144), ([257, 511], 8336, 400), ([129, 127, 256, 1, 0], 13328, 64),
       ([70] * 30 + [0] * 5, 2064, 272), ([1100], 4112, 2880), ([255, 3], 24592, 16), ([1060], 4112, 8336),
       ([900, 1], 528, 1136), ([40, 3, 90], 80, 192)]


@pytest.mark.parametrize("mode", ["plain", "weighted", "gathered"])
@pytest.mark.parametrize("case", range(len(BIG)), ids=["N%d-K%d-R%d" % (n, k, sum(c)) for c, n, k in BIG])
def test_product_of_many_columns(case, mode):
    import torch
    from mixture_experts_layer_03_amd import abi
    dev = need_gpu()
    counts, N, K = BIG[case]
    E, R, k = len(counts), sum(counts), 1
    print("GPU case big product", counts[:6], N, K, mode, flush=True)
    r = _rng(29 * case + 3)
    n = R
    if mode == "gathered":
        k = 4
        R += -R % k
    rows = R // k if mode == "gathered" else R
    aq, asc = S.quant_rows(_spread(r, (rows, K), True))
    slot = r.permutation(R).astype(np.int32)
    w = (r.random(R) + 0.1).astype(np.float32) if mode != "plain" else None
    off = _offsets(counts)
    av = S.row_values(aq, asc)
    if mode == "gathered":
        av = av[slot // k]
    bq = np.empty((E, N, K), np.uint8)
    bsc = np.empty((E, -(-N // 128), S.scale_cols(K)), np.uint8)
    for e in range(E):
        bq[e], bsc[e] = (t[0] for t in S.quant_weights(_spread(r, (1, N, K), True) / np.sqrt(K)))
    out = torch.full((R + 1, N), 9.0, dtype=torch.bfloat16, device=dev)
    again = torch.full((R, N), 9.0, dtype=torch.bfloat16, device=dev)
    args = (_u8(aq, dev), _u8(asc, dev), _i32(off, dev), _u8(bq, dev), _u8(bsc, dev),
            None if w is None else torch.from_numpy(w).to(dev))
    kw = dict(row_to_slot=_i32(slot, dev), k=k) if mode == "gathered" else {}
    abi.moe_grouped_gemm_fp8(*args, out[:R], **kw)
    abi.moe_grouped_gemm_fp8(*args, again, **kw)
    torch.cuda.synchronize()
    assert (out[n:] == 9.0).all() and torch.equal(out[:R], again)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            c, err = S.product(av[a:b], np.array([0, b - a]), [S.weight_values(bq[e], bsc[e])], None if w is None else w[a:b])
            _check(down(out[a:b]), c, err)


# rows per expert, d, f, k: big tiles; few rows with K = 64 mod 128, whose weight rows begin inside a line
BIG_FFN = [([300, 0, 260, 40], 272, 4112, 1), ([129, 255], 64, 8208, 2), ([600], 2880, 4144, 1), ([70] * 20, 144, 1040, 4),
           ([1, 0, 17, 30, 5], 576, 144, 1), ([64, 1, 3], 192, 400, 4), ([2, 1], 64, 128, 1), ([33] + [0] * 70 + [9], 8256, 80, 2)]


@pytest.mark.parametrize("case", range(len(BIG_FFN)), ids=["d%d-f%d-R%d-k%d" % (d, f, sum(c), k) for c, d, f, k in BIG_FFN])
def test_ffn_of_big_tiles_and_of_rows_that_begin_inside_a_line(case):
    import torch
    from mixture_experts_layer_03_amd import abi
    dev = need_gpu()
    counts, d, f, k = BIG_FFN[case]
    E, R = len(counts), sum(counts)
    assert R % k == 0
    print("GPU case big ffn", counts[:6], d, f, k, flush=True)
    r = _rng(23 * case + 11)
    xq, xsc = S.quant_rows(I.round_to_bf16(r.standard_normal((R // k, d)).astype(np.float32)))
    gq, gsc = S.quant_weights(_spread(r, (E, 2 * f, d), True) / np.sqrt(d) / 8)
    dq, dsc = S.quant_weights(r.standard_normal((E, d, f)) / np.sqrt(f))
    slot = r.permutation(R).astype(np.int32)
    w = (r.random(R) + 0.1).astype(np.float32)
    off = _offsets(counts)
    u8 = dict(dtype=torch.uint8, device=dev)
    h, hs = torch.full((R + 1, f), 77, **u8), torch.full((R + 1, S.scale_cols(f)), 77, **u8)
    y = torch.full((R + 1, d), 9.0, dtype=torch.bfloat16, device=dev)
    abi.moe_grouped_ffn_fwd_fp8(_u8(xq, dev), _u8(xsc, dev), _i32(off, dev), _u8(gq, dev), _u8(gsc, dev), _u8(dq, dev),
                                _u8(dsc, dev), torch.from_numpy(w).to(dev), h[:R], hs[:R], y[:R],
                                row_to_slot=_i32(slot, dev) if k > 1 else None, k=k)
    torch.cuda.synchronize()
    assert (h[R] == 77).all() and (hs[R] == 77).all() and (y[R] == 9.0).all()
    x = S.row_values(xq, xsc)
    x = x[slot // k] if k > 1 else x
    hq, hsc = h[:R].cpu().numpy(), hs[:R].cpu().numpy()
    got = S.row_values(hq, hsc)
    nb = -(-f // 128)
    assert (hsc[:, nb:] == 127).all()
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        gu, err = S.product(x[a:b], np.array([0, b - a]), [S.weight_values(gq[e], gsc[e])])
        ref = S.swiglu(gu)
        dh = 1.1 * err[:, :f] * (np.abs(gu[:, f:]) + err[:, f:]) + np.abs(gu[:, :f]) * err[:, f:] \
            + (2 * np.abs(gu[:, :f]) + 16) * U * np.abs(ref)
        rsc = S.quant_rows(ref)[1]
        step = np.repeat(np.exp2(np.maximum(hsc[a:b], rsc).astype(np.float64) - 127), 128, 1)[:, :f]
        half = np.maximum(np.maximum(np.abs(ref), np.abs(got[a:b])) * 2.0 ** -4, step * 2.0 ** -10)
        assert (np.abs(got[a:b] - ref) <= dh + half).all()
        for i in range(nb):
            v, s = np.abs(ref[:, i * 128:(i + 1) * 128]), hsc[a:b, i].astype(np.int64) - 127
            ee = dh[:, i * 128:(i + 1) * 128]
            lo = S.block_exponent(np.maximum((v - ee).max(1), 2.0 ** -140))
            assert ((s >= lo) & (s <= S.block_exponent((v + ee).max(1)))).all()
        c, err = S.product(got[a:b], np.array([0, b - a]), [S.weight_values(dq[e], dsc[e])], w[a:b])
        _check(down(y[a:b]), c, err)


@pytest.mark.parametrize("R", [4095, 4096])
def test_quant_rows_where_the_split_over_waves_ends(R):
    import torch
    from mixture_experts_layer_03_amd import abi
    dev = need_gpu()
    x = _spread(_rng(R), (R, 1168), False)
    q = torch.empty(R, 1168, dtype=torch.uint8, device=dev)
    sc = torch.empty(R, S.scale_cols(1168), dtype=torch.uint8, device=dev)
    abi.moe_quant_rows_fp8(torch.from_numpy(x).to(dev), q, sc)
    torch.cuda.synchronize()
    rq, rs = S.quant_rows(x)
    assert np.array_equal(sc.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("shift", [16, 64, 112])
@pytest.mark.parametrize("counts,d,f", [([3, 0, 20], 192, 144), ([600], 144, 4112), ([90, 70], 576, 272)],
                         ids=["few", "big", "mid"])
def test_pointers_aligned_to_16_bytes_only(counts, d, f, shift):
    """The results do not depend on where in a line the operands begin."""
    import torch
    from mixture_experts_layer_03_amd import abi
    dev = need_gpu()
    r = _rng(d + f)
    E, R = len(counts), sum(counts)

    def at(t):   # the same bytes, `shift` behind a line
        raw = t.contiguous().view(torch.uint8).reshape(-1)
        buf = torch.zeros(raw.numel() + 128 + shift, dtype=torch.uint8, device=dev)
        base = -buf.data_ptr() % 128 + shift
        buf[base:base + raw.numel()] = raw
        return buf[base:base + raw.numel()].view(t.dtype).view(t.shape)

    x = torch.from_numpy(r.standard_normal((R, d)).astype(np.float32)).to(dev).bfloat16()
    wg = torch.from_numpy(r.standard_normal((E, 2 * f, d)).astype(np.float32)).to(dev)
    wd = torch.from_numpy(r.standard_normal((E, d, f)).astype(np.float32)).to(dev)
    off = _i32(_offsets(counts), dev)
    out = []
    for put in (lambda t: t, at):
        u8 = dict(dtype=torch.uint8, device=dev)
        q, s = put(torch.zeros(R, d, **u8)), put(torch.zeros(R, S.scale_cols(d), **u8))
        abi.moe_quant_rows_fp8(put(x), q, s)
        gq, gs = put(torch.zeros(E, 2 * f, d, **u8)), put(torch.zeros(E, -(-2 * f // 128), S.scale_cols(d), **u8))
        abi.moe_quant_weights_fp8(put(wg), gq, gs)
        dq, ds = put(torch.zeros(E, d, f, **u8)), put(torch.zeros(E, -(-d // 128), S.scale_cols(f), **u8))
        dt, dts = put(torch.zeros(E, f, d, **u8)), put(torch.zeros(E, -(-f // 128), S.scale_cols(d), **u8))
        abi.moe_quant_weights_fp8(put(wd), dq, ds, dt, dts)
        h, hs = put(torch.zeros(R, f, **u8)), put(torch.zeros(R, S.scale_cols(f), **u8))
        y = put(torch.zeros(R, d, dtype=torch.bfloat16, device=dev))
        abi.moe_grouped_ffn_fwd_fp8(q, s, off, gq, gs, dq, ds, None, h, hs, y)
        torch.cuda.synchronize()
        out.append([q, s, gq, gs, dq, ds, dt, dts, h, hs, y])
    for a, b in zip(*out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _whole(gen, *shape):
    """Whole numbers up to 8 as e4m3, drawn a slice at a time."""
    import torch
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=gen.device)
    for i in range(shape[0]):
        out[i] = torch.randint(-8, 9, shape[1:], generator=gen, device=gen.device).to(torch.float8_e4m3fn)
    return out


def test_results_past_2_31_elements():
    import torch
    from mixture_experts_layer_03_amd import abi
    dev = need_gpu()
    gen = torch.Generator(device=dev).manual_seed(1)
    R, N, K, E = 70000, 32768, 64, 3
    a, b = _whole(gen, 1, R, K)[0], _whole(gen, E, N, K)
    one = dict(fill_value=127, dtype=torch.uint8, device=dev)
    asc, bsc = torch.full((R, 4), **one), torch.full((E, N // 128, 4), **one)
    off = [0, 1000, 69000, R]
    c = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    assert c.numel() > 2 ** 31
    abi.moe_grouped_gemm_fp8(a, asc, _i32(off, dev), b, bsc, None, c)
    torch.cuda.synchronize()
    for e, rows in enumerate([slice(0, 64), slice(65500, 65600), slice(R - 200, R)]):
        assert torch.equal(c[rows], (a[rows].float() @ b[e].float().T).bfloat16()), e   # exact, rounded once


@pytest.mark.parametrize("rows", [2, 40], ids=["few", "big"])
def test_weights_past_2_31_bytes(rows):
    import torch
    from mixture_experts_layer_03_amd import abi
    dev = need_gpu()
    gen = torch.Generator(device=dev).manual_seed(rows)
    E, N, K = 520, 2048, 2064
    R = E * rows
    a, b = _whole(gen, 1, R, K)[0], _whole(gen, E, N, K)
    assert b.numel() > 2 ** 31
    one = dict(fill_value=127, dtype=torch.uint8, device=dev)
    asc, bsc = torch.full((R, S.scale_cols(K)), **one), torch.full((E, N // 128, S.scale_cols(K)), **one)
    off = _i32(np.arange(E + 1) * rows, dev)
    c = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    abi.moe_grouped_gemm_fp8(a, asc, off, b, bsc, None, c)
    torch.cuda.synchronize()
    for e in (0, 259, 508, 519):
        i = slice(e * rows, (e + 1) * rows)
        assert torch.equal(c[i], (a[i].float() @ b[e].float().T).bfloat16()), e
    if rows > 2:
        return
    # gate/up over the same bytes: the last expert's rows by themselves give the same
    f, i = N // 2, slice(R - 2, R)
    dq, ds = _whole(gen, E, K, f), torch.full((E, -(-K // 128), S.scale_cols(f)), **one)

    def ffn(x, xs, o, e):
        n = x.shape[0]
        h, hs = torch.empty(n, f, dtype=torch.uint8, device=dev), torch.empty(n, S.scale_cols(f), dtype=torch.uint8, device=dev)
        y = torch.empty(n, K, dtype=torch.bfloat16, device=dev)
        abi.moe_grouped_ffn_fwd_fp8(x, xs, o, b[e], bsc[e].clone(), dq[e], ds[e].clone(), None, h, hs, y)
        torch.cuda.synchronize()
        return h, hs, y
    whole, last = ffn(a, asc, off, slice(0, E)), ffn(a[i].clone(), asc[i].clone(), _i32([0, 2], dev), slice(E - 1, E))
    for p, q in zip(whole, last):
        assert torch.equal(p[i], q)


def test_quantisation_past_2_31_elements():
    import torch
    from mixture_experts_layer_03_amd import abi
    dev = need_gpu()
    u8 = dict(dtype=torch.uint8, device=dev)
    x = torch.empty(300000, 8192, dtype=torch.bfloat16, device=dev).normal_()
    assert x.numel() > 2 ** 31
    q, s = torch.empty(x.shape, **u8), torch.empty(x.shape[0], 64, **u8)
    abi.moe_quant_rows_fp8(x, q, s)
    lq, ls = torch.empty(50, 8192, **u8), torch.empty(50, 64, **u8)
    abi.moe_quant_rows_fp8(x[-50:], lq, ls)
    torch.cuda.synchronize()
    assert torch.equal(q[-50:], lq) and torch.equal(s[-50:], ls)
    w = x.view(-1)[:600 * 2048 * 1936].view(600, 2048, 1936)
    sizes = [(2048, 1936), (16, 16), (1936, 2048), (16, 16)]
    out = [torch.empty(600, *z, **u8) for z in sizes]
    assert S.scale_cols(1936) == S.scale_cols(2048) == 16 and out[0].numel() > 2 ** 31
    abi.moe_quant_weights_fp8(w, *out)
    last = [torch.empty(1, *z, **u8) for z in sizes]
    abi.moe_quant_weights_fp8(w[-1:], *last)
    torch.cuda.synchronize()
    for p, q in zip(out, last):
        assert torch.equal(p[-1:], q)


@pytest.mark.parametrize("counts,d,f", [([1, 0, 3], 2880, 1040), ([2, 9, 1, 17], 512, 720), ([19], 720, 1296)],
                         ids=["d2880", "d512", "d720"])
def test_gate_up_of_few_rows_cuts_no_products(counts, d, f):
    """448 * 448 - 448 * 448 + u within 8 consecutive k is u, and silu(32) u = 32 u (e^-32 is below half a unit):
    whole numbers that h holds exactly."""
    import torch
    from mixture_experts_layer_03_amd import abi
    dev = need_gpu()
    print("GPU case few rows", counts, d, f, flush=True)
    E, R = len(counts), sum(counts)
    x, w = np.zeros((R, d)), np.zeros((E, 2 * f, d))
    x[:, 0::8], x[:, 1::8], x[:, 2::8] = 448, 448, 1
    j = np.arange(f)
    u = np.empty((E, f))
    for e in range(E):
        k = 8 * ((j + 5 * e) % (d // 8))
        u[e] = (j + e) % 7 + 1
        w[e, j, k + 2] = 32
        w[e, f + j, k], w[e, f + j, k + 1], w[e, f + j, k + 2] = 448, -448, u[e]
    one = dict(fill_value=127, dtype=torch.uint8, device=dev)
    u8 = dict(dtype=torch.uint8, device=dev)
    h, hs = torch.empty(R, f, **u8), torch.empty(R, S.scale_cols(f), **u8)
    y = torch.empty(R, d, dtype=torch.bfloat16, device=dev)
    abi.moe_grouped_ffn_fwd_fp8(_u8(S.to_e4m3(x), dev), torch.full((R, S.scale_cols(d)), **one), _i32(_offsets(counts), dev),
                                _u8(S.to_e4m3(w), dev), torch.full((E, -(-2 * f // 128), S.scale_cols(d)), **one),
                                torch.zeros(E, d, f, **u8), torch.full((E, -(-d // 128), S.scale_cols(f)), **one), None, h,
                                hs, y)
    torch.cuda.synchronize()
    assert np.array_equal(S.row_values(h.cpu().numpy(), hs.cpu().numpy()), 32 * np.repeat(u, counts, 0))
    assert (y == 0).all()
