"""The routing by scores and the block-scaled fp8 expert products, as they are measured.

Operators (the framework's calls, where ``own`` is true):

* ``route``   moe_route_scored, and moe_route_scored_bwd in a training step
* ``quant``   moe_quant_rows_fp8, moe_quant_weights_fp8
* ``product`` moe_quant_rows_fp8 + moe_grouped_gemm_fp8 (the gradient of the
  experts' input rows, through transposed weight blocks)
* ``ffn``     moe_quant_rows_fp8 + moe_grouped_ffn_fwd_fp8

The 8-bit format: e4m3 values, one power-of-two scale for each block of 128
along a row (weights: 128 x 128), stored as its exponent + 127 in a byte;
a scale row is padded to a multiple of four bytes (127 there).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding batch's routing: launch latency
        dict(name="route decode", op="route", train=False, T=16, E=256, k=8, score="sigmoid", bias=True,
             groups=8, keep=4, gtop=2, renorm=True, scale=2.5),
        # the routing of a large prompt batch
        dict(name="route prompt", op="route", train=False, T=32768, E=256, k=8, score="sigmoid", bias=True,
             groups=8, keep=4, gtop=2, renorm=True, scale=2.5),
        # a training step of a softmax router whose weights are not renormalised: a dense gradient
        dict(name="route train softmax", op="route", train=True, T=16384, E=128, k=8, score="softmax", bias=False,
             groups=1, keep=1, gtop=1, renorm=False, scale=1.0),
        # a training step with odd sizes and groups that are no power of two
        dict(name="route train sigmoid odd", op="route", train=True, T=5003, E=160, k=6, score="sigmoid", bias=True,
             groups=8, keep=3, gtop=1, renorm=True, scale=1.0),
        # activations of a prompt batch, quantised by rows
        dict(name="quant rows", op="quant", what="rows", R=32768, K=2048, dtype="bf16"),
        # all experts' gate/up weights quantised once after an update, with the copy that the input gradient reads
        dict(name="quant weights", op="quant", what="weights", E=32, N=5760, K=2880, dtype="bf16"),
        # the gradient of the rows at the gate/up product, ragged experts and sizes that end inside a block
        dict(name="product odd", op="product", E=13, R=5003, N=720, K=1136, skew=True, weighted=False),
        # the same at the benchmark layer
        dict(name="product layer", op="product", E=32, R=16384, N=2880, K=5760, skew=False, weighted=False),
        # one token: the weights of the chosen experts are all there is to read
        dict(name="ffn one token", op="ffn", T=1, d=2880, E=32, k=4, f=2880),
        # a decoding batch: every expert's weights, a few rows each
        dict(name="ffn decode 64", op="ffn", T=64, d=2880, E=32, k=4, f=2880),
        # the benchmark layer
        dict(name="ffn layer", op="ffn", T=4096, d=2880, E=32, k=4, f=2880),
        # the larger layer: many narrow experts
        dict(name="ffn many experts", op="ffn", T=32768, d=2048, E=128, k=8, f=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "quant", "product", "ffn", "ffn"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 10])
        E = groups * rng.randint(4, 40)
        k = rng.randint(1, min(10, E))
        size = E // groups
        keep = rng.randint(min(groups, -(-k // size)), groups)
        train = rng.random() < 0.5
        T = _log(rng, 1, 32768 if not train else 16384)
        return dict(op=op, train=train, T=T, E=E, k=k, score=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, gtop=rng.choice([1, 2]),
                    renorm=k > 1 and rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
    if op == "quant":
        if rng.random() < 0.5:
            return dict(op=op, what="rows", R=_log(rng, 1, 30000), K=16 * _log(rng, 2, 256),
                        dtype=rng.choice(["bf16", "fp32"]))
        return dict(op=op, what="weights", E=rng.randint(1, 16), N=16 * _log(rng, 2, 300),
                    K=16 * _log(rng, 2, 200), dtype=rng.choice(["bf16", "fp32"]))
    if op == "product":
        return dict(op=op, E=rng.randint(1, 64), R=_log(rng, 1, 12000), N=16 * _log(rng, 2, 180),
                    K=16 * _log(rng, 2, 240), skew=rng.random() < 0.5, weighted=rng.random() < 0.5)
    E = rng.choice([4, 8, 16, 32, 64])
    return dict(op=op, T=_log(rng, 1, 6000), d=16 * _log(rng, 8, 180), E=E, k=rng.randint(1, min(8, E)),
                f=16 * _log(rng, 8, 180))


# ---------------------------------------------------------------------- inputs

def _cols(K):
    """Bytes of one row of scales."""
    return (-(-K // 128) + 3) // 4 * 4


def _pow2(s):
    """2.0 ** s for integer tensors s, exact in 32 bits (-126 <= s <= 127)."""
    return ((s.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponents(amax):
    """The smallest s >= -127 with amax <= 448 * 2**s; 0 where amax is 0."""
    m, e = torch.frexp(amax)                      # amax = m * 2**e, 0.5 <= m < 1; 448 = 0.875 * 2**9
    s = torch.clamp(e.to(torch.int32) - 9 + (m > 0.875), min=-127)
    return torch.where(amax == 0, torch.zeros_like(s), s)


def _pad(t, rows, cols):
    return torch.nn.functional.pad(t, (0, cols - t.shape[-1], 0, rows - t.shape[-2]))


def _plain_rows(x):
    """(q [R, K], scale bytes [R, cols]) of x [R, K]."""
    R, K = x.shape
    nb = -(-K // 128)
    v = _pad(x.float(), R, nb * 128).view(R, nb, 128)
    s = _exponents(v.abs().amax(-1))
    q = (v * _pow2(-s)[..., None]).view(R, nb * 128)[:, :K].to(FP8)
    out = torch.full((R, _cols(K)), 127, dtype=torch.uint8, device=x.device)
    out[:, :nb] = (s + 127).to(torch.uint8)
    return q.contiguous(), out


def _plain_weights(w):
    """(q [E, N, K], scale bytes [E, N/128, cols]) of w [E, N, K]."""
    E, N, K = w.shape
    mb, nb = -(-N // 128), -(-K // 128)
    v = _pad(w.float(), mb * 128, nb * 128).view(E, mb, 128, nb, 128)
    s = _exponents(v.abs().amax((2, 4)))
    q = (v * _pow2(-s)[:, :, None, :, None]).view(E, mb * 128, nb * 128)[:, :N, :K].to(FP8)
    out = torch.full((E, mb, _cols(K)), 127, dtype=torch.uint8, device=w.device)
    out[:, :, :nb] = (s + 127).to(torch.uint8)
    return q.contiguous(), out


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _weights8(g, E, N, K):
    """Seeded expert weights [E, N, K] of spread 1/sqrt(K), in 8 bits; one expert at a time, to bound the memory."""
    parts = [_plain_weights(_randn(g, 1, N, K, scale=K ** -0.5, dtype=torch.bfloat16)) for _ in range(E)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        s = {"case": case, "logits": _randn(g, T, E, scale=1.5),
             "bias": _randn(g, E, scale=0.1) if case["bias"] else None,
             "idx": torch.empty(T, k, dtype=torch.int32, device=DEV),
             "w": torch.empty(T, k, device=DEV)}
        if case["train"]:
            s["d_rows"] = _randn(g, T * k)
            s["slot_to_row"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
            s["d_w"] = torch.empty(T, k, device=DEV)
            s["d_logits"] = torch.empty(T, E, device=DEV)
        return s
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}
    if op == "quant":
        if case["what"] == "rows":
            R, K = case["R"], case["K"]
            # activations: a spread that differs from row to row, a few large columns
            x = _randn(g, R, K) * torch.exp(_randn(g, R, 1)) * (1 + 20 * (torch.rand(K, generator=g, device=DEV) < 0.01))
            return {"case": case, "x": x.to(dt[case["dtype"]]), "q": torch.empty(R, K, dtype=FP8, device=DEV),
                    "scale": torch.empty(R, _cols(K), dtype=torch.uint8, device=DEV)}
        E, N, K = case["E"], case["N"], case["K"]
        w = torch.empty(E, N, K, dtype=dt[case["dtype"]], device=DEV)
        w.normal_(std=K ** -0.5, generator=g)
        u8 = dict(dtype=torch.uint8, device=DEV)
        return {"case": case, "w": w, "q": torch.empty(E, N, K, dtype=FP8, device=DEV),
                "scale": torch.empty(E, -(-N // 128), _cols(K), **u8),
                "qt": torch.empty(E, K, N, dtype=FP8, device=DEV),
                "scale_t": torch.empty(E, -(-K // 128), _cols(N), **u8)}
    if op == "product":
        E, R, N, K = case["E"], case["R"], case["N"], case["K"]
        p = torch.ones(E, device=DEV)
        if case["skew"]:                              # a hot expert, and one without rows
            p = 1.0 / torch.arange(1, E + 1, device=DEV, dtype=torch.float32)
            p[E // 2] = 0.0 if E > 1 else 1.0
        expert = torch.multinomial(p, R, replacement=True, generator=g)
        counts = torch.bincount(expert, minlength=E).cpu()
        b, bs = _weights8(g, E, N, K)
        return {"case": case, "a": _randn(g, R, K, scale=0.05, dtype=torch.bfloat16), "b": b, "b_scale": bs,
                "counts": counts.tolist(),
                "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32).to(DEV),
                "w": torch.rand(R, generator=g, device=DEV) if case["weighted"] else None,
                "q": torch.empty(R, K, dtype=FP8, device=DEV),
                "scale": torch.empty(R, _cols(K), dtype=torch.uint8, device=DEV),
                "c": torch.empty(R, N, dtype=torch.bfloat16, device=DEV)}
    T, d, E, k, f = (case[n] for n in ("T", "d", "E", "k", "f"))
    R = T * k
    expert = torch.rand(T, E, generator=g, device=DEV).topk(k, 1).indices.reshape(-1)   # slot -> expert
    order = torch.sort(expert, stable=True).indices
    counts = torch.bincount(expert, minlength=E).cpu()
    w_gu, w_gu_s = _weights8(g, E, 2 * f, d)
    w_dn, w_dn_s = _weights8(g, E, d, f)
    return {"case": case, "x": _randn(g, T, d, dtype=torch.bfloat16), "counts": counts.tolist(),
            "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32).to(DEV),
            "row_to_slot": order.to(torch.int32), "w": torch.rand(R, generator=g, device=DEV),
            "w_gu": w_gu, "w_gu_scale": w_gu_s, "w_down": w_dn, "w_down_scale": w_dn_s,
            "q": torch.empty(T, d, dtype=FP8, device=DEV),
            "scale": torch.empty(T, _cols(d), dtype=torch.uint8, device=DEV),
            "h": torch.empty(R, f, dtype=FP8, device=DEV),
            "h_scale": torch.empty(R, _cols(f), dtype=torch.uint8, device=DEV),
            "y": torch.empty(R, d, dtype=torch.bfloat16, device=DEV)}


# ---------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "quant": _own_quant, "product": _own_product, "ffn": _own_ffn}[op](state)
    return {"route": _route, "quant": _quant, "product": _product, "ffn": _ffn}[op](state)


def _own_route(s):
    from mixture_experts_layer_03_amd import abi
    c = s["case"]
    score = abi.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else abi.MOE_SCORE_SOFTMAX
    abi.moe_route_scored(s["logits"], s["bias"], c["k"], s["idx"], s["w"], score=score, n_group=c["groups"],
                         topk_group=c["keep"], group_top=c["gtop"], renorm=c["renorm"], scale=c["scale"])
    if not c["train"]:
        return {"idx": s["idx"], "w": s["w"]}
    abi.moe_route_scored_bwd(s["logits"], s["idx"], s["w"], s["d_rows"], s["slot_to_row"], s["d_w"], s["d_logits"],
                             score=score, renorm=c["renorm"], scale=c["scale"])
    return {"idx": s["idx"], "w": s["w"], "d_w": s["d_w"], "d_logits": s["d_logits"]}


def _own_quant(s):
    from mixture_experts_layer_03_amd import abi
    if s["case"]["what"] == "rows":
        abi.moe_quant_rows_fp8(s["x"], s["q"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    abi.moe_quant_weights_fp8(s["w"], s["q"], s["scale"], s["qt"], s["scale_t"])
    return {"q": s["q"], "scale": s["scale"], "qt": s["qt"], "scale_t": s["scale_t"]}


def _own_product(s):
    from mixture_experts_layer_03_amd import abi
    abi.moe_quant_rows_fp8(s["a"], s["q"], s["scale"])
    abi.moe_grouped_gemm_fp8(s["q"], s["scale"], s["offsets"], s["b"], s["b_scale"], s["w"], s["c"])
    return {"c": s["c"]}


def _own_ffn(s):
    from mixture_experts_layer_03_amd import abi
    abi.moe_quant_rows_fp8(s["x"], s["q"], s["scale"])
    abi.moe_grouped_ffn_fwd_fp8(s["q"], s["scale"], s["offsets"], s["w_gu"], s["w_gu_scale"], s["w_down"],
                                s["w_down_scale"], s["w"], s["h"], s["h_scale"], s["y"],
                                row_to_slot=s["row_to_slot"], k=s["case"]["k"])
    return {"y": s["y"]}


# ---------------------------------------------------------------------- the plain forms

def _scores(x, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _ranked(v, n):
    """Indices of the n largest along the last axis, equal values by lower index."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :n]


def _route(s):
    c, x, bias = s["case"], s["logits"], s["bias"]
    T, E = x.shape
    k, G = c["k"], c["groups"]
    # decisions in 64 bits: scores next to each other at a border differ by less than 32 bits hold
    x64 = x.double()
    score = _scores(x64, c["score"])
    rank = x64 if bias is None else score + bias.double()
    if c["keep"] < G:
        per = (rank if c["gtop"] == 1 else score if bias is None else rank).view(T, G, E // G)
        gs = torch.sort(per, dim=-1, descending=True).values[..., :c["gtop"]].sum(-1)
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, _ranked(gs, c["keep"]), True)
        rank = torch.where(kept[:, :, None].expand(T, G, E // G).reshape(T, E), rank, -math.inf)
    idx = _ranked(rank, k)
    p = _scores(x, c["score"])
    sel = p.gather(1, idx)
    w = (sel / sel.sum(1, keepdim=True) if c["renorm"] else sel) * c["scale"]
    if not c["train"]:
        return {"idx": idx.to(torch.int32), "w": w}
    g = s["d_rows"][s["slot_to_row"].long()].view(T, k)
    dsel = g * c["scale"]                                       # of the selected scores
    if c["renorm"]:
        tot = sel.sum(1, keepdim=True)
        dsel = (dsel - (dsel * sel / tot).sum(1, keepdim=True)) / tot
    ds = torch.zeros_like(p).scatter_(1, idx, dsel)
    if c["score"] == "sigmoid":
        dl = ds * p * (1.0 / (1.0 + torch.exp(x)))
    else:
        dl = p * (ds - (ds * p).sum(1, keepdim=True))
    return {"idx": idx.to(torch.int32), "w": w, "d_w": g, "d_logits": dl}


def _quant(s):
    if s["case"]["what"] == "rows":
        q, scale = _plain_rows(s["x"])
        return {"q": q, "scale": scale}
    q, scale = _plain_weights(s["w"])
    qt, scale_t = _plain_weights(s["w"].transpose(1, 2))
    return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}


def _values(q, scale):
    """What 8-bit rows [R, K] with their scales stand for, in 32 bits."""
    K = q.shape[1]
    return q.float() * _pow2(scale.int() - 127).repeat_interleave(128, 1)[:, :K]


def _weight(q, scale):
    """What an expert's 8-bit weights [N, K] stand for."""
    N, K = q.shape
    return q.float() * _pow2(scale.int() - 127).repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[:N]


def _product(s):
    a = _values(*_plain_rows(s["a"]))
    parts = a.split(s["counts"])
    c = torch.cat([r @ _weight(q, m).t() for r, q, m in zip(parts, s["b"], s["b_scale"]) if len(r)])
    return {"c": (c if s["w"] is None else c * s["w"][:, None]).to(torch.bfloat16)}


def _ffn(s):
    k, f = s["case"]["k"], s["case"]["f"]
    x = _values(*_plain_rows(s["x"]))[s["row_to_slot"].long() // k]
    gu = torch.cat([r @ _weight(q, m).t()
                    for r, q, m in zip(x.split(s["counts"]), s["w_gu"], s["w_gu_scale"]) if len(r)])
    g, u = gu[:, :f], gu[:, f:]
    h = _values(*_plain_rows(g / (1.0 + torch.exp(-g)) * u))
    y = torch.cat([r @ _weight(q, m).t()
                   for r, q, m in zip(h.split(s["counts"]), s["w_down"], s["w_down_scale"]) if len(r)])
    return {"y": (y * s["w"][:, None]).to(torch.bfloat16)}


# ---------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b, fl = 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), 10 * T * E
        if case["train"]:
            b, fl = b + 4 * T * E + 12 * T * k, fl + 4 * T * E
        return {"bytes": b, "flops": fl}
    if op == "quant":
        size = 2 if case["dtype"] == "bf16" else 4
        if case["what"] == "rows":
            n = case["R"] * case["K"]
            return {"bytes": n * (size + 1) + n // 128, "flops": 2 * n}
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": n * (size + 2), "flops": 2 * n}
    if op == "product":
        E, R, N, K = case["E"], case["R"], case["N"], case["K"]
        return {"bytes": 2 * R * K + min(E, R) * N * K + 2 * R * N, "flops": 2 * R * N * K}
    T, d, E, k, f = (case[n] for n in ("T", "d", "E", "k", "f"))
    touched = E * (1 - (1 - k / E) ** T)                          # experts that some token chose, on average
    return {"bytes": 2 * T * d + touched * 3 * d * f + 2 * T * k * d, "flops": 6 * T * k * d * f}


# ---------------------------------------------------------------------- the definition in 64 bits

def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _exact_route(s):
    c = s["case"]
    x, b = _np(s["logits"]), _np(s["bias"])
    T, E = x.shape
    k, G, keep = c["k"], c["groups"], c["keep"]
    if c["score"] == "sigmoid":
        log_s = -np.logaddexp(0.0, -x)
        rest = np.exp(-np.logaddexp(0.0, x))                      # 1 - s
    else:
        top = x.max(1, keepdims=True)
        log_s = x - top - np.log(np.exp(x - top).sum(1, keepdims=True))
        rest = None
    sc = np.exp(log_s)
    choice = x if b is None else sc + b
    if keep < G:
        per = (choice if c["gtop"] == 1 else sc if b is None else choice).reshape(T, G, E // G)
        gs = np.partition(per, E // G - c["gtop"], axis=2)[:, :, E // G - c["gtop"]:].sum(2)
        order = np.lexsort((np.broadcast_to(np.arange(G), gs.shape), -gs), axis=1)
        ok = np.zeros((T, G), bool)
        np.put_along_axis(ok, order[:, :keep], True, 1)
        choice = np.where(np.repeat(ok, E // G, 1), choice, -np.inf)
    idx = np.lexsort((np.broadcast_to(np.arange(E), choice.shape), -choice), axis=1)[:, :k]
    ls = np.take_along_axis(log_s, idx, 1)
    if c["renorm"]:
        e = np.exp(ls - ls.max(1, keepdims=True))
        p = e / e.sum(1, keepdims=True)
    else:
        p = np.exp(ls)
    w = p * c["scale"]
    out = {"idx": idx.astype(np.int32), "w": w}
    if not c["train"]:
        return out
    g = _np(s["d_rows"])[s["slot_to_row"].cpu().numpy()].reshape(T, k)
    mean = (g * p).sum(1, keepdims=True)
    dl = np.zeros((T, E))
    if c["score"] == "softmax" and not c["renorm"]:
        dl = -sc * mean * c["scale"]
        np.put_along_axis(dl, idx, np.take_along_axis(dl, idx, 1) + w * g, 1)
    else:
        t = w * (g - mean if c["renorm"] else g)
        if rest is not None:
            t = t * np.take_along_axis(rest, idx, 1)
        np.put_along_axis(dl, idx, t, 1)
    out.update(d_w=g, d_logits=dl)
    return out


def _round_e4m3(v):
    """The nearest e4m3 value, ties to even, of |v| <= 448 in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_blocks(v, dims):
    """(values rounded, exponents) of blocks of v whose axes `dims` share a scale."""
    amax = v.abs().amax(dims, keepdim=True)
    s = torch.ceil(torch.log2(amax / 448))
    s = torch.where(torch.exp2(s - 1) * 448 >= amax, s - 1, torch.where(torch.exp2(s) * 448 < amax, s + 1, s))
    s = torch.where(amax > 0, s.clamp(min=-127), torch.zeros_like(s))
    return _round_e4m3(v * torch.exp2(-s)), s


def _exact_rows(x):
    R, K = x.shape
    nb = -(-K // 128)
    v = torch.zeros(R, nb * 128, dtype=torch.float64, device=x.device)
    v[:, :K] = x
    q, s = _exact_blocks(v.view(R, nb, 128), 2)
    return q, s


def _exact_row_values(x):
    q, s = _exact_rows(x)
    return (q * torch.exp2(s)).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _exact_weight(q, scale):
    """[N, K] in 64 bits from the stored bytes."""
    n = torch.arange(q.shape[0], device=q.device) // 128
    kk = torch.arange(q.shape[1], device=q.device) // 128
    return q.double() * torch.exp2(scale.double() - 127)[n][:, kk]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "quant":
        if case["what"] == "rows":
            q, _ = _exact_rows(s["x"].double())
            return {"q": q.reshape(case["R"], -1)[:, :case["K"]], "scale": None}
        E, N, K = case["E"], case["N"], case["K"]
        mb, nb = -(-N // 128), -(-K // 128)
        out = torch.empty(E, N, K, dtype=torch.float64, device=DEV)
        for e in range(E):
            v = torch.zeros(mb * 128, nb * 128, dtype=torch.float64, device=DEV)
            v[:N, :K] = s["w"][e]
            q, _ = _exact_blocks(v.view(mb, 128, nb, 128), (1, 3))
            out[e] = q.reshape(mb * 128, nb * 128)[:N, :K]
        return {"q": out, "scale": None, "qt": out.transpose(1, 2).contiguous(), "scale_t": None}
    if op == "product":
        a = _exact_row_values(s["a"].double())
        c = torch.empty(case["R"], case["N"], dtype=torch.float64, device=DEV)
        at = 0
        for e, n in enumerate(s["counts"]):
            c[at:at + n] = a[at:at + n] @ _exact_weight(s["b"][e], s["b_scale"][e]).t()
            at += n
        return {"c": c if s["w"] is None else c * s["w"].double()[:, None]}
    f = case["f"]
    x = _exact_row_values(s["x"].double())
    token = s["row_to_slot"].long() // case["k"]
    y = torch.empty(case["T"] * case["k"], case["d"], dtype=torch.float64, device=DEV)
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            gu = x[token[at:at + n]] @ _exact_weight(s["w_gu"][e], s["w_gu_scale"][e]).t()
            h = _exact_row_values(gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:])
            y[at:at + n] = h @ _exact_weight(s["w_down"][e], s["w_down_scale"][e]).t()
        at += n
    return {"y": y * s["w"].double()[:, None]}
