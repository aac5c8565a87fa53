"""CPU oracle of the score routing and of the block-scaled 8-bit products, in fp64.

Test infrastructure only.  Plain numpy; shares no code with the HIP library.
"""
import numpy as np


# ------------------------------------------------------------------ routing

def scores(logits, sigmoid):
    """[T, E] scores; a row of softmax logits that are all -inf scores 0."""
    x = np.asarray(logits, np.float64)
    with np.errstate(all="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-x))
        m = x.max(1, keepdims=True)
        e = np.exp(x - np.where(m == -np.inf, 0.0, m))
        s = e.sum(1, keepdims=True)
        return np.where(s == 0.0, 0.0, e / np.where(s == 0.0, 1.0, s))


def _order(v):
    """Indices by value descending, equal values by lower index, NaN last."""
    return np.argsort(-v, axis=-1, kind="stable")


def route_scored(logits, bias, k, sigmoid, n_group=1, topk_group=1, group_top=1, renorm=True,
                 scale=1.0):
    """(idx [T, k] int32, w [T, k] float64)."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    s = scores(x, sigmoid)
    c = x if bias is None else s + np.asarray(bias, np.float64)
    size = E // n_group
    idx = np.empty((T, k), np.int32)
    for t in range(T):
        cand = np.arange(E)
        if topk_group < n_group:
            val = np.empty(n_group)
            for g in range(n_group):
                src = c if (bias is not None or group_top == 1) else s
                v = src[t, g * size:(g + 1) * size]
                v = np.sort(np.where(np.isnan(v), -np.inf, v))[::-1]
                val[g] = v[:group_top].sum()
            kept = np.sort(_order(np.where(np.isnan(val), -np.inf, val))[:topk_group])
            cand = np.concatenate([np.arange(g * size, (g + 1) * size) for g in kept])
        idx[t] = cand[_order(c[t, cand])[:k]]
    return idx, weights(x, idx, sigmoid, renorm, scale)


def weights(logits, idx, sigmoid, renorm=True, scale=1.0):
    x = np.asarray(logits, np.float64)
    v = np.take_along_axis(x, idx, 1)
    with np.errstate(all="ignore"):
        if not renorm:
            return scale * np.take_along_axis(scores(x, sigmoid), idx, 1)
        # log s up to a common constant, so that no score underflows
        ls = -np.logaddexp(0.0, -v) if sigmoid else v
        m = ls.max(1, keepdims=True)
        e = np.exp(ls - np.where(m == -np.inf, 0.0, m))
        tot = e.sum(1, keepdims=True)
        return np.where(tot == 0.0, 0.0, scale * e / np.where(tot == 0.0, 1.0, tot))


def route_scored_bwd(logits, idx, g, sigmoid, renorm=True, scale=1.0):
    """d_logits [T, E] for gradients g [T, k] of the weights."""
    x = np.asarray(logits, np.float64)
    g = np.asarray(g, np.float64)
    w = weights(x, idx, sigmoid, renorm, scale)
    p = w / scale
    m = (p * g).sum(1, keepdims=True)
    d = w * (g - m if renorm else g)
    out = np.zeros(x.shape)
    if sigmoid:
        with np.errstate(all="ignore"):
            d = d / (1.0 + np.exp(np.take_along_axis(x, idx, 1)))
    elif not renorm:
        out -= scale * scores(x, False) * m
    np.put_along_axis(out, idx, np.take_along_axis(out, idx, 1) + d, 1)
    return out


# ------------------------------------------------------------------ 8-bit blocks

def e4m3_table():
    """The value of each byte, NaN for 0x7f and 0xff."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


_TABLE = e4m3_table()
_POS = _TABLE[:127]                      # 0 .. 448, ascending


def to_e4m3(v):
    """Nearest e4m3 byte of |v| <= 448 (ties to the even byte); NaN -> 0x7f."""
    v = np.asarray(v, np.float64)
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = a - _POS[lo], _POS[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    b = np.where(up, hi, lo) | np.where(np.signbit(v), 128, 0)
    return np.where(np.isnan(v), 127, b).astype(np.uint8)


def scale_cols(K):
    return (-(-K // 128) + 3) // 4 * 4


def block_exponent(amax):
    """Smallest s >= -127 with amax <= 448 * 2**s; 0 for amax 0 (exact)."""
    m, e = np.frexp(np.asarray(amax, np.float64))
    s = np.maximum(e - 9 + (m > 0.875), -127)
    return np.where(amax == 0, 0, s).astype(np.int64)


def quant_rows(x):
    """(bytes [R, K], scale bytes [R, cols]) of x [R, K]."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    q = np.empty((R, K), np.uint8)
    sc = np.full((R, scale_cols(K)), 127, np.uint8)
    for b in range(-(-K // 128)):
        v = x[:, b * 128:(b + 1) * 128]
        s = block_exponent(np.where(np.isfinite(v), np.abs(v), 0).max(1))
        q[:, b * 128:(b + 1) * 128] = to_e4m3(np.where(np.isfinite(v), v, np.nan) * 2.0 ** -s[:, None])
        sc[:, b] = s + 127
    return q, sc


def quant_weights(w):
    """(bytes [E, N, K], scale bytes [E, N/128, cols]) of w [E, N, K]."""
    w = np.asarray(w, np.float64)
    E, N, K = w.shape
    q = np.empty((E, N, K), np.uint8)
    sc = np.full((E, -(-N // 128), scale_cols(K)), 127, np.uint8)
    for e in range(E):
        for a in range(-(-N // 128)):
            for b in range(-(-K // 128)):
                i, j = slice(a * 128, (a + 1) * 128), slice(b * 128, (b + 1) * 128)
                v = w[e, i, j]
                s = block_exponent(np.where(np.isfinite(v), np.abs(v), 0).max())
                q[e, i, j] = to_e4m3(np.where(np.isfinite(v), v, np.nan) * 2.0 ** -s)
                sc[e, a, b] = s + 127
    return q, sc


def row_values(q, sc):
    K = q.shape[1]
    return _TABLE[q] * np.repeat(2.0 ** (sc.astype(np.float64) - 127), 128, 1)[:, :K]


def weight_values(q, sc):
    """[N, K] of one expert."""
    N, K = q.shape
    return _TABLE[q] * np.repeat(np.repeat(2.0 ** (sc.astype(np.float64) - 127), 128, 1)[:, :K], 128, 0)[:N]


def _group_max(v):
    """Largest magnitude of each 8 consecutive values of a row."""
    return np.abs(v).reshape(v.shape[0], v.shape[1] // 8, 8).max(2)


def product(a, offsets, b, row_scale=None):
    """(c, err) of value rows a [R, K] and value weights b [E][N, K]: the
    exact product, and how far one may be off that cuts the products of each 8
    consecutive k at 2^-13 of the largest and adds in fp32 from there."""
    R, K = a.shape
    N = b[0].shape[0]
    c, err = np.zeros((R, N)), np.zeros((R, N))
    for e in range(len(b)):
        i = slice(int(offsets[e]), int(offsets[e + 1]))
        c[i] = a[i] @ b[e].T
        err[i] = (7 * 2.0 ** -13) * (_group_max(a[i]) @ _group_max(b[e]).T) \
            + ((K + 2) * 2.0 ** -24) * (np.abs(a[i]) @ np.abs(b[e]).T)
    if row_scale is not None:
        w = np.asarray(row_scale, np.float64)[:, None]
        c, err = c * w, err * np.abs(w)
    return c, err


def swiglu(gu):
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
