"""Oracle of the residual norms, the weighted combine and AdamW (test
infrastructure only): numpy in 64 bits, with the size of the sums' addends
beside each value, from which the tests count roundings.
"""
import numpy as np

U32 = 2.0 ** -24


def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def residual_norm(x, y, w_post, w_pre, gate, scale, eps, store):
    """(out, n, 1/rms of y, of out, size): out is rounded by `store` before its norm; size: |scale x| + |gate p|."""
    rp = rn = n = None
    p = y
    if w_post is not None:
        rp = rstd(y, eps)
        p = y * rp * w_post
    if gate is not None:
        p = p * gate
    sx = 0.0 if x is None else scale * x
    out = sx + p
    if w_pre is not None:
        s = store(out)
        rn = rstd(s, eps)
        n = s * rn * w_pre
    return out, n, rp, rn, abs(sx) + abs(p)


def residual_norm_bwd(d_out, d_n, out, y, w_post, w_pre, gate, scale, rp, rn):
    """{name: (value, size)} of the gradients; size: what the absolute values of all addends come to."""
    d = (d_out if d_out is not None else d_n).shape[1]
    D = np.zeros_like(d_out if d_out is not None else d_n)
    aD = np.zeros_like(D)
    r = {}
    if d_out is not None:
        D, aD = D + d_out, aD + abs(d_out)
    if w_pre is not None:
        q = d_n * w_pre
        D = D + rn * q - out * rn ** 3 / d * (q * out).sum(1, keepdims=True)
        aD = aD + abs(rn * q) + abs(out) * rn ** 3 / d * abs(q * out).sum(1, keepdims=True)
        t = d_n * out * rn
        r["d_w_pre"] = (t.sum(0), abs(t).sum(0))
    r["d_x"] = (scale * D, abs(scale) * aD)
    g = 1.0 if gate is None else gate
    P, aP = g * D, abs(g) * aD
    if w_post is None:
        r["d_y"] = (P, aP)
        p = y
    else:
        h = P * w_post
        r["d_y"] = (rp * (h - y * rp ** 2 / d * (h * y).sum(1, keepdims=True)),
                    rp * (aP * abs(w_post) + abs(y) * rp ** 2 / d * (aP * abs(w_post * y)).sum(1, keepdims=True)))
        r["d_w_post"] = ((P * y * rp).sum(0), (aP * abs(y) * rp).sum(0))
        p = y * rp * w_post
    if gate is not None:
        t, at = D * p, aD * abs(p)
        axis = 0 if gate.ndim == 1 else 1 if gate.shape[1] == 1 and d > 1 else None
        r["d_gate"] = (t, at) if axis is None else (t.sum(axis), at.sum(axis))
    return r


def combine_weighted(y_perm, slot_to_row, w):
    """(y, size)"""
    T, k = w.shape
    y, size = np.zeros((T, y_perm.shape[1])), np.zeros((T, y_perm.shape[1]))
    for t in range(T):
        for j in range(k):
            r = slot_to_row[t * k + j]
            if r >= 0:
                y[t] += w[t, j] * y_perm[r]
                size[t] += abs(w[t, j] * y_perm[r])
    return y, size


def combine_weighted_bwd(dy, y_perm, slot_to_row, w):
    """{row: (dy_perm, d_row_scale, size of the sum's addends)} of the rows that a slot names."""
    T, k = w.shape
    rows = {}
    for t in range(T):
        for j in range(k):
            r = slot_to_row[t * k + j]
            if r >= 0:
                a = dy[t] * y_perm[r]
                rows[int(r)] = (w[t, j] * dy[t], a.sum(), abs(a).sum())
    return rows


# ---------------------------------------------------------------- AdamW

def _mix(a):
    a = np.asarray(a, np.uint64) & np.uint64(0xFFFFFFFF)
    a = a ^ (a >> np.uint64(16))
    a = (a * np.uint64(0x971CBEF1)) & np.uint64(0xFFFFFFFF)
    a = a ^ (a >> np.uint64(15))
    a = (a * np.uint64(0x6A695495)) & np.uint64(0xFFFFFFFF)
    return a ^ (a >> np.uint64(16))


def random_bits(seed, step, tensor, n, start=0):
    """(low half of r, high half of r, high half of r * C) of n elements from `start` on."""
    m32 = np.uint64(0xFFFFFFFF)
    e = np.arange(start, start + n, dtype=np.uint64)
    key = _mix(_mix(_mix(_mix(seed & 0xFFFFFFFF) ^ np.uint64(seed >> 32)) ^ np.uint64(step)) ^ np.uint64(tensor))
    r = _mix((key ^ (e >> np.uint64(32))) ^ (e & m32))
    r2 = (r * np.uint64(0x30E9132D)) & m32
    return r & np.uint64(0xFFFF), r >> np.uint64(16), r2 >> np.uint64(16)


def moments(m, v, g, b1, b2):
    """The new moments in 32 bits, every operation rounded by itself: bit for bit what is defined."""
    f = np.float32
    m, v, g = (np.asarray(t, f) for t in (m, v, g))
    with np.errstate(all="ignore"):
        return m * f(b1) + g * f(1.0 - b1), v * f(b2) + g * f(1.0 - b2) * g


def updated(p, m, v, lr, b1, b2, eps, decay, step):
    """(p after the step in 64 bits, size of the update)."""
    p, m, v = (np.asarray(t, np.float64) for t in (p, m, v))
    u = lr / (1 - b1 ** step) * m / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * decay) - u, abs(u)


def grid(fmt):
    """The non-negative finite values of an 8-bit type by code."""
    mant, bias, codes = (3, 7, 0x7F) if fmt == "e4m3" else (2, 15, 0x7C)
    c = np.arange(codes)
    e, f = c >> mant, c & ((1 << mant) - 1)
    return np.where(e == 0, f * 2.0 ** (1 - bias - mant), (1 + f * 2.0 ** -mant) * 2.0 ** (e - bias))


def exponents(x, largest):
    """s of each block of 128 of x (padded with zeros)."""
    a = np.abs(np.asarray(x, np.float64))
    a = np.where(np.isfinite(a), a, 0.0)
    a = np.pad(a, (0, -len(a) % 128)).reshape(-1, 128).max(1)
    s = np.zeros(len(a), np.int64)
    for i, v in enumerate(a):
        if v > 0:
            e = -126
            while v > largest * 2.0 ** e:
                e += 1
            s[i] = e
    return s


def code_of(x, s, r16, fmt):
    """8-bit codes of x [n] with s [blocks]: between the neighbours lo and hi of |x| / 2^s the upper one where the
    place between them plus r16 / 2^16 reaches 1."""
    values = grid(fmt)
    sc = np.repeat(2.0 ** np.asarray(s, np.float64), 128)[:len(x)]
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x)
    a = np.where(bad, 0.0, np.abs(x)) / sc
    # what lies below the bits that 16 random ones reach is cut off
    mant = 3 if fmt == "e4m3" else 2
    lo = np.searchsorted(values, a, side="right") - 1
    hi = np.minimum(lo + 1, len(values) - 1)
    gap = np.where(hi > lo, values[hi] - values[lo], 1.0)
    place = np.floor((a - values[lo]) / gap * 2.0 ** (23 - mant)) * 2.0 ** -(23 - mant)
    code = np.where(place + r16 * 2.0 ** -16 >= 1.0, hi, lo)
    if fmt == "e4m3":
        code = code | np.where(np.signbit(x), 0x80, 0)
    else:
        code = np.where((x > 0) & (code == 0), 1, code)
    return np.where(bad, 0x7F, code).astype(np.uint8)


def bf16_up_or_down(p, r16):
    """fp32 p rounded to bf16 by 16 random bits, as fp32."""
    p = np.asarray(p, np.float32)
    b = p.view(np.uint32).astype(np.uint64)
    up = ((b + r16) & np.uint64(0xFFFF0000)).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(p), up, p)
