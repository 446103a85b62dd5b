"""Plain 64-bit forms of the operators around the recurrence, written from their formulas, with the error that
32-bit arithmetic may make of them: each function returns its results and beside each a bound.

U = 2^-24 is half a step of float32.  A scan's error obeys the scan's own recurrence: step t adds to what its state carries
over the errors of a_t and of the two products and the sum, at most (8 + 12 |l_t|) U of the magnitudes M_t met there:
6 |l| U from the exponent's own rounding (|l| log2(e) half a step, times ln 2), 2 U for the exponential, the rest for the
products, the sums and the products of decays over segments.  A logit's e^g is known to (|g| + 2) U of itself, since the
exponent g log2(e) is rounded to U |g| log2(e) and ln 2 times that is its relative error; 1 - a = e^g / (1 + e^g) takes that
error over (a = 1 / (1 + e^g) only e^g of it): (|g| + 6) U with its sum, reciprocal and product.
"""
import numpy as np

U = 2.0 ** -24
ROUND = {"bf16": 2.0 ** -8, "f32": U}


def gates(g, logit):
    """Clamped log gates and the derivative by the input."""
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        l = -np.logaddexp(g, 0.0) if logit else g
        slope = -1.0 / (1.0 + np.exp(-g)) if logit else np.ones_like(g)
    return np.clip(l, -5.0, 0.0), np.where((l < -5) | (l > 0), 0.0, slope)


def rest_error(g, l, logit):
    """The relative error of 1 - a, and of the sigmoid that is a logit's slope."""
    return (np.abs(np.minimum(np.asarray(g, np.float64), 5.0)) + 6) * U if logit else (6 + 12 * np.abs(l)) * U


def spans(lengths=None, cu=None):
    cu = np.concatenate([[0], np.cumsum(lengths)]) if cu is None else cu
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def scan(x, g, h0, where, logit=False, mix=False):
    """x, g [total, D], h0 [N, D]; where: (first, end) of each sequence.  Returns y, h, u and their bounds."""
    x, h0 = np.asarray(x, np.float64), np.asarray(h0, np.float64)
    l, _ = gates(g, logit)
    a = np.exp(l)
    w = -np.expm1(l) if mix else np.ones_like(l)
    tw = rest_error(g, l, logit) * np.abs(w) if mix else np.zeros_like(l)
    y, before, ty, tb = (np.zeros_like(x) for _ in range(4))
    h, th = h0.copy(), np.zeros_like(h0)
    for n, (i, j) in enumerate(where):
        s, m, d = h0[n].copy(), np.abs(h0[n]), np.zeros(x.shape[1])
        for t in range(i, j):
            before[t], tb[t] = s, d
            s = a[t] * s + w[t] * x[t]
            m = a[t] * m + np.abs(w[t] * x[t])
            d = a[t] * d + (8 + 12 * np.abs(l[t])) * U * m + tw[t] * np.abs(x[t])
            y[t], ty[t] = s, d
        h[n], th[n] = s, d
    u = before - x if mix else before
    return (y, ty), (h, th), (u, tb + U * np.abs(u))


def scan_grad(x, g, h0, dy, dh, where, logit=False, mix=False, u=None):
    """Gradients; u: the factor of the gates' gradient to use (else the exact one), taken as given."""
    dy, dh = np.asarray(dy, np.float64), np.asarray(dh, np.float64)
    l, slope = gates(g, logit)
    a = np.exp(l)
    w = -np.expm1(l) if mix else np.ones_like(l)
    if u is None:
        _, _, (u, tu) = scan(x, g, h0, where, logit, mix)
    else:
        u, tu = np.asarray(u, np.float64), np.zeros(dy.shape)
    tr = rest_error(g, l, logit)
    dx, dg, tx, tg = (np.zeros_like(dy) for _ in range(4))
    dh0, t0 = dh.copy(), np.zeros_like(dh)
    for n, (i, j) in enumerate(where):
        e, m, d = dh[n].copy(), np.abs(dh[n]), np.zeros(dy.shape[1])
        for t in range(j - 1, i - 1, -1):
            r, rm = dy[t] + e, np.abs(dy[t]) + m
            rd = d + U * rm
            dx[t], tx[t] = w[t] * r, w[t] * rd + (2 * U + (tr[t] if mix else 0)) * np.abs(w[t] * r)
            e, m = a[t] * r, a[t] * rm
            d = a[t] * rd + (8 + 12 * np.abs(l[t])) * U * m
            dg[t] = u[t] * e * slope[t]
            tg[t] = np.abs(slope[t]) * (np.abs(u[t]) * d + np.abs(e) * tu[t] + tu[t] * d) + (4 * U + (tr[t] if logit else 0)) * np.abs(dg[t])
        dh0[n], t0[n] = e, d
    return (dx, tx), (dg, tg), (dh0, t0)


def turned(z, angle, interleaved, sign=1.0):
    """The first 2R channels of z [tokens, H, D] turned by angle [tokens, R]."""
    out, r = z.copy(), angle.shape[1]
    for i in range(r):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        c, s = np.cos(angle[:, i])[:, None], sign * np.sin(angle[:, i])[:, None]
        out[..., p], out[..., q] = z[..., p] * c - z[..., q] * s, z[..., q] * c + z[..., p] * s
    return out


def _pair_size(z, r, interleaved):
    """|z_p| + |z_q| of a channel's pair, its own magnitude where it is not turned."""
    out = np.abs(z)
    for i in range(r):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        out[..., p] = out[..., q] = np.abs(z[..., p]) + np.abs(z[..., q])
    return out


def qk_norm(x, w, angle, rms, eps, interleaved, dy=None):
    """x [tokens, H, D]; angle [tokens, R].  y, and with dy also dx and dw, each with its bound.

    A row's sum of squares is rounded at most 19 times (16 in a lane, three exchanges), its root halves that, and the
    root, the products with r and w and the rotation (a fraction of a turn to 2^-25, 3.2 U in radians, sine and cosine 2 U
    each) add 14: 32 U of the two channels of a pair.  A row's dot is a sum of D terms of which each is known to 32 U
    and rounded at most 20 times; the weights' sums are rounded at most once a term."""
    x = np.asarray(x, np.float64)
    D, r = x.shape[-1], angle.shape[1]
    s = 1.0 / D if rms else 1.0
    w = np.ones(D) if w is None else np.asarray(w, np.float64)
    total = s * (x * x).sum(-1, keepdims=True) + eps
    with np.errstate(divide="ignore"):
        rr = np.where(total > 0, 1.0 / np.sqrt(total), 0.0)
    n = x * rr
    z = n * w
    y, ty = turned(z, angle, interleaved), 32 * U * _pair_size(z, r, interleaved)
    if dy is None:
        return y, ty
    dy = np.asarray(dy, np.float64)
    dz, tz = turned(dy, angle, interleaved, -1.0), 10 * U * _pair_size(dy, r, interleaved)
    dn = dz * w
    tn = tz * np.abs(w) + 2 * U * np.abs(dn)
    dot = s * (dn * n).sum(-1, keepdims=True)
    tdot = s * (tn * np.abs(n) + 52 * U * np.abs(dn * n)).sum(-1, keepdims=True)
    dx = rr * (dn - n * dot)
    tx = rr * (tn + np.abs(n) * tdot + 60 * U * (np.abs(n * dot) + np.abs(dn)))
    dw = (dz * n).sum((0, 1))
    tw = (tz * np.abs(n) + (24 + dy.shape[0] * dy.shape[1]) * U * np.abs(dz * n)).sum((0, 1))
    return (y, ty), (dx, tx), (dw, tw)


# every finite e4m3 magnitude, by its code
E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def pack8(x):
    """Codes, scale bytes and values of x [rows, cols] (finite), from the format's definition: the nearest of all
    codes, the even one of two equally near."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    codes, values = np.zeros(x.shape, np.uint8), np.zeros_like(x)
    scales = np.zeros((rows, -(-cols // 32)), np.uint8)
    for b in range(scales.shape[1]):
        v = x[:, 32 * b:32 * b + 32]
        amax = np.abs(v).max(1)
        e = np.full(rows, -120)
        while (amax > 448.0 * 2.0 ** e).any():
            e = e + (amax > 448.0 * 2.0 ** e)
        z = np.minimum(np.abs(v), 1.875 * 2.0 ** 127) / 2.0 ** e[:, None]
        hi = np.searchsorted(E4M3, z).clip(0, 126)
        lo = np.maximum(hi - 1, 0)
        up, down = E4M3[hi] - z, z - E4M3[lo]
        code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        scales[:, b] = e + 127
        codes[:, 32 * b:32 * b + 32] = code | (np.signbit(v) * 128)
        values[:, 32 * b:32 * b + 32] = np.copysign(E4M3[code] * 2.0 ** e[:, None], v)
    return codes, scales, values


def unpack8(codes, scales):
    values = np.concatenate([E4M3, [np.nan]])[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    return values * 2.0 ** (np.repeat(scales.astype(np.float64), 32, -1)[..., :codes.shape[-1]] - 127)
