"""Feature-row operators in float64 (oracle side; test infrastructure only): group norm with an
activation, its first and second derivatives, and counter-based dropout of whole channels.

Rows [N, dim] hold irrep blocks in the mul_ir layout.  Per block the channels are cut into groups;
for a segment of rows and a group of n values
    mu = mean(x) for even scalars (0e), 0 for other irreps;  r = (mean((x - mu)^2) + eps)^(-1/2)
    z = (x - mu) r,  t = weight z + bias (bias: 0e only),  y = m a(t)
with m the dropout factor and a the activation (SiLU on 0e channels, or none).  A mean, a bias or a
pointwise function of a component that rotates (or changes sign under inversion) would break
equivariance, so the other irreps only get the scale.

The derivatives are written segment by segment; the second one is the derivative of <grad_y, ydot>, ydot
the change of y along (u_x, u_weight, u_bias), because the first derivative's pairing with u is that number.

Each function also returns, where ``scale=True``, the sum of the absolute values of the terms that
were added for every output: the size on which rounding errors act.
"""

import numpy as np

from .irreps import parse_irreps

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox4x32(counter, key):
    """Four 32-bit words of Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3"),
    in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = M0 * c[0], M1 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + W0) & 0xFFFFFFFF, (k[1] + W1) & 0xFFFFFFFF]
    return c


def dropout_keep(irreps, n_rows, p, seed, offset=0, row0=0):
    """Per block a [n_rows, channels] array of the channels that stay."""
    thr = int(np.floor(p * 2.0 ** 32))
    key = (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)
    out = []
    for b, ir in enumerate(parse_irreps(irreps)):
        keep = np.zeros((n_rows, ir.mul), dtype=bool)
        for i in range(n_rows):
            for q in range(0, ir.mul, 4):
                words = philox4x32((q // 4, row0 + i, b, offset), key)
                for j, w in enumerate(words[:ir.mul - q]):
                    keep[i, q + j] = w >= thr
        out.append(keep)
    return out


def dropout_factor(irreps, n_rows, p, seed, offset=0, row0=0):
    """[n_rows, dim] dropout factors: 1 / (1 - p) or 0."""
    blocks = parse_irreps(irreps)
    keep = dropout_keep(irreps, n_rows, p, seed, offset, row0)
    return np.concatenate([np.repeat(k, 2 * ir.l + 1, axis=1) for ir, k in zip(blocks, keep)], axis=1) / (1.0 - p)


def _silu(t):
    s = 1.0 / (1.0 + np.exp(-t))
    return t * s, s * (1.0 + t * (1.0 - s)), s * (1.0 - s) * (2.0 + t * (1.0 - 2.0 * s))


class _Group:
    """One (segment, group): slices of the rows, columns, weights and biases."""

    def __init__(self, rows, cols, chan, bias, d):
        self.rows, self.cols, self.chan, self.bias, self.d = rows, cols, chan, bias, d
        self.scalar = bias is not None

    def take(self, t):
        return np.asarray(t, dtype=np.float64)[self.rows, self.cols]

    def spread(self, v, which):
        """Per-channel values over the group's columns."""
        if v is None or which is None:
            return 0.0
        return np.repeat(np.asarray(v, dtype=np.float64)[which], self.d)[None, :]

    def fold(self, t):
        """Sums over rows and components, per channel."""
        return t.reshape(t.shape[0], -1, self.d).sum(axis=(0, 2))

    def center(self, t):
        return t - t.mean() if self.scalar else t


def _groups(irreps, groups, row_ptr):
    for s, e in zip(row_ptr[:-1], row_ptr[1:]):
        if e <= s:
            continue
        col = chan = sc = 0
        for ir in parse_irreps(irreps):
            per, d = ir.mul // groups, 2 * ir.l + 1
            scalar = ir.l == 0 and ir.p == 1
            for g in range(groups):
                yield _Group(slice(s, e), slice(col + g * per * d, col + (g + 1) * per * d),
                             slice(chan + g * per, chan + (g + 1) * per),
                             slice(sc + g * per, sc + (g + 1) * per) if scalar else None, d)
            col += ir.dim
            chan += ir.mul
            sc += ir.mul if scalar else 0


def _sizes(irreps):
    blocks = parse_irreps(irreps)
    return sum(ir.mul for ir in blocks), sum(ir.mul for ir in blocks if ir.l == 0 and ir.p == 1)


def _common(q, x, weight, bias, eps, act, factor):
    """z, r, weights, a(t), a'(t), a''(t), dropout factor of one (segment, group)."""
    xg = q.take(x)
    mu = xg.mean() if q.scalar else 0.0
    r = 1.0 / np.sqrt(np.mean((xg - mu) ** 2) + eps)
    z = (xg - mu) * r
    w = q.spread(weight, q.chan) if weight is not None else 1.0
    t = w * z + q.spread(bias, q.bias)
    if act == "silu" and q.scalar:
        a0, a1, a2 = _silu(t)
    else:
        a0, a1, a2 = t, np.ones_like(t), np.zeros_like(t)
    m = 1.0 if factor is None else q.take(factor)
    return z, r, mu, w, a0, a1, a2, m


def group_norm(irreps, groups, row_ptr, x, weight=None, bias=None, eps=1e-5, act=None, factor=None, scale=False):
    """y [N, dim]; rows outside the segments are zero."""
    y, size = np.zeros(np.shape(x)), np.zeros(np.shape(x))
    for q in _groups(irreps, groups, row_ptr):
        z, r, mu, w, a0, _, _, m = _common(q, x, weight, bias, eps, act, factor)
        y[q.rows, q.cols] = m * a0
        size[q.rows, q.cols] = m * (np.abs(w) * (np.abs(z) + 2.0) + np.abs(q.spread(bias, q.bias)))
    return (y, size) if scale else y


def group_norm_backward(irreps, groups, row_ptr, x, grad_y, weight=None, bias=None, eps=1e-5, act=None, factor=None,
                        scale=False):
    """(grad_x, grad_weight, grad_bias)."""
    n_ch, n_sc = _sizes(irreps)
    gx, gw, gb = np.zeros(np.shape(x)), np.zeros(n_ch), np.zeros(n_sc)
    sx, sw, sb = np.zeros(np.shape(x)), np.zeros(n_ch), np.zeros(n_sc)
    for q in _groups(irreps, groups, row_ptr):
        z, r, _, w, _, a1, _, m = _common(q, x, weight, bias, eps, act, factor)
        gm = m * q.take(grad_y)
        h = gm * a1
        c = w * h
        gx[q.rows, q.cols] = r * (q.center(c) - z * np.mean(c * z))
        gw[q.chan] += q.fold(h * z)
        if q.scalar:
            gb[q.bias] += q.fold(h)
        ac = np.abs(w * gm) * (1.0 + np.abs(w) * (np.abs(z) + 2.0))  # a' moves with t: |a''| <= 1/2
        sx[q.rows, q.cols] = r * (ac + ac.mean() + (np.abs(z) + 1.0) * np.mean(ac * (np.abs(z) + 1.0)))
        ah = np.abs(gm) * (1.0 + np.abs(w) * (np.abs(z) + 2.0))
        sw[q.chan] += q.fold(ah * (np.abs(z) + 1.0))
        if q.scalar:
            sb[q.bias] += q.fold(ah)
    return (gx, gw, gb, sx, sw, sb) if scale else (gx, gw, gb)


def group_norm_double_backward(irreps, groups, row_ptr, x, grad_y, weight=None, bias=None, u_x=None, u_weight=None,
                               u_bias=None, eps=1e-5, act=None, factor=None, scale=False):
    """(d_grad_y, d_x, d_weight, d_bias) of <u_x, grad_x> + <u_weight, grad_weight> + <u_bias, grad_bias>."""
    n_ch, n_sc = _sizes(irreps)
    out = [np.zeros(np.shape(x)), np.zeros(np.shape(x)), np.zeros(n_ch), np.zeros(n_sc)]
    size = [np.zeros_like(t) for t in out]
    for q in _groups(irreps, groups, row_ptr):
        z, r, _, w, _, a1, a2, m = _common(q, x, weight, bias, eps, act, factor)
        g = m * q.take(grad_y)
        ux = np.zeros_like(z) if u_x is None else q.take(u_x)
        uw, ub = q.spread(u_weight, q.chan), q.spread(u_bias, q.bias)
        m2 = np.mean(z * ux)
        zd = r * (q.center(ux) - z * m2)
        td = w * zd + uw * z + ub
        h = g * a1
        c = w * h
        cz = np.mean(c * z)
        k = g * a2 * td
        C = w * k + uw * h - r * m2 * c - r * cz * ux
        out[0][q.rows, q.cols] = m * a1 * td
        out[1][q.rows, q.cols] = r * (q.center(C) - z * np.mean(z * C)) - r * z * np.mean(c * zd)
        out[2][q.chan] += q.fold(k * z + h * zd)
        if q.scalar:
            out[3][q.bias] += q.fold(k)
        # the same with absolute values; the derivatives of the activation are bounded by 1.1 and move
        # with t by at most 1/2 (a') and 1 (a'') a unit
        az, aw, au = np.abs(z) + 1.0, np.abs(w), np.abs(ux)
        move = 1.1 + aw * (az + 1.0)
        azd = r * (au + au.mean() + az * np.mean(az * au))
        atd = aw * azd + np.abs(uw) * az + np.abs(ub)
        ag = np.abs(g) * move
        ac = aw * ag
        ak = ag * atd if act == "silu" and q.scalar else 0.0 * atd
        aC = aw * ak + np.abs(uw) * ag + r * np.mean(az * au) * ac + r * np.mean(ac * az) * au
        size[0][q.rows, q.cols] = m * move * atd
        size[1][q.rows, q.cols] = r * (aC + aC.mean() + az * np.mean(az * aC)) + r * az * np.mean(ac * azd)
        size[2][q.chan] += q.fold(ak * az + ag * azd)
        if q.scalar:
            size[3][q.bias] += q.fold(ak)
    return tuple(out) + tuple(size) if scale else tuple(out)
