"""Serving in 8-bit floating point, restated in float64 (oracle; test use only).

* e4m3 codes with a power-of-two scale per block, and the linear with a scale per 128 input channels,
* rotary positions on part of a head with scaled frequencies,
* a paged cache of keys and values, appended to and read,
* attention over such a cache.

Inputs are float64 arrays holding bf16 (or coded) values exactly; codes are handled as the values they
stand for. Functions that feed a tolerance also return the magnitudes its derivation needs.
"""

import numpy as np


def e4m3(z):
    """Nearest e4m3 value (ties to even) of |z| <= 448: steps of 2^-3 of the leading power of two, of 2^-9 below 2^-6."""
    z = np.asarray(z, np.float64)
    _, e = np.frexp(np.maximum(np.abs(z), 2.0 ** -6))     # |z| = m 2^e, m in [1/2, 1)
    step = np.ldexp(1.0, e - 4)
    return np.rint(z / step) * step


def exponent(amax):
    """The least integer e >= -100 with amax <= 448 * 2^e."""
    m, e = np.frexp(np.asarray(amax, np.float64))           # 448 = 0.875 * 2^9
    return np.where(np.asarray(amax) > 0, np.maximum(e - 9 + (m > 0.875), -100), -100)


def quantize(x, smooth=None, rows=1):
    """(codes' values [M, K], exponents [ceil(M / rows), ceil(K / 128)]) of v = x * smooth, in blocks of
    `rows` x 128."""
    v = np.asarray(x, np.float64)
    if smooth is not None:
        v = v * np.asarray(smooth, np.float64)
    M, K = v.shape
    e = np.empty((-(-M // rows), -(-K // 128)), np.int64)
    codes = np.empty_like(v)
    for i in range(e.shape[0]):
        for p in range(e.shape[1]):
            b = (slice(rows * i, rows * (i + 1)), slice(128 * p, 128 * (p + 1)))
            e[i, p] = exponent(np.abs(v[b]).max())
            codes[b] = e4m3(np.ldexp(v[b], -int(e[i, p])))
    return codes, e


def gemm(codes, ascales, weight, wscales, bias=None):
    """(y, mag, cut): y = sum over blocks of 128 of ascales[p, m] * wscales[n // 128, p] * (codes @ weight^T), + bias;
    mag the same with absolute values and without the bias; cut a bound of what the matrix instruction drops.

    It adds products in groups of 8 neighbouring k, aligned to the largest exponent of the group (the sum of
    the two operands' exponents), and drops what lies below 2^-13 of it, towards zero (measured: beside 2^16 a
    product of 2^3 counts, one of 2^2 does not, 3.5 * 2^3 counts as 3 * 2^3). The largest itself, whose 8 bits reach
    2^-6, loses nothing; each of the other 7 less than 2^-13 of at most the product of the group's largest codes. Products
    within 2^7 of each other lose nothing, as 2^-6 of 2^-7 is still kept."""
    M, K = codes.shape
    N = weight.shape[0]
    y, mag, cut = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))

    def tops(z):
        z = np.pad(np.abs(z), ((0, 0), (0, -z.shape[1] % 8)))
        return z.reshape(len(z), -1, 8).max(2)

    for p in range(-(-K // 128)):
        s = np.asarray(ascales, np.float64)[p][:, None] * np.repeat(np.asarray(wscales, np.float64)[:, p], 128)[:N]
        k = slice(128 * p, 128 * (p + 1))
        y += s * (codes[:, k] @ weight[:, k].T)
        mag += np.abs(s) * (np.abs(codes[:, k]) @ np.abs(weight[:, k]).T)
        cut += np.abs(s) * 7 * 2.0 ** -13 * (tops(codes[:, k]) @ tops(weight[:, k]).T)
    return (y if bias is None else y + np.asarray(bias, np.float64)), mag, cut


def rope(z, positions, R, theta=10000.0, interleaved=False, factor=1.0, original=0, low=1.0, high=32.0, amplitude=1.0):
    """(out, mag, angle): pairs of the first R elements turned; mag = amplitude * (|u| + |w|) per element of a pair and 0
    for the rest; angle = |position * frequency| per element. Angles in long double."""
    z = np.asarray(z, np.float64)
    out, mag, far = z.copy(), np.zeros_like(z), np.zeros_like(z)
    tau = 2 * np.longdouble(np.pi) + np.longdouble(2.4492935982947064e-16)
    for i in range(R // 2):
        f = np.longdouble(theta) ** (np.longdouble(-2 * i) / R)
        kept = np.longdouble(0)
        if original:
            kept = min(max((original * f / tau - low) / (np.longdouble(high) - low), np.longdouble(0)), np.longdouble(1))
        f = f * (kept + (1 - kept) / np.longdouble(factor))
        angle = np.asarray(positions).astype(np.longdouble) * f
        c = np.cos(angle).astype(np.float64)[:, None] * amplitude
        s = np.sin(angle).astype(np.float64)[:, None] * amplitude
        iu, iw = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        u, w = z[:, :, iu], z[:, :, iw]
        out[:, :, iu], out[:, :, iw] = u * c - w * s, w * c + u * s
        mag[:, :, iu] = mag[:, :, iw] = amplitude * (np.abs(u) + np.abs(w))
        far[:, :, iu] = far[:, :, iw] = np.abs(angle).astype(np.float64)[:, None]
    return out, mag, far


class Cache:
    """A cache as values: codes [pages, Hk, page, D] (keys and values alike) and exponents [pages, Hk] (None: NaN)."""

    def __init__(self, pages, Hk, page, D):
        self.page = page
        self.codes = {n: np.zeros((pages, Hk, page, D)) for n in "kv"}
        self.exps = {n: np.full((pages, Hk), -100) for n in "kv"}
        self.nan = {n: np.zeros((pages, Hk), bool) for n in "kv"}

    def append(self, new, table, lengths, cu):
        """new = {"k": [T, Hk, D], "v": ...}; a page's tokens of the call at once."""
        pages = self.exps["k"].shape[0]
        for b in range(len(lengths)):
            at, i, end = max(int(lengths[b]), 0), cu[b], cu[b + 1]
            while i < end:
                blk, slot = at // self.page, at % self.page
                n = min(self.page - slot, end - i)
                p = table[b][blk] if blk < len(table[b]) else -1
                if 0 <= p < pages:
                    for name, z in new.items():
                        self._block(name, p, slot, z[i:i + n])
                at, i = at + n, i + n

    def _block(self, name, p, slot, z):
        codes, exps, nan = self.codes[name][p], self.exps[name][p], self.nan[name][p]
        for h in range(z.shape[1]):
            amax = np.abs(z[:, h]).max()
            if slot > 0 and nan[h]:
                continue
            nan[h] = not np.isfinite(amax)
            if nan[h]:
                continue
            e = int(exponent(amax))
            if slot > 0:
                e = max(e, int(exps[h]))
                codes[h, :slot] = e4m3(np.ldexp(codes[h, :slot], int(exps[h]) - e))
            exps[h] = e
            codes[h, slot:slot + len(z)] = e4m3(np.ldexp(z[:, h], -e))

    def values(self, name):
        z = np.ldexp(self.codes[name], self.exps[name][:, :, None, None])
        return np.where(self.nan[name][:, :, None, None], np.nan, z)


def gather(values, table, page, start, n):
    """Tokens start .. start + n - 1 of one sequence out of `values` [pages, Hk, page, D]; zeros without a page."""
    pages, Hk, _, D = values.shape
    out = np.zeros((n, Hk, D))
    for i in range(n):
        blk, slot = divmod(max(start, 0) + i, page)
        p = table[blk] if blk < len(table) else -1
        if 0 <= p < pages:
            out[i] = values[p, :, slot]
    return out


def attention(q, k, v, n, causal=True, scale=None):
    """One sequence: (o, tol) for its n queries q [n, H, D] over keys k, v [L, Hk, D]; tol bounds the device's error
    before the final rounding.

    The device's score is off by at most e_j = scale * (D + 8) * 2^-24 * sum |q| |k_j| (fp32 sums) + (2^-22 + 2^-23 |s_j -
    m|) (the exponent's subtraction, product and base 2, whose roundings are relative to it; 2^-22 the exponential's), which
    moves o by at most sum_j p_j e_j |v_j - o|. Each probability is rounded to bf16 (2^-8) for the product with v, the
    sum that divides it is taken before that: sum_j p_j 2^-8 |v_j|. First order; 5 % on top for the rest, plus the
    fp32 sums of the second product and of the probabilities, (L + 8) * 2^-24 * sum_j p_j (|v_j| + |o|)."""
    _, H, D = q.shape
    L, Hk = k.shape[:2]
    scale = D ** -0.5 if scale is None else scale
    o, tol = np.zeros((n, H, D)), np.zeros((n, H, D))
    for h in range(H):
        kk, vv = k[:, h // (H // Hk)], v[:, h // (H // Hk)]
        for lo in range(0, n, 256):
            i = np.arange(lo, min(n, lo + 256))
            last = L - n + i if causal else np.full(len(i), L - 1)
            some = last >= 0
            if not some.any():
                continue
            i, last = i[some], last[some]
            s = scale * (q[i, h] @ kk.T)
            e = scale * (D + 8) * 2.0 ** -24 * (np.abs(q[i, h]) @ np.abs(kk).T) + 2.0 ** -22
            s = np.where(np.arange(L)[None, :] <= last[:, None], s, -np.inf)
            d = s - s.max(1, keepdims=True)
            e = e + 2.0 ** -23 * np.where(np.isfinite(d), np.abs(d), 0.0)
            p = np.exp(d)
            p = p / p.sum(1, keepdims=True)
            # keys that are not seen have no say, whatever they hold
            live = np.where(p.any(0)[:, None], vv, 0.0)
            out = p @ live
            pv, pe = p @ np.abs(live), p * np.where(p > 0, e, 0.0)
            o[i, h] = out
            tol[i, h] = (1.05 * (2.0 ** -8 * pv + pe @ np.abs(live) + pe.sum(1, keepdims=True) * np.abs(out))
                         + (L + 8) * 2.0 ** -24 * (pv + np.abs(out)) + 1e-30)
    return o, tol
