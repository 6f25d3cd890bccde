"""Operators between a transformer block's linears, restated in float64 (oracle; test use only).

* the linear in 8-bit integers with a scale per token and per output channel,
* the norms before and after a block with its gate, residual scale and modulation,
* rotary positions with several axes and the per-head norm,
* attention over packed sequences with grouped heads.

Inputs are float64 arrays holding bf16 (or integer) values exactly. Functions that
feed a tolerance also return the magnitudes its derivation needs. The 8-bit codes
are defined by fp32 steps and are computed in NumPy float32, whose division,
product and rounding are the IEEE ones.
"""

import numpy as np


def quantize_int8(x, smooth=None):
    """Codes (int8) and scales (float32) of rows x [M, K]: v = x * smooth, codes =
    rne(v * (127 / max |v|)), scale = max |v| / 127, in float32 steps; rows whose 127 / max
    overflows (a zero row among them) give zeros."""
    v = np.asarray(x, np.float32)
    if smooth is not None:
        v = v * np.asarray(smooth, np.float32)
    a = np.abs(v).max(axis=1)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.float32(127.0) / a
    live = np.isfinite(inv)
    inv = np.where(live, inv, np.float32(0.0)).astype(np.float32)
    scale = np.where(live, a / np.float32(127.0), np.float32(0.0)).astype(np.float32)
    return np.rint(v * inv[:, None]).astype(np.int8), scale


def gemm_int8(codes, ascales, weight, wscales, bias=None):
    """(y, |main|): y = (codes @ weight^T) * ascales * wscales + bias in float64, sums exact."""
    acc = np.asarray(codes, np.float64) @ np.asarray(weight, np.float64).T
    main = acc * np.asarray(ascales, np.float64)[:, None] * np.asarray(wscales, np.float64)[None, :]
    y = main if bias is None else main + np.asarray(bias, np.float64)[None, :]
    return y, np.abs(main)


def _groups(M, cu, G):
    g = np.full(M, -1, np.int64)
    if cu is None:
        g[:] = 0
        return g
    for i in range(G):
        g[cu[i]:cu[i + 1]] = i
    return g


def norm_gated(h, block=None, post=None, gate=None, rs=1.0, pre=None, scale=None, cu=None, eps=1e-6):
    """(h_out, x_out, added, factor, rows): added = what the block adds to h, factor = x_out / h_out
    per element's multiplier, rows = the rows that belong to a group."""
    M, K = h.shape
    G = 1 if cu is None else len(cu) - 1
    g = _groups(M, cu, G)
    rows = g >= 0
    gi = np.maximum(g, 0)
    added = np.zeros((M, K))
    if block is not None:
        added = block / np.sqrt((block ** 2).mean(1, keepdims=True) + eps)
        if post is not None:
            added = added * post
        if gate is not None:
            added = added * gate[gi]
        added = rs * added
    h_out = h + added
    factor = 1.0 / np.sqrt((h_out ** 2).mean(1, keepdims=True) + eps)
    factor = np.broadcast_to(factor, (M, K)).copy()
    if pre is not None:
        factor = factor * pre
    if scale is not None:
        factor = factor * (1.0 + scale[gi])
    return h_out, h_out * factor, added, factor, rows


def rope_axes(z, positions, axis_dims, theta=10000.0, interleaved=True, weight=None, eps=1e-6):
    """(out, |u| + |w|) for z [T, H, D]: the sum of the magnitudes of each element's pair."""
    z = np.asarray(z, np.float64)
    T, H, D = z.shape
    if weight is not None:
        z = z / np.sqrt((z ** 2).mean(2, keepdims=True) + eps) * weight
    out = np.empty_like(z)
    mag = np.empty_like(z)
    p = 0
    for a, d in enumerate(axis_dims):
        for i in range(d // 2):
            angle = positions[:, a].astype(np.float64) * theta ** (-2.0 * i / d)
            c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
            iu, iw = (2 * p, 2 * p + 1) if interleaved else (p, p + D // 2)
            u, w = z[:, :, iu], z[:, :, iw]
            out[:, :, iu] = u * c - w * s
            out[:, :, iw] = w * c + u * s
            mag[:, :, iu] = mag[:, :, iw] = np.abs(u) + np.abs(w)
            p += 1
    return out, mag


def attention_packed(q, k, v, cu=None, causal=False, scale=None, queries=None):
    """(o, tol, rows): o [T, H, D] in float64, a bound on the device's error before the final
    rounding, and the rows that belong to a sequence (of `queries`, token numbers, if given: the others
    are left zero).

    The bound: the device's score is off by at most e_j = scale * (D + 8) * 2^-24 * sum |q| |k_j| (fp32
    sums) + 2^-21 (the exponent's own roundings), which moves o by at most sum_j p_j e_j |v_j - o|. Each
    probability is rounded to bf16 (2^-8) for the product with v, the sum that divides it is taken before
    that: sum_j p_j 2^-8 |v_j|. First order; 5 % on top for the rest, plus the fp32 sums of the second product
    and of the probabilities, (L + 8) * 2^-24 * sum_j p_j (|v_j| + |o|)."""
    T, H, D = q.shape
    Hk = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    cu = [0, T] if cu is None else list(cu)
    o = np.zeros((T, H, D))
    tol = np.zeros((T, H, D))
    rows = np.zeros(T, bool)
    for b in range(len(cu) - 1):
        r = slice(cu[b], cu[b + 1])
        L = cu[b + 1] - cu[b]
        if L <= 0:
            continue
        at = np.arange(cu[b], cu[b + 1])
        if queries is not None:
            at = np.intersect1d(at, queries)
        rows[at] = True
        for hd in range(H):
            qq, kk, vv = q[at, hd], k[r, hd // (H // Hk)], v[r, hd // (H // Hk)]
            s = scale * (qq @ kk.T)
            e = scale * (D + 8) * 2.0 ** -24 * (np.abs(qq) @ np.abs(kk).T) + 2.0 ** -21
            if causal:
                s = np.where(np.arange(L)[None, :] <= (at - cu[b])[:, None], s, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p = p / p.sum(1, keepdims=True)
            out = p @ vv
            o[at, hd] = out
            pe = p * e
            pv = p @ np.abs(vv)
            tol[at, hd] = (1.05 * (2.0 ** -8 * pv + pe @ np.abs(vv) + pe.sum(1, keepdims=True) * np.abs(out))
                          + (L + 8) * 2.0 ** -24 * (pv + np.abs(out)) + 1e-30)
    return o, tol, rows
