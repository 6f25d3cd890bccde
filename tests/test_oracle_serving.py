"""CPU: the oracle of the 8-bit floating-point operators against facts that can be written down, and mistakes
planted in it, which the GPU tests' comparisons have to see."""

import numpy as np
import pytest
import torch

from oracle import serving as S


def test_e4m3_grid_and_ties():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    every = np.unique(every[np.isfinite(every)])
    assert every.max() == 448 and np.array_equal(S.e4m3(every), every)
    mid = (every[1:] + every[:-1]) / 2
    codes = torch.from_numpy(mid).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(S.e4m3(mid), codes)
    assert S.e4m3(17.0) == 16 and S.e4m3(19.0) == 20 and S.e4m3(2.0 ** -10) == 0 and S.e4m3(1.5 * 2.0 ** -9) == 2.0 ** -8


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (0.0, -100), (1.0, -8),
                                    (2.0 ** -140, -100), (448 * 2.0 ** -100, -100), (449 * 2.0 ** -100, -99),
                                    (3.3895313892515355e38, 120)])
def test_exponent(amax, e):
    assert S.exponent(amax) == e


def test_growing_scale_keeps_what_was_there():
    c = S.Cache(2, 1, 16, 64)
    rng = np.random.default_rng(0)
    a, b = rng.standard_normal((5, 1, 64)), 100 * rng.standard_normal((3, 1, 64))
    table = [[1]]
    c.append({"k": a, "v": a}, table, [0], [0, 5])
    before = c.values("k")[1, 0, :5].copy()
    c.append({"k": b, "v": b}, table, [5], [0, 3])
    after = c.values("k")[1, 0]
    unit = 2.0 ** c.exps["k"][1, 0]
    # exact but for what falls below the least normal code
    big = np.abs(before) >= 2.0 ** -6 * unit
    assert big.any() and np.array_equal(after[:5][big], before[big])
    assert (np.abs(after[:5] - before) <= 2.0 ** -10 * unit).all()
    assert (np.abs(after[5:8] - b[:, 0]) <= np.maximum(2.0 ** -4 * np.abs(b[:, 0]), 2.0 ** -10 * unit)).all()


def _attention_case(seed=0, n=5, L=300):
    rng = np.random.default_rng(seed)
    q = rng.standard_normal((n, 4, 64))
    k, v = rng.standard_normal((L, 2, 64)), rng.standard_normal((L, 2, 64))
    for i in range(n):                      # each query aligned with its last key and the one after: both show
        for h in range(4):
            q[i, h] = 0.6 * (k[L - n + i, h // 2] + k[min(L - n + i + 1, L - 1), h // 2]) + 0.05 * k[20, h // 2]
    return q, k, v


@pytest.mark.parametrize("mistake", ["last key left out", "a key too many", "wrong group", "page order", "scale of another page"])
def test_planted_mistakes_pass_the_bound(mistake):
    q, k, v = _attention_case()
    n, L = len(q), len(k)
    ref, tol = S.attention(q, k, v, n)
    tol = (1 + 2.0 ** -8) * tol + 2.0 ** -8 * np.abs(ref)
    if mistake == "last key left out":
        got, _ = S.attention(q, k[:-1], v[:-1], n)
    elif mistake == "a key too many":
        got = ref.copy()
        got[:-1] = S.attention(q[:-1], k, v, n - 1)[0]
    elif mistake == "wrong group":
        got, _ = S.attention(q, k[:, ::-1], v[:, ::-1], n)
    elif mistake == "page order":
        swap = np.r_[16:32, 0:16, 32:L]
        got, _ = S.attention(q, k, v[swap], n)
    else:
        v2 = v.copy()
        v2[16:32] *= 4
        got, _ = S.attention(q, k, v2, n)
    assert (np.abs(got - ref) > tol).any()


def test_rows_without_keys_are_zero():
    q, k, v = _attention_case(1, 3, 300)
    o, tol = S.attention(np.concatenate([q, q]), k[:4], v[:4], 6)
    assert not o[:2].any() and not tol[:2].any() and o[2:].all()


def test_rope_by_parts_and_linear():
    z = np.random.default_rng(1).standard_normal((3, 2, 64))
    pos = np.array([0, 7, 100000])
    same, _, _ = S.rope(z, pos, 64, factor=1.0, original=4096)
    plain, _, _ = S.rope(z, pos, 64)
    assert np.allclose(same, plain, atol=1e-12)
    far, _, _ = S.rope(z, pos * 8, 64, factor=8.0)
    assert np.allclose(far, plain, atol=1e-9)
    # the first pair turns 4096 / 2 pi times and is kept, the last turns less than once and is divided
    mixed, _, _ = S.rope(z, pos, 64, factor=8.0, original=4096)
    assert np.allclose(mixed[:, :, 0], plain[:, :, 0], atol=1e-12)
    slow, _, _ = S.rope(z, pos, 64, factor=8.0)
    assert np.allclose(mixed[:, :, 31], slow[:, :, 31], atol=1e-12)
    part, mag, _ = S.rope(z, pos, 16, interleaved=True, amplitude=1.5)
    assert np.array_equal(part[:, :, 16:], z[:, :, 16:]) and not mag[:, :, 16:].any()
    assert np.allclose((part[:, :, :16] ** 2).sum(2), 2.25 * (z[:, :, :16] ** 2).sum(2))


def test_gemm_blocks():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((5, 400)), rng.standard_normal((200, 400))
    a, ea = S.quantize(x)
    b, eb = S.quantize(w, rows=128)
    assert ea.shape == (5, 4) and eb.shape == (2, 4)
    va = np.ldexp(a, np.repeat(ea, 128, 1)[:, :400])
    vb = np.ldexp(b, np.repeat(np.repeat(eb, 128, 0)[:200], 128, 1)[:, :400])
    y, mag, cut = S.gemm(a, 2.0 ** ea.T, b, 2.0 ** eb)
    assert (cut > 0).all() and (cut < 7 * 2.0 ** -13 * 8 * mag).all()
    assert np.allclose(y, va @ vb.T) and np.allclose(mag, np.abs(va) @ np.abs(vb).T)
    assert np.linalg.norm(y - x @ w.T) < 0.05 * np.linalg.norm(x @ w.T)
