"""Pins of oracle/block.py to something other than itself: exact rationals, closed forms, torch."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block as B


def bf16(a):
    return torch.tensor(np.asarray(a, np.float32)).bfloat16().double().numpy()


def test_quantize_int8_against_rationals():
    rng = np.random.default_rng(1)
    x = bf16(rng.standard_normal((6, 48)) * [[1e-3], [1], [50], [1e20], [1e-30], [7]])
    codes, scale = B.quantize_int8(x)
    for m in range(x.shape[0]):
        a = Fraction(float(np.abs(x[m]).max()))
        assert abs(Fraction(float(scale[m])) - a / 127) <= a / 127 * Fraction(1, 2 ** 24)
        for k in range(x.shape[1]):
            exact = Fraction(float(x[m, k])) * 127 / a
            # fp32 steps: within 2 units of 2^-24 of the exact quotient before rounding
            assert abs(Fraction(int(codes[m, k])) - exact) <= Fraction(1, 2) + abs(exact) * Fraction(2, 2 ** 24)
        assert abs(codes[m]).max() == 127


def test_quantize_int8_zero_and_tiny_rows():
    x = np.zeros((3, 16))
    x[1, 3] = 2.0 ** -126
    x[2, 5] = 2.0 ** -119
    codes, scale = B.quantize_int8(x)
    assert not codes[:2].any() and not scale[:2].any()
    assert codes[2, 5] == 127 and scale[2] > 0


def test_gemm_int8_integers():
    rng = np.random.default_rng(2)
    c = rng.integers(-127, 128, (3, 32))
    w = rng.integers(-128, 128, (4, 32))
    y, _ = B.gemm_int8(c, np.full(3, 0.5), w, np.full(4, 0.25))
    assert np.array_equal(y * 8, (c @ w.T).astype(float))


def test_norm_gated_closed_forms():
    h = np.full((2, 16), 3.0)
    b = np.full((2, 16), -2.0)
    ho, x, _, _, rows = B.norm_gated(h, b, rs=0.5, eps=0.0)
    assert np.allclose(ho, 2.5) and np.allclose(x, 1.0) and rows.all()
    ho, x, _, _, _ = B.norm_gated(h, b, gate=np.zeros((1, 16)), scale=np.full((1, 16), 1.0), eps=0.0)
    assert np.array_equal(ho, h) and np.allclose(x, 2.0)
    _, _, _, _, rows = B.norm_gated(np.ones((5, 16)), cu=[1, 1, 3])
    assert rows.tolist() == [False, True, True, False, False]


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_axes_rotates_and_keeps_relative_phase(interleaved):
    rng = np.random.default_rng(3)
    z = rng.standard_normal((4, 2, 64))
    pos = rng.integers(-50, 5000, (4, 3))
    out, _ = B.rope_axes(z, pos, (16, 24, 24), interleaved=interleaved)
    assert np.allclose((out ** 2).sum(2), (z ** 2).sum(2))
    zero, _ = B.rope_axes(z, 0 * pos, (16, 24, 24), interleaved=interleaved)
    assert np.array_equal(zero, z)
    # <R_p q, R_p' k> depends on p - p' alone
    q, k = z[:, :1], z[:, 1:]
    moved = pos + np.array([11, -7, 300])
    a = (B.rope_axes(q, pos, (16, 24, 24), interleaved=interleaved)[0][0]
         * B.rope_axes(k, pos, (16, 24, 24), interleaved=interleaved)[0][1]).sum()
    b = (B.rope_axes(q, moved, (16, 24, 24), interleaved=interleaved)[0][0]
         * B.rope_axes(k, moved, (16, 24, 24), interleaved=interleaved)[0][1]).sum()
    assert abs(a - b) < 1e-9


def test_rope_axes_first_pair_by_hand():
    z = np.zeros((1, 1, 64))
    z[0, 0, 0] = 1.0
    out, _ = B.rope_axes(z, np.array([[2, 0]]), (32, 32))
    assert np.isclose(out[0, 0, 0], np.cos(2.0)) and np.isclose(out[0, 0, 1], np.sin(2.0))
    out, _ = B.rope_axes(z, np.array([[2, 0]]), (32, 32), interleaved=False)
    assert np.isclose(out[0, 0, 0], np.cos(2.0)) and np.isclose(out[0, 0, 32], np.sin(2.0))


@pytest.mark.parametrize("causal", [False, True])
def test_attention_against_torch(causal):
    rng = np.random.default_rng(4)
    cu = [0, 5, 5, 12, 13]
    q, k, v = rng.standard_normal((14, 4, 64)), rng.standard_normal((14, 2, 64)), rng.standard_normal((14, 2, 64))
    o, tol, rows = B.attention_packed(q, k, v, cu, causal)
    assert rows.tolist() == [True] * 13 + [False] and (tol[:13] > 0).all()
    for a, b in zip(cu[:-1], cu[1:]):
        if a == b:
            continue
        t = [torch.tensor(z[a:b]).transpose(0, 1) for z in (q, np.repeat(k, 2, 1), np.repeat(v, 2, 1))]
        ref = torch.nn.functional.scaled_dot_product_attention(*t, is_causal=causal).transpose(0, 1).numpy()
        assert np.allclose(o[a:b], ref, atol=1e-12)


def test_attention_closed_forms():
    rng = np.random.default_rng(5)
    v = rng.standard_normal((6, 1, 64))
    o, _, _ = B.attention_packed(np.zeros((6, 1, 64)), rng.standard_normal((6, 1, 64)), v, causal=True)
    assert np.allclose(o[:, 0], np.cumsum(v[:, 0], 0) / np.arange(1, 7)[:, None])
