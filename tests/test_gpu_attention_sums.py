"""GPU: attention where the softmax sums are what can go wrong, against float64 on scores that are exact in
fp32 (few products per score, each of few bits), so that the tolerance holds the sums' own roundings alone."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("base,low,step", [
    (177, 0, 0.125), (164, 0, 0.125), (151, 0, 0.125), (138, 0, 0.125), (149, 0, 0.25), (166, 0, 0.25),
    (177, 1824, 2.0), (177, 1808, 32.0), (-177, -1826, 2.0), (-177, -1840, 32.0)])
def test_weights_across_a_raised_maximum(gpu_lib, base, low, step, D):
    """Keys of the first tile score s, those of the second s + step, with s up to 7.3e5, where the product of
    maximum and scale rounds by up to 2^-4; query 1 raises the maxima of its wave at the second tile. The last
    four cases cross the border from which the maximum is taken off the scores, in both directions.

    v is 1 and -1, so o = (1 - e) / (1 + e), e = exp(step). Roundings: a probability to bf16 (2^-8 of the sum of
    p |v|, here 1), o to bf16 (2^-8), and fp32 steps of the exponents' differences, sums and quotient, below
    2^-18 together."""
    T = 128
    q, k, v = (torch.zeros(T, 1, D) for _ in range(3))
    q[:, 0, 0], k[:, 0, 0] = base, 4096
    q[:, 0, 1], k[64:, 0, 1] = 1, step
    q[:, 0, 3:5] = 1
    k[:, 0, 3], k[:, 0, 4] = low // 32 * 32, low % 32
    q[1] = 0
    q[1, 0, 2], k[64:, 0, 2] = 64, 1
    v[:64], v[64:] = 1, -1
    o = gpu_lib.attention_packed(*(t.bfloat16().cuda() for t in (q, k, v)), scale=1.0)
    for t in (q, k):
        assert torch.equal(t.bfloat16().float(), t)
    ref = -np.tanh(step / 2)
    tol = 2.0 ** -8 + 2.0 ** -8 * abs(ref) + 2.0 ** -18
    got = o.double().cpu().numpy()
    rows = np.delete(got, 1, axis=0)
    assert (np.abs(rows - ref) <= tol).all(), float(np.abs(rows - ref).max() / tol)
    assert (np.abs(got[1] + 1) <= tol).all()


@pytest.mark.parametrize("empty", [0, 40])
def test_sum_of_a_long_sequence(gpu_lib, empty):
    """2^18 keys: one of score 0, the others of one score whose probability (0.5596) makes a running fp32 sum lose
    1e-3 of itself (simulated), which o shows where its value is near the border between two bf16 numbers: 64 columns of
    v are 1 up to different keys and 0 behind. (With empty sequences beside it the mean length takes four waves.)

    o = (1 + b (n - 1)) / (1 + (T - 1) p) with b = bf16(p), 0.25 of a step from a tie; the products of b add up exactly
    (8 bits times 18, 16 keys at a time). p is off by at most 4 units of 2^-24, a tile's sum by 17, the rest by 4 more: 2e-6, and 1e-5 is allowed."""
    T, D = 1 << 18, 64
    p = 0.5595654845237732
    s = torch.tensor(np.log(p), dtype=torch.float64)
    hi = s.bfloat16().double()
    lo = (s - hi).bfloat16().double()
    p = float(torch.exp(hi + lo))
    b = float(torch.tensor(p, dtype=torch.float64).float().bfloat16())
    assert abs(p - b) < 0.35 * 2.0 ** -8
    q, k, v = (torch.zeros(T, 1, D) for _ in range(3))
    q[:, 0, :2] = 1
    k[1:, 0, 0], k[1:, 0, 1] = hi, lo
    n = 64 * np.random.default_rng(1).integers(T // 128, T // 64 + 1, D)
    v[:, 0] = (torch.arange(T)[:, None] < torch.from_numpy(n)[None]).float()
    cu = torch.tensor([0] * (empty + 1) + [T], dtype=torch.int32).cuda()
    o = gpu_lib.attention_packed(*(t.bfloat16().cuda() for t in (q, k, v)), cu, scale=1.0)
    assert bool((o == o[0]).all())
    ref = (1 + b * (n - 1.0)) / (1 + (T - 1) * p)
    half = 2.0 ** (np.floor(np.log2(ref)) - 8)
    err = np.abs(o[0, 0].double().cpu().numpy() - ref)
    assert (err <= half + 1e-5 * ref).all(), float(((err - half) / ref).max())
