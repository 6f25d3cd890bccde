"""GPU: packed attention where every score lies so far below zero that its power of two leaves fp32: at scales above 1 such
scores are ordinary finite fp32 numbers, and a row answers with its best key's value, or the mean over equal ones."""

import numpy as np
import pytest
import torch

from tests.test_gpu_attention import dev, f64, make, offsets
from tests.test_gpu_attention_cache_far import best_keys, visible

pytestmark = pytest.mark.gpu

SHAPES = [([1, 2, 31, 33], 4, 2, 128), ([64, 0, 65, 1, 200], 3, 3, 64), ([700, 130], 6, 2, 64), ([1300], 2, 1, 128)]
IDS = ["-".join(map(str, s[0])) for s in SHAPES]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("scale", [64.0, 2.0 ** 20])
@pytest.mark.parametrize("lens,H,Hk,D", SHAPES, ids=IDS)
def test_best_key_of_scores_far_below_zero(gpu_lib, lens, H, Hk, D, scale, causal):
    print(f"[attention] far below: {lens} H={H} Hk={Hk} D={D} scale={scale} causal={causal}", flush=True)
    T, cu = sum(lens), offsets(lens)
    q, k, v = make(T, H, Hk, D, T + D)
    q, k = -(q.abs().float() * 2.0 ** 119).bfloat16(), k.abs()
    o = f64(gpu_lib.attention_packed(q, k, v, dev(cu), causal=causal, scale=scale))
    q, k, v = f64(q), f64(k), np.repeat(f64(v), H // Hk, 1)
    sure = 0
    for n, a in zip(lens, cu):
        r = slice(a, a + n)
        if n == 0:
            continue
        best, far = best_keys(q[r], k[r], scale, visible(n, n, causal))
        want = v[r][best, np.arange(H)[None]]
        assert np.array_equal(o[r][far], want[far]), n
        sure += int(far.sum())
    assert sure >= T * H // 2 and np.isfinite(o).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("lens,H,Hk,D", SHAPES + [([8200], 1, 1, 128)], ids=IDS + ["8200"])
def test_equal_scores_far_from_zero(gpu_lib, lens, H, Hk, D, sign, causal):
    """Scores of 2^20 * +-D 2^110 are exact, probabilities exactly 1 and so is their sum: o is the mean of the values that a row
    sees, off by fp32 sums (at most 2^-23 an addition) and one rounding to bf16."""
    T, cu = sum(lens), offsets(lens)
    _, _, v = make(T, H, Hk, D, T)
    q = torch.full((T, H, D), sign * 2.0 ** 110, dtype=torch.bfloat16, device="cuda")
    k = torch.ones((T, Hk, D), dtype=torch.bfloat16, device="cuda")
    o, v = f64(gpu_lib.attention_packed(q, k, v, dev(cu), causal=causal, scale=2.0 ** 20)), f64(v)
    for n, a in zip(lens, cu):
        seen = visible(n, n, causal)
        z = np.concatenate([np.zeros((1, Hk, D)), v[a:a + n]])
        count = np.maximum(seen, 1)[:, None, None]
        mean, mag = (np.repeat(np.cumsum(x, 0)[seen] / count, H // Hk, 1) for x in (z, np.abs(z)))
        tol = 2.0 ** -8 * np.abs(mean) + (1 + 2.0 ** -8) * (count + 8) * 2.0 ** -23 * mag
        assert (np.abs(o[a:a + n] - mean) <= tol).all(), n
