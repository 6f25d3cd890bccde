"""GPU: attention over the e4m3 cache where every score lies so far below zero that its power of two leaves fp32: a row
still answers with the keys it sees, not with the zeros of a row that sees none. At scales above 1 such scores are ordinary
finite fp32 numbers. Every kernel, whole and split, and both joins: the sizes of the choice's own test."""

import numpy as np
import pytest
import torch

from tests.test_attention_cache_plan import SIZES, plan
from tests.test_gpu_attention_cache import Case, f64

SCALES = [64.0, 2.0 ** 20]
IDS = [f"{k}-{s}-{D}" for k, s, _, _, _, D in SIZES]


def case(lib, seqs, H, Hk, D, page, seed):
    return Case(lib, [n for n, _ in seqs], [L for _, L in seqs], H, Hk, D, page, seed)


def visible(n, L, causal):
    """Keys that each of a sequence's n queries sees."""
    return np.maximum(L - n + 1 + np.arange(n), 0) if causal else np.full(n, L)


def best_keys(q, k, scale, seen):
    """(the best key's index [n, H], whether it is so by far): by more than 200 powers of two beyond what fp32 sums may be off
    by. q [n, H, D], k [L, Hk, D].

    A score is a sum of D exact products, off by at most D 2^-23 sum |q||k| (each addition by 2^-24 of its result where it
    rounds, twice that where it cuts off); 8 more for the products' own order. Every other key's probability is then below
    2^-149 and zero, the best key's is exactly 1, and o is exactly its value."""
    n, H, D = q.shape
    best, far = np.zeros((n, H), int), np.zeros((n, H), bool)
    for h in range(H):
        kk = k[:, h // (H // k.shape[1])]
        s = q[:, h] @ kk.T
        off = (D + 8) * 2.0 ** -23 * (np.abs(q[:, h]) @ np.abs(kk).T).max(1)
        s = np.where(np.arange(len(kk))[None] < seen[:, None], s, -np.inf)
        best[:, h] = s.argmax(1)
        far[:, h] = seen > 0
        if len(kk) > 1:
            top = np.sort(s, 1)[:, -2:]
            far[:, h] &= (seen == 1) | (top[:, 1] > top[:, 0] + 2 * off + 200 / (scale * np.log2(np.e)))
    return best, far


def all_below(c, gain):
    """Keys and queries of opposite sign, so that no score is above zero."""
    b = c.cache.k_codes.view(torch.uint8)
    b.copy_(torch.where(b == 0xFF, b, b & 0x7F))
    for kv in c.keys:
        kv[0] = np.abs(kv[0])
    c.q = -(c.q.float().abs() * gain).bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("kernel,splits,seqs,H,Hk,D", SIZES, ids=IDS)
def test_best_key_of_scores_far_below_zero(gpu_lib, kernel, splits, seqs, H, Hk, D, scale, causal):
    print(f"[attention_cache] far below: {kernel} / {splits} H={H} Hk={Hk} D={D} scale={scale} causal={causal}", flush=True)
    assert plan(seqs, H, Hk, D) == (kernel, splits)
    c = case(gpu_lib, seqs, H, Hk, D, 64, 50 + kernel + splits)
    all_below(c, 2.0 ** 119)       # the largest scores pass 2^126, every score times 64 log2 e passes 2^128 in most rows
    check_best(c, c.run(causal, scale=scale), causal, scale)


def check_best(c, o, causal, scale):
    o, q = f64(o), f64(c.q)
    assert np.isfinite(o).all()
    sure = rows = 0
    for b, (n, L) in enumerate(zip(c.new, c.lens)):
        r = slice(c.cu[b], c.cu[b + 1])
        seen = visible(n, L, causal)
        assert not o[r][seen == 0].any()
        if L == 0 or n == 0:
            continue
        best, far = best_keys(q[r], c.keys[b][0], scale, seen)
        v = np.repeat(c.keys[b][1], c.H // c.Hk, 1)
        want = v[best, np.arange(c.H)[None]]
        assert np.array_equal(o[r][far], want[far]), (b, n, L)
        sure, rows = sure + int(far.sum()), rows + int((seen > 0).sum()) * c.H
    assert sure >= rows // 2, (sure, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kernel,splits,seqs,H,Hk,D", SIZES, ids=IDS)
def test_equal_scores_far_from_zero(gpu_lib, kernel, splits, seqs, H, Hk, D, sign, causal):
    """Equal keys: each row's o is the mean of the values it sees. Scores of 2^20 * +-448 D 2^103 are exact, probabilities are
    exactly 1 and so is their sum. What is left are the fp32 sums, L additions of at most 2^-23 of what is added up, a few
    operations of the quotient, and one rounding to bf16."""
    print(f"[attention_cache] equal, far: {kernel} / {splits} H={H} Hk={Hk} D={D} sign={sign} causal={causal}", flush=True)
    c = case(gpu_lib, seqs, H, Hk, D, 32, 60 + kernel + splits)
    c.cache.k_codes.view(torch.uint8)[:] = 0x7E        # 448
    c.cache.k_scales[:] = 127
    c.q[:] = sign * 2.0 ** 103
    o = f64(c.run(causal, scale=2.0 ** 20))
    for b, (n, L) in enumerate(zip(c.new, c.lens)):
        seen = visible(n, L, causal)
        v = np.concatenate([np.zeros((1, c.Hk, c.D)), c.keys[b][1]])
        count = np.maximum(seen, 1)[:, None, None]
        mean, mag = (np.repeat(np.cumsum(x, 0)[seen] / count, c.H // c.Hk, 1) for x in (v, np.abs(v)))
        tol = 2.0 ** -8 * np.abs(mean) + (1 + 2.0 ** -8) * (count + 8) * 2.0 ** -23 * mag
        err = np.abs(o[c.cu[b]:c.cu[b + 1]] - mean)
        assert (err <= tol).all(), (b, n, L, float(np.nanmax(err - tol)))


@pytest.mark.gpu
@pytest.mark.parametrize("scale,gain", [(2.0 ** 20, 1.0), (2.0 ** 10, 2.0 ** 100), (1.0, 2.0 ** 110)])
@pytest.mark.parametrize("kernel,splits,seqs,H,Hk,D", SIZES, ids=IDS)
def test_best_key_of_extreme_scores(gpu_lib, kernel, splits, seqs, H, Hk, D, scale, gain):
    """Scores of either sign: by value, not only finite."""
    c = case(gpu_lib, seqs, H, Hk, D, 128, 70 + kernel + splits)
    c.q = (c.q.float() * gain).bfloat16()
    for causal in (False, True):
        check_best(c, c.run(causal, scale=scale), causal, scale)


def test_best_keys_of_a_written_out_case():
    """The helper itself, on the CPU: the least of scores below zero wins among the keys that a row sees."""
    k = np.array([[[4.0]], [[1.0]], [[2.0]]])
    q = np.array([[[-1.0]], [[-1.0]], [[-1.0]]])
    best, far = best_keys(q, k, 2.0 ** 20, visible(3, 3, True))
    assert best[:, 0].tolist() == [0, 1, 1] and far.all()
    best, far = best_keys(q, k, 1.0, np.array([0, 2, 3]))
    assert not far.any()
