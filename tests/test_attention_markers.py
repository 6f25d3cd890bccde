"""Attention where single keys decide: a query aligned with one key gives it all the weight, so a key left out,
read twice or taken from a neighbour moves o by as much as a value. (With independent normal values o shrinks as
1 / L and hides in the tolerance.) The CPU tests plant such mistakes in the oracle and see them pass the bound."""

import numpy as np
import pytest
import torch

from oracle import block as B


def offsets(lens, start=0):
    return [int(c) for c in np.cumsum([start] + list(lens))]


def marked(T, H, D, cu, causal, seed, rows=160, Hk=None):
    """q [T, H, D], k, v [T, Hk, D] (bf16 values) and the marked queries. Keys are normal; a marked query is 3 times one key:
    its score is 3 sqrt(D) (24 and 34) against normal ones of deviation 3. Its key is one that it may see (first, last,
    tile borders, its own) or, for a third of the rows, one just outside: behind the query where causal, else in the
    neighbouring sequence or behind the last."""
    rng = np.random.default_rng(seed)
    Hk = Hk or H
    q, k, v = (torch.from_numpy(rng.standard_normal((T, n, D))).bfloat16() for n in (H, Hk, Hk))
    picks = []
    for a, b in zip(cu[:-1], cu[1:]):
        L = b - a
        if L == 0:
            continue
        edges = [0, 1, 31, 32, 63, 64, 65, 127, 128, 255, 256, L // 2, L - 257, L - 256, L - 129, L - 65, L - 64, L - 63, L - 2, L - 1]
        edges = sorted({e for e in edges if 0 <= e < L})
        at = sorted(set(edges) | set(rng.integers(0, L, rows // (len(cu) - 1)).tolist()))
        for n, i in enumerate(at):
            if n % 3 == 2:
                j = i + 1 if causal else (-1 if n % 2 else L)
                j = min(max(a + j, 0), T - 1)
                if causal and j == a + i:
                    continue
            else:
                may = [e for e in edges if not causal or e <= i] + ([i] if causal else [])
                j = a + may[rng.integers(len(may))]
            picks.append(a + i)
            q[a + i] = (3.0 * k[j].float()).bfloat16().repeat_interleave(H // Hk, 0)
    return q, k, v, np.array(sorted(picks))


def reference(q, k, v, cu, causal, queries):
    ref, tol, _ = B.attention_packed(*(t.double().numpy() for t in (q, k, v)), cu, causal, None, queries)
    return ref, (1 + 2.0 ** -8) * tol + 2.0 ** -8 * np.abs(ref)


CASES = [([8192], 0, 0, 128), ([8300], 0, 0, 64), ([9001], 0, 0, 128), ([16700], 0, 0, 64), ([9000, 8250], 5, 3, 128), ([4100], 0, 0, 128),
         ([700, 65, 1, 190], 2, 1, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,start,behind,D", CASES, ids=lambda x: "-".join(map(str, x)) if isinstance(x, list) else str(x))
@pytest.mark.parametrize("causal", [False, True])
def test_marked_keys(gpu_lib, lens, start, behind, D, causal):
    print(f"[attention] marked {lens} D={D} causal={causal}", flush=True)
    cu = offsets(lens, start)
    T = cu[-1] + behind
    q, k, v, at = marked(T, 1, D, cu, causal, T)
    o = gpu_lib.attention_packed(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), causal=causal)
    ref, tol = reference(q, k, v, cu, causal, at)
    err = np.abs(o.double().cpu().numpy() - ref)[at]
    assert (err <= tol[at]).all(), float((err / tol[at]).max())


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk", [(8, 1), (12, 2), (6, 2), (16, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_marked_keys_of_head_groups(gpu_lib, H, Hk, causal):
    """Eight waves dealt to 8, 2, 1 and 8 heads of a group: rows of 32, 128, 256 and 32 queries."""
    print(f"[attention] marked groups {H} {Hk} causal={causal}", flush=True)
    T, D = 8200, 128
    q, k, v, at = marked(T, H, D, [0, T], causal, H, 12, Hk)
    o = gpu_lib.attention_packed(q.cuda(), k.cuda(), v.cuda(), causal=causal)
    ref, tol = reference(q, k, v, None, causal, at)
    err = np.abs(o.double().cpu().numpy() - ref)[at]
    assert (err <= tol[at]).all(), float((err / tol[at]).max())


@pytest.mark.parametrize("lens,D,drop", [([8300], 64, "last"), ([8300], 64, "first"), ([8192], 128, "tile"), ([9001], 128, "behind"),
                                         ([700, 65, 1, 190], 64, "neighbour"), ([700, 65, 1, 190], 64, "behind")])
def test_the_bound_sees_a_wrong_key(lens, D, drop):
    """The mistakes: the sequence's last or first key left out, a whole 64-key tile left out, the key behind a causal
    query taken in, a neighbour's first key taken in."""
    causal = drop == "behind"
    cu = offsets(lens)
    T = cu[-1]
    q, k, v, at = marked(T, 1, D, cu, causal, T, rows=40)
    at = at[at < cu[1]]
    ref, tol = reference(q, k, v, cu, causal, at)
    Q, K, V = (t[:, 0].double().numpy() for t in (q, k, v))
    keys = np.arange(cu[1])
    keys = {"last": keys[:-1], "first": keys[1:], "tile": np.delete(keys, slice(cu[1] - 320, cu[1] - 256)),
            "neighbour": np.arange(cu[1] + 1), "behind": keys}[drop]
    s = Q[at] @ K[keys].T / np.sqrt(D)
    if causal:
        s = np.where(keys[None] <= at[:, None] + 1, s, -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    wrong = (p / p.sum(1, keepdims=True)) @ V[keys]
    seen = (np.abs(wrong - ref[at, 0]) > 20 * tol[at, 0]).any(1)
    assert seen.sum() >= (2 if drop != "tile" else 1), int(seen.sum())
