"""The cached attention's choice of kernel and split: each is reached by named sizes and close to the best by the measured grid
(CPU), and is right there (GPU), its tiles in every form. A refit of the choice that leaves a kernel without a size
fails here."""

import os

import numpy as np
import pytest

from bit_w4a4_quantized_quantize_amd import _lib, ops
from tests.test_gpu_attention_cache import Case

RAGGED = [(70, 40), (129, 155), (1, 1), (128, 128), (0, 90), (200, 155), (33, 100), (257, 0), (64, 64), (65, 65), (127, 153),
          (190, 120), (3, 155), (128, 155), (256, 149), (190, 151), (100, 140), (2, 2), (300, 101)]
LONG = [(257, 6000), (1, 300), (130, 2900), (0, 700), (119, 64), (93, 4200)]
MIDDLE = [(700, 2838), (1001, 2500), (0, 5), (600, 599), (1, 2838), (700, 703), (490, 2740)]

# kernel, ways the keys are split, (queries, keys) of each sequence, H, Hk, D: both joins (up to eight ways, and more)
SIZES = [
    (0, 1, [(1, 92), (3, 40)], 4, 2, 64), (0, 1, [(5, 64), (1, 9)], 6, 2, 128),
    (0, 8, [(1, 1811)], 2, 1, 64), (0, 8, [(1, 1845), (1, 3)], 3, 1, 128),
    (0, 12, [(1, 2074), (2, 70)], 2, 1, 64), (0, 12, [(2, 2072)], 5, 1, 128),
    (1, 1, RAGGED, 24, 3, 64), (1, 1, RAGGED, 16, 2, 128), (1, 4, MIDDLE, 6, 2, 64), (1, 6, MIDDLE, 2, 1, 128),
    (1, 12, LONG, 12, 2, 64), (1, 16, LONG, 4, 1, 128)]


def plan(seqs, H, Hk, D):
    T = sum(n for n, _ in seqs)
    return ops.attention_cache_fp8_plan(T, len(seqs), H, Hk, D, max(L for _, L in seqs), True)


def kind(splits):
    return 0 if splits == 1 else 1 if splits <= 8 else 2


def test_every_kernel_and_join_has_its_sizes():
    kinds = set()
    for kernel, splits, seqs, H, Hk, D in SIZES:
        got = plan(seqs, H, Hk, D)
        assert got == (kernel, splits), (got, kernel, splits, H, Hk, D)
        kinds.add((kernel, kind(splits), D))
    assert len(kinds) == 12


def measured_grid():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles", "attention_cache_grid.txt")
    for line in open(path):
        if not line.startswith("#"):
            *sizes, = map(int, line.split()[:7])
            yield sizes, {tuple(map(int, t.split(":")[0].split("/"))): float(t.split(":")[1]) for t in line.split()[7:]}


def test_choice_against_the_measured_grid():
    """The chosen kernel and split, by the times measured for all of them: what a refit may lose, by the device's time, and
    where that is less than a call takes its caller."""
    loss, short = [], []
    for (H, Hk, D, B, n, before, longest), times in measured_grid():
        got = ops.attention_cache_fp8_plan(B * n, B, H, Hk, D, longest, n > 1)
        if got not in times:     # more ways than were measured at its size
            assert max(s for k, s in times if k == got[0]) < got[1], (H, Hk, D, B, n, before, got)
            continue
        best = min(times.values())
        (short if best < 14 else loss).append(times[got] / best)
    assert len(loss) > 150 and len(short) > 100
    assert np.mean(loss) <= 1.05 and max(loss) <= 1.35 and np.mean(short) <= 1.02 and max(short) <= 1.25


@pytest.mark.parametrize("sizes", [(0, 1, 4, 2, 128, 100), (1, 0, 4, 2, 128, 100), (1, 1, 5, 2, 128, 100), (1, 1, 4, 0, 128, 100),
                                   (1, 1, 4, 2, 96, 100), (1, 1, 4, 2, 128, 0)])
def test_plan_refusals(sizes):
    with pytest.raises(_lib.SvdqError):
        ops.attention_cache_fp8_plan(*sizes, True)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("kernel,splits,seqs,H,Hk,D", SIZES, ids=[f"{k}-{s}-{D}" for k, s, _, _, _, D in SIZES])
def test_kernel(gpu_lib, kernel, splits, seqs, H, Hk, D, causal, page):
    print(f"[attention_cache] kernel {kernel} / {splits} H={H} Hk={Hk} D={D} causal={causal} page={page}", flush=True)
    c = Case(gpu_lib, [n for n, _ in seqs], [L for _, L in seqs], H, Hk, D, page, kernel + splits)
    c.check(c.run(causal), causal)
