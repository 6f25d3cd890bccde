"""GPU: the gated norms around a block against the oracle in float64.

Error of the fp32 steps: a sum of K squares in any order is off by at most K 2^-24 relative, the norm's
factor by half of that, and at most 8 further roundings act on it: e = (K / 2 + 8) 2^-24. h_out is off by
dh = e |added| + 2^-24 |h_out| before its bf16 rounding (2^-8); x_out by factor * dh + |x| (e + |dh| / |h|)
(the second norm sees h's error in its sum) and its own bf16 rounding.
"""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(M, K, G, seed, full=True, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    bf = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    h = bf(M, K) * spread
    h[:, :: max(1, K // 3)] *= 20
    d = dict(h=h, block=bf(M, K) * 3)
    if full:
        d |= dict(post_weight=1 + 0.1 * bf(K), gate=bf(G, K).tanh(), pre_weight=1 + 0.1 * bf(K), scale=0.3 * bf(G, K))
    return {k: v.bfloat16().cuda() for k, v in d.items()}


def bounds(d, rs, eps, cu):
    ho, x, added, factor, rows = B.norm_gated(f64(d["h"]), f64(d.get("block")), f64(d.get("post_weight")),
                                              f64(d.get("gate")), rs, f64(d.get("pre_weight")), f64(d.get("scale")),
                                              cu, eps)
    K = ho.shape[1]
    e = (K / 2 + 8) * 2.0 ** -24
    dh = e * np.abs(added) + 2.0 ** -24 * np.abs(ho)
    if d.get("block") is None:
        dh = 0 * dh
    rel = np.linalg.norm(dh, axis=1, keepdims=True) / np.maximum(np.linalg.norm(ho, axis=1, keepdims=True), 1e-300)
    dx = np.abs(factor) * dh + np.abs(x) * (e + rel)
    tiny = 2.0 ** -133   # a bf16 denormal's half step
    return ho, 2.0 ** -8 * (np.abs(ho) + dh) + dh + tiny, x, 2.0 ** -8 * (np.abs(x) + dx) + dx + tiny, rows


def check(got, ref, tol, rows):
    err = np.abs(f64(got) - ref)[rows]
    assert (err <= tol[rows]).all(), float((err / tol[rows]).max())


CASES = [(1, 16, 1), (3, 48, 2), (77, 3840, 1), (5, 2048, 3), (4, 2064, 4), (9, 4096, 2), (6, 4112, 3), (5, 8192, 5),
         (3, 8208, 1), (4, 10240, 2), (2, 16384, 1), (3, 16400, 2), (2, 32768, 2), (1000, 256, 7), (2500, 1024, 6)]


@pytest.mark.parametrize("M,K,G", CASES)
@pytest.mark.parametrize("full", [True, False])
def test_against_oracle(gpu_lib, M, K, G, full):
    print(f"[norm] {M} {K} {G} full={full}", flush=True)
    d = make(M, K, G, M + K, full)
    edges = np.sort(np.random.default_rng(K).integers(0, M + 1, G - 1))
    cu = [0, *edges.tolist(), M]
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ho, x = gpu_lib.norm_gated(**d, residual_scale=0.5, cu_seqlens=cut, eps=1e-6)
    rh, th, rx, tx, rows = bounds(d, 0.5, 1e-6, cu)
    check(ho, rh, th, rows)
    check(x, rx, tx, rows)
    # the 8-bit form: the codes of the bf16 x_out, bit for bit
    for smooth in (None, (torch.rand(K) + 0.5).bfloat16().cuda()):
        h8, codes, scales = gpu_lib.norm_gated_int8(**d, residual_scale=0.5, cu_seqlens=cut, eps=1e-6, smooth=smooth)
        qc, qs = gpu_lib.quantize_int8(x, smooth)
        assert torch.equal(h8, ho) and torch.equal(codes, qc) and torch.equal(scales, qs)


@pytest.mark.parametrize("M,K", [(7, 272), (3, 3840)])
def test_optional_parts(gpu_lib, M, K):
    d = make(M, K, 1, 3)
    # before the first block: the norm alone
    first = dict(h=d["h"], pre_weight=d["pre_weight"], scale=d["scale"])
    none, x = gpu_lib.norm_gated(**first)
    assert none is None
    _, _, rx, tx, rows = bounds(first, 1.0, 1e-6, None)
    check(x, rx, tx, rows)
    # after the last block: no norm after it
    last = {k: d[k] for k in ("h", "block", "post_weight", "gate")}
    ho, none = gpu_lib.norm_gated(**last, pre=False)
    assert none is None
    rh, th, _, _, rows = bounds(last, 1.0, 1e-6, None)
    check(ho, rh, th, rows)
    # in place, the same bits
    h = d["h"].clone()
    want = gpu_lib.norm_gated(**d, residual_scale=-0.25)
    got = gpu_lib.norm_gated(**(d | dict(h=h)), residual_scale=-0.25, h_out=h)
    assert torch.equal(got[0], want[0]) and got[0] is h and torch.equal(got[1], want[1])


def test_zero_and_huge_rows(gpu_lib):
    """A zero row stays zero (eps keeps the factor finite); values near bf16's ends that square beyond
    float32 are outside the documented range and are not tried; 1e15 is inside it."""
    d = make(4, 256, 1, 5)
    d["h"][0] = 0
    d["block"][0] = 0
    d["h"][1] = 1e15
    d["block"][2] = 1e-20
    ho, x = gpu_lib.norm_gated(**d)
    rh, th, rx, tx, rows = bounds(d, 1.0, 1e-6, None)
    check(ho, rh, th, rows)
    check(x, rx, tx, rows)
    assert not x[0].any()
    _, codes, scales = gpu_lib.norm_gated_int8(**d)
    assert not codes[0].any() and scales[0] == 0


@pytest.mark.parametrize("K", [256, 1008, 3840, 10240])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_rows_stay_visible(gpu_lib, K, bad):
    """A NaN or infinity in a row leaves NaN or infinity in it, in the codes' scale too; other rows do not change."""
    d = make(5, K, 1, 6)
    want, want8 = gpu_lib.norm_gated(**d), gpu_lib.norm_gated_int8(**d)
    d["h"][1, K - 1] = bad
    d["block"][3, 0] = bad
    got, got8 = gpu_lib.norm_gated(**d), gpu_lib.norm_gated_int8(**d)
    for w, g in zip(want + want8, got + got8):
        assert torch.equal(w[[0, 2, 4]], g[[0, 2, 4]])
    assert not bool(torch.isfinite(got[1].float()).all(1)[[1, 3]].any())
    assert not bool(torch.isfinite(got8[2])[[1, 3]].any())


@pytest.mark.parametrize("cu", [[3, 3, 10, 40], [0, 0, 0, 0], [50, 50, 50, 50], [0, 64, 64, 64], [7, 20, 20, 64]])
def test_rows_outside_the_groups_are_left(gpu_lib, cu):
    M, K = 64, 528
    d = make(M, K, 3, 8)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ho, x = torch.full_like(d["h"], 7.0), torch.full_like(d["h"], 9.0)
    codes = torch.full((M, K), 5, dtype=torch.int8, device="cuda")
    scales = torch.full((M,), 3.0, device="cuda")
    gpu_lib.norm_gated(**d, cu_seqlens=cut, h_out=ho, x_out=x)
    rh, th, rx, tx, rows = bounds(d, 1.0, 1e-6, cu)
    check(ho, rh, th, rows)
    check(x, rx, tx, rows)
    out = torch.from_numpy(~rows).cuda()
    assert (ho[out] == 7).all() and (x[out] == 9).all()
    gpu_lib.norm_gated_int8(**d, cu_seqlens=cut, h_out=ho, codes=codes, scales=scales)
    assert (codes[out] == 5).all() and (scales[out] == 3).all()


@pytest.mark.parametrize("cu", [[-5, 10, 1 << 30], [40, 10, 64], [64, 0, 64], [0, 100, 30]])
def test_bad_offsets_stay_inside(gpu_lib, cu):
    """Offsets outside 0..M or decreasing: results are unspecified, nothing outside is touched."""
    M, K = 64, 272
    d = make(M, K, 2, 9)
    buf = torch.full((3, M, K), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.norm_gated(**d, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), h_out=buf[1])
    torch.cuda.synchronize()
    assert (buf[0] == 7).all() and (buf[2] == 7).all()


def test_many_groups_and_graph(gpu_lib):
    M, K, G = 700, 256, 333
    d = make(M, K, G, 11)
    cu = np.sort(np.random.default_rng(1).integers(0, M + 1, G + 1))
    cu[0], cu[-1] = 0, M
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    want = gpu_lib.norm_gated(**d, cu_seqlens=cut)
    rh, th, rx, tx, rows = bounds(d, 1.0, 1e-6, cu)
    check(want[0], rh, th, rows)
    check(want[1], rx, tx, rows)
    ho, x = torch.empty_like(want[0]), torch.empty_like(want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.norm_gated(**d, cu_seqlens=cut, h_out=ho, x_out=x)
    for _ in range(4):
        ho.zero_()
        x.zero_()
        gpu_lib.norm_gated(d["h"])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ho, want[0]) and torch.equal(x, want[1])


def test_most_rows(gpu_lib):
    """2^24 rows, sampled."""
    M, K = 1 << 24, 16
    g = torch.Generator(device="cuda").manual_seed(18)
    h, b = (torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ho, x = gpu_lib.norm_gated(h, b, residual_scale=0.5)
    pick = torch.tensor([0, 3, 4, 1 << 20, (1 << 22) + 1, M - 1], device="cuda")
    want = gpu_lib.norm_gated(h[pick], b[pick], residual_scale=0.5)
    assert torch.equal(ho[pick], want[0]) and torch.equal(x[pick], want[1])


def test_offsets_beyond_32_bits(gpu_lib):
    """h, block and the outputs of more than 2^32 bytes each: the last rows as those of a short call."""
    M, K = 140000, 16384
    h = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros_like(h)
    d = make(8, K, 1, 12)
    h[-8:], b[-8:] = d["h"], d["block"]
    want = gpu_lib.norm_gated(**d)
    ho, x = gpu_lib.norm_gated(**(d | dict(h=h, block=b)))
    assert torch.equal(ho[-8:], want[0]) and torch.equal(x[-8:], want[1])
    assert not x[:-8].any()


def test_empty(gpu_lib):
    d = make(1, 32, 1, 1, full=False)
    ho, x = gpu_lib.norm_gated(d["h"][:0], d["block"][:0])
    assert ho.shape == x.shape == (0, 32)
