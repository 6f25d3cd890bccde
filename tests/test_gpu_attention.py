"""GPU: attention over packed sequences against the oracle in float64, element by element within the bound
that oracle/block.py derives (fp32 scores and sums, probabilities rounded to bf16), plus the output's own
bf16 rounding (2^-8)."""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def make(T, H, Hk, D, seed, sharp=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, H, D, generator=g) * sharp).bfloat16().cuda()
    k = torch.randn(T, Hk, D, generator=g).bfloat16().cuda()
    v = torch.randn(T, Hk, D, generator=g).bfloat16().cuda()
    return q, k, v


def offsets(lens, start=0):
    return [int(c) for c in np.cumsum([start] + list(lens))]


def dev(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def check(o, q, k, v, cu=None, causal=False, scale=None, queries=None):
    ref, tol, rows = B.attention_packed(f64(q), f64(k), f64(v), cu, causal, scale, queries)
    tol = (1 + 2.0 ** -8) * tol + 2.0 ** -8 * np.abs(ref)
    err = np.abs(f64(o) - ref)[rows]
    assert (err <= tol[rows]).all(), float((err / tol[rows]).max())
    return torch.from_numpy(rows).cuda()


LENGTHS = [[1], [2], [31, 33], [64], [65], [5, 0, 64, 1, 200], [127, 129], [256], [257], [300, 513], [1000], [0, 0, 3, 0],
           [1] * 70, [17] * 150 + [0] * 20 + [400]]


@pytest.mark.parametrize("lens", LENGTHS, ids=lambda x: "-".join(map(str, x[:6])))
@pytest.mark.parametrize("H,Hk,D", [(4, 2, 128), (3, 3, 64), (5, 1, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_against_oracle(gpu_lib, lens, H, Hk, D, causal):
    print(f"[attention] {lens[:6]} H={H} Hk={Hk} D={D} causal={causal}", flush=True)
    T = sum(lens)
    q, k, v = make(T, H, Hk, D, T + D)
    cu = offsets(lens)
    o = gpu_lib.attention_packed(q, k, v, dev(cu), causal=causal)
    check(o, q, k, v, cu, causal)
    if len(lens) == 1:
        assert torch.equal(gpu_lib.attention_packed(q, k, v, causal=causal), o)


@pytest.mark.parametrize("T,H,Hk,D,causal", [(2500, 2, 1, 128, False), (2500, 2, 2, 64, True), (4100, 1, 1, 128, True)])
def test_long(gpu_lib, T, H, Hk, D, causal):
    print(f"[attention] long {T}", flush=True)
    q, k, v = make(T, H, Hk, D, 3)
    check(gpu_lib.attention_packed(q, k, v, causal=causal), q, k, v, None, causal)


@pytest.mark.parametrize("T,H,Hk,D", [(8192, 1, 1, 128), (8300, 2, 1, 64), (9001, 4, 1, 128), (16700, 3, 3, 64)])
@pytest.mark.parametrize("causal", [False, True])
def test_longest_sampled_queries(gpu_lib, T, H, Hk, D, causal):
    """Mean lengths from 8192 on take eight waves per workgroup; sampled queries, ends and tile borders."""
    print(f"[attention] longest {T} causal={causal}", flush=True)
    q, k, v = make(T, H, Hk, D, T)
    pick = np.unique(np.concatenate([[0, 1, 63, 64, 255, 256, T - 257, T - 65, T - 2, T - 1],
                                     np.random.default_rng(T).integers(0, T, 40)]))
    check(gpu_lib.attention_packed(q, k, v, causal=causal), q, k, v, None, causal, None, pick)


def test_two_long_sequences_eight_waves(gpu_lib):
    cu = offsets([9000, 8100], 3)
    T = cu[-1] + 2
    q, k, v = make(T, 2, 1, 128, 21)
    o = torch.full_like(q, 7.0)
    pick = np.array([3, 4, 9002, 9003, 9004, 9300, T - 3, 5000])
    gpu_lib.attention_packed(q, k, v, dev(cu), causal=True, out=o)
    check(o, q, k, v, cu, True, None, pick)
    assert (o[:3] == 7).all() and (o[-2:] == 7).all()


def test_thousands_of_sequences(gpu_lib):
    """More sequences than 64 * 64 lanes probe in two rounds; lengths 0 to 5."""
    lens = np.random.default_rng(3).integers(0, 6, 5000).tolist()
    cu = offsets(lens)
    q, k, v = make(cu[-1], 2, 2, 64, 22)
    o = gpu_lib.attention_packed(q, k, v, dev(cu), causal=True)
    check(o, q, k, v, cu, True)


@pytest.mark.parametrize("H,Hk", [(6, 1), (8, 1), (16, 1), (12, 2), (24, 8)])
@pytest.mark.parametrize("D,causal", [(128, True), (64, False)])
def test_head_groups(gpu_lib, H, Hk, D, causal):
    """Groups that fill a workgroup's waves, do not divide them, or exceed them."""
    lens = [70, 1, 200, 33]
    q, k, v = make(sum(lens), H, Hk, D, 24)
    cu = offsets(lens)
    check(gpu_lib.attention_packed(q, k, v, dev(cu), causal=causal), q, k, v, cu, causal)


@pytest.mark.parametrize("H,Hk", [(8, 1), (12, 2)])
def test_head_groups_eight_waves(gpu_lib, H, Hk):
    T = 8200
    q, k, v = make(T, H, Hk, 64, 25)
    pick = np.array([0, 31, 32, 63, 100, 4111, T - 33, T - 1])
    check(gpu_lib.attention_packed(q, k, v, causal=True), q, k, v, None, True, None, pick)


def test_most_tokens_and_sequences(gpu_lib):
    """T = 2^24 - 1 tokens in 65535 sequences: the last ones as those of a call of their own."""
    T, B, D = (1 << 24) - 1, 65535, 64
    g = torch.Generator(device="cuda").manual_seed(26)
    q, k, v = (torch.randn(T, 1, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    cu = (torch.arange(B + 1, device="cuda") * (T // B)).to(torch.int32)
    cu[-1] = T
    o = gpu_lib.attention_packed(q, k, v, cu, causal=True)
    for b in (0, 1, 63, 64, 40000, B - 1):
        r = slice(int(cu[b]), int(cu[b + 1]))
        one = gpu_lib.attention_packed(q[r], k[r], v[r], causal=True)
        assert torch.equal(o[r], one), b


def test_offsets_beyond_32_bits(gpu_lib):
    """A token stride of 2^20 elements: the last tokens lie more than 2^32 bytes in."""
    T, H, D, st = 2100, 1, 128, 1 << 20
    q, k, v = make(T, H, H, D, 23)
    buf = torch.empty(T * st, dtype=torch.bfloat16, device="cuda")
    views = [torch.as_strided(buf, (T, H, D), (st, D, 1), 512 * i) for i in range(4)]
    for dst, src in zip(views, (q, k, v)):
        dst.copy_(src)
    gpu_lib.attention_packed(*views[:3], out=views[3])
    assert torch.equal(views[3], gpu_lib.attention_packed(q, k, v))


@pytest.mark.parametrize("sharp", [8.0, 60.0])
@pytest.mark.parametrize("causal", [False, True])
def test_peaked_and_growing_scores(gpu_lib, sharp, causal):
    """Scores up to hundreds: the running maximum moves by more than any fixed step, in every tile."""
    T, D = 700, 128
    q, k, v = make(T, 2, 2, D, 5, sharp)
    ramp = torch.linspace(0.1, 3.0, T, device="cuda")[:, None, None]
    k = (k * ramp).bfloat16()
    check(gpu_lib.attention_packed(q, k, v, causal=causal), q, k, v, None, causal)
    k2 = torch.flip(k, [0])
    check(gpu_lib.attention_packed(q, k2, v, causal=causal), q, k2, v, None, causal)


@pytest.mark.parametrize("scale", [1e-6, 0.02, 1.0])
def test_scales_and_equal_scores(gpu_lib, scale):
    q, k, v = make(200, 2, 1, 64, 6)
    check(gpu_lib.attention_packed(q, k, v, scale=scale), q, k, v, None, False, scale)
    z = torch.zeros_like(q)
    check(gpu_lib.attention_packed(z, k, v, scale=scale, causal=True), z, k, v, None, True, scale)


@pytest.mark.parametrize("D", [64, 128])
def test_strided_views(gpu_lib, D):
    """A fused qkv buffer, head-major storage, and a padded output."""
    T, H, Hk = 333, 6, 2
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn(T, (H + 2 * Hk) * D, generator=g).bfloat16().cuda()
    q = qkv[:, : H * D].view(T, H, D)
    k = qkv[:, H * D: (H + Hk) * D].view(T, Hk, D)
    v = qkv[:, (H + Hk) * D:].view(T, Hk, D)
    cu = offsets([100, 233])
    want = gpu_lib.attention_packed(q.contiguous(), k.contiguous(), v.contiguous(), dev(cu))
    out = torch.full((T, H + 1, D + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.attention_packed(q, k, v, dev(cu), out=out[:, :H, :D])
    assert torch.equal(out[:, :H, :D], want)
    assert (out[:, H] == 3).all() and (out[:, :, D:] == 3).all()
    qh, kh, vh = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    oh = torch.empty(H, T, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    gpu_lib.attention_packed(qh, kh, vh, dev(cu), out=oh)
    assert torch.equal(oh, want)
    check(want, q, k, v, cu)


@pytest.mark.parametrize("causal", [False, True])
def test_rows_outside_the_sequences_are_left(gpu_lib, causal):
    T = 500
    q, k, v = make(T, 3, 1, 128, 8)
    for cu in ([0, 100, 400], [37, 37, 300], [500, 500, 500], [0, 0, 0], [130, 131, 131, 490]):
        o = torch.full_like(q, 7.0)
        gpu_lib.attention_packed(q, k, v, dev(cu), causal=causal, out=o)
        rows = check(o, q, k, v, cu, causal)
        assert (o[~rows] == 7).all()


@pytest.mark.parametrize("causal", [False, True])
def test_other_sequences_values_do_not_leak(gpu_lib, causal):
    """Infinities and NaN in the neighbours, and behind the last sequence."""
    q, k, v = make(400, 2, 2, 128, 9)
    cu = offsets([90, 110, 130])
    want = gpu_lib.attention_packed(q, k, v, dev(cu), causal=causal)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").bfloat16()
    for t in (q, k, v):
        t[:90] = bad[0]
        t[200:] = bad[1]
        t[250:] = bad[2]
        t[330:] = bad[0]
    got = gpu_lib.attention_packed(q, k, v, dev(cu), causal=causal)
    assert torch.equal(got[90:200], want[90:200])


@pytest.mark.parametrize("cu", [[-9, 50, 1 << 30], [300, 20, 200], [200, 0, 200], [0, 5000, 100], [-1, -1, -1]])
def test_bad_offsets_stay_inside(gpu_lib, cu):
    """Offsets outside 0..T or decreasing: results are unspecified, nothing outside is touched."""
    T = 200
    q, k, v = make(T, 2, 1, 64, 10)
    buf = torch.full((3, T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.attention_packed(q, k, v, dev(cu), out=buf[1])
    torch.cuda.synchronize()
    assert (buf[0] == 7).all() and (buf[2] == 7).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cu", [[0, 100, 200, 0, 300], [250, 300, 0, 200, 100, 300], [100, 200, 300, 0, 40, 300]])
def test_decreasing_offsets_stay_inside(gpu_lib, cu, causal):
    """Tiles are numbered by the offsets: decreasing ones can name a tile before its sequence's start. What
    stands around the output stays, and every written row is a mean of values of the tensor."""
    T, H, D, pad = 300, 2, 64, 400
    q, k, _ = make(T, H, H, D, 21)
    v = torch.full_like(k, 0.75)
    buf = torch.full((T + 2 * pad, H, D), 3.0, device="cuda", dtype=torch.bfloat16)
    gpu_lib.attention_packed(q, k, v, dev(cu), causal=causal, out=buf[pad:pad + T])
    assert bool((buf[:pad] == 3.0).all()) and bool((buf[pad + T:] == 3.0).all())
    mid = buf[pad:pad + T]
    assert bool(((mid == 3.0) | ((mid - 0.75).abs() <= 2.0 ** -7)).all())


@pytest.mark.parametrize("T", [1, 70, 300])
def test_far_negative_scores(gpu_lib, T):
    """Equal scores of -1.3e34 (q k^T = -128 * 1e16 * 1e16): the mean of the values, as for any equal scores.
    Probabilities are exactly 1, so only the fp32 sums (T 2^-24 of the magnitudes) and one rounding remain."""
    _, _, v = make(T, 2, 2, 128, 22)
    q = torch.full_like(v, 1e16)
    o = gpu_lib.attention_packed(q, -q, v)
    ref = f64(v).mean(0, keepdims=True)
    tol = 2.0 ** -8 * np.abs(ref) + 2 * T * 2.0 ** -24 * np.abs(f64(v)).mean(0, keepdims=True)
    assert (np.abs(f64(o) - ref) <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
def test_one_token_with_infinite_values(gpu_lib, D):
    """A sequence of one token answers with that token's values, infinities included."""
    q, k, v = make(1, 2, 2, D, 23)
    v[0, 0, 3], v[0, 1, 5] = float("inf"), float("-inf")
    for cu in (None, dev([0, 1])):
        assert torch.equal(gpu_lib.attention_packed(q, k, v, cu), v)


def test_repeats_streams_and_graph(gpu_lib):
    q, k, v = make(600, 4, 2, 128, 11)
    cu = dev(offsets([250, 1, 349]))
    want = gpu_lib.attention_packed(q, k, v, cu, causal=True)
    assert torch.equal(gpu_lib.attention_packed(q, k, v, cu, causal=True), want)
    o = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o.zero_()
        gpu_lib.attention_packed(q, k, v, cu, causal=True, out=o)
    s.synchronize()
    assert torch.equal(o, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.attention_packed(q, k, v, cu, causal=True, out=o)
    for _ in range(4):
        o.zero_()
        gpu_lib.attention_packed(q, k, v, cu)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)


def test_empty(gpu_lib):
    q, k, v = make(4, 2, 1, 64, 12)
    assert gpu_lib.attention_packed(q[:0], k[:0], v[:0]).shape == (0, 2, 64)
    o = torch.full_like(q, 2.0)
    gpu_lib.attention_packed(q, k, v, dev([2]), out=o)
    assert (o == 2).all()
