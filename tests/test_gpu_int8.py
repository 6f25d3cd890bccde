"""GPU: the linear in 8-bit integers against the oracle.

Codes and scales bit for bit. y: the sum over k is exact; its conversion to fp32, the two
scale products and the bias add round four times (2^-24 each, of |main| and |bias|), and y is
rounded once to bf16 (2^-8).
"""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def activations(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randperm(K, generator=g)[: max(1, K // 100)]] *= 20.0
    return x.bfloat16().cuda()


def weights(N, K, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8).cuda(),
            (torch.rand(N, generator=g) * 1e-3 + 1e-5).cuda(), (torch.randn(N, generator=g) * 0.1).bfloat16().cuda())


def check_y(y, codes, scales, w, ws, bias):
    ref, main = B.gemm_int8(codes, scales, f64(w), f64(ws), None if bias is None else f64(bias))
    mag = main + (0.0 if bias is None else np.abs(f64(bias)))
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * 4 * 2.0 ** -24 * mag + 1e-38
    err = np.abs(f64(y) - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (2, 2064), (5, 3840), (17, 4112), (4, 10240), (2, 20000), (3, 70000)])
@pytest.mark.parametrize("smooth", [False, True])
def test_quantize_bits(gpu_lib, M, K, smooth):
    print(f"[int8] quantize {M} {K} smooth={smooth}", flush=True)
    x = activations(M, K, 1)
    sm = (torch.rand(K) + 0.5).bfloat16().cuda() if smooth else None
    codes, scales = gpu_lib.quantize_int8(x, sm)
    rc, rs = B.quantize_int8(f64(x), None if sm is None else f64(sm))
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), rs.view(np.uint32))


def test_quantize_zero_tiny_and_tie_rows(gpu_lib):
    x = torch.zeros(5, 32)
    x[1, 3] = 2.0 ** -126
    x[2, 5] = 2.0 ** -119
    x[3] = torch.arange(32) * 0.5          # ties: maximum 15.5 -> not exact; next row exact halves
    x[4, 0] = 127.0
    x[4, 1:31] = torch.arange(30) + 0.5
    x = x.bfloat16().cuda()
    codes, scales = gpu_lib.quantize_int8(x)
    rc, rs = B.quantize_int8(f64(x))
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    assert codes[4, 1] == 0 and codes[4, 2] == 2 and codes[4, 3] == 2   # to even


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("M,K", [(5, 48), (5, 2064), (6, 3840), (9, 10240), (40, 512), (5, 20000)])
def test_non_finite_rows_stay_visible(gpu_lib, M, K, bad):
    """A row that holds an infinity or NaN has it as its scale and NaN as its y; the other rows do not change."""
    print(f"[int8] non-finite {M} {K} {bad}", flush=True)
    w, ws, bias = weights(24, K, 5)
    x = activations(M, K, 6)
    clean_codes, clean_scales = gpu_lib.quantize_int8(x)
    clean = gpu_lib.linear_int8(x, w, ws, bias)
    rows = [1, 3, 4]
    for r, k in zip(rows, (0, K - 1, K // 2)):
        x[r, k] = bad
    others = [m for m in range(M) if m not in rows]
    codes, scales = gpu_lib.quantize_int8(x)
    assert torch.equal(codes[others], clean_codes[others]) and torch.equal(scales[others], clean_scales[others])
    assert bool((torch.isnan(scales) if bad != bad else torch.isinf(scales))[rows].all())
    for y in (gpu_lib.linear_int8(x, w, ws, bias), gpu_lib.gemm_int8(codes, scales, w, ws, bias)):
        assert torch.equal(y[others], clean[others]) and bool(torch.isnan(y[rows]).all())


SHAPES = [(31, 1312, 70), (29, 1408, 33), (8, 5120, 48), (4, 10240, 40), (32, 1280, 50), (1, 16, 1), (1, 3840, 3840), (2, 272, 107), (5, 48, 33), (7, 10240, 65), (16, 3840, 257), (17, 64, 40),
          (31, 1040, 130), (33, 96, 64), (48, 3840, 1000), (64, 256, 512), (65, 528, 129), (100, 10240, 300),
          (129, 400, 257), (200, 3840, 1283), (333, 1024, 640), (513, 784, 769), (1000, 272, 96), (1030, 2064, 520),
          (333, 10240, 3840), (100, 10000, 300), (1, 40960, 40), (40, 4000, 48)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("bias", [False, True])
def test_linear_against_oracle(gpu_lib, M, K, N, bias):
    print(f"[int8] linear {M} {K} {N} bias={bias}", flush=True)
    x = activations(M, K, M + K)
    w, ws, b = weights(N, K, N)
    b = b if bias else None
    sm = (torch.rand(K) + 0.5).bfloat16().cuda()
    y = gpu_lib.linear_int8(x, w, ws, bias=b, smooth=sm)
    codes, scales = B.quantize_int8(f64(x), f64(sm))
    check_y(y, codes, scales, w, ws, b)
    y2 = gpu_lib.gemm_int8(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), w, ws, bias=b)
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))


@pytest.mark.parametrize("M,N,rows", [(4096, 10240, 24), (4000, 3840, 24), (2048, 11520, 24), (8200, 1290, 40)])
def test_large_sampled_rows(gpu_lib, M, N, rows):
    """Every tile shape of the large products, on sampled rows (first, last and scattered)."""
    K = 1040
    print(f"[int8] large {M} {K} {N}", flush=True)
    x = activations(M, K, 5)
    w, ws, b = weights(N, K, 6)
    y = gpu_lib.linear_int8(x, w, ws, bias=b)
    pick = np.unique(np.concatenate([[0, 1, M - 2, M - 1], np.random.default_rng(0).integers(0, M, rows)]))
    codes, scales = B.quantize_int8(f64(x[torch.from_numpy(pick).cuda()]))
    check_y(y[torch.from_numpy(pick).cuda()], codes, scales, w, ws, b)


# sizes that take each tile shape, with all of k (3 and 9 panels) and with k split; ragged rows and channels
TILES = [(1282, 11167, 272), (1547, 9399, 1040), (397, 8596, 9680), (423, 8360, 10096),
         (964, 10946, 272), (971, 10921, 1040), (197, 11199, 7440), (215, 10896, 8144),
         (388, 11118, 272), (401, 11050, 1040), (4421, 129, 7712), (4369, 136, 10976),
         (263, 10966, 272), (258, 11326, 1040), (5733, 66, 7056), (131, 5984, 4048),
         (646, 10933, 272), (642, 11105, 1040), (129, 11209, 4416), (130, 10960, 5344),
         (131, 10915, 272), (130, 11038, 1040), (67, 4257, 3568), (67, 3400, 6208),
         (65, 8285, 272), (65, 8213, 1040), (2755, 66, 2192), (65, 3056, 2720),
         (33, 60, 1040), (157, 273, 1296), (33, 61, 1200), (36, 72, 1168),
         (389, 5520, 8208), (404, 5385, 8048), (5479, 132, 6960), (5519, 130, 6176), (6699, 72, 6864),
         (6779, 69, 6160), (4171, 72, 4384), (4157, 66, 4544), (66, 2140, 3136), (69, 2054, 3120),
         (81, 60, 1696), (68, 61, 1952)]


@pytest.mark.parametrize("M,K,N", [(1, 3840, 5003), (3, 10240, 4500), (7, 1040, 4999), (16, 10240, 4100), (17, 1296, 6001),
                                   (32, 2048, 8190), (33, 2064, 1300), (48, 1040, 5003), (49, 400, 4097), (64, 2048, 333),
                                   (64, 1024, 9001), (63, 2064, 77), (9, 10240, 640), (24, 10240, 3840), (17, 4112, 4200), (20, 4096, 4096), (16, 48, 20000)])
@pytest.mark.parametrize("smooth", [False, True])
def test_few_tokens_many_channels(gpu_lib, M, K, N, smooth):
    """More channels than 16 for each CU take another kernel; 9 to 64 tokens take tiles above 2^17 codes or 2^24
    weights."""
    print(f"[int8] few {M} {K} {N} smooth={smooth}", flush=True)
    x = activations(M, K, 9)
    w, ws, b = weights(N, K, 10)
    sm = (torch.rand(K) + 0.5).bfloat16().cuda() if smooth else None
    y = gpu_lib.linear_int8(x, w, ws, bias=b, smooth=sm)
    codes, scales = gpu_lib.quantize_int8(x, sm)
    assert torch.equal(gpu_lib.gemm_int8(codes, scales, w, ws, bias=b), y)
    check_y(y, *B.quantize_int8(f64(x), None if sm is None else f64(sm)), w, ws, b)


@pytest.mark.parametrize("M,N,K", TILES)
def test_every_tile_shape(gpu_lib, M, N, K):
    print(f"[int8] tiles {M} {N} {K}", flush=True)
    x = activations(M, K, 7)
    w, ws, b = weights(N, K, 8)
    y = gpu_lib.linear_int8(x, w, ws, bias=b)
    pick = np.unique(np.concatenate([[0, 1, M - 2, M - 1], np.random.default_rng(1).integers(0, M, 20)]))
    at = torch.from_numpy(pick).cuda()
    codes, scales = B.quantize_int8(f64(x[at]))
    check_y(y[at], codes, scales, w, ws, b)


def test_most_rows(gpu_lib):
    """2^24 rows: quantiser and product, sampled."""
    M, K, N = 1 << 24, 16, 8
    g = torch.Generator(device="cuda").manual_seed(16)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    w, ws, b = weights(N, K, 17)
    codes, scales = gpu_lib.quantize_int8(x)
    y = gpu_lib.gemm_int8(codes, scales, w, ws, bias=b)
    pick = torch.tensor([0, 1, 4095, 1 << 20, (1 << 22) + 3, M - 2, M - 1], device="cuda")
    rc, rs = B.quantize_int8(f64(x[pick]))
    assert np.array_equal(codes[pick].cpu().numpy(), rc) and np.array_equal(scales[pick].cpu().numpy(), rs)
    check_y(y[pick], rc, rs, w, ws, b)


def test_offsets_beyond_32_bits(gpu_lib):
    """Codes of more than 2^32 bytes: the last rows as those of a short call."""
    M, K, N = 530000, 8192, 48
    c = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    s = torch.ones(M, device="cuda")
    w, ws, b = weights(N, K, 14)
    x = activations(40, K, 15)
    codes, scales = gpu_lib.quantize_int8(x)
    c[-40:], s[-40:] = codes, scales
    y = gpu_lib.gemm_int8(c, s, w, ws, bias=b)
    check_y(y[-40:], codes.cpu().numpy(), scales.cpu().numpy(), w, ws, b)
    check_y(y[:40], np.zeros((40, K), np.int8), np.ones(40), w, ws, b)


def test_extreme_codes_largest_k(gpu_lib):
    """K = 131072 with codes of +-127 and weights of -128: sums up to 2.13e9, inside int32."""
    K = 131072
    for M, N in ((2, 3), (70, 40)):
        c = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
        c[1] = -127
        w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        w[1] = 127
        s, ws = torch.full((M,), 1e-6, device="cuda"), torch.full((N,), 1e-3, device="cuda")
        y = gpu_lib.gemm_int8(c, s, w, ws)
        check_y(y, c.cpu().numpy(), s.cpu().numpy(), w, ws, None)


def test_outputs_and_workspace_are_used_whole(gpu_lib):
    """Given outputs are filled entirely and nothing outside them; a poisoned workspace does not matter;
    the same call twice gives the same bits."""
    for M, K, N in ((3, 272, 107), (70, 3840, 333), (300, 528, 200)):
        x = activations(M, K, 9)
        w, ws, b = weights(N, K, 10)
        want = gpu_lib.linear_int8(x, w, ws, bias=b)
        need = gpu_lib.linear_int8_workspace_bytes(M, N, K)
        wk = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        buf = torch.full((M * N + 4096,), float("nan"), dtype=torch.bfloat16, device="cuda")
        y = buf[2048:2048 + M * N].view(M, N)
        gpu_lib.linear_int8(x, w, ws, bias=b, y=y, workspace=wk[:need])
        assert torch.equal(y, want)
        assert torch.isnan(buf[:2048]).all() and torch.isnan(buf[2048 + M * N:]).all()
        assert (wk[need:] == 0x5A).all()


def test_side_stream_and_graph(gpu_lib):
    x = activations(40, 1024, 3)
    w, ws, b = weights(300, 1024, 4)
    want = gpu_lib.linear_int8(x, w, ws, bias=b)
    y = torch.empty_like(want)
    wk = torch.empty(gpu_lib.linear_int8_workspace_bytes(40, 300, 1024), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y.zero_()
        gpu_lib.linear_int8(x, w, ws, bias=b, y=y, workspace=wk)
    s.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.linear_int8(x, w, ws, bias=b, y=y, workspace=wk)
    for _ in range(4):
        y.zero_()
        wk.fill_(0x5A)
        gpu_lib.linear_int8(x, w, ws)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_empty(gpu_lib):
    w, ws, _ = weights(8, 32, 1)
    assert gpu_lib.linear_int8(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), w, ws).shape == (0, 8)
    x = activations(4, 32, 1)
    assert gpu_lib.linear_int8(x, w[:0], ws[:0]).shape == (4, 0)
    assert gpu_lib.quantize_int8(x[:0])[0].shape == (0, 32)
