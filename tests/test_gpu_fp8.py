"""GPU: the linear in 8-bit floating point against the oracle.

Codes and scales bit for bit. y: a block's 128 products are exact in fp32 and added in fp32, each addition
off by at most 2^-23 of the sum of magnitudes (twice half a step, whatever the unit's order); the product
of the two scales and the addition to the result round twice per block (2^-24), partial sums of up to 8 splits
and the bias once each: together below (128 * 2^-23 + (2 P + 12) * 2^-24) mag for P blocks. The matrix instruction
drops low bits of products that are small beside a neighbour; oracle/serving.py derives how much at most. Inputs whose
products stay within 2^7 of each other lose none, and are held to the first bound alone (`narrow`). y is rounded
once to bf16 (2^-8).
"""

import numpy as np
import pytest
import torch

from oracle import serving as S

pytestmark = pytest.mark.gpu


def f64(t):
    return t.float().double().cpu().numpy()


def activations(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randperm(K, generator=g)[: max(1, K // 100)]] *= 20.0
    return x.bfloat16().cuda()


def weights(N, K, seed):
    """Any codes but NaN, any scales."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K), generator=g, dtype=torch.int32).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x31
    scales = torch.rand(-(-N // 128), -(-K // 128), generator=g) * 1e-3 + 1e-5
    return codes.view(torch.float8_e4m3fn).cuda(), scales.cuda(), (torch.randn(N, generator=g) * 0.1).bfloat16().cuda()


def narrow_activations(M, K, seed):
    """Magnitudes in [1, 8): codes of three neighbouring exponents, four after a scale's rounding."""
    g = torch.Generator().manual_seed(seed)
    x = (1 + 6.9 * torch.rand(M, K, generator=g)) * torch.where(torch.rand(M, K, generator=g) < 0.5, -1.0, 1.0)
    return x.bfloat16().cuda()


def narrow_weights(N, K, seed):
    """Codes of four neighbouring exponents (1 to 15)."""
    g = torch.Generator().manual_seed(seed)
    codes = 56 + torch.randint(0, 32, (N, K), generator=g) + 128 * torch.randint(0, 2, (N, K), generator=g)
    _, scales, bias = weights(N, K, seed)
    return codes.to(torch.uint8).view(torch.float8_e4m3fn).cuda(), scales, bias


def check_y(y, codes, ascales, w, ws, bias, rows=None, narrow=False):
    ref, mag, cut = S.gemm(codes, ascales, f64(w), f64(ws), None if bias is None else f64(bias))
    P = -(-codes.shape[1] // 128)
    if bias is not None:
        mag = mag + np.abs(f64(bias))
    err = (128 * 2.0 ** -23 + (2 * P + 12) * 2.0 ** -24) * mag + (0.0 if narrow else cut)
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * err + 1e-38
    got = f64(y) if rows is None else f64(y[rows])
    err = np.abs(got - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (2, 2064), (5, 3840), (17, 4112), (4, 10240), (130, 400), (3, 70000)])
@pytest.mark.parametrize("smooth", [False, True])
def test_quantize_bits(gpu_lib, M, K, smooth):
    print(f"[fp8] quantize {M} {K} smooth={smooth}", flush=True)
    x = activations(M, K, 1)
    sm = (torch.rand(K) + 0.5).bfloat16().cuda() if smooth else None
    for rows, fn in ((1, gpu_lib.quantize_fp8), (128, gpu_lib.quantize_weight_fp8)):
        codes, scales = fn(x, sm)
        rc, e = S.quantize(f64(x), None if sm is None else f64(sm), rows)
        assert np.array_equal(f64(codes), rc)
        assert np.array_equal(f64(scales), 2.0 ** (e.T if rows == 1 else e))


def test_quantize_zero_tiny_tie_and_border_blocks(gpu_lib):
    x = torch.zeros(7, 128)
    x[1, 3] = 2.0 ** -126
    x[2, 5] = 2.0 ** -109 * 1.5            # under the least scale
    x[3, :8] = torch.tensor([448.0, 17.0, 18.0, 19.0, -17.0, 0.0029296875, 0.0009765625, 0.001953125])
    x[4, 0], x[4, 1] = 450.0, 1.0          # above 448: the next power
    x[5, 0] = 3.3895313892515355e38
    x[6] = torch.arange(128) * 3.5
    x = x.bfloat16().cuda()
    codes, scales = gpu_lib.quantize_fp8(x)
    rc, e = S.quantize(f64(x))
    assert np.array_equal(f64(codes), rc) and np.array_equal(f64(scales), 2.0 ** e.T)
    assert scales[0, 0] == 2.0 ** -100 and scales[0, 3] == 1.0 and scales[0, 4] == 2.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("M,K", [(5, 48), (5, 2064), (6, 3840), (40, 512), (300, 400)])
def test_non_finite_tokens_stay_visible(gpu_lib, M, K, bad):
    """A token's block that holds an infinity or NaN has scale NaN, and the token NaN as its y; the others do not change."""
    print(f"[fp8] non-finite {M} {K} {bad}", flush=True)
    w, ws, bias = weights(24, K, 5)
    x = activations(M, K, 6)
    clean_codes, clean_scales = gpu_lib.quantize_fp8(x)
    clean = gpu_lib.linear_fp8(x, w, ws, bias)
    rows, at = [1, 3, 4], (0, K - 1, K // 2)
    for r, k in zip(rows, at):
        x[r, k] = bad
    others = [m for m in range(M) if m not in rows]
    codes, scales = gpu_lib.quantize_fp8(x)
    assert torch.equal(codes[others].view(torch.uint8), clean_codes[others].view(torch.uint8))
    assert torch.equal(scales[:, others], clean_scales[:, others])
    for r, k in zip(rows, at):
        assert bool(torch.isnan(scales[k // 128, r])) and int(torch.isnan(scales[:, r]).sum()) == 1
    for y in (gpu_lib.linear_fp8(x, w, ws, bias), gpu_lib.gemm_fp8(codes, scales, w, ws, bias)):
        assert torch.equal(y[others], clean[others]) and bool(torch.isnan(y[rows]).all())


def test_nan_weight_code_and_scale(gpu_lib):
    for M in (3, 200):
        w, ws, _ = weights(300, 400, 7)
        x = activations(M, 400, 8)
        clean = gpu_lib.linear_fp8(x, w, ws)
        w.view(torch.uint8)[17, 399] = 0x7F
        ws[2, 1] = float("nan")
        y = gpu_lib.linear_fp8(x, w, ws)
        bad = torch.zeros(300, dtype=torch.bool, device="cuda")
        bad[17] = bad[256:] = True
        assert bool(torch.isnan(y[:, bad]).all()) and torch.equal(y[:, ~bad], clean[:, ~bad])


SHAPES = [(1, 16, 1), (1, 3840, 3840), (2, 272, 107), (5, 48, 33), (7, 10240, 65), (8, 5120, 48), (16, 3840, 257),
          (17, 64, 40), (31, 1040, 130), (32, 1280, 50), (33, 96, 64), (48, 3840, 1000), (64, 256, 512), (65, 528, 129),
          (100, 10240, 300), (129, 400, 257), (200, 3840, 1283), (333, 1024, 640), (513, 784, 769), (1000, 272, 96),
          (1030, 2064, 520), (333, 10240, 3840), (1, 40960, 40), (40, 4000, 48), (1500, 1552, 1100), (300, 144, 5000)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("bias", [False, True])
def test_linear_against_oracle(gpu_lib, M, K, N, bias):
    print(f"[fp8] linear {M} {K} {N} bias={bias}", flush=True)
    x = activations(M, K, M + K)
    w, ws, b = weights(N, K, N)
    b = b if bias else None
    sm = (torch.rand(K) + 0.5).bfloat16().cuda()
    y = gpu_lib.linear_fp8(x, w, ws, bias=b, smooth=sm)
    codes, e = S.quantize(f64(x), f64(sm))
    check_y(y, codes, 2.0 ** e.T, w, ws, b)
    # the same through codes, bit for bit
    qc, qs = gpu_lib.quantize_fp8(x, sm)
    assert torch.equal(gpu_lib.gemm_fp8(qc, qs, w, ws, bias=b).view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_of_narrow_values(gpu_lib, M, K, N):
    print(f"[fp8] narrow {M} {K} {N}", flush=True)
    x = narrow_activations(M, K, M + K)
    w, ws, b = narrow_weights(N, K, N)
    codes, e = S.quantize(f64(x))
    check_y(gpu_lib.linear_fp8(x, w, ws, bias=b), codes, 2.0 ** e.T, w, ws, b, narrow=True)


@pytest.mark.parametrize("M", [5, 200])
def test_what_the_matrix_instruction_drops(gpu_lib, M):
    """Products that cancel beside a small one, in its group of 8 and in another: the bound that the oracle states."""
    for near, small, kept in ((2, 2.0 ** 3, True), (2, 2.0 ** 2, False), (8, 2.0 ** -6, True), (127, 2.0 ** -6, True)):
        a, w = torch.zeros(M, 128), torch.zeros(40, 128)
        a[:, 0], a[:, 1], a[:, near] = 256.0, -256.0, 1.0
        w[:, :2], w[:, near] = 256.0, small
        y = gpu_lib.gemm_fp8(a.cuda().to(torch.float8_e4m3fn), torch.ones(1, M, device="cuda"), w.cuda().to(torch.float8_e4m3fn),
                             torch.ones(1, 1, device="cuda"))
        assert bool((y == (small if kept else 0.0)).all()), (near, small)


@pytest.mark.parametrize("M,K,N", [(3, 400, 200), (300, 400, 700), (90, 10240, 64)])
def test_any_activation_scales(gpu_lib, M, K, N):
    codes, _, _ = weights(M, K, 11)
    w, ws, b = weights(N, K, 12)
    scales = (torch.rand(-(-K // 128), M) * 3 + 0.01).cuda()
    scales[0, 0] = -0.75
    y = gpu_lib.gemm_fp8(codes, scales, w, ws, bias=b)
    check_y(y, f64(codes), f64(scales), w, ws, b)
    codes, _, _ = narrow_weights(M, K, 11)
    w, ws, b = narrow_weights(N, K, 12)
    check_y(gpu_lib.gemm_fp8(codes, scales, w, ws, bias=b), f64(codes), f64(scales), w, ws, b, narrow=True)


@pytest.mark.parametrize("M,N,K,rows", [(4096, 10240, 3840, 24), (4000, 3840, 3840, 24), (2048, 11520, 3840, 24),
                                        (8200, 1290, 3840, 40), (2050, 3840, 10240, 16)])
def test_large_sampled_rows(gpu_lib, M, N, K, rows):
    print(f"[fp8] large {M} {N}", flush=True)
    x = activations(M, K, 3)
    w, ws, b = weights(N, K, 4)
    y = gpu_lib.linear_fp8(x, w, ws, b)
    pick = sorted(set(np.random.default_rng(M).integers(0, M, rows)) | {0, 127, 255, 256, M - 1})
    codes, e = S.quantize(f64(x[pick]))
    check_y(y, codes, 2.0 ** e.T, w, ws, b, pick)
    x, (w, ws, b) = narrow_activations(M, K, 3), narrow_weights(N, K, 4)
    codes, e = S.quantize(f64(x[pick]))
    check_y(gpu_lib.linear_fp8(x, w, ws, b), codes, 2.0 ** e.T, w, ws, b, pick, narrow=True)


def test_each_block_meets_its_scales(gpu_lib):
    """Ones in a single block of k at a time: y is that block's scales' product, exactly."""
    for M in (5, 200):
        K, N = 1008, 400
        g = torch.Generator().manual_seed(1)
        ws = (2.0 ** torch.randint(-6, 6, (4, 8), generator=g).float()).cuda()
        scales = (2.0 ** torch.randint(-6, 6, (8, M), generator=g).float()).cuda()
        w = torch.ones(N, K, device="cuda").to(torch.float8_e4m3fn)
        for p in range(8):
            codes = torch.zeros(M, K, device="cuda")
            codes[:, 128 * p + 3] = 1.0
            y = gpu_lib.gemm_fp8(codes.to(torch.float8_e4m3fn), scales, w, ws)
            ref = scales[p][:, None] * ws[:, p].repeat_interleave(128)[:N]
            assert torch.equal(y.float(), ref)


def test_into_given_buffers_on_a_side_stream(gpu_lib):
    M, K, N = 333, 2064, 300
    x, (w, ws, b) = activations(M, K, 1), weights(N, K, 2)
    ref = gpu_lib.linear_fp8(x, w, ws, b)
    base = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = base[32:32 + M * N].view(M, N)
    need = gpu_lib.linear_fp8_workspace_bytes(M, N, K)
    work = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert gpu_lib.linear_fp8(x, w, ws, b, y=y, workspace=work[256:256 + need]) is y
    s.synchronize()
    assert torch.equal(y, ref) and bool((base[:32] == 7).all()) and bool((base[32 + M * N:] == 7).all())
    assert bool((work[:256] == 0xA5).all()) and bool((work[256 + need:] == 0xA5).all())


def test_empty(gpu_lib):
    w, ws, b = weights(40, 64, 1)
    assert gpu_lib.linear_fp8(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w, ws, b).shape == (0, 40)
    x = activations(5, 64, 1)
    none = torch.empty(0, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    assert gpu_lib.linear_fp8(x, none, torch.empty(0, 1, device="cuda")).shape == (5, 0)


def test_graph_replays(gpu_lib):
    """A few-token and a split product captured together, replayed between eager work."""
    cases = []
    for M, K, N in ((1, 3840, 640), (100, 10240, 300), (600, 400, 300)):
        w, ws, b = weights(N, K, M)
        cases.append((activations(M, K, M), w, ws, b, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"),
                      torch.empty(max(1, gpu_lib.linear_fp8_workspace_bytes(M, N, K)), dtype=torch.uint8, device="cuda")))

    def run():
        for x, w, ws, b, y, work in cases:
            gpu_lib.linear_fp8(x, w, ws, b, y=y, workspace=work)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(4):
        for i, c in enumerate(cases):
            c[0].copy_(activations(*c[0].shape, 100 * rep + i))
        ref = [gpu_lib.linear_fp8(x, w, ws, b) for x, w, ws, b, _, _ in cases]
        for c in cases:
            c[4].fill_(0)
            c[5].fill_(0x5A)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(c[4], r) for c, r in zip(cases, ref)), rep
