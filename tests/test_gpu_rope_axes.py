"""GPU: rotary positions with several axes against the oracle in float64.

Error: the angle is reduced in fp64 and rounded to fp32 as a fraction of a turn (2^-26 turns = 9.4e-8
rad), cosine and sine are within 2 units (2.4e-7), the rotation rounds three times (1.8e-7): together below
6e-7 (|u| + |w|) for a pair; the norm adds (D / 2 + 10) 2^-24 of it; bf16 rounds once (2^-8).
"""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(got, z, pos, axes, theta, inter, w, eps=1e-6):
    D = z.shape[2]
    ref, mag = B.rope_axes(f64(z), pos.cpu().numpy(), axes, theta, inter, f64(w), eps)
    e = 6e-7 + (0 if w is None else (D / 2 + 10) * 2.0 ** -24)
    tol = 2.0 ** -8 * np.abs(ref) + 1.01 * e * mag + 2.0 ** -133
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), float((err / tol).max())


def positions(T, A, far, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-far, far + 1, (T, A), generator=g, dtype=torch.int64).to(torch.int32).cuda()


@pytest.mark.parametrize("T,H,Hk,D,axes", [
    (1, 1, 1, 128, (32, 48, 48)), (77, 30, 30, 128, (32, 48, 48)), (5, 3, 1, 64, (16, 24, 24)), (300, 7, 2, 64, (64,)),
    (33, 32, 8, 128, (128,)), (64, 5, 5, 128, (2, 6, 118, 2)), (9, 40, 3, 64, (32, 32)), (3, 100, 7, 128, (64, 64)), (1025, 4, 4, 128, (16, 56, 56))])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_against_oracle(gpu_lib, T, H, Hk, D, axes, inter, norm):
    print(f"[rope] {T} {H} {Hk} {D} {axes} inter={inter} norm={norm}", flush=True)
    g = torch.Generator().manual_seed(T + D)
    qkv = torch.randn(T, (H + 2 * Hk) * D, generator=g).bfloat16().cuda()
    q = qkv[:, : H * D].view(T, H, D)
    k = qkv[:, H * D: (H + Hk) * D].view(T, Hk, D)
    qw = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16().cuda() if norm else None
    kw = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16().cuda() if norm else None
    pos = positions(T, len(axes), 4000, T)
    qo, ko = gpu_lib.rope_axes(q, k, pos, axes, theta=10000.0, interleaved=inter, q_weight=qw, k_weight=kw)
    check(qo, q, pos, axes, 10000.0, inter, qw)
    check(ko, k, pos, axes, 10000.0, inter, kw)
    # in place inside the fused buffer: the same bits, and v is left alone
    again = qkv.clone()
    q2, k2 = again[:, : H * D].view(T, H, D), again[:, H * D: (H + Hk) * D].view(T, Hk, D)
    gpu_lib.rope_axes(q2, k2, pos, axes, theta=10000.0, interleaved=inter, q_weight=qw, k_weight=kw, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    assert torch.equal(again[:, (H + Hk) * D:], qkv[:, (H + Hk) * D:])


def test_far_positions(gpu_lib):
    """Positions to the ends of int32: an fp32 product would lose the phase altogether."""
    T, D, axes = 64, 128, (64, 64)
    q = torch.randn(T, 2, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    pos = positions(T, 2, 2 ** 31 - 1, 2)
    pos[0] = torch.tensor([2 ** 31 - 1, -2 ** 31])
    for theta in (1.0, 256.0, 1e6):
        qo, none = gpu_lib.rope_axes(q, None, pos, axes, theta=theta)
        assert none is None
        # fp64: 2^31 turns at 2^-53 relative, twice (the oracle's own angle too): 2^31 * 2^-52 * 2 pi = 3e-6
        ref, mag = B.rope_axes(f64(q), pos.cpu().numpy(), axes, theta)
        tol = 2.0 ** -8 * np.abs(ref) + (6e-7 + 2 * 3e-6) * mag
        assert (np.abs(f64(qo) - ref) <= tol).all()


def test_strides_and_sides(gpu_lib):
    """Head-major storage, padded tokens, outputs of another layout, q or k alone."""
    T, H, D, axes = 37, 6, 64, (16, 24, 24)
    g = torch.Generator().manual_seed(4)
    pos = positions(T, 3, 100, 5)
    base = torch.randn(H, T, D, generator=g).bfloat16().cuda()
    q = base.transpose(0, 1)
    wide = torch.randn(T, H, D + 16, generator=g).bfloat16().cuda()
    k = wide[:, :, 8:8 + D]
    qo = torch.full((T, H, D + 8), 5.0, dtype=torch.bfloat16, device="cuda")[:, :, :D]
    ko = torch.full((H + 1, T, D), 5.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.rope_axes(q, k, pos, axes, q_out=qo, k_out=ko[:H].transpose(0, 1))
    check(qo, q, pos, axes, 10000.0, True, None)
    check(ko[:H].transpose(0, 1), k, pos, axes, 10000.0, True, None)
    assert (ko[H] == 5).all() and (qo.as_strided((T, H, 8), (H * (D + 8), D + 8, 1), D) == 5).all()
    only_q, _ = gpu_lib.rope_axes(q, None, pos, axes)
    _, only_k = gpu_lib.rope_axes(None, k, pos, axes)
    assert torch.equal(only_q, qo) and torch.equal(only_k, ko[:H].transpose(0, 1))
    one = q[:1].expand(1, H, D)
    assert torch.equal(gpu_lib.rope_axes(one, None, pos[:1], axes)[0], qo[:1])


def test_norm_on_one_side(gpu_lib):
    g = torch.Generator().manual_seed(8)
    q, k = torch.randn(21, 3, 128, generator=g).bfloat16().cuda(), torch.randn(21, 2, 128, generator=g).bfloat16().cuda()
    w = (1 + 0.1 * torch.randn(128, generator=g)).bfloat16().cuda()
    pos = positions(21, 1, 50, 9)
    for qw, kw in ((w, None), (None, w)):
        qo, ko = gpu_lib.rope_axes(q, k, pos, (128,), q_weight=qw, k_weight=kw, eps=1e-5)
        check(qo, q, pos, (128,), 10000.0, True, qw, 1e-5)
        check(ko, k, pos, (128,), 10000.0, True, kw, 1e-5)


def test_zero_heads_rows_and_eps(gpu_lib):
    """A head of zeros stays zero through the norm."""
    q = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    qo, _ = gpu_lib.rope_axes(q, None, positions(5, 1, 9, 1), (64,), q_weight=w)
    assert not qo.any()


@pytest.mark.parametrize("D,axes", [(64, (16, 24, 24)), (128, (32, 48, 48))])
@pytest.mark.parametrize("inter", [True, False])
def test_tiny_and_huge_heads(gpu_lib, D, axes, inter):
    """Mean squares among fp32's denormals (eps 0; 2^-64 squared is 2^-128), at the border of the fast square
    root, and up to 1e34: the norm's bound holds relative to the result for all of them. A sum of D denormal
    squares rounds to multiples of 2^-149, D 2^-150 of 2^-128 D here: 2^-22 of it."""
    T, H = 12, 5
    z = torch.randn(T, H, D, generator=torch.Generator().manual_seed(3))
    for h, size in enumerate((2.0 ** -64, 1e-15, 1.0, 1e8, 1e17)):
        z[:, h] *= size
    z = z.bfloat16().cuda()
    w = (1 + 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(4))).bfloat16().cuda()
    pos = positions(T, 3, 300, 5)
    zo, _ = gpu_lib.rope_axes(z, None, pos, axes, interleaved=inter, q_weight=w, eps=0.0)
    ref, mag = B.rope_axes(f64(z), pos.cpu().numpy(), axes, 10000.0, inter, f64(w), 0.0)
    tol = 2.0 ** -8 * np.abs(ref) + (6e-7 + (D / 2 + 10) * 2.0 ** -24 + 2.0 ** -22) * 1.01 * mag
    assert (np.abs(f64(zo) - ref) <= tol).all()


def test_non_finite_heads(gpu_lib):
    """A NaN makes its own head NaN under the norm and reaches no other head or token."""
    T, H, D, axes = 6, 4, 128, (64, 64)
    z = torch.randn(T, H, D, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    pos = positions(T, 2, 50, 7)
    want, _ = gpu_lib.rope_axes(z, None, pos, axes, q_weight=w)
    z[2, 1, 77] = float("nan")
    got, _ = gpu_lib.rope_axes(z, None, pos, axes, q_weight=w)
    assert bool(torch.isnan(got[2, 1]).all())
    rest = torch.ones(T, H, dtype=torch.bool, device="cuda")
    rest[2, 1] = False
    assert torch.equal(got[rest], want[rest])


def test_most_tokens(gpu_lib):
    T = (1 << 24) - 1
    q = torch.randn(T, 1, 64, generator=torch.Generator(device="cuda").manual_seed(12), device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)[:, None].contiguous()
    qo, _ = gpu_lib.rope_axes(q, None, pos, (64,))
    pick = torch.tensor([0, 15, 16, 1 << 20, T - 2, T - 1], device="cuda")
    assert torch.equal(qo[pick], gpu_lib.rope_axes(q[pick], None, pos[pick], (64,))[0])


def test_offsets_beyond_32_bits(gpu_lib):
    T, st, axes = 2100, 1 << 20, (64, 64)
    q = torch.randn(T, 1, 128, generator=torch.Generator().manual_seed(10)).bfloat16().cuda()
    pos = positions(T, 2, 300, 11)
    buf = torch.empty(T * st, dtype=torch.bfloat16, device="cuda")
    src, dst = (torch.as_strided(buf, (T, 1, 128), (st, 128, 1), 512 * i) for i in range(2))
    src.copy_(q)
    gpu_lib.rope_axes(src, None, pos, axes, q_out=dst)
    assert torch.equal(dst, gpu_lib.rope_axes(q, None, pos, axes)[0])


def test_graph_and_empty(gpu_lib):
    T, axes = 50, (32, 48, 48)
    q = torch.randn(T, 4, 128, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    pos = positions(T, 3, 300, 7)
    want, _ = gpu_lib.rope_axes(q, None, pos, axes)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.rope_axes(q, None, pos, axes, q_out=out)
    for _ in range(4):
        out.zero_()
        gpu_lib.rope_axes(q, q, pos, axes, theta=5.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    e, _ = gpu_lib.rope_axes(q[:0], None, pos[:0], axes)
    assert e.shape == (0, 4, 128)
