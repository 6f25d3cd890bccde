"""GPU: the operators between the linears run together, as the attention half of a block:

    codes = norm into 8 bits; qkv = 8-bit linear; q, k turned in place; attention; out = 8-bit linear;
    the gated norm back into the residual stream

on packed sequences. Each step is checked against the oracle on the device's own input of that step
(bf16 in, one step's bound), eagerly, and the whole chain replayed from a graph gives the eager bits."""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def test_attention_half_of_a_block(gpu_lib):
    ops = gpu_lib
    H, Hk, D, K = 6, 2, 64, 384
    axes = (16, 24, 24)
    lens = [70, 0, 129, 1]
    T = 210                                      # ten tokens of padding behind the last sequence
    cu = [0, 70, 70, 199, 200]
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    G = len(lens)
    h = rnd(T, K).bfloat16().cuda()
    pre, post, pre2, qw, kw = ((1 + 0.1 * rnd(n)).bfloat16().cuda() for n in (K, K, K, D, D))
    scale, gate, scale2 = (0.3 * rnd(G, K)).bfloat16().cuda(), rnd(G, K).tanh().bfloat16().cuda(), \
        (0.3 * rnd(G, K)).bfloat16().cuda()
    w1, ws1 = ops.quantize_int8((0.02 * rnd((H + 2 * Hk) * D, K)).bfloat16().cuda())
    w2, ws2 = ops.quantize_int8((0.02 * rnd(K, H * D)).bfloat16().cuda())
    bias = (0.01 * rnd(K)).bfloat16().cuda()
    pos = torch.stack([torch.arange(T) % 7, torch.arange(T) // 7, torch.arange(T) % 13], 1).to(torch.int32).cuda()

    codes = torch.zeros(T, K, dtype=torch.int8, device="cuda")
    cscale = torch.zeros(T, device="cuda")
    qkv = torch.empty(T, (H + 2 * Hk) * D, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    h2, x2 = torch.zeros_like(h), torch.zeros_like(h)
    need = max(ops.gemm_int8_workspace_bytes(T, qkv.shape[1], K), ops.linear_int8_workspace_bytes(T, K, H * D), 1)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    q, k, v = (t.view(T, -1, D) for t in qkv.split([H * D, Hk * D, Hk * D], 1))
    kept = {}

    def half(keep=False):
        ops.norm_gated_int8(h, pre_weight=pre, scale=scale, cu_seqlens=cut, codes=codes, scales=cscale)
        ops.gemm_int8(codes, cscale, w1, ws1, y=qkv, workspace=work)
        if keep:
            kept["qkv"] = qkv.clone()
        ops.rope_axes(q, k, pos, axes, theta=256.0, q_weight=qw, k_weight=kw, q_out=q, k_out=k)
        ops.attention_packed(q, k, v, cut, out=o)
        ops.linear_int8(o.view(T, H * D), w2, ws2, bias=bias, y=y, workspace=work)
        ops.norm_gated(h, y, post_weight=post, gate=gate, pre_weight=pre2, scale=scale2, cu_seqlens=cut, h_out=h2,
                       x_out=x2)

    half(keep=True)
    torch.cuda.synchronize()
    r = slice(0, 200)
    e = (K / 2 + 8) * 2.0 ** -24
    # norm into codes: as if the bf16 x had been written and quantised
    x = ops.norm_gated(h, pre_weight=pre, scale=scale, cu_seqlens=cut)[1]
    _, rx, _, _, _ = B.norm_gated(f64(h), None, None, None, 1.0, f64(pre), f64(scale), cu)
    assert (np.abs(f64(x) - rx)[r] <= (2.0 ** -8 + 2 * e) * np.abs(rx)[r] + 1e-30).all()
    rc, rs = B.quantize_int8(f64(x)[r])
    assert np.array_equal(codes.cpu().numpy()[r], rc) and np.array_equal(cscale.cpu().numpy()[r], rs)
    # qkv
    ref, main = B.gemm_int8(rc, rs, f64(w1), f64(ws1))
    assert (np.abs(f64(kept["qkv"])[r] - ref) <= 2.0 ** -8 * np.abs(ref) + 5 * 2.0 ** -24 * main + 1e-30).all()
    # rotary
    z = f64(kept["qkv"]).reshape(T, -1, D)
    for got, zin, w in ((q, z[:, :H], qw), (k, z[:, H:H + Hk], kw)):
        ref, mag = B.rope_axes(zin, pos.cpu().numpy(), axes, 256.0, True, f64(w))
        assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (6e-7 + (D / 2 + 10) * 2.0 ** -24) * 1.01 * mag).all()
    # attention
    ref, tol, rows = B.attention_packed(f64(q), f64(k), f64(v), cu)
    assert (np.abs(f64(o) - ref)[rows] <= ((1 + 2.0 ** -8) * tol + 2.0 ** -8 * np.abs(ref))[rows]).all()
    assert not o[200:].any()
    # out projection
    rc, rs = B.quantize_int8(f64(o).reshape(T, -1))
    ref, main = B.gemm_int8(rc, rs, f64(w2), f64(ws2), f64(bias))
    mag = main + np.abs(f64(bias))
    assert (np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 5 * 2.0 ** -24 * mag + 1e-30).all()
    # back into the residual stream
    rh, rx, added, factor, rows = B.norm_gated(f64(h), f64(y), f64(post), f64(gate), 1.0, f64(pre2), f64(scale2), cu)
    dh = e * np.abs(added) + 2.0 ** -24 * np.abs(rh)
    assert (np.abs(f64(h2) - rh)[rows] <= (2.0 ** -8 * (np.abs(rh) + dh) + dh)[rows]).all()
    assert not h2[200:].any()

    want = {n: t.clone() for n, t in dict(qkv=qkv, o=o, h2=h2, x2=x2).items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        half()
    for _ in range(4):
        for t in (qkv, o, h2, x2, y, codes, cscale):
            t.zero_()
        work.fill_(0x5A)
        ops.linear_int8(h, w1, ws1)              # unrelated eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in dict(o=o, h2=h2, x2=x2).items():
            assert torch.equal(t, want[n]), n
        assert torch.equal(qkv[r], want["qkv"][r])
