"""GPU: the serving operators together, as a decoder's attention half uses them: the 8-bit linear for q, k and v,
scaled rotary positions in place, appending to the cache, attention over it, the output linear. Prompts in chunks,
then tokens; the whole run in a graph for the tokens. Against the same steps in float64 from the oracle, which
takes each step's bf16 results as they are rounded on the device, so that every step's own bound holds."""

import numpy as np
import pytest
import torch

from oracle import serving as S

pytestmark = pytest.mark.gpu


def f64(t):
    return t.float().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Block:
    def __init__(self, lib, H=8, Hk=2, D=64, K=512, page=16, pages=60, width=12, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.lib, self.H, self.Hk, self.D, self.K = lib, H, Hk, D, K
        self.qkv = lib.quantize_weight_fp8((torch.randn((H + 2 * Hk) * D, K, generator=g) * K ** -0.5).bfloat16().cuda())
        self.out = lib.quantize_weight_fp8((torch.randn(K, H * D, generator=g) * 0.1).bfloat16().cuda())
        self.cache = lib.new_cache_fp8(pages, Hk, D, page)
        for t in (self.cache.k_codes, self.cache.v_codes, self.cache.k_scales, self.cache.v_scales):
            t.view(torch.uint8).fill_(0xFF)
        self.table = i32(np.random.default_rng(seed).permutation(pages).reshape(-1, width).tolist())

    def step(self, x, positions, before, after, cu=None):
        lib, H, Hk, D = self.lib, self.H, self.Hk, self.D
        T = x.shape[0]
        qkv = lib.linear_fp8(x, *self.qkv).view(T, H + 2 * Hk, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        raw = qkv.clone() if self.keep else None
        lib.rope_scaled(q, k, positions, rotary_dim=D // 2, factor=4.0, original_length=64, q_out=q, k_out=k)
        lib.cache_append_fp8(k, v, self.cache, self.table, before, cu)
        o = lib.attention_cache_fp8(q, self.cache, self.table, after, cu)
        y = lib.linear_fp8(o.view(T, H * D), *self.out)
        self.seen = (raw, qkv, o)
        return y

    keep = True


def check_step(blk, x, y, oracle, before, new, cu):
    raw, qkv, o = blk.seen
    H, Hk, D = blk.H, blk.Hk, blk.D

    def linear(a, got, w):
        codes, e = S.quantize(f64(a))
        ref, mag, cut = S.gemm(codes, 2.0 ** e.T, f64(w[0]), f64(w[1]))
        P = e.shape[1]
        tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((128 * 2.0 ** -23 + (2 * P + 12) * 2.0 ** -24) * mag + cut) + 1e-38
        assert (np.abs(f64(got) - ref) <= tol).all()

    T = x.shape[0]
    linear(x, raw.view(T, -1), blk.qkv)
    pos = np.concatenate([b + np.arange(n) for b, n in zip(before, new)])
    for part in (slice(0, H), slice(H, H + Hk)):
        ref, mag, far = S.rope(f64(raw[:, part]), pos, D // 2, factor=4.0, original=64)
        assert (np.abs(f64(qkv[:, part]) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * (7e-7 + 2.0 ** -51 * far) * mag).all()
    assert torch.equal(qkv[:, H + Hk:], raw[:, H + Hk:])
    table = blk.table.tolist()
    oracle.append({"k": f64(qkv[:, H:H + Hk]), "v": f64(qkv[:, H + Hk:])}, table, before, cu)
    kv = [oracle.values(n) for n in "kv"]
    for b, n in enumerate(new):
        if n == 0:
            continue
        r = slice(cu[b], cu[b + 1])
        L = before[b] + n
        k, v = (S.gather(z, table[b], oracle.page, 0, L) for z in kv)
        ref, tol = S.attention(f64(qkv[r, :H]), k, v, n)
        assert (np.abs(f64(o[r]) - ref) <= (1 + 2.0 ** -8) * tol + 2.0 ** -8 * np.abs(ref)).all(), b
    linear(o.view(T, -1), y, blk.out)


def test_chunks_then_tokens(gpu_lib):
    blk = Block(gpu_lib)
    oracle = S.Cache(60, blk.Hk, 16, blk.D)
    held = [0] * 5
    g = torch.Generator().manual_seed(1)
    for new in ([30, 1, 17, 0, 64], [20, 40, 1, 5, 33], [1] * 5, [1] * 5, [1, 1, 0, 1, 1]):
        x = torch.randn(sum(new), blk.K, generator=g).bfloat16().cuda()
        pos = np.concatenate([h + np.arange(n) for h, n in zip(held, new)])
        cu = [int(c) for c in np.cumsum([0] + new)]
        after = [h + n for h, n in zip(held, new)]
        one_each = new == [1] * 5
        y = blk.step(x, i32(pos.tolist()), i32(held), i32(after), None if one_each else i32(cu))
        check_step(blk, x, y, oracle, held, new, cu)
        held = after


def test_tokens_in_a_graph(gpu_lib):
    """A captured step whose inputs and lengths are updated in place, against an eager block of the same contents."""
    a, b = Block(gpu_lib), Block(gpu_lib)
    a.keep = b.keep = False
    g = torch.Generator().manual_seed(2)
    first = [30, 1, 17, 5, 100]
    cu = i32(np.cumsum([0] + first).tolist())
    x = torch.randn(sum(first), a.K, generator=g).bfloat16().cuda()
    pos = i32(np.concatenate([np.arange(n) for n in first]).tolist())
    for blk in (a, b):
        blk.step(x, pos, i32([0] * 5), i32(first), cu)
    x, before, after = torch.empty(5, a.K, dtype=torch.bfloat16, device="cuda"), i32(first), i32([n + 1 for n in first])
    x.normal_()
    warm = Block(gpu_lib)
    warm.keep = False
    warm.step(x, before, before, after)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = a.step(x, before, before, after)
    for t in range(6):
        x.copy_(torch.randn(5, a.K, generator=g).bfloat16())
        now = [n + t for n in first]
        before.copy_(i32(now))
        after.copy_(i32([n + 1 for n in now]))
        ref = b.step(x, before, before, after)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref), t
