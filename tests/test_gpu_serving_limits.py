"""GPU: serving in 8-bit floating point at the ends of its documented ranges: as many sequences and tokens as are allowed,
a table of the most tokens, whose one page is listed throughout."""

import numpy as np
import pytest
import torch

from oracle import serving as S

pytestmark = pytest.mark.gpu


def f64(t):
    return t.float().double().cpu().numpy()


def test_as_many_sequences_as_are_allowed(gpu_lib):
    """65535 single tokens appended, read back and attended to, a few keys each."""
    B, page, D = 65535, 16, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = gpu_lib.new_cache_fp8(B, 1, D, page)
    table = torch.randperm(B, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    keep_k, keep_v = [], []
    for step in range(3):
        k = torch.randn(B, 1, D, generator=g, device="cuda").bfloat16()
        v = torch.randn(B, 1, D, generator=g, device="cuda").bfloat16()
        at = torch.full((B,), step, dtype=torch.int32, device="cuda")
        gpu_lib.cache_append_fp8(k, v, cache, table, at)
        keep_k.append(k)
    for step in range(3):
        at = torch.full((B,), step, dtype=torch.int32, device="cuda")
        k, v = gpu_lib.cache_read_fp8(cache, table, at)
        # half a step of the code, and again where the page was rescaled into subnormal codes
        assert bool(((k.float() - keep_k[step].float()).abs() <= 2.0 ** -4 * keep_k[step].float().abs() + 2.0 ** -15).all())
        keep_k[step] = k
        keep_v.append(v)
    lens = torch.randint(0, 4, (B,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(B, 2, D, generator=g, device="cuda").bfloat16()
    o = gpu_lib.attention_cache_fp8(q, cache, table, lens).double()
    k, v = torch.stack(keep_k, 1).double(), torch.stack(keep_v, 1).double()        # [B, 3, 1, D]
    s = (q.double()[:, None] * k).sum(3) * D ** -0.5                               # [B, 3, 2]
    s = s.masked_fill(torch.arange(3, device="cuda")[None, :, None] >= lens[:, None, None], -torch.inf)
    p = torch.where(lens[:, None, None] > 0, s.softmax(1), 0.0).nan_to_num(0.0)[..., None]
    ref, mag = (p * v).sum(1), (p * v.abs()).sum(1)
    # the probabilities' and the output's roundings to bf16 (2^-8 each), fp32 sums and exponents far below 2e-4
    assert bool(((o - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2e-4) * mag).all())


def test_as_many_tokens_as_are_allowed(gpu_lib):
    """2^24 - 1 tokens in a call."""
    T, D, page = (1 << 24) - 1, 64, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn(T, 1, D, generator=g, device="cuda", dtype=torch.bfloat16)
    pages = -(-T // page)
    cache = gpu_lib.new_cache_fp8(pages, 1, D, page)
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    gpu_lib.cache_append_fp8(k, k.abs(), cache, table, zero, cu_seqlens=cu)
    back = gpu_lib.cache_read_fp8(cache, table, zero, cu_seqlens=cu, tokens=T)
    for x, sign in zip(back, (False, True)):
        for part, want in zip(x.split(1 << 21), k.split(1 << 21)):
            want = want.abs() if sign else want
            assert bool(((part.float() - want.float()).abs() <= 2.0 ** -4 * want.float().abs() + 2.0 ** -16).all())
    # one token that sees all of them: the mean of values, for keys of nothing
    cache.k_codes.view(torch.uint8).zero_()
    o = gpu_lib.attention_cache_fp8(torch.ones(1, 2, D, device="cuda").bfloat16(), cache, table, zero + T).double()
    mean = sum(v.double().sum(0) for v in back[1].split(1 << 20)) / T
    # Probabilities are 1 and their sum exact. Values of one sign: split 16 ways or more among four waves, 32 keys an
    # instruction, an accumulator is added to at most 2^13 times, 2^-24 of it each; the instruction's own sums and the join's are less
    splits = gpu_lib.attention_cache_fp8_plan(1, 1, 2, 1, D, T, False)[1]
    assert splits >= 16
    assert bool(((o - mean).abs() <= (2.0 ** -8 + 2.0 ** -10) * mean).all())


def test_as_many_rows_as_are_allowed(gpu_lib):
    M, K = 1 << 24, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    codes, scales = gpu_lib.quantize_fp8(x)
    pick = torch.tensor([0, 1, 31, 32, M // 2, M - 33, M - 2, M - 1])
    rc, e = S.quantize(f64(x[pick.cuda()]))
    assert np.array_equal(f64(codes.view(torch.uint8)[pick.cuda()].view(torch.float8_e4m3fn)), rc)
    assert np.array_equal(scales[:, pick.cuda()].double().cpu().numpy(), 2.0 ** e.T)


def test_positions_of_as_many_tokens_as_are_allowed(gpu_lib):
    T, D = (1 << 24) - 1, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(T, 1, D, generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    pick = torch.tensor([0, 1, 7, T // 2, T - 2, T - 1], device="cuda")
    for R, inter in ((16, False), (8, False), (8, True)):
        o, _ = gpu_lib.rope_scaled(q, None, pos, rotary_dim=R, interleaved=inter)
        part, _ = gpu_lib.rope_scaled(q[pick].contiguous(), None, pos[pick].contiguous(), rotary_dim=R, interleaved=inter)
        assert torch.equal(o[pick], part)


def test_a_table_of_as_many_tokens_as_are_allowed(gpu_lib):
    """2^30 keys, one page listed 2^23 times: o is the mean of its values."""
    D, page, width = 64, 128, 1 << 23
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = gpu_lib.new_cache_fp8(2, 1, D, page)
    v = torch.randn(page, 1, D, generator=g, device="cuda").abs().bfloat16()
    one = torch.ones((1, 1), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, page], dtype=torch.int32, device="cuda")
    gpu_lib.cache_append_fp8(torch.zeros_like(v), v, cache, one, one[0] - 1, cu_seqlens=cu)
    mean = gpu_lib.cache_read_fp8(cache, one, one[0] - 1, cu_seqlens=cu, tokens=page)[1].double().mean(0)
    table = torch.ones((1, width), dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, D, generator=g, device="cuda").bfloat16()
    length = torch.full((1,), 1 << 30, dtype=torch.int32, device="cuda")
    splits = gpu_lib.attention_cache_fp8_plan(1, 1, 2, 1, D, 1 << 30, False)[1]
    assert splits >= 64
    o = gpu_lib.attention_cache_fp8(q, cache, table, length).double()
    # an accumulator is added to 2^30 / (64 splits, 4 waves, 32 keys an instruction) = 2^17 times, at most 2^-25 of it each
    assert bool(((o - mean).abs() <= (2.0 ** -8 + 2.0 ** -8) * mean).all())
    with pytest.raises(gpu_lib.SvdqError):
        gpu_lib.attention_cache_fp8(q, cache, torch.ones((1, width + 1), dtype=torch.int32, device="cuda"), length)
