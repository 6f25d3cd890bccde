"""GPU: one token on a table of 2^30 keys, held to a bound that counts every addition of the second product's sums."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_mean_of_a_table_of_as_many_tokens_as_are_allowed(gpu_lib):
    """2^30 keys of nothing, one page listed 2^23 times: probabilities are exactly 1, their sums (of at most 2^24 in any place
    that adds ones) exact, and o is the mean of the page's values, all of one sign.

    An accumulator of the few-row kernel takes its share of the keys, 2^30 / (splits * 4 waves), 32 a matrix instruction:
    n additions, each off by at most 2^-24 of the sum where it rounds and 2^-23 where it cuts off. The instruction's own 31
    additions, the four waves', the splits' and the quotient add splits + 64 of those, o's rounding to bf16 2^-8."""
    D, page, width = 64, 128, 1 << 23
    g = torch.Generator(device="cuda").manual_seed(6)
    cache = gpu_lib.new_cache_fp8(2, 1, D, page)
    v = torch.randn(page, 1, D, generator=g, device="cuda").abs().bfloat16()
    one = torch.ones((1, 1), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, page], dtype=torch.int32, device="cuda")
    gpu_lib.cache_append_fp8(torch.zeros_like(v), v, cache, one, one[0] - 1, cu_seqlens=cu)
    mean = gpu_lib.cache_read_fp8(cache, one, one[0] - 1, cu_seqlens=cu, tokens=page)[1].double().mean(0)
    q = torch.randn(1, 2, D, generator=g, device="cuda").bfloat16()
    table = torch.ones((1, width), dtype=torch.int32, device="cuda")
    length = torch.full((1,), 1 << 30, dtype=torch.int32, device="cuda")
    kernel, splits = gpu_lib.attention_cache_fp8_plan(1, 1, 2, 1, D, 1 << 30, False)
    assert kernel == 0 and splits >= 64
    n = -(-(1 << 30) // (splits * 4 * 32))
    o = gpu_lib.attention_cache_fp8(q, cache, table, length).double()
    tol = 2.0 ** -8 + (1 + 2.0 ** -8) * (n + splits + 64) * 2.0 ** -23
    print(f"[attention_cache] 2^30 keys: {splits} splits, bound {tol:.2e}, off by {float(((o - mean).abs() / mean).max()):.2e}", flush=True)
    assert bool(((o - mean).abs() <= tol * mean).all())
