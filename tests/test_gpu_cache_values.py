"""GPU: values that come back from the e4m3 cache where earlier tests look at shapes and scales: single tokens without
offsets, and a page that held something not finite, written anew."""

import numpy as np
import pytest

from oracle import serving as S
from tests.test_gpu_cache import check_held, dirty, f64, i32, offsets, table_for, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hk,D", [(2, 128), (3, 64)])
def test_single_tokens_read_without_offsets(gpu_lib, page, Hk, D):
    lens = [100, 70, 1, 129]
    pages = sum(-(-n // page) for n in lens) + 2
    table = table_for(lens, page, pages, page)
    cache, oracle = dirty(gpu_lib, pages, Hk, page, D), S.Cache(pages, Hk, page, D)
    k, v = tokens(sum(lens), Hk, D, page + D)
    gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32([0] * 4), i32(offsets(lens)))
    oracle.append({"k": f64(k), "v": f64(v)}, table, [0] * 4, offsets(lens))
    for at in ([99, 69, 0, 128], [0, 0, 0, 0], [page - 1, 15, 0, page], [17, 33, 0, 64]):
        at = [min(i, n - 1) for i, n in zip(at, lens)]
        for name, got in zip("kv", gpu_lib.cache_read_fp8(cache, i32(table), i32(at))):
            assert got.shape == (4, Hk, D)
            for b in range(4):
                want = S.gather(oracle.values(name), table[b], page, at[b], 1)
                assert want.any() and np.array_equal(f64(got[b:b + 1]), want), (name, b, at)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_page_written_anew_after_something_not_finite(gpu_lib, bad):
    Hk, D, page = 3, 64, 16
    table = [[2, 0, 1]]
    cache, oracle = dirty(gpu_lib, 3, Hk, page, D), S.Cache(3, Hk, page, D)

    def append(k, v, at):
        gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32([at]), i32([0, len(k)]))
        oracle.append({"k": f64(k), "v": f64(v)}, table, [at], [0, len(k)])

    k, v = (t.clone() for t in tokens(40, Hk, D, 5))
    k[20, 1, 7] = bad
    v[25, 2, 0] = bad
    append(k, v, 0)
    check_held(gpu_lib, cache, oracle, table, [40])
    assert cache.k_scales[0, 1] == 255 and cache.v_scales[0, 2] == 255
    append(*tokens(9, Hk, D, 6), 16)            # slot 0 of that page, and part of it
    check_held(gpu_lib, cache, oracle, table, [25])
    append(*tokens(7, Hk, D, 7), 25)            # behind them
    check_held(gpu_lib, cache, oracle, table, [40])
    assert not bool((cache.k_scales == 255).any()) and not bool((cache.v_scales == 255).any())
