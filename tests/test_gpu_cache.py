"""GPU: writing to a paged e4m3 cache and reading it back, bit for bit against the oracle."""

import numpy as np
import pytest
import torch

from oracle import serving as S

pytestmark = pytest.mark.gpu


def f64(t):
    return t.float().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def tokens(T, Hk, D, seed, loud=0.1):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, 2 * Hk, D, generator=g)
    z *= torch.where(torch.rand(T, 2 * Hk, 1, generator=g) < loud, 2.0 ** torch.randint(-3, 7, (T, 2 * Hk, 1), generator=g), 1.0)
    z = z.bfloat16().cuda()
    return z[:, :Hk], z[:, Hk:]


def table_for(lens, page, pages, seed):
    """Pages in shuffled order, as many per sequence as its length takes; -1 past them."""
    order = np.random.default_rng(seed).permutation(pages).tolist()
    counts = [-(-n // page) for n in lens]
    assert sum(counts) <= pages
    width = max(1, max(counts))
    rows, at = [], 0
    for c in counts:
        rows.append(order[at:at + c] + [-1] * (width - c))
        at += c
    return rows


def offsets(lens):
    return [int(c) for c in np.cumsum([0] + list(lens))]


def dirty(lib, pages, Hk, page, D):
    """A cache full of NaN codes and scales."""
    c = lib.new_cache_fp8(pages, Hk, D, page)
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        t.view(torch.uint8).fill_(0xFF)
    return c


def codes_of(cache, name):
    """[pages, Hk, page, D] whatever the layout."""
    t = cache.k_codes if name == "k" else cache.v_codes.view(torch.uint8).transpose(2, 3).contiguous().view(torch.float8_e4m3fn)
    return f64(t)


def check_held(lib, cache, oracle, table, lens):
    """Every token that the sequences hold: scales, codes, and what cache_read gives."""
    read = dict(zip("kv", lib.cache_read_fp8(cache, i32(table), i32([0] * len(lens)), i32(offsets(lens)), sum(lens))))
    for name in "kv":
        exps = (cache.k_scales if name == "k" else cache.v_scales).cpu().numpy().astype(int) - 127
        codes, values = codes_of(cache, name), oracle.values(name)
        at = 0
        for row, n in zip(table, lens):
            for blk in range(-(-n // oracle.page)):
                p, held = row[blk], min(oracle.page, n - blk * oracle.page)
                if not 0 <= p < len(values):
                    assert not read[name][at:at + held].any()
                else:
                    assert np.array_equal(exps[p], np.where(oracle.nan[name][p], 128, oracle.exps[name][p])), (name, p)
                    live = ~oracle.nan[name][p]
                    assert np.array_equal(codes[p, live, :held], oracle.codes[name][p, live, :held]), (name, p)
                    got = f64(read[name][at:at + held])
                    # bf16 holds every value but 2^128, which the largest bf16 rounds up to in e4m3: infinity
                    ref = np.where(np.abs(values[p]) >= 2.0 ** 128, np.sign(values[p]) * np.inf, values[p])
                    assert np.array_equal(got, ref[:, :held].transpose(1, 0, 2), equal_nan=True), (name, p)
                at += held


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hk,D", [(1, 128), (3, 64), (8, 128)])
def test_appends_against_oracle(gpu_lib, page, Hk, D):
    """Prompts of many lengths, then ragged additions (none, one, many tokens), into shuffled pages."""
    print(f"[cache] append page={page} Hk={Hk} D={D}", flush=True)
    steps = [[1, 0, 15, 16, 17, page, page + 1, 3 * page - 1, 200], [1, 0, 1, 1, 1, 1, 1, 1, 1], [0, 5, 40, 0, 300, 2, 1, 129, 7],
             [3, 1, 0, 2 * page, 1, 0, 4, 1, 1]]
    total = [sum(s) for s in zip(*steps)]
    pages = sum(-(-n // page) for n in total) + 3
    table = table_for(total, page, pages, page)
    cache, oracle = dirty(gpu_lib, pages, Hk, page, D), S.Cache(pages, Hk, page, D)
    held = [0] * len(total)
    for i, new in enumerate(steps):
        k, v = tokens(sum(new), Hk, D, 10 * page + i)
        gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32(held), i32(offsets(new)))
        oracle.append({"k": f64(k), "v": f64(v)}, table, held, offsets(new))
        held = [a + b for a, b in zip(held, new)]
        check_held(gpu_lib, cache, oracle, table, held)
    # pages that no sequence has are as they were
    spare = [p for p in range(pages) if p not in sum(table, [])]
    assert spare and bool((cache.k_codes.view(torch.uint8)[spare] == 255).all())
    assert bool((cache.v_codes.view(torch.uint8)[spare] == 255).all()) and bool((cache.v_scales[spare] == 255).all())


@pytest.mark.parametrize("page,D", [(16, 64), (64, 128)])
def test_token_by_token(gpu_lib, page, D):
    """Single tokens without offsets, louder and louder: the scale grows many times."""
    B, Hk, n = 5, 2, 2 * page + 3
    table = table_for([n + b for b in range(B)], page, 40, 1)
    cache, oracle = dirty(gpu_lib, 40, Hk, page, D), S.Cache(40, Hk, page, D)
    held = list(range(B))
    k, v = tokens(B * B, Hk, D, 1)
    gpu_lib.cache_append_fp8(k[:sum(held)], v[:sum(held)], cache, i32(table), i32([0] * B), i32(offsets(held)))
    oracle.append({"k": f64(k[:sum(held)]), "v": f64(v[:sum(held)])}, table, [0] * B, offsets(held))
    for t in range(n - 1):
        k, v = tokens(B, Hk, D, 100 + t, 0.3)
        if t % 7 == 3:
            k, v = k * 2.0 ** (t // 4), v * 2.0 ** (t // 5)
        gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32(held))
        oracle.append({"k": f64(k), "v": f64(v)}, table, held, list(range(B + 1)))
        held = [h + 1 for h in held]
    check_held(gpu_lib, cache, oracle, table, held)


def test_slots_past_the_tokens_are_left_alone(gpu_lib):
    for page in (16, 64):
        Hk, D = 2, 64
        cache = dirty(gpu_lib, 4, Hk, page, D)
        k, v = tokens(9, Hk, D, 3)
        gpu_lib.cache_append_fp8(k, v, cache, i32([[2]]), i32([0]), i32([0, 9]))
        assert bool((cache.k_codes.view(torch.uint8)[2, :, 9:] == 255).all())
        assert bool((cache.v_codes.view(torch.uint8)[2, :, :, 9:] == 255).all())
        for p in (0, 1, 3):
            assert all(bool((t.view(torch.uint8)[p] == 255).all()) for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales))


def test_zero_tiny_and_huge_blocks(gpu_lib):
    cache, oracle = dirty(gpu_lib, 6, 1, 16, 64), S.Cache(6, 1, 16, 64)
    z = torch.zeros(6, 16, 1, 64)
    z[1] = 2.0 ** -126
    z[2, 3, 0, 5] = 448 * 2.0 ** -100
    z[3, 3, 0, 5] = 450 * 2.0 ** -100
    z[4, 15, 0, 63] = 3.3895313892515355e38
    z[5] = torch.randn(16, 1, 64) * 1e30
    z = z.bfloat16().view(96, 1, 64).cuda()
    table = [[5, 0, 3, 1, 2, 4]]
    gpu_lib.cache_append_fp8(z, z, cache, i32(table), i32([0]), i32([0, 96]))
    oracle.append({"k": f64(z), "v": f64(z)}, table, [0], [0, 96])
    check_held(gpu_lib, cache, oracle, table, [96])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_tokens_mark_their_page(gpu_lib, bad):
    Hk, D, page = 3, 64, 16
    table = [[0, 1, 2]]
    cache, oracle = dirty(gpu_lib, 3, Hk, page, D), S.Cache(3, Hk, page, D)
    k, v = tokens(40, Hk, D, 5)
    k, v = k.clone(), v.clone()
    k[20, 1, 7] = bad
    v[5, 2, 0] = bad
    held = 0
    for n in (19, 3, 10, 8):
        part = slice(held, held + n)
        gpu_lib.cache_append_fp8(k[part], v[part], cache, i32(table), i32([held]), i32([0, n]))
        oracle.append({"k": f64(k[part]), "v": f64(v[part])}, table, [held], [0, n])
        held += n
    assert cache.k_scales[1, 1] == 255 and cache.v_scales[0, 2] == 255
    assert int((cache.k_scales == 255).sum()) == 1 and int((cache.v_scales == 255).sum()) == 1
    check_held(gpu_lib, cache, oracle, table, [40])
    # slot 0 written again: as new
    k, v = tokens(16, Hk, D, 6)
    gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32([16]), i32([0, 16]))
    oracle.append({"k": f64(k), "v": f64(v)}, table, [16], [0, 16])
    assert not bool((cache.k_scales == 255).any())


def test_pages_that_the_table_does_not_have(gpu_lib):
    """Entries outside the cache and tokens past the table's width are left out, and read as zeros."""
    Hk, D, page = 2, 128, 16
    table = [[1, -1, 2], [7, 0, 2 ** 31 - 1], [-2 ** 31, 3, 4]]
    cache, oracle = dirty(gpu_lib, 5, Hk, page, D), S.Cache(5, Hk, page, D)
    lens = [48, 60, 48]
    k, v = tokens(sum(lens), Hk, D, 7)
    gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32([0] * 3), i32(offsets(lens)))
    oracle.append({"k": f64(k), "v": f64(v)}, table, [0] * 3, offsets(lens))
    check_held(gpu_lib, cache, oracle, table, [48, 48, 48])
    far, _ = gpu_lib.cache_read_fp8(cache, i32(table), i32([47, 1000, 2 ** 31 - 4]), i32([0, 4, 8, 10]), 10)
    assert far[0].any() and not far[1:].any()


@pytest.mark.parametrize("cu", [[0, 40, 20, 60], [-5, 10, 30, 60], [0, 10, 30, 1000], [50, 50, 50, 60], [60, 40, 20, 0]])
def test_bad_offsets_stay_inside(gpu_lib, cu):
    """Offsets outside 0..T or decreasing, negative lengths: nothing outside the tensors is touched."""
    Hk, D, page = 2, 64, 16
    cache = dirty(gpu_lib, 30, Hk, page, D)
    table = table_for([80] * 3, page, 30, 2)
    k, v = tokens(60, Hk, D, 8)
    gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32([3, -7, 0]), i32(cu))
    spare = [p for p in range(30) if p not in sum(table, [])]
    assert bool((cache.k_codes.view(torch.uint8)[spare] == 255).all())
    base = torch.full((80, Hk, D), 3.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.cache_read_fp8(cache, i32(table), i32([3, -7, 0]), i32(cu), 60, k=base[10:70], v=torch.empty_like(base[10:70]))
    assert bool((base[:10] == 3).all()) and bool((base[70:] == 3).all())


def test_read_parts_and_rows_outside(gpu_lib):
    Hk, D, page = 2, 128, 32
    table = table_for([100, 70], page, 9, 3)
    cache, oracle = dirty(gpu_lib, 9, Hk, page, D), S.Cache(9, Hk, page, D)
    k, v = tokens(170, Hk, D, 9)
    gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32([0, 0]), i32([0, 100, 170]))
    oracle.append({"k": f64(k), "v": f64(v)}, table, [0, 0], [0, 100, 170])
    out = torch.full((60, Hk, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((60, Hk, D), 7.0, dtype=torch.bfloat16, device="cuda")
    rk, rv = gpu_lib.cache_read_fp8(cache, i32(table), i32([31, 5]), i32([4, 40, 55]), k=out[0], v=out[1])
    assert rk is out[0] and rv is out[1]
    for got, name in ((rk, "k"), (rv, "v")):
        assert np.array_equal(f64(got[4:40]), S.gather(oracle.values(name), table[0], page, 31, 36))
        assert np.array_equal(f64(got[40:55]), S.gather(oracle.values(name), table[1], page, 5, 15))
        assert bool((got[:4] == 7).all()) and bool((got[55:] == 7).all())
    one, _ = gpu_lib.cache_read_fp8(cache, i32(table), i32([99, 0]))
    assert one.shape == (2, Hk, D) and torch.equal(one[0], gpu_lib.cache_read_fp8(cache, i32(table), i32([99, 0]))[0][0])


def test_strided_tokens_side_stream_and_graph(gpu_lib):
    Hk, D, page = 4, 64, 16
    table = i32(table_for([60, 60], page, 10, 4))
    g = torch.Generator().manual_seed(1)
    heads_first = torch.randn(2 * Hk, 50, D, generator=g).bfloat16().cuda()
    k, v = heads_first[:Hk].transpose(0, 1), heads_first[Hk:].transpose(0, 1)
    a, b, c = (dirty(gpu_lib, 10, Hk, page, D) for _ in range(3))
    start, cu = i32([7, 0]), i32([0, 20, 50])
    gpu_lib.cache_append_fp8(k.contiguous(), v.contiguous(), a, table, start, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gpu_lib.cache_append_fp8(k, v, b, table, start, cu)
    s.synchronize()

    def same(x, y):
        return all(torch.equal(getattr(x, n).view(torch.uint8), getattr(y, n).view(torch.uint8))
                   for n in ("k_codes", "v_codes", "k_scales", "v_scales"))

    assert same(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.cache_append_fp8(k, v, c, table, start, cu)
    for _ in range(3):
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            t.view(torch.uint8).fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(a, c)


def test_many_sequences(gpu_lib):
    """More sequences than the search probes at once, most of one token."""
    rng = np.random.default_rng(5)
    Hk, D, page, B = 1, 64, 16, 700
    new = np.where(rng.random(B) < 0.3, 0, np.where(rng.random(B) < 0.05, 40, 1)).tolist()
    held = rng.integers(0, 30, B).tolist()
    total = [a + b for a, b in zip(held, new)]
    pages = sum(-(-n // page) for n in total) + 1
    table = table_for(total, page, pages, 6)
    cache, oracle = dirty(gpu_lib, pages, Hk, page, D), S.Cache(pages, Hk, page, D)
    for n, at in ((held, [0] * B), (new, held)):
        k, v = tokens(sum(n), Hk, D, sum(n))
        gpu_lib.cache_append_fp8(k, v, cache, i32(table), i32(at), i32(offsets(n)))
        oracle.append({"k": f64(k), "v": f64(v)}, table, at, offsets(n))
    check_held(gpu_lib, cache, oracle, table, total)
