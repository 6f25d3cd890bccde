"""GPU: the cached attention's tiles (many rows) where a call can go wrong: missing and stale pages, contents that are not
finite, extreme scores, strides, streams, guards, bad offsets, graphs that share a workspace, more sequences than a wave has
lanes, a cache past 4 GiB. The batches are those that reach the tiles, whole and with keys split; each test asserts it."""

import numpy as np
import pytest
import torch

from tests.test_attention_cache_plan import LONG, RAGGED, plan
from tests.test_gpu_attention_cache import Case, i32

pytestmark = pytest.mark.gpu

# sequences, H, Hk, D: keys whole, and split
WHOLE, SPLIT = (RAGGED, 16, 2, 128), (LONG, 4, 1, 128)
NARROW = (RAGGED, 24, 3, 64)


def tiles(lib, batch, page, seed, **kw):
    seqs, H, Hk, D = batch
    assert plan(seqs, H, Hk, D)[0] == 1
    return Case(lib, [n for n, _ in seqs], [L for _, L in seqs], H, Hk, D, page, seed, **kw)


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("batch", [WHOLE, SPLIT, NARROW], ids=["whole", "split", "narrow"])
def test_stale_contents_and_missing_pages(gpu_lib, batch, page):
    c = tiles(gpu_lib, batch, page, 31, extra_width=2)
    clean = c.run()
    c.check(clean)
    spare = [p for p in range(c.cache.k_codes.shape[0]) if p not in sum(c.table, [])]
    own = [-(-L // page) for L in c.lens]
    for b, row in enumerate(c.table):          # past a sequence's end: pages of NaN
        row[own[b]:] = [spare[b % len(spare)]] * (len(row) - own[b])
    c.cache.k_scales[spare] = 255
    c.cache.v_scales[spare] = 255
    assert torch.equal(bits(c.run()), bits(clean))
    entries = (-1, -2 ** 31, 2 ** 31 - 1, c.cache.k_codes.shape[0])
    gone = [b for b, L in enumerate(c.lens) if L > page]
    for i, b in enumerate(gone):
        j = i % own[b]
        c.table[b][j] = entries[i % 4]
        for x in c.keys[b]:
            x[j * page:(j + 1) * page] = 0.0
    for causal in (True, False):
        c.check(c.run(causal), causal)
    c.lens[0] = -7
    o = c.run(max_length=max(c.lens))
    assert not o[: c.new[0]].any()


def test_lengths_past_the_table(gpu_lib):
    """Lengths past the table's width are what it holds."""
    c = tiles(gpu_lib, WHOLE, 32, 32)
    width = len(c.table[0]) * 32
    full = [b for b, L in enumerate(c.lens) if -(-L // 32) * 32 == width]
    lens = list(c.lens)
    for b in full:
        lens[b] = 2 ** 31 - 1
    c.cache.v_codes.view(torch.uint8)[[c.table[b][-1] for b in full], :, :, 31] = 0x7F      # past every length as given
    assert bool(torch.isfinite(c.run(False).float()).all())
    o = c.lib.attention_cache_fp8(c.q, c.cache, i32(c.table), i32(lens), cu_seqlens=i32(c.cu), causal=False, max_length=max(c.lens))
    for b in range(len(lens)):
        rows = o[c.cu[b]:c.cu[b + 1]].float()
        assert bool(torch.isnan(rows).all()) if b in full else bool(torch.isfinite(rows).all())


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("which", ["k_scales", "v_scales"])
def test_non_finite_pages_reach_only_their_sequence_and_head(gpu_lib, page, which):
    c = tiles(gpu_lib, WHOLE, page, 33)
    clean = c.run()
    b = RAGGED.index((64, 64))
    getattr(c.cache, which)[c.table[b][0], 1] = 255
    o = c.run()
    rows = slice(c.cu[b], c.cu[b + 1])
    assert bool(torch.isnan(o[rows, 8:].float()).all())
    ok = torch.ones_like(o, dtype=torch.bool)
    ok[rows, 8:] = False
    assert torch.equal(o[ok], clean[ok])


@pytest.mark.parametrize("page", [16, 128])
def test_future_keys_that_are_not_finite_are_not_seen(gpu_lib, page):
    c = tiles(gpu_lib, WHOLE, page, 34)
    clean = c.run()
    b = RAGGED.index((190, 151))
    c.cache.k_codes.view(torch.uint8)[c.table[b][150 // page], :, 150 % page, 5] = 0x7F
    o = c.run()
    last = c.cu[b + 1] - 1
    assert bool(torch.isnan(o[last].float()).all())
    o[last] = clean[last]
    assert torch.equal(bits(o), bits(clean))


@pytest.mark.parametrize("scale,gain", [(2.0 ** -10, 1.0), (1.0, 60.0), (2.0 ** 20, 1.0), (1e-30, 1.0), (2.0 ** 10, 1e30)])
@pytest.mark.parametrize("batch", [WHOLE, SPLIT], ids=["whole", "split"])
def test_extreme_scores(gpu_lib, batch, scale, gain):
    c = tiles(gpu_lib, batch, 64, 35)
    c.q = (c.q.float() * gain).bfloat16()
    o = c.run(scale=scale)
    assert bool(torch.isfinite(o.float()).all())
    if gain <= 60.0 and scale <= 1.0:
        c.check(o, scale=scale)


@pytest.mark.parametrize("batch", [NARROW, SPLIT], ids=["narrow", "split"])
def test_equal_keys_far_from_zero(gpu_lib, batch):
    for sign in (1.0, -1.0):
        c = tiles(gpu_lib, batch, 32, 36)
        c.cache.k_codes.view(torch.uint8)[:] = 0x7E        # 448
        c.cache.k_scales[:] = 200
        c.q[:] = sign * 3e7
        o = c.run(False)
        for b, L in enumerate(c.lens):
            rows = o[c.cu[b]:c.cu[b + 1]].double()
            if L == 0:
                assert not rows.any()
                continue
            v = torch.from_numpy(np.repeat(c.keys[b][1], c.H // c.Hk, 1)).cuda()
            assert bool(((rows - v.mean(0)).abs() <= 2.0 ** -7 * v.abs().mean(0)).all())


def test_old_keys_keep_their_weight(gpu_lib):
    """Scores that climb from key to key move the maximum often."""
    L, page, H, Hk, D = 2048, 64, 24, 3, 128
    c = tiles(gpu_lib, ([(512, L), (300, L), (1, 64)], H, Hk, D), page, 37)
    k = torch.zeros(L, D)
    k[:, 0] = torch.arange(L) // 16                                  # rounded below
    k = k.to(torch.float8_e4m3fn)
    for b in range(2):
        order = torch.tensor(c.table[b][: L // page])
        c.cache.k_codes.view(torch.uint8)[order] = k.view(torch.uint8).view(L // page, 1, page, D).cuda()
        c.keys[b][0] = np.repeat(k.double().numpy()[:, None], Hk, 1)
    c.cache.k_scales[:] = 127
    c.cache.k_codes.view(torch.uint8)[c.table[2][0]] = 0
    c.keys[2][0] = np.zeros((64, Hk, D))
    q = torch.zeros(sum(c.new), H, D)
    q[:, ::2, 0], q[:, 1::2, 0] = 1.5, -0.75
    c.q = q.bfloat16().cuda()
    for scale in (0.125, 2.0):
        c.check(c.run(False, scale=scale), False, scale)


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("batch", [WHOLE, SPLIT], ids=["whole", "split"])
def test_views_strides_streams_and_guards(gpu_lib, batch, page):
    c = tiles(gpu_lib, batch, page, 38)
    ref = c.run()
    T, H, D = c.q.shape
    fused = torch.randn(T, H + 3, D, device="cuda").bfloat16()
    fused[:, 1:H + 1] = c.q
    heads_first = torch.full((H, T + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = heads_first[:, 1:T + 1].transpose(0, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run(q=fused[:, 1:H + 1], out=out)
    s.synchronize()
    assert got is out and torch.equal(out, ref)
    assert bool((heads_first[:, 0] == 7).all()) and bool((heads_first[:, -1] == 7).all())
    need = gpu_lib.attention_cache_fp8_workspace_bytes(T, len(c.new), H, c.Hk, D, max(c.lens), True)
    assert (need > 0) == (batch is SPLIT)
    work = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.run(workspace=work[256:256 + need]), ref)
    assert bool((work[:256] == 0xA5).all()) and bool((work[256 + need:] == 0xA5).all())
    assert all(torch.equal(bits(c.run()), bits(ref)) for _ in range(3))


@pytest.mark.parametrize("batch", [WHOLE, SPLIT], ids=["whole", "split"])
def test_rows_outside_the_offsets_are_left_alone(gpu_lib, batch):
    c = tiles(gpu_lib, batch, 64, 39)
    q = torch.cat([c.q[:5], c.q, c.q[:9]])
    out = torch.full_like(q, 7.0)
    c.lib.attention_cache_fp8(q, c.cache, i32(c.table), i32(c.lens), cu_seqlens=i32([x + 5 for x in c.cu]),
                              max_length=max(c.lens), out=out)
    c.check(out[5:-9])
    assert bool((out[:5] == 7).all()) and bool((out[-9:] == 7).all())


@pytest.mark.parametrize("how", ["reversed", "before", "after", "up and down"])
@pytest.mark.parametrize("batch", [WHOLE, SPLIT], ids=["whole", "split"])
def test_bad_offsets_stay_inside(gpu_lib, batch, how):
    c = tiles(gpu_lib, batch, 32, 40)
    T = c.q.shape[0]
    cu = {"reversed": c.cu[::-1], "before": [x - T // 2 for x in c.cu], "after": [x + T // 2 for x in c.cu],
          "up and down": [T if i % 2 else 0 for i in range(len(c.cu))]}[how]
    base = torch.full((T + 20, *c.q.shape[1:]), 3.0, dtype=torch.bfloat16, device="cuda")
    c.lib.attention_cache_fp8(c.q, c.cache, i32(c.table), i32(c.lens), cu_seqlens=i32(cu), max_length=max(c.lens), out=base[10:-10])
    torch.cuda.synchronize()
    assert bool((base[:10] == 3).all()) and bool((base[-10:] == 3).all())


def test_graphs_sharing_a_workspace(gpu_lib):
    """Two captured calls with one workspace, replayed in turn between eager work; lengths change in between."""
    cases = [tiles(gpu_lib, SPLIT, 64, 41), tiles(gpu_lib, SPLIT, 16, 42)]
    need = gpu_lib.attention_cache_fp8_workspace_bytes(cases[0].q.shape[0], len(LONG), *SPLIT[1:], 6000, True)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for c in cases:
        st = dict(out=torch.empty_like(c.q), lens=i32(c.lens), table=i32(c.table), cu=i32(c.cu))

        def call(c=c, st=st):
            c.lib.attention_cache_fp8(c.q, c.cache, st["table"], st["lens"], cu_seqlens=st["cu"], max_length=6000, out=st["out"], workspace=work)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, c, st))
    for rep in range(4):
        for g, c, st in graphs:
            st["lens"].copy_(i32([max(0, x - 61 * rep) for x in c.lens]))
            ref = c.lib.attention_cache_fp8(c.q, c.cache, st["table"], st["lens"], cu_seqlens=st["cu"], max_length=6000)
            st["out"].zero_()
            work.fill_(0x5A)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(bits(st["out"]), bits(ref)), rep


@pytest.mark.parametrize("B", [63, 64, 65, 150])
def test_as_many_sequences_as_lanes_and_more(gpu_lib, B):
    """Up to 64 sequences are ordered by a wave, more are found by their offsets; equal lengths among them, and empty ones."""
    rng = np.random.default_rng(B)
    new = rng.choice([0, 1, 40, 64, 90, 120], B)
    new[-1] = 40
    lens = np.where(rng.random(B) < 0.3, 100, new + rng.integers(0, 130, B))
    seqs = list(zip(new.tolist(), lens.tolist()))
    for H, Hk, D, page in ((16, 2, 128, 32), (24, 3, 64, 64)):
        c = tiles(gpu_lib, (seqs, H, Hk, D), page, B)
        c.check(c.run())


@pytest.mark.parametrize("page", [32, 64])
def test_pages_past_32_bits(gpu_lib, page):
    """A cache of more than 4 GiB of codes: pages at its far end."""
    Hk, D = 2, 128
    pages = (9 << 29) // (Hk * page * D)          # 4.8 GB each for keys and values
    c = tiles(gpu_lib, WHOLE, page, 44)
    ref = c.run()
    big = gpu_lib.Fp8Cache(*(torch.zeros((pages, *t.shape[1:]), dtype=torch.uint8, device="cuda").view(t.dtype)
                             for t in (c.cache.k_codes, c.cache.v_codes, c.cache.k_scales, c.cache.v_scales)))
    n = c.cache.k_codes.shape[0]
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        getattr(big, name).view(torch.uint8)[pages - n:] = getattr(c.cache, name).view(torch.uint8)
    table = [[p + pages - n if p >= 0 else p for p in row] for row in c.table]
    o = gpu_lib.attention_cache_fp8(c.q, big, i32(table), i32(c.lens), cu_seqlens=i32(c.cu), max_length=max(c.lens))
    assert torch.equal(bits(o), bits(ref))
