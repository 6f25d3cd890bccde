"""GPU: attention over the paged e4m3 cache against the oracle in float64, element by element within the bound
that oracle/serving.py derives, plus the output's own bf16 rounding (2^-8).

Caches are built from codes and scales directly, so that the operator is tested by itself; pages lie in
shuffled order and hold NaN codes wherever no token is. Queries are aligned with the last key that they
see and the one after (CPU tests plant such mistakes in the oracle)."""

import numpy as np
import pytest
import torch

from oracle import serving as S

pytestmark = pytest.mark.gpu


def f64(t):
    return t.float().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(lens):
    return [int(c) for c in np.cumsum([0] + list(lens))]


class Case:
    """Sequences of new[b] queries on lens[b] keys in a cache."""

    def __init__(self, lib, new, lens, H, Hk, D, page, seed=0, sharp=1.0, extra_width=0):
        rng = np.random.default_rng(seed)
        self.lib, self.new, self.lens, self.H, self.Hk, self.D, self.page = lib, list(new), list(lens), H, Hk, D, page
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 2
        order = rng.permutation(pages).tolist()
        width = max(1, max(counts)) + extra_width
        self.table, at = [], 0
        for c in counts:
            self.table.append(order[at:at + c] + [-1] * (width - c))
            at += c
        codes = {n: torch.full((pages, Hk, page, D), 0xFF, dtype=torch.uint8) for n in "kv"}
        scales = {n: torch.from_numpy(rng.integers(120, 123, (pages, Hk))).to(torch.uint8) for n in "kv"}
        g = torch.Generator().manual_seed(seed)
        self.keys = []                 # per sequence: k, v [L, Hk, D] in float64
        for b, n in enumerate(lens):
            kv = []
            for name in "kv":
                z = (torch.randn(n, Hk, D, generator=g) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
                vals = z.double()
                for t0 in range(0, n, page):
                    p = self.table[b][t0 // page]
                    part = slice(t0, min(n, t0 + page))
                    codes[name][p, :, : z[part].shape[0]] = z[part].view(torch.uint8).transpose(0, 1)
                    vals[part] = vals[part] * 2.0 ** (scales[name][p].double() - 127.0)[None, :, None]
                kv.append(vals.numpy())
            self.keys.append(kv)
        self.cache = lib.Fp8Cache(codes["k"].view(torch.float8_e4m3fn).cuda(),
                                  codes["v"].transpose(2, 3).contiguous().view(torch.float8_e4m3fn).cuda(),
                                  scales["k"].cuda(), scales["v"].cuda())
        T = sum(new)
        q = torch.randn(T, H, D, generator=g).numpy().astype(np.float64)
        cu = offsets(new)
        for b, (n, L) in enumerate(zip(new, lens)):
            k = self.keys[b][0]
            for i in range(n):
                last = L - n + i
                for j in (last, last + 1):
                    if 0 <= j < L:
                        q[cu[b] + i] += 0.5 * np.repeat(k[j], H // Hk, 0)
        self.q = torch.from_numpy(q * sharp).to(torch.bfloat16).cuda()
        self.cu = cu

    def run(self, causal=True, packed=True, **kw):
        kw.setdefault("max_length", max(self.lens))
        return self.lib.attention_cache_fp8(kw.pop("q", self.q), self.cache, i32(self.table), i32(self.lens),
                                            cu_seqlens=i32(self.cu) if packed else None, causal=causal, **kw)

    def check(self, o, causal=True, scale=None, seqs=None):
        q, o = f64(self.q), f64(o)
        for b in range(len(self.new)) if seqs is None else seqs:
            r = slice(self.cu[b], self.cu[b + 1])
            ref, tol = S.attention(q[r], *self.keys[b], self.new[b], causal, scale)
            tol = (1 + 2.0 ** -8) * tol + 2.0 ** -8 * np.abs(ref)
            err = np.abs(o[r] - ref)
            assert (err <= tol).all(), (b, self.new[b], self.lens[b], float(np.nanmax(err / np.maximum(tol, 1e-30))))


HEADS = [(4, 2, 128), (3, 3, 64), (8, 1, 128), (6, 2, 64), (40, 2, 128)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hk,D", HEADS)
def test_single_tokens(gpu_lib, page, H, Hk, D):
    print(f"[attention_cache] decode page={page} H={H} Hk={Hk} D={D}", flush=True)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 1030]
    c = Case(gpu_lib, [1] * len(lens), lens, H, Hk, D, page, page + H)
    for causal in (True, False):
        o = c.run(causal, packed=False)
        c.check(o, causal)
    assert torch.equal(c.run(True, packed=True).view(torch.int16), o.view(torch.int16)) or H // Hk > 16
    c.check(c.run(True, packed=True), True)


LENGTHS = [([5], [5]), ([1], [1]), ([31, 33], [31, 100]), ([64, 1, 0, 7], [64, 300, 50, 8]), ([65], [400]), ([2, 2, 2], [70, 2, 200]),
           ([130, 17], [130, 1017]), ([300], [1300]), ([257, 3, 90], [300, 900, 95])]


@pytest.mark.parametrize("new,lens", LENGTHS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("H,Hk,D,page", [(4, 2, 128, 16), (3, 3, 64, 64), (5, 1, 128, 128), (14, 2, 64, 32)])
@pytest.mark.parametrize("causal", [False, True])
def test_chunks(gpu_lib, new, lens, H, Hk, D, page, causal):
    print(f"[attention_cache] chunks {new} {lens} H={H} Hk={Hk} D={D} page={page} causal={causal}", flush=True)
    c = Case(gpu_lib, new, lens, H, Hk, D, page, sum(lens) + D)
    c.check(c.run(causal), causal)


@pytest.mark.parametrize("n,L,H,Hk,D,page,causal", [
    (700, 2500, 2, 1, 128, 64, True), (2048, 4100, 1, 1, 64, 16, False), (1500, 1500, 4, 2, 128, 128, True),
    (16, 9000, 4, 1, 128, 32, True), (40, 5000, 8, 1, 128, 64, False), (200, 6001, 3, 1, 64, 128, True)])
def test_long_chunks(gpu_lib, n, L, H, Hk, D, page, causal):
    print(f"[attention_cache] long {n} {L} {H} {Hk} {D} {page} {causal}", flush=True)
    c = Case(gpu_lib, [n], [L], H, Hk, D, page, n)
    c.check(c.run(causal), causal)


@pytest.mark.parametrize("L,H,Hk,D,page", [(20000, 32, 8, 128, 64), (33333, 4, 4, 64, 16), (9999, 15, 1, 128, 128)])
def test_one_token_on_a_long_cache(gpu_lib, L, H, Hk, D, page):
    """Keys shared out among many workgroups, whatever bound of the length the caller gives."""
    print(f"[attention_cache] one token {L}", flush=True)
    c = Case(gpu_lib, [1], [L], H, Hk, D, page, L, extra_width=3)
    for bound in (L, None, 1, 300, 10 ** 7):
        c.check(c.run(packed=False, max_length=bound))


def test_mixed_short_and_long(gpu_lib):
    """Sequences that take one workgroup's share beside one that takes many, and empty ones."""
    lens = [3, 20000, 0, 64, 257, 1, 4000]
    c = Case(gpu_lib, [1] * 7, lens, 8, 2, 128, 32, 5)
    o = c.run(packed=False)
    c.check(o)
    assert not o[2].any()
    c = Case(gpu_lib, [2, 3, 0, 1, 4, 1, 7], lens, 8, 2, 128, 32, 6)
    c.check(c.run())


def test_rows_without_keys_are_zero(gpu_lib):
    """More queries than keys: the first see none."""
    for H, Hk, D in ((4, 2, 128), (3, 3, 64)):
        for new, lens in (([9, 5], [4, 0]), ([200, 300], [100, 0]), ([1, 70], [0, 3])):
            c = Case(gpu_lib, new, lens, H, Hk, D, 16, 9)
            out = torch.full_like(c.q, float("nan"))
            o = c.run(out=out)
            c.check(o)
            for b, (n, L) in enumerate(zip(new, lens)):
                assert not o[c.cu[b]: c.cu[b] + max(0, n - L)].any()
            # without a causal mask only sequences without keys are empty
            o = c.run(False)
            c.check(o, False)


def test_stale_contents_and_missing_pages(gpu_lib):
    """Pages past a sequence's end may hold anything; entries outside the cache count as zero keys and values."""
    for new in ([1, 1], [40, 200]):
        c = Case(gpu_lib, new, [300, 290], 4, 2, 128, 32, 11)
        clean = c.run()
        spare = [p for p in range(c.cache.k_codes.shape[0]) if p not in sum(c.table, [])]
        c.table[0] += [spare[0]] * 4
        c.table[1] += [spare[1]] * 4
        c.cache.k_scales[spare] = 255
        c.cache.v_scales[spare] = 255
        assert torch.equal(c.run().view(torch.int16), clean.view(torch.int16))
        for entry in (-1, -2 ** 31, 2 ** 31 - 1, c.cache.k_codes.shape[0]):
            c.table[1][3] = entry
            c.keys[1][0][96:128] = 0.0
            c.keys[1][1][96:128] = 0.0
            c.check(c.run())
        # lengths past the table's width are what it holds
        long = [len(c.table[0]) * 32 + 1000, 290]
        o = c.lib.attention_cache_fp8(c.q, c.cache, i32(c.table), i32(long), cu_seqlens=i32(c.cu))
        assert bool(torch.isnan(o[: new[0]].float()).any())   # the spare pages' NaN is in reach now
        assert bool(torch.isfinite(o[new[0]:].float()).all())
        o = c.lib.attention_cache_fp8(c.q, c.cache, i32(c.table), i32([-5, 290]), cu_seqlens=i32(c.cu))
        assert not o[: new[0]].any()


def test_non_finite_pages_reach_only_their_sequence_and_head(gpu_lib):
    for new in ([1, 1, 1], [30, 100, 7]):
        for which in ("k_scales", "v_scales"):
            c = Case(gpu_lib, new, [200, 210, 220], 4, 2, 128, 64, 12)
            clean = c.run()
            getattr(c.cache, which)[c.table[1][0], 1] = 255
            o = c.run()
            rows = slice(c.cu[1], c.cu[2])
            assert bool(torch.isnan(o[rows, 2:].float()).all())
            ok = torch.ones_like(o, dtype=torch.bool)
            ok[rows, 2:] = False
            assert torch.equal(o[ok], clean[ok])


def test_future_keys_that_are_not_finite_are_not_seen(gpu_lib):
    """A NaN key after a query's own does not reach it."""
    for n in (4, 100):
        c = Case(gpu_lib, [n], [n + 60], 4, 2, 128, 16, 13)
        clean = c.run()
        last = n + 59
        c.cache.k_codes.view(torch.uint8)[c.table[0][last // 16], :, last % 16, 5] = 0x7F
        o = c.run()
        assert torch.equal(o[:-1], clean[:-1]) and bool(torch.isnan(o[-1].float()).all())


@pytest.mark.parametrize("scale,gain", [(2.0 ** -10, 1.0), (1.0, 60.0), (2.0 ** 20, 1.0), (1e-30, 1.0), (2.0 ** 10, 1e30)])
def test_extreme_scores(gpu_lib, scale, gain):
    """Scores from nothing to the ends of fp32: single keys win, or all count the same; nothing becomes NaN."""
    for new in ([1, 1], [90, 8]):
        c = Case(gpu_lib, new, [500, 130], 4, 2, 128, 64, 14)
        c.q = (c.q.float() * gain).bfloat16()
        o = c.run(scale=scale)
        assert bool(torch.isfinite(o.float()).all())
        if gain <= 60.0 and scale <= 1.0:
            c.check(o, scale=scale)


def test_equal_keys_far_from_zero(gpu_lib):
    """Equal keys, whose scores are equal however large: o is the mean of v."""
    for new in ([1], [70]):
        for sign in (1.0, -1.0):
            c = Case(gpu_lib, new, [333], 2, 1, 64, 32, 15)
            c.cache.k_codes.view(torch.uint8)[:] = 0x7E        # 448
            c.cache.k_scales[:] = 200
            c.q[:] = sign * 3e7
            o = c.run(False)
            mean = torch.from_numpy(c.keys[0][1].mean(0)).cuda()
            err = (o.double() - mean).abs()
            assert bool((err <= 2.0 ** -7 * torch.from_numpy(np.abs(c.keys[0][1]).mean(0)).cuda()).all())


def test_old_keys_keep_their_weight(gpu_lib):
    """Scores that climb from key to key move the maximum often; sums over exact inputs show what rescaling loses."""
    L, page = 4096, 64
    for new in ([1], [40]):
        c = Case(gpu_lib, new, [L], 2, 1, 64, page, 16)
        k = torch.zeros(L, 64)
        k[:, 0] = torch.arange(L) // 16 * 0.5                    # values of e4m3 up to 128 in steps: rounded below
        k = k.to(torch.float8_e4m3fn)
        order = torch.tensor(c.table[0][: L // page])
        c.cache.k_codes.view(torch.uint8)[order, 0] = k.view(torch.uint8).view(L // page, page, 64).cuda()
        c.cache.k_scales[:] = 127
        c.keys[0][0] = k.double().numpy()[:, None]
        q = torch.zeros(sum(new), 2, 64)
        q[:, 0, 0], q[:, 1, 0] = 1.5, -0.75
        c.q = q.bfloat16().cuda()
        for scale in (0.125, 2.0):
            c.check(c.run(False, scale=scale), False, scale)


def test_views_strides_streams_and_guards(gpu_lib):
    for new, packed in (([1] * 5, False), ([3, 90, 1, 0, 40], True)):
        H, Hk, D = 6, 2, 128
        c = Case(gpu_lib, new, [100, 900, 64, 1, 77], H, Hk, D, 32, 17)
        ref = c.run(packed=packed)
        T = sum(new)
        fused = torch.randn(T, H + 3, D, device="cuda").bfloat16()
        fused[:, 1:H + 1] = c.q
        heads_first = torch.full((H, T + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
        out = heads_first[:, 1:T + 1].transpose(0, 1)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = c.run(packed=packed, q=fused[:, 1:H + 1], out=out)
        s.synchronize()
        assert got is out and torch.equal(out, ref)
        assert bool((heads_first[:, 0] == 7).all()) and bool((heads_first[:, -1] == 7).all())
        need = gpu_lib.attention_cache_fp8_workspace_bytes(T, len(new), H, Hk, D, 900, packed)
        work = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        assert torch.equal(c.run(packed=packed, workspace=work[256:256 + need]), ref)
        assert bool((work[:256] == 0xA5).all()) and bool((work[256 + need:] == 0xA5).all())


def test_rows_outside_the_offsets_are_left_alone(gpu_lib):
    for lens in ([100, 300], [100, 30000]):
        c = Case(gpu_lib, [3, 4], lens, 4, 2, 64, 64, 18)
        q = torch.cat([c.q[:2], c.q, c.q[:5]])
        out = torch.full_like(q, 7.0)
        c.lib.attention_cache_fp8(q, c.cache, i32(c.table), i32(c.lens), cu_seqlens=i32([2, 5, 9]), max_length=max(lens), out=out)
        c.check(out[2:9])   # (not bit for bit a call without the other rows: keys may be shared out differently)
        assert bool((out[:2] == 7).all()) and bool((out[9:] == 7).all())


@pytest.mark.parametrize("cu", [[0, 40, 20, 60], [-5, 10, 30, 60], [0, 10, 30, 1000], [60, 40, 20, 0], [50, 50, 50, 60]])
def test_bad_offsets_stay_inside(gpu_lib, cu):
    c = Case(gpu_lib, [20, 20, 20], [100, 5000, 64], 4, 2, 64, 16, 19)
    base = torch.full((80, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    c.lib.attention_cache_fp8(c.q, c.cache, i32(c.table), i32(c.lens), cu_seqlens=i32(cu), out=base[10:70])
    torch.cuda.synchronize()
    assert bool((base[:10] == 3).all()) and bool((base[70:] == 3).all())


def test_graphs_sharing_a_workspace(gpu_lib):
    """Two captured calls with one workspace, replayed in turn between eager work; lengths grow in between."""
    cases = [Case(gpu_lib, [1] * 3, [3000, 40, 700], 8, 2, 128, 64, 20), Case(gpu_lib, [20, 1, 9], [2000, 64, 900], 8, 2, 128, 64, 21)]
    need = max(gpu_lib.attention_cache_fp8_workspace_bytes(sum(c.new), 3, 8, 2, 128, 3000, p) for c, p in zip(cases, (False, True)))
    work = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    graphs = []
    for c, packed in zip(cases, (False, True)):
        st = dict(out=torch.empty_like(c.q), lens=i32(c.lens), table=i32(c.table), cu=i32(c.cu) if packed else None)

        def call(c=c, st=st):
            c.lib.attention_cache_fp8(c.q, c.cache, st["table"], st["lens"], cu_seqlens=st["cu"], max_length=3000, out=st["out"], workspace=work)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, c, st))
    for rep in range(4):
        for g, c, st in graphs:
            st["lens"].copy_(i32([max(n, x - 17 * rep) for n, x in zip(c.new, c.lens)]))
            ref = c.lib.attention_cache_fp8(c.q, c.cache, st["table"], st["lens"], cu_seqlens=st["cu"], max_length=3000)
            st["out"].zero_()
            work.fill_(0x5A)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(st["out"].view(torch.int16), ref.view(torch.int16)), rep


def test_results_repeat(gpu_lib):
    c = Case(gpu_lib, [1] * 4, [9000, 40, 300, 5000], 8, 2, 128, 64, 22)
    first = c.run(packed=False)
    assert all(torch.equal(c.run(packed=False), first) for _ in range(5))


def test_many_sequences(gpu_lib):
    rng = np.random.default_rng(3)
    new = np.where(rng.random(900) < 0.4, 0, np.where(rng.random(900) < 0.05, 30, 1)).tolist()
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 200, 900))]
    c = Case(gpu_lib, new, lens, 4, 2, 64, 16, 23)
    o = c.run()
    c.check(o, seqs=[b for b in range(900) if new[b] > 0][::7])


def test_pages_past_32_bits(gpu_lib):
    """A cache of more than 4 GiB of codes: pages at its far end."""
    pages, Hk, D, page = 36000, 8, 128, 128        # 4.7 GB each for keys and values
    c = Case(gpu_lib, [1, 70], [500, 300], 16, Hk, D, page, 24)
    ref = c.run()
    big = gpu_lib.Fp8Cache(*(torch.zeros((pages, *t.shape[1:]), dtype=torch.uint8, device="cuda").view(t.dtype)
                             for t in (c.cache.k_codes, c.cache.v_codes, c.cache.k_scales, c.cache.v_scales)))
    n = c.cache.k_codes.shape[0]
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        getattr(big, name).view(torch.uint8)[pages - n:] = getattr(c.cache, name).view(torch.uint8)
    table = [[p + pages - n if p >= 0 else p for p in row] for row in c.table]
    o = gpu_lib.attention_cache_fp8(c.q, big, i32(table), i32(c.lens), cu_seqlens=i32(c.cu), max_length=500)
    assert torch.equal(o.view(torch.int16), ref.view(torch.int16))
    # and tokens appended there come back
    k = torch.randn(3, Hk, D, device="cuda").bfloat16()
    gpu_lib.cache_append_fp8(k, k, big, i32([[pages - 1], [0], [pages - 2]]), i32([0, 0, 0]))
    back = gpu_lib.cache_read_fp8(big, i32([[pages - 1], [0], [pages - 2]]), i32([0, 0, 0]))
    assert all(bool(((x.float() - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -16).all()) for x in back)
