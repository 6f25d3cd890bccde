"""Measured cases of serving in 8-bit floating point: linears, rotary positions, and attention over a cache.

Four operators of a decoder step. The linear in 8-bit floating point (e4m3) with a scale per 128 input channels of
a token and per 128 x 128 block of the weight. Rotary positions on the first part of a head with frequencies scaled
for long contexts. Writing keys and values into pages of an e4m3 cache with a power-of-two scale per page and head,
with the values read back; and attention over such a cache, for single tokens and for chunks. The widths
are those of a diffusion transformer (3840, FFN 10240, 30 heads of 128) and of a text encoder with grouped heads
(32 heads of 128 on 8).

A cache holds keys as [pages, heads, page, D] and values as [pages, heads, D, page] codes, its scales are exponents
with a bias of 127; a table per sequence lists its pages in order.

run() is the plain form in elementary torch operations, or with `own` the framework's calls.
"""

import math
import random

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through an attention-sized linear: latency, the weight's bytes
        dict(name="fp8 linear, one token", op="linear", M=1, K=3840, N=3840, smooth=False, bias=True),
        # a ragged batch of prompt tokens through the FFN's down projection
        dict(name="fp8 linear, 333 tokens, w2", op="linear", M=333, K=10240, N=3840, smooth=True, bias=True),
        # the 1024^2 FFN up projection: the compute-bound case
        dict(name="fp8 linear, 1024 w1", op="linear", M=4096, K=3840, N=10240, smooth=True, bias=False),
        # a decoding batch's q and k, half of each head turned, far positions: latency
        dict(name="rotary, 32 decoded tokens", op="rope", T=32, H=32, Hk=8, D=128, R=64, interleaved=False,
             factor=8.0, original=8192, amplitude=1.2),
        # packed prompts, a quarter of each head of 64 turned, positions interpolated
        dict(name="rotary, packed prompts", op="rope", T=4099, H=24, Hk=8, D=64, R=16, interleaved=False, factor=4.0,
             original=0, amplitude=1.0),
        # a long document, whole heads, neighbouring pairs: bandwidth
        dict(name="rotary, long", op="rope", T=16896, H=30, Hk=30, D=128, R=128, interleaved=True, factor=4.0,
             original=4096, amplitude=1.1386),
        # a decoding batch's new keys and values into pages that are partly filled: latency
        dict(name="append, 32 decoded tokens", op="append", T=32, B=32, cuts=1, past=1000, Hk=8, D=128, page=64),
        # a batch of prompts behind ragged beginnings
        dict(name="append, packed prompts", op="append", T=16411, B=13, cuts=3, past=333, Hk=8, D=128, page=64),
        # one sequence with a long cache, a single token: the cache's bytes over the whole chip
        dict(name="attention, one token, long cache", op="attention", T=1, B=1, cuts=1, past=65536, H=32, Hk=8, D=128,
             page=64, causal=True),
        # a decoding batch of ragged lengths: the ordinary serving call
        dict(name="attention, 32 decoded tokens", op="attention", T=32, B=32, cuts=2, past=2500, H=32, Hk=8, D=128,
             page=64, causal=True),
        # prompts cut into chunks, each behind what is cached of it, small pages
        dict(name="attention, packed chunks", op="attention", T=4099, B=13, cuts=3, past=700, H=32, Hk=8, D=128,
             page=16, causal=True),
        # a chunk of image tokens that sees everything cached before it and itself: the largest
        dict(name="attention, chunk on a long cache", op="attention", T=2048, B=1, cuts=1, past=14848, H=30, Hk=30,
             D=128, page=128, causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "rope", "append", "attention", "attention"])
    if op == "linear":
        K, N = 16 * _log(rng, 16, 640), _log(rng, 100, 11520)
        return dict(op=op, M=_log(rng, 1, min(8192, 4096 * 3840 * 10240 // (K * N))), K=K, N=N,
                    smooth=rng.random() < 0.5, bias=rng.random() < 0.5)
    Hk = rng.choice([1, 4, 6, 8, 15])
    H = Hk * rng.choice([1, 2, 3, 4, 8] if Hk <= 8 else [1, 2])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        T = _log(rng, 1, min(16896, 16896 * 60 * 128 // ((H + Hk) * D)))
        return dict(op=op, T=T, H=H, Hk=Hk, D=D, R=8 * rng.randint(1, D // 8), interleaved=rng.random() < 0.5,
                    factor=rng.choice([1.0, 2.0, 8.0, 31.5]), original=rng.choice([0, 4096, 8192]),
                    amplitude=rng.choice([1.0, 1.2079]))
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    B = _log(rng, 1, 32)
    T = B if rng.random() < 0.4 else B * _log(rng, 1, 16411 // B if op == "append" else 2900 // B)
    if op == "append":
        return dict(op=op, T=T, B=B, cuts=rng.randrange(1000), past=_log(rng, 1, 2000), Hk=Hk, D=D, page=page)
    # keys behind each sequence's queries, so that neither the cache nor the products pass the largest case's
    past = min(65536 // B, 2048 * 16896 * 30 // (T * H) - 2 * T // B)
    return dict(op=op, T=T, B=B, cuts=rng.randrange(1000), past=_log(rng, 1, max(1, past)), H=H, Hk=Hk, D=D, page=page,
                causal=rng.random() < 0.7)


def _shares(total, parts, cuts):
    """`parts` lengths of sum `total`, each between about a quarter and twice the mean."""
    r = random.Random(cuts)
    w = [r.uniform(0.25, 1.75) for _ in range(parts)]
    edges = [int(round(total * sum(w[:i]) / sum(w))) for i in range(parts)] + [total]
    return [edges[i + 1] - edges[i] for i in range(parts)]


def _lengths(case):
    """Per sequence: its new tokens, and the tokens already there."""
    B = case["B"]
    new = [1] * B if case["T"] == B else _shares(case["T"], B, case["cuts"])
    return new, _shares(case["past"] * B, B, case["cuts"] + 1)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    edges = [0]
    for n in lens:
        edges.append(edges[-1] + n)
    return _ints(edges)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, M, K):
    """Activations of a transformer block: unit normal with one channel in a hundred 20 times larger."""
    x = _normal(gen, M, K)
    x[:, torch.randperm(K, generator=gen, device="cuda")[: K // 100]] *= 20.0
    return x.to(torch.bfloat16)


def _keys(gen, rows, heads, D):
    """Keys: a few channels of each head carry larger values."""
    x = _normal(gen, rows, heads, D)
    x[:, :, :: 16] *= 4.0
    return x


def _pages(gen, lens, page):
    """A table of pages for sequences of these lengths, in shuffled order, and their number (some are spare)."""
    counts = [-(-n // page) for n in lens]
    total = sum(counts) + 5
    order = torch.randperm(total, generator=gen, device="cuda").int()
    width = max(counts)
    first = torch.tensor([sum(counts[:i]) for i in range(len(counts))], device="cuda")
    at = torch.arange(width, device="cuda")
    held = at < torch.tensor(counts, device="cuda")[:, None]
    table = torch.where(held, order[(first[:, None] + at).clamp_max(total - 1)], torch.tensor(0, device="cuda").int())
    return table.int().contiguous(), total


def _block_exponent(amax):
    """The least e with amax <= 448 * 2^e, at least -100."""
    m, e = torch.frexp(amax)
    return (e - 8 - (m <= 0.875).int()).clamp_min(-100)


def _power(e):
    """2^e in 32 bits, -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(z):
    """e4m3 codes, ties to even, as bytes."""
    return z.to(torch.float8_e4m3fn).view(torch.uint8)


def _values_of(codes):
    return codes.view(torch.float8_e4m3fn).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = _activations(gen, M, K)
        # a weight held in 8 bits: codes and a scale (no power of two) per block of 128 x 128
        w = _normal(gen, N, K) * 0.02
        blocks = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128)).unflatten(1, (-1, 128)).unflatten(0, (-1, 128))
        s["ws"] = (blocks.abs().amax((1, 3)) / 448.0).contiguous()
        w = (w / s["ws"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]).clamp(-448.0, 448.0)
        s["w"] = w.to(torch.float8_e4m3fn)
        s["bias"] = (_normal(gen, N) * 0.01).to(torch.bfloat16) if case["bias"] else None
        s["smooth"] = None
        if case["smooth"]:
            s["smooth"] = s["x"].float().abs().amax(0).clamp_min(1e-6).rsqrt().to(torch.bfloat16)
        return s
    if op == "rope":
        T, H, Hk, D = case["T"], case["H"], case["Hk"], case["D"]
        qkv = _normal(gen, T, (H + 2 * Hk) * D).to(torch.bfloat16)
        s["q"] = qkv[:, : H * D].view(T, H, D)
        s["k"] = qkv[:, H * D: (H + Hk) * D].view(T, Hk, D)
        # positions of packed tokens, each run from somewhere in a long context
        start = torch.randint(0, 131072, (T // 512 + 1,), generator=gen, device="cuda")
        i = torch.arange(T, device="cuda")
        s["pos"] = (start[i // 512] + i % 512).int()
        return s
    Hk, D, page = case["Hk"], case["D"], case["page"]
    new, past = _lengths(case)
    T = sum(new)
    full = [n + p for n, p in zip(new, past)]
    s["table"], pages = _pages(gen, full, page)
    s["cu"] = None if case["T"] == case["B"] else _offsets(new)
    s["past"], s["lens"] = _ints(past), _ints(full)
    s["longest"], s["most"] = max(full), max(new)
    # the cache as it stands: every page holds tokens (new ones overwrite theirs)
    held = _keys(gen, pages * page, Hk, D).view(pages, page, Hk, D).transpose(1, 2)
    e = _block_exponent(held.abs().amax((2, 3)))
    s["kc"] = _codes((held * _power(-e)[:, :, None, None]).contiguous()).view(torch.float8_e4m3fn)
    s["ks"] = (e + 127).to(torch.uint8)
    held = _normal(gen, pages, Hk, D, page)
    e = _block_exponent(held.abs().amax((2, 3)))
    s["vc"] = _codes(held * _power(-e)[:, :, None, None]).view(torch.float8_e4m3fn)
    s["vs"] = (e + 127).to(torch.uint8)
    if op == "append":
        qkv = torch.cat([_keys(gen, T, Hk, D), _normal(gen, T, Hk, D)], 1)
        # a token in fifty is louder, so that scales of pages in use grow
        qkv *= torch.where(torch.rand(T, 1, 1, generator=gen, device="cuda") < 0.02, 8.0, 1.0)
        qkv = qkv.to(torch.bfloat16)
        s["k"], s["v"] = qkv[:, :Hk], qkv[:, Hk:]
        # what is read back: the pages that the new tokens fall into, up to their last token
        starts = [p // page * page for p in past]
        counts = [f - b for f, b in zip(full, starts)]
        s["starts"], s["back"], s["rows"] = _ints(starts), _offsets(counts), sum(counts)
    else:
        s["q"] = _normal(gen, T, case["H"] * D).to(torch.bfloat16).view(T, case["H"], D)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_linear(s):
    v = s["x"].float()
    M, K = v.shape
    if s["smooth"] is not None:
        v = v * s["smooth"].float()
    block = torch.arange(K, device=v.device) // 128
    amax = torch.nn.functional.pad(v.abs(), (0, -K % 128)).unflatten(1, (-1, 128)).amax(2)
    e = _block_exponent(amax)[:, block]
    a = _values_of(_codes(v * _power(-e))) * _power(e)
    w = s["w"].float() * s["ws"][torch.arange(s["w"].shape[0], device=v.device) // 128][:, block]
    y = a @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(torch.bfloat16)


def _plain_rope_one(z, c, cos, sin):
    R = c["R"]
    z, rest = z[..., :R].float(), z[..., R:]
    if c["interleaved"]:
        a, b = z[..., 0::2], z[..., 1::2]
    else:
        a, b = z.chunk(2, 2)
    a, b = a * cos - b * sin, b * cos + a * sin
    out = torch.stack([a, b], 3).flatten(2) if c["interleaved"] else torch.cat([a, b], 2)
    return torch.cat([out.to(torch.bfloat16), rest], 2)


def _plain_rope(s):
    c = s["case"]
    freq = 10000.0 ** (-2.0 * torch.arange(c["R"] // 2, device="cuda", dtype=torch.float64) / c["R"])
    if c["original"]:
        rotations = c["original"] * freq / (2.0 * math.pi)
        kept = ((rotations - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        freq = freq * (kept + (1.0 - kept) / c["factor"])
    else:
        freq = freq / c["factor"]
    angle = s["pos"].double()[:, None] * freq
    cos = (c["amplitude"] * angle.cos()).float()[:, None]
    sin = (c["amplitude"] * angle.sin()).float()[:, None]
    return _plain_rope_one(s["q"], c, cos, sin), _plain_rope_one(s["k"], c, cos, sin)


def _sequence_of(cu, rows):
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(rows, device=cu.device, dtype=torch.int32), right=True)


def _plain_append_one(new, codes, scales, page_of, slot):
    """Into codes [pages, heads, page, D] in bytes, a block of tokens per page: its scale grows to hold the new ones."""
    pages, Hk, P, D = codes.shape
    top = torch.zeros(pages, Hk, device=new.device).index_reduce_(0, page_of, new.abs().amax(2), "amax")
    first = torch.full((pages,), P, device=new.device).index_reduce_(0, page_of, slot, "amin")
    touched = (first < P).nonzero()[:, 0]
    first = first[touched][:, None]
    old = torch.where(first > 0, scales[touched].int() - 127, -100)
    e = torch.maximum(old, _block_exponent(top[touched]))
    # what was there, in units of the new scale
    block = codes[touched]
    again = _codes(_values_of(block) * _power(old - e)[:, :, None, None])
    grown = (e > old)[:, :, None, None] & (torch.arange(P, device=new.device) < first)[:, None, :, None]
    codes[touched] = torch.where(grown, again, block)
    scales[touched] = (e + 127).to(torch.uint8)
    at = scales[page_of].int() - 127
    codes[page_of, :, slot] = _codes(new * _power(-at)[:, :, None])


def _plain_append(s):
    P = s["case"]["page"]
    k, v = s["k"].float(), s["v"].float()
    T = k.shape[0]
    cu = s["cu"] if s["cu"] is not None else torch.arange(T + 1, device=k.device, dtype=torch.int32)
    b = _sequence_of(cu, T)
    pos = s["past"][b] + torch.arange(T, device=k.device) - cu[b]
    page_of, slot = s["table"][b, pos // P].long(), (pos % P).long()
    kc, vc = s["kc"].view(torch.uint8), s["vc"].view(torch.uint8)
    _plain_append_one(k, kc, s["ks"], page_of, slot)
    turned = vc.transpose(2, 3).contiguous()
    _plain_append_one(v, turned, s["vs"], page_of, slot)
    vc.copy_(turned.transpose(2, 3))
    # read back
    b = _sequence_of(s["back"], s["rows"])
    pos = s["starts"][b] + torch.arange(s["rows"], device=k.device) - s["back"][b]
    page_of, slot = s["table"][b, pos // P].long(), (pos % P).long()
    kb = _values_of(kc[page_of, :, slot]) * _power(s["ks"][page_of].int() - 127)[:, :, None]
    vb = _values_of(vc[page_of, :, :, slot]) * _power(s["vs"][page_of].int() - 127)[:, :, None]
    return kb.to(torch.bfloat16), vb.to(torch.bfloat16)


def _plain_attention(s):
    """The sequences padded to the longest, in queries and in keys, the padding masked."""
    c, q, table = s["case"], s["q"], s["table"].long()
    T, H, D = q.shape
    Hk, G, (B, W) = c["Hk"], c["H"] // c["Hk"], table.shape
    L, n = s["longest"], s["most"]
    k = _values_of(s["kc"].view(torch.uint8)[table]) * _power(s["ks"][table].int() - 127)[..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(B, Hk, D, W * c["page"])[..., :L].contiguous()
    v = _values_of(s["vc"].view(torch.uint8)[table]) * _power(s["vs"][table].int() - 127)[..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, Hk, W * c["page"], D)[:, :, :L].contiguous()
    cu = s["cu"] if s["cu"] is not None else torch.arange(T + 1, device=q.device, dtype=torch.int32)
    at = torch.arange(n, device=q.device)
    count = (cu[1:] - cu[:-1]).long()
    row = (cu[:-1, None].long() + at).clamp_max(T - 1)
    qp = q[row].float().view(B, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, D)
    p = torch.matmul(qp, k).mul_(D ** -0.5).view(B, Hk, G, n, L)
    j = torch.arange(L, device=q.device)
    last = s["lens"].long()[:, None] - 1 - ((count[:, None] - 1 - at) if c["causal"] else 0 * at)   # [B, n]
    p.masked_fill_((j > last[:, :, None])[:, None, None], -math.inf)
    p.sub_(p.amax(4, keepdim=True)).exp_()
    p.div_(p.sum(4, keepdim=True))
    o = torch.matmul(p.view(B, Hk, G * n, L), v).view(B, Hk, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H, D)
    return o[at < count[:, None]].to(torch.bfloat16)


def run(s):
    if own:
        return _run_own(s)
    return {"linear": _plain_linear, "rope": _plain_rope, "append": _plain_append, "attention": _plain_attention}[s["op"]](s)


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    from bit_w4a4_quantized_quantize_amd import ops
    c, op = s["case"], s["op"]
    if op == "linear":
        return ops.linear_fp8(s["x"], s["w"], s["ws"], bias=s["bias"], smooth=s["smooth"])
    if op == "rope":
        return ops.rope_scaled(s["q"], s["k"], s["pos"], rotary_dim=c["R"], theta=10000.0,
                               interleaved=c["interleaved"], factor=c["factor"], original_length=c["original"],
                               low_rotations=1.0, high_rotations=32.0, amplitude=c["amplitude"])
    cache = ops.Fp8Cache(s["kc"], s["vc"], s["ks"], s["vs"])
    if op == "append":
        ops.cache_append_fp8(s["k"], s["v"], cache, s["table"], s["past"], cu_seqlens=s["cu"])
        return ops.cache_read_fp8(cache, s["table"], s["starts"], s["back"], s["rows"])
    return ops.attention_cache_fp8(s["q"], cache, s["table"], s["lens"], cu_seqlens=s["cu"], causal=c["causal"],
                                   max_length=s["longest"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + N * K + 4 * -(-N // 128) * -(-K // 128) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "rope":
        n = case["T"] * (case["H"] + case["Hk"])
        return {"bytes": 4 * n * case["D"] + 4 * case["T"], "flops": 3 * n * case["R"]}
    new, past = _lengths(case)
    Hk, D, P = case["Hk"], case["D"], case["page"]
    if op == "append":
        # the new tokens read, their codes written; the pages' tokens read back and written as bf16
        back = sum(n + p % P for n, p in zip(new, past))
        return {"bytes": 2 * Hk * D * (3 * sum(new) + 3 * back), "flops": 4 * Hk * D * sum(new)}
    H = case["H"]
    pairs = sum(n * p + (n * (n + 1) // 2 if case["causal"] else n * n) for n, p in zip(new, past))
    return {"bytes": 4 * case["T"] * H * D + 2 * Hk * D * sum(n + p for n, p in zip(new, past)), "flops": 4 * H * D * pairs}


# ---------------------------------------------------------------- in 64 bits

def _two_to(e):
    """2^e exactly (pow and exp2 may be off in the last place, which would break ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _least_power(top):
    """The exponent of the least power of two that `top` is at most 448 times as large as, at least -100."""
    e = torch.ceil(torch.log2(top / 448.0)).clamp_min(-100.0)
    e = torch.where(top > 448.0 * _two_to(e), e + 1, e)
    return torch.where((top <= 448.0 * _two_to(e - 1)) & (e > -100), e - 1, e)


def _e4m3(z):
    """The nearest value of 3 fraction bits and exponents from -6 on, ties to even."""
    step = _two_to(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3.0)
    return torch.round(z / step) * step


def _exact_linear(s):
    v, w = s["x"].double(), s["w"].float().double()
    if s["smooth"] is not None:
        v = v * s["smooth"].double()
    y = torch.zeros(v.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for p, k in enumerate(range(0, v.shape[1], 128)):
        u = _two_to(_least_power(v[:, k: k + 128].abs().max(1, keepdim=True).values))
        scale = s["ws"][:, p].double().repeat_interleave(128)[: w.shape[0]]
        y += (_e4m3(v[:, k: k + 128] / u) * u) @ (w[:, k: k + 128] * scale[:, None]).T
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_rope(z, s):
    c, R = s["case"], s["case"]["R"]
    out = z.double()
    src = out.clone()
    for i in range(R // 2):
        f = 10000.0 ** (-2.0 * i / R)
        share = 0.0
        if c["original"]:
            share = min(1.0, max(0.0, (c["original"] * f / math.tau - 1.0) / 31.0))
        f = share * f + (1.0 - share) * f / c["factor"]
        turn = torch.polar(torch.full((z.shape[0], 1), c["amplitude"], dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * f)
        lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
        r = torch.complex(src[:, :, lo], src[:, :, hi]) * turn
        out[:, :, lo], out[:, :, hi] = r.real, r.imag
    return out


def _values(codes, scales, pages, turned):
    """Tokens of these pages in order, [tokens, heads, D], in 64 bits."""
    z = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float().double() * _two_to(scales[pages].int() - 127)[:, :, None, None]
    return (z.permute(0, 3, 1, 2) if turned else z.permute(0, 2, 1, 3)).flatten(0, 1)


def _exact_append(s, new, codes, scales, turned):
    out = []
    P, edges = s["case"]["page"], (list(range(s["case"]["B"] + 1)) if s["cu"] is None else s["cu"].tolist())
    for b, past in enumerate(s["past"].tolist()):
        z = new[edges[b]: edges[b + 1]].double()
        first = past // P
        while z.shape[0]:
            page, held = s["table"][b, first].item(), past % P
            took, z = z[: P - held], z[P - held:]
            e = _least_power(took.abs().amax((0, 2)))
            if held:
                e = torch.maximum(e, scales[page].double() - 127.0)
                was = _values(codes, scales, [page], turned)[:held]
                out.append(_e4m3(was / _two_to(e)[:, None]) * _two_to(e)[:, None])
            out.append(_e4m3(took / _two_to(e)[:, None]) * _two_to(e)[:, None])
            past, first = (first + 1) * P, first + 1
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_linear(s)
    if op == "rope":
        return _exact_rope(s["q"], s), _exact_rope(s["k"], s)
    if op == "append":
        return _exact_append(s, s["k"], s["kc"], s["ks"], False), _exact_append(s, s["v"], s["vc"], s["vs"], True)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    new, past = _lengths(case)
    start = 0
    for b, (n, held) in enumerate(zip(new, past)):
        pages = s["table"][b, : -(-(n + held) // case["page"])].tolist()
        k = _values(s["kc"], s["ks"], pages, False)[: n + held]
        v = _values(s["vc"], s["vs"], pages, True)[: n + held]
        rows = slice(start, start + n)
        start += n
        for h in range(case["H"]):
            kv = h // (case["H"] // case["Hk"])
            a = s["q"][rows, h].double() @ k[:, kv].T / math.sqrt(case["D"])
            if case["causal"]:
                a += torch.triu(torch.full_like(a, -math.inf), 1 + held)
            out[rows, h] = torch.softmax(a, 1) @ v[:, kv]
    return out
