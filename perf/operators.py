"""Measured cases of the operators between a transformer block's quantised linears.

Four operators: the linear in 8-bit integers, the norms before and after a block with its gate and residual
scale, rotary positions with several axes, and attention over packed sequences. The cases are those of a
diffusion transformer of width 3840 (30 heads of 128, FFN width 10240) at 1024^2 (4096 tokens) and 2048px
(16384 image + 512 text tokens), its single-token and text-only calls, packed prompts of a text encoder with
grouped heads, and video tokens with heads of 64.

run() is the plain form in elementary torch operations, or with `own` the framework's calls.
"""

import math
import random

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a single token through a modulation-sized linear: latency, the weight's bytes
        dict(name="int8 linear, one token", op="linear", M=1, K=3840, N=3840, smooth=False, bias=True),
        # a ragged batch of text tokens through the FFN's down projection
        dict(name="int8 linear, 333 tokens, w2", op="linear", M=333, K=10240, N=3840, smooth=True, bias=True),
        # the 1024^2 FFN up projection, the compute-bound case
        dict(name="int8 linear, 1024 w1", op="linear", M=4096, K=3840, N=10240, smooth=True, bias=False),
        # block boundary whose norm hands its codes to the next 8-bit linear (attention's out width)
        dict(name="norm into int8 linear, 1024", op="norm_linear", M=4096, K=3840, N=3840, G=1, cuts=1),
        # block boundary of a prompt's text tokens: latency
        dict(name="norm, 77 tokens", op="norm", M=77, K=3840, G=1, cuts=1),
        # block boundary of three packed images of 2048px in all: bandwidth
        dict(name="norm, 2048 packed", op="norm", M=16896, K=3840, G=3, cuts=2),
        # a text prompt's q and k: latency
        dict(name="rotary, 77 tokens", op="rope", T=77, H=30, Hk=30, D=128, axes="32,48,48", norm=True,
             interleaved=True),
        # 2048px image tokens, q and k read out of the fused qkv output
        dict(name="rotary, 2048", op="rope", T=16896, H=30, Hk=30, D=128, axes="32,48,48", norm=True,
             interleaved=True),
        # video tokens, grouped heads of 64, half-split pairs, no head norm
        dict(name="rotary, video", op="rope", T=8190, H=24, Hk=8, D=64, axes="16,24,24", norm=False,
             interleaved=False),
        # a text encoder's packed prompts: causal, grouped heads, odd lengths
        dict(name="attention, packed prompts", op="attention", T=4099, B=13, cuts=3, H=32, Hk=8, D=128, causal=True),
        # 1024^2 image, full
        dict(name="attention, 1024", op="attention", T=4096, B=1, cuts=1, H=30, Hk=30, D=128, causal=False),
        # 2048px image with its text, full: the largest
        dict(name="attention, 2048", op="attention", T=16896, B=1, cuts=1, H=30, Hk=30, D=128, causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "norm_linear", "norm", "rope", "attention"])
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 8192), K=16 * _log(rng, 16, 640), N=_log(rng, 100, 11520),
                    smooth=rng.random() < 0.5, bias=rng.random() < 0.5)
    if op == "norm_linear":
        M = _log(rng, 1, 8192)
        return dict(op=op, M=M, K=16 * _log(rng, 16, 640), N=_log(rng, 100, 11520), G=rng.randint(1, min(4, M)),
                    cuts=rng.randrange(1000))
    if op == "norm":
        M = _log(rng, 1, 16896)
        return dict(op=op, M=M, K=16 * _log(rng, 16, 640), G=rng.randint(1, min(6, M)), cuts=rng.randrange(1000))
    Hk = rng.choice([4, 6, 8, 15])
    H = Hk * rng.choice([1, 2, 4] if Hk <= 8 else [1, 2])
    D = rng.choice([64, 128])
    if op == "rope":
        axes = rng.choice({64: ["64", "16,24,24", "32,32"], 128: ["128", "32,48,48", "64,64", "16,56,56"]}[D])
        return dict(op=op, T=_log(rng, 1, 16896), H=H, Hk=Hk, D=D, axes=axes, norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5)
    T = _log(rng, 1, 12000)
    return dict(op=op, T=T, B=rng.randint(1, max(1, min(24, T // 4))), cuts=rng.randrange(1000), H=H, Hk=Hk, D=D,
                causal=rng.random() < 0.5)


def _lengths(total, parts, cuts):
    """`parts` lengths between about a quarter and twice the mean, of sum `total`."""
    r = random.Random(cuts)
    w = [r.uniform(0.25, 1.75) for _ in range(parts)]
    edges = [0]
    for i in range(parts):
        edges.append(int(round(total * sum(w[: i + 1]) / sum(w))))
    edges[-1] = total
    return [edges[i + 1] - edges[i] for i in range(parts)]


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, M, K):
    """Activations of a transformer block: unit normal with one channel in a hundred 20 times larger."""
    x = _normal(gen, M, K)
    x[:, torch.randperm(K, generator=gen, device="cuda")[: K // 100]] *= 20.0
    return x.to(torch.bfloat16)


def _int8_weight(gen, N, K):
    """A weight held in 8 bits: codes and one scale per output channel."""
    w = _normal(gen, N, K) * 0.02
    s = w.abs().amax(1) / 127.0
    return torch.round(w / s[:, None]).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op in ("linear", "norm_linear"):
        M, K, N = case["M"], case["K"], case["N"]
        s["w"], s["ws"] = _int8_weight(gen, N, K)
        s["bias"] = (_normal(gen, N) * 0.01).to(torch.bfloat16) if case.get("bias") else None
        s["smooth"] = None
    if op == "linear":
        s["x"] = _activations(gen, M, K)
        if case["smooth"]:
            s["smooth"] = s["x"].float().abs().amax(0).clamp_min(1e-6).rsqrt().to(torch.bfloat16)
    if op in ("norm", "norm_linear"):
        M, K, G = case["M"], case["K"], case["G"]
        s["h"] = _activations(gen, M, K)
        s["b"] = _normal(gen, M, K).to(torch.bfloat16)
        s["post"] = (1.0 + 0.1 * _normal(gen, K)).to(torch.bfloat16)
        s["pre"] = (1.0 + 0.1 * _normal(gen, K)).to(torch.bfloat16)
        s["gate"] = torch.tanh(_normal(gen, G, K)).to(torch.bfloat16)
        s["scale"] = (0.3 * _normal(gen, G, K)).to(torch.bfloat16)
        s["cu"] = _cu(_lengths(M, G, case["cuts"]))
    if op == "rope":
        T, H, Hk, D = case["T"], case["H"], case["Hk"], case["D"]
        qkv = _normal(gen, T, (H + 2 * Hk) * D).to(torch.bfloat16)
        s["q"] = qkv[:, : H * D].view(T, H, D)
        s["k"] = qkv[:, H * D: (H + Hk) * D].view(T, Hk, D)
        s["qw"] = (1.0 + 0.1 * _normal(gen, D)).to(torch.bfloat16) if case["norm"] else None
        s["kw"] = (1.0 + 0.1 * _normal(gen, D)).to(torch.bfloat16) if case["norm"] else None
        s["axes"] = tuple(int(a) for a in case["axes"].split(","))
        # text tokens first (time alone runs), then a grid of image or video tokens
        text = min(T, 512)
        side = max(1, math.isqrt(max(1, T - text)))
        i = torch.arange(T, device="cuda")
        j = (i - text).clamp_min(0)
        grid = torch.stack([torch.where(i < text, i, text + j // (4 * side)), j // side, j % side], 1)
        s["pos"] = grid[:, : len(s["axes"])].to(torch.int32).contiguous()
    if op == "attention":
        T, H, Hk, D = case["T"], case["H"], case["Hk"], case["D"]
        qkv = _normal(gen, T, (H + 2 * Hk) * D).to(torch.bfloat16)
        s["q"] = qkv[:, : H * D].view(T, H, D)
        s["k"] = qkv[:, H * D: (H + Hk) * D].view(T, Hk, D)
        s["v"] = qkv[:, (H + Hk) * D:].view(T, Hk, D)
        s["lens"] = _lengths(T, case["B"], case["cuts"])
        s["cu"] = _cu(s["lens"])
        s["longest"] = max(s["lens"])
    return s


# ---------------------------------------------------------------- plain forms

def _rows_group(cu, rows):
    return torch.searchsorted(cu[1:], torch.arange(rows, device=cu.device, dtype=torch.int32), right=True)


def _plain_quantize(v):
    amax = v.abs().amax(1, keepdim=True)
    inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    return torch.round(v * inv), amax / 127.0


def _plain_linear(codes, scales, w, ws, bias):
    y = (codes @ w.float().t()) * scales * ws
    if bias is not None:
        y = y + bias.float()
    return y.to(torch.bfloat16)


def _plain_norm(s):
    group = _rows_group(s["cu"], s["h"].shape[0])
    b = s["b"].float()
    b = b * torch.rsqrt((b * b).mean(1, keepdim=True) + EPS) * s["post"].float()
    h = s["h"].float() + 0.5 * s["gate"].float()[group] * b
    x = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["pre"].float() * (1.0 + s["scale"].float()[group])
    return h.to(torch.bfloat16), x.to(torch.bfloat16)


def _plain_rope_one(z, w, cos, sin, interleaved):
    z = z.float()
    if w is not None:
        z = z * torch.rsqrt((z * z).mean(2, keepdim=True) + EPS) * w.float()
    if interleaved:
        a, b = z[..., 0::2], z[..., 1::2]
    else:
        a, b = z.chunk(2, 2)
    a, b = a * cos - b * sin, b * cos + a * sin
    out = torch.stack([a, b], 3).flatten(2) if interleaved else torch.cat([a, b], 2)
    return out.to(torch.bfloat16)


def _plain_rope(s):
    dev = s["q"].device
    sizes = torch.tensor([a // 2 for a in s["axes"]], device=dev)
    axis = torch.repeat_interleave(torch.arange(len(s["axes"]), device=dev), sizes,
                                   output_size=s["q"].shape[2] // 2)
    first = (torch.cumsum(sizes, 0) - sizes)[axis]
    freq = 10000.0 ** (-(torch.arange(axis.numel(), device=dev, dtype=torch.float64) - first) / sizes[axis])
    angle = s["pos"].double()[:, axis] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    inter = s["case"]["interleaved"]
    return _plain_rope_one(s["q"], s["qw"], cos, sin, inter), _plain_rope_one(s["k"], s["kw"], cos, sin, inter)


def _plain_attention(s):
    """The sequences padded to the longest, the padding masked."""
    q, k, v, cu, L = s["q"], s["k"], s["v"], s["cu"].long(), s["longest"]
    T, H, D = q.shape
    B, Hk = cu.numel() - 1, k.shape[1]
    at = torch.arange(L, device=q.device)
    there = at < (cu[1:] - cu[:-1])[:, None]                       # [B, L]
    row = (cu[:-1, None] + at).clamp_max(T - 1)                    # [B, L]
    qp = q[row].float().view(B, L, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, (H // Hk) * L, D)
    kp = k[row].float().permute(0, 2, 3, 1).contiguous()           # [B, Hk, D, L]
    vp = v[row].float().permute(0, 2, 1, 3).contiguous()           # [B, Hk, L, D]
    p = torch.matmul(qp, kp).mul_(D ** -0.5).view(B, Hk, H // Hk, L, L)
    hide = ~there[:, None, None, None, :]
    if s["case"]["causal"]:
        hide = hide | (at[None, :] > at[:, None])
    p.masked_fill_(hide, -math.inf)
    p.sub_(p.amax(4, keepdim=True)).exp_()
    p.div_(p.sum(4, keepdim=True))
    o = torch.matmul(p.view(B, Hk, (H // Hk) * L, L), vp)
    o = o.view(B, Hk, H // Hk, L, D).permute(0, 3, 1, 2, 4).reshape(B, L, H, D)
    return o[there].to(torch.bfloat16)


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "linear":
        v = s["x"].float()
        if s["smooth"] is not None:
            v = v * s["smooth"].float()
        return _plain_linear(*_plain_quantize(v), s["w"], s["ws"], s["bias"])
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_linear":
        h, x = _plain_norm(s)
        return h, _plain_linear(*_plain_quantize(x.float()), s["w"], s["ws"], s["bias"])
    if op == "rope":
        return _plain_rope(s)
    return _plain_attention(s)


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    from bit_w4a4_quantized_quantize_amd import ops
    op = s["op"]
    if op == "linear":
        return ops.linear_int8(s["x"], s["w"], s["ws"], bias=s["bias"], smooth=s["smooth"])
    if op == "norm":
        return ops.norm_gated(s["h"], s["b"], post_weight=s["post"], gate=s["gate"], residual_scale=0.5,
                              pre_weight=s["pre"], scale=s["scale"], cu_seqlens=s["cu"], eps=EPS)
    if op == "norm_linear":
        h, codes, scales = ops.norm_gated_int8(s["h"], s["b"], post_weight=s["post"], gate=s["gate"],
                                               residual_scale=0.5, pre_weight=s["pre"], scale=s["scale"],
                                               cu_seqlens=s["cu"], eps=EPS)
        return h, ops.gemm_int8(codes, scales, s["w"], s["ws"], bias=s["bias"])
    if op == "rope":
        return ops.rope_axes(s["q"], s["k"], s["pos"], s["axes"], theta=10000.0,
                             interleaved=s["case"]["interleaved"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
    return ops.attention_packed(s["q"], s["k"], s["v"], s["cu"], causal=s["case"]["causal"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N, "flops": 2 * M * N * K}
    if op == "norm":
        M, K = case["M"], case["K"]
        return {"bytes": 8 * M * K + 4 * K * (1 + case["G"]), "flops": 14 * M * K}
    if op == "norm_linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 6 * M * K + 4 * K * (1 + case["G"]) + N * K + 4 * N + 2 * M * N, "flops": 2 * M * N * K}
    if op == "rope":
        T, n = case["T"], (case["H"] + case["Hk"]) * case["D"]
        return {"bytes": 4 * T * n + 4 * T * len(case["axes"].split(",")), "flops": 6 * T * n}
    T, H, Hk, D = case["T"], case["H"], case["Hk"], case["D"]
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _lengths(T, case["B"], case["cuts"]))
    return {"bytes": 4 * T * D * (H + Hk), "flops": 4 * H * D * pairs}


# ---------------------------------------------------------------- in 64 bits

def _exact_int8(v, s):
    """Rounding to 8 bits is part of the operator; the rest is exact."""
    top = v.abs().max(dim=1).values
    unit = top / 127.0
    codes = torch.where(top[:, None] > 0, torch.round(v * 127.0 / top[:, None]), 0.0)
    y = torch.einsum("mk,nk->mn", codes, s["w"].double()) * torch.outer(unit, s["ws"].double())
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_norm(s):
    hs, xs = [], []
    edges = s["cu"].tolist()
    for g in range(len(edges) - 1):
        rows = slice(edges[g], edges[g + 1])
        b = s["b"][rows].double()
        b = b / torch.sqrt(b.square().sum(1, keepdim=True) / b.shape[1] + EPS)
        h = s["h"][rows].double() + 0.5 * (s["gate"][g].double() * s["post"].double()) * b
        hs.append(h)
        xs.append(h / torch.sqrt(h.square().sum(1, keepdim=True) / h.shape[1] + EPS)
                  * (s["pre"].double() * (1.0 + s["scale"][g].double())))
    return torch.cat(hs), torch.cat(xs)


def _exact_rope(z, w, s):
    z = z.double()
    if w is not None:
        z = z / torch.sqrt(z.square().mean(2, keepdim=True) + EPS) * w.double()
    out = torch.empty_like(z)
    p = 0
    for a, d in enumerate(s["axes"]):
        for i in range(d // 2):
            angle = s["pos"][:, a].double() * 10000.0 ** (-2.0 * i / d)
            turn = torch.polar(torch.ones_like(angle), angle)[:, None]
            lo, hi = (2 * p, 2 * p + 1) if s["case"]["interleaved"] else (p, p + z.shape[2] // 2)
            r = torch.complex(z[:, :, lo], z[:, :, hi]) * turn
            out[:, :, lo], out[:, :, hi] = r.real, r.imag
            p += 1
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        v = s["x"].double()
        return _exact_int8(v if s["smooth"] is None else v * s["smooth"].double(), s)
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_linear":
        h, x = _exact_norm(s)
        return h, _exact_int8(x.to(torch.bfloat16).double(), s)
    if op == "rope":
        return _exact_rope(s["q"], s["qw"], s), _exact_rope(s["k"], s["kw"], s)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for n in s["lens"]:
        rows = slice(start, start + n)
        start += n
        for h in range(case["H"]):
            kv = h // (case["H"] // case["Hk"])
            a = s["q"][rows, h].double() @ s["k"][rows, kv].double().T / math.sqrt(case["D"])
            if case["causal"]:
                a += torch.triu(torch.full_like(a, -math.inf), 1)
            out[rows, h] = torch.softmax(a, 1) @ s["v"][rows, kv].double()
    return out
