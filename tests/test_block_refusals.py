"""Refusals of the operators between the linears, on any host: the C ABI's checks with fake device
addresses (never dereferenced; every case fails validation or is an empty problem), and the Python
binding's checks with CPU tensors."""

import ctypes

import pytest
import torch

from bit_w4a4_quantized_quantize_amd import _lib, ops

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-pointer validation cases run on CPU-only hosts")
bf, f32, i8, i32 = torch.bfloat16, torch.float32, torch.int8, torch.int32


def fake(i):
    return 0x7F0000000000 + i * 0x100000000


def err():
    return _lib.lib().svdq_last_error().decode()


def quant(**kw):
    a = dict(x=fake(1), smooth=fake(2), M=64, K=256, codes=fake(3), ascales=fake(4))
    a.update(kw)
    return _lib.lib().svdq_quantize_int8(*a.values(), None)


@no_gpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 2), (dict(K=24), 2), (dict(K=0), 2), (dict(K=1 << 25), 3), (dict(M=(1 << 24) + 1), 3),
    (dict(x=None), 1), (dict(codes=None), 1), (dict(ascales=None), 1), (dict(smooth=fake(2) + 8), 4),
    (dict(codes=fake(3) + 4), 4), (dict(codes=fake(1)), 6), (dict(ascales=fake(3) + 64), 6), (dict(codes=fake(2) + 256), 6),
])
def test_quantize_int8(kw, code):
    assert quant(**kw) == code and err()


def gemm(fn="svdq_gemm_int8", **kw):
    a = dict(codes=fake(1), ascales=fake(2), weight=fake(3), wscales=fake(4), bias=None, M=64, N=128, K=256, y=fake(5),
             ws=fake(6), ws_bytes=1 << 30)
    a.update(kw)
    return getattr(_lib.lib(), fn)(*a.values(), None)


@no_gpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 2), (dict(N=-1), 2), (dict(K=40), 2), (dict(K=131072 + 16), 3), (dict(N=(1 << 24) + 1), 3),
    (dict(M=1 << 24, N=1 << 15), 3), (dict(weight=None), 1), (dict(wscales=None), 1), (dict(y=None), 1), (dict(codes=None), 1),
    (dict(bias=fake(7) + 2), 4), (dict(y=fake(5) + 2), 4),
    (dict(y=fake(3) + 128), 6), (dict(y=fake(4)), 6), (dict(y=fake(1)), 6), (dict(bias=fake(5)), 6),
])
def test_gemm_and_linear_int8(kw, code):
    assert gemm(**kw) == code and err()
    # the layer takes x and smooth where the product takes codes and scales
    assert gemm("svdq_linear_int8", **kw) == code and err()


@no_gpu_only
def test_int8_workspace_and_empty():
    L = _lib.lib()
    need = L.svdq_linear_int8_workspace_bytes(64, 128, 256)
    assert need >= 64 * 256 + 64 * 4
    assert gemm("svdq_linear_int8", ws_bytes=need - 1) == 5
    assert gemm("svdq_linear_int8", ws=None) == 1
    assert gemm("svdq_linear_int8", ws=fake(6) + 8) == 4
    assert gemm("svdq_linear_int8", ws=fake(5) - 1024) == 6
    assert gemm("svdq_linear_int8", M=0, codes=None) == 0
    assert gemm(N=0) == 0 and gemm(M=0) == 0 and quant(M=0, x=None) == 0
    assert L.svdq_linear_int8_workspace_bytes(0, 128, 256) == 0
    assert gemm("svdq_linear_int8", ascales=fake(2) + 8) == 4       # smooth


def norm(fn="svdq_norm_gated", **kw):
    a = dict(h=fake(1), block=fake(2), post=fake(3), gate=fake(4), rs=1.0, pre=fake(5), scale=fake(6), cu=fake(7), G=3,
             M=64, K=256, eps=1e-6, h_out=fake(8), a=fake(9), b=None, c=None)
    if fn.endswith("int8"):
        a.update(a=fake(10), b=fake(11), c=fake(12))      # smooth, codes, ascales
    a.update(kw)
    v = list(a.values())
    return getattr(_lib.lib(), fn)(*(v if fn.endswith("int8") else v[:-2]), None)


@no_gpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 2), (dict(K=8), 2), (dict(K=32784), 3), (dict(G=0), 2), (dict(G=(1 << 24) + 1), 3), (dict(cu=None), 8),
    (dict(eps=-1e-6), 8), (dict(eps=float("nan")), 8), (dict(eps=float("inf")), 8), (dict(rs=float("inf")), 8),
    (dict(rs=float("nan")), 8),
    (dict(block=None), 8), (dict(block=None, h_out=None), 8), (dict(h_out=None), 1), (dict(h=None), 1),
    (dict(h=fake(1) + 8), 4), (dict(gate=fake(4) + 2), 4), (dict(cu=fake(7) + 4), 4),
    (dict(h_out=fake(2)), 6), (dict(h_out=fake(1) + 512), 6), (dict(h_out=fake(4) + 1024), 6), (dict(h_out=fake(7)), 6),
])
def test_norm_gated(kw, code):
    assert norm(**kw) == code and err()
    assert norm("svdq_norm_gated_int8", **kw) == code and err()


@no_gpu_only
def test_norm_gated_forms():
    assert norm(block=None, h_out=None, post=None, gate=None, a=None) == 8             # nothing to do
    assert norm(a=None) == 8                                                         # pre_weight without x_out
    assert norm(a=fake(1)) == 6 and norm(a=fake(8) + 64) == 6                        # x_out over h, over h_out
    assert norm("svdq_norm_gated_int8", b=None) == 1 and norm("svdq_norm_gated_int8", c=None) == 1
    assert norm("svdq_norm_gated_int8", a=fake(10) + 8) == 4
    assert norm("svdq_norm_gated_int8", b=fake(8)) == 6 and norm("svdq_norm_gated_int8", c=fake(11) + 16) == 6
    assert norm(M=0, h=None, block=None, post=None, gate=None, h_out=None) == 0


def rope(**kw):
    a = dict(q=fake(1), qst=1536, qsh=128, H=4, k=fake(1) + 1024, kst=1536, ksh=128, Hk=4, qw=fake(2), kw=fake(3),
             eps=1e-6, pos=fake(4), dims=(32, 48, 48), axes=3, theta=1e4, inter=1, T=16, D=128, qo=fake(5), qost=512,
             qosh=128, ko=fake(6), kost=512, kosh=128)
    a.update(kw)
    if a["dims"] is not None:
        a["dims"] = (ctypes.c_int32 * len(a["dims"]))(*a["dims"])
    return _lib.lib().svdq_rope_axes(*a.values(), None)


@no_gpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 2), (dict(T=1 << 24), 3), (dict(D=96), 3), (dict(H=-1), 2), (dict(H=65536), 3),
    (dict(axes=0), 2), (dict(axes=5, dims=(32, 32, 32, 16, 16)), 2), (dict(dims=None), 1), (dict(dims=(32, 48, 46)), 2),
    (dict(dims=(31, 49, 48)), 2), (dict(dims=(128, 0, 0)), 2), (dict(theta=0.5), 8), (dict(theta=float("nan")), 8),
    (dict(eps=-1.0), 8), (dict(pos=None), 1), (dict(pos=fake(4) + 4), 4), (dict(qw=fake(2) + 2), 4),
    (dict(q=None), 1), (dict(H=0), 8), (dict(qo=None), 1), (dict(q=fake(1) + 8), 4), (dict(qst=1540), 4),
    (dict(qsh=64), 2), (dict(qst=64), 2), (dict(qst=-128), 2), (dict(qst=1 << 24), 3),
    (dict(qost=256), 2),                                                            # heads of tokens overlap
    (dict(qo=fake(1), qost=1536), 0), (dict(qo=fake(1) + 1024, qost=1536), 6),      # in place; q_out over k
    (dict(qo=fake(1), qost=1024), 6), (dict(qo=fake(1) + 16, qost=1536), 6),
    (dict(qo=fake(6)), 6), (dict(qo=fake(4)), 6), (dict(qo=fake(3)), 6),
    (dict(H=0, Hk=0), 2),
])
def test_rope_axes(kw, code):
    if code == 0:      # the in-place form passes the overlap checks: stop it at the next one
        kw = kw | dict(ko=fake(4))
        assert rope(**kw) == 6 and "positions" in err()
        return
    assert rope(**kw) == code and err()


@no_gpu_only
def test_rope_axes_fused_views_in_place():
    """q and k of one fused buffer, both in place, interleave without sharing an element."""
    both = dict(qo=fake(1), qost=1536, ko=fake(1) + 1024, kost=1536)
    assert rope(**both, T=0) == 0
    assert rope(**both, qw=fake(1) + 64) == 6 and "q_weight" in err()
    assert rope(**both | dict(k=fake(1) + 768, ko=fake(1) + 768)) == 6              # heads shared
    assert rope(**both | dict(k=fake(1) + 2304, ko=fake(1) + 2304)) == 6             # wraps into the next token's q


def attn(**kw):
    a = dict(q=fake(1), qst=512, qsh=128, k=fake(2), kst=256, ksh=128, v=fake(3), vst=256, vsh=128, cu=fake(4), B=3,
             T=64, H=4, Hk=2, D=128, causal=0, scale=0.1, o=fake(5), ost=512, osh=128)
    a.update(kw)
    return _lib.lib().svdq_attention_packed(*a.values(), None)


@no_gpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 2), (dict(T=1 << 24), 3), (dict(D=80), 3), (dict(H=3), 2), (dict(H=0), 2), (dict(Hk=0), 2),
    (dict(B=-1), 2), (dict(B=65536), 3), (dict(H=65538), 3), (dict(cu=None), 8),
    (dict(scale=0.0), 8), (dict(scale=-1.0), 8), (dict(scale=float("nan")), 8), (dict(scale=float("inf")), 8),
    (dict(scale=2e6), 8), (dict(T=(1 << 24) - 1, H=256, qst=1 << 15, ost=1 << 15), 3),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1),
    (dict(k=fake(2) + 8), 4), (dict(vst=260), 4), (dict(cu=fake(4) + 4), 4), (dict(kst=1 << 24), 3), (dict(ksh=64), 2),
    (dict(kst=0), 2), (dict(ost=256), 2),
    (dict(o=fake(1)), 6), (dict(o=fake(2) + 64), 6), (dict(o=fake(3)), 6), (dict(o=fake(4) - 128), 6),
])
def test_attention_packed(kw, code):
    assert attn(**kw) == code and err()


@no_gpu_only
def test_attention_empty():
    assert attn(T=0, q=None) == 0 and attn(B=0) == 0


# ---- the binding, with CPU tensors

def z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def refused(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_int8():
    x, w, ws = z(4, 32), z(8, 32, dtype=i8), z(8, dtype=f32)
    refused("GPU tensor", ops.linear_int8, x, w, ws)
    refused("must be torch.bfloat16", ops.linear_int8, x.float(), w, ws)
    refused("must be torch.int8", ops.linear_int8, x, w.int(), ws)
    refused("weight has K", ops.linear_int8, x, z(8, 48, dtype=i8), ws)
    refused("wscales must have shape", ops.linear_int8, x, w, z(9, dtype=f32))
    refused("multiple of 16", ops.linear_int8, z(4, 24), z(8, 24, dtype=i8), ws)
    refused("bias must have shape", ops.linear_int8, x, w, ws, bias=z(7))
    refused("smooth must have shape", ops.linear_int8, x, w, ws, smooth=z(16))
    refused("y must have shape", ops.linear_int8, x, w, ws, y=z(4, 9))
    refused("workspace has", ops.linear_int8, z(64, 32), w, ws, workspace=z(8, dtype=torch.uint8))
    refused("contiguous", ops.linear_int8, z(32, 4).t(), w, ws)
    refused("ascales must have shape", ops.gemm_int8, z(4, 32, dtype=i8), z(3, dtype=f32), w, ws)
    refused("codes must be", ops.gemm_int8, x, z(4, dtype=f32), w, ws)
    refused("codes must have shape", ops.quantize_int8, x, codes=z(4, 31, dtype=i8))
    refused("scales must be", ops.quantize_int8, x, scales=z(4))
    refused("GPU tensor", ops.quantize_int8, x)


def test_binding_norm():
    h = z(4, 32)
    refused("GPU tensor", ops.norm_gated, h, h.clone())
    refused("block must have shape", ops.norm_gated, h, z(4, 48))
    refused("gate must have shape", ops.norm_gated, h, h.clone(), gate=z(2, 32))
    refused("scale must have shape", ops.norm_gated, h, scale=z(32))
    refused("cu_seqlens must be", ops.norm_gated, h, cu_seqlens=z(2, dtype=torch.int64))
    refused("cu_seqlens has", ops.norm_gated, h, cu_seqlens=z(1, dtype=i32))
    refused("post_weight must have shape", ops.norm_gated, h, h.clone(), post_weight=z(31))
    refused("x_out must have shape", ops.norm_gated, h, x_out=z(4, 31))
    refused("pre=False", ops.norm_gated, h, h.clone(), pre=False, x_out=h.clone())
    refused("smooth must have shape", ops.norm_gated_int8, h, smooth=z(31))
    refused("scales must have shape", ops.norm_gated_int8, h, scales=z(3, dtype=f32))


def test_binding_rope():
    q, k, pos = z(4, 2, 64), z(4, 1, 64), z(4, 3, dtype=i32)
    refused("GPU tensor", ops.rope_axes, q, k, pos, (16, 24, 24))
    refused("q or k", ops.rope_axes, None, None, pos, (16, 24, 24))
    refused("positions must have shape", ops.rope_axes, q, k, pos, (32, 32))
    refused("positions must be", ops.rope_axes, q, k, pos.long(), (16, 24, 24))
    refused("k must have shape", ops.rope_axes, q, z(5, 1, 64), pos, (16, 24, 24))
    refused("3 dims", ops.rope_axes, z(4, 64), None, pos, (16, 24, 24))
    refused("contiguous", ops.rope_axes, z(4, 2, 128)[:, :, ::2], None, pos, (16, 24, 24))
    refused("q_weight must have shape", ops.rope_axes, q, k, pos, (16, 24, 24), q_weight=z(32))
    refused("q_out must have shape", ops.rope_axes, q, k, pos, (16, 24, 24), q_out=z(4, 3, 64))
    refused("need k", ops.rope_axes, q, None, pos, (16, 24, 24), k_out=k)


def test_binding_attention():
    q, k = z(4, 2, 64), z(4, 1, 64)
    refused("GPU tensor", ops.attention_packed, q, k, k.clone())
    refused("k must have shape", ops.attention_packed, q, z(5, 1, 64), k)
    refused("v must have shape", ops.attention_packed, q, k, z(4, 2, 64))
    refused("cu_seqlens must be", ops.attention_packed, q, k, k, z(2, dtype=torch.int64))
    refused("cu_seqlens has", ops.attention_packed, q, k, k, z(0, dtype=i32))
    refused("out must have shape", ops.attention_packed, q, k, k, out=z(4, 2, 128))
    refused("must be torch.bfloat16", ops.attention_packed, q.half(), k, k)
    refused("contiguous", ops.attention_packed, z(4, 2, 128)[:, :, ::2], k, k)
