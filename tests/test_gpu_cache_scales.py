"""GPU: appending to pages whose scale bytes were not made by this library: any byte but 255 is a power of two, from 2^-127
to 2^127, and tokens added behind it are coded by it, bit for bit as the oracle does."""

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.test_gpu_cache import check_held, dirty, f64, i32

pytestmark = pytest.mark.gpu

BYTES = [0, 1, 26, 27, 127, 246, 247, 248, 252, 253, 254]


@pytest.mark.parametrize("page,D", [(16, 64), (32, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("byte", BYTES)
def test_append_behind_a_scale_from_elsewhere(gpu_lib, byte, page, D):
    """A page of 5 tokens with this scale gets 9 more: quiet ones, which leave the scale, and ones as loud as bf16 has them."""
    print(f"[cache] append behind scale {byte} page={page} D={D}", flush=True)
    Hk, held, new = 2, 5, 9
    g = torch.Generator().manual_seed(byte + page)
    for loud in (0.0, 2.0 ** (byte - 127 + 3), 2.0 ** 125):
        cache, oracle = dirty(gpu_lib, 2, Hk, page, D), S.Cache(2, Hk, page, D)
        for name in "kv":
            z = (torch.randn(Hk, held, D, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            oracle.codes[name][1, :, :held] = z.double().numpy()
            oracle.exps[name][1] = byte - 127
            z = z.view(torch.uint8).cuda()
            if name == "k":
                cache.k_codes.view(torch.uint8)[1, :, :held] = z
            else:
                cache.v_codes.view(torch.uint8)[1, :, :, :held] = z.transpose(1, 2)
        cache.k_scales[1] = byte
        cache.v_scales[1] = byte
        z = torch.rand(new, 2 * Hk, D, generator=g).clamp(min=0.25) * torch.randn(new, 2 * Hk, D, generator=g).sign()
        z = (z.double() * min(loud, 2.0 ** 127)).float().bfloat16().cuda()
        k, v = z[:, :Hk], z[:, Hk:]
        gpu_lib.cache_append_fp8(k, v, cache, i32([[1]]), i32([held]), i32([0, new]))
        oracle.append({"k": f64(k), "v": f64(v)}, [[1]], [held], [0, new])
        if byte == 254 and loud:
            assert np.abs(oracle.codes["k"][1, :, held:held + new]).max() > 0
        check_held(gpu_lib, cache, oracle, [[1]], [held + new])
        # and a token by itself
        one = z[:1]
        gpu_lib.cache_append_fp8(one[:, :Hk], one[:, Hk:], cache, i32([[1]]), i32([held + new]))
        oracle.append({"k": f64(one[:, :Hk]), "v": f64(one[:, Hk:])}, [[1]], [held + new], [0, 1])
        check_held(gpu_lib, cache, oracle, [[1]], [held + new + 1])


def to_bf16(v):
    """Nearest bf16 in float64, subnormals and the overflow to infinity included."""
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -126))
    step = np.ldexp(1.0, e - 8)
    z = np.rint(v / step) * step
    return np.where(np.abs(z) >= 2.0 ** 128, np.copysign(np.inf, z), z)


def test_every_scale_byte(gpu_lib):
    """A head for each byte, every code: what is read back, and what a row answers that sees one key."""
    Hk, page, D = 256, 16, 128
    codes = torch.arange(256, dtype=torch.uint8)
    codes[0x7F] = codes[0xFF] = 0                                    # the NaN codes
    k = torch.zeros(1, Hk, page, D, dtype=torch.uint8)
    k[:, :, :2] = codes.view(1, 1, 2, D)
    scales = torch.arange(256, dtype=torch.uint8)[None].cuda()
    held = gpu_lib.Fp8Cache(k.view(torch.float8_e4m3fn).cuda(), k.transpose(2, 3).contiguous().view(torch.float8_e4m3fn).cuda(),
                            scales, scales.clone())
    value = codes.view(torch.float8_e4m3fn).double().view(2, 1, D) * 2.0 ** (torch.arange(256).double() - 127).view(1, 256, 1)
    want = to_bf16(value.numpy())[:, :255]
    for got in gpu_lib.cache_read_fp8(held, i32([[0]]), i32([0]), i32([0, 2]), 2):
        assert np.array_equal(f64(got)[:, :255], want) and np.isnan(f64(got)[:, 255]).all()
    held.k_codes.view(torch.uint8).zero_()
    held.k_scales.fill_(127)
    for T, H in ((1, 256), (1, 512), (200, 256)):
        q = torch.ones(T, H, D, device="cuda").bfloat16()
        o = f64(gpu_lib.attention_cache_fp8(q, held, i32([[0]]), i32([1]), cu_seqlens=i32([0, T]), causal=False))
        o = o.reshape(T, 256, H // 256, D)
        assert np.array_equal(o[:, :255], np.broadcast_to(want[0][None, :, None], o[:, :255].shape))
        assert np.isnan(o[:, 255]).all()
