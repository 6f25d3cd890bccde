"""The largest attention calls: what the checks let through fits a grid of fewer than 2^32 work items, and what does
not is refused on the host (fake device addresses; a call that is let through ends at a later check)."""

import pytest
import torch

from bit_w4a4_quantized_quantize_amd import _lib

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-pointer validation cases run on CPU-only hosts")


def fake(i):
    return 0x7F0000000000 + i * 0x10000000000


def attn(T, B, H, Hk, D):
    """With o on its own queries: refused as an overlap once the sizes have passed."""
    s = (H * D, D)
    return _lib.lib().svdq_attention_packed(fake(1), *s, fake(2), Hk * D, D, fake(3), Hk * D, D, fake(4), B, T, H, Hk, D,
                                            0, 0.1, fake(1), *s, None)


def work_items(T, B, H, Hk, D):
    """Grid times workgroup as the launch makes them, for either number of waves."""
    most = 0
    for lg_waves in (2, 3):
        lg = 0
        while (2 << lg) <= 1 << lg_waves and (H // Hk) % (2 << lg) == 0:
            lg += 1
        total = (T // (32 << (lg_waves - lg)) + B) * (H >> lg)
        most = max(most, (total + 7) // 8 * 8 * (64 << lg_waves))
    return most


@no_gpu_only
@pytest.mark.parametrize("T,B,H", [(31417 * 256, 1, 267), (31418 * 256 - 1, 1, 267), (2 ** 21 - 257, 1, 1024), (2 ** 21 - 259, 1, 1024),
                                   (2 ** 21 - 255, 1, 1024), (32768, 65407, 128), (100, 8200, 1023), (2 ** 24 - 1, 1, 127),
                                   (2 ** 24 - 1, 1, 128), (7, 65535, 127), (7, 65535, 128)])
def test_grid_of_the_largest_calls(T, B, H):
    code = attn(T, B, H, H, 64)
    assert code in (3, 6), (code, _lib.lib().svdq_last_error().decode())
    if code == 6:
        assert work_items(T, B, H, H, 64) < 2 ** 32
    else:
        assert 2 * T * H + 512 * B * H >= 2 ** 32 - 4096
