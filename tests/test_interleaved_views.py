"""Head views of one buffer that interleave without sharing an element: the overlap checks against a count of
elements (fake device addresses, never dereferenced), and on the GPU against calls on tensors of their own."""

import ctypes
import random

import pytest
import torch

from bit_w4a4_quantized_quantize_amd import _lib

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-pointer validation cases run on CPU-only hosts")
D = 64


def fake(i):
    return 0x7F0000000000 + i * 0x100000000


def elements(off, T, H, st, sh):
    return {off + t * st + h * sh + 8 * e for t in range(T) for h in range(H) for e in range(D // 8)}


def k_against_q_out(T, Hk, k, H, qo):
    """Whether the checks call k (off, st, sh) and q_out overlapping. q_out lies on the positions too, which is looked at
    afterwards, so no call gets past the checks."""
    base = fake(1)
    dims = (ctypes.c_int32 * 1)(D)
    code = _lib.lib().svdq_rope_axes(fake(2), H * D, D, H, base + 2 * k[0], k[1], k[2], Hk, None, None, 1e-6,
                                     base + 2 * qo[0], dims, 1, 1e4, 1, T, D, base + 2 * qo[0], qo[1], qo[2],
                                     fake(3), Hk * D, D, None)
    msg = _lib.lib().svdq_last_error().decode()
    assert code == 6 and "output q_out overlaps input" in msg, (code, msg)
    return msg.endswith("input k")


@no_gpu_only
@pytest.mark.parametrize("same", [True, False])
def test_overlap_checks_against_a_count(same):
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        T, H, Hk = rng.randint(1, 5), rng.randint(1, 4), rng.randint(1, 4)
        st, sh = (8 * rng.randint(8, 64) for _ in range(2))
        if rng.random() < 0.5:      # layouts that are made: heads of n tensors beside each other, tokens or heads outside
            n = rng.randint(1, 3)
            st, sh = rng.choice([(n * 4 * D, n * D), (n * D, n * 5 * D), (D, n * 5 * D), (n * 4 * D + 8, n * D)])
        k = (1 << 20, st, sh)
        qo = (k[0] + 8 * rng.randint(-200, 200), st, sh)
        if not same:
            qo = (qo[0], 8 * rng.randint(8, 64), 8 * rng.randint(8, 64))
        if T > 1 and H > 1 and qo[1] < (H - 1) * qo[2] + D and qo[2] < (T - 1) * qo[1] + D:
            continue                # refused for its own heads
        shared = bool(elements(k[0], T, Hk, *k[1:]) & elements(qo[0], T, H, *qo[1:]))
        told = k_against_q_out(T, Hk, k, H, qo)
        if same:
            assert told == shared, (T, H, Hk, k, qo)
        assert told or not shared, (T, H, Hk, k, qo)
        seen[shared] += 1
    assert min(seen.values()) > 200


@no_gpu_only
def test_many_heads_interleaved():
    """As many heads as there may be."""
    T, H = 64, 65535
    assert not k_against_q_out(T, H, (0, 3 * H * D, 3 * D), H, (D, 3 * H * D, 3 * D))
    assert k_against_q_out(T, H, (0, 3 * H * D, 3 * D), H, (3 * D * (H - 1), 3 * H * D, 3 * D))


LAYOUTS = {
    "T H 3 D": lambda b, T, H: [b.view(T, H, 3, D)[:, :, i] for i in range(3)],
    "H T 3 D": lambda b, T, H: [b.view(H, T, 3, D)[:, :, i].transpose(0, 1) for i in range(3)],
    "H 3 T D": lambda b, T, H: [b.view(H, 3, T, D)[:, i].transpose(0, 1) for i in range(3)],
    "T 3 H D": lambda b, T, H: [b.view(T, 3, H, D)[:, i] for i in range(3)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H", [(77, 4), (1, 4), (40, 1)])
def test_rotary_and_attention_in_one_buffer(gpu_lib, layout, T, H):
    """q and k turned in place, then attention from them, and into q's place from a copy of it: as on tensors of their own."""
    print(f"[views] {layout} T={T} H={H}", flush=True)
    x = torch.randn(T * H * 3 * D, generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    q, k, v = LAYOUTS[layout](x, T, H)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
    apart = [t.contiguous() for t in (q, k, v)]
    q1, k1 = gpu_lib.rope_axes(apart[0], apart[1], pos, (D,))
    gpu_lib.rope_axes(q, k, pos, (D,), q_out=q, k_out=k)
    assert torch.equal(q, q1) and torch.equal(k, k1) and torch.equal(v, apart[2])
    want = gpu_lib.attention_packed(q1, k1, apart[2])
    assert torch.equal(gpu_lib.attention_packed(q, k, v), want)
    gpu_lib.attention_packed(q1, k, v, out=q)
    assert torch.equal(q, want) and torch.equal(k, k1) and torch.equal(v, apart[2])


@pytest.mark.gpu
def test_heads_of_no_elements_are_refused(gpu_lib):
    z = torch.zeros(4, 2, 0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(_lib.SvdqError, match="head size"):
        gpu_lib.attention_packed(z, z, z)
    with pytest.raises(_lib.SvdqError, match="head size"):
        gpu_lib.rope_axes(z, None, torch.zeros(4, 1, dtype=torch.int32, device="cuda"), (2,))
