"""GPU: rotary positions on part of a head with scaled frequencies, against the oracle (angles in long double).

Error: the angle in turns is a product in fp64 (2^-51 of it, the frequency's rounding included), reduced and
rounded to fp32 (2^-26 turns = 9.4e-8 rad), cosine and sine are within 2 units (2.4e-7), the amplitude rounds once
(6e-8), the rotation three times (1.8e-7): together below (7e-7 + 2^-51 |angle|) amplitude (|u| + |w|) for a pair;
bf16 rounds once (2^-8). The rest of a head is copied bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import serving as S

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def check(got, z, pos, R, **kw):
    ref, mag, far = S.rope(f64(z), pos.cpu().numpy(), R, **kw)
    tol = 2.0 ** -8 * np.abs(ref) + 1.01 * (7e-7 + 2.0 ** -51 * far) * mag + np.where(mag > 0, 2.0 ** -133, 0.0)
    err = np.abs(f64(got) - ref)
    tol[:, :, R:] = 0.0
    assert (err <= tol).all(), float((err - tol).max())


def make(T, H, Hk, D, far, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (H + 2 * Hk) * D, generator=g).bfloat16().cuda()
    pos = torch.randint(-far, far + 1, (T,), generator=g, dtype=torch.int64).to(torch.int32).cuda()
    return qkv[:, : H * D].view(T, H, D), qkv[:, H * D: (H + Hk) * D].view(T, Hk, D), pos


SCALINGS = [dict(), dict(factor=4.0), dict(factor=8.0, original=8192), dict(factor=31.5, original=4096, low=1.0, high=4.0, amplitude=1.25)]


def call(lib, q, k, pos, R, inter, kw, **more):
    return lib.rope_scaled(q, k, pos, rotary_dim=R, interleaved=inter, factor=kw.get("factor", 1.0),
                           original_length=kw.get("original", 0), low_rotations=kw.get("low", 1.0),
                           high_rotations=kw.get("high", 32.0), amplitude=kw.get("amplitude", 1.0), **more)


@pytest.mark.parametrize("T,H,Hk,D,R", [(1, 1, 1, 8, 8), (77, 30, 30, 128, 128), (5, 3, 1, 64, 16), (300, 7, 2, 80, 24),
                                        (33, 32, 8, 128, 64), (64, 5, 5, 96, 96), (9, 40, 3, 64, 8), (3, 100, 7, 256, 256),
                                        (1025, 4, 4, 256, 40), (2000, 1, 1, 16, 8), (11, 1, 1, 64, 64)])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()) or "plain")
def test_against_oracle(gpu_lib, T, H, Hk, D, R, inter, kw):
    print(f"[rope_scaled] {T} {H} {Hk} {D} {R} {inter} {kw}", flush=True)
    q, k, pos = make(T, H, Hk, D, 200000, T + D)
    qo, ko = call(gpu_lib, q, k, pos, R, inter, kw)
    check(qo, q, pos, R, interleaved=inter, **kw)
    check(ko, k, pos, R, interleaved=inter, **kw)


def test_positions_to_the_ends_of_int32(gpu_lib):
    q, k, _ = make(6, 3, 2, 128, 1, 1)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, -1, 2 ** 30 + 12345, 1], dtype=torch.int32, device="cuda")
    for kw in SCALINGS:
        qo, ko = call(gpu_lib, q, k, pos, 128, True, kw)
        check(qo, q, pos, 128, interleaved=True, **kw)
        check(ko, k, pos, 128, interleaved=True, **kw)


@pytest.mark.parametrize("R", [32, 128])
@pytest.mark.parametrize("inter", [True, False])
def test_in_place_one_side_and_views(gpu_lib, R, inter):
    q, k, pos = make(130, 6, 2, 128, 5000, 2)
    qo, ko = call(gpu_lib, q, k, pos, R, inter, {})
    only_q, none = call(gpu_lib, q, None, pos, R, inter, {})
    assert none is None and torch.equal(only_q, qo)
    none, only_k = call(gpu_lib, None, k, pos, R, inter, {})
    assert none is None and torch.equal(only_k, ko)
    # q in place, k into a new tensor
    q2 = q.clone()
    a, b = call(gpu_lib, q2, k, pos, R, inter, {}, q_out=q2)
    assert a is q2 and torch.equal(q2, qo) and torch.equal(b, ko)
    # both in place in the fused buffer, what lies beside them untouched
    buf = torch.randn(130, 11, 128, device="cuda").bfloat16()
    buf[:, 1:7], buf[:, 8:10] = q, k
    was = buf.clone()
    call(gpu_lib, buf[:, 1:7], buf[:, 8:10], pos, R, inter, {}, q_out=buf[:, 1:7], k_out=buf[:, 8:10])
    assert torch.equal(buf[:, 1:7], qo) and torch.equal(buf[:, 8:10], ko)
    assert all(torch.equal(buf[:, i], was[:, i]) for i in (0, 7, 10))
    # heads before tokens
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(call(gpu_lib, qt, None, pos, R, inter, {})[0], qo)


def test_equals_the_axes_operator_unscaled(gpu_lib):
    """One axis, whole heads, no scaling: the same frequencies as rope_axes, within a rounding of bf16."""
    q, k, pos = make(200, 5, 3, 128, 100000, 3)
    for inter in (True, False):
        a = gpu_lib.rope_axes(q, k, pos[:, None].contiguous(), (128,), interleaved=inter)
        b = gpu_lib.rope_scaled(q, k, pos, interleaved=inter)
        for x, y in zip(a, b):
            assert bool(((x.float() - y.float()).abs() <= 2.0 ** -7 * y.float().abs() + 1e-5).all())


def test_non_finite_elements_stay_in_their_pair(gpu_lib):
    q, _, pos = make(20, 3, 1, 64, 100, 4)
    q = q.contiguous()
    clean = gpu_lib.rope_scaled(q, None, pos, rotary_dim=32)[0]
    q[3, 1, 5] = float("nan")
    q[4, 2, 40] = float("inf")       # past the turned part: copied
    out = gpu_lib.rope_scaled(q, None, pos, rotary_dim=32)[0]
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[3, 1, 5] = bad[3, 1, 21] = True
    assert bool(torch.isnan(out[bad]).all()) and torch.isinf(out[4, 2, 40])
    bad[4, 2, 40] = True
    assert torch.equal(out[~bad], clean[~bad])


def test_side_stream_graph_and_empty(gpu_lib):
    q, k, pos = make(100, 6, 2, 128, 5000, 5)
    ref = gpu_lib.rope_scaled(q, k, pos, rotary_dim=64)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.rope_scaled(q, k, pos, rotary_dim=64, q_out=qo, k_out=ko)
    for _ in range(3):
        qo.zero_(), ko.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, ref[0]) and torch.equal(ko, ref[1])
        assert torch.equal(gpu_lib.rope_scaled(q, k, pos, rotary_dim=64)[0], ref[0])
    none, _ = gpu_lib.rope_scaled(q[:0], None, pos[:0])
    assert none.shape == (0, 6, 128)
