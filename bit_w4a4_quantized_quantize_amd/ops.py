"""PyTorch-facing binding of the HIP library: argument marshalling only.

Every function checks dtype/device/contiguity, allocates outputs with torch
(device memory and the current stream are the only things torch provides),
and calls the C ABI with raw pointers. All arithmetic happens in the HIP
kernels; there is no CPU or PyTorch fallback.

Tensors (bf16 unless stated): x [M, K]; smooth [K]; qweight uint8 [N, K/2]
(low nibble = even k); wscales uint8 [K/16, N] (e4m3fn bytes; a
torch.float8_e4m3fn tensor is accepted and viewed as bytes); wcscales [N];
wtscale [1]; proj_down [K, R]; proj_up [N, R]; bias [N] or None.
"""

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import ACT_CANONICAL, ACT_MXFP4, ACT_PACKED, WEIGHT_CANONICAL, WEIGHT_PACKED, SvdqError  # noqa: F401


def _bytes(t):
    if t.dtype == torch.float8_e4m3fn or t.dtype == torch.int8:
        return t.view(torch.uint8)
    return t


def _need(t, name, dtype, ndim=None, shape=None, min_numel=None):
    """Check a tensor argument before its pointer reaches the C ABI, which cannot see
    sizes: dtype, rank, exact shape or a minimum element count, and contiguity. The
    device is checked separately (_devices), after every size check of the call, so a
    size mistake is reported as such on any host."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None:
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    elif ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} has {t.numel()} elements, at least {int(min_numel)} needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _devices(**tensors):
    """Every given tensor (None skipped) is a GPU tensor, all on one device; returns it."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return dev


def _k_ok(K):
    if K <= 0 or K % 16 != 0:
        raise ValueError(f"K = {K} must be a positive multiple of 16")


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(device=None):
    return torch.cuda.current_stream(device).cuda_stream


def set_gemm_tile(tile):
    """Tile shape of the W4A4 GEMM on packed operands, process-wide (tests and tuning):
    0 automatic, 1 256 x 320, 2 256 x 256, 3 128 x 320, 4 128 x 160. Returns the previous
    value. Results are bit-identical for every shape."""
    prev = ctypes.c_int(0)
    _lib.check("svdq_set_gemm_tile", _lib.lib().svdq_set_gemm_tile(int(tile), ctypes.byref(prev)))
    return prev.value


def quantize_act(x, smooth, proj_down=None, qact=None, ascales=None, lora_act=None, packed=False,
                 workspace=None, mx=False):
    """quant(x * smooth) and, with proj_down, lora_act = x @ proj_down.

    Returns (qact, ascales, lora_act): canonical qact uint8 [M, K/2] and ascales
    uint8 [K/16, M]; or, with packed=True, one packed uint8 buffer (the packed
    weight layout with rows = tokens) and ascales None; or, with mx=True, the
    MXFP4 variant's code and scale buffers (as quantize_act_mxfp4 gives them).
    lora_act bf16 [M, R] or None. workspace: optional uint8 device tensor of at
    least quantize_act_workspace_bytes(M, K, R) bytes (allocated here when None).
    """
    if mx and packed:
        raise ValueError("packed and mx are two different layouts")
    return _quantize_act(x, smooth, None, proj_down, qact, ascales, lora_act, packed, workspace, mx)


def quantize_act_static(x, smooth, act_gscale, proj_down=None, qact=None, ascales=None, lora_act=None,
                        packed=False, workspace=None):
    """As quantize_act, with the block scales relative to the static global activation
    scale act_gscale (bf16 [1] device tensor, e.g. from calibrate_act_gscale)."""
    _need(act_gscale, "act_gscale", torch.bfloat16, shape=(1,))
    return _quantize_act(x, smooth, act_gscale, proj_down, qact, ascales, lora_act, packed, workspace)


def calibrate_act_gscale(x, smooth, act_gscale=None, workspace=None):
    """Static global activation scale from a calibration batch x [M, K] (bf16):
    bf16(max |x * smooth| / (6 * 448)), or 1 when that maximum is 0. Returns bf16 [1]."""
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    _k_ok(K)
    _need(smooth, "smooth", torch.bfloat16, shape=(K,))
    dev = x.device
    if act_gscale is None:
        act_gscale = torch.empty(1, dtype=torch.bfloat16, device=dev)
    _need(act_gscale, "act_gscale", torch.bfloat16, shape=(1,))
    L = _lib.lib()
    nbytes = L.svdq_calibrate_workspace_bytes(M, K)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, 1, min_numel=nbytes)
    _devices(x=x, smooth=smooth, act_gscale=act_gscale, workspace=workspace)
    _lib.check("svdq_calibrate_act_gscale", L.svdq_calibrate_act_gscale(
        _p(x), _p(smooth), M, K, _p(act_gscale), _p(workspace), workspace.numel(), _stream(dev)))
    return act_gscale


def _quantize_act(x, smooth, act_gscale, proj_down, qact, ascales, lora_act, packed, workspace, mx=False):
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    _k_ok(K)
    dev = x.device
    _need(smooth, "smooth", torch.bfloat16, shape=(K,))
    R = 0
    if proj_down is not None:
        _need(proj_down, "proj_down", torch.bfloat16, 2)
        R = proj_down.shape[1]
        _need(proj_down, "proj_down", torch.bfloat16, shape=(K, R))
    L = _lib.lib()
    if mx:
        if K % 128 != 0:
            raise ValueError(f"K={K}: the MXFP4 layout needs K a multiple of 128")
        if qact is None or ascales is None:
            c, sc = mx_buffers(M, K, dev)
            qact = c if qact is None else qact
            ascales = sc if ascales is None else ascales
        _check_mx_operands(qact, ascales, M, K, "act")
    elif packed:
        nbytes = L.svdq_packed_act_bytes(M, K)
        if qact is None:
            qact = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
        _need(qact, "qact (packed)", torch.uint8, 1, min_numel=nbytes)
        if ascales is not None:
            raise ValueError("ascales must be None with packed=True (the packed buffer holds the scales)")
    else:
        if qact is None:
            qact = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
        if ascales is None:
            ascales = torch.empty((K // 16, M), dtype=torch.uint8, device=dev)
        _need(qact, "qact", torch.uint8, shape=(M, K // 2))
        _need(_bytes(ascales), "ascales", torch.uint8, shape=(K // 16, M))
    if R > 0:
        if lora_act is None:
            lora_act = torch.empty((M, R), dtype=torch.bfloat16, device=dev)
        _need(lora_act, "lora_act", torch.bfloat16, shape=(M, R))
    ws_need = quantize_act_workspace_bytes(M, K, R)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=dev)
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = _need(workspace, "workspace", torch.uint8, 1, min_numel=ws_need).numel()
    _devices(x=x, smooth=smooth, act_gscale=act_gscale, proj_down=proj_down, qact=qact, ascales=ascales,
             lora_act=lora_act, workspace=workspace)
    layout = ACT_MXFP4 if mx else ACT_PACKED if packed else ACT_CANONICAL
    rest = (_p(proj_down), R, layout, _p(qact), _p(_bytes(ascales)) if ascales is not None else None,
            _p(lora_act) if R > 0 else None, _p(workspace), ws_bytes, _stream(dev))
    if act_gscale is None:
        _lib.check("svdq_quantize_act", L.svdq_quantize_act(_p(x), _p(smooth), M, K, *rest))
    else:
        _lib.check("svdq_quantize_act_static", L.svdq_quantize_act_static(_p(x), _p(smooth), _p(act_gscale), M, K,
                                                                          *rest))
    return qact, ascales, (lora_act if R > 0 else None)


def quantize_act_workspace_bytes(M, K, R):
    """Scratch bytes svdq_quantize_act needs (fp32 partials when K is split)."""
    return int(_lib.lib().svdq_quantize_act_workspace_bytes(M, K, R))


def repack_weight(qweight, wscales):
    """qweight [N, K/2] + wscales [K/16, N] -> packed uint8 buffer (MFMA order)."""
    qweight = _need(_bytes(qweight), "qweight", torch.uint8, 2)
    N, Kh = qweight.shape
    K = 2 * Kh
    _k_ok(K)
    wscales = _need(_bytes(wscales), "wscales", torch.uint8, shape=(K // 16, N))
    L = _lib.lib()
    nbytes = L.svdq_repack_weight_bytes(N, K)
    packed = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=qweight.device)
    _devices(qweight=qweight, wscales=wscales)
    _lib.check("svdq_repack_weight", L.svdq_repack_weight(
        _p(qweight), _p(wscales), N, K, _p(packed), nbytes, _stream(qweight.device)))
    return packed


def unpack_weight(packed, N, K):
    """Inverse of repack_weight: -> (qweight uint8 [N, K/2], wscales uint8 [K/16, N])."""
    _k_ok(K)
    _need(packed, "packed", torch.uint8, 1, min_numel=_lib.lib().svdq_repack_weight_bytes(N, K))
    _devices(packed=packed)
    qweight = torch.empty((N, K // 2), dtype=torch.uint8, device=packed.device)
    wscales = torch.empty((K // 16, N), dtype=torch.uint8, device=packed.device)
    L = _lib.lib()
    _lib.check("svdq_unpack_weight", L.svdq_unpack_weight(
        _p(packed), packed.numel(), N, K, _p(qweight), _p(wscales), _stream(packed.device)))
    return qweight, wscales


@dataclass
class SVDQLinearWeights:
    """One quantised linear layer's tensors, on the GPU.

    weight is qweight [N, K/2] (layout WEIGHT_CANONICAL, wscales given) or a
    buffer from repack_weight (layout WEIGHT_PACKED, wscales None).
    """
    N: int
    K: int
    weight: torch.Tensor
    wscales: Optional[torch.Tensor]
    wcscales: torch.Tensor
    wtscale: torch.Tensor
    smooth: torch.Tensor
    proj_down: Optional[torch.Tensor]
    proj_up: Optional[torch.Tensor]
    bias: Optional[torch.Tensor] = None
    layout: int = WEIGHT_CANONICAL

    @property
    def R(self):
        return 0 if self.proj_down is None else int(self.proj_down.shape[1])

    def packed(self):
        """A copy of this layer with the weight repacked (load-time step)."""
        if self.layout == WEIGHT_PACKED:
            return self
        buf = repack_weight(self.weight, self.wscales)
        return SVDQLinearWeights(self.N, self.K, buf, None, self.wcscales, self.wtscale, self.smooth,
                                 self.proj_down, self.proj_up, self.bias, WEIGHT_PACKED)


def _layer_tensors(w: SVDQLinearWeights):
    return dict(weight=w.weight, wscales=w.wscales, wcscales=w.wcscales, wtscale=w.wtscale, smooth=w.smooth,
                proj_down=w.proj_down, proj_up=w.proj_up, bias=w.bias)


def _check_layer(w: SVDQLinearWeights):
    """Every tensor of the layer against (N, K, R): dtype, shape (or size), device."""
    N, K = int(w.N), int(w.K)
    _k_ok(K)
    if w.layout == WEIGHT_CANONICAL:
        _need(_bytes(w.weight), "qweight", torch.uint8, shape=(N, K // 2))
        if w.wscales is None:
            raise ValueError("wscales is required with the canonical weight layout")
        dev = w.weight.device
        _need(_bytes(w.wscales), "wscales", torch.uint8, shape=(K // 16, N))
    elif w.layout == WEIGHT_PACKED:
        _need(w.weight, "packed weight", torch.uint8, 1, min_numel=_lib.lib().svdq_repack_weight_bytes(N, K))
        if w.wscales is not None:
            raise ValueError("wscales must be None with the packed weight layout (the buffer holds them)")
        dev = w.weight.device
    else:
        raise ValueError(f"unknown weight layout {w.layout}")
    _need(w.wcscales, "wcscales", torch.bfloat16, shape=(N,))
    _need(w.wtscale, "wtscale", torch.bfloat16, shape=(1,))
    _need(w.smooth, "smooth", torch.bfloat16, shape=(K,))
    R = w.R
    if R > 0:
        _need(w.proj_down, "proj_down", torch.bfloat16, shape=(K, R))
        _need(w.proj_up, "proj_up", torch.bfloat16, shape=(N, R))
    if w.bias is not None:
        _need(w.bias, "bias", torch.bfloat16, shape=(N,))
    return dev


def gemm_w4a4(qact, ascales, lora_act, w: SVDQLinearWeights, y=None, M=None):
    """The scaled GEMM + low-rank up-projection + epilogue from quantised activations.

    Canonical activations: qact [M, K/2], ascales [K/16, M]. Packed activations
    (from quantize_act(..., packed=True)): qact is the packed buffer, ascales
    None, and M must be given. Either weight layout goes with either.
    """
    dev = _check_layer(w)
    K = w.K
    L = _lib.lib()
    act_packed = ascales is None
    if act_packed:
        if M is None:
            raise ValueError("M is required with packed activations")
        _need(qact, "qact (packed)", torch.uint8, 1, min_numel=L.svdq_packed_act_bytes(M, K))
    else:
        _need(qact, "qact", torch.uint8, 2)
        M = qact.shape[0]
        _need(qact, "qact", torch.uint8, shape=(M, K // 2))
        ascales = _need(_bytes(ascales), "ascales", torch.uint8, shape=(K // 16, M))
    if w.R > 0:
        _need(lora_act, "lora_act", torch.bfloat16, shape=(M, w.R))
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, shape=(M, w.N))
    _devices(**_layer_tensors(w), qact=qact, ascales=ascales, lora_act=lora_act, y=y)
    _lib.check("svdq_gemm_w4a4", L.svdq_gemm_w4a4(
        _p(qact), _p(ascales), ACT_PACKED if act_packed else ACT_CANONICAL,
        _p(lora_act) if w.R > 0 else None,
        _p(_bytes(w.weight)), _p(_bytes(w.wscales)) if w.wscales is not None else None, w.layout,
        _p(w.wcscales), _p(w.wtscale), _p(w.proj_up) if w.R > 0 else None, _p(w.bias),
        M, w.N, w.K, w.R, _p(y), _stream(qact.device)))
    return y


def linear_workspace_bytes(M, N, K, R):
    return _lib.lib().svdq_linear_workspace_bytes(M, N, K, R)


def linear_w4a4(x, w: SVDQLinearWeights, y=None, workspace=None):
    """The whole layer: y [M, N] bf16."""
    return _linear(x, w, None, y, workspace)


def linear_w4a4_static(x, w: SVDQLinearWeights, act_gscale, y=None, workspace=None):
    """The whole layer with static activation scales relative to act_gscale (bf16 [1])."""
    _need(act_gscale, "act_gscale", torch.bfloat16, shape=(1,))
    return _linear(x, w, act_gscale, y, workspace)


def _linear(x, w, act_gscale, y, workspace):
    dev = _check_layer(w)
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    if K != w.K:
        raise ValueError(f"x has K={K}, the layer K={w.K}")
    _need(x, "x", torch.bfloat16, shape=(M, K))
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, shape=(M, w.N))
    L = _lib.lib()
    nbytes = L.svdq_linear_workspace_bytes(M, w.N, K, w.R)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, 1, min_numel=nbytes)
    _devices(**_layer_tensors(w), x=x, y=y, workspace=workspace, act_gscale=act_gscale)
    rest = (_p(_bytes(w.weight)), _p(_bytes(w.wscales)) if w.wscales is not None else None, w.layout,
            _p(w.wcscales), _p(w.wtscale), _p(w.proj_down) if w.R > 0 else None,
            _p(w.proj_up) if w.R > 0 else None, _p(w.bias), M, w.N, K, w.R,
            _p(y), _p(workspace), workspace.numel(), _stream(x.device))
    if act_gscale is None:
        _lib.check("svdq_linear_w4a4", L.svdq_linear_w4a4(_p(x), _p(w.smooth), *rest))
    else:
        _lib.check("svdq_linear_w4a4_static", L.svdq_linear_w4a4_static(_p(x), _p(w.smooth), _p(act_gscale), *rest))
    return y


def linear_w4a4_noalloc(x, w: SVDQLinearWeights, y):
    """The whole layer with the library's static device scratch as workspace (no
    allocation by the library; y [M, N] bf16 must be given). Raises SvdqError
    (SVDQ_ERR_WORKSPACE) when the problem needs more than noalloc_scratch_bytes()."""
    dev = _check_layer(w)
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    if K != w.K:
        raise ValueError(f"x has K={K}, the layer K={w.K}")
    _need(y, "y", torch.bfloat16, shape=(M, w.N))
    _devices(**_layer_tensors(w), x=x, y=y)
    L = _lib.lib()
    _lib.check("svdq_linear_w4a4_noalloc", L.svdq_linear_w4a4_noalloc(
        _p(x), _p(w.smooth), _p(_bytes(w.weight)),
        _p(_bytes(w.wscales)) if w.wscales is not None else None, w.layout,
        _p(w.wcscales), _p(w.wtscale), _p(w.proj_down) if w.R > 0 else None,
        _p(w.proj_up) if w.R > 0 else None, _p(w.bias), M, w.N, K, w.R, _p(y), _stream(dev)))
    return y


def noalloc_scratch_bytes():
    return int(_lib.lib().svdq_noalloc_scratch_bytes())


def _check_gated(w: SVDQLinearWeights):
    if w.layout != WEIGHT_PACKED:
        raise ValueError("the gated layer needs the packed weight layout (use .packed())")
    if w.N % 2 != 0:
        raise ValueError(f"the gated layer has 2F output channels, got N={w.N}")
    _check_layer(w)
    return w.N // 2


def gemm_w4a4_gated(qact, lora_act, w: SVDQLinearWeights, M, h=None):
    """Gated FFN step from packed activations: h [M, F] = silu(y[:, :F]) * y[:, F:]
    of the 2F-channel layer w (w1 and w3 as one layer), bf16."""
    F_out = _check_gated(w)
    dev = w.weight.device
    L = _lib.lib()
    _need(qact, "qact (packed)", torch.uint8, 1, min_numel=L.svdq_packed_act_bytes(M, w.K))
    if w.R > 0:
        _need(lora_act, "lora_act", torch.bfloat16, shape=(M, w.R))
    if h is None:
        h = torch.empty((M, F_out), dtype=torch.bfloat16, device=dev)
    _need(h, "h", torch.bfloat16, shape=(M, F_out))
    _devices(**_layer_tensors(w), qact=qact, lora_act=lora_act, h=h)
    _lib.check("svdq_gemm_w4a4_gated", L.svdq_gemm_w4a4_gated(
        _p(qact), _p(lora_act) if w.R > 0 else None, _p(_bytes(w.weight)), _p(w.wcscales),
        _p(w.wtscale), _p(w.proj_up) if w.R > 0 else None, _p(w.bias), M, F_out, w.K, w.R,
        _p(h), _stream(qact.device)))
    return h


def gemm_w4a4_gated_quant(qact, lora_act, w: SVDQLinearWeights, M, next_smooth, h=None, next_qact=None):
    """Gated FFN step from packed activations that also quantises h for the next layer
    (w2) with w2's smooth factor: returns (h [M, F] bf16, next_qact packed uint8 buffer of
    the [M, F] activation, as quantize_act(h, next_smooth, packed=True) would give)."""
    F_out = _check_gated(w)
    dev = w.weight.device
    L = _lib.lib()
    _need(qact, "qact (packed)", torch.uint8, 1, min_numel=L.svdq_packed_act_bytes(M, w.K))
    if w.R > 0:
        _need(lora_act, "lora_act", torch.bfloat16, shape=(M, w.R))
    _need(next_smooth, "next_smooth", torch.bfloat16, shape=(F_out,))
    if h is None:
        h = torch.empty((M, F_out), dtype=torch.bfloat16, device=dev)
    _need(h, "h", torch.bfloat16, shape=(M, F_out))
    nbytes = L.svdq_packed_act_bytes(M, F_out)
    if next_qact is None:
        next_qact = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(next_qact, "next_qact", torch.uint8, 1, min_numel=nbytes)
    _devices(**_layer_tensors(w), qact=qact, lora_act=lora_act, h=h, next_smooth=next_smooth, next_qact=next_qact)
    _lib.check("svdq_gemm_w4a4_gated_quant", L.svdq_gemm_w4a4_gated_quant(
        _p(qact), _p(lora_act) if w.R > 0 else None, _p(_bytes(w.weight)), _p(w.wcscales), _p(w.wtscale),
        _p(w.proj_up) if w.R > 0 else None, _p(w.bias), M, F_out, w.K, w.R, _p(h), _p(next_smooth),
        _p(next_qact), next_qact.numel(), _stream(dev)))
    return h, next_qact


def lowrank_down(x, proj_down, lora_act=None, workspace=None):
    """lora_act [M, R] = bf16(x @ proj_down) alone (x [M, K], proj_down [K, R], bf16)."""
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    _k_ok(K)
    _need(proj_down, "proj_down", torch.bfloat16, 2)
    R = proj_down.shape[1]
    _need(proj_down, "proj_down", torch.bfloat16, shape=(K, R))
    dev = x.device
    if lora_act is None:
        lora_act = torch.empty((M, R), dtype=torch.bfloat16, device=dev)
    _need(lora_act, "lora_act", torch.bfloat16, shape=(M, R))
    need = quantize_act_workspace_bytes(M, K, R)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = _need(workspace, "workspace", torch.uint8, 1, min_numel=need).numel()
    _devices(x=x, proj_down=proj_down, lora_act=lora_act, workspace=workspace)
    L = _lib.lib()
    _lib.check("svdq_lowrank_down", L.svdq_lowrank_down(_p(x), _p(proj_down), M, K, R, _p(lora_act),
                                                         _p(workspace), ws_bytes, _stream(dev)))
    return lora_act


def linear_w4a4_gated(x, w: SVDQLinearWeights, h=None, workspace=None):
    """The whole gated step from x: h [M, F] bf16 (w is the 2F-channel w1/w3 layer)."""
    F_out = _check_gated(w)
    dev = w.weight.device
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    if K != w.K:
        raise ValueError(f"x has K={K}, the layer K={w.K}")
    _need(x, "x", torch.bfloat16, shape=(M, K))
    if h is None:
        h = torch.empty((M, F_out), dtype=torch.bfloat16, device=dev)
    _need(h, "h", torch.bfloat16, shape=(M, F_out))
    L = _lib.lib()
    nbytes = L.svdq_linear_gated_workspace_bytes(M, F_out, K, w.R)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, 1, min_numel=nbytes)
    _devices(**_layer_tensors(w), x=x, h=h, workspace=workspace)
    _lib.check("svdq_linear_w4a4_gated", L.svdq_linear_w4a4_gated(
        _p(x), _p(w.smooth), _p(_bytes(w.weight)), _p(w.wcscales), _p(w.wtscale),
        _p(w.proj_down) if w.R > 0 else None, _p(w.proj_up) if w.R > 0 else None, _p(w.bias),
        M, F_out, K, w.R, _p(h), _p(workspace), workspace.numel(), _stream(x.device)))
    return h


def linear_bf16(x, weight, bias=None, y=None):
    """A linear kept in bf16: y [M, N] = bf16(x @ weight^T + bias), with x [M, K],
    weight [N, K] and bias [N] (or None), all bf16."""
    _need(x, "x", torch.bfloat16, 2)
    _need(weight, "weight", torch.bfloat16, 2)
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"x has K={K}, weight has K={weight.shape[1]}")
    dev = x.device
    _need(weight, "weight", torch.bfloat16, shape=(N, K))
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, shape=(N,))
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, shape=(M, N))
    L = _lib.lib()
    _devices(x=x, weight=weight, bias=bias, y=y)
    _lib.check("svdq_linear_bf16", L.svdq_linear_bf16(
        _p(x), _p(weight), _p(bias), M, N, K, _p(y), _stream(x.device)))
    return y


def prepare_workspace_bytes(N, K, R):
    return _lib.lib().svdq_prepare_workspace_bytes(N, K, R)


def _prep_outputs(N, K, R, dev):
    u8 = torch.uint8
    return dict(qweight=torch.empty((N, K // 2), dtype=u8, device=dev),
                wscales=torch.empty((K // 16, N), dtype=u8, device=dev),
                wcscales=torch.empty(N, dtype=torch.bfloat16, device=dev),
                wtscale=torch.empty(1, dtype=torch.bfloat16, device=dev))


def prepare_weight(weight, smooth, omega=None, iters=2, bias=None, workspace=None):
    """SVDQuant preparation of a bf16 weight [N, K] with smooth [K]: the rank-R
    split (R = omega.shape[1]; omega [K, R] float32 Gaussian, or None for R = 0),
    the residual's two-level scales and NVFP4 codes. Returns SVDQLinearWeights
    (canonical layout)."""
    _need(weight, "weight", torch.bfloat16, 2)
    N, K = weight.shape
    _k_ok(K)
    dev = weight.device
    _need(smooth, "smooth", torch.bfloat16, shape=(K,))
    R = 0
    if omega is not None:
        _need(omega, "omega", torch.float32, 2)
        if omega.shape[0] != K:
            raise ValueError(f"omega must be [K={K}, R], got {tuple(omega.shape)}")
        R = omega.shape[1]
        _need(omega, "omega", torch.float32, shape=(K, R))
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, shape=(N,))
    out = _prep_outputs(N, K, R, dev)
    pd = torch.empty((K, R), dtype=torch.bfloat16, device=dev) if R else None
    pu = torch.empty((N, R), dtype=torch.bfloat16, device=dev) if R else None
    L = _lib.lib()
    nbytes = L.svdq_prepare_workspace_bytes(N, K, R)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, 1, min_numel=nbytes)
    _devices(weight=weight, smooth=smooth, omega=omega, bias=bias, workspace=workspace)
    _lib.check("svdq_prepare_weight", L.svdq_prepare_weight(
        _p(weight), _p(smooth), _p(omega), N, K, R, iters, _p(out["qweight"]), _p(out["wscales"]),
        _p(out["wcscales"]), _p(out["wtscale"]), _p(pd), _p(pu), _p(workspace), workspace.numel(),
        _stream(dev)))
    return SVDQLinearWeights(N=N, K=K, weight=out["qweight"], wscales=out["wscales"], wcscales=out["wcscales"],
                             wtscale=out["wtscale"], smooth=smooth, proj_down=pd, proj_up=pu, bias=bias)


def prepare_residual(weight, smooth, proj_down=None, proj_up=None, workspace=None):
    """Steps 3-5 of the preparation for given bf16 factors: returns
    (qweight, wscales, wcscales, wtscale)."""
    _need(weight, "weight", torch.bfloat16, 2)
    N, K = weight.shape
    _k_ok(K)
    dev = weight.device
    _need(smooth, "smooth", torch.bfloat16, shape=(K,))
    if proj_down is not None:
        _need(proj_down, "proj_down", torch.bfloat16, 2)
    R = 0 if proj_down is None else proj_down.shape[1]
    if R:
        _need(proj_down, "proj_down", torch.bfloat16, shape=(K, R))
        _need(proj_up, "proj_up", torch.bfloat16, shape=(N, R))
    out = _prep_outputs(N, K, R, dev)
    L = _lib.lib()
    nbytes = L.svdq_prepare_workspace_bytes(N, K, R)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, 1, min_numel=nbytes)
    _devices(weight=weight, smooth=smooth, proj_down=proj_down, proj_up=proj_up, workspace=workspace)
    _lib.check("svdq_prepare_residual", L.svdq_prepare_residual(
        _p(weight), _p(smooth), _p(proj_down), _p(proj_up), N, K, R, _p(out["qweight"]), _p(out["wscales"]),
        _p(out["wcscales"]), _p(out["wtscale"]), _p(workspace), workspace.numel(), _stream(dev)))
    return out["qweight"], out["wscales"], out["wcscales"], out["wtscale"]


def mx_buffers(rows, K, dev):
    L = _lib.lib()
    return (torch.empty(L.svdq_mx_codes_bytes(rows, K), dtype=torch.uint8, device=dev),
            torch.empty(L.svdq_mx_scales_bytes(rows, K), dtype=torch.uint8, device=dev))


def _check_mx_operands(codes, scales, rows, K, name):
    L = _lib.lib()
    _need(codes, f"{name}_codes", torch.uint8, 1, min_numel=L.svdq_mx_codes_bytes(rows, K))
    _need(scales, f"{name}_scales", torch.uint8, 1, min_numel=L.svdq_mx_scales_bytes(rows, K))


def reround_weight_mxfp4(w: "SVDQLinearWeights"):
    """MXFP4 variant: the layer's canonical NVFP4 weight re-rounded to MX codes and
    scales (load time). Returns (mx_codes, mx_scales) uint8 buffers."""
    _check_layer(w)
    if w.layout != WEIGHT_CANONICAL:
        raise ValueError("re-rounding reads the canonical weight layout")
    codes, scales = mx_buffers(w.N, w.K, w.weight.device)
    L = _lib.lib()
    _devices(**_layer_tensors(w), codes=codes, scales=scales)
    _lib.check("svdq_reround_weight_mxfp4", L.svdq_reround_weight_mxfp4(
        _p(_bytes(w.weight)), _p(_bytes(w.wscales)), w.N, w.K, _p(codes), _p(scales), _stream(w.weight.device)))
    return codes, scales


def quantize_act_mxfp4(x, smooth):
    """MX(x * smooth): returns (mx_codes, mx_scales) uint8 buffers."""
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    _k_ok(K)
    _need(smooth, "smooth", torch.bfloat16, shape=(K,))
    codes, scales = mx_buffers(M, K, x.device)
    L = _lib.lib()
    _devices(x=x, smooth=smooth)
    _lib.check("svdq_quantize_act_mxfp4", L.svdq_quantize_act_mxfp4(
        _p(x), _p(smooth), M, K, _p(codes), _p(scales), _stream(x.device)))
    return codes, scales


def gemm_mxfp4(act_codes, act_scales, lora_act, w_codes, w_scales, w: "SVDQLinearWeights", M, y=None):
    """The variant's GEMM + low-rank up-projection + epilogue: y [M, N] bf16."""
    dev = _check_layer(w)
    L = _lib.lib()
    _check_mx_operands(act_codes, act_scales, M, w.K, "act")
    _check_mx_operands(w_codes, w_scales, w.N, w.K, "w")
    if w.R > 0:
        _need(lora_act, "lora_act", torch.bfloat16, shape=(M, w.R))
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, shape=(M, w.N))
    _devices(**_layer_tensors(w), act_codes=act_codes, act_scales=act_scales, lora_act=lora_act, w_codes=w_codes,
             w_scales=w_scales, y=y)
    _lib.check("svdq_gemm_mxfp4", L.svdq_gemm_mxfp4(
        _p(act_codes), _p(act_scales), _p(lora_act) if w.R > 0 else None, _p(w_codes), _p(w_scales),
        _p(w.wcscales), _p(w.wtscale), _p(w.proj_up) if w.R > 0 else None, _p(w.bias), M, w.N, w.K, w.R,
        _p(y), _stream(act_codes.device)))
    return y


def linear_mxfp4(x, w: "SVDQLinearWeights", w_codes, w_scales, y=None, workspace=None):
    """The whole MXFP4 variant layer from x (w supplies smooth, wcscales, wtscale,
    the low-rank factors and bias; w_codes / w_scales from reround_weight_mxfp4)."""
    dev = _check_layer(w)
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    if K != w.K:
        raise ValueError(f"x has K={K}, the layer K={w.K}")
    _need(x, "x", torch.bfloat16, shape=(M, K))
    _check_mx_operands(w_codes, w_scales, w.N, K, "w")
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, shape=(M, w.N))
    L = _lib.lib()
    nbytes = L.svdq_linear_mxfp4_workspace_bytes(M, K, w.R)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, 1, min_numel=nbytes)
    _devices(**_layer_tensors(w), x=x, w_codes=w_codes, w_scales=w_scales, y=y, workspace=workspace)
    _lib.check("svdq_linear_mxfp4", L.svdq_linear_mxfp4(
        _p(x), _p(w.smooth), _p(w_codes), _p(w_scales), _p(w.wcscales), _p(w.wtscale),
        _p(w.proj_down) if w.R > 0 else None, _p(w.proj_up) if w.R > 0 else None, _p(w.bias),
        M, w.N, K, w.R, _p(y), _p(workspace), workspace.numel(), _stream(x.device)))
    return y


# the current stream's handle without the Stream object around it (1.6 us less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _stream
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(name, dev, *args):
    """Call the C entry point `name` on dev's current stream, with dev the current HIP device."""
    fn = getattr(_lib.lib(), name)
    index = dev.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        _lib.check(name, status)


def _on_one_device(index, **tensors):
    """Every given tensor (None skipped) is on GPU `index`; the error is _devices'."""
    for t in tensors.values():
        if t is not None and t.get_device() != index:
            _devices(**tensors)
    if index < 0:
        _devices(**tensors)


def _workspace(workspace, need, dev):
    """The given workspace, checked, or a new one (None when no bytes are needed); and its size."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return workspace, _need(workspace, "workspace", torch.uint8, 1, min_numel=need).numel()


def quantize_int8(x, smooth=None, codes=None, scales=None):
    """8-bit codes with one scale per row: v = x * smooth, scales = max |v| / 127 (float32
    [M]), codes = round(v * (127 / max |v|)) (int8 [M, K]). x [M, K] bf16, smooth [K] bf16 or
    None. The same rule quantises activations (rows = tokens) and weights (rows = output
    channels, smooth = 1 / the layer's smooth). Returns (codes, scales)."""
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    _k_ok(K)
    if smooth is not None:
        _need(smooth, "smooth", torch.bfloat16, shape=(K,))
    dev = x.device
    if codes is None:
        codes = torch.empty_like(x, dtype=torch.int8)
    else:
        _need(codes, "codes", torch.int8, shape=(M, K))
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=dev)
    else:
        _need(scales, "scales", torch.float32, shape=(M,))
    _on_one_device(x.get_device(), x=x, smooth=smooth, codes=codes, scales=scales)
    _launch("svdq_quantize_int8", dev, _p(x), _p(smooth), M, K, _p(codes), _p(scales))
    return codes, scales


def _check_int8_weight(weight, wscales, bias, K):
    _need(weight, "weight", torch.int8, 2)
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"the activations have K={K}, weight has K={weight.shape[1]}")
    _need(weight, "weight", torch.int8, shape=(N, K))
    _need(wscales, "wscales", torch.float32, shape=(N,))
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, shape=(N,))
    return N


def gemm_int8_workspace_bytes(M, N, K):
    """Scratch bytes gemm_int8 needs."""
    return _lib.lib().svdq_gemm_int8_workspace_bytes(M, N, K)


def gemm_int8_plan(M, N, K):
    """How gemm_int8 runs a size (tests and tuning): (tile, ways k is split), tile 0..7 as in svdq.h or -1 for
    the kernel for few tokens."""
    tile, splits = ctypes.c_int(0), ctypes.c_int(0)
    _lib.check("svdq_gemm_int8_plan", _lib.lib().svdq_gemm_int8_plan(M, N, K, ctypes.byref(tile), ctypes.byref(splits)))
    return tile.value, splits.value


def linear_int8_workspace_bytes(M, N, K):
    """Scratch bytes linear_int8 needs."""
    return _lib.lib().svdq_linear_int8_workspace_bytes(M, N, K)


def gemm_int8(codes, ascales, weight, wscales, bias=None, y=None, workspace=None):
    """y [M, N] bf16 = (codes @ weight^T) * ascales[m] * wscales[n] + bias from 8-bit codes:
    codes int8 [M, K], ascales float32 [M] (quantize_int8 or norm_gated_int8), weight int8
    [N, K], wscales float32 [N], bias bf16 [N] or None. K <= 131072."""
    _need(codes, "codes", torch.int8, 2)
    M, K = codes.shape
    _k_ok(K)
    _need(ascales, "ascales", torch.float32, shape=(M,))
    N = _check_int8_weight(weight, wscales, bias, K)
    dev = codes.device
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    else:
        _need(y, "y", torch.bfloat16, shape=(M, N))
    workspace, ws_bytes = _workspace(workspace, gemm_int8_workspace_bytes(M, N, K), dev)
    _on_one_device(codes.get_device(), codes=codes, ascales=ascales, weight=weight, wscales=wscales, bias=bias, y=y,
                   workspace=workspace)
    _launch("svdq_gemm_int8", dev, _p(codes), _p(ascales), _p(weight), _p(wscales), _p(bias), M, N, K, _p(y),
            _p(workspace), ws_bytes)
    return y


def linear_int8(x, weight, wscales, bias=None, smooth=None, y=None, workspace=None):
    """The whole linear in 8-bit integers: quantize_int8(x, smooth), then gemm_int8. x [M, K]
    bf16, weight int8 [N, K], wscales float32 [N]; returns y [M, N] bf16."""
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    _k_ok(K)
    N = _check_int8_weight(weight, wscales, bias, K)
    if smooth is not None:
        _need(smooth, "smooth", torch.bfloat16, shape=(K,))
    dev = x.device
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    else:
        _need(y, "y", torch.bfloat16, shape=(M, N))
    workspace, ws_bytes = _workspace(workspace, linear_int8_workspace_bytes(M, N, K), dev)
    _on_one_device(x.get_device(), x=x, smooth=smooth, weight=weight, wscales=wscales, bias=bias, y=y,
                   workspace=workspace)
    _launch("svdq_linear_int8", dev, _p(x), _p(smooth), _p(weight), _p(wscales), _p(bias), M, N, K, _p(y),
            _p(workspace), ws_bytes)
    return y


def _check_norm(h, block, post_weight, gate, pre_weight, scale, cu_seqlens, h_out):
    """Arguments common to the two norms; returns (M, K, G, h_out)."""
    _need(h, "h", torch.bfloat16, 2)
    M, K = h.shape
    _k_ok(K)
    G = 1
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1, min_numel=2)
        G = cu_seqlens.numel() - 1
    if block is not None:
        _need(block, "block", torch.bfloat16, shape=(M, K))
        if h_out is None:
            h_out = torch.empty_like(h)
        else:
            _need(h_out, "h_out", torch.bfloat16, shape=(M, K))
    if post_weight is not None:
        _need(post_weight, "post_weight", torch.bfloat16, shape=(K,))
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, shape=(G, K))
    if pre_weight is not None:
        _need(pre_weight, "pre_weight", torch.bfloat16, shape=(K,))
    if scale is not None:
        _need(scale, "scale", torch.bfloat16, shape=(G, K))
    return M, K, G, h_out


def norm_gated(h, block=None, post_weight=None, gate=None, residual_scale=1.0, pre_weight=None, scale=None,
               cu_seqlens=None, eps=1e-6, h_out=None, x_out=None, pre=True):
    """The norms between two transformer blocks, in one pass:

        h_out = h + residual_scale * gate[g] * rms(block) * post_weight
        x_out = rms(h_out) * pre_weight * (1 + scale[g])

    h, block [M, K] bf16 (block None before the first block: x_out from h, and h_out None);
    weights [K] or None (1); gate, scale [G, K] or None (1 and 0); cu_seqlens int32 [G + 1] row
    offsets of the groups, or None for one group. Rows outside cu_seqlens are not written. h_out
    may be h (in place). pre=False leaves x_out out (after the last block). Returns (h_out, x_out)."""
    M, K, G, h_out = _check_norm(h, block, post_weight, gate, pre_weight, scale, cu_seqlens, h_out)
    if pre:
        if x_out is None:
            x_out = torch.empty_like(h)
        else:
            _need(x_out, "x_out", torch.bfloat16, shape=(M, K))
    elif x_out is not None:
        raise ValueError("x_out must be None with pre=False")
    _on_one_device(h.get_device(), h=h, block=block, post_weight=post_weight, gate=gate, pre_weight=pre_weight,
                   scale=scale, cu_seqlens=cu_seqlens, h_out=h_out, x_out=x_out)
    _launch("svdq_norm_gated", h.device, _p(h), _p(block), _p(post_weight), _p(gate), residual_scale, _p(pre_weight),
            _p(scale), _p(cu_seqlens), G, M, K, eps, _p(h_out), _p(x_out))
    return h_out, x_out


def norm_gated_int8(h, block=None, post_weight=None, gate=None, residual_scale=1.0, pre_weight=None, scale=None,
                    cu_seqlens=None, eps=1e-6, h_out=None, smooth=None, codes=None, scales=None):
    """norm_gated whose x_out leaves as 8-bit codes for gemm_int8, those of
    quantize_int8(x_out, smooth) bit for bit. Returns (h_out, codes int8 [M, K], scales float32 [M])."""
    M, K, G, h_out = _check_norm(h, block, post_weight, gate, pre_weight, scale, cu_seqlens, h_out)
    if smooth is not None:
        _need(smooth, "smooth", torch.bfloat16, shape=(K,))
    if codes is None:
        codes = torch.empty_like(h, dtype=torch.int8)
    else:
        _need(codes, "codes", torch.int8, shape=(M, K))
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=h.device)
    else:
        _need(scales, "scales", torch.float32, shape=(M,))
    _on_one_device(h.get_device(), h=h, block=block, post_weight=post_weight, gate=gate, pre_weight=pre_weight,
                   scale=scale, cu_seqlens=cu_seqlens, h_out=h_out, smooth=smooth, codes=codes, scales=scales)
    _launch("svdq_norm_gated_int8", h.device, _p(h), _p(block), _p(post_weight), _p(gate), residual_scale,
            _p(pre_weight), _p(scale), _p(cu_seqlens), G, M, K, eps, _p(h_out), _p(smooth), _p(codes), _p(scales))
    return h_out, codes, scales


def _need_heads(t, name, shape=None):
    """Check a [tokens, heads, D] bf16 tensor, a view with any token and head strides (the D
    elements of a head are contiguous), and return it as the C ABI takes it: pointer, strides."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    have, strides = t.shape, t.stride()
    if len(have) != 3:
        raise ValueError(f"{name} must have 3 dims [tokens, heads, D], got shape {tuple(have)}")
    if shape is not None and have != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(have)}")
    if strides[2] != 1 and t.numel() > 0:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return t.data_ptr(), strides[0], strides[1]


_NO_HEADS = (None, 0, 0)


def rope_axes(q, k, positions, axis_dims, theta=10000.0, interleaved=True, q_weight=None, k_weight=None, eps=1e-6,
              q_out=None, k_out=None):
    """Rotary positions with several axes, after the per-head norm when a weight is given, for
    q [T, H, D] and k [T, Hk, D] (bf16 views with any token and head strides, as out of a fused
    qkv buffer; either may be None). positions int32 [T, A]; axis_dims: A even sizes of sum
    D: the i-th pair of axis a turns by positions[t, a] * theta^(-2i / axis_dims[a]). interleaved: pairs
    are neighbours, else halves of the head. q_weight, k_weight [D] bf16. q_out / k_out may be q / k
    themselves (in place); new ones are laid out like their input. Returns (q_out, k_out)."""
    if q is None and k is None:
        raise ValueError("q or k is required")
    given = q if q is not None else k
    qa, ka, qoa, koa, H, Hk = _NO_HEADS, _NO_HEADS, _NO_HEADS, _NO_HEADS, 0, 0
    if q is not None:
        qa = _need_heads(q, "q")
        H = q.shape[1]
    if k is not None:
        ka = _need_heads(k, "k")
        Hk = k.shape[1]
    T, _, D = given.shape
    if q is not None and k is not None and (k.shape[0] != T or k.shape[2] != D):
        raise ValueError(f"k must have shape {[T, Hk, D]}, got {list(k.shape)}")
    axis_dims = tuple(axis_dims)
    _need(positions, "positions", torch.int32, shape=(T, len(axis_dims)))
    if q_weight is not None:
        _need(q_weight, "q_weight", torch.bfloat16, shape=(D,))
    if k_weight is not None:
        _need(k_weight, "k_weight", torch.bfloat16, shape=(D,))
    if q is not None:
        q_out = torch.empty_like(q) if q_out is None else q_out
        qoa = _need_heads(q_out, "q_out", q.shape)
    elif q_weight is not None or q_out is not None:
        raise ValueError("q_weight and q_out need q")
    if k is not None:
        k_out = torch.empty_like(k) if k_out is None else k_out
        koa = _need_heads(k_out, "k_out", k.shape)
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    _on_one_device(given.get_device(), q=q, k=k, positions=positions, q_weight=q_weight, k_weight=k_weight,
                   q_out=q_out, k_out=k_out)
    _launch("svdq_rope_axes", given.device, *qa, H, *ka, Hk, _p(q_weight), _p(k_weight), eps, positions.data_ptr(),
            (ctypes.c_int32 * len(axis_dims))(*axis_dims), len(axis_dims), theta, 1 if interleaved else 0, T, D, *qoa,
            *koa)
    return q_out, k_out


def attention_packed(q, k, v, cu_seqlens=None, causal=False, scale=None, out=None):
    """softmax(scale * q k^T) v over whole packed sequences. q [T, H, D], k, v [T, Hk, D] bf16 (views
    with any token and head strides; H a multiple of Hk, D 64 or 128); cu_seqlens int32 [B + 1] token
    offsets of the sequences (None: one sequence); causal: a token sees itself and those before it
    in its sequence. scale defaults to D ** -0.5. Rows of a given `out` outside cu_seqlens are left as
    they were (a new one, laid out like q, is not initialised there). Returns out [T, H, D]."""
    qa = _need_heads(q, "q")
    T, H, D = q.shape
    ka = _need_heads(k, "k")
    Hk = k.shape[1]
    if k.shape[0] != T or k.shape[2] != D:
        raise ValueError(f"k must have shape {[T, Hk, D]}, got {list(k.shape)}")
    va = _need_heads(v, "v", k.shape)
    B = 1
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1, min_numel=1)
        B = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    oa = _need_heads(out, "out", q.shape)
    _on_one_device(q.get_device(), q=q, k=k, v=v, cu_seqlens=cu_seqlens, out=out)
    _launch("svdq_attention_packed", q.device, *qa, *ka, *va, _p(cu_seqlens), B, T, H, Hk, D, 1 if causal else 0,
            scale if scale is not None else D ** -0.5 if D > 0 else 1.0, *oa)   # D = 0 is refused there
    return out
