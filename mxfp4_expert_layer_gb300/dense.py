"""Torch-facing wrappers of the dense operators around the expert layer: the norms
before and after a block, the gated feed-forward block, and products of a few tokens
with MXFP4 weights.

    s, y = block_norm(z, r, norm_weight=wp, gate=g, residual_scale=a, next_weight=wn)
    grads = block_norm_backward(ds, dy, z, s, norm_weight=wp, gate=g, residual_scale=a, next_weight=wn)
    out, gu = ffn_forward(x, w_gateup, w_down, save=True)
    d_x, d_w_gateup, d_w_down = ffn_backward(d_out, x, gu, w_gateup, w_down)
    gateup = MatvecMXFP4(codes, scales, kind=MOE_WEIGHTS_GATEUP)
    h = gateup(x)                       # x [T <= 64, K] -> silu(gate) * up, [T, rows / 2]

Gradients are explicit calls; nothing here registers with autograd.  Every call runs on
the current stream of its tensors' device, takes its workspace from torch's allocator
(so calls on other streams and captured graphs never share one) and keeps no state.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib as L

_DTYPES = {torch.bfloat16: L.MOE_DTYPE_BF16, torch.float16: L.MOE_DTYPE_F16, torch.float32: L.MOE_DTYPE_F32}


class _Library:
    """The library's functions, looked up once each."""

    def __getattr__(self, name):
        fn = getattr(L.load(), name)
        setattr(self, name, fn)
        return fn


_C = _Library()
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _dtype16(t: torch.Tensor) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None or d == L.MOE_DTYPE_F32:
        raise ValueError(f"bf16 or f16 tensors are needed, got {t.dtype}")
    return d


def _need(name: str, t: Optional[torch.Tensor], shape, dtype, device) -> Optional[int]:
    """The address of a contiguous tensor of this shape, type and device (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on {device} is needed, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _call(device: torch.device, fn, *args) -> None:
    """One library call on the current stream of `device`, with it current."""
    if device.type != "cuda":
        raise ValueError("CUDA tensors are needed")
    index = device.index
    if index == _current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        raise L.MoEError(fn.__name__, st)


@functools.lru_cache(maxsize=None)
def _ffn_bytes(T: int, H: int, I: int, backward: int) -> int:
    return _C.moe_ffn_workspace_bytes(T, H, I, backward)


@functools.lru_cache(maxsize=None)
def _matvec_bytes(T: int, K: int) -> int:
    return _C.moe_matvec_workspace_bytes(T, K)


@functools.lru_cache(maxsize=None)
def _norm_bytes(T: int, H: int) -> int:
    return _C.moe_block_norm_workspace_bytes(T, H)


# ------------------------------------------------------------------ norms around a block
def _gate(gate: Optional[torch.Tensor], T: int, H: int, dtype, device) -> Tuple[int, Optional[int]]:
    if gate is None:
        return L.MOE_GATE_NONE, None
    if gate.dim() == 1:
        return L.MOE_GATE_FEATURE, _need("gate", gate, (H,), dtype, device)
    if gate.shape == (T, 1):
        return L.MOE_GATE_TOKEN, _need("gate", gate, (T, 1), torch.float32, device)
    return L.MOE_GATE_FULL, _need("gate", gate, (T, H), dtype, device)


def block_norm(block: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
               norm_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               residual_scale: float = 1.0, next_weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
               residual_out: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """s = residual_scale * residual + gate * RMSNorm(block) and out = RMSNorm(s)
    (moe_block_norm); returns (s, out), out None without ``next_weight``.

    block [T, H] bf16 or f16; ``residual`` of the same type or f32 (the type of s);
    ``norm_weight`` None: no norm after the block; ``gate``: None, [H] or [T, H] of
    block's type, or f32 [T, 1].  ``residual_out`` may be ``residual``."""
    T, H = block.shape
    dt, dev = block.dtype, block.device
    code = _dtype16(block)
    sdt = residual.dtype if residual is not None else residual_out.dtype if residual_out is not None else dt
    if sdt != dt and sdt != torch.float32:
        raise ValueError(f"the residual stream is {dt} or float32, got {sdt}")
    kind, gate_ptr = _gate(gate, T, H, dt, dev)
    if residual_out is None:
        residual_out = torch.empty_like(block, dtype=sdt)
    if next_weight is None:
        if out is not None:
            raise ValueError("out needs next_weight")
    elif out is None:
        out = torch.empty_like(block)
    _call(dev, _C.moe_block_norm, _need("block", block, (T, H), dt, dev),
          _need("norm_weight", norm_weight, (H,), dt, dev), gate_ptr, kind, _need("residual", residual, (T, H), sdt, dev),
          residual_scale, _need("next_weight", next_weight, (H,), dt, dev), eps, T, H, code, _DTYPES[sdt],
          _need("residual_out", residual_out, (T, H), sdt, dev), _need("out", out, (T, H), dt, dev))
    return residual_out, out


class BlockNormGrads(NamedTuple):
    """Gradients of block_norm; None for an argument that the call did not have."""
    block: torch.Tensor
    residual: Optional[torch.Tensor]
    norm_weight: Optional[torch.Tensor]   # f32 [H]
    gate: Optional[torch.Tensor]          # f32 [H], f32 [T, 1], or [T, H] of the gate's type
    next_weight: Optional[torch.Tensor]   # f32 [H]


def block_norm_backward(d_residual_out: Optional[torch.Tensor], d_out: Optional[torch.Tensor], block: torch.Tensor,
                        residual_out: Optional[torch.Tensor] = None, *, norm_weight: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                        next_weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
                        has_residual: bool = True) -> BlockNormGrads:
    """Every gradient of block_norm (moe_block_norm_backward).  ``residual_out`` is the s
    that the forward returned; ``d_residual_out`` and ``d_out`` the gradients of its two
    results (None for one that nothing read); ``has_residual`` False: no residual was added."""
    T, H = block.shape
    dt, dev = block.dtype, block.device
    code = _dtype16(block)
    like = d_residual_out if d_residual_out is not None else residual_out
    sdt = like.dtype if like is not None else dt
    if sdt != dt and sdt != torch.float32:
        raise ValueError(f"the residual stream is {dt} or float32, got {sdt}")
    kind, gate_ptr = _gate(gate, T, H, dt, dev)
    nbytes = _norm_bytes(T, H)
    if nbytes == 0:
        raise L.MoEError("moe_block_norm_backward", L.MOE_ERR_UNSUPPORTED_SHAPE)
    d_block = torch.empty_like(block)
    d_residual = torch.empty(block.shape, dtype=sdt, device=dev) if has_residual else None
    f32 = dict(dtype=torch.float32, device=dev)
    d_norm = torch.empty(H, **f32) if norm_weight is not None else None
    d_next = torch.empty(H, **f32) if next_weight is not None else None
    if gate is None:
        d_gate = None
    else:
        d_gate = torch.empty_like(gate) if kind == L.MOE_GATE_FULL else torch.empty(gate.shape, **f32)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call(dev, _C.moe_block_norm_backward, _need("d_residual_out", d_residual_out, (T, H), sdt, dev),
          _need("d_out", d_out, (T, H), dt, dev), _need("block", block, (T, H), dt, dev),
          _need("norm_weight", norm_weight, (H,), dt, dev), gate_ptr, kind,
          _need("residual_out", residual_out, (T, H), sdt, dev), residual_scale,
          _need("next_weight", next_weight, (H,), dt, dev), eps, T, H, code, _DTYPES[sdt], d_block.data_ptr(),
          None if d_residual is None else d_residual.data_ptr(), None if d_norm is None else d_norm.data_ptr(),
          None if d_gate is None else d_gate.data_ptr(), None if d_next is None else d_next.data_ptr(), ws.data_ptr(),
          nbytes)
    return BlockNormGrads(d_block, d_residual, d_norm, d_gate, d_next)


# ------------------------------------------------------------------ gated feed-forward block
def _ffn_shape(x: torch.Tensor, w_gateup: torch.Tensor) -> Tuple[int, int, int]:
    T, H = x.shape
    return T, H, w_gateup.shape[0] // 2


def ffn_forward(x: torch.Tensor, w_gateup: torch.Tensor, w_down: torch.Tensor, *, act: int = L.MOE_ACT_SILU,
                save: bool = False, out: Optional[torch.Tensor] = None):
    """out = (act(x W_gate^T) * (x W_up^T)) W_down^T (moe_ffn_forward): x [T, H],
    w_gateup [2I, H] (gate rows, then up rows) and w_down [H, I], all bf16 or all f16.
    With ``save``, (out, gateup): the products before the activation, f32 [T, 2I], for
    ffn_backward."""
    T, H, I = _ffn_shape(x, w_gateup)
    code, dt, dev = _dtype16(x), x.dtype, x.device
    nbytes = _ffn_bytes(T, H, I, 0)
    if nbytes == 0:
        raise L.MoEError("moe_ffn_forward", L.MOE_ERR_UNSUPPORTED_SHAPE)
    if out is None:
        out = torch.empty(T, H, dtype=dt, device=dev)
    gateup = torch.empty(T, 2 * I, dtype=torch.float32, device=dev) if save else None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call(dev, _C.moe_ffn_forward, _need("x", x, (T, H), dt, dev), _need("w_gateup", w_gateup, (2 * I, H), dt, dev),
          _need("w_down", w_down, (H, I), dt, dev), T, H, I, act, code, None if gateup is None else gateup.data_ptr(),
          _need("out", out, (T, H), dt, dev), ws.data_ptr(), nbytes)
    return (out, gateup) if save else out


class FfnGrads(NamedTuple):
    """Gradients of ffn_forward; None for one that was not asked for."""
    x: Optional[torch.Tensor]          # [T, H]
    w_gateup: Optional[torch.Tensor]   # [2I, H]
    w_down: Optional[torch.Tensor]     # [H, I]


def ffn_backward(d_out: torch.Tensor, x: torch.Tensor, gateup: torch.Tensor, w_gateup: torch.Tensor,
                 w_down: torch.Tensor, *, act: int = L.MOE_ACT_SILU, need_x: bool = True,
                 need_weights: bool = True) -> FfnGrads:
    """The gradients of ffn_forward (moe_ffn_backward) from its inputs, the ``gateup`` it
    saved and ``act`` as given there; all of x's type."""
    T, H, I = _ffn_shape(x, w_gateup)
    code, dt, dev = _dtype16(x), x.dtype, x.device
    nbytes = _ffn_bytes(T, H, I, 1)
    if nbytes == 0:
        raise L.MoEError("moe_ffn_backward", L.MOE_ERR_UNSUPPORTED_SHAPE)
    d_x = torch.empty(T, H, dtype=dt, device=dev) if need_x else None
    d_wgu = torch.empty(2 * I, H, dtype=dt, device=dev) if need_weights else None
    d_wd = torch.empty(H, I, dtype=dt, device=dev) if need_weights else None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call(dev, _C.moe_ffn_backward, _need("d_out", d_out, (T, H), dt, dev), _need("x", x, (T, H), dt, dev),
          _need("gateup", gateup, (T, 2 * I), torch.float32, dev), _need("w_gateup", w_gateup, (2 * I, H), dt, dev),
          _need("w_down", w_down, (H, I), dt, dev), T, H, I, act, code, None if d_x is None else d_x.data_ptr(),
          None if d_wgu is None else d_wgu.data_ptr(), None if d_wd is None else d_wd.data_ptr(), ws.data_ptr(), nbytes)
    return FfnGrads(d_x, d_wgu, d_wd)


def dense_status() -> int:
    """The feed-forward GEMMs' device status word on the current device (0 = healthy), read
    after the current stream and cleared (moe_dense_status)."""
    st = ctypes.c_int(0)
    rc = _C.moe_dense_status(ctypes.byref(st), torch.cuda.current_stream().cuda_stream)
    if rc not in (L.MOE_OK, L.MOE_ERR_DEVICE_TIMEOUT):
        raise L.MoEError("moe_dense_status", rc)
    return st.value


# ------------------------------------------------------------------ a few tokens x MXFP4 weights
class MatvecMXFP4:
    """MXFP4 weights [rows, K] laid out once for products of 1 to 64 tokens
    (moe_prepare_matvec, moe_matvec_mxfp4): codes uint8 [rows, K/2], scales uint8
    [rows, K/32].  kind MOE_WEIGHTS_DOWN: y = x W^T + bias, [T, rows].  kind
    MOE_WEIGHTS_GATEUP: act(gate) * up of the gate rows [0, rows/2) and the up rows,
    [T, rows/2].  ``bias``: f32 [rows] or None."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, kind: int = L.MOE_WEIGHTS_DOWN,
                 bias: Optional[torch.Tensor] = None, act: int = L.MOE_ACT_SILU):
        rows, half = codes.shape
        self.rows, self.K, self.kind, self.act, self.bias = rows, 2 * half, kind, act, bias
        dev = codes.device
        nbytes = _C.moe_prepared_matvec_bytes(rows, self.K, kind)
        if nbytes == 0:
            raise L.MoEError("moe_prepare_matvec", L.MOE_ERR_UNSUPPORTED_SHAPE)
        _need("bias", bias, (rows,), torch.float32, dev)
        self.n_out = rows // 2 if kind == L.MOE_WEIGHTS_GATEUP else rows
        self.weight = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _call(dev, _C.moe_prepare_matvec, _need("codes", codes, (rows, half), torch.uint8, dev),
              _need("scales", scales, (rows, self.K // 32), torch.uint8, dev), rows, self.K, kind,
              self.weight.data_ptr(), nbytes)

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        T = x.shape[0]
        code = _dtype16(x)
        dev = self.weight.device
        if out is None:
            out = torch.empty(T, self.n_out, dtype=x.dtype, device=dev)
        bias = self.bias
        nbytes = _matvec_bytes(T, self.K)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        _call(dev, _C.moe_matvec_mxfp4, _need("x", x, (T, self.K), x.dtype, dev), self.weight.data_ptr(),
              None if bias is None else bias.data_ptr(), T, self.rows, self.K, self.kind, self.act, code,
              _need("out", out, (T, self.n_out), x.dtype, dev), None if ws is None else ws.data_ptr(), nbytes)
        return out

    __call__ = forward
