"""Torch-facing wrappers of the dense operators around the expert layer: the norms
before and after a block, the gated feed-forward block, and products of a few tokens
with MXFP4 weights.

    s, y = block_norm(z, r, norm_weight=wp, gate=g, residual_scale=a, next_weight=wn)
    grads = block_norm_backward(ds, dy, z, s, norm_weight=wp, gate=g, residual_scale=a, next_weight=wn)
    out, gu = ffn_forward(x, w_gateup, w_down, save=True)
    d_x, d_w_gateup, d_w_down = ffn_backward(d_out, x, gu, w_gateup, w_down)
    gateup = MatvecMXFP4(codes, scales, kind=MOE_WEIGHTS_GATEUP)
    h = gateup(x)                       # x [T <= 64, K] -> silu(gate) * up, [T, rows / 2]

Gradients are explicit calls; nothing here registers with autograd.  Where autograd
records, a tensor that requires grad is therefore refused (of a backward call: an incoming
gradient that does); under ``torch.no_grad()`` it is as any other.  Every call runs on the
current stream of its tensors' device, takes its workspace from torch's allocator (so calls
on other streams and captured graphs never share one) and keeps no state; the checks and
allocations are native (csrc/dense_binding.cpp).
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib as L
from .build import EXT_PATH


def _load_ext():
    """The native binding (raises if it was never built)."""
    L.load()
    if not os.path.exists(EXT_PATH):
        raise RuntimeError(f"{EXT_PATH} is missing: build it with mxfp4_expert_layer_gb300.build.build()")
    spec = importlib.util.spec_from_file_location(__package__ + "._dense_ext", EXT_PATH)
    ext = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ext)
    ext.set_error(L.MoEError)
    return ext


_ext = _load_ext()


# ------------------------------------------------------------------ norms around a block
def block_norm(block: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
               norm_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               residual_scale: float = 1.0, next_weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
               residual_out: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """s = residual_scale * residual + gate * RMSNorm(block) and out = RMSNorm(s)
    (moe_block_norm); returns (s, out), out None without ``next_weight``.

    block [T, H] bf16 or f16; ``residual`` of the same type or f32 (the type of s);
    ``norm_weight`` None: no norm after the block; ``gate``: None, [H] or [T, H] of
    block's type, or f32 [T, 1].  ``residual_out`` may be ``residual``, ``out`` may be
    ``block``.  Small results of one type share a storage."""
    return _ext.block_norm(block, residual, norm_weight, gate, residual_scale, next_weight, eps, residual_out, out)


class BlockNormGrads(NamedTuple):
    """Gradients of block_norm; None for an argument that the call did not have.  The f32 [H]
    ones share a storage (3 H values at most)."""
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
    return BlockNormGrads._make(_ext.block_norm_backward(d_residual_out, d_out, block, residual_out, norm_weight, gate,
                                                         residual_scale, next_weight, eps, has_residual))


# ------------------------------------------------------------------ gated feed-forward block
def ffn_forward(x: torch.Tensor, w_gateup: torch.Tensor, w_down: torch.Tensor, *, act: int = L.MOE_ACT_SILU,
                save: bool = False, out: Optional[torch.Tensor] = None):
    """out = (act(x W_gate^T) * (x W_up^T)) W_down^T (moe_ffn_forward): x [T, H],
    w_gateup [2I, H] (gate rows, then up rows) and w_down [H, I], all bf16 or all f16.
    ``out`` may be ``x``.  With ``save``, (out, gateup): the products before the activation,
    f32 [T, 2I], for ffn_backward, which needs x as it was."""
    r = _ext.ffn_forward(x, w_gateup, w_down, act, save, out)
    return r if save else r[0]


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
    return FfnGrads._make(_ext.ffn_backward(d_out, x, gateup, w_gateup, w_down, act, need_x, need_weights))


def dense_status() -> int:
    """The dense operators' device status words on the current device, as one (0 = healthy),
    read after the current stream and cleared (moe_dense_status)."""
    st = ctypes.c_int(0)
    rc = L.moe_dense_status(ctypes.byref(st), torch.cuda.current_stream().cuda_stream)
    if rc not in (L.MOE_OK, L.MOE_ERR_DEVICE_TIMEOUT):
        raise L.MoEError("moe_dense_status", rc)
    return st.value


# ------------------------------------------------------------------ a few tokens x MXFP4 weights
class MatvecMXFP4:
    """MXFP4 weights [rows, K] laid out once for products of 1 to 64 tokens
    (moe_prepare_matvec, moe_matvec_mxfp4): codes uint8 [rows, K/2], scales uint8
    [rows, K/32].  kind MOE_WEIGHTS_DOWN: y = x W^T + bias, [T, rows].  kind
    MOE_WEIGHTS_GATEUP: act(gate) * up of the gate rows [0, rows/2) and the up rows,
    [T, rows/2].  ``bias``: f32 [rows] or None.  ``out`` may not overlap ``x``."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, kind: int = L.MOE_WEIGHTS_DOWN,
                 bias: Optional[torch.Tensor] = None, act: int = L.MOE_ACT_SILU):
        rows, half = codes.shape
        self.rows, self.K, self.kind, self.act, self.bias = rows, 2 * half, kind, act, bias
        dev = codes.device
        nbytes = L.moe_prepared_matvec_bytes(rows, self.K, kind)
        if nbytes == 0:
            raise L.MoEError("moe_prepare_matvec", L.MOE_ERR_UNSUPPORTED_SHAPE)
        for name, t, shape, dtype in (("codes", codes, (rows, half), torch.uint8),
                                      ("scales", scales, (rows, half // 16), torch.uint8),
                                      ("bias", bias, (rows,), torch.float32)):
            if t is not None and (t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_cuda
                                  or not t.is_contiguous()):
                raise ValueError(f"{name}: a contiguous {dtype} CUDA tensor of shape {shape} is needed")
        self.weight = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        with torch.cuda.device(dev):
            L.check("moe_prepare_matvec", L.moe_prepare_matvec(codes.data_ptr(), scales.data_ptr(), rows, self.K, kind,
                                                               self.weight.data_ptr(), nbytes,
                                                               torch.cuda.current_stream().cuda_stream))

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        return _ext.matvec(x, self.weight, self.bias, self.rows, self.K, self.kind, self.act, out)

    __call__ = forward
