"""Torch-facing wrappers of the dense operators around the expert layer: the norms
before and after a block, the gated feed-forward block, projections with bias, activation
and residual, tokens sorted by expert and back, and products of a few tokens with MXFP4 weights.

    s, y = block_norm(z, r, norm_weight=wp, gate=g, residual_scale=a, next_weight=wn)
    s, codes, scales, y = block_norm_8bit(z, r, norm_weight=wp, gate=g, residual_scale=a, next_weight=wn, with_out=True)
    grads = block_norm_backward(ds, dy, z, s, norm_weight=wp, gate=g, residual_scale=a, next_weight=wn)
    out, gu = ffn_forward(x, w_gateup, w_down, save=True)
    d_x, d_w_gateup, d_w_down = ffn_backward(d_out, x, gu, w_gateup, w_down)
    out, pre = linear_forward(x, weight, bias, residual, act=MOE_ACT_GELU, save=True)
    d_x, d_weight, d_bias = linear_backward(d_out, x, weight, pre, act=MOE_ACT_GELU)
    s = sort_tokens(x, topk_idx, E)     # s.rows: x by expert; experts of one's own give y [T*k, H]
    out = unsort_tokens(y, s.inv_perm, topk_w)
    d_y, d_topk_w = unsort_tokens_backward(d_out, y, s.inv_perm, topk_w)
    d_logits = route_backward(d_topk_w, logits, topk_idx, topk_w)
    d_x = sort_tokens_backward(d_rows, s.inv_perm)
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


class BlockNorm8(NamedTuple):
    """What block_norm_8bit returns; small results share a storage."""
    residual: torch.Tensor            # s [T, H]
    codes: torch.Tensor               # float8_e4m3fn [T, H]: out / scale
    scales: torch.Tensor              # "mx": float8_e8m0fnu [T, H / 32]; "row": f32 [T, 1]
    out: Optional[torch.Tensor]       # [T, H] of block's type, with ``with_out``


_SCALES = {"mx": L.MOE_SCALE_MX, "row": L.MOE_SCALE_ROW}


def block_norm_8bit(block: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                    norm_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                    residual_scale: float = 1.0, next_weight: torch.Tensor, eps: float = 1e-5, scales: str = "mx",
                    with_out: bool = False) -> BlockNorm8:
    """block_norm with out in 8 bits (moe_block_norm_8bit): E4M3 codes, and scales that are powers
    of two for 32 values each ("mx", H a multiple of 32) or one for a row ("row").  codes and
    scales are as sort_tokens takes them.  ``with_out``: out in block's type as well.  Its
    gradients are block_norm_backward's, the rounding passing d_out through."""
    if scales not in _SCALES:
        raise ValueError(f'scales: "mx" or "row", got {scales!r}')
    return BlockNorm8._make(_ext.block_norm_8bit(block, residual, norm_weight, gate, residual_scale, next_weight, eps,
                                                 _SCALES[scales], with_out))


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


# ------------------------------------------------------------------ projections
def linear_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, *, act: int = L.MOE_ACT_NONE,
                   out_dtype: Optional[torch.dtype] = None, save: bool = False, out: Optional[torch.Tensor] = None):
    """out = act(x W^T + bias) + residual (moe_linear_forward): x [T, K] and weight [N, K] bf16
    or f16, ``bias`` f32 [N]; ``residual`` and out [T, N] of x's type or f32 (``out_dtype``, or
    as the residual is).  ``out`` may be ``residual``.  With ``save``, (out, pre): what the
    activation was taken of, f32 [T, N], for linear_backward (None without an activation)."""
    if out_dtype is not None and out_dtype not in (x.dtype, torch.float32):
        raise ValueError(f"out_dtype: x's type or float32, got {out_dtype}")
    wide = None if out_dtype is None else out_dtype == torch.float32
    r = _ext.linear_forward(x, weight, bias, residual, act, wide, save, out)
    return r if save else r[0]


class LinearGrads(NamedTuple):
    """Gradients of linear_forward; None for one that was not asked for.  The residual's is d_out."""
    x: Optional[torch.Tensor]        # [T, K]
    weight: Optional[torch.Tensor]   # [N, K]
    bias: Optional[torch.Tensor]     # f32 [N]


def linear_backward(d_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, pre: Optional[torch.Tensor] = None, *,
                    act: int = L.MOE_ACT_NONE, need_x: bool = True, need_weight: bool = True,
                    need_bias: bool = True) -> LinearGrads:
    """The gradients of linear_forward (moe_linear_backward) from its inputs, the ``pre`` it
    saved and ``act`` as given there; d_out [T, N] of the type that out had."""
    return LinearGrads._make(_ext.linear_backward(d_out, x, weight, pre, act, need_x, need_weight, need_bias))


# ------------------------------------------------------------------ tokens sorted by expert
class SortedTokens(NamedTuple):
    """Token rows in expert order.  The three integer arrays share a storage, where the rows are
    small (64 KB) with them."""
    rows: torch.Tensor                # [T*k, H]: by expert, then by token; what was dropped comes last, as zeros
    scales: Optional[torch.Tensor]    # [T*k, S]: the rows' scales
    offsets: torch.Tensor             # i32 [E + 1]: rows of expert e are [offsets[e], offsets[e + 1])
    perm: torch.Tensor                # i32 [T*k]: assignment t*k + j of each row; -1 - it where dropped
    inv_perm: torch.Tensor            # i32 [T, k]: row of each assignment; -1 - it where dropped


def sort_tokens(x: torch.Tensor, topk_idx: torch.Tensor, n_experts: int, *,
                scales: Optional[torch.Tensor] = None) -> SortedTokens:
    """The rows of x [T, H] (any type, rows of a multiple of 16 bytes) in the order of the
    experts that topk_idx (i32 [T, k]) names (moe_sort_tokens).  An index outside
    [0, n_experts) drops its assignment.  ``scales`` [T, S] go with their rows."""
    return SortedTokens._make(_ext.sort_tokens(x, topk_idx, n_experts, scales))


def sort_tokens_backward(d_rows: torch.Tensor, inv_perm: torch.Tensor,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """d_x [T, H], the gradient of sort_tokens: each token's rows of d_rows [T*k, H] (bf16, f16
    or f32) summed (moe_unsort_tokens)."""
    return _ext.sort_tokens_backward(d_rows, inv_perm, out)


def unsort_tokens(y: torch.Tensor, inv_perm: torch.Tensor, topk_w: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum_j topk_w[t, j] * y[inv_perm[t, j]] over the j that were not dropped
    (moe_unsort_tokens): y [T*k, H] bf16, f16 or f32 in the order of sort_tokens, topk_w
    f32 [T, k] (None: 1).  ``out`` may not overlap an input."""
    return _ext.unsort_tokens(y, inv_perm, topk_w, out)


class UnsortGrads(NamedTuple):
    """Gradients of unsort_tokens; None for one that was not asked for.  Small ones share a storage."""
    y: Optional[torch.Tensor]         # [T*k, H]; 0 in the rows of what was dropped
    topk_w: Optional[torch.Tensor]    # f32 [T, k]; 0 where dropped


def unsort_tokens_backward(d_out: torch.Tensor, y: Optional[torch.Tensor], inv_perm: torch.Tensor,
                           topk_w: Optional[torch.Tensor] = None, *, need_y: bool = True,
                           need_w: bool = True) -> UnsortGrads:
    """The gradients of unsort_tokens from its arguments (moe_unsort_tokens_backward); without
    ``need_w``, y may be None."""
    return UnsortGrads._make(_ext.unsort_tokens_backward(d_out, y, inv_perm, topk_w, need_y, need_w))


def route_backward(d_topk_w: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor, *,
                   gating: int = 0) -> torch.Tensor:
    """d_logits f32 [T, E] from the gradient of route's weights and what route returned
    (moe_route_backward): the indices as routed, before any were dropped."""
    return _ext.route_backward(d_topk_w, logits, topk_idx, topk_w, gating)


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
