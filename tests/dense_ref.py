"""Plain 64-bit statements of the dense operators (test references, torch on any device)
and the error bounds their 32-bit kernels are held to."""

from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24  # half a step of an f32 value, relative
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def half_step(dtype) -> float:
    """Relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


def floor_of(dtype) -> float:
    """Absolute error of one rounding among the subnormals."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def rms(v, eps):
    return torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def block_norm(z, r, w, g, a, v, eps, store=None):
    """(s, y); `store` rounds the stream as it is kept."""
    n = z if w is None else z / rms(z, eps) * w
    s = n if g is None else g * n
    if r is not None:
        s = a * r + s
    kept = s if store is None else store(s)
    return s, None if v is None else kept / rms(kept, eps) * v


def block_norm_grads(ds, dy, z, s, w, g, a, v, eps):
    """Values and magnitudes (the sums with every term taken absolute) of the gradients."""
    out, mag = {}, {}
    d = torch.zeros_like(z) if ds is None else ds
    D = d.abs()
    if v is not None:
        rs, u = 1 / rms(s, eps), dy * v
        d = d + rs * u - s * rs ** 3 * (u * s).mean(1, keepdim=True)
        D = D + rs * u.abs() + s.abs() * rs ** 3 * (u * s).abs().mean(1, keepdim=True)
        out["next_weight"], mag["next_weight"] = (dy * s * rs).sum(0), (dy * s * rs).abs().sum(0)
    out["residual"], mag["residual"] = a * d, abs(a) * D
    rz = 1 / rms(z, eps) if w is not None else torch.ones_like(z[:, :1])
    wv = w if w is not None else torch.ones_like(z[0])
    p, P = (d, D) if g is None else (d * g, D * g.abs())
    if g is not None:
        dg, DG = d * z * rz * wv, D * (z * rz * wv).abs()
        if g.dim() == 1:
            dg, DG = dg.sum(0), DG.sum(0)
        elif g.shape[1] == 1:
            dg, DG = dg.sum(1, keepdim=True), DG.sum(1, keepdim=True)
        out["gate"], mag["gate"] = dg, DG
    q, Q = p * wv, P * wv.abs()
    if w is not None:
        out["norm_weight"], mag["norm_weight"] = (p * z * rz).sum(0), (P * (z * rz).abs()).sum(0)
        out["block"] = rz * q - z * rz ** 3 * (q * z).mean(1, keepdim=True)
        mag["block"] = rz * Q + z.abs() * rz ** 3 * (Q * z.abs()).mean(1, keepdim=True)
    else:
        out["block"], mag["block"] = q, Q
    return out, mag


def act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def dequantise(codes, scales):
    """MXFP4 [rows, K/2] codes and [rows, K/32] scales -> f64 [rows, K]."""
    mag = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    c = codes.long()
    w = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for odd in (0, 1):
        v = (c >> (4 * odd)) & 15
        w[:, odd::2] = mag[v & 7] * (1 - 2 * (v >> 3)).double()
    return w * torch.pow(2.0, scales.double().repeat_interleave(32, 1) - 127)


def within(got, ref, tol):
    """Assert |got - ref| <= tol element by element, saying where it fails.  A value past
    its type's largest by half a step or more rounds to infinity."""
    top = torch.finfo(got.dtype).max * (1 + torch.finfo(got.dtype).eps / 4)
    got, ref = got.double(), ref.double()
    bad = (got - ref).abs() > tol
    bad |= torch.isfinite(ref) != torch.isfinite(got)
    beyond = torch.isfinite(ref) & (ref.abs() + tol >= top) & (got == torch.sign(ref) * float("inf"))
    bad &= ~beyond
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        g, r = got.flatten()[i].item(), ref.flatten()[i].item()
        t = tol.expand_as(ref).flatten()[i].item() if isinstance(tol, torch.Tensor) else tol
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {i}: {g} for {r}, tolerance {t}")
