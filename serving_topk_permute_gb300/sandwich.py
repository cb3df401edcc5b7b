"""Binding of the sandwich norm (include/moe.h): a block's post-norm, gate, scaled residual and the next
block's pre-norm in one pass, and its gradient. Argument checks and marshalling only, as in block.py.
"""
from __future__ import annotations

import ctypes
from ctypes import byref
from typing import NamedTuple

import torch

from . import block
from .block import (F32, I32, I64, P, SZ, Quantized, _at_device, _current_device, _device_of, _fail, _flat, _matrix,
                    _on, _row_stride, _stream)
from .moe import MOE_OK

GATES = {"none": 0, "token": 1, "channel": 2}

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8


class SandwichC(ctypes.Structure):
    _fields_ = [("gamma_post", P), ("gamma_pre", P), ("gate", P), ("gate_kind", I32), ("residual_scale", F32),
                ("eps", F32)]


_lib = block.declare({
    "moe_sandwich_norm": [I32, I32, P, P, I64, P, I64, P, I64, P, I64, P, P, P],
    "moe_sandwich_norm_workspace_size": [I32, I32, P],
    "moe_sandwich_norm_backward": [I32, I32, P, P, I64, P, I64, P, P, I64, P, I64, P, I64, P, I64, P, P, P, P, SZ, P],
})


def _params(shape, dev: int, gamma_post, gamma_pre, gate, gate_kind, alpha: float, eps: float) -> SandwichC:
    """The library's argument. A gate's kind follows from its length, unless rows and H agree."""
    rows, H = shape
    _flat("gamma_post", gamma_post, _F32, H, dev)
    _flat("gamma_pre", gamma_pre, _F32, H, dev)
    if gate is None:
        if gate_kind not in (None, "none"):
            raise ValueError(f"a gate of kind {gate_kind!r} must be given")
        return SandwichC(gamma_post.data_ptr(), gamma_pre.data_ptr(), None, 0, alpha, eps)
    if gate_kind is None:
        n = gate.numel()
        if n == rows and n == H:
            raise ValueError(f"a gate of {n} elements may be one for each token or each channel here: give gate_kind")
        gate_kind = "token" if n == rows else "channel"
    if gate_kind not in ("token", "channel"):
        raise ValueError(f"gate_kind must be 'token' or 'channel', got {gate_kind!r}")
    _flat("gate", gate, _F32, rows if gate_kind == "token" else H, dev)
    return SandwichC(gamma_post.data_ptr(), gamma_pre.data_ptr(), gate.data_ptr(), GATES[gate_kind], alpha, eps)


def sandwich_norm(f: torch.Tensor, residual: torch.Tensor, gamma_post: torch.Tensor, gamma_pre: torch.Tensor,
                  gate: torch.Tensor | None = None, gate_kind: str | None = None, alpha: float = 1.0,
                  eps: float = 1e-6, sum_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  quantized: Quantized | None = None, stats: torch.Tensor | None = None, stream=None):
    """moe_sandwich_norm: z = alpha residual + gate gamma_post f / rms(f), h = gamma_pre z / rms(z).

    f (the block's output), residual, sum_out (receives z), out (receives h): bf16 [rows, H]; gammas: fp32 [H];
    gate: fp32 [rows] or [H] (gate_kind "token" or "channel" says which where rows == H); quantized: receives h in
    its format; stats: fp32 [rows, 2], receives what the backward pass needs. Without out and quantized, out is
    allocated. Returns out if there is one, else quantized."""
    shape = _matrix("f", f)
    rows, H = shape
    dev = _device_of("f", f)
    ldf = _row_stride("f", f, _BF16, shape, dev)
    ldr = _row_stride("residual", residual, _BF16, shape, dev)
    c = _params(shape, dev, gamma_post, gamma_pre, gate, gate_kind, alpha, eps)
    if out is None and quantized is None:
        with _on(stream):
            out = torch.empty((rows, H), dtype=_BF16, device=f.device)
    po = ps = pq = pt = None
    ldo = lds = 0
    if out is not None:
        ldo = _row_stride("out", out, _BF16, shape, dev)
        po = out.data_ptr()
    if sum_out is not None:
        lds = _row_stride("sum_out", sum_out, _BF16, shape, dev)
        ps = sum_out.data_ptr()
    if quantized is not None:
        if quantized.shape != shape:
            raise ValueError(f"quantized holds {quantized.shape}, f is {tuple(shape)}")
        pq = quantized._arg(dev)
    if stats is not None:
        _flat("stats", stats, _F32, 2 * rows, dev)
        pt = stats.data_ptr()
    fn = _lib().moe_sandwich_norm
    call = fn if dev == _current_device() else _at_device(fn, dev)
    st = call(rows, H, byref(c), f.data_ptr(), ldf, residual.data_ptr(), ldr, ps, lds, po, ldo, pq, pt,
              _stream(stream, dev))
    if st:
        _fail("moe_sandwich_norm", st)
    return out if out is not None else quantized


def sandwich_norm_workspace_size(rows: int, hidden: int) -> int:
    """Bytes of the backward pass's workspace."""
    n = SZ()
    st = _lib().moe_sandwich_norm_workspace_size(rows, hidden, byref(n))
    if st != MOE_OK:
        _fail("moe_sandwich_norm_workspace_size", st)
    return n.value


class SandwichGrads(NamedTuple):
    """Gradients of a sandwich norm: f and residual bf16 [rows, H], gate fp32 [rows] or [H] (None without a gate),
    gammas fp32 [H]."""
    f: torch.Tensor
    residual: torch.Tensor
    gate: torch.Tensor | None
    gamma_post: torch.Tensor | None
    gamma_pre: torch.Tensor | None


def sandwich_norm_backward(f: torch.Tensor, residual: torch.Tensor, gamma_post: torch.Tensor, gamma_pre: torch.Tensor,
                           stats: torch.Tensor, gate: torch.Tensor | None = None, gate_kind: str | None = None,
                           alpha: float = 1.0, d_sum: torch.Tensor | None = None, d_out: torch.Tensor | None = None,
                           d_f: torch.Tensor | None = None, d_residual: torch.Tensor | None = None,
                           gammas: bool = True, workspace: torch.Tensor | None = None, stream=None) -> SandwichGrads:
    """The gradients of sum(d_sum z) + sum(d_out h). f, residual, gammas, gate and alpha as sandwich_norm had them,
    stats as it wrote them; d_sum and d_out bf16 [rows, H], one of them may be None. d_f and d_residual are written
    if given (each may be d_sum or d_out), else allocated. gammas=False leaves the gammas' gradients out (and a
    channel gate's)."""
    shape = _matrix("f", f)
    rows, H = shape
    dev = _device_of("f", f)
    ldf = _row_stride("f", f, _BF16, shape, dev)
    ldr = _row_stride("residual", residual, _BF16, shape, dev)
    c = _params(shape, dev, gamma_post, gamma_pre, gate, gate_kind, alpha, 0.0)
    _flat("stats", stats, _F32, 2 * rows, dev)
    ps = po = None
    lds = ldo = 0
    if d_sum is not None:
        lds = _row_stride("d_sum", d_sum, _BF16, shape, dev)
        ps = d_sum.data_ptr()
    if d_out is not None:
        ldo = _row_stride("d_out", d_out, _BF16, shape, dev)
        po = d_out.data_ptr()
    if ps is None and po is None:
        raise ValueError("one of d_sum and d_out must be given")
    empty, device = torch.empty, f.device
    d_gate = d_post = d_pre = None
    with _on(stream):
        if d_f is None:
            d_f = empty((rows, H), dtype=_BF16, device=device)
        if d_residual is None:
            d_residual = empty((rows, H), dtype=_BF16, device=device)
        if gammas:
            d_post, d_pre = empty(H, dtype=_F32, device=device), empty(H, dtype=_F32, device=device)
        if c.gate_kind == 1 or (c.gate_kind == 2 and gammas):
            d_gate = empty(rows if c.gate_kind == 1 else H, dtype=_F32, device=device)
        if workspace is None and gammas:
            workspace = empty(sandwich_norm_workspace_size(rows, H), dtype=_U8, device=device)
    ldd = _row_stride("d_f", d_f, _BF16, shape, dev)
    ldg = _row_stride("d_residual", d_residual, _BF16, shape, dev)
    pw, n = None, 0
    if workspace is not None:
        if workspace.get_device() != dev or workspace.dtype is not _U8 or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{dev}")
        pw, n = workspace.data_ptr(), workspace.numel()
    fn = _lib().moe_sandwich_norm_backward
    call = fn if dev == _current_device() else _at_device(fn, dev)
    st = call(rows, H, byref(c), f.data_ptr(), ldf, residual.data_ptr(), ldr, stats.data_ptr(), ps, lds, po, ldo,
              d_f.data_ptr(), ldd, d_residual.data_ptr(), ldg, None if d_gate is None else d_gate.data_ptr(),
              None if d_post is None else d_post.data_ptr(), None if d_pre is None else d_pre.data_ptr(), pw, n,
              _stream(stream, dev))
    if st:
        _fail("moe_sandwich_norm_backward", st)
    return SandwichGrads(d_f, d_residual, d_gate, d_post, d_pre)
