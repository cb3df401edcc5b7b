"""Binding of the operators around the experts (include/moe.h, "around the experts"): residual
add with RMSNorm and quantised outputs, the router with its balance loss, and the linear
product in the microscaled formats. Argument checks and marshalling only: every step runs in
the library's CUDA kernels, on the current stream unless one is given.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from ctypes import byref
from dataclasses import dataclass

import torch

from .moe import FORMATS, MOE_OK, MoeError, lib

SF_LAYOUTS = {"rows": 0, "atoms": 1}
SF_BLOCK = {"mxfp8": 32, "nvfp4": 16, "mxfp4": 32}
VALUES_PER_BYTE = {"mxfp8": 1, "nvfp4": 2, "mxfp4": 2}
LOGITS = {torch.float32: 0, torch.bfloat16: 1}

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_device = torch.cuda.device

P, I32, I64, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class QuantC(ctypes.Structure):
    _fields_ = [("format", I32), ("sf_layout", I32), ("codes", P), ("sf", P), ("row_scale", P)]


class RouterConfigC(ctypes.Structure):
    _fields_ = [("num_experts", I32), ("top_k", I32), ("renormalize", I32), ("logits_type", I32),
                ("balance_coef", F32)]


class LinearConfigC(ctypes.Structure):
    _fields_ = [("out_features", I32), ("in_features", I32), ("max_tokens", I32), ("format", I32)]


class LinearWeightC(ctypes.Structure):
    _fields_ = [("codes", P), ("sf", P), ("global_scale", P)]


_SIGNATURES = {
    "moe_quant_sf_size": [I32, I32, I64, I64, P],
    "moe_quantize": [I32, I32, P, I64, P, P],
    "moe_add_rmsnorm": [I32, I32, P, I64, P, I64, P, F32, P, I64, P, I64, P, P],
    "moe_router_workspace_size": [P, I32, P],
    "moe_router_forward": [P, I32, P, I64, P, P, P, P, P, P, P, P, SZ, P],
    "moe_router_backward": [P, I32, P, I64, P, P, P, P, P, P, P, I64, P],
    "moe_linear_config_validate": [P],
    "moe_linear_plan": [P, P],
    "moe_linear_plan_destroy": [P],
    "moe_linear_set_wait_timeout": [P, ctypes.c_uint64],
    "moe_linear_weight_sf_size": [P, P],
    "moe_linear_transform_weight": [P, P, P, P],
    "moe_linear_workspace_size": [P, I32, P],
    "moe_linear_forward": [P, I32, P, I64, P, P, I64, P, SZ, P],
    "moe_linear_forward_quantized": [P, I32, P, P, P, I64, P, SZ, P],
    "moe_linear_last_status": [P, P, P, P],
}
_fns = None


def _lib():
    global _fns
    if _fns is None:
        L = lib()
        for name, args in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        _fns = L
    return _fns


def declare(signatures):
    """The library with these functions declared, as a function that loads it at its first call."""
    done = []

    def get():
        if not done:
            L = _lib()
            for name, args in signatures.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = ctypes.c_int
            done.append(L)
        return done[0]
    return get


def _fail(fn: str, status: int):
    raise MoeError(fn, status)


def _at_device(fn, dev: int):
    """The library's call with that device current: it launches on the current one, whatever device the
    addresses belong to. (Calls come here where another one is current.)"""
    def call(*args):
        with _device(dev):
            return fn(*args)
    return call


def _stream(stream, dev: int) -> int:
    """The given stream's handle. Where none is given, calls take _raw_stream: a torch.cuda.Stream object
    costs microseconds to make."""
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    return stream.cuda_stream


def _device_of(name: str, t: torch.Tensor) -> int:
    """The number of the CUDA device that t is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
    return dev


def _on(stream):
    """Where a call allocates what it was not given: memory that is freed then goes back to the
    stream that uses it."""
    return nullcontext() if stream is None else torch.cuda.stream(stream)


def _row_stride(name: str, t: torch.Tensor, dtype, shape, dev: int) -> int:
    """The row stride of a 2-D tensor of this type and shape on this device whose rows are contiguous."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor of shape {tuple(shape)} on cuda:{dev}, "
                         f"got {tuple(t.shape)} on {t.device}")
    stride = t.stride()
    if stride[1] != 1 and shape[1] > 1 and shape[0] > 0:
        raise ValueError(f"{name} must have contiguous rows")
    return stride[0]


def _matrix(name: str, t: torch.Tensor):
    """The shape of a 2-D tensor."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return shape


def _flat(name: str, t: torch.Tensor, dtype, numel: int, dev: int):
    """A contiguous tensor of numel elements on this device."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != numel or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {numel} elements on cuda:{dev}, got {t.numel()} on "
                         f"{t.device}")


# ----------------------------------------------------------------------------- quantised rows

def sf_size(fmt: str, sf_layout: str, rows: int, K: int) -> int:
    """Bytes of the block scales of [rows, K] (moe_quant_sf_size)."""
    n = SZ()
    st = _lib().moe_quant_sf_size(FORMATS[fmt], SF_LAYOUTS[sf_layout], rows, K, byref(n))
    if st != MOE_OK:
        _fail("moe_quant_sf_size", st)
    return n.value


def _set_once(self, name, value):
    if name in self.__dict__:
        raise AttributeError(f"{type(self).__name__}.{name} cannot be replaced: make a new one")
    self.__dict__[name] = value


def _places(tensors):
    """Calls that say where the tensors' elements lie and how many there are, and their answers: what
    resize_, set_, an assignment to .data and a resized storage change behind a handle's back."""
    ask = [method for t in tensors for method in (t.data_ptr, t.numel)]
    return ask, [f() for f in ask]


class Quantized:
    """Quantised rows: codes [rows, K / values per byte], block scales and, for NVFP4, one fp32
    scale per row (moe_quant_t). Codes and scales are byte tensors (uint8 or a float8 type). The
    tensors can be neither replaced nor resized afterwards."""

    def __init__(self, fmt: str, shape, codes: torch.Tensor, sf: torch.Tensor, row_scale: torch.Tensor | None,
                 sf_layout: str = "rows"):
        rows, K = shape
        vpb = VALUES_PER_BYTE[fmt]
        if codes.element_size() != 1 or sf.element_size() != 1:
            raise ValueError("codes and scales must be byte tensors")
        dev = _device_of("codes", codes)
        if not codes.is_contiguous() or codes.numel() != rows * K // vpb:
            raise ValueError(f"codes must be a contiguous CUDA tensor of {rows * K // vpb} bytes")
        if sf.get_device() != dev or not sf.is_contiguous() or sf.numel() < sf_size(fmt, sf_layout, rows, K):
            raise ValueError(f"scales must be a contiguous tensor of sf_size(...) bytes on cuda:{dev}")
        if (row_scale is not None) != (fmt == "nvfp4"):
            raise ValueError("NVFP4, and only NVFP4, has a scale per row")
        if row_scale is not None:
            _flat("row_scale", row_scale, torch.float32, rows, dev)
        self._dev = dev
        self.fmt, self.shape, self.sf_layout = fmt, torch.Size((rows, K)), sf_layout
        self.codes, self.sf, self.row_scale = codes, sf, row_scale
        self._ask, self._at = _places((codes, sf) if row_scale is None else (codes, sf, row_scale))
        self._c = QuantC(FORMATS[fmt], SF_LAYOUTS[sf_layout], codes.data_ptr(), sf.data_ptr(),
                         None if row_scale is None else row_scale.data_ptr())
        self._ref = byref(self._c)

    __setattr__ = _set_once

    def _arg(self, dev: int):
        """The library's argument."""
        if self._dev != dev:
            raise ValueError(f"the Quantized is on cuda:{self._dev}, the other tensors are on cuda:{dev}")
        if [f() for f in self._ask] != self._at:
            raise ValueError("a tensor of the Quantized was resized or given other memory: make a new one")
        return self._ref

    @classmethod
    def alloc(cls, fmt: str, rows: int, K: int, sf_layout: str = "atoms", device=None) -> "Quantized":
        device = device or torch.device("cuda", torch.cuda.current_device())
        return cls(fmt, (rows, K),
                   torch.empty((rows, K // VALUES_PER_BYTE[fmt]), dtype=torch.uint8, device=device),
                   torch.empty(sf_size(fmt, sf_layout, rows, K), dtype=torch.uint8, device=device),
                   torch.empty(rows, dtype=torch.float32, device=device) if fmt == "nvfp4" else None, sf_layout)


def quantize(x: torch.Tensor, fmt: str, sf_layout: str = "atoms", out: Quantized | None = None,
             stream=None) -> Quantized:
    """moe_quantize: the rows of x (bf16 [rows, K]) in a microscaled format."""
    shape = _matrix("x", x)
    dev = _device_of("x", x)
    ldx = _row_stride("x", x, _BF16, shape, dev)
    if out is None:
        with _on(stream):
            out = Quantized.alloc(fmt, shape[0], shape[1], sf_layout, x.device)
    elif out.shape != shape or out.fmt != fmt:
        raise ValueError(f"out holds {out.fmt} {out.shape}, x is {tuple(shape)} for {fmt}")
    fn = (_fns or _lib()).moe_quantize
    call = fn if dev == _current_device() else _at_device(fn, dev)
    st = call(shape[0], shape[1], x.data_ptr(), ldx, out._arg(dev), _stream(stream, dev))
    if st:
        _fail("moe_quantize", st)
    return out


def add_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                sum_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                quantized: Quantized | None = None, stream=None):
    """moe_add_rmsnorm: z = x + residual, y = gamma * z / sqrt(mean(z^2) + eps).

    x, residual, sum_out (receives z), out (receives y): bf16 [rows, H]; gamma: fp32 [H];
    quantized: receives y in its format. Without out and quantized, out is allocated.
    Returns out if there is one, else quantized."""
    shape = _matrix("x", x)
    rows, H = shape
    dev = _device_of("x", x)
    ldx = _row_stride("x", x, _BF16, shape, dev)
    _flat("gamma", gamma, _F32, H, dev)
    if out is None and quantized is None:
        with _on(stream):
            out = torch.empty((rows, H), dtype=_BF16, device=x.device)
    po = pr = ps = pq = None
    ldo = ldr = lds = 0
    if out is not None:
        ldo = _row_stride("out", out, _BF16, shape, dev)
        po = out.data_ptr()
    if residual is not None:
        ldr = _row_stride("residual", residual, _BF16, shape, dev)
        pr = residual.data_ptr()
    if sum_out is not None:
        lds = _row_stride("sum_out", sum_out, _BF16, shape, dev)
        ps = sum_out.data_ptr()
    if quantized is not None:
        if quantized.shape != shape:
            raise ValueError(f"quantized holds {quantized.shape}, x is {tuple(shape)}")
        pq = quantized._arg(dev)
    fn = (_fns or _lib()).moe_add_rmsnorm
    call = fn if dev == _current_device() else _at_device(fn, dev)
    st = call(rows, H, x.data_ptr(), ldx, pr, ldr, gamma.data_ptr(), eps, ps, lds, po, ldo, pq, _stream(stream, dev))
    if st:
        _fail("moe_add_rmsnorm", st)
    return out if out is not None else quantized


# ----------------------------------------------------------------------------- router

@dataclass(frozen=True)
class RouterConfig:
    """What a Router is built for. It cannot be changed: another coefficient or top_k is another Router."""
    num_experts: int
    top_k: int
    renormalize: bool = True
    balance_coef: float = 0.0


class RouterOutput:
    """Buffers of one Router.forward: topk_ids int32 [T, k] (-1: no expert), topk_weights fp32
    [T, k], counts int32 [E], num_valid int32 [1] and, when training, prob_mean fp32 [E] and
    loss fp32 [1]; workspace uint8. counts, num_valid, prob_mean and loss may be None. A buffer is
    replaced by assigning another tensor."""

    def __init__(self, topk_ids: torch.Tensor, topk_weights: torch.Tensor, counts: torch.Tensor | None,
                 num_valid: torch.Tensor | None, prob_mean: torch.Tensor | None, loss: torch.Tensor | None,
                 workspace: torch.Tensor):
        self.topk_ids, self.topk_weights, self.counts, self.num_valid = topk_ids, topk_weights, counts, num_valid
        self.prob_mean, self.loss, self.workspace = prob_mean, loss, workspace

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_args"] = None  # checked again by the next forward

    def __getstate__(self):
        return {**self.__dict__, "_args": None}  # a copy's buffers are its own

    def _check(self, T: int, E: int, k: int, dev: int):
        """The library's arguments for T tokens, after checks that hold while the buffers stay where they are."""
        _flat("topk_ids", self.topk_ids, _I32, T * k, dev)
        _flat("topk_weights", self.topk_weights, _F32, T * k, dev)
        for name, dtype, n in (("counts", _I32, E), ("num_valid", _I32, 1), ("prob_mean", _F32, E), ("loss", _F32, 1)):
            t = getattr(self, name)
            if t is not None:
                _flat(name, t, dtype, n, dev)
        if self.workspace.dtype is not _U8 or self.workspace.get_device() != dev or not self.workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{dev}")
        all_of = (self.topk_ids, self.topk_weights, self.counts, self.num_valid, self.prob_mean, self.loss,
                  self.workspace)
        there = [t for t in all_of if t is not None]
        if any(t.data_ptr() == 0 and t.numel() for t in there):
            raise ValueError("a buffer of the RouterOutput has no memory")
        ptr = [None if t is None else t.data_ptr() for t in all_of]
        self.__dict__["_args"] = ((T, E, k, dev), (*ptr, self.workspace.numel()), *_places(there))


class Router:
    """Softmax router: top-k experts, their weights, per-expert counts and the balance loss
    (moe_router_forward, moe_router_backward)."""

    def __init__(self, cfg: RouterConfig):
        # buffers are checked by what the library was told, whatever becomes of cfg
        self._cfg, self._E, self._k = cfg, cfg.num_experts, cfg.top_k
        self._c = {d: RouterConfigC(cfg.num_experts, cfg.top_k, 1 if cfg.renormalize else 0, code, cfg.balance_coef)
                   for d, code in LOGITS.items()}
        self._ref = {d: byref(c) for d, c in self._c.items()}
        n = SZ()
        st = _lib().moe_router_workspace_size(byref(self._c[torch.float32]), 0, byref(n))
        if st != MOE_OK:
            _fail("moe_router_workspace_size", st)

    @property
    def cfg(self) -> RouterConfig:
        return self._cfg

    def workspace_size(self, num_tokens: int) -> int:
        n = SZ()
        st = _lib().moe_router_workspace_size(byref(self._c[torch.float32]), num_tokens, byref(n))
        if st != MOE_OK:
            _fail("moe_router_workspace_size", st)
        return n.value

    def alloc(self, num_tokens: int, training: bool = False, device=None) -> RouterOutput:
        device = device or torch.device("cuda", torch.cuda.current_device())
        E, k, T = self._E, self._k, num_tokens
        empty = torch.empty
        return RouterOutput(
            empty((T, k), dtype=torch.int32, device=device), empty((T, k), dtype=torch.float32, device=device),
            empty(E, dtype=torch.int32, device=device), empty(1, dtype=torch.int32, device=device),
            empty(E, dtype=torch.float32, device=device) if training else None,
            empty(1, dtype=torch.float32, device=device) if training else None,
            empty(max(self.workspace_size(T), 1), dtype=torch.uint8, device=device))

    def _inputs(self, logits: torch.Tensor, token_mask: torch.Tensor | None):
        """Number of tokens, the logits' device and row stride, and the mask's address."""
        shape = _matrix("logits", logits)
        dtype = logits.dtype
        if dtype not in LOGITS:
            raise ValueError(f"logits must be float32 or bfloat16, got {dtype}")
        dev = _device_of("logits", logits)
        ld = _row_stride("logits", logits, dtype, shape, dev)
        if shape[1] != self._E:
            raise ValueError(f"logits must be [T, {self._E}], got {tuple(shape)}")
        if token_mask is None:
            return shape[0], dev, ld, None
        if token_mask.dtype not in (torch.bool, _U8):
            raise ValueError("token_mask must be bool or uint8")
        _flat("token_mask", token_mask, token_mask.dtype, shape[0], dev)
        return shape[0], dev, ld, token_mask.data_ptr()

    def forward(self, logits: torch.Tensor, token_mask: torch.Tensor | None = None, out: RouterOutput | None = None,
                training: bool = False, stream=None) -> RouterOutput:
        """logits fp32 or bf16 [T, E]; token_mask bool [T] (False: padding). With out, its buffers
        are written (prob_mean and loss when it has them); else they are allocated."""
        T, dev, ld, mask = self._inputs(logits, token_mask)
        E, k = self._E, self._k
        if out is None:
            with _on(stream):
                out = self.alloc(T, training, logits.device)
        o = out
        args = o._args
        if args is None or args[0] != (T, E, k, dev) or [f() for f in args[2]] != args[3]:
            o._check(T, E, k, dev)
            args = o._args
        fn = _fns.moe_router_forward
        call = fn if dev == _current_device() else _at_device(fn, dev)
        st = call(self._ref[logits.dtype], T, logits.data_ptr(), ld, mask, *args[1], _stream(stream, dev))
        if st:
            _fail("moe_router_forward", st)
        return o

    def backward(self, logits: torch.Tensor, topk_ids: torch.Tensor, counts: torch.Tensor | None = None,
                 num_valid: torch.Tensor | None = None, d_weights: torch.Tensor | None = None,
                 d_loss: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The gradient of sum(d_weights * topk_weights) + d_loss * loss with respect to logits
        (counts held constant), in the logits' type."""
        T, dev, ld, mask = self._inputs(logits, token_mask)
        E, k = self._E, self._k
        if out is None:
            with _on(stream):
                out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
        ldo = _row_stride("out", out, logits.dtype, logits.shape, dev)
        _flat("topk_ids", topk_ids, _I32, T * k, dev)
        pw = pl = pc = pn = None
        if d_weights is not None:
            _flat("d_weights", d_weights, _F32, T * k, dev)
            pw = d_weights.data_ptr()
        if d_loss is not None:
            if counts is None or num_valid is None:
                raise ValueError("the loss's gradient needs counts and num_valid")
            _flat("d_loss", d_loss, _F32, 1, dev)
            _flat("counts", counts, _I32, E, dev)
            _flat("num_valid", num_valid, _I32, 1, dev)
            pl, pc, pn = d_loss.data_ptr(), counts.data_ptr(), num_valid.data_ptr()
        fn = _fns.moe_router_backward
        call = fn if dev == _current_device() else _at_device(fn, dev)
        st = call(self._ref[logits.dtype], T, logits.data_ptr(), ld, mask, topk_ids.data_ptr(), pc, pn, pw, pl,
                  out.data_ptr(), ldo, _stream(stream, dev))
        if st:
            _fail("moe_router_backward", st)
        return out


# ----------------------------------------------------------------------------- linear product

@dataclass(frozen=True)
class LinearConfig:
    """What a LinearPlan is built for. It cannot be changed."""
    out_features: int
    in_features: int
    max_tokens: int
    fmt: str = "nvfp4"

    def to_c(self) -> LinearConfigC:
        return LinearConfigC(self.out_features, self.in_features, self.max_tokens, FORMATS[self.fmt])


def linear_validate(cfg: LinearConfig) -> int:
    return _lib().moe_linear_config_validate(byref(cfg.to_c()))


class LinearWeight:
    """A weight in the kernel layout (LinearPlan.transform_weight): codes, scale atoms (both bytes) and, for
    NVFP4, the global scale; the format and the shape [N, K] that they were laid out for, where that is
    known. Its tensors can be neither replaced nor resized."""

    __setattr__ = _set_once

    def __init__(self, codes: torch.Tensor, sf: torch.Tensor, global_scale: torch.Tensor | None,
                 fmt: str | None = None, shape=None):
        dev = _device_of("codes", codes)
        for name, t in (("codes", codes), ("sf", sf)):
            if t.element_size() != 1 or t.get_device() != dev or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous byte tensor on cuda:{dev}")
        if global_scale is not None:
            _flat("global_scale", global_scale, _F32, 1, dev)
        self._dev = dev
        self.codes, self.sf, self.global_scale = codes, sf, global_scale
        self.fmt, self.shape = fmt, None if shape is None else tuple(shape)
        self._bytes = (codes.numel(), sf.numel(), global_scale is not None)
        self._ask, self._at = _places((codes, sf) if global_scale is None else (codes, sf, global_scale))
        self._c = LinearWeightC(codes.data_ptr(), sf.data_ptr(),
                                None if global_scale is None else global_scale.data_ptr())
        self._ref = byref(self._c)

    def _arg(self, dev: int):
        """The library's argument."""
        if self._dev != dev:
            raise ValueError(f"the weight is on cuda:{self._dev}, the plan is for cuda:{dev}")
        if [f() for f in self._ask] != self._at:
            raise ValueError("a tensor of the LinearWeight was resized or given other memory: make a new one")
        return self._ref


class LinearPlan:
    """out[t, n] = sum_k x[t, k] W[n, k] with x and W in a microscaled format (moe_linear_*), on the device that
    is current when the plan is made."""

    def __init__(self, cfg: LinearConfig):
        # tensors are checked by what the library was told, whatever becomes of cfg
        self._cfg, self._N, self._K, self._fmt = cfg, cfg.out_features, cfg.in_features, cfg.fmt
        h = ctypes.c_void_p()
        st = _lib().moe_linear_plan(byref(cfg.to_c()), byref(h))
        if st != MOE_OK:
            _fail("moe_linear_plan", st)
        self._h, self._dev = h, _current_device()
        n = SZ()
        st = _lib().moe_linear_weight_sf_size(h, byref(n))
        if st != MOE_OK:
            _fail("moe_linear_weight_sf_size", st)
        # what a weight of this plan looks like
        self._weight_bytes = (self._N * self._K // VALUES_PER_BYTE[self._fmt], n.value, self._fmt == "nvfp4")

    def __del__(self):
        if getattr(self, "_h", None) and _fns is not None:
            _fns.moe_linear_plan_destroy(self._h)
            self._h = None

    @property
    def cfg(self) -> LinearConfig:
        return self._cfg

    def workspace_size(self, num_tokens: int) -> int:
        n = SZ()
        st = _lib().moe_linear_workspace_size(self._h, num_tokens, byref(n))
        if st != MOE_OK:
            _fail("moe_linear_workspace_size", st)
        return n.value

    def alloc_workspace(self, num_tokens: int, device=None) -> torch.Tensor:
        return torch.zeros(max(self.workspace_size(num_tokens), 1), dtype=torch.uint8,
                           device=device or torch.device("cuda", self._dev))

    def transform_weight(self, codes: torch.Tensor, sf: torch.Tensor, global_scale: torch.Tensor | None = None,
                         stream=None) -> LinearWeight:
        """Checkpoint codes [N, K / values per byte] and row-major block scales [N, K / g] (bytes), with
        the NVFP4 global scale (fp32 [1]), in the kernel layout. The codes are shared, not copied."""
        N, K, fmt = self._N, self._K, self._fmt
        for name, t, n in (("codes", codes, N * K // VALUES_PER_BYTE[fmt]), ("sf", sf, N * K // SF_BLOCK[fmt])):
            if t.element_size() != 1 or t.get_device() != self._dev or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{name} must be a contiguous byte tensor of {n} bytes on cuda:{self._dev}")
        with _on(stream):
            dst = LinearWeight(codes, torch.empty(self._weight_bytes[1], dtype=torch.uint8, device=codes.device),
                               global_scale, fmt, (N, K))
        src = LinearWeightC(codes.data_ptr(), sf.data_ptr(), None if global_scale is None else global_scale.data_ptr())
        fn = _lib().moe_linear_transform_weight
        call = fn if self._dev == _current_device() else _at_device(fn, self._dev)
        st = call(self._h, byref(src), byref(dst._c), _stream(stream, self._dev))
        if st != MOE_OK:
            _fail("moe_linear_transform_weight", st)
        return dst

    def _refuse_weight(self, w: LinearWeight):
        N, K, fmt = self._N, self._K, self._fmt
        raise ValueError(f"the weight holds {w.fmt or 'codes'} {w.shape or ''} of {w._bytes[0]} code and {w._bytes[1]} "
                         f"scale bytes{' with' if w._bytes[2] else ' without'} a global scale; this plan takes {fmt} "
                         f"{(N, K)}, {self._weight_bytes[0]} and {self._weight_bytes[1]} bytes")

    def forward(self, x, weight: LinearWeight, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x: bf16 [T, K] (quantised by the call) or a Quantized with scales in atoms; out bf16 [T, N]."""
        N, dev = self._N, self._dev
        quantized = type(x) is Quantized
        shape = x.shape if quantized else _matrix("x", x)
        T = shape[0]
        if shape[1] != self._K:
            raise ValueError(f"x must be [T, {self._K}], got {tuple(shape)}")
        if weight._bytes != self._weight_bytes or \
                (weight.shape is not None and (weight.fmt != self._fmt or weight.shape != (N, self._K))):
            self._refuse_weight(weight)
        if not quantized:
            ldx = _row_stride("x", x, _BF16, shape, dev)
        if out is None:
            with _on(stream):
                out = torch.empty((T, N), dtype=_BF16, device=weight.codes.device)
        ldo = _row_stride("out", out, _BF16, (T, N), dev)
        if workspace is None:
            with _on(stream):
                workspace = self.alloc_workspace(T, out.device)
        elif workspace.get_device() != dev or workspace.dtype is not _U8 or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{dev}")
        s = _stream(stream, dev)
        if quantized:
            fn = _fns.moe_linear_forward_quantized
            call = fn if dev == _current_device() else _at_device(fn, dev)
            st = call(self._h, T, x._arg(dev), weight._arg(dev), out.data_ptr(), ldo, workspace.data_ptr(),
                      workspace.numel(), s)
        else:
            fn = _fns.moe_linear_forward
            call = fn if dev == _current_device() else _at_device(fn, dev)
            st = call(self._h, T, x.data_ptr(), ldx, weight._arg(dev), out.data_ptr(), ldo, workspace.data_ptr(),
                      workspace.numel(), s)
        if st:
            _fail("moe_linear_forward", st)
        return out

    def set_wait_timeout(self, ns: int):
        """Limit of each bounded wait in the product's kernels (0: the default, 2 s)."""
        st = _lib().moe_linear_set_wait_timeout(self._h, ns)
        if st != MOE_OK:
            _fail("moe_linear_set_wait_timeout", st)

    def last_status(self, workspace: torch.Tensor, stream=None) -> int:
        """The status of the last forward in this workspace, which is waited for (moe_linear_last_status)."""
        v = I32()
        least = self.workspace_size(0)  # the status words lie at its start, as many for every number of tokens
        if workspace.get_device() != self._dev or workspace.dtype is not _U8 or not workspace.is_contiguous() or \
                workspace.numel() < least:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of {least} bytes or more on "
                             f"cuda:{self._dev}, got {workspace.numel()} {workspace.dtype} on {workspace.device}")
        fn = _lib().moe_linear_last_status
        call = fn if self._dev == _current_device() else _at_device(fn, self._dev)
        st = call(self._h, workspace.data_ptr(), _stream(stream, self._dev), byref(v))
        if st != MOE_OK:
            _fail("moe_linear_last_status", st)
        return v.value
