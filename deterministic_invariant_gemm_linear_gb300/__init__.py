"""Deterministic, batch-invariant BF16 contractions for GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/rlk.h`` (librlk.so, built
in-tree by ``build.py``).  This module only marshals arguments: PyTorch is used
for device memory and streams; every step of every operator runs in the
library's CUDA kernels.  There is no CPU or PyTorch fallback — if the library
is missing, or the device is not sm_103, calls raise.

Operators (web pages of the RL-Kernel project):
  * ``linear_logp`` — "feat(linear-logp): add batch-invariant fused SM90
    operator": log_softmax(hidden . W^T + bias)[target] and the log-sum-exp,
    with a vocabulary split that depends on V only.  Forward only: inputs that
    require grad are rejected (the page's author notes: backward is outside
    the contract and fails closed).
  * ``det_gemm_fwd / det_gemm_da / det_gemm_db`` — "feat(musa): add native
    deterministic gemm kernel": C = A B, dA = dC B^T, dB = A^T dC with FP32
    accumulation in a fixed ascending K order, BF16 or FP32 output; an FP32 dC
    is rounded to BF16 first (that page's review comment).
  * ``linear_logp_trainable``, ``det_gemm_trainable``, ``det_linear_trainable`` —
    opt-in torch.autograd wiring of the forward entries to the library's
    backward entries (gradients bitwise equal to calling those entries).

Operators of a training loop around them (on-policy distillation):
  * ``sample_logits`` — one token a row from logits by temperature, top-k, top-p
    and min-p, from one given uniform number a row; the token depends on its
    row alone, bit for bit.
  * ``linear_distill``, ``linear_distill_backward``,
    ``linear_distill_trainable`` — T^2 KL(teacher || student) of hidden . W^T
    over a teacher's top logits without the [N, V] logits of the student, and
    its gradients (the trainable form keeps the FP32 logits between forward and
    backward where they fit KEEP_LOGITS_BYTES; keep_logits=False does not).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import operator
import os

import torch
from torch.autograd.function import once_differentiable

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# RLK_LIBRARY=debug selects the debug build (store checks, phase trace) of the
# same library; anything else, or unset, the release build.
LIB_PATH = os.path.join(_PKG_DIR, "librlk_debug.so" if os.environ.get("RLK_LIBRARY") == "debug"
                        else "librlk.so")

RLK_OK = 0
RLK_BF16, RLK_FP32, RLK_FP64 = 0, 1, 2
RLK_GEMM_FWD, RLK_GEMM_DA, RLK_GEMM_DB = 0, 1, 2
RLK_GEMM_LINEAR_FWD, RLK_GEMM_LINEAR_DX, RLK_GEMM_LINEAR_DW, RLK_GEMM_FWD_ACCUM = 3, 4, 5, 6
STATUS_NAMES = {0: "RLK_OK", 1: "RLK_ERR_NULL", 2: "RLK_ERR_SHAPE", 3: "RLK_ERR_DTYPE",
                4: "RLK_ERR_ALIGN", 5: "RLK_ERR_WORKSPACE", 6: "RLK_ERR_UNSUPPORTED_DEVICE",
                7: "RLK_ERR_CUDA", 8: "RLK_ERR_TIMEOUT", 9: "RLK_ERR_BOUNDS",
                10: "RLK_ERR_NOT_DEBUG_BUILD", 11: "RLK_ERR_VALUE"}
RLK_DEVERR_TIMEOUT, RLK_DEVERR_BOUNDS = 0x1, 0x2
TRACE_FIELDS, TRACE_MAX_CTAS = 16, 1024


class RlkError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


_P, _I64, _SZ, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
_F = ctypes.c_float

# name -> (restype, argtypes); mirrors include/rlk.h
SIGNATURES = {
    "rlk_status_string": (ctypes.c_char_p, [_I]),
    "rlk_numerics_version": (_I, []),
    "rlk_device_check": (_I, []),
    "rlk_get_device_error": (_I, [_P, ctypes.POINTER(ctypes.c_uint32)]),
    "rlk_selftest_bounded_wait": (_I, [ctypes.c_uint32, _P]),
    "rlk_is_debug_build": (_I, []),
    "rlk_selftest_store_check": (_I, [_P]),
    "rlk_debug_trace_read": (_I, [_P, _I64, ctypes.POINTER(_I64)]),
    "rlk_vocab_split_policy": (_I, [_I64, ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                                    ctypes.POINTER(_I64)]),
    "rlk_linear_logp_workspace_size": (_SZ, [_P, _I64, _I64, _I64, _P, _I64, _I64]),
    "rlk_linear_logp": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64,
                             _P, _P, _P, _P, _SZ, _P]),
    "rlk_linear_logp_partials": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64,
                                      _P, _SZ, _P]),
    "rlk_linear_logp_combine": (_I, [_I64, _I64, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "rlk_linear_logp_noalloc": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64,
                                     _P, _P, _P, _P]),
    "rlk_throughput_split_count": (_I, [_I64, _I64, ctypes.c_int32, ctypes.POINTER(_I64)]),
    "rlk_det_gemm_tile_plan": (_I, [_I, _I64, _I64, _I64, ctypes.c_int32,
                                    ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(_I64),
                                    ctypes.POINTER(ctypes.c_int32)]),
    "rlk_vocab_shard_range": (_I, [_I64, _I64, _I64, ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                                   ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "rlk_linear_logp_shard_workspace_size": (_SZ, [_P, _I64, _I64, _I64, _P, _I64, _I64, _I64,
                                                   _I64]),
    "rlk_linear_logp_shard_partials": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I64, _P,
                                            _P, _I64, _P, _I64, _P, _P, _SZ, _P]),
    "rlk_linear_logp_combine_shards": (_I, [_I64, _I64, _P, _I64, _I64, _P, _P, _I64, _I64, _P,
                                            _I64, _P, _P, _P, _P]),
    "rlk_linear_logp_splits_workspace_size": (_SZ, [_P, _I64, _I64, _I64, _P, _I64, _I64, _I64]),
    "rlk_linear_logp_splits": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64,
                                    _P, _P, _P, _I64, _P, _SZ, _P]),
    "rlk_linear_logp_backward_workspace_size": (_SZ, [_I64, _I64]),
    "rlk_linear_logp_backward_workspace_size_for": (_SZ, [_P, _I64, _I64, _I64, _P, _I64, _I64]),
    "rlk_linear_logp_backward": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _P, _P,
                                      _P, _I, _I64, _P, _I, _I64, _P, _P, _SZ, _P]),
    "rlk_sample_logits_workspace_size": (_SZ, [_I, _I64, _I64]),
    "rlk_sample_logits": (_I, [_P, _I, _I64, _I64, _I64, _P, _I, _P, _F, _P, ctypes.c_int32, _P, _F,
                               _P, _F, _P, _P, _P, _SZ, _P]),
    "rlk_linear_distill_workspace_size": (_SZ, [_P, _I64, _I64, _I64, _P, _I64, _I64, _I64]),
    "rlk_linear_distill": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _P, _I, _I64,
                                _I64, _P, _F, _P, _P, _P, _I64, _P, _SZ, _P]),
    "rlk_linear_distill_backward_workspace_size": (_SZ, [_P, _I64, _I64, _I64, _P, _I64, _I64, _I64,
                                                         _I]),
    "rlk_linear_distill_backward": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _P, _I,
                                         _I64, _I64, _P, _F, _P, _P, _I64, _P, _P, _I, _I64, _P, _I,
                                         _I64, _P, _P, _SZ, _P]),
    "rlk_det_gemm_workspace_size": (_SZ, [_I, _P, _I, _I64, _I64, _I64, _P, _I, _I64, _I64, _I64]),
    "rlk_det_gemm_fwd": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _I, _I64, _P, _SZ, _P]),
    "rlk_det_gemm_da": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _P, _I, _I64, _P, _SZ, _P]),
    "rlk_det_gemm_db": (_I, [_P, _I64, _I64, _I64, _P, _I, _I64, _I64, _P, _I, _I64, _P, _SZ, _P]),
    "rlk_det_gemm_fwd_accum_fp32": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _SZ,
                                         _P]),
    "rlk_sum_partials_ordered": (_I, [_P, _I64, _I64, _I64, _I64, _I64, _P, _I, _I64, _P]),
    "rlk_det_linear_fwd": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _I, _I64, _P, _SZ, _P]),
    "rlk_det_linear_dx": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _P, _I, _I64, _P, _SZ, _P]),
    "rlk_det_linear_dw": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _P, _I, _I64, _P, _SZ, _P]),
    "rlk_det_gemm_backward_workspace_size": (_SZ, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _P,
                                                   _I64]),
    "rlk_det_gemm_backward": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _I,
                                   _I64, _P, _I, _I64, _P, _SZ, _P]),
    "rlk_det_linear_backward_workspace_size": (_SZ, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _P,
                                                     _I64]),
    "rlk_det_linear_backward": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _I,
                                     _I64, _P, _I, _I64, _P, _SZ, _P]),
}

_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded librlk.so; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"librlk.so is not built ({LIB_PATH}); build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        cdll = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(cdll, name)
            f.restype = res
            f.argtypes = args
        _LIB = cdll
    return _LIB


def status_string(status: int) -> str:
    return lib().rlk_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != RLK_OK:
        raise RlkError(status, what)


def numerics_version() -> int:
    return int(lib().rlk_numerics_version())


def vocab_split_policy(V: int):
    """(num_splits, vtiles_per_split, num_vtiles) for a vocabulary of V ids."""
    s, v, t = _I64(), _I64(), _I64()
    _check(lib().rlk_vocab_split_policy(V, ctypes.byref(s), ctypes.byref(v), ctypes.byref(t)),
           "rlk_vocab_split_policy")
    return s.value, v.value, t.value


def device_error(stream=None) -> int:
    """Reads and clears the library's device error word (synchronises the stream)."""
    flags = ctypes.c_uint32(0)
    st = lib().rlk_get_device_error(_stream_ptr(stream), ctypes.byref(flags))
    if st not in (RLK_OK, 8, 9):
        _check(st, "rlk_get_device_error")
    return flags.value


def is_debug_build() -> bool:
    return bool(lib().rlk_is_debug_build())


def debug_trace(max_ctas: int = TRACE_MAX_CTAS):
    """Debug build: the linear-logp kernels' per-CTA phase timestamps (ns) since the
    last read, as a list of TRACE_FIELDS-tuples indexed by CTA (then cleared)."""
    import numpy as np
    out = np.zeros((max_ctas, TRACE_FIELDS), dtype=np.uint64)
    n = _I64()
    _check(lib().rlk_debug_trace_read(out.ctypes.data_as(ctypes.c_void_p), max_ctas,
                                      ctypes.byref(n)), "rlk_debug_trace_read")
    return out[:n.value]


# A small call's time is its host side: addresses pass as plain integers, the current stream
# and device are asked for without building their Python objects (0.1 us for 2.9, and 0.3 for
# 1.5 where the device is current already, on the Grace host).
def _stream_ptr(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


_HERE = contextlib.nullcontext()


def _on(device):
    """The device made current for a with block."""
    return _HERE if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def _used_by(stream, tensors):
    """Marks the memory of CUDA tensors as in use by a stream that it was not allocated on."""
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)


def _streamed(call):
    """An entry point's stream argument: the whole call, its copies and allocations included, is
    made with that stream current, so what it makes and drops is ordered and reused there.  The
    caller orders the stream after the inputs, and its own work after the stream; inputs and
    outputs may be dropped on either side."""
    @functools.wraps(call)
    def run(*args, stream=None, **named):
        if stream is None:
            return call(*args, **named)
        here = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            out = call(*args, **named)
        if stream != here:
            _used_by(stream, args)
            _used_by(stream, named.values())
            _used_by(here, out if isinstance(out, tuple) else (out,))
        return out
    return run


def _matrix(t: torch.Tensor, name: str):
    """(tensor, leading dimension) for a 2-D row-major operand (unit column stride)."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(shape)}")
    rows, cols = shape
    ld, step = t.stride()
    if step != 1 or (rows > 1 and ld < cols):
        t = t.contiguous()
        ld = t.stride(0)
    return t, ld if rows > 1 or ld > cols else cols


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("rlk operates on CUDA tensors only (no CPU fallback)")


_DT = {torch.bfloat16: RLK_BF16, torch.float32: RLK_FP32}


# ------------------------------------------------------------------ linear-logp
def linear_logp_workspace(hidden2d, weight, ldh, ldw, N, H, V) -> torch.Tensor:
    n = lib().rlk_linear_logp_workspace_size(_ptr(hidden2d), N, H, ldh, _ptr(weight), V, ldw)
    if n == 0 and N > 0:
        raise RlkError(2, "rlk_linear_logp_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=hidden2d.device)


def throughput_split_count(N: int, V: int, sm_count: int = 0) -> int:
    """The occupancy-driven split count of the throughput-mode ablation (depends on N)."""
    s = _I64()
    _check(lib().rlk_throughput_split_count(N, V, sm_count, ctypes.byref(s)),
           "rlk_throughput_split_count")
    return s.value


def det_gemm_tile_plan(op: int, out_rows: int, out_cols: int, red: int, sm_count: int) -> dict:
    """The output tiling of det_gemm op (RLK_GEMM_*) for these extents on sm_count SMs
    (host arithmetic): {"tile_cols": 256 | 224 | 128, "split_blocks": wide blocks run as
    halves, "launches": 1 | 2}."""
    t, b, n = ctypes.c_int32(), _I64(), ctypes.c_int32()
    _check(lib().rlk_det_gemm_tile_plan(op, out_rows, out_cols, red, sm_count, ctypes.byref(t),
                                        ctypes.byref(b), ctypes.byref(n)), "rlk_det_gemm_tile_plan")
    return {"tile_cols": t.value, "split_blocks": b.value, "launches": n.value}


@_streamed
def linear_logp(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                bias: torch.Tensor | None = None, *, return_target_logit: bool = False,
                stream=None, num_splits: int | None = None):
    """logp, lse (FP32, shaped like hidden's leading dims) [, target logit].

    hidden [..., H] bf16, weight [V, H] bf16, target [...] int64 (any strides,
    including an expanded zero-stride target), bias [V] fp32 or None.
    num_splits (ablation only): an explicit vocabulary split count instead of
    the V-only policy (rlk_linear_logp_splits); 0 means the V-only policy.
    """
    if hidden.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad):
        raise RuntimeError("linear_logp is forward-only: inputs that require grad are rejected")
    _require_cuda(hidden, weight, target, bias)
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise TypeError("hidden and weight must be bfloat16")
    if target.dtype != torch.int64:
        raise TypeError("target must be int64")
    if bias is not None and (bias.dtype != torch.float32 or bias.dim() != 1):
        raise TypeError("bias must be a 1-D float32 tensor")
    lead = hidden.shape[:-1]
    H = hidden.size(-1)
    h2, ldh = _matrix(hidden.reshape(-1, H), "hidden")
    w2, ldw = _matrix(weight, "weight")
    N, V = h2.size(0), w2.size(0)
    if w2.size(1) != H:
        raise ValueError("weight must be [V, H] with the hidden size H")
    t1 = target.reshape(-1)
    if t1.numel() != N:
        raise ValueError("target must have one id per hidden row")
    tstride = t1.stride(0) if N > 1 else 1
    if bias is not None:
        bias = bias.contiguous()
        if bias.numel() != V:
            raise ValueError("bias must have V entries")
    dev = hidden.device
    logp = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    zt = torch.empty(N, dtype=torch.float32, device=dev) if return_target_logit else None
    with _on(dev):
        if num_splits is None:
            ws = linear_logp_workspace(h2, w2, ldh, ldw, N, H, V)
            st = lib().rlk_linear_logp(_ptr(h2), N, H, ldh, _ptr(w2), V, ldw, _ptr(bias), _ptr(t1),
                                       tstride, _ptr(logp), _ptr(lse), _ptr(zt), _ptr(ws),
                                       ws.numel(), _stream_ptr(stream))
        else:
            n = lib().rlk_linear_logp_splits_workspace_size(_ptr(h2), N, H, ldh, _ptr(w2), V, ldw,
                                                            num_splits)
            if n == 0 and N > 0:
                raise RlkError(2, "rlk_linear_logp_splits_workspace_size")
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
            st = lib().rlk_linear_logp_splits(_ptr(h2), N, H, ldh, _ptr(w2), V, ldw, _ptr(bias),
                                              _ptr(t1), tstride, _ptr(logp), _ptr(lse), _ptr(zt),
                                              num_splits, _ptr(ws), ws.numel(),
                                              _stream_ptr(stream))
    _check(st, "rlk_linear_logp")
    out = (logp.reshape(lead), lse.reshape(lead))
    if return_target_logit:
        out = out + (zt.reshape(lead),)
    return out


class LinearLogpCall:
    """A prepared linear-logp call on fixed tensors (outputs and workspace
    allocated once), runnable as the whole operator or as its two stages."""

    def __init__(self, hidden, weight, target, bias=None, *, target_logit: bool = False,
                 num_splits: int | None = None):
        _require_cuda(hidden, weight, target, bias)
        self.num_splits = num_splits      # None: the operator; an int: the ablation entry point
        self.h, self.ldh = _matrix(hidden, "hidden")
        self.w, self.ldw = _matrix(weight, "weight")
        self.t = target.reshape(-1)
        self.bias = None if bias is None else bias.contiguous()
        self.N, self.H = self.h.shape
        self.V = self.w.size(0)
        self.tstride = self.t.stride(0) if self.N > 1 else 1
        dev = hidden.device
        self.logp = torch.empty(self.N, dtype=torch.float32, device=dev)
        self.lse = torch.empty(self.N, dtype=torch.float32, device=dev)
        self.zt = torch.empty(self.N, dtype=torch.float32, device=dev) if target_logit else None
        with _on(dev):
            if num_splits is None:
                self.ws = linear_logp_workspace(self.h, self.w, self.ldh, self.ldw, self.N, self.H,
                                                self.V)
            else:
                n = lib().rlk_linear_logp_splits_workspace_size(
                    _ptr(self.h), self.N, self.H, self.ldh, _ptr(self.w), self.V, self.ldw,
                    num_splits)
                if n == 0 and self.N > 0:
                    raise RlkError(2, "rlk_linear_logp_splits_workspace_size")
                self.ws = torch.empty(n, dtype=torch.uint8, device=dev)

    def _use(self, stream):
        if stream is not None and stream != torch.cuda.current_stream(stream.device):
            _used_by(stream, (self.h, self.w, self.t, self.bias, self.logp, self.lse, self.zt, self.ws))

    def partials(self, stream=None):
        if self.num_splits is not None:
            raise RuntimeError("the two-stage calls use the V-only split")
        self._use(stream)
        _check(lib().rlk_linear_logp_partials(
            _ptr(self.h), self.N, self.H, self.ldh, _ptr(self.w), self.V, self.ldw, _ptr(self.bias),
            _ptr(self.t), self.tstride, _ptr(self.ws), self.ws.numel(), _stream_ptr(stream)),
            "rlk_linear_logp_partials")

    def combine(self, stream=None):
        if self.num_splits is not None:
            raise RuntimeError("the two-stage calls use the V-only split")
        self._use(stream)
        _check(lib().rlk_linear_logp_combine(
            self.N, self.V, _ptr(self.t), self.tstride, _ptr(self.logp), _ptr(self.lse),
            _ptr(self.zt), _ptr(self.ws), self.ws.numel(), _stream_ptr(stream)),
            "rlk_linear_logp_combine")

    def __call__(self, stream=None):
        self._use(stream)
        if self.num_splits is None:
            _check(lib().rlk_linear_logp(
                _ptr(self.h), self.N, self.H, self.ldh, _ptr(self.w), self.V, self.ldw,
                _ptr(self.bias), _ptr(self.t), self.tstride, _ptr(self.logp), _ptr(self.lse),
                _ptr(self.zt), _ptr(self.ws), self.ws.numel(), _stream_ptr(stream)),
                "rlk_linear_logp")
        else:
            _check(lib().rlk_linear_logp_splits(
                _ptr(self.h), self.N, self.H, self.ldh, _ptr(self.w), self.V, self.ldw,
                _ptr(self.bias), _ptr(self.t), self.tstride, _ptr(self.logp), _ptr(self.lse),
                _ptr(self.zt), self.num_splits, _ptr(self.ws), self.ws.numel(),
                _stream_ptr(stream)), "rlk_linear_logp_splits")
        return self.logp, self.lse


# ------------------------------------------------------------ vocabulary shards
def vocab_shard_range(V: int, num_shards: int, shard: int):
    """(split_begin, split_end, v_begin, v_end) of shard `shard` in the balanced
    partition of the V-only splits into num_shards contiguous runs."""
    out = [_I64() for _ in range(4)]
    _check(lib().rlk_vocab_shard_range(V, num_shards, shard, *[ctypes.byref(x) for x in out]),
           "rlk_vocab_shard_range")
    return tuple(x.value for x in out)


@_streamed
def linear_logp_shard_partials(hidden: torch.Tensor, weight_shard: torch.Tensor,
                               target: torch.Tensor, V: int, split_begin: int, split_end: int,
                               bias_shard: torch.Tensor | None = None, *, ld_partials: int = 0,
                               stream=None):
    """Partials of one vocabulary shard: (partials [N, ld, 2] fp32 with the shard's
    (m, s) pairs in its first split_end - split_begin columns, target logits [N]
    fp32, NaN for rows whose target the shard does not hold).

    weight_shard [v_end - v_begin, H] bf16 holds the weight rows of the shard's
    vocabulary ids, bias_shard the matching bias entries; V is the whole
    vocabulary; target holds global ids.
    """
    _require_cuda(hidden, weight_shard, target, bias_shard)
    h2, ldh = _matrix(hidden.reshape(-1, hidden.size(-1)), "hidden")
    w2, ldw = _matrix(weight_shard, "weight_shard")
    N, H = h2.shape
    t1 = target.reshape(-1)
    tstride = t1.stride(0) if N > 1 else 1
    n = split_end - split_begin
    ld = max(ld_partials, n, 1)
    if bias_shard is not None:
        bias_shard = bias_shard.contiguous()
    dev = hidden.device
    partials = torch.empty(N, ld, 2, dtype=torch.float32, device=dev)
    zt = torch.full((N,), float("nan"), dtype=torch.float32, device=dev)
    with _on(dev):
        nb = lib().rlk_linear_logp_shard_workspace_size(_ptr(h2), N, H, ldh, _ptr(w2), V,
                                                        split_begin, split_end, ldw)
        if nb == 0:
            raise RlkError(2, "rlk_linear_logp_shard_workspace_size")
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        _check(lib().rlk_linear_logp_shard_partials(
            _ptr(h2), N, H, ldh, _ptr(w2), V, split_begin, split_end, ldw, _ptr(bias_shard),
            _ptr(t1), tstride, _ptr(partials), ld, _ptr(zt), _ptr(ws), nb, _stream_ptr(stream)),
            "rlk_linear_logp_shard_partials")
    return partials, zt


@_streamed
def linear_logp_combine_shards(partials: torch.Tensor, target_logits: torch.Tensor,
                               split_offsets, target: torch.Tensor, V: int, *,
                               return_target_logit: bool = False, stream=None):
    """The fixed-order merge over gathered shard outputs.

    partials [R, N, ld, 2] fp32 (shard q's pairs in its first
    split_offsets[q+1] - split_offsets[q] columns), target_logits [R, N] fp32,
    split_offsets R + 1 split indices (0 .. S).  Returns logp, lse [, target logit],
    bitwise equal to linear_logp on the whole vocabulary.
    """
    _require_cuda(partials, target_logits, target)
    if partials.dim() != 4 or partials.size(-1) != 2 or partials.dtype != torch.float32:
        raise ValueError("partials must be a float32 [R, N, ld, 2] tensor")
    partials = partials.contiguous()
    target_logits = target_logits.contiguous()
    R, N, ld, _ = partials.shape
    if len(split_offsets) != R + 1:
        raise ValueError("split_offsets needs one entry per shard plus one")
    if tuple(target_logits.shape) != (R, N):
        raise ValueError("target_logits must be [R, N] like the partials' first two dims")
    offs = (ctypes.c_int64 * (R + 1))(*[int(x) for x in split_offsets])
    t1 = target.reshape(-1)
    tstride = t1.stride(0) if N > 1 else 1
    dev = partials.device
    logp = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    zt = torch.empty(N, dtype=torch.float32, device=dev) if return_target_logit else None
    with _on(dev):
        _check(lib().rlk_linear_logp_combine_shards(
            N, V, _ptr(t1), tstride, R, offs, _ptr(partials), ld, N * ld, _ptr(target_logits), N,
            _ptr(logp), _ptr(lse), _ptr(zt), _stream_ptr(stream)), "rlk_linear_logp_combine_shards")
    return (logp, lse, zt) if return_target_logit else (logp, lse)


def _all_gather(t: torch.Tensor, group=None) -> torch.Tensor:
    """Every rank's equally shaped tensor, stacked in rank order on t's device.
    With the NCCL backend device tensors are exchanged directly; with gloo they
    travel through host copies."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    dev = t.device
    x = t.contiguous()
    if dist.get_backend(group) != "nccl":
        x = x.cpu()
    parts = [torch.empty_like(x) for _ in range(world)]
    dist.all_gather(parts, x, group=group)
    return torch.stack(parts).to(dev)


def exchange_shard_partials(partials: torch.Tensor, target_logit: torch.Tensor, group=None):
    """All-gather every rank's shard output: ([R, N, ld, 2], [R, N]) in rank order.

    Every rank passes partials padded to the same [N, ld, 2] (the widest shard).
    With the NCCL backend the device tensors are exchanged directly; with gloo the
    tensors travel through host copies and come back on the caller's device.
    """
    return _all_gather(partials, group), _all_gather(target_logit, group)


@_streamed
def sum_partials_ordered(parts: torch.Tensor, out_dtype=torch.float32, *, stream=None):
    """out = parts[0] + parts[1] + ... (FP32, ascending part order) for parts [P, rows, cols]
    fp32, written as out_dtype (bf16 rounds to nearest even)."""
    _require_cuda(parts)
    if parts.dim() != 3 or parts.dtype != torch.float32:
        raise ValueError("parts must be a float32 [P, rows, cols] tensor")
    parts = parts.contiguous()
    P, rows, cols = parts.shape
    out = torch.empty(rows, cols, dtype=out_dtype, device=parts.device)
    with _on(parts.device):
        _check(lib().rlk_sum_partials_ordered(_ptr(parts), P, rows, cols, cols, rows * cols,
                                              _ptr(out), _DT[out_dtype], cols, _stream_ptr(stream)),
               "rlk_sum_partials_ordered")
    return out


def det_gemm_db_row_sharded(A_local: torch.Tensor, dC_local: torch.Tensor,
                            out_dtype=torch.bfloat16, *, group=None):
    """dB = A^T . dC when the rows of A and dC are divided between the ranks of `group`:
    each rank forms its FP32 partial product (det_gemm_db over its own rows), the ranks
    all-gather the partials, and every rank adds them in rank order
    (sum_partials_ordered).  The result is the same bits on every rank and run to
    run; it depends on the row partition, not on the exchange."""
    local = det_gemm_db(A_local, dC_local, out_dtype=torch.float32)
    return sum_partials_ordered(_all_gather(local, group), out_dtype)


def vocab_parallel_linear_logp(hidden: torch.Tensor, weight_shard: torch.Tensor,
                               target: torch.Tensor, V: int,
                               bias_shard: torch.Tensor | None = None, *, group=None,
                               return_target_logit: bool = False):
    """linear_logp with the vocabulary divided between the ranks of `group`.

    Rank q holds the weight rows (and bias entries) of its balanced shard,
    vocab_shard_range(V, world, q); every rank passes the same hidden and target.
    Each rank computes its shard's partials, the ranks exchange them
    (exchange_shard_partials), and every rank merges all of them in the fixed
    order: the results equal single-device linear_logp bit for bit.
    """
    import torch.distributed as dist
    world, rank = dist.get_world_size(group), dist.get_rank(group)
    ranges = [vocab_shard_range(V, world, q) for q in range(world)]
    j0, j1, v0, v1 = ranges[rank]
    if weight_shard.size(0) != v1 - v0:
        raise ValueError(f"rank {rank} holds vocabulary ids [{v0}, {v1}): weight_shard needs "
                         f"{v1 - v0} rows, got {weight_shard.size(0)}")
    widest = max(r[1] - r[0] for r in ranges)
    partials, zt = linear_logp_shard_partials(hidden, weight_shard, target, V, j0, j1, bias_shard,
                                              ld_partials=widest)
    gp, gz = exchange_shard_partials(partials, zt, group)
    offsets = [r[0] for r in ranges] + [ranges[-1][1]]
    out = linear_logp_combine_shards(gp, gz, offsets, target, V,
                                     return_target_logit=return_target_logit)
    lead = hidden.shape[:-1]
    return tuple(o.reshape(lead) for o in out)


@_streamed
def linear_logp_backward(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                         lse: torch.Tensor, grad_logp: torch.Tensor, bias: torch.Tensor | None = None,
                         *, grad_hidden: bool = True, grad_weight: bool = True,
                         grad_bias: bool | None = None, out_dtype=torch.bfloat16,
                         return_grad_logits: bool = False, stream=None):
    """(grad_hidden [..., H], grad_weight [V, H], grad_bias [V] | None) for logp = linear_logp(...).

    lse is the forward's lse; grad_logp is dL/dlogp (same leading shape as hidden's rows).
    With return_grad_logits, also returns G = dL/dz as the BF16 [N, V] view the kernels used.
    """
    _require_cuda(hidden, weight, target, lse, grad_logp, bias)
    lead = hidden.shape[:-1]
    H = hidden.size(-1)
    h2, ldh = _matrix(hidden.reshape(-1, H), "hidden")
    w2, ldw = _matrix(weight, "weight")
    N, V = h2.size(0), w2.size(0)
    t1 = target.reshape(-1)
    tstride = t1.stride(0) if N > 1 else 1
    l1 = lse.reshape(-1).contiguous().float()
    g1 = grad_logp.reshape(-1).contiguous().float()
    if bias is not None:
        bias = bias.contiguous()
    if grad_bias is None:
        grad_bias = bias is not None
    dev = hidden.device
    gh = torch.empty(N, H, dtype=out_dtype, device=dev) if grad_hidden else None
    gw = torch.empty(V, H, dtype=out_dtype, device=dev) if grad_weight else None
    gb = torch.empty(V, dtype=torch.float32, device=dev) if grad_bias else None
    with _on(dev):
        n = lib().rlk_linear_logp_backward_workspace_size_for(_ptr(h2), N, H, ldh, _ptr(w2), V, ldw)
        if n == 0:
            raise RlkError(2, "rlk_linear_logp_backward_workspace_size_for")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        dt = _DT[out_dtype]
        _check(lib().rlk_linear_logp_backward(
            _ptr(h2), N, H, ldh, _ptr(w2), V, ldw, _ptr(bias), _ptr(t1), tstride, _ptr(l1), _ptr(g1),
            _ptr(gh), dt, H, _ptr(gw), dt, H, _ptr(gb), _ptr(ws), n, _stream_ptr(stream)),
            "rlk_linear_logp_backward")
    out = (None if gh is None else gh.reshape(*lead, H), gw, gb)
    if return_grad_logits:
        ldG = -(-V // 8) * 8
        G = ws[:N * ldG * 2].view(torch.bfloat16).view(N, ldG)[:, :V]
        out = out + (G,)
    return out


class _LinearLogpGrad(torch.autograd.Function):
    """Autograd wiring of rlk_linear_logp (forward) and rlk_linear_logp_backward: the
    forward keeps lse, the backward asks the library for the gradients autograd
    needs (BF16 for hidden and weight, FP32 for the bias).  lse is returned as a
    constant: gradients flow through logp only."""

    @staticmethod
    def forward(ctx, hidden, weight, bias, target):
        with torch.no_grad():
            logp, lse = linear_logp(hidden.detach(), weight.detach(), target,
                                    None if bias is None else bias.detach())
        ctx.save_for_backward(hidden, weight, bias, target, lse)
        ctx.mark_non_differentiable(lse)
        return logp, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logp, _grad_lse):
        hidden, weight, bias, target, lse = ctx.saved_tensors
        want_h, want_w, want_b = ctx.needs_input_grad[:3]
        if grad_logp is None or not (want_h or want_w or want_b):
            return None, None, None, None
        gh, gw, gb = linear_logp_backward(hidden, weight, target, lse, grad_logp, bias,
                                          grad_hidden=want_h, grad_weight=want_w,
                                          grad_bias=bool(want_b and bias is not None))
        return gh, gw, gb, None


def linear_logp_trainable(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                          bias: torch.Tensor | None = None):
    """logp, lse as linear_logp, differentiable through logp with respect to hidden,
    weight and bias (the fused backward: G = g * (onehot(target) - softmax(z)), then
    grad_hidden = G . W and grad_weight = G^T . hidden in fixed order).  lse carries
    no gradient.  linear_logp itself stays forward-only and rejects inputs that
    require grad."""
    return _LinearLogpGrad.apply(hidden, weight, bias, target)


# ------------------------------------------------------------------ sampling
def _per_row(value, name: str, N: int, dtype):
    """(tensor or None, scalar) of a sampling setting given per row or for all rows."""
    if not isinstance(value, torch.Tensor):
        return None, value
    _require_cuda(value)
    if value.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor or a number")
    if value.numel() != N:
        raise ValueError(f"{name} must have one value per row")
    return value.reshape(-1).contiguous(), 0


@_streamed
def sample_logits(logits: torch.Tensor, uniform: torch.Tensor, *, temperature=1.0, top_k=0,
                  top_p=1.0, min_p=0.0, stream=None):
    """token (int64), logp (FP32), shaped like logits' leading dims: one token a row.

    logits [..., V] bf16 or fp32; uniform [...] fp32 or fp64, one number in [0, 1) a row (fp64
    reaches all 2^31 steps).  temperature, top_k, top_p and min_p are numbers or per-row tensors
    (float32; int32 for top_k).  Kept are the top_k largest, of those the smallest leading set
    whose probability reaches top_p, of those the ids at least min_p times as probable as the
    likeliest; logp is the token's log-probability among what is kept.  temperature 0 is greedy;
    top_k <= 0, top_p = 1 and min_p = 0 keep all.  Equal logits are ordered by id.  The token is
    a function of its row alone, bit for bit.  A row without a distribution (NaN or +inf among
    its logits or settings, or every id banned with -inf) gives token -1 and logp NaN.
    """
    _require_cuda(logits, uniform)
    if logits.dtype not in _DT:
        raise TypeError("logits must be bfloat16 or float32")
    if uniform.dtype not in (torch.float32, torch.float64):
        raise TypeError("uniform must be float32 or float64")
    lead, V = logits.shape[:-1], logits.size(-1)
    if uniform.shape != lead:
        raise ValueError("uniform must have one number per row of logits")
    z, ld = _matrix(logits.reshape(-1, V) if logits.dim() != 2 else logits, "logits")
    N = z.size(0)
    u = uniform.reshape(-1).contiguous()
    tau, tau_all = _per_row(temperature, "temperature", N, torch.float32)
    k, k_all = _per_row(top_k, "top_k", N, torch.int32)
    if k is None:                         # any whole number: the C call takes 32 bits
        k_all = max(0, min(operator.index(k_all), V))
    p, p_all = _per_row(top_p, "top_p", N, torch.float32)
    m, m_all = _per_row(min_p, "min_p", N, torch.float32)
    dev = logits.device
    token = torch.empty(N, dtype=torch.int64, device=dev)
    logp = torch.empty(N, dtype=torch.float32, device=dev)
    nb = lib().rlk_sample_logits_workspace_size(_DT[z.dtype], N, V)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    with _on(dev):
        _check(lib().rlk_sample_logits(
            _ptr(z), _DT[z.dtype], N, V, ld, _ptr(u),
            RLK_FP32 if u.dtype == torch.float32 else RLK_FP64, _ptr(tau), tau_all, _ptr(k), k_all,
            _ptr(p), p_all, _ptr(m), m_all, _ptr(token), _ptr(logp), _ptr(ws), nb,
            _stream_ptr(stream)), "rlk_sample_logits")
    return token.reshape(lead), logp.reshape(lead)


# ------------------------------------------------------------------ distillation
class _Distill:
    """A distillation call's sizes and settings, checked, and its operands: tensors with unit
    column stride and their leading dimensions."""

    __slots__ = ("lead", "h", "ldh", "w", "ldw", "ids", "ldi", "tl", "ldt", "tdt", "bias", "tlse",
                 "N", "H", "V", "K", "T")

    def __init__(self, hidden, weight, teacher_ids, teacher_logits, bias, teacher_lse, temperature):
        _require_cuda(hidden, weight, teacher_ids, teacher_logits, bias, teacher_lse)
        if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
            raise TypeError("hidden and weight must be bfloat16")
        if teacher_ids.dtype != torch.int64:
            raise TypeError("teacher_ids must be int64")
        if teacher_logits.dtype not in _DT:
            raise TypeError("teacher_logits must be bfloat16 or float32")
        shape = hidden.shape
        self.lead = shape[:-1]
        if teacher_ids.shape != teacher_logits.shape or teacher_ids.shape[:-1] != self.lead:
            raise ValueError(
                "teacher_ids and teacher_logits must be [..., K] with hidden's leading shape")
        self.H, self.K = shape[-1], teacher_ids.shape[-1]
        self.N = shape[0] if len(shape) == 2 else hidden.numel() // self.H if self.H else 0
        if weight.dim() != 2 or weight.shape[1] != self.H:
            raise ValueError("weight must be [V, H] with the hidden size H")
        self.V = weight.shape[0]
        if bias is not None:
            if bias.dtype != torch.float32 or bias.dim() != 1:
                raise TypeError("bias must be a 1-D float32 tensor")
            if bias.numel() != self.V:
                raise ValueError("bias must have V entries")
        if teacher_lse is not None:
            if teacher_lse.dtype != torch.float32 or teacher_lse.shape != self.lead:
                raise ValueError("teacher_lse must be float32 with hidden's leading shape")
        self.T = temperature
        self.tdt = _DT[teacher_logits.dtype]
        self.hold(hidden, weight, teacher_ids, teacher_logits, bias, teacher_lse)

    def hold(self, hidden, weight, teacher_ids, teacher_logits, bias, teacher_lse):
        """Takes operands of the sizes and types that were checked."""
        if len(self.lead) != 1:
            hidden = hidden.reshape(self.N, self.H)
            teacher_ids = teacher_ids.reshape(self.N, self.K)
            teacher_logits = teacher_logits.reshape(self.N, self.K)
        self.h, self.ldh = _matrix(hidden, "hidden")
        self.w, self.ldw = _matrix(weight, "weight")
        self.ids, self.ldi = _matrix(teacher_ids, "teacher_ids")
        self.tl, self.ldt = _matrix(teacher_logits, "teacher_logits")
        self.bias = None if bias is None else bias.contiguous()
        self.tlse = None if teacher_lse is None else teacher_lse.reshape(-1).contiguous()

    def drop(self):
        """Lets go of the operands."""
        self.h = self.w = self.ids = self.tl = self.bias = self.tlse = None

    def forward(self, keep_logits: bool, stream=None):
        """loss [N], lse [N], logits [N, 8 ceil(V / 8)] or None."""
        h, w, dev = self.h, self.w, self.h.device
        N, H, V, K = self.N, self.H, self.V, self.K
        loss = torch.empty(N, dtype=torch.float32, device=dev)
        lse = torch.empty(N, dtype=torch.float32, device=dev)
        ldz = -(-V // 8) * 8
        logits = torch.empty((N, ldz), dtype=torch.float32, device=dev) if keep_logits else None
        lib_ = lib()
        with _on(dev):
            n = lib_.rlk_linear_distill_workspace_size(_ptr(h), N, H, self.ldh, _ptr(w), V, self.ldw,
                                                       K)
            if n == 0:
                raise RlkError(2, "rlk_linear_distill_workspace_size")
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
            _check(lib_.rlk_linear_distill(
                _ptr(h), N, H, self.ldh, _ptr(w), V, self.ldw, _ptr(self.bias), _ptr(self.ids),
                self.ldi, _ptr(self.tl), self.tdt, self.ldt, K, _ptr(self.tlse), self.T, _ptr(loss),
                _ptr(lse), _ptr(logits), ldz, _ptr(ws), n, _stream_ptr(stream)),
                "rlk_linear_distill")
        return loss, lse, logits

    def backward(self, lse, grad_loss, logits, want, out_dtype, stream=None):
        """grad_hidden [N, H], grad_weight, grad_bias (those of `want`, else None), workspace."""
        h, w, dev = self.h, self.w, self.h.device
        N, H, V, K = self.N, self.H, self.V, self.K
        gh = torch.empty((N, H), dtype=out_dtype, device=dev) if want[0] else None
        gw = torch.empty((V, H), dtype=out_dtype, device=dev) if want[1] else None
        gb = torch.empty(V, dtype=torch.float32, device=dev) if want[2] else None
        logits, ldz = (None, 0) if logits is None else _kept_logits(logits, N, V)
        dt = _DT[out_dtype]
        lib_ = lib()
        with _on(dev):
            n = lib_.rlk_linear_distill_backward_workspace_size(_ptr(h), N, H, self.ldh, _ptr(w), V,
                                                                self.ldw, K, int(want[2]))
            if n == 0:
                raise RlkError(2, "rlk_linear_distill_backward_workspace_size")
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
            _check(lib_.rlk_linear_distill_backward(
                _ptr(h), N, H, self.ldh, _ptr(w), V, self.ldw, _ptr(self.bias), _ptr(self.ids),
                self.ldi, _ptr(self.tl), self.tdt, self.ldt, K, _ptr(self.tlse), self.T, _ptr(lse),
                _ptr(logits), ldz, _ptr(grad_loss), _ptr(gh), dt, H, _ptr(gw), dt, H, _ptr(gb),
                _ptr(ws), n, _stream_ptr(stream)), "rlk_linear_distill_backward")
        return gh, gw, gb, ws


def _kept_logits(z: torch.Tensor, N: int, V: int):
    """(logits, pitch) as the backward reads them: rows of whole 32-byte sectors, 8 ceil(V / 8)
    readable numbers each.  linear_distill's own are; others are copied into such rows."""
    width = -(-V // 8) * 8
    ld = z.stride(0) if N > 1 else width
    room = z.untyped_storage().nbytes() // 4 - z.storage_offset()
    if ld >= width and ld % 8 == 0 and z.data_ptr() % 32 == 0 and room >= (N - 1) * ld + width and \
            (V == 1 or z.stride(1) == 1):
        return z, ld
    rows = torch.zeros((N, width), dtype=torch.float32, device=z.device)
    rows[:, :V] = z[:, :V]
    return rows, width


@_streamed
def linear_distill(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor,
                   teacher_logits: torch.Tensor, bias: torch.Tensor | None = None, *,
                   temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                   return_logits: bool = False, stream=None):
    """loss, lse (FP32, shaped like hidden's leading dims): T^2 KL(teacher || student) over the
    teacher's top logits, and the student's log-sum-exp at temperature T.

    hidden [..., H] bf16, weight [V, H] bf16, bias [V] fp32 or None; teacher_ids [..., K] int64
    with the teacher's logits there, teacher_logits [..., K] bf16 or fp32.  A slot whose id is
    outside [0, V) (pad with -1) or whose logit is -inf is empty; a row without used slots has
    loss 0.  The teacher's probabilities are normalised over its slots, or by teacher_lse [...]
    fp32 (its log-sum-exp over its whole vocabulary at this temperature, 1e-4 .. 100).  With return_logits
    also the student's logits z [N, V] fp32 (bias included, not divided by T), which
    linear_distill_backward can take in place of forming them again.  Forward only: use
    linear_distill_trainable for gradients.
    """
    if hidden.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad):
        raise RuntimeError("linear_distill is forward-only: inputs that require grad are rejected")
    d = _Distill(hidden, weight, teacher_ids, teacher_logits, bias, teacher_lse, temperature)
    loss, lse, logits = d.forward(return_logits, stream)
    if len(d.lead) != 1:
        loss, lse = loss.reshape(d.lead), lse.reshape(d.lead)
    return (loss, lse, logits[:, :d.V]) if return_logits else (loss, lse)


@_streamed
def linear_distill_backward(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor,
                            teacher_logits: torch.Tensor, lse: torch.Tensor,
                            grad_loss: torch.Tensor, bias: torch.Tensor | None = None, *,
                            temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                            logits: torch.Tensor | None = None, grad_hidden: bool = True,
                            grad_weight: bool = True, grad_bias: bool | None = None,
                            out_dtype=torch.bfloat16, return_grad_logits: bool = False, stream=None):
    """(grad_hidden [..., H], grad_weight [V, H], grad_bias [V] | None) of linear_distill's loss.

    lse is the forward's lse; grad_loss is dL/dloss (one value a row); logits are those of
    linear_distill(..., return_logits=True), or None to form them again (the same bits).  With
    return_grad_logits, also returns G = dL/dz as the BF16 [N, V] view the products read.
    """
    d = _Distill(hidden, weight, teacher_ids, teacher_logits, bias, teacher_lse, temperature)
    _require_cuda(lse, grad_loss, logits)
    l1 = lse.reshape(-1).contiguous().float()
    g1 = grad_loss.reshape(-1).contiguous().float()
    if l1.numel() != d.N or g1.numel() != d.N:
        raise ValueError("lse and grad_loss must have one value per hidden row")
    if logits is not None and (logits.dtype != torch.float32 or tuple(logits.shape) != (d.N, d.V)):
        raise ValueError("logits must be those of linear_distill(..., return_logits=True)")
    if grad_bias is None:
        grad_bias = bias is not None
    gh, gw, gb, ws = d.backward(l1, g1, logits, (grad_hidden, grad_weight, grad_bias), out_dtype,
                                stream)
    out = (None if gh is None else gh.reshape(*d.lead, d.H), gw, gb)
    if return_grad_logits:
        ldG = -(-d.V // 8) * 8
        out = out + (ws[:d.N * ldG * 2].view(torch.bfloat16).view(d.N, ldG)[:, :d.V],)
    return out


# Most bytes of FP32 logits that linear_distill_trainable keeps from the forward for the
# backward.  Kept, the backward reads 4 bytes a logit where it would spend 2 H operations:
# forward and backward of N = 2048, H = 4096, V = 151936 take 5.0 ms with the 1.2 GB kept and
# 6.2 ms without; N = 255, H = 2048, V = 32003 16 us of G against 38 us.  8 GiB is 14,000 rows
# of that vocabulary, a thirtieth of the GPU's memory.
KEEP_LOGITS_BYTES = 8 << 30


class _LinearDistillGrad(torch.autograd.Function):
    """Autograd wiring of rlk_linear_distill and rlk_linear_distill_backward; lse is returned
    as a constant and the teacher's tensors carry no gradient.  Whatever the backward needs is
    saved with autograd, the kept logits too, which frees it after the backward."""

    @staticmethod
    def forward(ctx, hidden, weight, bias, teacher_ids, teacher_logits, teacher_lse, temperature,
                keep_logits):
        d = _Distill(hidden, weight, teacher_ids, teacher_logits, bias, teacher_lse, temperature)
        if keep_logits is None:
            keep_logits = 4 * d.N * d.V <= KEEP_LOGITS_BYTES
        loss, lse, logits = d.forward(keep_logits)
        ctx.save_for_backward(hidden, weight, bias, teacher_ids, teacher_logits, teacher_lse, lse,
                              logits)
        d.drop()
        ctx.call = d
        ctx.mark_non_differentiable(lse)
        if len(d.lead) != 1:
            loss, lse = loss.reshape(d.lead), lse.reshape(d.lead)
            ctx.mark_non_differentiable(lse)
        return loss, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, _grad_lse):
        want_h, want_w, want_b = ctx.needs_input_grad[:3]
        if grad_loss is None or not (want_h or want_w or want_b):
            return (None,) * 8
        hidden, weight, bias, ids, teacher_logits, teacher_lse, lse, logits = ctx.saved_tensors
        d = ctx.call
        d.hold(hidden, weight, ids, teacher_logits, bias, teacher_lse)
        if grad_loss.dim() != 1 or not grad_loss.is_contiguous():
            grad_loss = grad_loss.reshape(-1).contiguous()
        gh, gw, gb, _ = d.backward(lse, grad_loss, logits, (want_h, want_w, want_b),
                                   torch.bfloat16)
        d.drop()
        if gh is not None and hidden.dim() != 2:
            gh = gh.reshape(hidden.shape)
        return gh, gw, gb, None, None, None, None, None


def linear_distill_trainable(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor,
                             teacher_logits: torch.Tensor, bias: torch.Tensor | None = None, *,
                             temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                             keep_logits: bool | None = None):
    """loss, lse as linear_distill, differentiable through loss with respect to hidden, weight and
    bias (BF16 gradients of hidden and weight, FP32 of the bias).  lse carries no gradient.

    keep_logits: hold the logits in FP32 (4 N V bytes) from the forward to the backward, which
    otherwise forms them again; the gradients' bits are the same.  None: up to
    KEEP_LOGITS_BYTES.  Where nothing asks for a gradient they are not kept.
    """
    if not (torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad or
                                         (bias is not None and bias.requires_grad))):
        keep_logits = False
    return _LinearDistillGrad.apply(hidden, weight, bias, teacher_ids, teacher_logits, teacher_lse,
                                    temperature, keep_logits)


# ------------------------------------------------------------------ det_gemm
def _gemm_ws(op, x, xdt, xld, y, ydt, yld, device):
    n = lib().rlk_det_gemm_workspace_size(op, _ptr(x), xdt, x.size(0), x.size(1), xld,
                                          _ptr(y), ydt, y.size(0), y.size(1), yld)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device), n


def _flatten_rows(t: torch.Tensor) -> torch.Tensor:
    return t.reshape(-1, t.size(-1)) if t.dim() != 2 else t


@_streamed
def det_gemm_fwd(A: torch.Tensor, B: torch.Tensor, out_dtype=torch.bfloat16, *, stream=None):
    """C = A . B; A [..., M, K] bf16 (leading dims flattened into rows), B [K, N] bf16."""
    _require_cuda(A, B)
    lead = A.shape[:-1]
    A2, lda = _matrix(_flatten_rows(A), "A")
    B2, ldb = _matrix(B, "B")
    M, K = A2.shape
    if B2.size(0) != K:
        raise ValueError("A and B disagree on K")
    N = B2.size(1)
    C = torch.empty(M, N, dtype=out_dtype, device=A.device)
    with _on(A.device):
        ws, n = _gemm_ws(RLK_GEMM_FWD, A2, RLK_BF16, lda, B2, RLK_BF16, ldb, A.device)
        _check(lib().rlk_det_gemm_fwd(_ptr(A2), M, K, lda, _ptr(B2), N, ldb, _ptr(C), _DT[out_dtype],
                                      N, _ptr(ws), n, _stream_ptr(stream)), "rlk_det_gemm_fwd")
    return C.reshape(*lead, N)


@_streamed
def det_gemm_da(dC: torch.Tensor, B: torch.Tensor, out_dtype=torch.bfloat16, *, stream=None):
    """dA = dC . B^T; dC [..., M, N] bf16 or fp32 (fp32 is rounded to bf16 first), B [K, N]."""
    _require_cuda(dC, B)
    lead = dC.shape[:-1]
    d2, lddc = _matrix(_flatten_rows(dC), "dC")
    B2, ldb = _matrix(B, "B")
    M, N = d2.shape
    K = B2.size(0)
    if B2.size(1) != N:
        raise ValueError("dC and B disagree on N")
    dA = torch.empty(M, K, dtype=out_dtype, device=dC.device)
    with _on(dC.device):
        ws, n = _gemm_ws(RLK_GEMM_DA, d2, _DT[d2.dtype], lddc, B2, RLK_BF16, ldb, dC.device)
        _check(lib().rlk_det_gemm_da(_ptr(d2), _DT[d2.dtype], M, N, lddc, _ptr(B2), K, ldb, _ptr(dA),
                                     _DT[out_dtype], K, _ptr(ws), n, _stream_ptr(stream)),
               "rlk_det_gemm_da")
    return dA.reshape(*lead, K)


@_streamed
def det_gemm_db(A: torch.Tensor, dC: torch.Tensor, out_dtype=torch.bfloat16, *, stream=None):
    """dB = A^T . dC summed over every row; A [..., M, K] bf16, dC [..., M, N] bf16 or fp32."""
    _require_cuda(A, dC)
    A2, lda = _matrix(_flatten_rows(A), "A")
    d2, lddc = _matrix(_flatten_rows(dC), "dC")
    M, K = A2.shape
    if d2.size(0) != M:
        raise ValueError("A and dC disagree on M")
    N = d2.size(1)
    dB = torch.empty(K, N, dtype=out_dtype, device=A.device)
    with _on(A.device):
        ws, n = _gemm_ws(RLK_GEMM_DB, A2, RLK_BF16, lda, d2, _DT[d2.dtype], lddc, A.device)
        _check(lib().rlk_det_gemm_db(_ptr(A2), M, K, lda, _ptr(d2), _DT[d2.dtype], N, lddc, _ptr(dB),
                                     _DT[out_dtype], N, _ptr(ws), n, _stream_ptr(stream)),
               "rlk_det_gemm_db")
    return dB


@_streamed
def det_gemm_fwd_accum_fp32_(C: torch.Tensor, A: torch.Tensor, B: torch.Tensor, *, stream=None):
    """In place: C (fp32 [M, N]) += A . B, the product formed as by det_gemm_fwd and
    added to C once, after the full K reduction."""
    _require_cuda(C, A, B)
    if C.dtype != torch.float32:
        raise TypeError("C must be float32")
    A2, lda = _matrix(A, "A")
    B2, ldb = _matrix(B, "B")
    if C.dim() != 2 or C.stride(1) != 1:
        raise ValueError("C must be a 2-D row-major tensor (it is updated in place)")
    M, K = A2.shape
    N = B2.size(1)
    if B2.size(0) != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch")
    ldc = C.stride(0) if M > 1 else N
    with _on(A.device):
        ws, n = _gemm_ws(RLK_GEMM_FWD_ACCUM, A2, RLK_BF16, lda, B2, RLK_BF16, ldb, A.device)
        _check(lib().rlk_det_gemm_fwd_accum_fp32(_ptr(A2), M, K, lda, _ptr(B2), N, ldb, _ptr(C), ldc,
                                                 _ptr(ws), n, _stream_ptr(stream)),
               "rlk_det_gemm_fwd_accum_fp32")
    return C


@_streamed
def det_linear(X: torch.Tensor, W: torch.Tensor, out_dtype=torch.bfloat16, *, stream=None):
    """Y = X . W^T with the weight stored [N, K]; X [..., K] bf16 (leading dims are rows)."""
    _require_cuda(X, W)
    lead = X.shape[:-1]
    X2, ldx = _matrix(_flatten_rows(X), "X")
    W2, ldw = _matrix(W, "W")
    M, K = X2.shape
    N = W2.size(0)
    if W2.size(1) != K:
        raise ValueError("W must be [N, K]")
    Y = torch.empty(M, N, dtype=out_dtype, device=X.device)
    with _on(X.device):
        ws, n = _gemm_ws(RLK_GEMM_LINEAR_FWD, X2, RLK_BF16, ldx, W2, RLK_BF16, ldw, X.device)
        _check(lib().rlk_det_linear_fwd(_ptr(X2), M, K, ldx, _ptr(W2), N, ldw, _ptr(Y), _DT[out_dtype],
                                        N, _ptr(ws), n, _stream_ptr(stream)), "rlk_det_linear_fwd")
    return Y.reshape(*lead, N)


@_streamed
def det_linear_dx(dY: torch.Tensor, W: torch.Tensor, out_dtype=torch.bfloat16, *, stream=None):
    """dX = dY . W for Y = X . W^T; dY [..., N] bf16 or fp32 (fp32 rounded to bf16 first)."""
    _require_cuda(dY, W)
    lead = dY.shape[:-1]
    d2, lddy = _matrix(_flatten_rows(dY), "dY")
    W2, ldw = _matrix(W, "W")
    M, N = d2.shape
    K = W2.size(1)
    if W2.size(0) != N:
        raise ValueError("W must be [N, K]")
    dX = torch.empty(M, K, dtype=out_dtype, device=dY.device)
    with _on(dY.device):
        ws, n = _gemm_ws(RLK_GEMM_LINEAR_DX, d2, _DT[d2.dtype], lddy, W2, RLK_BF16, ldw, dY.device)
        _check(lib().rlk_det_linear_dx(_ptr(d2), _DT[d2.dtype], M, N, lddy, _ptr(W2), K, ldw, _ptr(dX),
                                       _DT[out_dtype], K, _ptr(ws), n, _stream_ptr(stream)),
               "rlk_det_linear_dx")
    return dX.reshape(*lead, K)


@_streamed
def det_linear_dw(dY: torch.Tensor, X: torch.Tensor, out_dtype=torch.bfloat16, *, stream=None):
    """dW [N, K] = dY^T . X summed over every row; dY [..., N] bf16 or fp32, X [..., K] bf16."""
    _require_cuda(dY, X)
    d2, lddy = _matrix(_flatten_rows(dY), "dY")
    X2, ldx = _matrix(_flatten_rows(X), "X")
    M, N = d2.shape
    if X2.size(0) != M:
        raise ValueError("dY and X disagree on the row count")
    K = X2.size(1)
    dW = torch.empty(N, K, dtype=out_dtype, device=dY.device)
    with _on(dY.device):
        ws, n = _gemm_ws(RLK_GEMM_LINEAR_DW, d2, _DT[d2.dtype], lddy, X2, RLK_BF16, ldx, dY.device)
        _check(lib().rlk_det_linear_dw(_ptr(d2), _DT[d2.dtype], M, N, lddy, _ptr(X2), K, ldx, _ptr(dW),
                                       _DT[out_dtype], K, _ptr(ws), n, _stream_ptr(stream)),
               "rlk_det_linear_dw")
    return dW


def _two_grads(fn, size_fn, g, x, w, out_shapes, out_dtype, want, stream):
    g2, ldg = _matrix(_flatten_rows(g), "grad")
    x2, ldx = _matrix(_flatten_rows(x), "x")
    w2, ldw = _matrix(w, "w")
    M, N = g2.shape
    K = x2.size(1)
    dev = g.device
    outs = [torch.empty(*shp, dtype=out_dtype, device=dev) if want[i] else None
            for i, shp in enumerate(out_shapes(M, N, K))]
    gdt = _DT[g2.dtype]
    with _on(dev):
        n = size_fn(_ptr(g2), gdt, M, N, ldg, _ptr(x2), K, ldx, _ptr(w2), ldw)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
        dt = _DT[out_dtype]
        lds = [o.size(1) if o is not None else 1 for o in outs]
        _check(fn(_ptr(g2), gdt, M, N, ldg, _ptr(x2), K, ldx, _ptr(w2), ldw, _ptr(outs[0]), dt,
                  lds[0], _ptr(outs[1]), dt, lds[1], _ptr(ws), n, _stream_ptr(stream)),
               fn.__name__)
    return tuple(outs)


@_streamed
def det_gemm_backward(dC: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                      out_dtype=torch.bfloat16, *, grad_a: bool = True, grad_b: bool = True,
                      stream=None):
    """(dA = dC . B^T, dB = A^T . dC) for C = A . B, from one dC (bf16 or fp32; an fp32
    dC is rounded to bf16 once and shared by both products).  Bitwise equal to
    det_gemm_da and det_gemm_db."""
    _require_cuda(dC, A, B)
    lib_ = lib()
    return _two_grads(lib_.rlk_det_gemm_backward, lib_.rlk_det_gemm_backward_workspace_size, dC, A,
                      B, lambda M, N, K: ((M, K), (K, N)), out_dtype, (grad_a, grad_b),
                      stream)


@_streamed
def det_linear_backward(dY: torch.Tensor, X: torch.Tensor, W: torch.Tensor,
                        out_dtype=torch.bfloat16, *, grad_x: bool = True, grad_w: bool = True,
                        stream=None):
    """(dX = dY . W, dW = dY^T . X) for Y = X . W^T with W [N, K], from one dY (an fp32 dY
    is rounded to bf16 once).  Bitwise equal to det_linear_dx and det_linear_dw."""
    _require_cuda(dY, X, W)
    lib_ = lib()
    return _two_grads(lib_.rlk_det_linear_backward, lib_.rlk_det_linear_backward_workspace_size, dY,
                      X, W, lambda M, N, K: ((M, K), (N, K)), out_dtype, (grad_x, grad_w),
                      stream)


# ------------------------------------------------------------------ autograd wiring
class _DetGemmGrad(torch.autograd.Function):
    """C = A . B under autograd: det_gemm_fwd forward; det_gemm_backward for the
    gradients autograd needs (an FP32 dC, from an FP32-output forward, is rounded
    to BF16 once before both products)."""

    @staticmethod
    def forward(ctx, A, B, out_dtype):
        with torch.no_grad():
            C = det_gemm_fwd(A.detach(), B.detach(), out_dtype)
        ctx.save_for_backward(A, B)
        return C

    @staticmethod
    @once_differentiable
    def backward(ctx, dC):
        A, B = ctx.saved_tensors
        want_a, want_b = ctx.needs_input_grad[:2]
        if not (want_a or want_b):
            return None, None, None
        dA, dB = det_gemm_backward(dC, A, B, grad_a=want_a, grad_b=want_b)
        return (None if dA is None else dA.reshape(A.shape)), dB, None


class _DetLinearGrad(torch.autograd.Function):
    """Y = X . W^T (W stored [N, K]) under autograd: det_linear forward,
    det_linear_backward for dX and dW."""

    @staticmethod
    def forward(ctx, X, W, out_dtype):
        with torch.no_grad():
            Y = det_linear(X.detach(), W.detach(), out_dtype)
        ctx.save_for_backward(X, W)
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, W = ctx.saved_tensors
        want_x, want_w = ctx.needs_input_grad[:2]
        if not (want_x or want_w):
            return None, None, None
        dX, dW = det_linear_backward(dY, X, W, grad_x=want_x, grad_w=want_w)
        return (None if dX is None else dX.reshape(X.shape)), dW, None


def det_gemm_trainable(A: torch.Tensor, B: torch.Tensor, out_dtype=torch.bfloat16):
    """det_gemm_fwd(A, B) differentiable with respect to A and B (BF16 gradients from
    the fixed-order det_gemm backward products)."""
    return _DetGemmGrad.apply(A, B, out_dtype)


def det_linear_trainable(X: torch.Tensor, W: torch.Tensor, out_dtype=torch.bfloat16):
    """det_linear(X, W) differentiable with respect to X and W: a deterministic,
    batch-invariant stand-in for a bias-free nn.Linear forward and backward."""
    return _DetLinearGrad.apply(X, W, out_dtype)
