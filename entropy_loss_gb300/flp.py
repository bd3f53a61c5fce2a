"""ctypes binding of ``libflp.so`` (the C ABI in ``include/flp.h``).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch is used for device memory, streams and dtype bookkeeping.
Loading fails loudly (``FlpError``) when the library is missing; there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libflp.so")

FLP_OK = 0
FLP_ERR_INVALID_ARG = 1
FLP_ERR_UNSUPPORTED = 2
FLP_ERR_WORKSPACE = 3
FLP_ERR_CUDA = 4
FLP_ERR_BAD_TARGET = 5
FLP_ERR_TIMEOUT = 6
FLP_F32 = 0
FLP_BF16 = 1

EXPORTS = ("flp_workspace_query", "flp_workspace_query_ex", "flp_forward", "flp_backward", "flp_get_error",
           "flp_set_phase_events", "flp_status_string", "flp_last_error_message",
           "flp_forward_noalloc", "flp_selftest_wait_timeout", "flp_loss", "flp_backward_ex",
           "flp_backward_plan", "flp_backward_schedule", "flp_selftest_dependency_timeout",
           "flp_selftest_dz_wait_timeout", "flp_policy_loss", "flp_layer_norm", "flp_layer_norm_workspace",
           "flp_layer_norm_backward", "flp_checkpoint_pack", "flp_checkpoint_unpack",
           "flp_checkpoint_weight_grad_workspace", "flp_checkpoint_weight_grad", "flp_selftest_weight_grad_timeout",
           "flp_balance_loss_workspace", "flp_balance_loss", "flp_balance_loss_ex")
FLP_LOSS_NLL_MEAN = 1
FLP_LOSS_CLIPPED_SURROGATE = 2
FLP_LOSS_NLL_SUM = 3
FLP_IS_TOKEN = 0
FLP_IS_SEQUENCE = 1
FLP_AGG_TOKEN_MEAN = 0
FLP_AGG_SEQUENCE_MEAN = 1
FLP_AGG_SUM_OVER = 2
SELFTEST_WORKSPACE_BYTES = 1 << 20
SELFTEST_WEIGHT_GRAD_BYTES = 3 << 20
SELFTEST_WEIGHT_GRAD_OUTPUT_OFFSET = 2 << 20
SELFTEST_OUTPUT_OFFSET = 768 << 10  # the forward self-test's logprob, lse, entropy (fp32 [256] each)
STATIC_SCRATCH_BYTES = 16 << 20
FLP_BWD_AUTO = 0
FLP_BWD_SPLIT = 1
FLP_BWD_FUSED = 2
FLP_BWD_VSPLIT = 3
SCHEDULES = {"auto": FLP_BWD_AUTO, "split": FLP_BWD_SPLIT, "fused": FLP_BWD_FUSED,
             "vsplit": FLP_BWD_VSPLIT}
# phase k of flp_set_phase_events is recorded around events 2k, 2k+1; the
# backward records phase 2 (split: first wave's dZ launch; vsplit: first
# vocabulary chunk's; fused: the whole backward launch) and, except for the
# fused schedule, phase 3 (the matching dX and dW launch)
PHASES = ("fwd", "merge", "dz", "bwd_gemm")


class FlpError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load the CUDA library (built by ``entropy_loss_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FlpError(FLP_ERR_CUDA, f"{path} is missing: build it with entropy_loss_gb300.build.build()")
    lib = ctypes.CDLL(path)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.flp_workspace_query.argtypes = [i64, i64, i64, i32, ctypes.POINTER(ctypes.c_size_t),
                                        ctypes.POINTER(ctypes.c_size_t)]
    lib.flp_workspace_query_ex.argtypes = [i64, i64, i64, i32, i64, ctypes.POINTER(ctypes.c_size_t),
                                           ctypes.POINTER(ctypes.c_size_t)]
    lib.flp_forward.argtypes = [p, p, p, i64, i64, i64, i64, ctypes.c_float, i32, p, p, p, p,
                                ctypes.c_size_t, p]
    lib.flp_backward.argtypes = [p, p, p, i64, i64, i64, i64, ctypes.c_float, i32, p, p, p, p, p,
                                 i32, p, i32, i32, p, ctypes.c_size_t, p]
    lib.flp_backward_ex.argtypes = [p, p, p, i64, i64, i64, i64, ctypes.c_float, i32, p, p, p, p,
                                    p, i32, p, i32, i32, p, ctypes.c_size_t, i32, p]
    lib.flp_backward_ex.restype = i32
    lib.flp_backward_plan.argtypes = [i64, i64, i64, ctypes.c_size_t, i32,
                                      ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                                      ctypes.POINTER(ctypes.c_int)]
    lib.flp_backward_plan.restype = i32
    lib.flp_backward_schedule.argtypes = [i64, i64, i64, ctypes.c_size_t, i32, i32,
                                          ctypes.POINTER(ctypes.c_int32), i64,
                                          ctypes.POINTER(ctypes.c_int64)]
    lib.flp_backward_schedule.restype = i32
    lib.flp_forward_noalloc.argtypes = [p, p, p, i64, i64, i64, i64, ctypes.c_float, i32, p, p, p,
                                        p]
    lib.flp_forward_noalloc.restype = i32
    lib.flp_selftest_wait_timeout.argtypes = [p, ctypes.c_size_t, i32, i64, p]
    lib.flp_selftest_wait_timeout.restype = i32
    lib.flp_selftest_dependency_timeout.argtypes = [p, ctypes.c_size_t, i32, i64, p]
    lib.flp_selftest_dependency_timeout.restype = i32
    lib.flp_selftest_dz_wait_timeout.argtypes = [p, ctypes.c_size_t, i32, i64, p]
    lib.flp_selftest_dz_wait_timeout.restype = i32
    lib.flp_loss.argtypes = [p, p, i64, i64, i32, p, p, p, ctypes.c_float, ctypes.c_float,
                             ctypes.c_float, p, p, p, p]
    lib.flp_loss.restype = i32
    lib.flp_policy_loss.argtypes = [p, p, i64, i64, p, i64, p, p, p, ctypes.c_float, ctypes.c_float,
                                    ctypes.c_float, i32, i32, ctypes.c_double, p, p, p, p]
    lib.flp_policy_loss.restype = i32
    f32, size = ctypes.c_float, ctypes.POINTER(ctypes.c_size_t)
    for name, args in (
            ("flp_layer_norm", [p, i64, i32, p, p, i32, i64, i64, f32, p, i64, p, p, p, p, p]),
            ("flp_layer_norm_workspace", [i64, i64, size]),
            ("flp_layer_norm_backward", [p, i64, p, i64, p, p, i32, p, i32, p, p, i64, i64, p, i64, p, p, p,
                                         ctypes.c_size_t, p]),
            ("flp_checkpoint_pack", [p, i64, i32, i64, i64, p, p, p]),
            ("flp_checkpoint_unpack", [p, p, i64, i64, p, i64, i32, p]),
            ("flp_checkpoint_weight_grad_workspace", [p, i64, i64, i64, i64, i32, size]),
            ("flp_checkpoint_weight_grad", [p, i64, p, p, i64, i64, i64, p, i32, i32, p, ctypes.c_size_t, p]),
            ("flp_selftest_weight_grad_timeout", [p, ctypes.c_size_t, i32, i32, i64, p]),
            ("flp_balance_loss_workspace", [i64, i64, size]),
            ("flp_balance_loss", [p, i64, i32, p, p, i64, i64, i64, f32, p, p, p, p, ctypes.c_size_t, p]),
            ("flp_balance_loss_ex", [p, i64, i32, p, p, i64, i64, i64, f32, p, p, i32, p, p, ctypes.c_size_t, p])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, i32
    lib.flp_get_error.argtypes = [p, p]
    lib.flp_set_phase_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), i32]
    lib.flp_set_phase_events.restype = i32
    lib.flp_status_string.argtypes = [i32]
    lib.flp_status_string.restype = ctypes.c_char_p
    lib.flp_last_error_message.argtypes = []
    lib.flp_last_error_message.restype = ctypes.c_char_p
    for name in ("flp_workspace_query", "flp_workspace_query_ex", "flp_forward", "flp_backward",
                 "flp_get_error"):
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


def _check(status: int, what: str) -> None:
    if status != FLP_OK:
        lib = load()
        msg = lib.flp_status_string(status).decode()
        detail = lib.flp_last_error_message().decode()
        raise FlpError(status, f"{what}: {msg}" + (f" ({detail})" if detail else ""))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def workspace_query(M: int, H: int, V: int, compute_entropy: bool = True, chunk_rows: int = 0):
    """(forward bytes, backward bytes) on the current device; chunk_rows > 0
    sizes the backward for row waves of that many rows (flp_workspace_query_ex),
    else for the default waves (flp_workspace_query)."""
    f = ctypes.c_size_t(0)
    b = ctypes.c_size_t(0)
    lib = load()
    if chunk_rows > 0:
        _check(lib.flp_workspace_query_ex(M, H, V, int(compute_entropy), chunk_rows, ctypes.byref(f),
                                          ctypes.byref(b)), "flp_workspace_query_ex")
    else:
        _check(lib.flp_workspace_query(M, H, V, int(compute_entropy), ctypes.byref(f), ctypes.byref(b)),
               "flp_workspace_query")
    return f.value, b.value


def alloc_workspace(M: int, H: int, V: int, compute_entropy: bool = True, chunk_rows: int = 0,
                    device=None) -> torch.Tensor:
    """One uint8 device buffer large enough for both forward and backward."""
    f, b = workspace_query(M, H, V, compute_entropy, chunk_rows)
    return torch.empty(max(f, b), dtype=torch.uint8, device=device or "cuda")


def _need(t, dtype, shape, name):
    """t must be a contiguous CUDA tensor of `dtype` (or one of a tuple of
    dtypes) and `shape`: the C ABI sees only its data pointer."""
    ok_dtype = t.dtype in dtype if isinstance(dtype, tuple) else t.dtype == dtype
    if not ok_dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _need_opt(t, dtype, shape, name):
    if t is not None:
        _need(t, dtype, shape, name)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _workspace(t):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("workspace: expected a contiguous CUDA tensor")
    return _ptr(t), _nbytes(t)


def forward(X, W, y, *, ignore_index: int = -100, scale: float = 1.0, compute_entropy: bool = True,
            workspace=None, logprob=None, lse=None, entropy=None, stream=None):
    """Per-row (logprob, lse, entropy-or-None) of softmax(scale * X W^T)."""
    M, H = X.shape
    V = W.shape[0]
    _need(X, torch.bfloat16, (M, H), "X")
    _need(W, torch.bfloat16, (V, H), "W")
    _need(y, torch.int64, (M,), "targets")
    dev = X.device
    logprob = torch.empty(M, dtype=torch.float32, device=dev) if logprob is None else logprob
    lse = torch.empty(M, dtype=torch.float32, device=dev) if lse is None else lse
    if compute_entropy and entropy is None:
        entropy = torch.empty(M, dtype=torch.float32, device=dev)
    if not compute_entropy:
        entropy = None
    for t, name in ((logprob, "logprob"), (lse, "lse"), (entropy, "entropy")):
        _need_opt(t, torch.float32, (M,), name)
    if workspace is None:
        workspace = alloc_workspace(M, H, V, compute_entropy, device=dev)
    ws_ptr, ws_bytes = _workspace(workspace)
    _check(load().flp_forward(_ptr(X), _ptr(W), _ptr(y), M, H, V, ignore_index, float(scale),
                              int(compute_entropy), _ptr(logprob), _ptr(lse), _ptr(entropy),
                              ws_ptr, ws_bytes, _stream(stream)), "flp_forward")
    return logprob, lse, entropy


def forward_noalloc(X, W, y, logprob, lse, entropy=None, *, ignore_index: int = -100,
                    scale: float = 1.0, compute_entropy: bool = True, stream=None):
    """flp_forward_noalloc: the forward without a workspace, for callers that
    cannot allocate device memory; its scratch is the library's fixed 16 MiB
    device array, shared by every call (calls that overlap on the GPU race).
    The outputs are caller-provided; nothing is allocated here."""
    M, H = X.shape
    V = W.shape[0]
    _need(X, torch.bfloat16, (M, H), "X")
    _need(W, torch.bfloat16, (V, H), "W")
    _need(y, torch.int64, (M,), "targets")
    _need(logprob, torch.float32, (M,), "logprob")
    _need(lse, torch.float32, (M,), "lse")
    if compute_entropy:
        _need(entropy, torch.float32, (M,), "entropy")
    _check(load().flp_forward_noalloc(_ptr(X), _ptr(W), _ptr(y), M, H, V, ignore_index,
                                      float(scale), int(compute_entropy), _ptr(logprob), _ptr(lse),
                                      _ptr(entropy if compute_entropy else None), _stream(stream)),
           "flp_forward_noalloc")
    return logprob, lse, entropy


def backward_plan(M: int, H: int, V: int, workspace_bytes: int, schedule: str = "auto"):
    """(wave rows, waves, schedule name) that `backward` runs with for this
    workspace size (for "vsplit", waves counts vocabulary chunks); host
    arithmetic only."""
    rows = ctypes.c_int64(0)
    waves = ctypes.c_int64(0)
    used = ctypes.c_int(0)
    _check(load().flp_backward_plan(M, H, V, workspace_bytes, SCHEDULES[schedule],
                                    ctypes.byref(rows), ctypes.byref(waves), ctypes.byref(used)),
           "flp_backward_plan")
    name = {v: k for k, v in SCHEDULES.items()}[used.value]
    return rows.value, waves.value, name


def backward_schedule(M: int, H: int, V: int, workspace_bytes: int, schedule: str = "auto",
                      pairs: int = 76):
    """The backward's units in ticket order as an int32 array of rows
    (launch, kind, wave, a, b); kind 0 dZ, 1 dX, 2 dW (see include/flp.h)."""
    import numpy as np
    lib = load()
    n = ctypes.c_int64(0)
    _check(lib.flp_backward_schedule(M, H, V, workspace_bytes, SCHEDULES[schedule], pairs, None, 0,
                                     ctypes.byref(n)), "flp_backward_schedule")
    out = np.zeros((n.value, 5), dtype=np.int32)
    _check(lib.flp_backward_schedule(M, H, V, workspace_bytes, SCHEDULES[schedule], pairs,
                                     out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), n.value,
                                     ctypes.byref(n)), "flp_backward_schedule")
    return out


def backward(X, W, y, lse, entropy, grad_logprob, grad_entropy, *, ignore_index: int = -100,
             scale: float = 1.0, compute_entropy: bool = True, dX=None, dW=None,
             dx_dtype=torch.bfloat16, dw_dtype=torch.float32, accumulate_dW: bool = False,
             workspace=None, schedule: str = "auto", stream=None):
    """(dX, dW) for upstream gradients of logprob and entropy (None = zero).
    dW may be fp32 (accumulated in fp32 across waves) or bf16 (one wave only).
    schedule: "auto", "split" (per wave a dZ launch, then a dX/dW launch),
    "fused" (one persistent launch for every wave) or "vsplit" (all rows at
    once, the vocabulary in chunks: dX accumulates over the chunks in fp32)."""
    M, H = X.shape
    V = W.shape[0]
    _need(X, torch.bfloat16, (M, H), "X")
    _need(W, torch.bfloat16, (V, H), "W")
    _need(y, torch.int64, (M,), "targets")
    _need(lse, torch.float32, (M,), "lse")
    if compute_entropy:
        _need(entropy, torch.float32, (M,), "entropy")
    _need_opt(grad_logprob, torch.float32, (M,), "grad_logprob")
    if compute_entropy:
        _need_opt(grad_entropy, torch.float32, (M,), "grad_entropy")
    if schedule not in SCHEDULES:
        raise ValueError(f"schedule must be one of {sorted(SCHEDULES)}")
    dev = X.device
    if dX is None:
        dX = torch.empty(M, H, dtype=dx_dtype, device=dev)
    if dW is None:
        dW = torch.empty(V, H, dtype=dw_dtype, device=dev)
    _need(dX, (torch.bfloat16, torch.float32), (M, H), "dX")
    _need(dW, (torch.bfloat16, torch.float32), (V, H), "dW")
    dxt = FLP_F32 if dX.dtype == torch.float32 else FLP_BF16
    dwt = FLP_F32 if dW.dtype == torch.float32 else FLP_BF16
    if workspace is None:
        workspace = alloc_workspace(M, H, V, compute_entropy, device=dev)
    ws_ptr, ws_bytes = _workspace(workspace)
    _check(load().flp_backward_ex(_ptr(X), _ptr(W), _ptr(y), M, H, V, ignore_index, float(scale),
                                  int(compute_entropy), _ptr(lse),
                                  _ptr(entropy if compute_entropy else None), _ptr(grad_logprob),
                                  _ptr(grad_entropy if compute_entropy else None), _ptr(dX), dxt,
                                  _ptr(dW), dwt, int(accumulate_dW), ws_ptr, ws_bytes,
                                  SCHEDULES[schedule], _stream(stream)),
           "flp_backward_ex")
    return dX, dW


def set_phase_events(events) -> None:
    """Instrument the next calls on this thread: `events` is a list of up to 10
    torch.cuda.Event (or None) recorded around the kernel phases (start, stop)
    of PHASES in order; None turns the instrumentation off."""
    if not events:
        _check(load().flp_set_phase_events(None, 0), "flp_set_phase_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[(e.cuda_event if e is not None else None)
                                            for e in events])
    _check(load().flp_set_phase_events(arr, len(events)), "flp_set_phase_events")


def selftest_wait_timeout(stall_after: int, wait_limit_ns: int, workspace=None, stream=None) -> int:
    """Run the forward kernel with its producers stopped after `stall_after`
    stages (< 0: no stall) and every wait bounded by `wait_limit_ns`; returns
    the error status the run leaves (FLP_ERR_TIMEOUT when the stall was
    detected, FLP_OK for a normal run)."""
    if workspace is None:
        workspace = torch.empty(SELFTEST_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return int(load().flp_selftest_wait_timeout(_ptr(workspace), _nbytes(workspace), stall_after,
                                                wait_limit_ns, _stream(stream)))


def selftest_dz_wait_timeout(stall_after: int, wait_limit_ns: int, workspace=None, stream=None) -> int:
    """Run the backward's dZ kernel on one internal 256 x 512 tile with its
    producers stopped after `stall_after` stages (< 0: no stall) and every wait
    bounded by `wait_limit_ns`; returns the error status the run leaves
    (FLP_ERR_TIMEOUT when the stall was detected, FLP_OK for a normal run)."""
    if workspace is None:
        workspace = torch.empty(SELFTEST_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return int(load().flp_selftest_dz_wait_timeout(_ptr(workspace), _nbytes(workspace), stall_after,
                                                   wait_limit_ns, _stream(stream)))


def selftest_dependency_timeout(broken: bool, wait_limit_ns: int, workspace=None, stream=None) -> int:
    """Run one fused-schedule backward launch on a small internal problem;
    with `broken` its dX tile waits on a dZ tile that is never scheduled, so
    the dependency wait must give up after `wait_limit_ns`.  Returns the error
    status the run leaves (FLP_ERR_TIMEOUT when broken, FLP_OK otherwise)."""
    if workspace is None:
        workspace = torch.empty(SELFTEST_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return int(load().flp_selftest_dependency_timeout(_ptr(workspace), _nbytes(workspace),
                                                      int(bool(broken)), wait_limit_ns,
                                                      _stream(stream)))


def selftest_weight_grad_timeout(odd: bool, stall_after: int, wait_limit_ns: int, workspace=None, stream=None) -> int:
    """Run a small weight gradient with its producers stopped after
    `stall_after` 64-row blocks (< 0: no stall) and every wait bounded by
    `wait_limit_ns`; with `odd` its dW is written through partial tiles.
    Returns the error status the run leaves."""
    if workspace is None:
        workspace = torch.empty(SELFTEST_WEIGHT_GRAD_BYTES, dtype=torch.uint8, device="cuda")
    return int(load().flp_selftest_weight_grad_timeout(_ptr(workspace), _nbytes(workspace), int(bool(odd)), stall_after,
                                                       wait_limit_ns, _stream(stream)))


def loss(logprob, y, kind=FLP_LOSS_NLL_MEAN, *, ignore_index: int = -100, old_logprob=None,
         advantage=None, ref_logprob=None, eps_low: float = 0.2, eps_high: float = 0.2,
         beta: float = 0.0, per_token=True, stream=None):
    """Loss head on per-row log-probs: (scalar loss [1], grad_logprob [M],
    per-token terms [M] or None).  grad_logprob is the upstream gradient for
    `backward`."""
    M = logprob.shape[0]
    _need(logprob, torch.float32, (M,), "logprob")
    _need(y, torch.int64, (M,), "targets")
    for t, name in ((old_logprob, "old_logprob"), (advantage, "advantage"), (ref_logprob, "ref_logprob")):
        _need_opt(t, torch.float32, (M,), name)
    dev = logprob.device
    out = torch.empty(1, dtype=torch.float32, device=dev)
    grad = torch.empty(M, dtype=torch.float32, device=dev)
    per = torch.empty(M, dtype=torch.float32, device=dev) if per_token else None
    _check(load().flp_loss(_ptr(logprob), _ptr(y), M, ignore_index, int(kind), _ptr(old_logprob),
                           _ptr(advantage), _ptr(ref_logprob), float(eps_low), float(eps_high),
                           float(beta), _ptr(per), _ptr(grad), _ptr(out), _stream(stream)),
           "flp_loss")
    return out, grad, per


def policy_loss(logprob, y, old_logprob, advantage, *, seq_offsets=None, ignore_index: int = -100,
                ref_logprob=None, eps_low: float = 0.2, eps_high: float = 0.2, beta: float = 0.0,
                is_level: int = FLP_IS_TOKEN, aggregation: int = FLP_AGG_TOKEN_MEAN,
                normalizer: float = 0.0, per_token=True, stream=None):
    """Clipped-surrogate loss over sequences (flp_policy_loss): (scalar loss
    [1], grad_logprob [M], per-token terms [M] or None).  seq_offsets: int64
    [B + 1] device tensor of the sequences' row offsets (None: one sequence).
    aggregation FLP_AGG_SUM_OVER with normalizer = num_items_in_batch is dapo."""
    M = logprob.shape[0]
    _need(logprob, torch.float32, (M,), "logprob")
    _need(y, torch.int64, (M,), "targets")
    _need(old_logprob, torch.float32, (M,), "old_logprob")
    _need(advantage, torch.float32, (M,), "advantage")
    _need_opt(ref_logprob, torch.float32, (M,), "ref_logprob")
    B = 0
    if seq_offsets is not None:
        B = seq_offsets.shape[0] - 1
        _need(seq_offsets, torch.int64, (B + 1,), "seq_offsets")
    dev = logprob.device
    out = torch.empty(1, dtype=torch.float32, device=dev)
    grad = torch.empty(M, dtype=torch.float32, device=dev)
    per = torch.empty(M, dtype=torch.float32, device=dev) if per_token else None
    _check(load().flp_policy_loss(_ptr(logprob), _ptr(y), M, ignore_index, _ptr(seq_offsets), B,
                                  _ptr(old_logprob), _ptr(advantage), _ptr(ref_logprob),
                                  float(eps_low), float(eps_high), float(beta), int(is_level),
                                  int(aggregation), float(normalizer), _ptr(per), _ptr(grad),
                                  _ptr(out), _stream(stream)),
           "flp_policy_loss")
    return out, grad, per


# ---------------------------------------------------------------- training-step operators
#
# The norm in front of the head, 8-bit checkpoints of activations with their
# use in the backward pass, and the router balance loss (include/flp.h has the
# formulas).  Row matrices may have any row pitch (a view of a wider tensor);
# their last dimension is contiguous.

CHECKPOINT_BLOCK = 32  # columns that share a step
_DTYPE = {torch.float32: FLP_F32, torch.bfloat16: FLP_BF16}


class Checkpoint8(NamedTuple):
    """An 8-bit checkpoint of a [rows, cols] activation: q int8 [rows, padded
    cols], scale uint8 [rows, padded cols / 32], and the type it reads back as."""
    q: torch.Tensor
    scale: torch.Tensor
    cols: int
    dtype: torch.dtype

    @property
    def shape(self):
        return (self.q.shape[0], self.cols)


def _dtype(t, name):
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: expected bf16 or fp32, got {t.dtype}")
    return code


def _rows(t, name, shape=None, dtype=None):
    """(address, row pitch) of a CUDA matrix whose rows are contiguous."""
    size = t.shape
    if len(size) != 2 or not t.is_cuda or (shape is not None and size != shape) or (
            dtype is not None and t.dtype is not dtype):
        raise ValueError(f"{name}: expected a CUDA matrix{'' if shape is None else f' of shape {tuple(shape)}'}"
                         f"{'' if dtype is None else f' of {dtype}'}, got {t.dtype} {tuple(size)} on {t.device}")
    pitch, unit = t.stride()
    rows, cols = size
    if (unit != 1 and cols > 1) or (pitch < cols and rows > 1):
        raise ValueError(f"{name}: rows must be contiguous and must not overlap, got strides {t.stride()}")
    return t.data_ptr(), pitch if rows > 1 else cols


def _check_checkpoint(c, name):
    q, scale = c.q, c.scale
    rows, padded = q.shape
    blocks = -(-c.cols // CHECKPOINT_BLOCK)
    if (q.dtype is not torch.int8 or scale.dtype is not torch.uint8 or not q.is_cuda or not scale.is_cuda
            or padded != blocks * CHECKPOINT_BLOCK or scale.shape != (rows, blocks)
            or not q.is_contiguous() or not scale.is_contiguous()):
        raise ValueError(f"{name}: not an 8-bit checkpoint: q {q.dtype} {tuple(q.shape)}, scale {scale.dtype} "
                         f"{tuple(scale.shape)}, {c.cols} columns")


def _new_checkpoint(rows, cols, dtype, device):
    blocks = -(-cols // CHECKPOINT_BLOCK)
    return Checkpoint8(torch.empty((rows, blocks * CHECKPOINT_BLOCK), dtype=torch.int8, device=device),
                       torch.empty((rows, blocks), dtype=torch.uint8, device=device), cols, dtype)


def _norm_param(t, cols, dtype, name):
    """(address, dtype code) of a norm parameter: [cols], the activations' type or fp32."""
    if t is None:
        return None, None
    d = t.dtype
    if (d is not dtype and d is not torch.float32) or t.shape != (cols,) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} or fp32 of shape ({cols},), "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr(), _DTYPE[d]


# Workspace sizes by device and problem: a pure function of both, remembered
# because asking costs as much as a small launch.
@functools.lru_cache(maxsize=4096)
def _workspace_bytes(fn: str, device: int, *args) -> int:
    n = ctypes.c_size_t(0)
    _check(getattr(load(), fn)(*args, ctypes.byref(n)), fn)
    return n.value


def _scratch(workspace, device, need):
    """(address, bytes, owner) of the caller's workspace, or of a new one of `need` bytes (none for 0)."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace.data_ptr(), need, workspace
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous CUDA tensor")
    return workspace.data_ptr(), _nbytes(workspace), workspace


def _on_stream(stream, fn, *args, **kw):
    """fn on `stream`, which its new tensors and workspace then belong to."""
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _stream_of(device):
    return torch.cuda.current_stream(device).cuda_stream


# The current stream's handle, where torch has it without the Stream object around
# it (which costs as much as a small launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, checkpoint: bool = False, out=None, stream=None):
    """Layer norm of each row of x [M, H] (bf16 or fp32; weight and bias in x's
    type or both fp32): (y, mean, rstd), and with `checkpoint` also the
    Checkpoint8 of x, written from the same read."""
    if stream is not None:
        return _on_stream(stream, layer_norm, x, weight, bias, eps=eps, checkpoint=checkpoint, out=out)
    xp, ldx = _rows(x, "x")
    M, H = shape = x.shape
    dt, dev = x.dtype, x.device
    code = _dtype(x, "x")
    wp, wt = _norm_param(weight, H, dt, "weight")
    bp, bt = _norm_param(bias, H, dt, "bias")
    if wt != bt and wt is not None and bt is not None:
        raise ValueError(f"weight and bias must have one type, got {weight.dtype} and {bias.dtype}")
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
        yp, ldy = out.data_ptr(), H
    else:
        yp, ldy = _rows(out, "out", shape, dt)
    mean = torch.empty(M, dtype=torch.float32, device=dev)
    rstd = torch.empty(M, dtype=torch.float32, device=dev)
    qp = sp = None
    if checkpoint:
        kept = _new_checkpoint(M, H, dt, dev)
        qp, sp = kept.q.data_ptr(), kept.scale.data_ptr()
    param = wt if wt is not None else bt if bt is not None else code
    status = load().flp_layer_norm(xp, ldx, code, wp, bp, param, M, H, eps, yp, ldy, mean.data_ptr(),
                                   rstd.data_ptr(), qp, sp, _raw_stream(dev.index))
    if status:
        _check(status, "flp_layer_norm")
    return (out, mean, rstd, kept) if checkpoint else (out, mean, rstd)


def layer_norm_backward(dy, x, weight, mean, rstd, *, dx=None, want_dweight: bool = True, want_dbias: bool = True,
                        workspace=None, stream=None):
    """(dx, dweight, dbias) of layer_norm; x is the activation (dy's type) or
    its Checkpoint8, mean and rstd the forward's.  dx has dy's type, dweight
    and dbias are fp32, or None where they are not wanted.  Without a weight its
    gradient is the one of all ones."""
    if stream is not None:
        return _on_stream(stream, layer_norm_backward, dy, x, weight, mean, rstd, dx=dx, want_dweight=want_dweight,
                          want_dbias=want_dbias, workspace=workspace)
    dyp, lddy = _rows(dy, "dy")
    M, H = shape = dy.shape
    dt, dev = dy.dtype, dy.device
    code = _dtype(dy, "dy")
    xp = qp = sp = None
    ldx = 0
    if isinstance(x, Checkpoint8):
        _check_checkpoint(x, "x")
        if x.cols != H or x.q.shape[0] != M:
            raise ValueError(f"x: checkpoint of shape {x.shape}, expected {(M, H)}")
        qp, sp = x.q.data_ptr(), x.scale.data_ptr()
    else:
        xp, ldx = _rows(x, "x", shape, dt)
    wp, wt = _norm_param(weight, H, dt, "weight")
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype is not torch.float32 or t.shape != (M,) or not t.is_cuda or not t.is_contiguous():
            _need(t, torch.float32, (M,), name)
    if dx is None:
        dx = torch.empty(shape, dtype=dt, device=dev)
        dxp, lddx = dx.data_ptr(), H
    else:
        dxp, lddx = _rows(dx, "dx", shape, dt)
    dweight = torch.empty(H, dtype=torch.float32, device=dev) if want_dweight else None
    dbias = torch.empty(H, dtype=torch.float32, device=dev) if want_dbias else None
    device = dev.index
    ws, ws_bytes, _keep = _scratch(workspace, dev, 0 if workspace is not None or not (want_dweight or want_dbias) else
                                   _workspace_bytes("flp_layer_norm_workspace", device, M, H))
    status = load().flp_layer_norm_backward(dyp, lddy, xp, ldx, qp, sp, code, wp, code if wt is None else wt,
                                            mean.data_ptr(), rstd.data_ptr(), M, H, dxp, lddx,
                                            dweight.data_ptr() if want_dweight else None,
                                            dbias.data_ptr() if want_dbias else None, ws, ws_bytes, _raw_stream(device))
    if status:
        _check(status, "flp_layer_norm_backward")
    return dx, dweight, dbias


def checkpoint_pack(x, *, stream=None) -> Checkpoint8:
    """The 8-bit checkpoint of x [M, H] (bf16 or fp32): 33/32 bytes an element."""
    if stream is not None:
        return _on_stream(stream, checkpoint_pack, x)
    xp, ldx = _rows(x, "x")
    M, H = x.shape
    code, dev = _dtype(x, "x"), x.device
    kept = _new_checkpoint(M, H, x.dtype, dev)
    status = load().flp_checkpoint_pack(xp, ldx, code, M, H, kept.q.data_ptr(), kept.scale.data_ptr(),
                                        _raw_stream(dev.index))
    if status:
        _check(status, "flp_checkpoint_pack")
    return kept


def checkpoint_unpack(kept: Checkpoint8, *, dtype=None, out=None, stream=None):
    """The values a checkpoint stands for, in its own type or the given one."""
    if stream is not None:
        return _on_stream(stream, checkpoint_unpack, kept, dtype=dtype, out=out)
    _check_checkpoint(kept, "checkpoint")
    q, H = kept.q, kept.cols
    M, dev = q.shape[0], q.device
    if out is None:
        out = torch.empty((M, H), dtype=dtype or kept.dtype, device=dev)
        xp, ldx = out.data_ptr(), H
    else:
        if dtype is not None and out.dtype is not dtype:
            raise ValueError(f"out: expected {dtype}, got {out.dtype}")
        xp, ldx = _rows(out, "out", (M, H))
    status = load().flp_checkpoint_unpack(q.data_ptr(), kept.scale.data_ptr(), M, H, xp, ldx, _dtype(out, "out"),
                                          _raw_stream(dev.index))
    if status:
        _check(status, "flp_checkpoint_unpack")
    return out


def checkpoint_weight_grad(dY, kept: Checkpoint8, *, dW=None, dw_dtype=torch.float32, accumulate: bool = False,
                           workspace=None, stream=None):
    """dW [N, K] = dY^T x of a linear layer whose input x [M, K] was kept as a
    checkpoint; dY bf16 [M, N].  With `accumulate` it is added to dW (fp32).  A
    timeout on the GPU leaves NaN in dW and FLP_ERR_TIMEOUT in the workspace."""
    if stream is not None:
        return _on_stream(stream, checkpoint_weight_grad, dY, kept, dW=dW, dw_dtype=dw_dtype, accumulate=accumulate,
                          workspace=workspace)
    _check_checkpoint(kept, "checkpoint")
    yp, ldy = _rows(dY, "dY", dtype=torch.bfloat16)
    M, N = dY.shape
    K, dev = kept.cols, dY.device
    if kept.q.shape[0] != M:
        raise ValueError(f"dY has {M} rows, the checkpoint {kept.q.shape[0]}")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs the dW to add to")
        dW = torch.empty((N, K), dtype=dw_dtype, device=dev)
    _need(dW, (torch.bfloat16, torch.float32), (N, K), "dW")
    code = _DTYPE[dW.dtype]
    device = dev.index
    # of the address only its alignment matters
    ws, ws_bytes, _keep = _scratch(workspace, dev, 0 if workspace is not None else
                                   _workspace_bytes("flp_checkpoint_weight_grad_workspace", device, yp % 16, ldy, M, N,
                                                    K, code))
    status = load().flp_checkpoint_weight_grad(yp, ldy, kept.q.data_ptr(), kept.scale.data_ptr(), M, N, K,
                                               dW.data_ptr(), code, accumulate, ws, ws_bytes, _raw_stream(device))
    if status:
        _check(status, "flp_checkpoint_weight_grad")
    return dW


def balance_loss(logits, top_k: int, *, experts=None, mask=None, coef: float = 1.0, grad: bool = True, grad_dtype=None,
                 workspace=None, stream=None):
    """Balance loss of router logits [T, E]: (loss [1], its gradient by the
    logits in their type or fp32 (grad_dtype), or None, counts int64 [E]).  mask: bool [T], the tokens that count;
    experts: int64 [T, top_k], the router's own choice (default: the top_k
    largest logits, ties to the lowest index)."""
    if stream is not None:
        return _on_stream(stream, balance_loss, logits, top_k, experts=experts, mask=mask, coef=coef, grad=grad,
                          grad_dtype=grad_dtype, workspace=workspace)
    zp, ld = _rows(logits, "logits")
    T, E = shape = logits.shape
    code, dev = _dtype(logits, "logits"), logits.device
    if mask is not None:
        _need(mask, torch.bool, (T,), "mask")
    if experts is not None:
        _need(experts, torch.int64, (T, top_k), "experts")
    loss_out = torch.empty(1, dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int64, device=dev)
    grad_dtype = logits.dtype if grad_dtype is None else grad_dtype
    if grad_dtype not in (logits.dtype, torch.float32):
        raise ValueError(f"grad_dtype: expected {logits.dtype} or fp32, got {grad_dtype}")
    g = torch.empty(shape, dtype=grad_dtype, device=dev) if grad else None
    device = dev.index
    ws, ws_bytes, _keep = _scratch(workspace, dev, 0 if workspace is not None else
                                   _workspace_bytes("flp_balance_loss_workspace", device, T, E))
    status = load().flp_balance_loss_ex(zp, ld, code, None if mask is None else mask.data_ptr(),
                                        None if experts is None else experts.data_ptr(), T, E, top_k, coef,
                                        loss_out.data_ptr(), None if g is None else g.data_ptr(), _DTYPE[grad_dtype],
                                        counts.data_ptr(), ws, ws_bytes, _raw_stream(device))
    if status:
        _check(status, "flp_balance_loss")
    return loss_out, g, counts


def get_error(workspace, stream=None) -> int:
    """Synchronise the stream and return the workspace's error status code."""
    return int(load().flp_get_error(_ptr(workspace), _stream(stream)))


class FusedLinearLogprob(torch.autograd.Function):
    """autograd wrapper: returns (logprob, entropy-or-empty) of softmax(scale X W^T)."""

    @staticmethod
    def forward(ctx, X, W, y, ignore_index, scale, compute_entropy, workspace):
        lp, lse, ent = forward(X, W, y, ignore_index=ignore_index, scale=scale,
                               compute_entropy=compute_entropy, workspace=workspace)
        ctx.save_for_backward(X, W, y, lse, ent if ent is not None else lse.new_empty(0))
        ctx.cfg = (ignore_index, scale, compute_entropy, workspace)
        return lp, (ent if ent is not None else lse.new_empty(0))

    @staticmethod
    def backward(ctx, g_lp, g_ent):
        X, W, y, lse, ent = ctx.saved_tensors
        ignore_index, scale, compute_entropy, workspace = ctx.cfg
        g_lp = None if g_lp is None else g_lp.contiguous().float()
        g_ent = None if (g_ent is None or not compute_entropy) else g_ent.contiguous().float()
        # a bf16 weight gets its bf16 gradient straight from the epilogue when
        # one backward wave covers every row; otherwise fp32 waves, then a cast
        M, H, V = X.shape[0], X.shape[1], W.shape[0]
        wave_rows, _, _ = backward_plan(M, H, V, _nbytes(workspace))
        direct = W.dtype == torch.bfloat16 and wave_rows >= M
        dX, dW = backward(X, W, y, lse, ent if compute_entropy else None, g_lp, g_ent,
                          ignore_index=ignore_index, scale=scale, compute_entropy=compute_entropy,
                          dx_dtype=X.dtype, dw_dtype=torch.bfloat16 if direct else torch.float32,
                          workspace=workspace)
        return dX, dW.to(W.dtype), None, None, None, None, None


def fused_linear_logprob(X, W, y, ignore_index: int = -100, scale: float = 1.0,
                         compute_entropy: bool = True, workspace=None):
    """Differentiable per-row log-prob (and entropy) of the LM head."""
    if workspace is None:
        workspace = alloc_workspace(X.shape[0], X.shape[1], W.shape[0], compute_entropy,
                                    device=X.device)
    return FusedLinearLogprob.apply(X, W, y, ignore_index, scale, compute_entropy, workspace)


class _Once(torch.autograd.Function):
    """The tensors that fn() gives, which depend on `inputs` in a way that autograd
    does not see: differentiating them is an error."""

    @staticmethod
    def forward(ctx, fn, *inputs):
        return fn()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of the training-step operators cannot be differentiated again")


def _once(fn, *inputs):
    """fn() inside a backward pass, whose gradients with create_graph must not pass for constants."""
    return _Once.apply(fn, *inputs) if torch.is_grad_enabled() else fn()


class FusedLayerNorm(torch.autograd.Function):
    """autograd wrapper of layer_norm; with `checkpoint` the input is kept for the
    backward pass in 8 bits instead of its own type."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, checkpoint):
        checkpoint = checkpoint and any(ctx.needs_input_grad)  # a checkpoint only for a backward pass
        y, mean, rstd, *kept = layer_norm(x, weight, bias, eps=eps, checkpoint=checkpoint)
        ctx.save_for_backward(*((kept[0].q, kept[0].scale) if checkpoint else (x, None)), weight, bias, mean, rstd)
        ctx.kept = (x.shape[1], x.dtype) if checkpoint else None
        return y

    @staticmethod
    def backward(ctx, dy):
        saved, scale, weight, bias, mean, rstd = ctx.saved_tensors
        x = saved if ctx.kept is None else Checkpoint8(saved, scale, *ctx.kept)
        _, want_dweight, want_dbias, _, _ = ctx.needs_input_grad
        dx, dweight, dbias = _once(lambda: layer_norm_backward(dy.contiguous(), x, weight, mean, rstd,
                                                               want_dweight=want_dweight, want_dbias=want_dbias),
                                   dy, saved, weight)
        return (dx, dweight.to(weight.dtype) if want_dweight else None,
                dbias.to(bias.dtype) if want_dbias else None, None, None)


def fused_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, checkpoint: bool = False):
    """Differentiable layer norm of the rows of x [M, H]."""
    # a Function's forward cannot tell that nothing is recorded
    return FusedLayerNorm.apply(x, weight, bias, eps, checkpoint and torch.is_grad_enabled())


class CheckpointLinear(torch.autograd.Function):
    """y = x W^T whose input is kept in 8 bits for the weight gradient.  The two
    products with W are library GEMMs."""

    @staticmethod
    def forward(ctx, x, W):
        if ctx.needs_input_grad[1]:
            for t, name in ((x, "x"), (W, "W")):
                if t.dtype is not torch.bfloat16:
                    raise ValueError(f"{name}: expected bf16 (its gradient is taken on the tensor cores), got {t.dtype}")
            kept = checkpoint_pack(x)
            ctx.save_for_backward(kept.q, kept.scale, W)
        else:
            ctx.save_for_backward(None, None, W)
        ctx.kept = (x.shape[1], x.dtype)
        return x @ W.t()

    @staticmethod
    def backward(ctx, dy):
        q, scale, W = ctx.saved_tensors
        dx = dy @ W if ctx.needs_input_grad[0] else None
        dW = None
        if ctx.needs_input_grad[1]:
            dW = _once(lambda: checkpoint_weight_grad(dy.contiguous(), Checkpoint8(q, scale, *ctx.kept),
                                                      dw_dtype=W.dtype), dy)
        return dx, dW


def checkpoint_linear(x, W):
    """Differentiable x W^T for bf16 x [M, K] and W [N, K] that keeps x in 8 bits
    (where W needs no gradient, of any type, and x is not kept)."""
    return CheckpointLinear.apply(x, W) if torch.is_grad_enabled() else x @ W.t()


class FusedBalanceLoss(torch.autograd.Function):
    """autograd wrapper of balance_loss: (scalar loss, counts)."""

    @staticmethod
    def forward(ctx, logits, top_k, experts, mask, coef):
        # kept in fp32: a gradient rounded to bf16 and then scaled is rounded twice, and a
        # factor near 1 is lost altogether
        loss_out, grad, counts = balance_loss(logits, top_k, experts=experts, mask=mask, coef=coef,
                                              grad=ctx.needs_input_grad[0], grad_dtype=torch.float32)
        ctx.save_for_backward(logits, grad)
        ctx.mark_non_differentiable(counts)
        return loss_out[0], counts

    @staticmethod
    def backward(ctx, g, _):
        logits, grad = ctx.saved_tensors
        dz = _once(lambda: torch.mul(grad, g.view(1, 1), out=torch.empty_like(grad, dtype=logits.dtype)), g, logits)
        return dz, None, None, None, None


def fused_balance_loss(logits, top_k: int, experts=None, mask=None, coef: float = 1.0):
    """Differentiable balance loss of router logits [T, E]: (scalar loss, counts [E])."""
    if not torch.is_grad_enabled():
        loss_out, _, counts = balance_loss(logits, top_k, experts=experts, mask=mask, coef=coef, grad=False)
        return loss_out[0], counts
    return FusedBalanceLoss.apply(logits, top_k, experts, mask, coef)
