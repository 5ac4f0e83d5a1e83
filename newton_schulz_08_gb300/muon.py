"""ctypes binding of libmuon.so (include/muon.h): argument marshalling only.

Every step of the Muon update runs inside the library's CUDA kernels; this
module turns torch tensors into device pointers and the current torch stream
into a cudaStream_t, allocates the workspace with torch when the caller does
not pass one, and raises ``MuonError`` on a non-OK status.  It loads the
library on first use and fails loudly if it has not been built.
"""

import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmuon.so")
#: the same library with device-side checks (tests and debugging)
DEBUG_LIB_PATH = os.path.join(_PKG, "lib", "libmuon_debug.so")

MUON_OK = 0
MUON_WARN_NONFINITE = 1
MUON_ERR_INVALID_ARG = -1
MUON_ERR_MISALIGNED = -2
MUON_ERR_ALIASING = -3
MUON_ERR_WORKSPACE_TOO_SMALL = -4
MUON_ERR_CUDA = -5
MUON_ERR_DEVICE_TIMEOUT = -6
MUON_ERR_UNSUPPORTED_DEVICE = -7
MUON_ERR_TOO_LARGE = -8
MUON_ERR_SCRATCH_LIMIT = -9
MUON_ERR_HOST_MEMORY = -10
MUON_BF16 = 0
MUON_F32 = 1

#: every symbol include/muon.h declares
EXPORTS = ["muon_workspace_size", "muon_step", "ns5_workspace_size", "ns5", "ns5_bank",
           "ns5_bank_workspace_size", "muon_device_status", "muon_status_str",
           "ns5_workspace_layout", "muon_set_debug", "muon_kernel_times", "ns5_noalloc", "ns5_noalloc_status",
           "muon_partition", "adam_step", "fp8_mm", "muon_plan_cache_clear",
           "fp8_mm_backward", "fp8_mm_backward_workspace_size", "muon_debug_check_failures",
           "adamw_step", "adamw_plan_create", "adamw_plan_set_grads", "adamw_plan_set_rates", "adamw_plan_step",
           "adamw_plan_destroy", "token_logprobs", "token_logprobs_backward", "token_logprobs_loss", "balance_loss",
           "balance_loss_workspace_size", "balance_loss_backward"]

#: bytes of the static device scratch ns5_noalloc uses (MUON_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 64 << 20

#: kernel kinds reported by muon_kernel_times
KERNEL_KINDS = ["momentum_cast", "normalise", "gram", "poly", "update", "apply", "update_apply", "fp8_quantize",
                "fp8_mm", "fp8_transpose", "fp8_mm_bwd", "fp8_reduce"]


class MuonError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {muon_status_str(status)} (status {status})")


class muon_mat_desc(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("buf", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class muon_ws_layout(ctypes.Structure):
    _fields_ = [("x_offset", ctypes.c_size_t * 2), ("a_offset", ctypes.c_size_t),
                ("b_offset", ctypes.c_size_t), ("ldx", ctypes.c_int64), ("lda", ctypes.c_int64),
                ("m", ctypes.c_int64), ("n", ctypes.c_int64)]


class adam_tensor_desc(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class adamw_tensor_desc(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("numel", ctypes.c_int64), ("lr", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("state_bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def load(path):
    """A ctypes handle on the library at `path` with every entry point's
    signature declared (the release library, or the debug build)."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m newton_schulz_08_gb300.build` (or __graft_entry__.build())")
    L = ctypes.CDLL(path)
    c_int, c_i64, c_sz, c_vp, c_f = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    P = ctypes.POINTER
    L.muon_workspace_size.argtypes = [P(muon_mat_desc), c_int]
    L.muon_workspace_size.restype = c_sz
    L.muon_step.argtypes = [P(muon_mat_desc), c_int, c_f, c_f, c_int, c_int, c_vp, c_sz, c_vp]
    L.muon_step.restype = c_int
    L.ns5_workspace_size.argtypes = [c_int, c_i64, c_i64]
    L.ns5_workspace_size.restype = c_sz
    L.ns5.argtypes = [c_vp, c_int, c_vp, c_int, c_i64, c_i64, c_int, c_vp, c_sz, c_vp]
    L.ns5.restype = c_int
    L.ns5_bank.argtypes = [P(c_vp), P(ctypes.c_int32), P(c_vp), P(c_i64), P(c_i64), c_int, c_int,
                           c_vp, c_sz, c_vp]
    L.ns5_bank.restype = c_int
    L.ns5_bank_workspace_size.argtypes = [P(c_i64), P(c_i64), c_int]
    L.ns5_bank_workspace_size.restype = c_sz
    L.muon_device_status.argtypes = [c_vp, c_vp]
    L.muon_device_status.restype = c_int
    L.muon_status_str.argtypes = [c_int]
    L.muon_status_str.restype = ctypes.c_char_p
    L.ns5_workspace_layout.argtypes = [c_int, c_i64, c_i64, P(muon_ws_layout)]
    L.ns5_workspace_layout.restype = c_int
    L.muon_set_debug.argtypes = [ctypes.c_char_p, ctypes.c_longlong]
    L.muon_set_debug.restype = c_int
    L.muon_kernel_times.argtypes = [P(ctypes.c_double), P(c_int), c_int]
    L.muon_kernel_times.restype = c_int
    L.ns5_noalloc.argtypes = [c_vp, c_int, c_vp, c_int, c_i64, c_i64, c_int, c_vp]
    L.ns5_noalloc.restype = c_int
    L.ns5_noalloc_status.argtypes = [c_vp]
    L.ns5_noalloc_status.restype = c_int
    L.muon_partition.argtypes = [P(c_i64), P(c_i64), c_int, c_int, P(c_int)]
    L.muon_partition.restype = c_int
    L.adam_step.argtypes = [P(adam_tensor_desc), c_int, c_f, c_f, c_f, c_f, c_f, c_int, c_int, c_vp]
    L.adam_step.restype = c_int
    L.fp8_mm.argtypes = [c_vp, c_vp, c_f, c_f, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_vp, c_sz, c_vp]
    L.fp8_mm.restype = c_int
    L.fp8_mm_backward_workspace_size.argtypes = [c_i64, c_i64, c_i64]
    L.fp8_mm_backward_workspace_size.restype = c_sz
    L.fp8_mm_backward.argtypes = [c_vp, c_vp, c_vp, c_f, c_f, c_f, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_vp,
                                  c_sz, c_vp]
    L.fp8_mm_backward.restype = c_int
    c_d, c_u64 = ctypes.c_double, ctypes.c_uint64
    L.adamw_step.argtypes = [P(adamw_tensor_desc), c_int, c_d, c_d, c_d, c_int, c_i64, c_u64, c_vp, c_vp]
    L.adamw_step.restype = c_int
    L.adamw_plan_create.argtypes = [P(adamw_tensor_desc), c_int, P(c_vp)]
    L.adamw_plan_create.restype = c_int
    L.adamw_plan_set_grads.argtypes = [c_vp, P(c_vp), P(ctypes.c_int32)]
    L.adamw_plan_set_grads.restype = c_int
    L.adamw_plan_set_rates.argtypes = [c_vp, P(c_d), P(c_d)]
    L.adamw_plan_set_rates.restype = c_int
    L.adamw_plan_step.argtypes = [c_vp, c_d, c_d, c_d, c_int, c_i64, c_u64, c_vp, c_vp]
    L.adamw_plan_step.restype = c_int
    L.adamw_plan_destroy.argtypes = [c_vp]
    L.adamw_plan_destroy.restype = None
    L.token_logprobs.argtypes = [c_vp, c_int, c_i64, c_i64, c_i64, c_vp, c_f, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]
    L.token_logprobs.restype = c_int
    L.token_logprobs_backward.argtypes = [c_vp, c_int, c_i64, c_i64, c_i64, c_vp, c_f, c_vp, c_vp, c_vp, c_vp, c_vp,
                                          c_i64, c_vp]
    L.token_logprobs_backward.restype = c_int
    L.token_logprobs_loss.argtypes = [c_vp, c_int, c_i64, c_i64, c_i64, c_vp, c_f, c_int, c_vp, c_vp, c_vp, c_vp, c_vp,
                                      c_vp, c_vp, c_vp, c_i64, c_vp]
    L.token_logprobs_loss.restype = c_int
    L.balance_loss.argtypes = [c_vp, c_int, c_i64, c_int, c_i64, c_vp, c_int, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp,
                               c_vp, c_sz, c_vp]
    L.balance_loss.restype = c_int
    L.balance_loss_workspace_size.argtypes = [c_i64, c_int, c_i64]
    L.balance_loss_workspace_size.restype = c_sz
    L.balance_loss_backward.argtypes = [c_vp, c_int, c_i64, c_int, c_i64, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp,
                                        c_i64, c_vp]
    L.balance_loss_backward.restype = c_int
    L.muon_plan_cache_clear.argtypes = []
    L.muon_plan_cache_clear.restype = None
    L.muon_debug_check_failures.argtypes = [P(ctypes.c_longlong)]
    L.muon_debug_check_failures.restype = c_int
    return L


def muon_status_str(status):
    return lib().muon_status_str(int(status)).decode()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _tensors(out):
    if isinstance(out, torch.Tensor):
        yield out
    elif isinstance(out, (tuple, list)):
        for t in out:
            yield from _tensors(t)


def _on(stream, tensor, fn, *args):
    """fn(*args) under `stream` of the tensor's device: what the call allocates
    belongs to that stream, so that neither a workspace nor an output is memory
    that the caller's own stream still uses or is given next.  What it returns
    may be used on the caller's stream, which must wait for `stream` as for
    any work there, and freed at any time."""
    if not tensor.is_cuda:
        return fn(*args)  # refuses it
    if getattr(stream, "device", tensor.device) != tensor.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {tensor.device}")
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == torch._C._cuda_getCurrentRawStream(tensor.get_device()):
        return fn(*args)
    own = torch.cuda.current_stream(tensor.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(handle, tensor.device) if handle
                  else torch.cuda.default_stream(tensor.device))
    with torch.cuda.stream(stream):
        out = fn(*args)
    for t in _tensors(out):
        if t.is_cuda:
            t.record_stream(own)
    return out


def _check(status, where, ok=(MUON_OK,)):
    if status not in ok:
        raise MuonError(status, where)
    return status


def _device_of(tensors, what):
    """The one CUDA device all `tensors` live on (raises otherwise).  The
    library works on the current device with device pointers, so a CPU
    tensor or a tensor of another GPU must never reach it."""
    dev = None
    for t in tensors:
        if not t.is_cuda:
            raise ValueError(f"{what}: every tensor must be a CUDA tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{what}: tensors are on {dev} and {t.device}; all must share one device")
    return dev


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    if t.dtype == torch.float32:
        return MUON_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _descs(params, grads, bufs):
    n = len(params)
    if len(grads) != n or len(bufs) != n:
        raise ValueError("params, grads and bufs must have the same length")
    arr = (muon_mat_desc * max(n, 1))()
    for i, (p, g, b) in enumerate(zip(params, grads, bufs)):
        if p.dim() != 2 or g.shape != p.shape or b.shape != p.shape:
            raise ValueError(f"matrix {i}: param, grad and buf must be 2-D of one shape")
        if p.dtype != torch.float32 or b.dtype != torch.float32:
            raise TypeError(f"matrix {i}: param and buf must be float32")
        if not (p.is_contiguous() and g.is_contiguous() and b.is_contiguous()):
            raise ValueError(f"matrix {i}: tensors must be contiguous")
        arr[i] = muon_mat_desc(p.data_ptr(), g.data_ptr(), b.data_ptr(), p.shape[0], p.shape[1],
                               _dtype_code(g), 0)
    return arr, n


def muon_workspace_size(shapes):
    """Workspace bytes for a bank given as a list of (rows, cols)."""
    n = len(shapes)
    arr = (muon_mat_desc * max(n, 1))()
    for i, (r, c) in enumerate(shapes):
        arr[i] = muon_mat_desc(0, 0, 0, r, c, MUON_BF16, 0)
    return lib().muon_workspace_size(arr, n)


def new_workspace(nbytes, device=None):
    device = device or torch.device("cuda", torch.cuda.current_device())
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def muon_step(params, grads, bufs, lr=0.02, momentum=0.95, nesterov=True, ns_steps=5,
              workspace=None, stream=None):
    """One Muon step over a bank (lists of 2-D CUDA tensors), in place."""
    if stream is not None and workspace is None and len(params):
        return _on(stream, params[0], muon_step, params, grads, bufs, lr, momentum, nesterov, ns_steps)
    arr, n = _descs(params, grads, bufs)
    if n == 0:
        return workspace
    dev = _device_of(list(params) + list(grads) + list(bufs) + ([workspace] if workspace is not None else []),
                     "muon_step")
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(lib().muon_workspace_size(arr, n), dev)
        st = lib().muon_step(arr, n, float(lr), float(momentum), int(bool(nesterov)), int(ns_steps),
                             ctypes.c_void_p(workspace.data_ptr()), workspace.numel(), _stream(stream))
    _check(st, "muon_step")
    return workspace


class StepGraph:
    """One muon_step recorded in a CUDA graph for fixed tensors, scalars and
    workspace; replay() runs the step's launches (momentum pass, normalise,
    the Newton-Schulz launches) with one host call.  The recording itself
    runs nothing: params and bufs are first changed by the first replay.
    The graph holds the tensors' addresses, so they must stay alive and in
    place; a change of lr, momentum or ns_steps needs a new StepGraph.
    Kernel-event recording (muon_set_debug "record_kernel_events") must be
    off while recording."""

    def __init__(self, params, grads, bufs, lr=0.02, momentum=0.95, nesterov=True, ns_steps=5, workspace=None):
        self.tensors = (list(params), list(grads), list(bufs))
        arr, n = _descs(*self.tensors)
        if n == 0:
            raise ValueError("StepGraph needs at least one matrix")
        dev = _device_of(self.tensors[0] + self.tensors[1] + self.tensors[2]
                         + ([workspace] if workspace is not None else []), "StepGraph")
        with torch.cuda.device(dev):
            if workspace is None:
                workspace = new_workspace(lib().muon_workspace_size(arr, n), dev)
            self.workspace = workspace
            self.stream = torch.cuda.Stream(dev)
            self.graph = torch.cuda.CUDAGraph()
            self.stream.wait_stream(torch.cuda.current_stream(dev))
            # relaxed: the first call of a bank also sets kernel attributes and
            # queries occupancy, which are not stream work
            with torch.cuda.graph(self.graph, stream=self.stream, capture_error_mode="relaxed"):
                muon_step(params, grads, bufs, lr=lr, momentum=momentum, nesterov=nesterov, ns_steps=ns_steps,
                          workspace=workspace, stream=self.stream)

    def replay(self):
        """Runs the recorded step (on the graph's stream, ordered after the
        current stream's work so far; the current stream waits for it)."""
        cur = torch.cuda.current_stream(self.stream.device)
        self.stream.wait_stream(cur)
        with torch.cuda.stream(self.stream):
            self.graph.replay()
        cur.wait_stream(self.stream)


def ns5_workspace_size(batch, rows, cols):
    return lib().ns5_workspace_size(int(batch), int(rows), int(cols))


def ns5(G, ns_steps=5, out=None, workspace=None, stream=None):
    """zeropower_via_newtonschulz5 on a (batch x) rows x cols CUDA tensor -> bf16."""
    if stream is not None:
        return _on(stream, G, ns5, G, ns_steps, out, workspace)
    squeeze = G.dim() == 2
    G3 = G.unsqueeze(0) if squeeze else G
    if G3.dim() != 3 or not G3.is_contiguous():
        raise ValueError("G must be a contiguous 2-D or 3-D tensor")
    batch, rows, cols = G3.shape
    if out is None:
        out = torch.empty(G3.shape, dtype=torch.bfloat16, device=G.device)
    if out.shape != G3.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bfloat16 tensor shaped like G")
    dev = _device_of([G3, out] + ([workspace] if workspace is not None else []), "ns5")
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(ns5_workspace_size(batch, rows, cols) if batch else 256, dev)
        st = lib().ns5(ctypes.c_void_p(G3.data_ptr()), _dtype_code(G3), ctypes.c_void_p(out.data_ptr()),
                       batch, rows, cols, int(ns_steps), ctypes.c_void_p(workspace.data_ptr()),
                       workspace.numel(), _stream(stream))
    _check(st, "ns5")
    return out[0] if squeeze else out


def ns5_bank_workspace_size(shapes):
    n = len(shapes)
    rows = (ctypes.c_int64 * max(n, 1))(*[s[0] for s in shapes])
    cols = (ctypes.c_int64 * max(n, 1))(*[s[1] for s in shapes])
    return lib().ns5_bank_workspace_size(rows, cols, n)


def ns5_bank(Gs, ns_steps=5, outs=None, workspace=None, stream=None):
    """Newton-Schulz on a list of differently shaped 2-D CUDA tensors -> bf16 list."""
    if stream is not None and len(Gs):
        return _on(stream, Gs[0], ns5_bank, Gs, ns_steps, outs, workspace)
    n = len(Gs)
    if outs is None:
        outs = [torch.empty(g.shape, dtype=torch.bfloat16, device=g.device) for g in Gs]
    if len(outs) != n:
        raise ValueError("outs must have one tensor per G")
    for g, o in zip(Gs, outs):
        if (g.dim() != 2 or not g.is_contiguous() or o.shape != g.shape or o.dtype != torch.bfloat16
                or not o.is_contiguous()):
            raise ValueError("each G must be 2-D contiguous with a contiguous bf16 out of the same shape")
    if n == 0:
        return outs
    dev = _device_of(list(Gs) + list(outs) + ([workspace] if workspace is not None else []), "ns5_bank")
    gp = (ctypes.c_void_p * max(n, 1))(*[g.data_ptr() for g in Gs])
    op = (ctypes.c_void_p * max(n, 1))(*[o.data_ptr() for o in outs])
    dt = (ctypes.c_int32 * max(n, 1))(*[_dtype_code(g) for g in Gs])
    rows = (ctypes.c_int64 * max(n, 1))(*[g.shape[0] for g in Gs])
    cols = (ctypes.c_int64 * max(n, 1))(*[g.shape[1] for g in Gs])
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(lib().ns5_bank_workspace_size(rows, cols, n), dev)
        st = lib().ns5_bank(gp, dt, op, rows, cols, n, int(ns_steps),
                            ctypes.c_void_p(workspace.data_ptr()), workspace.numel(), _stream(stream))
    _check(st, "ns5_bank")
    return outs


def muon_device_status(workspace, stream=None):
    """Synchronise and read the workspace's device status word (an int code)."""
    return lib().muon_device_status(ctypes.c_void_p(workspace.data_ptr()), _stream(stream))


def ns5_workspace_layout(batch, rows, cols):
    out = muon_ws_layout()
    _check(lib().ns5_workspace_layout(int(batch), int(rows), int(cols), ctypes.byref(out)),
           "ns5_workspace_layout")
    return {"x_offset": (out.x_offset[0], out.x_offset[1]), "a_offset": out.a_offset,
            "b_offset": out.b_offset, "ldx": out.ldx, "lda": out.lda, "m": out.m, "n": out.n}


def muon_plan_cache_clear():
    """Drop the library's prepared calls (host memory only)."""
    lib().muon_plan_cache_clear()


def muon_set_debug(key, value):
    if lib().muon_set_debug(key.encode(), int(value)) != 0:
        raise KeyError(key)


def muon_kernel_times():
    """{kind: (total_ms, launches)} for launches recorded since the last call."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    if lib().muon_kernel_times(ms, cnt, n) != 0:
        raise RuntimeError("muon_kernel_times failed")
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}


def ns5_noalloc(G, ns_steps=5, out=None, stream=None):
    """ns5 without a workspace: the library's own static device scratch is
    used (for callers that may not allocate device memory; see include/muon.h).
    Only `out` is allocated here when the caller does not pass one."""
    if stream is not None:
        return _on(stream, G, ns5_noalloc, G, ns_steps, out)
    squeeze = G.dim() == 2
    G3 = G.unsqueeze(0) if squeeze else G
    if G3.dim() != 3 or not G3.is_contiguous():
        raise ValueError("G must be a contiguous 2-D or 3-D tensor")
    batch, rows, cols = G3.shape
    if out is None:
        out = torch.empty(G3.shape, dtype=torch.bfloat16, device=G.device)
    if out.shape != G3.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bfloat16 tensor shaped like G")
    dev = _device_of([G3, out], "ns5_noalloc")
    # the library's scratch array and the default stream are the current
    # device's: make G's device current for the call
    with torch.cuda.device(dev):
        st = lib().ns5_noalloc(ctypes.c_void_p(G3.data_ptr()), _dtype_code(G3),
                               ctypes.c_void_p(out.data_ptr()), batch, rows, cols, int(ns_steps),
                               _stream(stream))
    _check(st, "ns5_noalloc")
    return out[0] if squeeze else out


def ns5_noalloc_status(stream=None, device=None):
    """Device status of the last ns5_noalloc call on `device` (default: the
    current one), read after synchronising `stream`: MUON_OK,
    MUON_WARN_NONFINITE or MUON_ERR_DEVICE_TIMEOUT (see include/muon.h)."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return lib().ns5_noalloc_status(_stream(stream))


def partition(shapes, world):
    """Owner rank of each matrix of a bank of (rows, cols) shapes when the
    step runs on `world` processes: heaviest Newton-Schulz work first, each
    matrix to the least-loaded rank (muon_partition; host only)."""
    n = len(shapes)
    rows = (ctypes.c_int64 * max(n, 1))(*[int(r) for r, _ in shapes])
    cols = (ctypes.c_int64 * max(n, 1))(*[int(c) for _, c in shapes])
    owner = (ctypes.c_int * max(n, 1))()
    _check(lib().muon_partition(rows, cols, n, int(world), owner), "muon_partition")
    return [owner[i] for i in range(n)]


def adam_step(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
              weight_decay=0.0, cautious=True, stream=None):
    """Adam step with cautious weight decay over lists of CUDA tensors, in
    place (fp32 params and moments; bf16 or fp32 grads).  See adam_step in
    include/muon.h for the arithmetic."""
    n = len(params)
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == n):
        raise ValueError("params, grads, exp_avgs, exp_avg_sqs must have the same length")
    arr = (adam_tensor_desc * max(n, 1))()
    for i, (p, g, m, v) in enumerate(zip(params, grads, exp_avgs, exp_avg_sqs)):
        for t in (p, m, v):
            if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError("params and moments must be contiguous float32 CUDA tensors")
        if not (p.numel() == g.numel() == m.numel() == v.numel()) or not g.is_contiguous():
            raise ValueError("tensor sizes differ or a gradient is not contiguous")
        arr[i] = adam_tensor_desc(p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), p.numel(),
                                  _dtype_code(g), 0)
    if n == 0:
        return
    dev = _device_of(list(params) + list(grads) + list(exp_avgs) + list(exp_avg_sqs), "adam_step")
    with torch.cuda.device(dev):
        st = lib().adam_step(arr, n, float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                             int(step), int(bool(cautious)), _stream(stream))
    _check(st, "adam_step")


def fp8_mm(x, w, x_s, w_s, out=None, x_f8=None, w_f8=None, workspace=None, stream=None):
    """FP8 scaled product of bf16 CUDA tensors x (M x K) and w (N x K):
    returns (out, x_f8, w_f8), out = bf16(x_s w_s (x_f8 . w_f8^T)) with
    x_f8 = E4M3(bf16(x / x_s)), w_f8 = E4M3(bf16(w / w_s)) as float8_e4m3fn
    tensors.  See fp8_mm in include/muon.h."""
    if stream is not None:
        return _on(stream, x, fp8_mm, x, w, x_s, w_s, out, x_f8, w_f8, workspace)
    for t in (x, w):
        if t.dim() != 2 or t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("x and w must be contiguous 2-D bfloat16 CUDA tensors")
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("x and w must have the same number of columns")
    dev = x.device
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if out is None else out
    x_f8 = torch.empty((M, K), dtype=torch.uint8, device=dev) if x_f8 is None else x_f8
    w_f8 = torch.empty((N, K), dtype=torch.uint8, device=dev) if w_f8 is None else w_f8
    # the library writes exactly these sizes: check the caller's buffers
    if out.shape != (M, N) or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous M x N bfloat16 tensor on x's device")
    for t, shape in ((x_f8, (M, K)), (w_f8, (N, K))):
        if (t.shape != shape or t.element_size() != 1 or not t.is_contiguous() or t.device != dev
                or t.dtype not in (torch.uint8, torch.float8_e4m3fn)):
            raise ValueError("x_f8 / w_f8 must be contiguous one-byte (uint8 or float8_e4m3fn) tensors "
                             "shaped like x / w, on x's device")
    x_f8, w_f8 = x_f8.view(torch.uint8), w_f8.view(torch.uint8)
    if w.device != dev:
        raise ValueError("x and w must be on the same device")
    _device_of([x, w, out, x_f8, w_f8] + ([workspace] if workspace is not None else []), "fp8_mm")
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(256, dev)
        st = lib().fp8_mm(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(w.data_ptr()), float(x_s), float(w_s),
                          ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(x_f8.data_ptr()),
                          ctypes.c_void_p(w_f8.data_ptr()), M, N, K, ctypes.c_void_p(workspace.data_ptr()),
                          workspace.numel(), _stream(stream))
    _check(st, "fp8_mm")
    return out, x_f8.view(torch.float8_e4m3fn), w_f8.view(torch.float8_e4m3fn)


def fp8_mm_backward_workspace_size(M, N, K):
    return lib().fp8_mm_backward_workspace_size(int(M), int(N), int(K))


def fp8_mm_backward(g, x_f8, w_f8, x_s, w_s, grad_s, grad_x=None, grad_w=None, g_f8=None, workspace=None,
                    stream=None):
    """Backward of the FP8 scaled product: g (M x N bf16) and the forward's
    x_f8 (M x K) and w_f8 (N x K) E4M3 codes -> (grad_x, grad_w, g_f8):
    grad_x = bf16(grad_s w_s (g_f8 . w_f8)), grad_w = bf16(grad_s x_s
    (g_f8^T . x_f8)), g_f8 = E5M2(bf16(g / grad_s)) as a float8_e5m2 tensor.
    See fp8_mm_backward in include/muon.h."""
    if stream is not None:
        return _on(stream, g, fp8_mm_backward, g, x_f8, w_f8, x_s, w_s, grad_s, grad_x, grad_w, g_f8, workspace)
    if g.dim() != 2 or g.dtype != torch.bfloat16 or not g.is_contiguous():
        raise ValueError("g must be a contiguous 2-D bfloat16 CUDA tensor")
    M, N = g.shape
    for t, shape in ((x_f8, None), (w_f8, None)):
        if t.dim() != 2 or t.element_size() != 1 or not t.is_contiguous():
            raise ValueError("x_f8 / w_f8 must be contiguous 2-D one-byte tensors")
    K = x_f8.shape[1]
    if x_f8.shape != (M, K) or w_f8.shape != (N, K):
        raise ValueError("x_f8 must be M x K and w_f8 N x K for g of M x N")
    dev = _device_of([g, x_f8, w_f8] + [t for t in (grad_x, grad_w, g_f8, workspace) if t is not None],
                     "fp8_mm_backward")
    grad_x = torch.empty((M, K), dtype=torch.bfloat16, device=dev) if grad_x is None else grad_x
    grad_w = torch.empty((N, K), dtype=torch.bfloat16, device=dev) if grad_w is None else grad_w
    g_f8 = torch.empty((M, N), dtype=torch.uint8, device=dev) if g_f8 is None else g_f8
    for t, shape in ((grad_x, (M, K)), (grad_w, (N, K))):
        if t.shape != shape or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("grad_x / grad_w must be contiguous bfloat16 tensors of M x K / N x K")
    if (g_f8.shape != (M, N) or g_f8.element_size() != 1 or not g_f8.is_contiguous()
            or g_f8.dtype not in (torch.uint8, torch.float8_e5m2)):
        raise ValueError("g_f8 must be a contiguous M x N one-byte tensor (uint8 or float8_e5m2)")
    g_f8 = g_f8.view(torch.uint8)
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(fp8_mm_backward_workspace_size(M, N, K), dev)
        st = lib().fp8_mm_backward(ctypes.c_void_p(g.data_ptr()), ctypes.c_void_p(x_f8.data_ptr()),
                                   ctypes.c_void_p(w_f8.data_ptr()), float(x_s), float(w_s), float(grad_s),
                                   ctypes.c_void_p(grad_x.data_ptr()), ctypes.c_void_p(grad_w.data_ptr()),
                                   ctypes.c_void_p(g_f8.data_ptr()), M, N, K, ctypes.c_void_p(workspace.data_ptr()),
                                   workspace.numel(), _stream(stream))
    _check(st, "fp8_mm_backward")
    return grad_x, grad_w, g_f8.view(torch.float8_e5m2)


# The operators below are called for a few microseconds of GPU work at a time:
# their host side avoids temporary objects (tensor devices, stream objects,
# context managers, ctypes wrappers).

def _index_of(what, *tensors):
    """Index of the one CUDA device that all tensors (None: left out) are on."""
    index = -1
    for t in tensors:
        if t is None:
            continue
        i = t.get_device()
        if i < 0 or (i != index and index >= 0):
            _device_of([u for u in tensors if u is not None], what)  # raises with the reason
        index = i
    return index


def _call(fn, what, index, stream, *args):
    """fn(*args, stream) with device `index` current; raises on an error."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    else:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != MUON_OK:
        raise MuonError(status, what)


#: elements that share one scale of an 8-bit moment
ADAMW_BLOCK = 256


def adamw_state(param, bits=32):
    """Zero moments for one parameter of an AdamW step: (exp_avg, exp_avg_sq)
    float32, or with bits=8 (exp_avg, exp_avg_scale, exp_avg_sq,
    exp_avg_sq_scale): float8_e4m3fn and float8_e5m2 codes with one float32
    scale per 256 elements.  8 bits are for tensors whose gradients differ by
    no more than 2^12 within 256 neighbouring elements (include/muon.h says
    what happens beyond)."""
    if bits == 32:
        return tuple(torch.zeros(param.numel(), dtype=torch.float32, device=param.device) for _ in range(2))
    if bits != 8:
        raise ValueError("bits must be 32 or 8")
    out = []
    for kind in (torch.float8_e4m3fn, torch.float8_e5m2):
        out.append(torch.zeros(param.numel(), dtype=torch.uint8, device=param.device).view(kind))
        out.append(torch.zeros(-(-param.numel() // ADAMW_BLOCK), dtype=torch.float32, device=param.device))
    return tuple(out)


def adamw_state_values(state):
    """The float32 values (exp_avg, exp_avg_sq) that a state stands for."""
    if len(state) == 2:
        return state
    value = lambda c, s: c.float() * s.repeat_interleave(ADAMW_BLOCK)[:c.numel()]  # noqa: E731
    return value(state[0], state[1]), value(state[2], state[3])


def _per_tensor(x, n, what):
    x = [float(x)] * n if isinstance(x, (int, float)) else [float(v) for v in x]
    if len(x) != n:
        raise ValueError(f"{what}: one number, or one per tensor")
    return x


def _adamw_descs(params, grads, states, lr, weight_decay):
    """(descriptors, number, every tensor) of an AdamW step, checked."""
    n = len(params)
    if len(states) != n or (grads is not None and len(grads) != n):
        raise ValueError("params, grads and states must have the same length")
    lr, weight_decay = _per_tensor(lr, n, "lr"), _per_tensor(weight_decay, n, "weight_decay")
    f32, m8, v8 = torch.float32, torch.float8_e4m3fn, torch.float8_e5m2
    codes = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16}
    arr, every = (adamw_tensor_desc * max(n, 1))(), []
    for i, (p, s) in enumerate(zip(params, states)):
        size = p.numel()
        if len(s) == 2:
            m, v = s
            ms = vs = None
            fits = m.dtype == f32 and v.dtype == f32
        elif len(s) == 4:
            m, ms, v, vs = s
            fits = m.dtype == m8 and v.dtype == v8
            blocks = -(-size // ADAMW_BLOCK)
            if ms.dtype != f32 or vs.dtype != f32 or ms.numel() != blocks or vs.numel() != blocks:
                raise ValueError(f"tensor {i}: scales must be float32, one per {ADAMW_BLOCK} elements")
        else:
            raise ValueError(f"tensor {i}: a state has 2 tensors (32 bits) or 4 (8 bits)")
        if not fits or m.numel() != size or v.numel() != size:
            raise ValueError(f"tensor {i}: moments must have the parameter's size and be float32, or float8_e4m3fn "
                             "and float8_e5m2")
        g = None if grads is None else grads[i]
        used = (p, m, v) if ms is None else (p, m, v, ms, vs)
        if g is not None:
            if g.numel() != size:
                raise ValueError(f"tensor {i}: the gradient must have the parameter's size")
            used += (g,)
        for t in used:
            if not t.is_contiguous():
                raise ValueError(f"tensor {i}: tensors must be contiguous")
        every += used
        kind, grad_kind = codes.get(p.dtype, -1), MUON_F32 if g is None else codes.get(g.dtype, -1)
        if kind < 0 or grad_kind < 0:
            raise TypeError(f"tensor {i}: parameters and gradients must be bfloat16 or float32")
        arr[i] = (p.data_ptr(), 0 if g is None else g.data_ptr(), m.data_ptr(), v.data_ptr(),
                  0 if ms is None else ms.data_ptr(), 0 if vs is None else vs.data_ptr(), size, lr[i],
                  weight_decay[i], kind, grad_kind, 32 if ms is None else 8, 0)
    return arr, n, every


def _grad_scale(t, index):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1 or t.get_device() != index:
        raise ValueError("grad_scale must be one float32 value on the parameters' device")
    return t.data_ptr()


def adamw_step(params, grads, states, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
               cautious=False, grad_scale=None, seed=0, stream=None):
    """AdamW step over lists of CUDA tensors, in place: float32 or bfloat16
    params and grads, states from adamw_state (32 or 8 bits, tensor by
    tensor).  lr and weight_decay: one number, or one per tensor.  grad_scale:
    a one-element float32 CUDA tensor that the gradients are multiplied with
    (a clipping factor).  seed: of the stochastic rounding of 8-bit states and
    bfloat16 parameters.  A call recorded in a CUDA graph repeats its own step
    number.  See adamw_step in include/muon.h; AdamW keeps what is the same in
    every step (this call describes every tensor anew)."""
    arr, n, every = _adamw_descs(params, grads, states, lr, weight_decay)
    if n == 0:
        return
    index = _index_of("adamw_step", *every)
    _call(lib().adamw_step, "adamw_step", index, stream, arr, n, float(beta1), float(beta2), float(eps),
          int(bool(cautious)), int(step), int(seed) & (2 ** 64 - 1), _grad_scale(grad_scale, index))


class AdamW:
    """AdamW over a fixed list of parameters, the checked descriptors kept
    between steps (adamw_plan in include/muon.h), so that a step costs one
    launch per combination of types.

    states   from adamw_state (default: zeros, 32 bits for every tensor, or
             `bits`);
    grads    the gradients' tensors when they stay in place (a bucket);
             otherwise pass them to step();
    step     steps already taken.

    The addresses of the tensors are kept, and their memory with them: a
    parameter or moment that is given other memory afterwards (``p.data = ...``,
    ``module.to(...)``) is not followed and needs a new AdamW.
    """

    def __init__(self, params, grads=None, states=None, bits=32, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                 weight_decay=0.01, cautious=False, seed=0, step=0):
        self.params = list(params)
        self.grads = None if grads is None else list(grads)
        self.states = [adamw_state(p, bits) for p in self.params] if states is None else list(states)
        self.beta1, self.beta2, self.eps, self.cautious = float(beta1), float(beta2), float(eps), int(bool(cautious))
        self.seed, self.steps = int(seed) & (2 ** 64 - 1), int(step)
        self._plan = ctypes.c_void_p()
        if not self.params:
            raise ValueError("AdamW needs at least one parameter")
        arr, n, every = _adamw_descs(self.params, self.grads, self.states, lr, weight_decay)
        self._index = _index_of("AdamW", *every)
        self._memory = [t.untyped_storage() for t in every]
        _check(lib().adamw_plan_create(arr, n, ctypes.byref(self._plan)), "AdamW")

    def __del__(self):
        if getattr(self, "_plan", None):
            lib().adamw_plan_destroy(self._plan)
            self._plan = None

    def set_rates(self, lr, weight_decay):
        """Learning rate and weight decay from the next step on: one number, or one per tensor."""
        n = len(self.params)
        lr, wd = _per_tensor(lr, n, "lr"), _per_tensor(weight_decay, n, "weight_decay")
        double = ctypes.c_double * n
        _check(lib().adamw_plan_set_rates(self._plan, double(*lr), double(*wd)), "AdamW.set_rates")

    def set_grads(self, grads):
        """Other gradient tensors from the next step on.  Every tensor is
        checked again: gradients that stay in place are given once."""
        n, grads = len(self.params), list(grads)
        if len(grads) != n or any(g.numel() != p.numel() or not g.is_contiguous()
                                  for g, p in zip(grads, self.params)):
            raise ValueError("AdamW: one contiguous gradient of the parameter's size per parameter")
        if _index_of("AdamW", *grads) != self._index:
            raise ValueError("AdamW: gradients must be on the parameters' device")
        ptrs = (ctypes.c_void_p * n)(*[g.data_ptr() for g in grads])
        kinds = (ctypes.c_int32 * n)(*[_dtype_code(g) for g in grads])
        _check(lib().adamw_plan_set_grads(self._plan, ptrs, kinds), "AdamW.set_grads")
        self.grads = grads

    def step(self, grads=None, grad_scale=None, stream=None):
        """One step, in place; `grads` replaces the gradients' tensors."""
        if grads is not None:
            self.set_grads(grads)
        elif self.grads is None:
            raise ValueError("AdamW.step: no gradients given, here or at construction")
        _call(lib().adamw_plan_step, "AdamW.step", self._index, stream, self._plan, self.beta1, self.beta2, self.eps,
              self.cautious, self.steps + 1, self.seed, _grad_scale(grad_scale, self._index))
        self.steps += 1

    def state_values(self):
        """The float32 moments (exp_avg, exp_avg_sq) of each parameter."""
        return [adamw_state_values(s) for s in self.states]


class TokenLogprobs(NamedTuple):
    """What token_logprobs gives for each row."""
    logprobs: torch.Tensor
    lse: torch.Tensor
    entropy: torch.Tensor
    top_logprobs: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]
    grad: Optional[torch.Tensor] = None


def _matrix(t, what):
    """(rows, columns, row pitch) of a 2-D CUDA tensor with unit column stride."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{what} must be 2-D with contiguous rows")
    rows, cols = t.shape
    pitch = t.stride(0) if rows > 1 else cols
    if pitch < cols:
        raise ValueError(f"{what}: rows overlap")
    return rows, cols, pitch


def _per_row(t, rows, dtype, what):
    if t is None:
        return None
    if t.shape != (rows,) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor with one entry per row")
    return t.data_ptr()


def _score_outputs(rows, top, dev):
    """(tensors, pointers) of logprobs, lse, entropy, top_logprobs, top_ids."""
    out = torch.empty((3, rows), dtype=torch.float32, device=dev)
    p = out.data_ptr()
    pointers = (p, p + 4 * rows, p + 8 * rows)
    if not top:
        return (*out.unbind(), None, None), (*pointers, None, None)
    values = torch.empty((rows, top), dtype=torch.float32, device=dev)
    ids = torch.empty((rows, top), dtype=torch.int64, device=dev)
    return (*out.unbind(), values, ids), (*pointers, values.data_ptr(), ids.data_ptr())


def _grad_out(out, logits):
    if out is None:
        return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    if out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("out must have the logits' shape and dtype")
    return out


def token_logprobs(logits, targets, top=0, scale=1.0, stream=None):
    """Log probabilities of the targets (int64, one per row; negative: the row
    is left out) under softmax(scale * logits), with log-sum-exp, entropy and
    the `top` (<= 32) most likely entries: a TokenLogprobs.  logits: rows x
    vocab, bfloat16 or float32, any row pitch.  See include/muon.h."""
    if stream is not None:
        return _on(stream, logits, token_logprobs, logits, targets, top, scale)
    rows, vocab, pitch = _matrix(logits, "logits")
    index = _index_of("token_logprobs", logits, targets)
    y = _per_row(targets, rows, torch.int64, "targets")
    out, p = _score_outputs(rows, top, logits.device)
    _call(lib().token_logprobs, "token_logprobs", index, stream, logits.data_ptr(), _dtype_code(logits), rows, vocab,
          pitch, y, scale, top, *p)
    return TokenLogprobs(*out)


def token_logprobs_backward(logits, targets, lse, grad_logprobs, entropy=None, grad_entropy=None, scale=1.0, out=None,
                            stream=None):
    """Gradient with respect to the logits from those with respect to
    logprobs and, with `entropy` as token_logprobs gave it, entropy.  `out`
    may be the logits themselves.  See include/muon.h."""
    if stream is not None:
        return _on(stream, logits, token_logprobs_backward, logits, targets, lse, grad_logprobs, entropy, grad_entropy,
                   scale, out)
    rows, vocab, pitch = _matrix(logits, "logits")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs entropy")
    out = _grad_out(out, logits)
    index = _index_of("token_logprobs_backward", logits, targets, lse, grad_logprobs, entropy, grad_entropy, out)
    f32 = torch.float32
    _call(lib().token_logprobs_backward, "token_logprobs_backward", index, stream, logits.data_ptr(),
          _dtype_code(logits), rows, vocab, pitch, _per_row(targets, rows, torch.int64, "targets"), scale,
          _per_row(lse, rows, f32, "lse"), _per_row(entropy, rows, f32, "entropy"),
          _per_row(grad_logprobs, rows, f32, "grad_logprobs"), _per_row(grad_entropy, rows, f32, "grad_entropy"),
          out.data_ptr(), _matrix(out, "out")[2])
    return out


def token_logprobs_loss(logits, targets, grad_logprobs, grad_entropy=None, top=0, scale=1.0, out=None, stream=None):
    """token_logprobs together with the gradient with respect to the logits
    (TokenLogprobs.grad), for a loss whose gradients with respect to logprobs
    and entropy are known beforehand; `out` may be the logits themselves.
    See include/muon.h."""
    if stream is not None:
        return _on(stream, logits, token_logprobs_loss, logits, targets, grad_logprobs, grad_entropy, top, scale, out)
    rows, vocab, pitch = _matrix(logits, "logits")
    out = _grad_out(out, logits)
    index = _index_of("token_logprobs_loss", logits, targets, grad_logprobs, grad_entropy, out)
    f32 = torch.float32
    gl, ge = _per_row(grad_logprobs, rows, f32, "grad_logprobs"), _per_row(grad_entropy, rows, f32, "grad_entropy")
    y = _per_row(targets, rows, torch.int64, "targets")
    got, p = _score_outputs(rows, top, logits.device)
    _call(lib().token_logprobs_loss, "token_logprobs_loss", index, stream, logits.data_ptr(), _dtype_code(logits),
          rows, vocab, pitch, y, scale, top, gl, ge, *p, out.data_ptr(), _matrix(out, "out")[2])
    return TokenLogprobs(*got, out)


class BalanceLoss(NamedTuple):
    """What balance_loss gives: the losses (0-d), int32 counts (groups x
    experts) and token numbers (groups), mean router probabilities (groups x
    experts), and `saved`, which balance_loss_backward reads."""
    balance: torch.Tensor
    z: torch.Tensor
    counts: torch.Tensor
    tokens: torch.Tensor
    mean_probs: torch.Tensor
    saved: torch.Tensor


@functools.lru_cache(maxsize=256)
def balance_loss_workspace_size(tokens, experts, groups=1):
    return lib().balance_loss_workspace_size(int(tokens), int(experts), int(groups))


def _mask(mask, tokens):
    if mask is None:
        return None
    if mask.shape != (tokens,) or mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous():
        raise ValueError("mask must be a contiguous bool tensor with one entry per token")
    return mask.data_ptr()


def balance_loss(logits, ids, mask=None, groups=1, workspace=None, stream=None):
    """Balance loss and z loss of a router, with the experts' counts: logits
    tokens x experts (bfloat16 or float32, any row pitch), ids tokens x top
    int64 (the experts each token goes to), mask one bool per token (False:
    left out), `groups` sequences of equal length.  See include/muon.h."""
    if stream is not None:
        return _on(stream, logits, balance_loss, logits, ids, mask, groups, workspace)
    tokens, experts, pitch = _matrix(logits, "logits")
    if ids.dim() != 2 or ids.shape[0] != tokens or ids.dtype != torch.int64 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous tokens x top int64 tensor")
    index = _index_of("balance_loss", logits, ids, mask, workspace)
    dev, f32 = logits.device, torch.float32
    # saved: the four statistics, then the weights
    saved = torch.empty(4 + groups * experts, dtype=f32, device=dev)
    counts = torch.empty((groups, experts), dtype=torch.int32, device=dev)
    n_tokens = torch.empty(groups, dtype=torch.int32, device=dev)
    mean = torch.empty((groups, experts), dtype=f32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(balance_loss_workspace_size(tokens, experts, groups), 256), dtype=torch.uint8,
                                device=dev)
    stats = saved.data_ptr()
    _call(lib().balance_loss, "balance_loss", index, stream, logits.data_ptr(), _dtype_code(logits), tokens, experts,
          pitch, ids.data_ptr(), ids.shape[1], _mask(mask, tokens), groups, stats, counts.data_ptr(),
          n_tokens.data_ptr(), mean.data_ptr(), stats + 16, workspace.data_ptr(), workspace.numel())
    return BalanceLoss(saved.select(0, 0), saved.select(0, 1), counts, n_tokens, mean, saved)


def balance_loss_backward(logits, result, grad_balance, grad_z, mask=None, out=None, stream=None):
    """Gradient of grad_balance * balance + grad_z * z (one-element float32
    CUDA tensors) with respect to the logits; `result` is balance_loss's for
    the same logits and mask.  `out` may be the logits themselves."""
    if stream is not None:
        return _on(stream, logits, balance_loss_backward, logits, result, grad_balance, grad_z, mask, out)
    tokens, experts, pitch = _matrix(logits, "logits")
    out = _grad_out(out, logits)
    groups, columns = result.counts.shape
    if columns != experts:
        raise ValueError("result is of other logits")
    if (grad_balance.dtype != torch.float32 or grad_z.dtype != torch.float32 or grad_balance.numel() != 1
            or grad_z.numel() != 1):
        raise ValueError("grad_balance and grad_z must be one-element float32 tensors")
    stats = result.saved.data_ptr()
    index = _index_of("balance_loss_backward", logits, mask, grad_balance, grad_z, out, result.saved)
    _call(lib().balance_loss_backward, "balance_loss_backward", index, stream, logits.data_ptr(), _dtype_code(logits),
          tokens, experts, pitch, _mask(mask, tokens), groups, stats, stats + 16, grad_balance.data_ptr(),
          grad_z.data_ptr(), out.data_ptr(), _matrix(out, "out")[2])
    return out
