"""ctypes binding of libspecverify.so with the same entry-point names as include/spec_verify.h.

Argument marshalling only: tensors are checked and their device pointers handed to the C ABI
on the current CUDA stream; every step of verification runs in the library's CUDA kernels.
PyTorch supplies device memory (outputs, the workspace) and the stream.  There is no CPU
fallback: if the library is not built or no GPU is present, these functions raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
from typing import NamedTuple, Optional

import torch

from . import _build

BF16, FP32, FP16, E4M3 = 0, 1, 2, 3
MODE_GREEDY, MODE_REJECTION, MODE_TREE, MODE_BLOCK = 0, 1, 2, 3
OK, EINVAL, EWORKSPACE, ECUDA, ETOOBIG = 0, -1, -2, -3, -4
NOALLOC_SCRATCH_BYTES = 4 << 20
DEV_OK, DEV_BAD_TOKEN, DEV_BAD_ROW, DEV_BAD_TREE, DEV_DUP_SIBLING = 0, 1, 2, 3, 4
DEV_BAD_KV_POSITION, DEV_BAD_KV_SLOT, DEV_TIMEOUT = 5, 6, 7

_lib = None
_lock = threading.Lock()


class Options(ctypes.Structure):
    """spec_verify_options: a temperature per request (device float32 [B], 0 = greedy) or one
    temperature for all, and the relaxed thresholds of target-only decisions (1 = exact)."""
    _fields_ = [("temperatures", ctypes.c_void_p), ("temperature", ctypes.c_float),
                ("threshold_single", ctypes.c_float), ("threshold_acc", ctypes.c_float),
                ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p)]


def library_path() -> str:
    return _build.LIB_PATH


def _declare(lib):
    """Argument and result types of every entry point of include/spec_verify.h."""
    vp, i32, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_float,
                             ctypes.c_size_t)
    lib.spec_verify_greedy.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, vp, sz, vp, vp]
    lib.spec_verify_greedy.restype = i32
    lib.spec_verify_rejection.argtypes = [vp, i32, vp, vp, i32, i32, i32, f32, u64, u64, vp,
                                          vp, vp, vp, sz, vp, vp]
    lib.spec_verify_rejection.restype = i32
    lib.spec_verify_block.argtypes = [vp, i32, vp, vp, i32, i32, i32, f32, u64, u64, vp, vp,
                                      vp, sz, vp, vp]
    lib.spec_verify_block.restype = i32
    lib.spec_verify_tree.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, f32, u64, u64, vp,
                                     vp, vp, vp, sz, vp, vp]
    lib.spec_verify_tree.restype = i32
    lib.spec_verify_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.spec_verify_workspace_bytes.restype = sz
    lib.spec_verify_strerror.argtypes = [i32]
    lib.spec_verify_strerror.restype = ctypes.c_char_p
    lib.spec_verify_philox.argtypes = [u64, u64, i32, i32, vp, vp]
    lib.spec_verify_philox.restype = i32
    lib.spec_verify_rejection_noalloc.argtypes = [vp, i32, vp, vp, i32, i32, i32, f32, u64,
                                                  u64, vp, vp, vp, vp, vp]
    lib.spec_verify_rejection_noalloc.restype = i32
    lib.spec_verify_kv_compact.argtypes = [vp, ctypes.c_int64, sz, i32, sz, vp, i32, vp, vp,
                                           vp, vp, i32, i32, vp, vp]
    lib.spec_verify_kv_compact.restype = i32
    OP = ctypes.POINTER(Options)
    lib.spec_verify_rejection_ex.argtypes = [vp, i32, vp, vp, i32, i32, i32, OP, u64, u64, vp,
                                             vp, vp, vp, sz, vp, vp]
    lib.spec_verify_rejection_ex.restype = i32
    lib.spec_verify_tree_ex.argtypes = [vp, i32, vp, vp, i32, i32, i32, OP, u64, u64, vp, vp,
                                        vp, vp, sz, vp, vp]
    lib.spec_verify_tree_ex.restype = i32
    lib.spec_verify_plan_budget.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.spec_verify_plan_budget.restype = i32
    lib.spec_verify_plan_budget_workspace_bytes.argtypes = [i32, i32]
    lib.spec_verify_plan_budget_workspace_bytes.restype = sz
    i64 = ctypes.c_int64
    lib.spec_verify_kv_append.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, i64, i64, i64, vp,
                                          i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                          vp, vp]
    lib.spec_verify_kv_append.restype = i32
    lib.spec_verify_attention.argtypes = [vp, i32, i64, vp, vp, i64, i64, i64, vp, i32, vp, vp, vp, i32,
                                          i32, i32, i32, i32, f32, vp, vp, vp, sz, vp, vp]
    lib.spec_verify_attention.restype = i32
    lib.spec_verify_attention_workspace_bytes.argtypes = [i32] * 6
    lib.spec_verify_attention_workspace_bytes.restype = sz
    lib.spec_verify_kv_e4m3_row_bytes.argtypes = [i32, i32]
    lib.spec_verify_kv_e4m3_row_bytes.restype = sz
    lib.spec_verify_kv_append_ex.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, i32, i64, i64, i64, vp,
                                             i32, vp, vp, vp, vp, i32, i32, i32, vp, vp, f32, i32, i32, i32, i32,
                                             i32, vp, vp]
    lib.spec_verify_kv_append_ex.restype = i32
    lib.spec_verify_kv_read.argtypes = [vp, vp, i32, i64, i64, i64, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp,
                                        i32, vp, vp]
    lib.spec_verify_kv_read.restype = i32
    lib.spec_verify_attention_e4m3.argtypes = lib.spec_verify_attention.argtypes
    lib.spec_verify_attention_e4m3.restype = i32
    lib.spec_verify_attention_e4m3_workspace_bytes.argtypes = [i32] * 6
    lib.spec_verify_attention_e4m3_workspace_bytes.restype = sz
    lib.spec_verify_attention_chunk.argtypes = [vp, i32, i64, vp, vp, i32, i64, i64, i64, vp, i32, vp, vp, i32, i32,
                                                i32, i32, i32, f32, vp, vp, vp, sz, vp, vp]
    lib.spec_verify_attention_chunk.restype = i32
    lib.spec_verify_attention_chunk_workspace_bytes.argtypes = [i32] * 6
    lib.spec_verify_attention_chunk_workspace_bytes.restype = sz
    lib.spec_verify_logprobs.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, f32, i32, vp, vp, vp,
                                         vp, vp, vp, sz, vp, vp]
    lib.spec_verify_logprobs.restype = i32
    lib.spec_verify_logprobs_workspace_bytes.argtypes = [i32] * 4
    lib.spec_verify_logprobs_workspace_bytes.restype = sz
    lib.spec_verify_debug_wait_clocks.argtypes = [ctypes.c_int64]
    lib.spec_verify_debug_wait_clocks.restype = i32
    lib.spec_verify_capture_id.argtypes = [vp, ctypes.POINTER(u64)]
    lib.spec_verify_capture_id.restype = i32
    lib.spec_verify_debug_fault.argtypes = [ctypes.POINTER(ctypes.c_uint64)]
    lib.spec_verify_debug_fault.restype = i32
    lib.spec_verify_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint64)]
    lib.spec_verify_wait_timeouts.restype = i32
    return lib


def load_library():
    """Load libspecverify.so (in-tree).  Raises when it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with __graft_entry__.build() (nvcc, sm_103a)")
        _lib = _declare(ctypes.CDLL(path))
        return _lib


def load_debug_library():
    """The range-checked build (libspecverify_debug.so, compiled on first use): the same entry
    points, every kernel's global-memory indices checked (spec_verify_debug_fault reports)."""
    return _declare(ctypes.CDLL(_build.build_debug()))


@contextlib.contextmanager
def using_library(lib):
    """Route this module's wrappers through another build of the library (e.g. the debug one)."""
    global _lib
    load_library()
    with _lock:
        prev, _lib = _lib, lib
    try:
        yield lib
    finally:
        with _lock:
            _lib = prev


def spec_verify_debug_fault(lib=None) -> int:
    """The first out-of-range index recorded by a debug build since the last read (0: none)."""
    lib = lib or load_library()
    w = ctypes.c_uint64(0)
    rc = lib.spec_verify_debug_fault(ctypes.byref(w))
    if rc != OK:
        raise SpecVerifyError("spec_verify_debug_fault", rc)
    return int(w.value)


def spec_verify_wait_timeouts(lib=None) -> int:
    """Waits inside kernels that ran out of time since the last read (0 in normal operation).  Rows of
    the top-k / top-p ring kernel were then finished by the general threshold kernel; attention and log
    probabilities are undefined (device status 7)."""
    lib = lib or load_library()
    n = ctypes.c_uint64(0)
    rc = lib.spec_verify_wait_timeouts(ctypes.byref(n))
    if rc != OK:
        raise SpecVerifyError("spec_verify_wait_timeouts", rc)
    return int(n.value)


def spec_verify_debug_wait_clocks(clocks: int, lib) -> None:
    """The limit of waits inside a debug build's kernels, in SM clocks (a test aid; see the header)."""
    rc = lib.spec_verify_debug_wait_clocks(clocks)
    if rc != OK:
        raise SpecVerifyError("spec_verify_debug_wait_clocks", rc)


def spec_verify_strerror(code: int) -> str:
    return load_library().spec_verify_strerror(int(code)).decode()


def spec_verify_workspace_bytes(mode: int, B: int, k_or_N: int, V: int) -> int:
    return int(load_library().spec_verify_workspace_bytes(mode, B, k_or_N, V))


class SpecVerifyError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code}: {spec_verify_strerror(code)}")
        self.code = code


# --------------------------------------------------------------------------------------------
# Marshalling helpers
# --------------------------------------------------------------------------------------------
_current_device = torch._C._cuda_getDevice  # (torch.cuda.current_device looks first whether CUDA is set up)


def _on(device: int, entry):
    """An entry point of the library with that device current: it launches on, and keeps its kernels' attributes
    for, the current one, and raw stream handles are that device's."""
    if device == _current_device():
        return entry

    def call(*args):
        with torch.cuda.device(device):
            return entry(*args)

    return call


def _capture_id(device: int, stream: Optional[torch.cuda.Stream], raw: int) -> int:
    """The id of the graph capture that a stream (None: the device's current one) is under; 0: none."""
    if raw == 0:
        return 0  # (the default stream cannot be captured)
    if stream is None and device == _current_device() and not torch.cuda.is_current_stream_capturing():
        return 0
    found = ctypes.c_uint64(0)
    rc = _on(device, load_library().spec_verify_capture_id)(raw, ctypes.byref(found))
    if rc != OK:
        raise SpecVerifyError("spec_verify_capture_id", rc)
    return found.value


class _Workspaces:
    """Device buffers kept per (device, stream).

    A call under graph capture takes one that was made within that capture: its memory is the graph's, its
    fill is a node ahead of the calls that need it, and every replay begins with it, whatever ran before and
    in whatever order graphs are replayed.  So no graph holds a buffer that calls outside it use, or that is
    given back when one of them needs a larger."""

    def __init__(self, make):
        self.make, self.kept, self.captured = make, {}, {}

    def get(self, nbytes: int, device: int, stream: Optional[torch.cuda.Stream], raw: int) -> torch.Tensor:
        key, capture = (device, raw), _capture_id(device, stream, raw)
        if capture:
            of, ws = self.captured.get(key, (0, None))
            if of != capture:
                ws = None
        else:
            ws = self.kept.get(key)
        if ws is None or ws.numel() < nbytes:
            with torch.cuda.stream(stream):  # the fill is in the order of the stream that uses it
                ws = self.make(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
            if capture:
                self.captured[key] = capture, ws
            else:
                self.kept[key] = ws
        return ws

    def forget(self):
        self.kept.clear()


# The library leaves a workspace's counters zero after each call, so one zero-fill suffices.
_workspaces = _Workspaces(torch.zeros)
# Not the verifiers' workspace: the planner overwrites its buffer, whose counter region the
# verifiers need to stay zero.
_plan_workspaces = _Workspaces(torch.empty)
# Nor are chunks' parts the verifiers' (52 MB a stream): they need no fill, a call writes what it reads.
_chunk_workspaces = _Workspaces(torch.empty)


def workspace_for(nbytes: int, device: torch.device, stream: torch.cuda.Stream) -> torch.Tensor:
    """A uint8 device buffer of at least nbytes for calls on this stream, zero-filled when it was made."""
    return _workspaces.get(nbytes, device.index, stream, stream.cuda_stream)


def spec_verify_reset_workspaces() -> None:
    """Forget the buffers kept for calls without a workspace: the next call on each stream takes a new,
    zero-filled one.  Needed after device status 7 (a wait inside a kernel ran out), which leaves counters
    behind on which later calls would join too early; and a way to give their memory back, the planner's and the
    chunks' too.  A graph's calls begin with a fill and need it not; a caller's own workspace is the caller's to
    zero."""
    for kept in (_workspaces, _plan_workspaces, _chunk_workspaces):
        kept.forget()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _logits_dtype(logits: torch.Tensor) -> int:
    if logits.dtype == torch.bfloat16:
        return BF16
    if logits.dtype == torch.float32:
        return FP32
    raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")


def _check_dev(name: str, t: torch.Tensor, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _ws_and_status(nbytes, device, stream, workspace, dev_status):
    if workspace is None:
        workspace = workspace_for(nbytes, device, stream)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=device)
    return workspace, dev_status


class Result(NamedTuple):
    out_tokens: torch.Tensor
    accept_len: torch.Tensor
    dev_status: torch.Tensor
    accept_index: Optional[torch.Tensor] = None
    out_probs: Optional[torch.Tensor] = None


# --------------------------------------------------------------------------------------------
# Entry points
# --------------------------------------------------------------------------------------------
def spec_verify_greedy(logits: torch.Tensor, draft_ids: torch.Tensor, *, out_tokens=None,
                       accept_len=None, workspace=None, dev_status=None, stream=None) -> Result:
    """logits [B, k+1, V] (bf16 / fp32), draft_ids [B, k] int32 -> Result."""
    lib = load_library()
    _check_dev("logits", logits)
    B, k1, V = logits.shape
    k = k1 - 1
    _check_dev("draft_ids", draft_ids, torch.int32)
    if tuple(draft_ids.shape) != (B, k):
        raise ValueError("draft_ids must be [B, k]")
    dev = logits.device
    stream = stream or torch.cuda.current_stream(dev)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, k1), dtype=torch.int32, device=dev)
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    nbytes = spec_verify_workspace_bytes(MODE_GREEDY, B, k, V)
    workspace, dev_status = _ws_and_status(nbytes, dev, stream, workspace, dev_status)
    rc = _on(dev.index, lib.spec_verify_greedy)(_ptr(logits), _logits_dtype(logits), _ptr(draft_ids), B, k, V,
                                _ptr(out_tokens), _ptr(accept_len), _ptr(workspace),
                                workspace.numel(), _ptr(dev_status),
                                ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_greedy", rc)
    return Result(out_tokens, accept_len, dev_status)


def spec_verify_rejection(logits: torch.Tensor, draft_ids: torch.Tensor,
                          draft_probs: Optional[torch.Tensor] = None, *, temperature: float,
                          seed: int, offset: int, out_tokens=None, accept_len=None,
                          out_probs=None, want_probs: bool = False, workspace=None,
                          dev_status=None, stream=None) -> Result:
    """Standard rejection (draft_probs [B, k, V] fp32) or one-hot (draft_probs None)."""
    lib = load_library()
    _check_dev("logits", logits)
    B, k1, V = logits.shape
    k = k1 - 1
    _check_dev("draft_ids", draft_ids, torch.int32)
    if tuple(draft_ids.shape) != (B, k):
        raise ValueError("draft_ids must be [B, k]")
    if draft_probs is not None:
        _check_dev("draft_probs", draft_probs, torch.float32)
        if tuple(draft_probs.shape) != (B, k, V):
            raise ValueError("draft_probs must be [B, k, V]")
    dev = logits.device
    stream = stream or torch.cuda.current_stream(dev)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, k1), dtype=torch.int32, device=dev)
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    if out_probs is None and want_probs:
        out_probs = torch.empty((B, k1, 3), dtype=torch.float32, device=dev)
    nbytes = spec_verify_workspace_bytes(MODE_REJECTION, B, k, V)
    workspace, dev_status = _ws_and_status(nbytes, dev, stream, workspace, dev_status)
    rc = _on(dev.index, lib.spec_verify_rejection)(_ptr(logits), _logits_dtype(logits), _ptr(draft_ids),
                                   _ptr(draft_probs), B, k, V, float(temperature),
                                   int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                                   _ptr(out_tokens), _ptr(accept_len), _ptr(out_probs),
                                   _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                   ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_rejection", rc)
    return Result(out_tokens, accept_len, dev_status, None, out_probs)


def spec_verify_block(logits: torch.Tensor, draft_ids: torch.Tensor,
                      draft_probs: Optional[torch.Tensor] = None, *, temperature: float,
                      seed: int, offset: int, out_tokens=None, accept_len=None, workspace=None,
                      dev_status=None, stream=None) -> Result:
    """Block verification of a chain: draft_probs [B, k, V] fp32, or None for one-hot drafts."""
    lib = load_library()
    _check_dev("logits", logits)
    B, k1, V = logits.shape
    k = k1 - 1
    _check_dev("draft_ids", draft_ids, torch.int32)
    if tuple(draft_ids.shape) != (B, k):
        raise ValueError("draft_ids must be [B, k]")
    if draft_probs is not None:
        _check_dev("draft_probs", draft_probs, torch.float32)
        if tuple(draft_probs.shape) != (B, k, V):
            raise ValueError("draft_probs must be [B, k, V]")
    dev = logits.device
    stream = stream or torch.cuda.current_stream(dev)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, k1), dtype=torch.int32, device=dev)
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    nbytes = spec_verify_workspace_bytes(MODE_BLOCK, B, k, V)
    workspace, dev_status = _ws_and_status(nbytes, dev, stream, workspace, dev_status)
    rc = _on(dev.index, lib.spec_verify_block)(_ptr(logits), _logits_dtype(logits), _ptr(draft_ids), _ptr(draft_probs),
                               B, k, V, float(temperature), int(seed) & (2**64 - 1),
                               int(offset) & (2**64 - 1), _ptr(out_tokens), _ptr(accept_len),
                               _ptr(workspace), workspace.numel(), _ptr(dev_status),
                               ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_block", rc)
    return Result(out_tokens, accept_len, dev_status)


def spec_verify_tree(logits: torch.Tensor, node_tokens: torch.Tensor, parents: torch.Tensor, *,
                     mode: int, temperature: float = 1.0, seed: int = 0, offset: int = 0,
                     out_tokens=None, accept_index=None, accept_len=None, workspace=None,
                     dev_status=None, stream=None) -> Result:
    """logits [B, N, V]; node_tokens, parents [B, N] int32; mode 0 greedy, 1 target-only."""
    lib = load_library()
    _check_dev("logits", logits)
    B, N, V = logits.shape
    _check_dev("node_tokens", node_tokens, torch.int32)
    _check_dev("parents", parents, torch.int32)
    if tuple(node_tokens.shape) != (B, N) or tuple(parents.shape) != (B, N):
        raise ValueError("node_tokens and parents must be [B, N]")
    dev = logits.device
    stream = stream or torch.cuda.current_stream(dev)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, N), dtype=torch.int32, device=dev)
    accept_index = accept_index if accept_index is not None else torch.empty((B, N), dtype=torch.int32, device=dev)
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    nbytes = spec_verify_workspace_bytes(MODE_TREE, B, N, V)
    workspace, dev_status = _ws_and_status(nbytes, dev, stream, workspace, dev_status)
    rc = _on(dev.index, lib.spec_verify_tree)(_ptr(logits), _logits_dtype(logits), _ptr(node_tokens),
                              _ptr(parents), B, N, V, int(mode), float(temperature),
                              int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                              _ptr(out_tokens), _ptr(accept_index), _ptr(accept_len),
                              _ptr(workspace), workspace.numel(), _ptr(dev_status),
                              ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_tree", rc)
    return Result(out_tokens, accept_len, dev_status, accept_index)


def spec_verify_philox(seed: int, offset: int, n_slot: int, n_req: int, out=None,
                       device=None, stream=None) -> torch.Tensor:
    """Raw Philox4x32-10 words [n_slot, n_req, 4] (as int32 bit patterns) for the library's
    counter layout (slot, request, offset)."""
    lib = load_library()
    device = torch.device(device or "cuda")
    stream = stream or torch.cuda.current_stream(device)
    if out is None:
        out = torch.empty((n_slot, n_req, 4), dtype=torch.int32, device=device)
    rc = _on(out.get_device(), lib.spec_verify_philox)(int(seed) & (2**64 - 1), int(offset) & (2**64 - 1), n_slot, n_req,
                                _ptr(out), ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_philox", rc)
    return out


def spec_verify_rejection_noalloc(logits: torch.Tensor, draft_ids: torch.Tensor,
                                  draft_probs: Optional[torch.Tensor] = None, *, temperature: float,
                                  seed: int, offset: int, out_tokens: torch.Tensor,
                                  accept_len: torch.Tensor, out_probs=None, dev_status=None,
                                  stream=None) -> Result:
    """spec_verify_rejection without a workspace, for callers that cannot allocate device memory
    while they verify: the library's built-in scratch is used instead.  The caller passes every
    output buffer (and dev_status, or None), so this wrapper allocates nothing either."""
    lib = load_library()
    _check_dev("logits", logits)
    B, k1, V = logits.shape
    k = k1 - 1
    _check_dev("draft_ids", draft_ids, torch.int32)
    if draft_probs is not None:
        _check_dev("draft_probs", draft_probs, torch.float32)
    _check_dev("out_tokens", out_tokens, torch.int32)
    _check_dev("accept_len", accept_len, torch.int32)
    stream = stream or torch.cuda.current_stream(logits.device)
    rc = _on(logits.device.index, lib.spec_verify_rejection_noalloc)(_ptr(logits), _logits_dtype(logits), _ptr(draft_ids),
                                           _ptr(draft_probs), B, k, V, float(temperature),
                                           int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                                           _ptr(out_tokens), _ptr(accept_len), _ptr(out_probs),
                                           _ptr(dev_status), ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_rejection_noalloc", rc)
    return Result(out_tokens, accept_len, dev_status, None, out_probs)


def spec_verify_kv_compact(kv_pool: torch.Tensor, slot_table: torch.Tensor,
                           committed: torch.Tensor, accept_index: torch.Tensor,
                           accept_len: torch.Tensor, *, stacked: bool = False, committed_out=None,
                           dev_status=None, stream=None):
    """Move each request's accepted-path KV rows (as spec_verify_tree reports them) to the
    positions right after its committed prefix, in place in kv_pool, and return
    (committed_out, dev_status).

    kv_pool is [num_slots, ...] with contiguous slot rows, or with stacked=True
    [planes, num_slots, ...] (one plane per layer and K or V) where each plane is contiguous and
    planes may be any 16-byte multiple apart; a slot row's bytes must be a multiple of 16.
    slot_table [B, max_pos], committed [B], accept_index [B, N] and accept_len [B] are int32
    CUDA tensors."""
    lib = load_library()
    if not kv_pool.is_cuda:
        raise ValueError("kv_pool must be a CUDA tensor")
    for name, t in (("slot_table", slot_table), ("committed", committed),
                    ("accept_index", accept_index), ("accept_len", accept_len)):
        _check_dev(name, t, torch.int32)
    B, N = accept_index.shape
    if slot_table.dim() != 2 or slot_table.shape[0] != B or tuple(committed.shape) != (B,) \
            or tuple(accept_len.shape) != (B,):
        raise ValueError("slot_table must be [B, max_pos], committed and accept_len [B]")
    if stacked:
        if kv_pool.dim() < 3 or not kv_pool[0].is_contiguous():
            raise ValueError("a stacked kv_pool is [planes, num_slots, ...] with contiguous planes")
        planes, num_slots = kv_pool.shape[0], kv_pool.shape[1]
        row_bytes = kv_pool[0, 0].numel() * kv_pool.element_size()
        plane_stride = kv_pool.stride(0) * kv_pool.element_size()
    else:
        if kv_pool.dim() < 2 or not kv_pool.is_contiguous():
            raise ValueError("kv_pool must be a contiguous [num_slots, ...] tensor")
        planes, num_slots = 1, kv_pool.shape[0]
        row_bytes = kv_pool[0].numel() * kv_pool.element_size()
        plane_stride = 0
    dev = kv_pool.device
    stream = stream or torch.cuda.current_stream(dev)
    if committed_out is None:
        committed_out = torch.empty(B, dtype=torch.int32, device=dev)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
    rc = _on(dev.index, lib.spec_verify_kv_compact)(_ptr(kv_pool), int(num_slots), int(row_bytes), int(planes),
                                    int(plane_stride), _ptr(slot_table), slot_table.shape[1],
                                    _ptr(committed), _ptr(committed_out), _ptr(accept_index),
                                    _ptr(accept_len), B, N, _ptr(dev_status),
                                    ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_kv_compact", rc)
    return committed_out, dev_status


def _options(temperatures, temperature, threshold_single, threshold_acc, B, device, top_k=None,
             top_p=None):
    for name, t, dt in (("temperatures", temperatures, torch.float32), ("top_k", top_k, torch.int32),
                        ("top_p", top_p, torch.float32)):
        if t is not None:
            _check_dev(name, t, dt)
            if tuple(t.shape) != (B,) or t.device != device:
                raise ValueError(f"{name} must be a [B] {dt} tensor on the logits' device")
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return Options(ptr(temperatures), float(temperature), float(threshold_single), float(threshold_acc),
                   ptr(top_k), ptr(top_p))


def spec_verify_rejection_ex(logits: torch.Tensor, draft_ids: torch.Tensor,
                             draft_probs: Optional[torch.Tensor] = None, *, temperatures=None,
                             temperature: float = 1.0, threshold_single: float = 1.0,
                             threshold_acc: float = 1.0, top_k=None, top_p=None, seed: int = 0,
                             offset: int = 0,
                             out_tokens=None, accept_len=None, out_probs=None, workspace=None,
                             dev_status=None, stream=None) -> Result:
    """spec_verify_rejection with a temperature per request (temperatures [B], 0 = greedy
    request), relaxed thresholds for target-only decisions, and per-request top-k / top-p
    (top_k [B] int32, top_p [B] float32) on the target distribution."""
    lib = load_library()
    _check_dev("logits", logits)
    B, k1, V = logits.shape
    k = k1 - 1
    _check_dev("draft_ids", draft_ids, torch.int32)
    if draft_probs is not None:
        _check_dev("draft_probs", draft_probs, torch.float32)
    dev = logits.device
    stream = stream or torch.cuda.current_stream(dev)
    opt = _options(temperatures, temperature, threshold_single, threshold_acc, B, dev, top_k, top_p)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, k1), dtype=torch.int32, device=dev)
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    nbytes = spec_verify_workspace_bytes(MODE_REJECTION, B, k, V)
    workspace, dev_status = _ws_and_status(nbytes, dev, stream, workspace, dev_status)
    rc = _on(dev.index, lib.spec_verify_rejection_ex)(_ptr(logits), _logits_dtype(logits), _ptr(draft_ids),
                                      _ptr(draft_probs), B, k, V, ctypes.byref(opt),
                                      int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                                      _ptr(out_tokens), _ptr(accept_len), _ptr(out_probs),
                                      _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                      ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_rejection_ex", rc)
    return Result(out_tokens, accept_len, dev_status, None, out_probs)


def spec_verify_tree_ex(logits: torch.Tensor, node_tokens: torch.Tensor, parents: torch.Tensor, *,
                        temperatures=None, temperature: float = 1.0, threshold_single: float = 1.0,
                        threshold_acc: float = 1.0, top_k=None, top_p=None, seed: int = 0,
                        offset: int = 0, out_tokens=None,
                        accept_index=None, accept_len=None, workspace=None, dev_status=None,
                        stream=None) -> Result:
    """spec_verify_tree where a request with temperature 0 walks by argmax and the others by the
    target-only rule at their temperature, with relaxed thresholds."""
    lib = load_library()
    _check_dev("logits", logits)
    B, N, V = logits.shape
    _check_dev("node_tokens", node_tokens, torch.int32)
    _check_dev("parents", parents, torch.int32)
    dev = logits.device
    stream = stream or torch.cuda.current_stream(dev)
    opt = _options(temperatures, temperature, threshold_single, threshold_acc, B, dev, top_k, top_p)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, N), dtype=torch.int32, device=dev)
    accept_index = accept_index if accept_index is not None else torch.empty((B, N), dtype=torch.int32, device=dev)
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    nbytes = spec_verify_workspace_bytes(MODE_TREE, B, N, V)
    workspace, dev_status = _ws_and_status(nbytes, dev, stream, workspace, dev_status)
    rc = _on(dev.index, lib.spec_verify_tree_ex)(_ptr(logits), _logits_dtype(logits), _ptr(node_tokens),
                                 _ptr(parents), B, N, V, ctypes.byref(opt), int(seed) & (2**64 - 1),
                                 int(offset) & (2**64 - 1), _ptr(out_tokens), _ptr(accept_index),
                                 _ptr(accept_len), _ptr(workspace), workspace.numel(),
                                 _ptr(dev_status), ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_tree_ex", rc)
    return Result(out_tokens, accept_len, dev_status, accept_index)


def spec_verify_plan_budget(conf: torch.Tensor, cost: torch.Tensor, num_drafts=None, *,
                            admitted=None, budget=None, best_rate=None, stream=None):
    """Adaptive verification budget: conf [B, K] float32, cost [B*K + 1] float64, num_drafts [B]
    int32 or None (CUDA tensors).  Returns (admitted [B] int32, budget [1] int32, best_rate [1]
    float64), all on the device."""
    lib = load_library()
    _check_dev("conf", conf, torch.float32)
    _check_dev("cost", cost, torch.float64)
    B, K = conf.shape
    if cost.numel() != B * K + 1:
        raise ValueError("cost must hold B*K + 1 entries")
    if num_drafts is not None:
        _check_dev("num_drafts", num_drafts, torch.int32)
    dev = conf.device
    stream = stream or torch.cuda.current_stream(dev)
    admitted = admitted if admitted is not None else torch.empty(B, dtype=torch.int32, device=dev)
    budget = budget if budget is not None else torch.empty(1, dtype=torch.int32, device=dev)
    best_rate = best_rate if best_rate is not None else torch.empty(1, dtype=torch.float64, device=dev)
    nbytes = int(lib.spec_verify_plan_budget_workspace_bytes(B, K))
    if nbytes == 0:
        raise ValueError("the budget planner takes B * K <= 16384 slots and K <= 64")
    ws = _plan_workspaces.get(nbytes, dev.index, stream, stream.cuda_stream)
    rc = _on(dev.index, lib.spec_verify_plan_budget)(_ptr(conf), _ptr(num_drafts), B, K, _ptr(cost), _ptr(admitted),
                                     _ptr(budget), _ptr(best_rate), _ptr(ws), ws.numel(),
                                     ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SpecVerifyError("spec_verify_plan_budget", rc)
    return admitted, budget, best_rate


# --------------------------------------------------------------------------------------------
# Around verification: the cache's new rows, attention over it, log probabilities
# --------------------------------------------------------------------------------------------
class Attention(NamedTuple):
    out: torch.Tensor
    lse: Optional[torch.Tensor]


class Logprobs(NamedTuple):
    logprobs: torch.Tensor
    entropy: torch.Tensor
    ranks: torch.Tensor
    top_ids: Optional[torch.Tensor]
    top_logprobs: Optional[torch.Tensor]


_HALF = {torch.bfloat16: BF16, torch.float16: FP16}
_INT32, _FP32 = torch.int32, torch.float32


def _half_dtype(q: torch.Tensor) -> int:
    code = _HALF.get(q.dtype)
    if code is None:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    return code


def _same(what, device: int, **tensors):
    """What the first tensor's type and device are, the others' have to be."""
    for name, t in tensors.items():
        if t.dtype is not what:
            raise TypeError(f"{name} must be {what}, got {t.dtype}")
        if t.get_device() != device:
            raise ValueError(f"{name} must be on cuda:{device}")


def _device_of(name: str, t: torch.Tensor) -> int:
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return device


def _row_stride(name: str, t: torch.Tensor, B: int, N: int, H: int, D: int) -> int:
    """Elements from one [heads, D] row of [B, N, heads, D] to the next: heads contiguous, rows evenly
    spaced (a view into a projection's output will do)."""
    sb, sn, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name}'s heads must be contiguous")
    if N == 1:
        return sb if B > 1 else max(sn, H * D)
    if B > 1 and sb != N * sn:
        raise ValueError(f"{name}'s rows must be evenly spaced")
    return sn


def _slot_stride(name: str, t: torch.Tensor, H: int, D: int) -> int:
    """Elements from one slot of [num_slots, Hkv, D] to the next: slots contiguous, any distance apart."""
    ss, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name}'s slots must be contiguous")
    return ss if t.shape[0] > 1 else max(ss, H * D)


def _index(name: str, t: torch.Tensor, shape, device: int) -> int:
    """An int32 index tensor's address."""
    if t.dtype is not _INT32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on cuda:{device}")
    return t.data_ptr()


def _result(name: str, t: Optional[torch.Tensor], shape, dtype, device: int, stream) -> torch.Tensor:
    """A caller's output checked, or a new one that the stream's work may write at once: from memory that its
    earlier work has had, kept until the current stream's work of the time it is dropped is done."""
    if t is None:
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=device)
        t.record_stream(torch.cuda.current_stream(device))
    elif t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{device}")
    return t


def _status(dev_status: Optional[torch.Tensor], device: int):
    if dev_status is None:
        return None
    if dev_status.dtype is not _INT32 or dev_status.get_device() != device:
        raise ValueError(f"dev_status must be an int32 tensor on cuda:{device}")
    return dev_status.data_ptr()


def _raw_stream(stream, device: int) -> int:
    # (torch.cuda.current_stream builds an object for each call, a tenth of a small call's host time.)
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _angles(cos_sin: Optional[torch.Tensor], device: int):
    """(address, positions, rotary_dim) of a table of cosines and sines; None: no rotation."""
    if cos_sin is None:
        return 0, 0, 0
    if cos_sin.dtype is not _FP32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous() or cos_sin.get_device() != device:
        raise ValueError(f"cos_sin must be a contiguous float32 [positions, rotary_dim] tensor on cuda:{device}")
    return cos_sin.data_ptr(), *cos_sin.shape


def spec_verify_kv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, slot_table: torch.Tensor, committed: torch.Tensor,
                          cos_sin: Optional[torch.Tensor], *, parents=None, num_nodes=None,
                          interleaved: bool = False, q_out=None, dev_status=None,
                          stream=None) -> torch.Tensor:
    """Write a verify forward's keys (rotated by position) and values into one layer's paged cache,
    in place, and return the rotated queries.

    q [B, N, Hq, D], k and v [B, N, Hkv, D] (bf16 / fp16; may be views into one projection's rows),
    k_cache and v_cache [num_slots, Hkv, D], slot_table [B, max_pos] and committed [B] int32,
    cos_sin [positions, rotary_dim] fp32 (cosines, then sines; None: no rotation), parents [B, N]
    int32 (None: a chain or a prompt), num_nodes [B] int32 (None: all N).  Without dev_status,
    faults in the data show in the returned rows alone (NaN)."""
    lib = _lib or load_library()
    code, dt, dev = _half_dtype(q), q.dtype, _device_of("q", q)
    B, N, Hq, D = q.shape
    S, Hkv, _ = csh = k_cache.shape
    if csh[2] != D or v_cache.shape != csh:
        raise ValueError("k_cache and v_cache must be [num_slots, Hkv, D]")
    if k.shape != (B, N, Hkv, D) or v.shape != (B, N, Hkv, D):
        raise ValueError(f"k and v must be {[B, N, Hkv, D]}")
    _same(dt, dev, k=k, v=v, k_cache=k_cache, v_cache=v_cache)
    cs, rot_positions, rot = _angles(cos_sin, dev)
    max_pos = slot_table.shape[-1]
    q_out = _result("q_out", q_out, (B, N, Hq, D), dt, dev, stream)
    rc = _on(dev, lib.spec_verify_kv_append)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), code, _row_stride("q", q, B, N, Hq, D),
        _row_stride("k", k, B, N, Hkv, D), _row_stride("v", v, B, N, Hkv, D), q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), S, _slot_stride("k_cache", k_cache, Hkv, D),
        _slot_stride("v_cache", v_cache, Hkv, D), _index("slot_table", slot_table, (B, max_pos), dev), max_pos,
        _index("committed", committed, (B,), dev),
        None if parents is None else _index("parents", parents, (B, N), dev),
        None if num_nodes is None else _index("num_nodes", num_nodes, (B,), dev), cs, rot_positions, rot,
        bool(interleaved), B, N, Hq, Hkv, D, _status(dev_status, dev), _raw_stream(stream, dev))
    if rc != OK:
        raise SpecVerifyError("spec_verify_kv_append", rc)
    return q_out


@functools.lru_cache(maxsize=256)
def spec_verify_attention_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, D: int, max_pos: int) -> int:
    return int(load_library().spec_verify_attention_workspace_bytes(B, N, Hq, Hkv, D, max_pos))


def spec_verify_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          slot_table: torch.Tensor, committed: torch.Tensor, *, parents=None,
                          num_nodes=None, scale: Optional[float] = None, out=None, lse=None,
                          want_lse: bool = False, workspace=None, dev_status=None,
                          stream=None) -> Attention:
    """Attention of the verify step's nodes (N = 1: plain decoding) over one layer's paged cache:
    each sees the committed positions and the nodes on its path from the root.

    q [B, N, Hq, D] rotated, the cache and its tables as spec_verify_kv_append left them; scale
    defaults to D ** -0.5.  Returns out [B, N, Hq, D] and, when wanted or given, lse [B, N, Hq] fp32.
    Without dev_status, faults in the data show in the returned rows alone (NaN).  A wait inside the kernel
    that runs out (status 7) does not show there but in dev_status and spec_verify_wait_timeouts;
    spec_verify_reset_workspaces has to follow it."""
    lib = _lib or load_library()
    code, dt, dev = _half_dtype(q), q.dtype, _device_of("q", q)
    B, N, Hq, D = q.shape
    S, Hkv, _ = csh = k_cache.shape
    if csh[2] != D or v_cache.shape != csh:
        raise ValueError("k_cache and v_cache must be [num_slots, Hkv, D]")
    _same(dt, dev, k_cache=k_cache, v_cache=v_cache)
    max_pos = slot_table.shape[-1]
    out = _result("out", out, (B, N, Hq, D), dt, dev, stream)
    if lse is not None or want_lse:
        lse = _result("lse", lse, (B, N, Hq), _FP32, dev, stream)
    raw = _raw_stream(stream, dev)
    if workspace is None:
        nbytes = spec_verify_attention_workspace_bytes(B, N, Hq, Hkv, D, max_pos)
        workspace = _workspaces.get(nbytes, dev, stream, raw)
    rc = _on(dev, lib.spec_verify_attention)(
        q.data_ptr(), code, _row_stride("q", q, B, N, Hq, D), k_cache.data_ptr(), v_cache.data_ptr(), S,
        _slot_stride("k_cache", k_cache, Hkv, D), _slot_stride("v_cache", v_cache, Hkv, D),
        _index("slot_table", slot_table, (B, max_pos), dev), max_pos, _index("committed", committed, (B,), dev),
        None if parents is None else _index("parents", parents, (B, N), dev),
        None if num_nodes is None else _index("num_nodes", num_nodes, (B,), dev), B, N, Hq, Hkv, D,
        D ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _status(dev_status, dev), raw)
    if rc != OK:
        raise SpecVerifyError("spec_verify_attention", rc)
    return Attention(out, lse)


@functools.lru_cache(maxsize=256)
def spec_verify_logprobs_workspace_bytes(B: int, T: int, V: int, top_n: int) -> int:
    return int(load_library().spec_verify_logprobs_workspace_bytes(B, T, V, top_n))


def spec_verify_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, row_index=None, temperatures=None,
                         temperature: float = 1.0, top_n: int = 0, logprobs=None, entropy=None, ranks=None,
                         top_ids=None, top_logprobs=None, workspace=None, dev_status=None,
                         stream=None) -> Logprobs:
    """Log probability, rank, entropy and top_n alternatives of given tokens: logits [B, rows, V] (bf16
    / fp32) as verified, tokens [B, T] int32 (verification's out_tokens; -1: nothing there), row_index
    [B, T] int32 (a tree's accept_index; None: token t belongs to row t), temperatures [B] fp32.
    Without dev_status, faults in the data show in the returned entries alone (NaN, -1).  Status 7 as for
    spec_verify_attention."""
    lib = _lib or load_library()
    dev = _device_of("logits", logits)
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    B, rows, V = logits.shape
    T = tokens.shape[-1]
    if temperatures is not None and (temperatures.dtype is not _FP32 or temperatures.shape != (B,)
                                     or temperatures.get_device() != dev or not temperatures.is_contiguous()):
        raise ValueError(f"temperatures must be a contiguous float32 tensor [{B}] on cuda:{dev}")
    logprobs = _result("logprobs", logprobs, (B, T), _FP32, dev, stream)
    entropy = _result("entropy", entropy, (B, T), _FP32, dev, stream)
    ranks = _result("ranks", ranks, (B, T), _INT32, dev, stream)
    if top_n:
        top_ids = _result("top_ids", top_ids, (B, T, top_n), _INT32, dev, stream)
        top_logprobs = _result("top_logprobs", top_logprobs, (B, T, top_n), _FP32, dev, stream)
    else:
        top_ids = top_logprobs = None
    raw = _raw_stream(stream, dev)
    if workspace is None:
        workspace = _workspaces.get(spec_verify_logprobs_workspace_bytes(B, T, V, top_n), dev, stream, raw)
    rc = _on(dev, lib.spec_verify_logprobs)(
        logits.data_ptr(), _logits_dtype(logits), _index("tokens", tokens, (B, T), dev),
        None if row_index is None else _index("row_index", row_index, (B, T), dev), B, rows, T, V,
        None if temperatures is None else temperatures.data_ptr(), temperature, top_n, logprobs.data_ptr(),
        entropy.data_ptr(), ranks.data_ptr(), None if top_ids is None else top_ids.data_ptr(),
        None if top_logprobs is None else top_logprobs.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _status(dev_status, dev), raw)
    if rc != OK:
        raise SpecVerifyError("spec_verify_logprobs", rc)
    return Logprobs(logprobs, entropy, ranks, top_ids, top_logprobs)
