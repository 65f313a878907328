"""Batched speculative-decoding verification on GB300 (sm_103a).

A thin ctypes binding over ``libspecverify.so``, whose C ABI is declared in
``include/specverify.h``.  Every step of the verification runs in the
library's CUDA kernels; this module only checks tensor shapes and dtypes,
allocates outputs and scratch with PyTorch, and passes device pointers and
the current CUDA stream.  There is no CPU fallback: if the library is not
built, the calls raise.

Notation (nextadmin.net "Speculative Decoding", § Core algorithm): q is the
target distribution, p the draft distribution, d_i the K drafted tokens.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

from .build import LIB as _LIB_PATH

try:   # the current stream's handle, in a twentieth of the public way's 2 us
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

__all__ = [
    "SpecVerifyError", "Aux", "Filters", "spec_filter_sample", "spec_verify_filtered", "spec_filter_workspace_bytes",
    "spec_verify_window_attention",
    "spec_verify", "spec_verify_greedy", "spec_verify_shortlist",
    "spec_workspace_bytes", "spec_philox_words", "spec_draft_sample", "spec_kv_commit", "spec_verify_tree_greedy", "spec_tree_mask",
    "spec_kv_commit_quant", "spec_kv_read_quant", "spec_verify_attention", "spec_attention_workspace_bytes",
    "spec_verify_shortlist_pos", "spec_status_string", "spec_launch_count", "spec_verify_static", "library_path", "load",
]

SPEC_F32, SPEC_BF16 = 0, 1
STATUS = {0: "SPEC_OK", 1: "SPEC_ERR_INVALID_ARG", 2: "SPEC_ERR_NONFINITE", 3: "SPEC_ERR_TOKEN_RANGE",
          4: "SPEC_ERR_SHORTLIST", 5: "SPEC_ERR_UNSUPPORTED", 6: "SPEC_ERR_CUDA", 7: "SPEC_ERR_TIMEOUT"}


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({spec_status_string(code)})")
        self.code = code


class _AuxStruct(ctypes.Structure):
    _fields_ = [("q_draft", ctypes.c_void_p), ("p_draft", ctypes.c_void_p),
                ("residual_mass", ctypes.c_void_p), ("row_lse", ctypes.c_void_p),
                ("device_status", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libspecverify.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise ImportError(f"{_LIB_PATH} is missing: build it first "
                                  "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(_LIB_PATH)
            P, I, U64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_float
            Z = ctypes.c_size_t
            lib.spec_workspace_bytes.argtypes = [I, I, I, I]
            lib.spec_workspace_bytes.restype = Z
            lib.spec_verify.argtypes = [P, I, P, I, I, P, I, I, I, F, U64, P, P, P, Z, P, P]
            lib.spec_verify.restype = I
            lib.spec_verify_greedy.argtypes = [P, I, P, I, I, I, P, P, P, Z, P, P]
            lib.spec_verify_greedy.restype = I
            lib.spec_verify_shortlist.argtypes = [P, I, P, I, I, P, I, P, I, I, I, F, U64, P, P, P, Z, P, P]
            lib.spec_verify_shortlist.restype = I
            lib.spec_philox_words.argtypes = [U64, ctypes.c_uint32, I, I, P, P]
            lib.spec_philox_words.restype = I
            lib.spec_status_string.argtypes = [I]
            lib.spec_status_string.restype = ctypes.c_char_p
            lib.spec_verify_static.argtypes = [P, I, P, P, I, I, I, F, U64, P, P, P, P]
            lib.spec_verify_static.restype = I
            L64 = ctypes.c_longlong
            lib.spec_verify_shortlist_pos.argtypes = [P, I, P, I, P, L64, L64, P, I, P, I, I, I, F, U64, P, P, P,
                                                      Z, P, P]
            lib.spec_verify_shortlist_pos.restype = I
            lib.spec_tree_workspace_bytes.argtypes = [I, I, I]
            lib.spec_tree_workspace_bytes.restype = Z
            lib.spec_verify_tree_greedy.argtypes = [P, I, P, P, I, I, I, P, P, P, P, Z, P, P]
            lib.spec_verify_tree_greedy.restype = I
            lib.spec_tree_mask.argtypes = [P, I, I, P, P, P]
            lib.spec_tree_mask.restype = I
            lib.spec_kv_commit.argtypes = [P, P, I, I, I, I, Z, P, P, P, P]
            lib.spec_kv_commit.restype = I
            lib.spec_kv_commit_quant.argtypes = [P, P, P, I, P, I, I, I, I, I, I, I, P, P, P, P]
            lib.spec_kv_commit_quant.restype = I
            lib.spec_kv_read_quant.argtypes = [P, P, P, P, I, I, I, I, I, I, P, I, P, P]
            lib.spec_kv_read_quant.restype = I
            lib.spec_attention_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
            lib.spec_attention_workspace_bytes.restype = Z
            lib.spec_verify_attention.argtypes = [P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, I, F, P, P, P, Z, P, P]
            lib.spec_verify_attention.restype = I
            lib.spec_verify_window_attention.argtypes = [P, P, P, I, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P, Z, P, P]
            lib.spec_verify_window_attention.restype = I
            lib.spec_draft_sample.argtypes = [P, I, I, I, I, F, U64, P, P, P, P]
            lib.spec_draft_sample.restype = I
            lib.spec_filter_sample.argtypes = [P, I, P, I, I, I, P, P, P, P, P]
            lib.spec_filter_sample.restype = I
            lib.spec_filter_workspace_bytes.argtypes = [I, I, I]
            lib.spec_filter_workspace_bytes.restype = Z
            lib.spec_verify_filtered.argtypes = [P, I, P, P, P, I, I, I, P, P, P, P, P, Z, P, P]
            lib.spec_verify_filtered.restype = I
            lib.spec_launch_count.argtypes = []
            lib.spec_launch_count.restype = U64
            _lib = lib
    return _lib


def spec_launch_count() -> int:
    """Kernels the library has launched in this process (all entry points)."""
    return int(load().spec_launch_count())


def spec_status_string(code: int) -> str:
    return load().spec_status_string(int(code)).decode()


def spec_workspace_bytes(B: int, K: int, V: int, S: int = 0) -> int:
    return int(load().spec_workspace_bytes(int(B), int(K), int(V), int(S)))


class Aux:
    """Optional per-call outputs (device tensors, any may be None).  Asking for
    q_draft, p_draft or row_lse makes the call evaluate every position."""

    def __init__(self, q_draft=None, p_draft=None, residual_mass=None, row_lse=None, device_status=None):
        self.q_draft, self.p_draft, self.residual_mass = q_draft, p_draft, residual_mass
        self.row_lse, self.device_status = row_lse, device_status

    @classmethod
    def alloc(cls, B: int, K: int, device, full: bool = True) -> "Aux":
        f = dict(dtype=torch.float32, device=device)
        nan = float("nan")
        return cls(q_draft=torch.full((B, K), nan, **f) if full else None,
                   p_draft=torch.full((B, K), nan, **f) if full else None,
                   residual_mass=torch.full((B,), nan, **f),
                   row_lse=torch.full((B, 2 * K + 1), nan, **f) if full else None,
                   device_status=torch.full((1,), -1, dtype=torch.int32, device=device))

    def _struct(self, B, K):
        def ptr(t, shape, dtype):
            if t is None:
                return None
            _check(t, shape, (dtype,), "aux")
            return t.data_ptr()
        return _AuxStruct(ptr(self.q_draft, (B, K), torch.float32), ptr(self.p_draft, (B, K), torch.float32),
                          ptr(self.residual_mass, (B,), torch.float32),
                          ptr(self.row_lse, (B, 2 * K + 1), torch.float32),
                          ptr(self.device_status, (1,), torch.int32))


class _FiltersStruct(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p)]


class Filters:
    """What each sequence asks for: device tensors [B], or None where it is off.
    temperature float32 (0: the largest logit alone; None: 1), top_k int32 (<= 0:
    all), top_p float32 (>= 1: all), min_p float32 (<= 0: all).  They apply in this
    order: see spec_filters_t in include/specverify.h."""
    __slots__ = ("temperature", "top_k", "top_p", "min_p")

    def __init__(self, temperature=None, top_k=None, top_p=None, min_p=None):
        self.temperature, self.top_k, self.top_p, self.min_p = temperature, top_k, top_p, min_p

    @classmethod
    def fill(cls, B: int, device, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0,
             min_p: float = 0.0) -> "Filters":
        """The same for B sequences."""
        return cls(torch.full((B,), temperature, dtype=torch.float32, device=device),
                   torch.full((B,), top_k, dtype=torch.int32, device=device),
                   torch.full((B,), top_p, dtype=torch.float32, device=device),
                   torch.full((B,), min_p, dtype=torch.float32, device=device))

    def _struct(self, B, index, name):
        shape = (B,)

        def ptr(t, dtype, what):
            if t is None:
                return None
            _need(t, shape, dtype, index, name, what)
            return t.data_ptr()
        return _FiltersStruct(ptr(self.temperature, torch.float32, ".temperature"),
                              ptr(self.top_k, torch.int32, ".top_k"), ptr(self.top_p, torch.float32, ".top_p"),
                              ptr(self.min_p, torch.float32, ".min_p"))


# ------------------------------------------------------------------ helpers
def _check(t, shape, dtypes, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.shape != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _index(t, name):
    """The device of a call's first tensor, which must be the current one: the launches go there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    index = t.get_device()
    if index != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{index}, but cuda:{torch.cuda.current_device()} is the current device")
    return index


def _need(t, shape, dtype, index, name, more=""):
    """_check for one type, and the tensors of a call lie on one device."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    _check(t, shape, (dtype,), name + more)
    raise ValueError(f"{name}{more} is on {t.device}, the call's other tensors on cuda:{index}")


def _own_workspace(workspace, index):
    """The caller's: its bytes are counted by its elements, so these lie side by side."""
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index:
        raise TypeError(f"workspace must be a CUDA tensor on cuda:{index}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _dt(t):
    return SPEC_BF16 if t.dtype == torch.bfloat16 else SPEC_F32


_HERE = contextlib.nullcontext()


class _On:
    """torch.cuda.stream in half its time."""
    __slots__ = ("stream", "before", "device")

    def __init__(self, stream, device):
        self.stream, self.device = stream, torch.cuda.current_device()
        self.before = torch.cuda.current_stream(device)

    def __enter__(self):
        torch.cuda.set_stream(self.stream)
        return self.before

    def __exit__(self, *exc):
        torch.cuda.set_stream(self.before)
        if self.device != self.before.device_index:
            torch.cuda.set_device(self.device)


def _on(device, stream):
    """A context in which the stream that a call goes to (None: the current one) is
    the current one: memory for the call comes from that stream's pool, and what is
    asked of the current stream is asked of it.  Gives the stream that was current,
    or None where that is the same."""
    if stream is None:
        return _HERE
    raw = _stream(device, stream)
    if raw == _stream(device, None):
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    return _On(stream, device)


def _new(shape, dtype, device, before):
    """An output, made inside `_on`.  It comes from the pool of the stream that the
    call goes to, as memory of another's may have work pending there, and the
    allocator learns that the stream that was current, `before`, is to use it."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if before is not None:
        t.record_stream(before)
    return t


class _Kept(threading.local):
    """Device memory kept from call to call, each thread its own: a call is more
    than one launch, and those of two threads on one stream may interleave.
    Freed as its thread ends."""

    def __init__(self):
        self.workspaces: dict = {}
        self.scratch: dict = {}


_kept = _Kept()


def _workspace(device, st, nbytes, sizes):
    """This thread's workspace for (device, st), the current stream.  The library
    leaves it ready for the next call with the same sizes; when the sizes change, it
    is zero-filled again (on the same stream) before the call.  A call under capture
    gets one of its own from the graph's pool, zero-filled by every replay: other
    calls may have used the kept one with other sizes since, or have replaced it."""
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, st)
    ent = _kept.workspaces.get(key)
    if ent is None or ent[0].numel() < nbytes:
        ent = [torch.zeros(max(nbytes, 1 << 16), dtype=torch.uint8, device=device), sizes]
        _kept.workspaces[key] = ent
    elif ent[1] != sizes:
        ent[0].zero_()
        ent[1] = sizes
    return ent[0]


def _outs(B, K, device, out_tokens, out_accept_len, before):
    if out_tokens is None:
        out_tokens = _new((B, K + 1), torch.int32, device, before)
    if out_accept_len is None:
        out_accept_len = _new((B,), torch.int32, device, before)
    _check(out_tokens, (B, K + 1), (torch.int32,), "out_tokens")
    _check(out_accept_len, (B,), (torch.int32,), "out_accept_len")
    return out_tokens, out_accept_len


def _stream(device, stream):
    if stream is None:
        index = device.index
        return _raw_stream(torch.cuda.current_device() if index is None else index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ws_args(device, st, nbytes, workspace, sizes):
    if workspace is None:
        workspace = _workspace(device, st, nbytes, sizes)
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    return workspace, workspace.numel() * workspace.element_size()


# ------------------------------------------------------------------ entry points
def spec_verify(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor, T: float, seed: int,
                *, draft_is_probs: bool = False, out_tokens=None, out_accept_len=None, workspace=None,
                aux: Aux | None = None, stream=None):
    """One verification round for B sequences.

    target [B][K+1][V] float32/bfloat16 logits; draft [B][K][V] logits of the
    same dtype, or float32 probabilities with ``draft_is_probs``; draft_tokens
    [B][K] int32.  T == 0 runs the greedy rule.  Returns (out_tokens [B][K+1],
    out_accept_len [B]) on the device, asynchronously on the current stream.
    """
    B, K1, V = target.shape
    K = K1 - 1
    _check(target, (B, K + 1, V), (torch.float32, torch.bfloat16), "target")
    _check(draft, (B, K, V), (torch.float32,) if draft_is_probs else (target.dtype,), "draft")
    _check(draft_tokens, (B, K), (torch.int32,), "draft_tokens")
    dev = target.device
    st = _stream(dev, stream)
    with _on(dev, stream) as before:
        out_tokens, out_accept_len = _outs(B, K, dev, out_tokens, out_accept_len, before)
        workspace, wsb = _ws_args(dev, st, spec_workspace_bytes(B, K, V, 0), workspace, (B, K, V, 0))
    ax = aux._struct(B, K) if aux is not None else None
    rc = load().spec_verify(target.data_ptr(), _dt(target), draft.data_ptr(), _dt(draft), int(draft_is_probs),
                            draft_tokens.data_ptr(), B, K, V, float(T), int(seed) & (2**64 - 1),
                            out_tokens.data_ptr(), out_accept_len.data_ptr(), workspace.data_ptr(), wsb,
                            ctypes.byref(ax) if ax is not None else None, st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify")
    return out_tokens, out_accept_len


def spec_verify_greedy(target: torch.Tensor, draft_tokens: torch.Tensor, *, out_tokens=None,
                       out_accept_len=None, workspace=None, aux: Aux | None = None, stream=None):
    """Greedy verification: accept d_i while d_i == argmax q_i (lowest index on ties)."""
    B, K1, V = target.shape
    K = K1 - 1
    _check(target, (B, K + 1, V), (torch.float32, torch.bfloat16), "target")
    _check(draft_tokens, (B, K), (torch.int32,), "draft_tokens")
    dev = target.device
    st = _stream(dev, stream)
    with _on(dev, stream) as before:
        out_tokens, out_accept_len = _outs(B, K, dev, out_tokens, out_accept_len, before)
        workspace, wsb = _ws_args(dev, st, spec_workspace_bytes(B, K, V, 0), workspace, (B, K, V, 0))
    ax = aux._struct(B, K) if aux is not None else None
    rc = load().spec_verify_greedy(target.data_ptr(), _dt(target), draft_tokens.data_ptr(), B, K, V,
                                   out_tokens.data_ptr(), out_accept_len.data_ptr(), workspace.data_ptr(), wsb,
                                   ctypes.byref(ax) if ax is not None else None, st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify_greedy")
    return out_tokens, out_accept_len


def spec_verify_static(target: torch.Tensor, draft: torch.Tensor | None, draft_tokens: torch.Tensor, T: float,
                       seed: int, *, out_tokens=None, out_accept_len=None, aux: Aux | None = None, stream=None):
    """spec_verify without a workspace: the library's own 256-byte scratch
    (see include/specverify.h).  Draft logits only; T == 0 is greedy (draft
    may be None).  Raises SpecVerifyError (SPEC_ERR_UNSUPPORTED) for shapes
    that need a workspace.  Calls must not overlap on the GPU."""
    B, K1, V = target.shape
    K = K1 - 1
    _check(target, (B, K + 1, V), (torch.float32, torch.bfloat16), "target")
    if T > 0:
        _check(draft, (B, K, V), (target.dtype,), "draft")
    _check(draft_tokens, (B, K), (torch.int32,), "draft_tokens")
    dev = target.device
    st = _stream(dev, stream)
    with _on(dev, stream) as before:
        out_tokens, out_accept_len = _outs(B, K, dev, out_tokens, out_accept_len, before)
    ax = aux._struct(B, K) if aux is not None else None
    rc = load().spec_verify_static(target.data_ptr(), _dt(target), draft.data_ptr() if (draft is not None and T > 0)
                                   else None, draft_tokens.data_ptr(), B, K, V, float(T), int(seed),
                                   out_tokens.data_ptr(), out_accept_len.data_ptr(),
                                   ctypes.byref(ax) if ax is not None else None, st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify_static")
    return out_tokens, out_accept_len


def spec_verify_shortlist(target: torch.Tensor, draft_sl: torch.Tensor, shortlist_idx: torch.Tensor,
                          draft_tokens: torch.Tensor, T: float, seed: int, *, draft_is_probs: bool = False,
                          out_tokens=None, out_accept_len=None, workspace=None, aux: Aux | None = None,
                          stream=None):
    """Verification with a draft defined on a per-sequence shortlist.

    draft_sl [B][K][S] (logits of the target's dtype, or float32 probabilities),
    shortlist_idx [B][S] int32 strictly ascending inside [0, V)."""
    B, K1, V = target.shape
    K = K1 - 1
    S = shortlist_idx.shape[-1]
    _check(target, (B, K + 1, V), (torch.float32, torch.bfloat16), "target")
    _check(draft_sl, (B, K, S), (torch.float32,) if draft_is_probs else (target.dtype,), "draft_sl")
    _check(shortlist_idx, (B, S), (torch.int32,), "shortlist_idx")
    _check(draft_tokens, (B, K), (torch.int32,), "draft_tokens")
    dev = target.device
    st = _stream(dev, stream)
    with _on(dev, stream) as before:
        out_tokens, out_accept_len = _outs(B, K, dev, out_tokens, out_accept_len, before)
        workspace, wsb = _ws_args(dev, st, spec_workspace_bytes(B, K, V, S), workspace, (B, K, V, S))
    ax = aux._struct(B, K) if aux is not None else None
    rc = load().spec_verify_shortlist(target.data_ptr(), _dt(target), draft_sl.data_ptr(), _dt(draft_sl),
                                      int(draft_is_probs), shortlist_idx.data_ptr(), S, draft_tokens.data_ptr(),
                                      B, K, V, float(T), int(seed) & (2**64 - 1), out_tokens.data_ptr(),
                                      out_accept_len.data_ptr(), workspace.data_ptr(), wsb,
                                      ctypes.byref(ax) if ax is not None else None, st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify_shortlist")
    return out_tokens, out_accept_len


def spec_philox_words(seed: int, tag: int, B: int, P: int, device=None, stream=None) -> torch.Tensor:
    """The Philox4x32-10 words the kernels draw: [B][P][4] (int32 storage of uint32)."""
    device = torch.device(device if device is not None else "cuda")
    st = _stream(device, stream)
    with _on(device, stream) as before:
        out = _new((B, P, 4), torch.int32, device, before)
    rc = load().spec_philox_words(int(seed) & (2**64 - 1), int(tag), B, P, out.data_ptr(), st)
    if rc:
        raise SpecVerifyError(rc, "spec_philox_words")
    return out


def spec_draft_sample(draft: torch.Tensor, T: float, seed: int, *, out_tokens=None, out_prob=None,
                      device_status=None, stream=None):
    """Draft tokens d_i ~ softmax(draft[b][i] / T) by inverse CDF on Philox
    uniforms (counter (i, b, 1, 0)), with p_i(d_i).  draft [B][K][V] float32 or
    bfloat16 logits.  T == 0 takes the first argmax (probability 1).  Returns
    (out_tokens [B][K] int32, out_prob [B][K] float32) on the device."""
    B, K, V = draft.shape
    _check(draft, (B, K, V), (torch.float32, torch.bfloat16), "draft")
    dev = draft.device
    with _on(dev, stream) as before:
        if out_tokens is None:
            out_tokens = _new((B, K), torch.int32, dev, before)
        if out_prob is None:
            out_prob = _new((B, K), torch.float32, dev, before)
    _check(out_tokens, (B, K), (torch.int32,), "out_tokens")
    _check(out_prob, (B, K), (torch.float32,), "out_prob")
    if device_status is not None:
        _check(device_status, (1,), (torch.int32,), "device_status")
    st = _stream(dev, stream)
    rc = load().spec_draft_sample(draft.data_ptr(), _dt(draft), B, K, V, float(T), int(seed) & (2**64 - 1),
                                  out_tokens.data_ptr(), out_prob.data_ptr(),
                                  device_status.data_ptr() if device_status is not None else None, st)
    if rc:
        raise SpecVerifyError(rc, "spec_draft_sample")
    return out_tokens, out_prob


def spec_filter_sample(logits: torch.Tensor, uniforms: torch.Tensor, filters: Filters | None = None, *,
                       out_tokens=None, out_prob=None, device_status=None, stream=None):
    """Tokens drawn from rows of logits under each sequence's filters by given
    random numbers: logits [B][K][V] float32 or bfloat16, uniforms [B][K] float32 in
    [0, 1).  Returns (out_tokens [B][K] int32, out_prob [B][K] float32, the tokens'
    probabilities among what the filters keep) on the device."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3:
        raise TypeError("logits must be a CUDA tensor [B][K][V]")
    B, K, V = shape = logits.shape
    index, dtype = _index(logits, "logits"), logits.dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16 or not logits.is_contiguous():
        _check(logits, shape, (torch.float32, torch.bfloat16), "logits")
    rows = (B, K)
    _need(uniforms, rows, torch.float32, index, "uniforms")
    if device_status is not None:
        _need(device_status, (1,), torch.int32, index, "device_status")
    fs = ctypes.byref(filters._struct(B, index, "filters")) if filters is not None else None
    if out_tokens is None or out_prob is None:
        dev = logits.device
        with _on(dev, stream) as before:
            if out_tokens is None:
                out_tokens = _new(rows, torch.int32, dev, before)
            if out_prob is None:
                out_prob = _new(rows, torch.float32, dev, before)
    _need(out_tokens, rows, torch.int32, index, "out_tokens")
    _need(out_prob, rows, torch.float32, index, "out_prob")
    st = _raw_stream(index) if stream is None else _stream(logits.device, stream)
    rc = (_lib or load()).spec_filter_sample(
        logits.data_ptr(), 1 if dtype is torch.bfloat16 else 0, uniforms.data_ptr(), B, K, V, fs,
        out_tokens.data_ptr(), out_prob.data_ptr(), None if device_status is None else device_status.data_ptr(), st)
    if rc:
        raise SpecVerifyError(rc, "spec_filter_sample")
    return out_tokens, out_prob


def spec_filter_workspace_bytes(B: int, K: int, V: int) -> int:
    return int(load().spec_filter_workspace_bytes(int(B), int(K), int(V)))


_filter_bytes = functools.lru_cache(maxsize=256)(spec_filter_workspace_bytes)


def spec_verify_filtered(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor,
                         uniforms: torch.Tensor, filters: Filters | None = None, *,
                         draft_filters: Filters | None = None, out_tokens=None, out_accept_len=None, workspace=None,
                         device_status=None, stream=None):
    """Verification between filtered distributions: target [B][K+1][V] and draft
    [B][K][V] float32 or bfloat16 logits, draft_tokens [B][K] int32 drawn from the
    draft's rows under draft_filters (default: filters; spec_filter_sample draws
    them), uniforms [B][K+1][2] float32 in [0, 1): at position i the acceptance
    number, and the number that draws the emitted token if the round ends there.
    Returns (out_tokens [B][K+1], out_accept_len [B]) as spec_verify does.  Without
    workspace (uint8, spec_filter_workspace_bytes(...) elements, one per call in flight)
    the call takes scratch that its thread keeps for the stream, as
    spec_verify_attention does."""
    if not isinstance(target, torch.Tensor) or target.dim() != 3:
        raise TypeError("target must be a CUDA tensor [B][K+1][V]")
    B, K1, V = shape = target.shape
    K = K1 - 1
    index, dtype = _index(target, "target"), target.dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16 or not target.is_contiguous():
        _check(target, shape, (torch.float32, torch.bfloat16), "target")
    _need(draft, (B, K, V), dtype, index, "draft")
    _need(draft_tokens, (B, K), torch.int32, index, "draft_tokens")
    _need(uniforms, (B, K1, 2), torch.float32, index, "uniforms")
    if device_status is not None:
        _need(device_status, (1,), torch.int32, index, "device_status")
    fs = ctypes.byref(filters._struct(B, index, "filters")) if filters is not None else None
    ds = ctypes.byref(draft_filters._struct(B, index, "draft_filters")) if draft_filters is not None else None
    dev = target.device
    st = _stream(dev, stream)
    with _on(dev, stream) as before:
        if out_tokens is None:
            out_tokens = _new((B, K1), torch.int32, dev, before)
        if out_accept_len is None:
            out_accept_len = _new((B,), torch.int32, dev, before)
        if workspace is None:
            workspace = _scratch(_filter_bytes(B, K, V), dev, st)
        else:
            _own_workspace(workspace, index)
    _need(out_tokens, (B, K1), torch.int32, index, "out_tokens")
    _need(out_accept_len, (B,), torch.int32, index, "out_accept_len")
    rc = (_lib or load()).spec_verify_filtered(
        target.data_ptr(), 1 if dtype is torch.bfloat16 else 0, draft.data_ptr(), draft_tokens.data_ptr(),
        uniforms.data_ptr(), B, K, V, fs, ds, out_tokens.data_ptr(), out_accept_len.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, None if device_status is None else device_status.data_ptr(), st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify_filtered")
    return out_tokens, out_accept_len


def spec_kv_commit(cache: torch.Tensor, staged: torch.Tensor | None, accept_len: torch.Tensor,
                   seq_len: torch.Tensor, *, K: int | None = None, device_status=None, stream=None):
    """Commit the accepted drafts' KV entries: cache [NL][B][L][...] (any
    dtype), staged [NL][B][K][...] of the same dtype and entry shape (None:
    entries written in place, then K must be given), accept_len [B] int32 (as
    spec_verify returns it), seq_len [B] int32 updated in place."""
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda or cache.dim() < 4 or not cache.is_contiguous():
        raise TypeError("cache must be a contiguous CUDA tensor [NL][B][L][...]")
    NL, B, L = cache.shape[:3]
    entry = cache[0, 0, 0]
    W = entry.numel() * cache.element_size()
    if staged is not None:
        K = staged.shape[2]
        _check(staged, (NL, B, K) + tuple(cache.shape[3:]), (cache.dtype,), "staged")
    elif K is None:
        raise ValueError("K is needed when the entries were written in place")
    _check(accept_len, (B,), (torch.int32,), "accept_len")
    _check(seq_len, (B,), (torch.int32,), "seq_len")
    if device_status is not None:
        _check(device_status, (1,), (torch.int32,), "device_status")
    st = _stream(cache.device, stream)
    rc = load().spec_kv_commit(cache.data_ptr(), staged.data_ptr() if staged is not None else None, NL, B, int(K), L,
                               W, accept_len.data_ptr(), seq_len.data_ptr(),
                               device_status.data_ptr() if device_status is not None else None, st)
    if rc:
        raise SpecVerifyError(rc, "spec_kv_commit")
    return seq_len


def spec_kv_commit_quant(cache: torch.Tensor, scale: torch.Tensor, staged: torch.Tensor, accept_len: torch.Tensor,
                         seq_len: torch.Tensor, *, nodes: torch.Tensor | None = None, lead: int = 0,
                         device_status=None, stream=None):
    """Commit the accepted drafts' KV entries to an 8-bit cache: cache
    [NL][B][L][2][Hkv][D] float8_e4m3fn with scale [NL][B][L][2][Hkv] uint8
    (element = code * 2^(byte - 127)), staged [NL][B][K][2][Hkv][D] float32 or
    bfloat16, accept_len [B] int32 (as the verification returns it), seq_len [B]
    int32 updated in place.  nodes [B][K] int32: the staged entries of an
    accepted tree path (spec_verify_tree_greedy's out_nodes).  lead = 1: staged
    entry 0, that of the last emitted token, is committed ahead of them."""
    if not isinstance(cache, torch.Tensor) or cache.dim() != 6:
        raise TypeError("cache must be a CUDA tensor [NL][B][L][2][Hkv][D]")
    if not isinstance(staged, torch.Tensor) or staged.dim() != 6:
        raise TypeError("staged must be a CUDA tensor [NL][B][K][2][Hkv][D]")
    NL, B, L, _, H, D = cache.shape
    K = staged.shape[2]
    _check(cache, (NL, B, L, 2, H, D), (torch.float8_e4m3fn,), "cache")
    _check(scale, (NL, B, L, 2, H), (torch.uint8,), "scale")
    _check(staged, (NL, B, K, 2, H, D), (torch.float32, torch.bfloat16), "staged")
    _check(accept_len, (B,), (torch.int32,), "accept_len")
    _check(seq_len, (B,), (torch.int32,), "seq_len")
    if nodes is not None:
        _check(nodes, (B, K), (torch.int32,), "nodes")
    if device_status is not None:
        _check(device_status, (1,), (torch.int32,), "device_status")
    rc = load().spec_kv_commit_quant(cache.data_ptr(), scale.data_ptr(), staged.data_ptr(), _dt(staged),
                                     nodes.data_ptr() if nodes is not None else None, int(lead), NL, B, K, L, H, D,
                                     accept_len.data_ptr(), seq_len.data_ptr(),
                                     device_status.data_ptr() if device_status is not None else None,
                                     _stream(cache.device, stream))
    if rc:
        raise SpecVerifyError(rc, "spec_kv_commit_quant")
    return seq_len


def spec_kv_read_quant(cache: torch.Tensor, scale: torch.Tensor, start: torch.Tensor | None, seq_len: torch.Tensor,
                       count: int, *, dtype=torch.bfloat16, out=None, device_status=None,
                       stream=None) -> torch.Tensor:
    """Entries start[b] .. start[b] + count - 1 (start None: from 0) of an 8-bit
    cache [NL][B][L][2][Hkv][D] in bfloat16 (exact for scale bytes 3 to 246) or
    float32 (exact to 246), zero at and past seq_len[b].  Returns [NL][B][count][2][Hkv][D]."""
    if not isinstance(cache, torch.Tensor) or cache.dim() != 6:
        raise TypeError("cache must be a CUDA tensor [NL][B][L][2][Hkv][D]")
    NL, B, L, _, H, D = cache.shape
    count = int(count)
    _check(cache, (NL, B, L, 2, H, D), (torch.float8_e4m3fn,), "cache")
    _check(scale, (NL, B, L, 2, H), (torch.uint8,), "scale")
    if start is not None:
        _check(start, (B,), (torch.int32,), "start")
    _check(seq_len, (B,), (torch.int32,), "seq_len")
    if out is None:
        if count < 1:
            raise ValueError("count must be at least 1")
        with _on(cache.device, stream) as before:
            out = _new((NL, B, count, 2, H, D), dtype, cache.device, before)
    _check(out, (NL, B, count, 2, H, D), (torch.float32, torch.bfloat16), "out")
    if device_status is not None:
        _check(device_status, (1,), (torch.int32,), "device_status")
    rc = load().spec_kv_read_quant(cache.data_ptr(), scale.data_ptr(), start.data_ptr() if start is not None else None,
                                   seq_len.data_ptr(), NL, B, L, count, H, D, out.data_ptr(), _dt(out),
                                   device_status.data_ptr() if device_status is not None else None,
                                   _stream(cache.device, stream))
    if rc:
        raise SpecVerifyError(rc, "spec_kv_read_quant")
    return out


def spec_attention_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, D: int, P: int, L: int) -> int:
    return int(load().spec_attention_workspace_bytes(int(B), int(T), int(Hq), int(Hkv), int(D), int(P), int(L)))


_attention_bytes = functools.lru_cache(maxsize=256)(spec_attention_workspace_bytes)


def _scratch(nbytes, device, st):
    """This thread's scratch for (device, st), the current stream: it needs no
    zero-fill and is handed to one of the thread's calls after another on that
    stream.  It comes from the allocator's pool of the stream, so a smaller one that
    is dropped is handed out again only to later work of it.  A call under capture
    gets scratch of its own from the graph's pool: the graph keeps the address."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, st)
    buf = _kept.scratch.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = _kept.scratch[key] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
    return buf


def spec_verify_attention(q: torch.Tensor, cache: torch.Tensor, seq_len: torch.Tensor, *,
                          staged: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                          prefix: torch.Tensor | None = None, cache_scale: torch.Tensor | None = None,
                          prefix_scale: torch.Tensor | None = None, sm_scale: float | None = None, out=None,
                          lse=None, workspace=None, device_status=None, stream=None):
    """Attention of the verification pass: q [B][T][Hq][D] bfloat16 attends to a
    prefix [P][2][Hkv][D] that the batch shares, to the sequence's own cache
    entries [0, seq_len[b]) (cache [B][L][2][Hkv][D], one layer) and to the
    pass's own entries staged [B][T][2][Hkv][D], under mask [B][T][T] uint8
    (spec_tree_mask) or causally.  Prefix and cache are bfloat16, or both
    float8_e4m3fn with cache_scale [B][L][2][Hkv] and prefix_scale [P][2][Hkv]
    uint8.  sm_scale defaults to 1 / sqrt(D).  Returns (out [B][T][Hq][D]
    bfloat16, lse [B][T][Hq] float32); a row that sees nothing has 0 and -inf.
    There is no backward pass: the outputs carry no gradient.  Without workspace
    (uint8, spec_attention_workspace_bytes(...) elements, one per call in flight) the
    call takes scratch that its thread keeps for the stream, as large as the largest
    call so far, until the thread ends."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise TypeError("q must be a CUDA tensor [B][T][Hq][D]")
    if not isinstance(cache, torch.Tensor) or cache.dim() != 5:
        raise TypeError("cache must be a CUDA tensor [B][L][2][Hkv][D]")
    B, T, Hq, D = q.shape
    L, H = cache.shape[1], cache.shape[3]
    dev = q.device
    quant = cache.dtype == torch.float8_e4m3fn
    kind = (cache.dtype,) if quant else (torch.bfloat16,)
    _check(q, (B, T, Hq, D), (torch.bfloat16,), "q")
    _check(cache, (B, L, 2, H, D), kind, "cache")
    _check(seq_len, (B,), (torch.int32,), "seq_len")
    if quant != (cache_scale is not None):
        raise ValueError("cache_scale goes with a float8_e4m3fn cache")
    if quant:
        _check(cache_scale, (B, L, 2, H), (torch.uint8,), "cache_scale")
    P = 0
    if prefix is not None:
        P = prefix.shape[0]
        _check(prefix, (P, 2, H, D), kind, "prefix")
    if (quant and prefix is not None) != (prefix_scale is not None):
        raise ValueError("prefix_scale goes with a float8_e4m3fn prefix")
    if prefix_scale is not None:
        _check(prefix_scale, (P, 2, H), (torch.uint8,), "prefix_scale")
    if staged is not None:
        _check(staged, (B, T, 2, H, D), (torch.bfloat16,), "staged")
    if mask is not None:
        _check(mask, (B, T, T), (torch.uint8,), "mask")
    if out is not None:
        _check(out, (B, T, Hq, D), (torch.bfloat16,), "out")
    if lse is not None:
        _check(lse, (B, T, Hq), (torch.float32,), "lse")
    if device_status is not None:
        _check(device_status, (1,), (torch.int32,), "device_status")
    if workspace is not None and (not isinstance(workspace, torch.Tensor) or not workspace.is_cuda):
        raise TypeError("workspace must be a CUDA tensor")
    nbytes = 0 if workspace is not None else _attention_bytes(B, T, Hq, H, D, P, L)
    if workspace is None and nbytes == 0:
        raise SpecVerifyError(1, "spec_verify_attention")
    st = _stream(dev, stream)
    lib = load()
    with _on(dev, stream) as before:
        if out is None:
            out = _new((B, T, Hq, D), torch.bfloat16, dev, before)
        if lse is None:
            lse = _new((B, T, Hq), torch.float32, dev, before)
        if workspace is None:
            workspace = _scratch(nbytes, dev, st)

    def ptr(t):
        return t.data_ptr() if t is not None else None
    rc = lib.spec_verify_attention(q.data_ptr(), ptr(prefix), ptr(prefix_scale), cache.data_ptr(), ptr(cache_scale),
                                   int(quant), seq_len.data_ptr(), ptr(staged), ptr(mask), B, T, Hq, H, D, P, L,
                                   float(sm_scale) if sm_scale is not None else D ** -0.5, out.data_ptr(),
                                   lse.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), ptr(device_status), st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify_attention")
    return out, lse


def spec_verify_window_attention(q: torch.Tensor, cache: torch.Tensor, seq_len: torch.Tensor, window: int, *,
                                 sinks: int = 0, staged: torch.Tensor | None = None,
                                 mask: torch.Tensor | None = None, cache_scale: torch.Tensor | None = None,
                                 sm_scale: float | None = None, out=None, lse=None, workspace=None,
                                 device_status=None, stream=None):
    """spec_verify_attention for a layer with a sliding window and sinks: q
    [B][T][Hq][D] bfloat16, cache [B][L][2][Hkv][D] bfloat16, or float8_e4m3fn with
    cache_scale [B][L][2][Hkv] uint8, staged [B][T][2][Hkv][D] bfloat16 under mask
    [B][T][T] uint8 or causally.  Of its sequence's entries [0, seq_len[b]) and the
    pass's that it is shown, in this order, a token sees the first ``sinks`` and the
    last ``window``, itself included.  Returns (out [B][T][Hq][D] bfloat16, lse
    [B][T][Hq] float32); a row that sees nothing has 0 and -inf.  No backward pass;
    workspace and scratch as in spec_verify_attention (P = 0)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise TypeError("q must be a CUDA tensor [B][T][Hq][D]")
    if not isinstance(cache, torch.Tensor) or cache.dim() != 5:
        raise TypeError("cache must be a CUDA tensor [B][L][2][Hkv][D]")
    B, T, Hq, D = shape = q.shape
    _, L, _, H, _ = cache.shape
    index = _index(q, "q")
    quant = cache.dtype is torch.float8_e4m3fn
    _need(q, shape, torch.bfloat16, index, "q")
    _need(cache, (B, L, 2, H, D), cache.dtype if quant else torch.bfloat16, index, "cache")
    _need(seq_len, (B,), torch.int32, index, "seq_len")
    if quant != (cache_scale is not None):
        raise ValueError("cache_scale goes with a float8_e4m3fn cache")
    if quant:
        _need(cache_scale, (B, L, 2, H), torch.uint8, index, "cache_scale")
    if staged is not None:
        _need(staged, (B, T, 2, H, D), torch.bfloat16, index, "staged")
    if mask is not None:
        _need(mask, (B, T, T), torch.uint8, index, "mask")
    if device_status is not None:
        _need(device_status, (1,), torch.int32, index, "device_status")
    window, sinks = int(window), int(sinks)
    if window < 1 or sinks < 0:
        raise ValueError("window must be at least 1 and sinks at least 0")
    dev = q.device
    st = _stream(dev, stream)
    with _on(dev, stream) as before:
        if out is None:
            out = _new(shape, torch.bfloat16, dev, before)
        if lse is None:
            lse = _new((B, T, Hq), torch.float32, dev, before)
        if workspace is None:
            nbytes = _attention_bytes(B, T, Hq, H, D, 0, L)
            if nbytes == 0:
                raise SpecVerifyError(1, "spec_verify_window_attention")
            workspace = _scratch(nbytes, dev, st)
        else:
            _own_workspace(workspace, index)
    _need(out, shape, torch.bfloat16, index, "out")
    _need(lse, (B, T, Hq), torch.float32, index, "lse")

    def ptr(t):
        return t.data_ptr() if t is not None else None
    # past 2^31 a window or sinks are everything
    rc = (_lib or load()).spec_verify_window_attention(
        q.data_ptr(), cache.data_ptr(), ptr(cache_scale), int(quant), seq_len.data_ptr(), ptr(staged), ptr(mask),
        min(window, 2**31 - 1), min(sinks, 2**31 - 1), B, T, Hq, H, D, L,
        D ** -0.5 if sm_scale is None else float(sm_scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, ptr(device_status), st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify_window_attention")
    return out, lse


def spec_verify_tree_greedy(target: torch.Tensor, tree_tokens: torch.Tensor, parent: torch.Tensor, *,
                            workspace=None, device_status=None, stream=None):
    """Greedy verification of a draft tree: target [B][N][V] logits (row n: the
    prediction after node n), tree_tokens and parent [B][N] int32 (parent[0]
    == -1, parent[n] < n).  Returns (out_tokens [B][N], out_nodes [B][N],
    out_accept_len [B])."""
    B, N, V = target.shape
    _check(target, (B, N, V), (torch.float32, torch.bfloat16), "target")
    _check(tree_tokens, (B, N), (torch.int32,), "tree_tokens")
    _check(parent, (B, N), (torch.int32,), "parent")
    dev = target.device
    nbytes = int(load().spec_tree_workspace_bytes(B, N, V))
    if nbytes == 0:
        raise SpecVerifyError(1, "spec_verify_tree_greedy")
    with _on(dev, stream) as before:
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        out_t = _new((B, N), torch.int32, dev, before)
        out_n = _new((B, N), torch.int32, dev, before)
        out_l = _new((B,), torch.int32, dev, before)
    if device_status is not None:
        _check(device_status, (1,), (torch.int32,), "device_status")
    st = _stream(dev, stream)
    rc = load().spec_verify_tree_greedy(target.data_ptr(), _dt(target), tree_tokens.data_ptr(), parent.data_ptr(),
                                        B, N, V, out_t.data_ptr(), out_n.data_ptr(), out_l.data_ptr(),
                                        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                        device_status.data_ptr() if device_status is not None else None, st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify_tree_greedy")
    return out_t, out_n, out_l


def spec_tree_mask(parent: torch.Tensor, *, out=None, device_status=None, stream=None) -> torch.Tensor:
    """Tree attention mask: uint8 [B][N][N], 1 where node j is node i or an ancestor of it."""
    B, N = parent.shape
    _check(parent, (B, N), (torch.int32,), "parent")
    if out is None:
        with _on(parent.device, stream) as before:
            out = _new((B, N, N), torch.uint8, parent.device, before)
    _check(out, (B, N, N), (torch.uint8,), "out")
    if device_status is not None:
        _check(device_status, (1,), (torch.int32,), "device_status")
    rc = load().spec_tree_mask(parent.data_ptr(), B, N, out.data_ptr(),
                               device_status.data_ptr() if device_status is not None else None,
                               _stream(parent.device, stream))
    if rc:
        raise SpecVerifyError(rc, "spec_tree_mask")
    return out


def spec_verify_shortlist_pos(target: torch.Tensor, draft_sl: torch.Tensor, shortlist_idx: torch.Tensor,
                              draft_tokens: torch.Tensor, T: float, seed: int, *, shortlist_len=None,
                              out_tokens=None, out_accept_len=None, workspace=None, aux: Aux | None = None,
                              stream=None):
    """Verification with per-position shortlists: shortlist_idx [B][K][S] (one
    list per position), [B][S] (one per sequence) or [S] (one shared list), int32
    strictly ascending; draft_sl [B][K][S] logits of the target's dtype, row
    (b, i) holding shortlist_len[i] entries (a host sequence of K ints; default S)."""
    B, K1, V = target.shape
    K = K1 - 1
    S = shortlist_idx.shape[-1]
    _check(target, (B, K + 1, V), (torch.float32, torch.bfloat16), "target")
    _check(draft_sl, (B, K, S), (target.dtype,), "draft_sl")
    _check(draft_tokens, (B, K), (torch.int32,), "draft_tokens")
    if shortlist_idx.dim() == 3:
        _check(shortlist_idx, (B, K, S), (torch.int32,), "shortlist_idx")
        seq, pos = K * S, S
    elif shortlist_idx.dim() == 2:
        _check(shortlist_idx, (B, S), (torch.int32,), "shortlist_idx")
        seq, pos = S, 0
    else:
        _check(shortlist_idx, (S,), (torch.int32,), "shortlist_idx")
        seq, pos = 0, 0
    lens = None
    if shortlist_len is not None:
        lens = (ctypes.c_int32 * K)(*[int(x) for x in shortlist_len])
    dev = target.device
    st = _stream(dev, stream)
    with _on(dev, stream) as before:
        out_tokens, out_accept_len = _outs(B, K, dev, out_tokens, out_accept_len, before)
        workspace, wsb = _ws_args(dev, st, spec_workspace_bytes(B, K, V, S), workspace, (B, K, V, S))
    ax = aux._struct(B, K) if aux is not None else None
    rc = load().spec_verify_shortlist_pos(target.data_ptr(), _dt(target), draft_sl.data_ptr(), _dt(draft_sl),
                                          shortlist_idx.data_ptr(), seq, pos, lens, S, draft_tokens.data_ptr(),
                                          B, K, V, float(T), int(seed) & (2**64 - 1), out_tokens.data_ptr(),
                                          out_accept_len.data_ptr(), workspace.data_ptr(), wsb,
                                          ctypes.byref(ax) if ax is not None else None, st)
    if rc:
        raise SpecVerifyError(rc, "spec_verify_shortlist_pos")
    return out_tokens, out_accept_len
