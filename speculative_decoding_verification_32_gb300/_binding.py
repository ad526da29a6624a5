"""ctypes binding of libspecverify.so: argument marshalling only.

Takes torch CUDA tensors, passes their device pointers, the current CUDA
stream and a cached workspace to the C ABI declared in
include/specverify.h, and returns the output tensors.  Every step of the
computation runs in the library's kernels; there is no other code path.
"""
import ctypes
import functools
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SPEC_F32, SPEC_BF16, SPEC_F16, SPEC_E4M3 = 0, 1, 2, 3
SPEC_STOCHASTIC, SPEC_GREEDY = 0, 1
SPEC_ERR_WORKSPACE = 7
ROW_STATUS = {0: "OK", 1: "NONFINITE", 2: "BAD_TOKEN", 3: "BAD_UNIFORM", 4: "BAD_PARENT",
              5: "EMPTY", 6: "TIMEOUT", 7: "BAD_TEMPERATURE", 8: "BAD_SLOT"}

_c = ctypes
_P = _c.c_void_p


class SpecChainArgs(_c.Structure):
    _fields_ = [("B", _c.c_int32), ("K", _c.c_int32), ("V", _c.c_int32), ("dtype", _c.c_int32),
                ("mode", _c.c_int32), ("margin_kappa", _c.c_float),
                ("target_logits", _P), ("draft_logits", _P), ("draft_tokens", _P),
                ("temperature", _P), ("u_accept", _P), ("u_sample", _P)]


class SpecChainOut(_c.Structure):
    _fields_ = [("accepted_len", _P), ("out_tokens", _P), ("num_emitted", _P),
                ("row_status", _P), ("p_at_draft", _P), ("q_at_draft", _P), ("resid_mass", _P)]


class SpecTreeArgs(_c.Structure):
    _fields_ = [("B", _c.c_int32), ("N", _c.c_int32), ("V", _c.c_int32), ("dtype", _c.c_int32),
                ("margin_kappa", _c.c_float), ("target_logits", _P), ("parent", _P),
                ("node_tokens", _P), ("temperature", _P)]


class SpecTreeOut(_c.Structure):
    _fields_ = [("accepted_len", _P), ("path_nodes", _P), ("out_tokens", _P),
                ("num_emitted", _P), ("row_status", _P)]


class SpecTruncation(_c.Structure):
    _fields_ = [("top_k", _P), ("top_p", _P)]


class SpecKvCompactArgs(_c.Structure):
    _fields_ = [("B", _c.c_int32), ("N", _c.c_int32), ("planes", _c.c_int32), ("pad", _c.c_int32),
                ("S_max", _c.c_int64), ("entry_bytes", _c.c_int64), ("plane_stride", _c.c_int64),
                ("row_stride", _c.c_int64), ("tok_stride", _c.c_int64), ("kv", _P),
                ("kv_len_in", _P), ("accepted_len", _P), ("path_nodes", _P)]


class SpecAdaptiveParams(_c.Structure):
    _fields_ = [("alpha", _c.c_double), ("divisor", _c.c_double), ("ema0", _c.c_double),
                ("shallow", _c.c_int32 * 3), ("deep", _c.c_int32 * 3), ("start", _c.c_int32 * 3),
                ("breaker", _c.c_int32)]


class SpecKvCache(_c.Structure):
    _fields_ = [("rows", _c.c_int32), ("heads", _c.c_int32), ("head_dim", _c.c_int32),
                ("dtype", _c.c_int32), ("slots", _c.c_int64), ("row_stride", _c.c_int64),
                ("tok_stride", _c.c_int64), ("k", _P), ("v", _P)]


class SpecKvAppendArgs(_c.Structure):
    _fields_ = [("cache", SpecKvCache), ("N", _c.c_int32), ("src_dtype", _c.c_int32), ("k", _P),
                ("v", _P), ("k_stride", _c.c_int64 * 3), ("v_stride", _c.c_int64 * 3),
                ("kv_len", _P), ("count", _P)]


class SpecKvReadArgs(_c.Structure):
    _fields_ = [("cache", SpecKvCache), ("T", _c.c_int32), ("out_dtype", _c.c_int32),
                ("k_out", _P), ("v_out", _P), ("start", _P), ("length", _P)]


class SpecAttentionArgs(_c.Structure):
    _fields_ = [("cache", SpecKvCache), ("prefix", SpecKvCache), ("prefix_len", _c.c_int64),
                ("N", _c.c_int32), ("q_heads", _c.c_int32), ("q_dtype", _c.c_int32),
                ("scale", _c.c_float), ("q", _P), ("q_stride", _c.c_int64 * 3),
                ("kv_len", _P), ("count", _P), ("parent", _P)]


class SpecLogprobsArgs(_c.Structure):
    _fields_ = [("B", _c.c_int32), ("npos", _c.c_int32), ("V", _c.c_int32), ("dtype", _c.c_int32),
                ("m", _c.c_int32), ("pad", _c.c_int32), ("row_stride", _c.c_int64),
                ("logits", _P), ("tokens", _P), ("temperature", _P)]


class SpecLogprobsOut(_c.Structure):
    _fields_ = [("logprob", _P), ("entropy", _P), ("top_ids", _P), ("top_logprobs", _P),
                ("status", _P)]


class SpecError(RuntimeError):
    """A spec_* entry point returned a non-zero spec_status."""

    def __init__(self, code, msg):
        super().__init__(msg)
        self.code = code


_lib = None
_lib_lock = threading.Lock()


def lib(path=None):
    """The loaded C library (raises if it was never built)."""
    global _lib
    if path is not None:
        return _bind(_c.CDLL(path))
    with _lib_lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            _lib = _bind(_c.CDLL(LIB_PATH))
    return _lib


def _bind(L):
    i32, u64, sz = _c.c_int32, _c.c_uint64, _c.c_size_t
    L.spec_verify_chain_workspace_size.argtypes = [i32, i32, i32]
    L.spec_verify_chain_workspace_size.restype = sz
    L.spec_verify_chain_truncated_workspace_size.argtypes = [i32, i32, i32]
    L.spec_verify_chain_truncated_workspace_size.restype = sz
    L.spec_verify_tree_workspace_size.argtypes = [i32, i32, i32]
    L.spec_verify_tree_workspace_size.restype = sz
    L.spec_verify_chain.argtypes = [_c.POINTER(SpecChainArgs), _c.POINTER(SpecChainOut), _P, sz, _P]
    L.spec_verify_chain.restype = _c.c_int
    L.spec_verify_chain_static.argtypes = [_c.POINTER(SpecChainArgs), _c.POINTER(SpecChainOut), _P]
    L.spec_verify_chain_static.restype = _c.c_int
    L.spec_verify_tree.argtypes = [_c.POINTER(SpecTreeArgs), _c.POINTER(SpecTreeOut), _P, sz, _P]
    L.spec_verify_tree.restype = _c.c_int
    L.spec_verify_chain_truncated.argtypes = [_c.POINTER(SpecChainArgs), _c.POINTER(SpecTruncation),
                                              _c.POINTER(SpecChainOut), _P, sz, _P]
    L.spec_verify_chain_truncated.restype = _c.c_int
    L.spec_drift_residuals.argtypes = [_c.POINTER(SpecChainArgs), i32, _P, _P, _P, _P, sz, _P]
    L.spec_drift_residuals.restype = _c.c_int
    L.spec_kv_compact_tree.argtypes = [_c.POINTER(SpecKvCompactArgs), _P, _P]
    L.spec_kv_compact_tree.restype = _c.c_int
    L.spec_adaptive_tree_policy.argtypes = [_c.POINTER(SpecAdaptiveParams), i32, _P, _P, _P, _P,
                                            _P, _P, _P]
    L.spec_adaptive_tree_policy.restype = _c.c_int
    L.spec_rollback_lengths.argtypes = [i32, i32, _P, _P, _P, _P, i32, _P, _P, _P, _P]
    L.spec_rollback_lengths.restype = _c.c_int
    L.spec_kv_entry_bytes.argtypes = [i32, i32, i32]
    L.spec_kv_entry_bytes.restype = sz
    L.spec_kv_append.argtypes = [_c.POINTER(SpecKvAppendArgs), _P, _P]
    L.spec_kv_append.restype = _c.c_int
    L.spec_kv_read.argtypes = [_c.POINTER(SpecKvReadArgs), _P, _P]
    L.spec_kv_read.restype = _c.c_int
    L.spec_prefix_attention_workspace_size.argtypes = [_c.POINTER(SpecAttentionArgs)]
    L.spec_prefix_attention_workspace_size.restype = sz
    L.spec_prefix_attention.argtypes = [_c.POINTER(SpecAttentionArgs), _P, _P, _P, _P, sz, _P]
    L.spec_prefix_attention.restype = _c.c_int
    L.spec_token_logprobs.argtypes = [_c.POINTER(SpecLogprobsArgs), _c.POINTER(SpecLogprobsOut), _P]
    L.spec_token_logprobs.restype = _c.c_int
    L.spec_workspace_init.argtypes = [_P, sz, _P]
    L.spec_workspace_init.restype = _c.c_int
    L.spec_status_string.argtypes = [_c.c_int]
    L.spec_status_string.restype = _c.c_char_p
    L.spec_set_wait_timeout_ns.argtypes = [u64]
    L.spec_set_wait_timeout_ns.restype = None
    L.spec_get_wait_timeout_ns.argtypes = []
    L.spec_get_wait_timeout_ns.restype = u64
    L.spec_debug_force_wait_timeout.argtypes = [_c.c_int]
    L.spec_debug_force_wait_timeout.restype = None
    return L


def _check(code):
    if code != 0:
        raise SpecError(code, lib().spec_status_string(code).decode())


def _ptr(t):
    return None if t is None else _P(t.data_ptr())


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _req(t, name, device, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# Workspaces: one buffer per (device, stream), grown on demand.  The library
# needs no particular contents; it keeps a small header at the buffer's end
# between calls, so the same buffer is always passed with its full size.
_ws = {}
_ws_lock = threading.Lock()


def workspace(device, nbytes, handle, stream=None):
    """The workspace of the stream with this handle.  `stream`: that stream, if it
    may not be the current one: a new buffer is filled, and a replaced one is
    given back, in its order."""
    key = (device, handle)
    with _ws_lock:
        buf = _ws.get(key)
        if buf is None or buf.numel() < nbytes:
            with _here if stream is None else torch.cuda.stream(stream):
                buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
            _ws[key] = buf
    return buf


# A call enqueues several kernels that hand data to one another through the
# stream's workspace, and other host threads run meanwhile: a call's kernels are
# enqueued as a whole before another call's on the same stream.  (Reentrant: an
# allocation may run a finaliser that makes a call of its own.)
_enqueue_locks = {}


def _enqueuing(key):
    """The lock of the workspace with this key."""
    return _enqueue_locks.setdefault(key, threading.RLock())


class _Here:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_here = _Here()
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(device, stream=None):
    """The context of a call's launches: its tensors' device is the current one."""
    if device.type != "cuda":
        raise ValueError(f"the library's calls need CUDA tensors, got tensors on {device}")
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return _here if _current_device() == device.index else torch.cuda.device(device)


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s, _P(s.cuda_stream)


def spec_verify_chain(target_logits, draft_logits, draft_tokens, temperature=None,
                      u_accept=None, u_sample=None, mode="stochastic", margin_kappa=0.0,
                      diagnostics=False, out=None, stream=None, top_k=None, top_p=None):
    """Verify B draft chains (see spec_verify_chain in include/specverify.h).

    target_logits [B,K+1,V] and draft_logits [B,K,V] (bf16 or fp32, CUDA),
    draft_tokens [B,K] int32, temperature [B] fp32 or None, u_accept [B,K] and
    u_sample [B,K+1] fp32 (stochastic mode).  mode: "stochastic" | "greedy".
    Returns a dict of CUDA tensors: accepted_len, out_tokens, num_emitted,
    row_status (+ p_at_draft, q_at_draft, resid_mass with diagnostics=True).
    top_k [B] int32 / top_p [B] float32 (stochastic mode, optional) truncate
    p and q (spec_verify_chain_truncated).
    """
    dev = target_logits.device
    greedy = mode == "greedy"
    _req(target_logits, "target_logits", dev)
    B, K1, V = target_logits.shape
    K = K1 - 1
    dt = _dtype_code(target_logits)
    if not greedy or draft_logits is not None:
        _req(draft_logits, "draft_logits", dev, target_logits.dtype)
    _req(draft_tokens, "draft_tokens", dev, torch.int32)
    _req(temperature, "temperature", dev, torch.float32)
    _req(u_accept, "u_accept", dev, torch.float32)
    _req(u_sample, "u_sample", dev, torch.float32)
    if out is None:
        out = dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty(B, K + 1, dtype=torch.int32, device=dev),
                   num_emitted=torch.empty(B, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
        if diagnostics and not greedy:
            for k in ("p_at_draft", "q_at_draft", "resid_mass"):
                out[k] = torch.empty(B, K, dtype=torch.float32, device=dev)
    args = SpecChainArgs(B, K, V, dt, SPEC_GREEDY if greedy else SPEC_STOCHASTIC,
                         float(margin_kappa), _ptr(target_logits),
                         None if greedy else _ptr(draft_logits), _ptr(draft_tokens),
                         _ptr(temperature), None if greedy else _ptr(u_accept),
                         None if greedy else _ptr(u_sample))
    o = SpecChainOut(_ptr(out["accepted_len"]), _ptr(out["out_tokens"]),
                     _ptr(out["num_emitted"]), _ptr(out["row_status"]),
                     _ptr(out.get("p_at_draft")), _ptr(out.get("q_at_draft")),
                     _ptr(out.get("resid_mass")))
    L = lib()
    truncated = top_k is not None or top_p is not None
    nbytes = (L.spec_verify_chain_truncated_workspace_size if truncated
              else L.spec_verify_chain_workspace_size)(B, K, V)
    on = _device(dev, stream)
    s, sp = _stream(dev, stream)
    with on, _enqueuing((dev, s.cuda_stream)):
        ws = workspace(dev, nbytes, s.cuda_stream, stream)
        if not truncated:
            _check(L.spec_verify_chain(_c.byref(args), _c.byref(o), _ptr(ws), ws.numel(), sp))
        else:
            if greedy:
                raise ValueError("top_k / top_p apply to mode='stochastic' only")
            _req(top_k, "top_k", dev, torch.int32)
            _req(top_p, "top_p", dev, torch.float32)
            t = SpecTruncation(_ptr(top_k), _ptr(top_p))
            _check(L.spec_verify_chain_truncated(_c.byref(args), _c.byref(t), _c.byref(o), _ptr(ws),
                                                 ws.numel(), sp))
    return out


def spec_verify_tree(target_logits, parent, node_tokens, temperature=None, margin_kappa=0.0,
                     out=None, stream=None):
    """Verify one draft tree per row (see spec_verify_tree in include/specverify.h).

    target_logits [B,N,V] (bf16 or fp32), parent [B,N] int32, node_tokens
    [B,N] int32.  Returns accepted_len, path_nodes, out_tokens, num_emitted,
    row_status.
    """
    dev = target_logits.device
    _req(target_logits, "target_logits", dev)
    B, N, V = target_logits.shape
    dt = _dtype_code(target_logits)
    _req(parent, "parent", dev, torch.int32)
    _req(node_tokens, "node_tokens", dev, torch.int32)
    _req(temperature, "temperature", dev, torch.float32)
    if out is None:
        out = dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
                   path_nodes=torch.empty(B, N, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty(B, N, dtype=torch.int32, device=dev),
                   num_emitted=torch.empty(B, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
    args = SpecTreeArgs(B, N, V, dt, float(margin_kappa), _ptr(target_logits), _ptr(parent),
                        _ptr(node_tokens), _ptr(temperature))
    o = SpecTreeOut(_ptr(out["accepted_len"]), _ptr(out["path_nodes"]), _ptr(out["out_tokens"]),
                    _ptr(out["num_emitted"]), _ptr(out["row_status"]))
    L = lib()
    nbytes = L.spec_verify_tree_workspace_size(B, N, V)
    on = _device(dev, stream)
    s, sp = _stream(dev, stream)
    with on, _enqueuing((dev, s.cuda_stream)):
        ws = workspace(dev, nbytes, s.cuda_stream, stream)
        _check(L.spec_verify_tree(_c.byref(args), _c.byref(o), _ptr(ws), ws.numel(), sp))
    return out


def spec_rollback_lengths(kv_len_in, accepted_len, num_emitted, out_tokens, eos_id=-1,
                          max_len=None, stream=None):
    """Committed KV lengths (see spec_rollback_lengths in include/specverify.h).

    Returns (committed_kv_len [B], num_emitted_out [B]) int32 CUDA tensors.
    """
    dev = out_tokens.device
    for t, n in ((kv_len_in, "kv_len_in"), (accepted_len, "accepted_len"),
                 (num_emitted, "num_emitted"), (out_tokens, "out_tokens"), (max_len, "max_len")):
        _req(t, n, dev, torch.int32)
    B, max_emit = out_tokens.shape
    committed = torch.empty(B, dtype=torch.int32, device=dev)
    n_out = torch.empty(B, dtype=torch.int32, device=dev)
    on = _device(dev, stream)
    _, sp = _stream(dev, stream)
    with on:
        _check(lib().spec_rollback_lengths(B, max_emit, _ptr(kv_len_in), _ptr(accepted_len),
                                           _ptr(num_emitted), _ptr(out_tokens), int(eos_id),
                                           _ptr(max_len), _ptr(committed), _ptr(n_out), sp))
    return committed, n_out


def spec_drift_residuals(target_logits, draft_logits, temperature=None, m=32, stream=None):
    """Top-m target support and log p - log q on it at every drafted position
    (see spec_drift_residuals in include/specverify.h).  Returns (support
    [B,K,m] int32, residual [B,K,m] float32, row_status [B] int32)."""
    dev = target_logits.device
    _req(target_logits, "target_logits", dev)
    _req(draft_logits, "draft_logits", dev, target_logits.dtype)
    _req(temperature, "temperature", dev, torch.float32)
    B, K1, V = target_logits.shape
    K = K1 - 1
    sup = torch.empty(B, K, m, dtype=torch.int32, device=dev)
    res = torch.empty(B, K, m, dtype=torch.float32, device=dev)
    st = torch.empty(B, dtype=torch.int32, device=dev)
    args = SpecChainArgs(B, K, V, _dtype_code(target_logits), SPEC_STOCHASTIC, 0.0,
                         _ptr(target_logits), _ptr(draft_logits), None, _ptr(temperature),
                         None, None)
    L = lib()
    nbytes = L.spec_verify_chain_truncated_workspace_size(B, K, V)
    on = _device(dev, stream)
    s, sp = _stream(dev, stream)
    with on, _enqueuing((dev, s.cuda_stream)):
        ws = workspace(dev, nbytes, s.cuda_stream, stream)
        _check(L.spec_drift_residuals(_c.byref(args), int(m), _ptr(sup), _ptr(res), _ptr(st),
                                      _ptr(ws), ws.numel(), sp))
    return sup, res, st


def spec_kv_compact_tree(kv, kv_len_in, accepted_len, path_nodes, stream=None):
    """Compact each row's accepted tree path in place (see spec_kv_compact_tree
    in include/specverify.h).

    kv: a CUDA tensor [planes, B, S_max, ...] whose trailing dimensions form
    one token's entry (contiguous, any dtype); path_nodes [B, N] int32.
    Returns row_status [B] int32.
    """
    dev = kv.device
    if not kv.is_contiguous() or kv.dim() < 3:
        raise ValueError("kv must be a contiguous [planes, B, S_max, ...] tensor")
    for t, n in ((kv_len_in, "kv_len_in"), (accepted_len, "accepted_len"),
                 (path_nodes, "path_nodes")):
        _req(t, n, dev, torch.int32)
    planes, B, S_max = kv.shape[:3]
    E = kv[0, 0, 0].numel() * kv.element_size() if kv.numel() else 0
    status = torch.empty(B, dtype=torch.int32, device=dev)
    a = SpecKvCompactArgs(B, path_nodes.shape[1], planes, 0, S_max, E, B * S_max * E, S_max * E, E,
                          _ptr(kv), _ptr(kv_len_in), _ptr(accepted_len), _ptr(path_nodes))
    on = _device(dev, stream)
    _, sp = _stream(dev, stream)
    with on:
        _check(lib().spec_kv_compact_tree(_c.byref(a), _ptr(status), sp))
    return status


def spec_adaptive_tree_policy(accepted_len, depth, draft_top1, ema, zero_run, alpha=0.3,
                              divisor=1.0, shallow=(3, 4, 4), deep=(7, 1, 8), start=(3, 4, 4),
                              ema0=0.0, breaker=5, stream=None):
    """One policy step for B sequences (see spec_adaptive_tree_policy in
    include/specverify.h).  ema (float64) and zero_run (int32) are updated in
    place; returns shape [B, 3] int32 = (nsteps, top-k, ndt)."""
    dev = accepted_len.device
    for t, n, dt in ((accepted_len, "accepted_len", torch.int32), (depth, "depth", torch.int32),
                     (draft_top1, "draft_top1", torch.float32), (ema, "ema", torch.float64),
                     (zero_run, "zero_run", torch.int32)):
        _req(t, n, dev, dt)
    B = accepted_len.shape[0]
    shape = torch.empty(B, 3, dtype=torch.int32, device=dev)
    q = SpecAdaptiveParams(float(alpha), float(divisor), float(ema0), (_c.c_int32 * 3)(*shallow),
                           (_c.c_int32 * 3)(*deep), (_c.c_int32 * 3)(*start), int(breaker))
    on = _device(dev, stream)
    _, sp = _stream(dev, stream)
    with on:
        _check(lib().spec_adaptive_tree_policy(_c.byref(q), B, _ptr(accepted_len), _ptr(depth),
                                               _ptr(draft_top1), _ptr(ema), _ptr(zero_run),
                                               _ptr(shape), sp))
    return shape


# The cache, attention and log-probability operators are called once per layer
# or step, often on a handful of tokens, so their marshalling is kept short:
# argument structures are packed in one go (same layout as the Structures
# above), sizes that depend on numbers alone are remembered, pointers go
# through as integers.
_CACHE = "4i3q2Q"
_PACK_APPEND = struct.Struct("<" + _CACHE + "2i2Q6q2Q")
_PACK_READ = struct.Struct("<" + _CACHE + "2i4Q")
_PACK_ATTENTION = struct.Struct("<" + _CACHE + _CACHE + "q3ifQ3q3Q")
_PACK_LOGPROBS = struct.Struct("<6iq3Q")
_PACK_LOGPROBS_OUT = struct.Struct("<5Q")
for _s, _t in ((_PACK_APPEND, SpecKvAppendArgs), (_PACK_READ, SpecKvReadArgs),
               (_PACK_ATTENTION, SpecAttentionArgs), (_PACK_LOGPROBS, SpecLogprobsArgs),
               (_PACK_LOGPROBS_OUT, SpecLogprobsOut)):
    assert _s.size == _c.sizeof(_t), _t

_KV_DTYPES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing
_fast = {}


def _fn(name, nargs):
    """The C entry point `name`, taking packed structures (bytes) and addresses (int)."""
    f = _fast.get(name)
    if f is None:
        f = lib()[name]
        f.argtypes = [_P] * nargs
        f.restype = _c.c_int
        _fast[name] = f
    return f


class _On:
    """A call on a stream that the caller names: tensors made inside `with`
    come from that stream's pool, and use() tells the allocator that the
    stream reads or writes tensors of another's, so none is handed out again
    too early."""

    def __init__(self, stream, *tensors):
        self.stream = stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx.__enter__()

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


def _on(device, stream, *tensors):
    """The context in which a call makes its outputs and launches: on `stream`,
    or (None) on the current stream of `device`."""
    on = _device(device, stream)
    return on if stream is None else _On(stream, *tensors)


def _enter(device, stream, *tensors):
    """That context, entered (the calls skip it where it would do nothing)."""
    on = _on(device, stream, *tensors)
    on.__enter__()
    return on


def _leave(on):
    if on is not None:
        on.__exit__(None, None, None)


def _scratch(dev, key, nbytes):
    """A workspace of these calls' own (the verify calls keep a header and
    stamped records in theirs): the stream's, or a larger one in its place.  A
    call captured into a graph gets one from the graph's pool: a replay may run
    beside later calls, and after the stream's has been replaced."""
    buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    if not _capturing():
        with _ws_lock:
            _ws[key] = buf
    return buf


def _kv_dtype(dtype, name):
    if dtype not in _KV_DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return _KV_DTYPES[dtype]


@functools.lru_cache(maxsize=None)
def spec_kv_entry_bytes(heads, head_dim, dtype=torch.uint8):
    """Bytes of one token's entry in one plane of a cache (see spec_kv_cache in
    include/specverify.h): dtype torch.uint8 (e4m3 codes and scale bytes),
    torch.bfloat16 or torch.float16."""
    code = SPEC_E4M3 if dtype == torch.uint8 else _kv_dtype(dtype, "dtype")
    n = lib().spec_kv_entry_bytes(int(heads), int(head_dim), code)
    if n == 0:
        raise ValueError(f"no cache entry of {heads} heads of {head_dim} in {dtype}")
    return n


def _kv_cache(cache, heads, head_dim, dev, name):
    """The fields of a cache tensor's C descriptor: [2, rows, slots, heads,
    head_dim] bfloat16 / float16, or [2, rows, slots, entry bytes] uint8 (e4m3)."""
    if not isinstance(cache, torch.Tensor) or cache.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")
    dtype = cache.dtype
    if dtype == torch.uint8:
        code, e, entry = SPEC_E4M3, 1, spec_kv_entry_bytes(heads, head_dim)
        want, dense = (entry,), (1,)
    elif dtype == torch.bfloat16 or dtype == torch.float16:
        code, e = _KV_DTYPES[dtype], 2
        spec_kv_entry_bytes(heads, head_dim, dtype)
        want, dense = (heads, head_dim), (head_dim, 1)
    else:
        raise TypeError(f"{name} must be bfloat16, float16 or uint8 (e4m3 entries), got {dtype}")
    shape, stride = cache.shape, cache.stride()
    if len(shape) != 3 + len(want) or shape[0] != 2 or shape[3:] != want:
        raise ValueError(f"{name} must be [2, rows, slots, {', '.join(map(str, want))}], "
                         f"got {tuple(shape)}")
    if stride[3:] != dense and any(a != b and n != 1 for a, b, n in zip(stride[3:], dense, want)):
        raise ValueError(f"{name}: one token's entry must be contiguous")
    k = cache.data_ptr()
    return (shape[1], heads, head_dim, code, shape[2], stride[1] * e, stride[2] * e, k, k + stride[0] * e)


def _i32(t, name, dev, shape):
    """The address of an int32 tensor of this shape, or 0 for None."""
    if t is None:
        return 0
    _req(t, name, dev, torch.int32)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def spec_kv_append(cache, k, v, kv_len, count=None, stream=None):
    """Write the keys and values of newly fed tokens into the KV cache (see
    spec_kv_append in include/specverify.h): token i of row b goes to slot
    kv_len[b] + i.

    cache [2, B, S, heads, D] (bfloat16 / float16) or [2, B, S, entry bytes]
    uint8 (e4m3 codes and power-of-two scales); k, v [B, N, heads, D]
    (float32, bfloat16 or float16, any strides with a dense last dimension);
    kv_len [B] int32; count [B] int32 or None (all N tokens).  Returns
    row_status [B] int32.
    """
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a [B, N, heads, head_dim] tensor")
    dev, shape, dtype = k.device, k.shape, k.dtype
    if not isinstance(v, torch.Tensor) or v.device != dev or v.shape != shape:
        raise ValueError(f"v must be a tensor like k, on {dev}")
    if v.dtype != dtype:
        raise TypeError(f"v must be {dtype}, got {v.dtype}")
    B, N, heads, D = shape
    ks, vs = k.stride(), v.stride()
    if (ks[3] != 1 or vs[3] != 1) and D > 1:
        raise ValueError("k and v: the last dimension must be dense")
    c = _kv_cache(cache, heads, D, dev, "cache")
    if c[0] != B:
        raise ValueError(f"cache has {c[0]} rows, k has {B}")
    if kv_len is None:
        raise ValueError("kv_len is needed")
    a = _PACK_APPEND.pack(*c, N, _kv_dtype(dtype, "k"), k.data_ptr(), v.data_ptr(), *ks[:3], *vs[:3],
                          _i32(kv_len, "kv_len", dev, (B,)), _i32(count, "count", dev, (B,)))
    index = dev.index
    on = None if stream is None and k.is_cuda and index == _current_device() else _enter(dev, stream, cache, k, v, kv_len, count)
    try:
        status = (torch.empty if N else torch.zeros)(B, dtype=torch.int32, device=dev)
        _check(_fn("spec_kv_append", 3)(a, status.data_ptr(), _raw_stream(index)))
    finally:
        _leave(on)
    return status


def spec_kv_read(cache, length, T, heads=None, head_dim=None, start=None, dtype=torch.bfloat16,
                 stream=None):
    """Read cache entries back as dense numbers (see spec_kv_read in
    include/specverify.h): entry t < length[b] of row b is slot start[b] + t
    (start None: 0); zeros from there to T.  heads and head_dim are needed for
    a uint8 (e4m3) cache.  Returns (k [B, T, heads, D], v, row_status [B])."""
    if not isinstance(cache, torch.Tensor) or cache.dim() < 4:
        raise ValueError("cache must be a [2, rows, slots, ...] tensor")
    dev = cache.device
    if cache.dtype != torch.uint8 and cache.dim() == 5:
        heads, head_dim = cache.shape[3:5]
    if heads is None or head_dim is None:
        raise ValueError("heads and head_dim are needed for a uint8 cache")
    c = _kv_cache(cache, heads, head_dim, dev, "cache")
    B = c[0]
    if length is None:
        raise ValueError("length is needed")
    code, n, s = _kv_dtype(dtype, "dtype"), _i32(length, "length", dev, (B,)), _i32(start, "start", dev, (B,))
    index = dev.index
    on = None if stream is None and cache.is_cuda and index == _current_device() else _enter(dev, stream, cache, length, start)
    try:
        k = torch.empty(B, T, heads, head_dim, dtype=dtype, device=dev)
        v = torch.empty_like(k)
        status = (torch.empty if T else torch.zeros)(B, dtype=torch.int32, device=dev)
        a = _PACK_READ.pack(*c, T, code, k.data_ptr(), v.data_ptr(), s, n)
        _check(_fn("spec_kv_read", 3)(a, status.data_ptr(), _raw_stream(index)))
    finally:
        _leave(on)
    return k, v, status


_NO_CACHE = (0,) * 9


def _attention_bytes(a):
    f = _fast.get("spec_prefix_attention_workspace_size")
    if f is None:
        f = lib()["spec_prefix_attention_workspace_size"]
        f.argtypes, f.restype = [_P], _c.c_size_t
        _fast["spec_prefix_attention_workspace_size"] = f
    return f(a)


def spec_prefix_attention(q, cache, kv_len, prefix=None, prefix_len=None, parent=None, count=None,
                          scale=None, kv_heads=None, stream=None):
    """The verify pass's attention over a shared prefix and each row's own cache
    (see spec_prefix_attention in include/specverify.h).

    q [B, N, q_heads, D] (bfloat16 or float16, any strides with a dense last
    dimension): the pass's tokens, already appended at slots kv_len[b] + i of
    cache [2, B, S, kv_heads, D] (q's dtype) or [2, B, S, entry bytes] uint8
    (kv_heads needed); prefix: a cache tensor whose row 0 holds the shared
    entries, the first prefix_len of them used (None: all); parent [B, N]
    int32 for draft trees (None: chains); count [B] int32 queries per row
    (None: N); scale: 1/sqrt(D) if None.  Returns (out like q, dense; lse
    [B, N, q_heads] float32; row_status [B] int32).
    """
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B, N, q_heads, head_dim] tensor")
    dev, shape, dtype = q.device, q.shape, q.dtype
    if dtype != torch.bfloat16 and dtype != torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    B, N, heads, D = shape
    qs = q.stride()
    if qs[3] != 1 and D > 1:
        raise ValueError("q: the last dimension must be dense")
    if kv_heads is None:
        if not isinstance(cache, torch.Tensor) or cache.dim() != 5:
            raise ValueError("kv_heads is needed for a uint8 cache")
        kv_heads = cache.shape[3]
    c = _kv_cache(cache, kv_heads, D, dev, "cache")
    if c[0] != B:
        raise ValueError(f"cache has {c[0]} rows, q has {B}")
    if prefix is not None:
        pc = _kv_cache(prefix, kv_heads, D, dev, "prefix")
        P = pc[4] if prefix_len is None else int(prefix_len)
    else:
        if prefix_len:
            raise ValueError("prefix_len without a prefix")
        pc, P = _NO_CACHE, 0
    if kv_len is None:
        raise ValueError("kv_len is needed")
    a = _PACK_ATTENTION.pack(*c, *pc, P, N, heads, _KV_DTYPES[dtype], D ** -0.5 if scale is None else scale,
                             q.data_ptr(), *qs[:3], _i32(kv_len, "kv_len", dev, (B,)),
                             _i32(count, "count", dev, (B,)), _i32(parent, "parent", dev, (B, N)))
    index = dev.index
    on = None if stream is None and q.is_cuda and index == _current_device() else \
        _enter(dev, stream, q, cache, kv_len, prefix, parent, count)
    try:
        out = torch.empty(shape, dtype=dtype, device=dev)
        lse = torch.empty(B, N, heads, dtype=torch.float32, device=dev)
        status = (torch.empty if N else torch.zeros)(B, dtype=torch.int32, device=dev)
        s = _raw_stream(index)
        f, code, key = _fn("spec_prefix_attention", 7), SPEC_ERR_WORKSPACE, (index, "scratch", s)
        with _enqueue_locks.get(key) or _enqueuing(key):
            ws = None if _capturing() else _ws.get(key)
            if ws is not None:  # the call itself says if that is too small, before it launches anything
                code = f(a, out.data_ptr(), lse.data_ptr(), status.data_ptr(), ws.data_ptr(), ws.numel(), s)
            if code == SPEC_ERR_WORKSPACE:
                ws = _scratch(dev, key, _attention_bytes(a))
                code = f(a, out.data_ptr(), lse.data_ptr(), status.data_ptr(), ws.data_ptr(), ws.numel(), s)
        _check(code)
    finally:
        _leave(on)
    return out, lse, status


def spec_token_logprobs(logits, tokens=None, temperature=None, m=0, stream=None):
    """Log probabilities of given tokens, entropy and the top m alternatives
    (see spec_token_logprobs in include/specverify.h).

    logits [B, npos, V] (bfloat16 or float32; positions may be spaced wider
    than V); tokens [B, npos] int32 (-1: skip the position) or None (no given
    tokens); temperature [B] float32 or None.  Returns a dict: logprob and
    entropy [B, npos] float32 (logprob only with tokens), top_ids [B, npos, m]
    int32, top_logprobs [B, npos, m] float32, status [B, npos] int32.
    """
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3:
        raise ValueError("logits must be a [B, npos, V] tensor")
    dev, st = logits.device, logits.stride()
    B, npos, V = logits.shape
    dt = _dtype_code(logits)
    pitch = st[1] if npos > 1 else st[0] if B > 1 else V
    if (V > 1 and st[2] != 1) or (B > 1 and st[0] != npos * pitch):
        raise ValueError("logits: positions must be evenly spaced with a dense last dimension")
    tk = _i32(tokens, "tokens", dev, (B, npos))
    if temperature is not None:
        _req(temperature, "temperature", dev, torch.float32)
        if temperature.shape != (B,):
            raise ValueError(f"temperature must be [{B}], got {list(temperature.shape)}")
    a = _PACK_LOGPROBS.pack(B, npos, V, dt, m, 0, pitch, logits.data_ptr(), tk,
                            0 if temperature is None else temperature.data_ptr())
    f32 = torch.float32
    index = dev.index
    on = None if stream is None and logits.is_cuda and index == _current_device() else _enter(dev, stream, logits, tokens, temperature)
    try:
        out = dict(entropy=torch.empty(B, npos, dtype=f32, device=dev),
                   status=torch.empty(B, npos, dtype=torch.int32, device=dev),
                   top_ids=torch.empty(B, npos, m, dtype=torch.int32, device=dev),
                   top_logprobs=torch.empty(B, npos, m, dtype=f32, device=dev))
        if tokens is not None:
            out["logprob"] = torch.empty(B, npos, dtype=f32, device=dev)
        o = _PACK_LOGPROBS_OUT.pack(out["logprob"].data_ptr() if tokens is not None else 0,
                                    out["entropy"].data_ptr(), out["top_ids"].data_ptr(),
                                    out["top_logprobs"].data_ptr(), out["status"].data_ptr())
        _check(_fn("spec_token_logprobs", 3)(a, o, _raw_stream(index)))
    finally:
        _leave(on)
    return out


def set_wait_timeout_ns(ns):
    lib().spec_set_wait_timeout_ns(int(ns))


def get_wait_timeout_ns():
    return lib().spec_get_wait_timeout_ns()


def debug_force_wait_timeout(on):
    lib().spec_debug_force_wait_timeout(int(on))
