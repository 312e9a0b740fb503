"""ctypes binding of libspec_verify.so (argument marshalling only).

Every step of the verification runs in the library's CUDA kernels; this module
checks tensor shapes/dtypes, allocates outputs and the workspace with torch on
the caller's device, passes raw device pointers and the current stream, and
raises on a non-zero return code.  There is no CPU fallback: if the library
cannot be loaded the call fails.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspec_verify.so")

F32, BF16 = 0, 1
OK, ERR_INVALID_ARG, ERR_WORKSPACE, ERR_CUDA, ERR_UNSUPPORTED = 0, 1, 2, 3, 4
ST_NONFINITE, ST_BAD_TOKEN, ST_BAD_GAMMA, ST_ZERO_RESIDUAL = 1, 2, 4, 8
ST_GUARDED, ST_TIMEOUT, ST_BAD_TEMPERATURE, ST_BAD_UNIFORM = 16, 32, 64, 128
ST_BAD_PENALTY, ST_BAD_LENGTH = 256, 512

_lock = threading.Lock()
_lib = None


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} (code {code})")


def lib(path: str | None = None) -> ctypes.CDLL:
    """Load the shared library (built by ``build.build()``) and set signatures."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise FileNotFoundError(
                f"{p} is missing: build it with `python -m speculative_decoding_verification_26_gb300.build`")
        L = ctypes.CDLL(p)
        P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.spec_workspace_bytes.argtypes = [I, I, I]
        L.spec_workspace_bytes.restype = SZ
        L.spec_status_string.argtypes = [I]
        L.spec_status_string.restype = ctypes.c_char_p
        L.spec_request_status_string.argtypes = [I]
        L.spec_request_status_string.restype = ctypes.c_char_p
        L.spec_launch_count.argtypes = []
        L.spec_launch_count.restype = ctypes.c_uint64
        L.spec_profile_next_call.argtypes = [P, P]
        L.spec_profile_next_call.restype = I
        L.spec_set_wait_limit.argtypes = [ctypes.c_longlong]
        L.spec_set_wait_limit.restype = I
        L.spec_verify_greedy.argtypes = [P, I, I, I, I, P, P, P, P, P, P, SZ, P]
        L.spec_verify_greedy.restype = I
        L.spec_verify_sample.argtypes = [P, P, I, I, I, I, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.spec_verify_sample.restype = I
        L.spec_verify_onehot.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P, P, P, SZ, P]
        L.spec_verify_onehot.restype = I
        L.spec_draft_signals.argtypes = [P, I, I, I, I, P, P, P, P, P, P, SZ, P]
        L.spec_divergence_stats.argtypes = [P, P, I, I, I, I, P, P, P, P, P]
        L.spec_divergence_stats.restype = I
        L.spec_gamma_select.argtypes = [P, P, P, I, P, P, P]
        L.spec_filter_top_k_top_p.argtypes = [P, I, I, I, P, P, P, P, P]
        L.spec_filter_top_k_top_p.restype = I
        L.spec_gamma_select.restype = I
        L.spec_draft_signals.restype = I
        F = ctypes.c_float
        L.spec_topk_logits.argtypes = [P, I, I, I, I, P, P, P, P, P, P]
        L.spec_topk_logits.restype = I
        L.spec_distill_topk.argtypes = [P, I, I, I, I, P, P, P, P, P, P, F, F, F, P, P, P, P, P]
        L.spec_distill_topk.restype = I
        L.spec_linear_ce_workspace_bytes.argtypes = [I, I, I, I]
        L.spec_linear_ce_workspace_bytes.restype = SZ
        L.spec_linear_ce_forward.argtypes = [P, P, I, I, I, I, P, P, P, P, P, SZ, P]
        L.spec_linear_ce_forward.restype = I
        L.spec_linear_ce_backward.argtypes = [P, P, I, I, I, I, P, P, P, P, P, P, SZ, P]
        L.spec_linear_ce_backward.restype = I
        L.spec_w4_quantize.argtypes = [P, I, I, I, I, P, P, P, P, P]
        L.spec_w4_quantize.restype = I
        L.spec_w4_dequantize.argtypes = [P, P, P, I, I, I, P, I, P]
        L.spec_w4_dequantize.restype = I
        L.spec_linear_w4.argtypes = [P, I, I, P, P, P, I, I, I, P, I, P]
        L.spec_linear_w4.restype = I
        L.spec_adjust_logits.argtypes = [P, P, I, I, I, I, P, I, P, P, P, I, P, P, P, P, P, P, I, P, P, P]
        L.spec_adjust_logits.restype = I
        if path is None:
            _lib = L
        return L


def status_string(code: int) -> str:
    return lib().spec_status_string(int(code)).decode()


def request_status_string(bit: int) -> str:
    return lib().spec_request_status_string(int(bit)).decode()


def workspace_bytes(B: int, G: int, V: int) -> int:
    return int(lib().spec_workspace_bytes(int(B), int(G), int(V)))


def launch_count() -> int:
    return int(lib().spec_launch_count())


def set_wait_limit(cycles: int) -> None:
    """Testing aid: internal waits of later calls give up after `cycles` SM
    cycles (<= 0 restores the default); see spec_set_wait_limit."""
    rc = lib().spec_set_wait_limit(int(cycles))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_set_wait_limit")


def profile_next_call(begin, end) -> None:
    """Record torch.cuda.Event `begin`/`end` around the verify kernel of
    the next call made by this thread (see spec_profile_next_call)."""
    rc = lib().spec_profile_next_call(ctypes.c_void_p(begin.cuda_event), ctypes.c_void_p(end.cuda_event))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_profile_next_call")


# ----------------------------------------------------------------------------
# torch-facing wrappers

def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _check(t, name, dtype=None, shape=None, device=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


_ws_locks: dict = {}


def _ws_lock(device: int, stream: int):
    """The lock of a stream's cached workspaces, held from taking one to the end
    of the C call: a call is several launches, and another host thread on the same
    stream must not put its own between them."""
    lock = _ws_locks.get((device, stream))
    return _ws_locks.setdefault((device, stream), threading.Lock()) if lock is None else lock


_ws_cache: dict = {}


def workspace(B, G, V, device):
    """A cached workspace tensor for these sizes on `device` (reused by calls
    on the same stream; calls sharing it must not overlap on the device, nor be
    made by several host threads at once: the calls that take it by default see
    to that)."""
    torch = _torch()
    torch.cuda.init()
    device = torch.device(device)
    i = torch.cuda.current_device() if device.index is None else device.index
    return _cached_ws(B, G, V, device, (i, _raw_stream(i)))


def _cached_ws(B, G, V, device, key):
    n = workspace_bytes(B, G, V)
    if n == 0:
        raise ValueError("sizes outside the library limits")
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < n:
        torch = _torch()
        ws = _ws_cache[key] = torch.empty(n, dtype=torch.uint8, device=device)
    return ws


class _Held:
    """A verification call's workspace while the call is made: the caller's, or
    the stream's cached one under its lock."""
    __slots__ = ("ws", "sizes", "dev", "lock")

    def __init__(self, ws, B, G, V, dev):
        self.ws, self.sizes, self.dev, self.lock = ws, (B, G, V), dev, None

    def __enter__(self):
        if self.ws is not None:
            return self.ws
        i = self.dev.index
        stream = _raw_stream(i)
        lock = _ws_lock(i, stream)
        lock.acquire()
        self.lock = lock
        try:
            return _cached_ws(*self.sizes, self.dev, (i, stream))
        except BaseException:
            lock.release()
            raise

    def __exit__(self, *exc):
        if self.lock is not None:
            self.lock.release()


def _out(o, key, make):
    t = o.get(key)
    return make() if t is None else t


def _raw_stream(i):
    """The current stream's handle on device i (torch.cuda.current_stream builds an object)."""
    return _torch()._C._cuda_getCurrentRawStream(i)


def _stream(device):
    return ctypes.c_void_p(_raw_stream(device.index))


def verify_greedy(target, draft_tokens, gamma=None, *, ws=None, out=None):
    """Greedy verification.  target [B, G+1, V] bf16/f32; draft_tokens [B, G] int32."""
    torch = _torch()
    B, Gp1, V = target.shape
    G = Gp1 - 1
    dev = target.device
    _check(target, "target", device=dev)
    _check(draft_tokens, "draft_tokens", torch.int32, (B, G), dev)
    _check(gamma, "gamma", torch.int32, (B,), dev)
    o = out or {}
    acc = _out(o, "accept_len", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    tok = _out(o, "tokens", lambda: torch.empty(B, G + 1, dtype=torch.int32, device=dev))
    st = _out(o, "status", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    with _Held(ws, B, G, V, dev) as ws:
        rc = lib().spec_verify_greedy(_ptr(target), _dtype_code(target), B, G, V, _ptr(draft_tokens), _ptr(gamma),
                                      _ptr(acc), _ptr(tok), _ptr(st), _ptr(ws), ws.numel(), _stream(dev))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_verify_greedy")
    return {"accept_len": acc, "tokens": tok, "status": st}


def verify_sample(target, draft, draft_tokens, gamma, temperature, uniforms, *, signals=True,
                  accept_prob=False, ws=None, out=None):
    """Full-q stochastic verification (+ optional draft signals / accept_prob)."""
    torch = _torch()
    B, Gp1, V = target.shape
    G = Gp1 - 1
    dev = target.device
    _check(target, "target", device=dev)
    _check(draft, "draft", target.dtype, (B, G, V), dev)
    _check(draft_tokens, "draft_tokens", torch.int32, (B, G), dev)
    _check(gamma, "gamma", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    _check(uniforms, "uniforms", torch.float32, (B, G + 1), dev)
    o = out or {}
    acc = _out(o, "accept_len", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    tok = _out(o, "tokens", lambda: torch.empty(B, G + 1, dtype=torch.int32, device=dev))
    st = _out(o, "status", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    sig = (_out(o, "signals", lambda: torch.empty(B, 4, dtype=torch.float32, device=dev))) if signals else None
    ap = (_out(o, "accept_prob", lambda: torch.empty(B, G, dtype=torch.float32, device=dev))) if accept_prob else None
    with _Held(ws, B, G, V, dev) as ws:
        rc = lib().spec_verify_sample(_ptr(target), _ptr(draft), _dtype_code(target), B, G, V, _ptr(draft_tokens),
                                      _ptr(gamma), _ptr(temperature), _ptr(uniforms), _ptr(acc), _ptr(tok), _ptr(sig),
                                      _ptr(ap), _ptr(st), _ptr(ws), ws.numel(), _stream(dev))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_verify_sample")
    r = {"accept_len": acc, "tokens": tok, "status": st}
    if sig is not None:
        r["signals"] = sig
    if ap is not None:
        r["accept_prob"] = ap
    return r


def verify_onehot(target, draft_tokens, gamma, temperature, uniforms, *, accept_prob=False, ws=None, out=None):
    """One-hot-q stochastic verification."""
    torch = _torch()
    B, Gp1, V = target.shape
    G = Gp1 - 1
    dev = target.device
    _check(target, "target", device=dev)
    _check(draft_tokens, "draft_tokens", torch.int32, (B, G), dev)
    _check(gamma, "gamma", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    _check(uniforms, "uniforms", torch.float32, (B, G + 1), dev)
    o = out or {}
    acc = _out(o, "accept_len", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    tok = _out(o, "tokens", lambda: torch.empty(B, G + 1, dtype=torch.int32, device=dev))
    st = _out(o, "status", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    ap = (_out(o, "accept_prob", lambda: torch.empty(B, G, dtype=torch.float32, device=dev))) if accept_prob else None
    with _Held(ws, B, G, V, dev) as ws:
        rc = lib().spec_verify_onehot(_ptr(target), _dtype_code(target), B, G, V, _ptr(draft_tokens), _ptr(gamma),
                                      _ptr(temperature), _ptr(uniforms), _ptr(acc), _ptr(tok), _ptr(ap), _ptr(st),
                                      _ptr(ws), ws.numel(), _stream(dev))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_verify_onehot")
    r = {"accept_len": acc, "tokens": tok, "status": st}
    if ap is not None:
        r["accept_prob"] = ap
    return r


def divergence_stats(target, draft, gamma, temperature, *, out=None):
    """Per-position divergence statistics.  target [B, G+1, V], draft [B, G, V];
    returns {"stats": [B, G, 5] (A, L1, KL(p||q), KL(q||p), H(p), bits),
    "status": [B]}."""
    torch = _torch()
    B, G, V = draft.shape
    dev = draft.device
    _check(target, "target", shape=(B, G + 1, V), device=dev)
    _check(draft, "draft", device=dev)
    if target.dtype != draft.dtype:
        raise TypeError("target and draft dtypes differ")
    _check(gamma, "gamma", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    o = out or {}
    stats = _out(o, "stats", lambda: torch.empty(B, G, 5, dtype=torch.float32, device=dev))
    st = _out(o, "status", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    rc = lib().spec_divergence_stats(_ptr(target), _ptr(draft), _dtype_code(draft), B, G, V, _ptr(gamma),
                                     _ptr(temperature), _ptr(stats), _ptr(st), _stream(dev))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_divergence_stats")
    return {"stats": stats, "status": st}


def filter_top_k_top_p(logits, top_k=None, top_p=None, temperature=None, *, status=None):
    """Top-k / top-p filtering of the rows of `logits` ([..., V], contiguous,
    fp32 or bf16) in place; top_k [n] int32, top_p [n] fp32, temperature [n]
    fp32, each optional (n = rows).  Returns the per-row status tensor."""
    torch = _torch()
    V = logits.shape[-1]
    n = logits.numel() // V
    dev = logits.device
    _check(logits, "logits", device=dev)
    _check(top_k, "top_k", torch.int32, (n,), dev)
    _check(top_p, "top_p", torch.float32, (n,), dev)
    _check(temperature, "temperature", torch.float32, (n,), dev)
    st = status if status is not None else torch.empty(n, dtype=torch.int32, device=dev)
    rc = lib().spec_filter_top_k_top_p(_ptr(logits), _dtype_code(logits), n, V, _ptr(top_k), _ptr(top_p),
                                       _ptr(temperature), _ptr(st), _stream(dev))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_filter_top_k_top_p")
    return st


GAMMA_MODEL_FLOATS = 141


def gamma_select(signals, model, comp=None, *, out=None):
    """SpecKV gamma selection.  signals [B, 4] fp32 (mean H, max H, mean c,
    min c), model [141] fp32, comp [B] fp32 or None; returns {"gamma": [B]
    int32 (2, 4, 6, 8; -1 for non-finite features), "expected": [B, 4]}."""
    torch = _torch()
    B = signals.shape[0]
    dev = signals.device
    _check(signals, "signals", torch.float32, (B, 4), dev)
    _check(model, "model", torch.float32, (GAMMA_MODEL_FLOATS,), dev)
    _check(comp, "comp", torch.float32, (B,), dev)
    o = out or {}
    g = _out(o, "gamma", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    e = _out(o, "expected", lambda: torch.empty(B, 4, dtype=torch.float32, device=dev))
    rc = lib().spec_gamma_select(_ptr(signals), _ptr(comp), _ptr(model), B, _ptr(g), _ptr(e), _stream(dev))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_gamma_select")
    return {"gamma": g, "expected": e}


def draft_signals(draft, gamma, temperature, *, row_signals=False, ws=None, out=None):
    """SpecKV draft signals only.  draft [B, G, V]."""
    torch = _torch()
    B, G, V = draft.shape
    dev = draft.device
    _check(draft, "draft", device=dev)
    _check(gamma, "gamma", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    o = out or {}
    sig = _out(o, "signals", lambda: torch.empty(B, 4, dtype=torch.float32, device=dev))
    rs = (_out(o, "row_signals", lambda: torch.empty(B, G, 2, dtype=torch.float32, device=dev))) if row_signals else None
    st = _out(o, "status", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    with _Held(ws, B, G, V, dev) as ws:
        rc = lib().spec_draft_signals(_ptr(draft), _dtype_code(draft), B, G, V, _ptr(gamma), _ptr(temperature),
                                      _ptr(sig), _ptr(rs), _ptr(st), _ptr(ws), ws.numel(), _stream(dev))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_draft_signals")
    r = {"signals": sig, "status": st}
    if rs is not None:
        r["row_signals"] = rs
    return r


MAX_TOPK = 256
DISTILL_MAX_V = 1 << 20


class _Hot:
    """What the calls below need of torch and the library, looked up once.  They
    take a few microseconds on the device for few rows, so their host side is kept
    short: addresses as plain integers, checks with the common case first, and the
    raw handle of the current stream (torch.cuda.current_stream builds an object)."""

    def __init__(self):
        import torch
        L = lib()
        self.torch, self.empty = torch, torch.empty
        self.f32, self.i32, self.bf16 = torch.float32, torch.int32, torch.bfloat16
        self.code = {torch.float32: F32, torch.bfloat16: BF16}
        self.device, self.stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self.topk, self.distill = L.spec_topk_logits, L.spec_distill_topk
        self.ce_forward, self.ce_backward = L.spec_linear_ce_forward, L.spec_linear_ce_backward
        self.quantize, self.dequantize = L.spec_w4_quantize, L.spec_w4_dequantize
        self.linear_w4, self.adjust = L.spec_linear_w4, L.spec_adjust_logits
        self.u8 = torch.uint8


_hot_state = None


def _hot():
    global _hot_state
    if _hot_state is None:
        _hot_state = _Hot()
    return _hot_state


def _call(h, dev, f, *args):
    """Call the C entry point f with `dev` current and its current stream last."""
    i = dev.index
    if h.device() == i:
        rc = f(*args, h.stream(i))
    else:
        with h.torch.cuda.device(dev):
            rc = f(*args, h.stream(i))
    if rc != OK:
        raise SpecVerifyError(rc, f.__name__)


def _addr(t):
    return None if t is None else t.data_ptr()


def _want(t, name, dtype, shape, device):
    """_check of a tensor or None, with the common case first."""
    if t is not None and not (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        _check(t, name, dtype, shape, device)


def _result(out, key, shape, dtype, dev):
    """out[key], checked, or a new tensor."""
    t = out.get(key)
    if t is None:
        return _hot().empty(shape, dtype=dtype, device=dev)
    _check(t, key, dtype, shape, dev)
    return t


def topk_logits(logits, K, temperature=None, *, out=None):
    """The record of teacher rows: logits [..., V] (n rows, fp32 or bf16),
    temperature [n] fp32 or None; returns {"top_logits": [n, K] fp32,
    "top_index": [n, K] int32, "tail_lse": [n], "status": [n]} (see
    spec_topk_logits)."""
    h = _hot()
    f32, i32 = h.f32, h.i32
    _check(logits, "logits")
    V = logits.shape[-1]
    n = logits.numel() // V
    dev = logits.device
    if temperature is not None:
        _want(temperature, "temperature", f32, (n,), dev)
    if out is None:
        empty = h.empty
        top, idx = empty((n, K), dtype=f32, device=dev), empty((n, K), dtype=i32, device=dev)
        tail, st = empty((n,), dtype=f32, device=dev), empty((n,), dtype=i32, device=dev)
    else:
        top, idx = _result(out, "top_logits", (n, K), f32, dev), _result(out, "top_index", (n, K), i32, dev)
        tail, st = _result(out, "tail_lse", (n,), f32, dev), _result(out, "status", (n,), i32, dev)
    code = h.code.get(logits.dtype)
    _call(h, dev, h.topk, logits.data_ptr(), _dtype_code(logits) if code is None else code, n, V, K,
          _addr(temperature), top.data_ptr(), idx.data_ptr(), tail.data_ptr(), st.data_ptr())
    return {"top_logits": top, "top_index": idx, "tail_lse": tail, "status": st}


def distill_topk(logits, top_logits, top_index, tail_lse=None, *, label=None, row_weight=None, temperature=None,
                 kl=1.0, tv=0.0, ce=0.0, grad=False, out=None):
    """The loss of student rows `logits` [..., V] (n rows, fp32 or bf16) against
    records (topk_logits), and with `grad` its gradient by the logits; label [n]
    int32, row_weight [n], temperature [n] fp32, each optional.  Returns
    {"loss": [n], "parts": [n, 3] (KL, TV, CE), "status": [n]} and "grad" (as
    `logits`; out={"grad": logits} overwrites them).  See spec_distill_topk."""
    h = _hot()
    f32, i32 = h.f32, h.i32
    _check(logits, "logits")
    V = logits.shape[-1]
    n = logits.numel() // V
    dev = logits.device
    K = top_logits.shape[-1]
    rows = (n,)
    _want(top_logits, "top_logits", f32, (n, K), dev)
    _want(top_index, "top_index", i32, (n, K), dev)
    _want(tail_lse, "tail_lse", f32, rows, dev)
    _want(label, "label", i32, rows, dev)
    _want(row_weight, "row_weight", f32, rows, dev)
    _want(temperature, "temperature", f32, rows, dev)
    if out is None:
        empty = h.empty
        loss, parts = empty(rows, dtype=f32, device=dev), empty((n, 3), dtype=f32, device=dev)
        st = empty(rows, dtype=i32, device=dev)
        g = empty(logits.shape, dtype=logits.dtype, device=dev) if grad else None
    else:
        loss, parts = _result(out, "loss", rows, f32, dev), _result(out, "parts", (n, 3), f32, dev)
        st = _result(out, "status", rows, i32, dev)
        g = _result(out, "grad", logits.shape, logits.dtype, dev) if grad else None
    code = h.code.get(logits.dtype)
    _call(h, dev, h.distill, logits.data_ptr(), _dtype_code(logits) if code is None else code, n, V, K,
          top_logits.data_ptr(), top_index.data_ptr(), _addr(tail_lse), _addr(label), _addr(row_weight),
          _addr(temperature), kl, tv, ce, loss.data_ptr(), parts.data_ptr(), _addr(g), st.data_ptr())
    r = {"loss": loss, "parts": parts, "status": st}
    if grad:
        r["grad"] = g
    return r


def linear_ce_workspace_bytes(n: int, H: int, V: int, backward: bool) -> int:
    return int(lib().spec_linear_ce_workspace_bytes(int(n), int(H), int(V), int(bool(backward))))


_ce_ws_cache: dict = {}


def linear_ce_workspace(n, H, V, device, *, backward):
    """A cached workspace of linear_ce_forward / linear_ce_backward for these
    sizes (reused by calls on the same stream; calls sharing it must not overlap
    on the device, nor be made by several host threads at once: the calls that
    take it by default see to that).  Under stream capture it is new: a graph
    keeps its own."""
    h = _hot()
    device = h.torch.device(device)
    need = linear_ce_workspace_bytes(n, H, V, backward)
    if need == 0:
        raise ValueError("sizes outside the library limits")
    if h.torch.cuda.is_current_stream_capturing():
        return h.empty(need, dtype=h.torch.uint8, device=device)
    i = h.device() if device.index is None else device.index
    key = (i, h.stream(i))
    ws = _ce_ws_cache.get(key)
    if ws is None or ws.numel() < need:
        _ce_ws_cache.pop(key, None)
        ws = _ce_ws_cache[key] = h.empty(need, dtype=h.torch.uint8, device=device)
    return ws


def _ce_inputs(h, hidden, weight, label):
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError("hidden is [n, H] and weight [V, H]")
    n, H = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    _check(hidden, "hidden", h.bf16)
    _want(weight, "weight", h.bf16, (V, H), dev)
    _want(label, "label", h.i32, (n,), dev)
    return n, H, V, dev


def _ce_call(h, dev, ws, backward, f, hidden, weight, dtype, n, H, V, *rest):
    """_call with the workspace ws, or the stream's cached one."""
    if ws is not None:
        _check(ws, "ws", h.torch.uint8, device=dev)
        return _call(h, dev, f, hidden, weight, dtype, n, H, V, *rest, ws.data_ptr(), ws.numel())
    with _ws_lock(dev.index, h.stream(dev.index)):
        ws = linear_ce_workspace(n, H, V, dev, backward=backward)
        _call(h, dev, f, hidden, weight, dtype, n, H, V, *rest, ws.data_ptr(), ws.numel())


def linear_ce_forward(hidden, weight, label, *, ws=None, out=None):
    """Cross entropy of the projection hidden [n, H] times weight [V, H] (bf16)
    against label [n] int32 (-1: the row takes no part), without its logits.
    Returns {"loss": [n], "lse": [n], "status": [n]} (see spec_linear_ce_forward)."""
    h = _hot()
    n, H, V, dev = _ce_inputs(h, hidden, weight, label)
    o = out or {}
    loss, lse = _result(o, "loss", (n,), h.f32, dev), _result(o, "lse", (n,), h.f32, dev)
    st = _result(o, "status", (n,), h.i32, dev)
    _ce_call(h, dev, ws, False, h.ce_forward, hidden.data_ptr(), weight.data_ptr(), BF16, n, H, V, label.data_ptr(),
             loss.data_ptr(), lse.data_ptr(), st.data_ptr())
    return {"loss": loss, "lse": lse, "status": st}


def linear_ce_backward(hidden, weight, label, lse, grad_loss=None, *, need_hidden=True, need_weight=True, ws=None,
                       out=None):
    """Gradients of sum(grad_loss * loss) by hidden and weight; lse as
    linear_ce_forward returned it, grad_loss [n] fp32 or None (= 1).  Returns
    {"grad_hidden": [n, H] bf16, "grad_weight": [V, H] bf16}, without the one
    that is not needed (see spec_linear_ce_backward)."""
    h = _hot()
    n, H, V, dev = _ce_inputs(h, hidden, weight, label)
    _want(lse, "lse", h.f32, (n,), dev)
    _want(grad_loss, "grad_loss", h.f32, (n,), dev)
    o = out or {}
    gh = _result(o, "grad_hidden", (n, H), h.bf16, dev) if need_hidden else None
    gw = _result(o, "grad_weight", (V, H), h.bf16, dev) if need_weight else None
    _ce_call(h, dev, ws, True, h.ce_backward, hidden.data_ptr(), weight.data_ptr(), BF16, n, H, V, label.data_ptr(),
             lse.data_ptr(), _addr(grad_loss), _addr(gh), _addr(gw))
    r = {}
    if need_hidden:
        r["grad_hidden"] = gh
    if need_weight:
        r["grad_weight"] = gw
    return r


W4_GROUPS = (32, 64, 128)
MAX_HISTORY, MAX_BIASES = 1 << 28, 4096


def _code(h, t):
    code = h.code.get(t.dtype)
    return _dtype_code(t) if code is None else code


def _take(t, name, dtype, shape, dev):
    """The address of a tensor of this dtype and shape on `dev`, checked; None of None."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev.index and t.is_contiguous()):
        _check(t, name, dtype, shape, dev)
    return t.data_ptr()


def _w4_sizes(packed, group):
    """(V, H, the shape of scales) of 4-bit weights."""
    if packed.dim() != 2:
        raise ValueError("packed is [V, H / 2]")
    if group not in W4_GROUPS:
        raise ValueError(f"group must be one of {W4_GROUPS}, got {group}")
    V, H = packed.shape
    H *= 2
    return V, H, (V, -(-H // group))


def quantize_w4(weight, group=128, *, zero=False, out=None):
    """weight [V, H] (fp32 or bf16, H a multiple of 32) in 4 bits, with a bf16
    scale and, with `zero`, a zero point for each `group` of 32, 64 or 128
    weights of a row.  Returns {"packed": [V, H / 2] uint8, "scale": [V,
    ceil(H / group)] bf16, "status": [V]} and "zero" ([V, ceil(H / group)]
    uint8) (see spec_w4_quantize)."""
    h = _hot()
    if weight.dim() != 2:
        raise ValueError("weight is [V, H]")
    if group not in W4_GROUPS:
        raise ValueError(f"group must be one of {W4_GROUPS}, got {group}")
    V, H = weight.shape
    dev = weight.device
    _check(weight, "weight")
    per = (V, -(-H // group))
    if out is None:
        empty = h.empty
        packed, scale = empty((V, H // 2), dtype=h.u8, device=dev), empty(per, dtype=h.bf16, device=dev)
        z = empty(per, dtype=h.u8, device=dev) if zero else None
        st = empty((V,), dtype=h.i32, device=dev)
    else:
        packed, scale = _result(out, "packed", (V, H // 2), h.u8, dev), _result(out, "scale", per, h.bf16, dev)
        z = _result(out, "zero", per, h.u8, dev) if zero else None
        st = _result(out, "status", (V,), h.i32, dev)
    _call(h, dev, h.quantize, weight.data_ptr(), _code(h, weight), V, H, group, packed.data_ptr(), scale.data_ptr(),
          _addr(z), st.data_ptr())
    r = {"packed": packed, "scale": scale, "status": st}
    if zero:
        r["zero"] = z
    return r


def dequantize_w4(packed, scale, zero=None, *, group=128, dtype=None, out=None):
    """The weights [V, H] that quantize_w4's results stand for, in `dtype` (bf16
    by default, or fp32).  Zero points are 0 to 15, not checked.  Returns
    {"weight": [V, H]} (see spec_w4_dequantize)."""
    h = _hot()
    V, H, per = _w4_sizes(packed, group)
    dev = packed.device
    _check(packed, "packed", h.u8)
    s, z = _take(scale, "scale", h.bf16, per, dev), _take(zero, "zero", h.u8, per, dev)
    dtype = dtype or h.bf16
    w = h.empty((V, H), dtype=dtype, device=dev) if out is None else _result(out, "weight", (V, H), dtype, dev)
    _call(h, dev, h.dequantize, packed.data_ptr(), s, z, V, H, group, w.data_ptr(), _code(h, w))
    return {"weight": w}


def linear_w4(hidden, packed, scale, zero=None, *, group=128, dtype=None, out=None):
    """hidden [..., H] (bf16) times 4-bit weights (quantize_w4), transposed:
    {"logits": [..., V]} in `dtype` (bf16 by default, or fp32).  Zero points are 0 to
    15, not checked (see spec_linear_w4)."""
    h = _hot()
    V, H, per = _w4_sizes(packed, group)
    dev = packed.device
    _check(packed, "packed", h.u8)
    s, z = _take(scale, "scale", h.bf16, per, dev), _take(zero, "zero", h.u8, per, dev)
    shape = hidden.shape
    if len(shape) < 1 or shape[-1] != H:
        raise ValueError(f"hidden must have shape [..., {H}], got {tuple(shape)}")
    if not (hidden.dtype is h.bf16 and hidden.get_device() == dev.index and hidden.is_contiguous()):
        _check(hidden, "hidden", h.bf16, device=dev)
    dtype = dtype or h.bf16
    if out is None:
        y = h.empty((*shape[:-1], V), dtype=dtype, device=dev)
    else:
        y = _result(out, "logits", (*shape[:-1], V), dtype, dev)
    _call(h, dev, h.linear_w4, hidden.data_ptr(), BF16, hidden.numel() // H, packed.data_ptr(), s, z, V, H, group,
          y.data_ptr(), _code(h, y))
    return {"logits": y}


def adjust_logits(logits, history=None, history_len=None, *, prompt_len=None, draft_tokens=None, gamma=None,
                  repetition=None, frequency=None, presence=None, bias_index=None, bias_value=None, mask=None, out=None):
    """Penalties for repeated tokens, biases and masks on the rows of logits
    [B, R, V] (fp32 or bf16), in place unless out={"logits": other} is given: row
    i has the history of request b (history [B, L] int32, history_len [B]; the
    first prompt_len [B] entries are its prompt) and its draft tokens y_0 ..
    y_{i-1} (draft_tokens [B, D], D >= R - 1, gamma [B] of them).  repetition,
    frequency, presence [B] fp32; bias_index [B, N] int32 with bias_value [B, N]
    fp32; mask [B, R, ceil(V / 32)] int32, bit v % 32 of word v // 32 for token v,
    1 where it is allowed; each optional.  Returns {"logits", "status": [B]} (see
    spec_adjust_logits)."""
    h = _hot()
    f32, i32 = h.f32, h.i32
    if logits.dim() != 3:
        raise ValueError("logits is [B, R, V]")
    B, R, V = logits.shape
    dev = logits.device
    _check(logits, "logits")
    L = D = N = 0
    told = drafts = index = value = None
    per = (B,)
    if history is not None:
        if history.dim() != 2:
            raise ValueError("history is [B, L]")
        L = history.shape[1]
        told = _take(history, "history", i32, (B, L), dev)
    elif history_len is not None or prompt_len is not None:
        raise ValueError("history_len and prompt_len are those of a history")
    if draft_tokens is not None:
        if draft_tokens.dim() != 2:
            raise ValueError("draft_tokens is [B, D]")
        D = draft_tokens.shape[1]
        drafts = _take(draft_tokens, "draft_tokens", i32, (B, D), dev)
        if D < R - 1:
            raise ValueError(f"draft_tokens has {D} tokens for {R} rows")
    if (bias_index is None) != (bias_value is None):
        raise ValueError("bias_index and bias_value go together")
    if bias_index is not None:
        if bias_index.dim() != 2:
            raise ValueError("bias_index is [B, N]")
        N = bias_index.shape[1]
        index, value = _take(bias_index, "bias_index", i32, (B, N), dev), _take(bias_value, "bias_value", f32, (B, N), dev)
    y = None if out is None else out.get("logits")
    if y is None:
        y = logits
    to = logits.data_ptr() if y is logits else _take(y, "out['logits']", logits.dtype, logits.shape, dev)
    st = None if out is None else out.get("status")
    if st is None:
        st = h.empty(per, dtype=i32, device=dev)
    _call(h, dev, h.adjust, logits.data_ptr(), to, _code(h, logits), B, R, V, told, L,
          _take(history_len, "history_len", i32, per, dev), _take(prompt_len, "prompt_len", i32, per, dev), drafts, D,
          _take(gamma, "gamma", i32, per, dev), _take(repetition, "repetition", f32, per, dev),
          _take(frequency, "frequency", f32, per, dev), _take(presence, "presence", f32, per, dev), index, value, N,
          _take(mask, "mask", i32, (B, R, (V + 31) // 32), dev), _take(st, "status", i32, per, dev))
    return {"logits": y, "status": st}


STATIC_WORKSPACE_BYTES = 8 << 20


def verify_sample_static(target, draft, draft_tokens, gamma, temperature, uniforms, *, signals=True,
                         accept_prob=False, out=None):
    """verify_sample on the library's own static scratch (spec_verify_sample_static).

    The C call allocates nothing; this wrapper allocates outputs only when
    `out` does not supply them.  Calls on one device must not overlap."""
    torch = _torch()
    L = lib()
    f = L.spec_verify_sample_static
    if f.argtypes is None:
        P, I = ctypes.c_void_p, ctypes.c_int
        f.argtypes = [P, P, I, I, I, I, P, P, P, P, P, P, P, P, P, P]
        f.restype = I
    B, Gp1, V = target.shape
    G = Gp1 - 1
    dev = target.device
    _check(target, "target", device=dev)
    _check(draft, "draft", target.dtype, (B, G, V), dev)
    _check(draft_tokens, "draft_tokens", torch.int32, (B, G), dev)
    _check(gamma, "gamma", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    _check(uniforms, "uniforms", torch.float32, (B, G + 1), dev)
    o = out or {}
    acc = _out(o, "accept_len", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    tok = _out(o, "tokens", lambda: torch.empty(B, G + 1, dtype=torch.int32, device=dev))
    st = _out(o, "status", lambda: torch.empty(B, dtype=torch.int32, device=dev))
    sig = (_out(o, "signals", lambda: torch.empty(B, 4, dtype=torch.float32, device=dev))) if signals else None
    ap = (_out(o, "accept_prob", lambda: torch.empty(B, G, dtype=torch.float32, device=dev))) if accept_prob else None
    rc = f(_ptr(target), _ptr(draft), _dtype_code(target), B, G, V, _ptr(draft_tokens), _ptr(gamma),
           _ptr(temperature), _ptr(uniforms), _ptr(acc), _ptr(tok), _ptr(sig), _ptr(ap), _ptr(st), _stream(dev))
    if rc != OK:
        raise SpecVerifyError(rc, "spec_verify_sample_static")
    r = {"accept_len": acc, "tokens": tok, "status": st}
    if sig is not None:
        r["signals"] = sig
    if ap is not None:
        r["accept_prob"] = ap
    return r
