"""GB300 (sm_103a) kernelized linear attention, phi(x) = elu(x) + 1.

Thin Python binding over the C ABI of include/linattn.h.  The functions carry
the C names and only marshal arguments: torch supplies device memory and the
current CUDA stream; every step of the computation runs in liblinattn.so.

    la_forward_causal(Q, K, V, ...)      V'_i = phi(Q_i)^T S_i / phi(Q_i)^T Z_i, j <= i
    la_backward_causal(Q, K, V, dOut, ...)
    la_forward_noncausal(Q, K, V, ...)   phi(Q)(phi(K)^T V) / phi(Q) sum phi(K)
    la_decode_step(q, k, v, S, Z, ...)   S += phi(k)v^T, Z += phi(k); read with q
    la_forward_gated_scan(A, X, ...)     h_t = a_t h_{t-1} + x_t per channel; its backward and step
    la_page_map, la_paged_append, la_paged_decode_step   softmax attention over a paged KV cache

Shapes: Q, K [B,H,N,D]; V [B,H,N,M]; S [B,H,D,M] fp32; Z [B,H,D] fp32.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native

_lib = _native.lib

_DT = {torch.float32: _native.LA_DTYPE_F32, torch.bfloat16: _native.LA_DTYPE_BF16}


class LinAttnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_lib.la_status_string(status).decode()}: {msg}")
        self.status = status


def _check(status: int) -> None:
    if status != _native.LA_OK:
        raise LinAttnError(status, (_lib.la_last_error_message() or b"").decode())


def _stream_handle(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _dims(Q, V):
    if Q.dim() != 4 or V.dim() != 4:
        raise ValueError("Q/K must be [B,H,N,D] and V [B,H,N,M]")
    B, H, N, D = Q.shape
    if tuple(V.shape[:3]) != (B, H, N):
        raise ValueError(f"V shape {tuple(V.shape)} does not match Q {tuple(Q.shape)}")
    return B, H, N, D, V.shape[3]


def _dtype(t):
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return _DT[t.dtype]


def la_causal_ckpt_floats(B, H, N, D, M):
    """fp32 words of the optional state checkpoints (la_forward_causal(ckpt=...))."""
    return int(_lib.la_causal_ckpt_floats(B, H, N, D, M))


def la_forward_causal(Q, K, V, out=None, S_init=None, Z_init=None, return_state=False,
                      den=None, ckpt=None, stream=None):
    """Causal forward.  Returns Out, or (Out, S_final, Z_final) with return_state.

    den: optional fp32 [B, H, N] tensor that receives the normaliser
    phi(Q_i).Z_i of every token, to hand to la_backward_causal(Den=...).
    ckpt: optional fp32 tensor of la_causal_ckpt_floats(B, H, N, D, M) elements
    that receives state checkpoints, to hand to la_backward_causal(Ckpt=...)."""
    B, H, N, D, M = _dims(Q, V)
    dev = Q.device
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _need(t, n, Q.dtype, dev)
    if K.shape != Q.shape:
        raise ValueError("K must have the shape of Q")
    if out is None:
        out = torch.empty((B, H, N, M), dtype=Q.dtype, device=dev)
    _need(out, "out", Q.dtype, dev)
    if (S_init is None) != (Z_init is None):
        raise ValueError("give both S_init and Z_init, or neither")
    if S_init is not None:
        _need(S_init, "S_init", torch.float32, dev)
        _need(Z_init, "Z_init", torch.float32, dev)
    if den is not None:
        _need(den, "den", torch.float32, dev)
        if tuple(den.shape) != (B, H, N):
            raise ValueError(f"den must be [B, H, N] = {(B, H, N)}, got {tuple(den.shape)}")
    _check_ckpt(ckpt, "ckpt", B, H, N, D, M, dev)
    S_f = Z_f = None
    if return_state:
        S_f = torch.empty((B, H, D, M), dtype=torch.float32, device=dev)
        Z_f = torch.empty((B, H, D), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(_lib.la_forward_causal(_ptr(Q), _ptr(K), _ptr(V), _ptr(out), B, H, N, D, M,
                                      _dtype(Q), _ptr(S_init), _ptr(Z_init), _ptr(S_f), _ptr(Z_f),
                                      _ptr(den), _ptr(ckpt), _stream_handle(stream)))
    return (out, S_f, Z_f) if return_state else out


def _check_ckpt(c, name, B, H, N, D, M, dev):
    if c is None:
        return
    _need(c, name, torch.float32, dev)
    if c.numel() != la_causal_ckpt_floats(B, H, N, D, M):
        raise ValueError(f"{name} must hold la_causal_ckpt_floats(...) = "
                         f"{la_causal_ckpt_floats(B, H, N, D, M)} floats, got {c.numel()}")


def la_backward_causal(Q, K, V, dOut, Out=None, dQ=None, dK=None, dV=None, Den=None,
                       Ckpt=None, stream=None):
    """Causal backward; returns (dQ, dK, dV).  Out (the forward output), Den
    (its normaliser, fp32 [B, H, N]) and Ckpt (its state checkpoints) are optional."""
    B, H, N, D, M = _dims(Q, V)
    dev = Q.device
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (dOut, "dOut")):
        _need(t, n, Q.dtype, dev)
    if Out is not None:
        _need(Out, "Out", Q.dtype, dev)
    if Den is not None:
        _need(Den, "Den", torch.float32, dev)
        if tuple(Den.shape) != (B, H, N):
            raise ValueError(f"Den must be [B, H, N] = {(B, H, N)}, got {tuple(Den.shape)}")
    _check_ckpt(Ckpt, "Ckpt", B, H, N, D, M, dev)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    for t, n in ((dQ, "dQ"), (dK, "dK"), (dV, "dV")):
        _need(t, n, Q.dtype, dev)
    with torch.cuda.device(dev):
        _check(_lib.la_backward_causal(_ptr(Q), _ptr(K), _ptr(V), _ptr(Out), _ptr(dOut), _ptr(dQ),
                                       _ptr(dK), _ptr(dV), B, H, N, D, M, _dtype(Q), _ptr(Den),
                                       _ptr(Ckpt), _stream_handle(stream)))
    return dQ, dK, dV


def la_forward_noncausal(Q, K, V, out=None, stream=None):
    B, H, N, D, M = _dims(Q, V)
    dev = Q.device
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _need(t, n, Q.dtype, dev)
    if out is None:
        out = torch.empty((B, H, N, M), dtype=Q.dtype, device=dev)
    _need(out, "out", Q.dtype, dev)
    with torch.cuda.device(dev):
        _check(_lib.la_forward_noncausal(_ptr(Q), _ptr(K), _ptr(V), _ptr(out), B, H, N, D, M,
                                         _dtype(Q), _stream_handle(stream)))
    return out


def la_backward_noncausal(Q, K, V, dOut, Out=None, dQ=None, dK=None, dV=None, stream=None):
    """Backward of la_forward_noncausal; returns (dQ, dK, dV).  Out is optional."""
    B, H, N, D, M = _dims(Q, V)
    dev = Q.device
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (dOut, "dOut")):
        _need(t, n, Q.dtype, dev)
    if K.shape != Q.shape or dOut.shape != V.shape:
        raise ValueError("K must have the shape of Q and dOut the shape of V")
    if Out is not None:
        _need(Out, "Out", Q.dtype, dev)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    for t, n in ((dQ, "dQ"), (dK, "dK"), (dV, "dV")):
        _need(t, n, Q.dtype, dev)
    with torch.cuda.device(dev):
        _check(_lib.la_backward_noncausal(_ptr(Q), _ptr(K), _ptr(V), _ptr(Out), _ptr(dOut), _ptr(dQ),
                                          _ptr(dK), _ptr(dV), B, H, N, D, M, _dtype(Q),
                                          _stream_handle(stream)))
    return dQ, dK, dV


def la_forward_noncausal_noalloc(Q, K, V, out=None, stream=None):
    """la_forward_noncausal for callers that may not allocate device memory.

    The library side allocates nothing (its scratch is a fixed 16 MiB device
    array); pass `out` to keep this Python wrapper from allocating the output.
    Calls that overlap on the GPU share that array and must be serialised.
    """
    B, H, N, D, M = _dims(Q, V)
    dev = Q.device
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _need(t, n, Q.dtype, dev)
    if out is None:
        out = torch.empty((B, H, N, M), dtype=Q.dtype, device=dev)
    _need(out, "out", Q.dtype, dev)
    with torch.cuda.device(dev):
        _check(_lib.la_forward_noncausal_noalloc(_ptr(Q), _ptr(K), _ptr(V), _ptr(out), B, H, N, D,
                                                 M, _dtype(Q), _stream_handle(stream)))
    return out


def la_decode_step(q, k, v, S, Z, out=None, stream=None):
    """One decode step; updates S, Z in place and returns out [B,H,M] fp32."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q/k must be [B,H,D] and v [B,H,M]")
    B, H, D = q.shape
    M = v.shape[2]
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(S, "S", torch.float32, dev)
    _need(Z, "Z", torch.float32, dev)
    if tuple(S.shape) != (B, H, D, M) or tuple(Z.shape) != (B, H, D):
        raise ValueError("S must be [B,H,D,M] and Z [B,H,D]")
    if out is None:
        out = torch.empty((B, H, M), dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev)
    with torch.cuda.device(dev):
        _check(_lib.la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(S), _ptr(Z), _ptr(out), B, H, D,
                                   M, _dtype(q), _stream_handle(stream)))
    return out


def la_workspace_bytes(op, B, H, N, D, M, dtype, saved=0, num_sms=0):
    """Scratch bytes one call of entry point `op` takes from the library pool.

    dtype: torch.float32 or torch.bfloat16.  saved: OR of LA_SAVED_OUT,
    LA_SAVED_DEN, LA_SAVED_CKPT (la_backward_causal's optional inputs).
    num_sms <= 0 asks the current device for its SM count."""
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    n = _lib.la_workspace_bytes(op.encode(), B, H, N, D, M, _DT[dtype], int(saved), int(num_sms))
    if n == _native.SIZE_MAX:
        raise LinAttnError(_native.LA_ERR_INVALID_ARG, la_last_error_message())
    return int(n)


def la_scratch_peak_bytes(reset=False):
    """Peak bytes of the library's scratch pool held at once on the current device."""
    n = _lib.la_scratch_peak_bytes(1 if reset else 0)
    if n == _native.SIZE_MAX:
        raise LinAttnError(_native.LA_ERR_CUDA, la_last_error_message())
    return int(n)


LA_SAVED_OUT, LA_SAVED_DEN, LA_SAVED_CKPT = (_native.LA_SAVED_OUT, _native.LA_SAVED_DEN,
                                             _native.LA_SAVED_CKPT)


def la_forward_poly2(Q, K, V, causal=True, out=None, stream=None):
    """Attention with similarity (Q_i . K_j)^2 through its degree-2 feature map (D = 32)."""
    B, H, N, D, M = _dims(Q, V)
    dev = Q.device
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _need(t, n, Q.dtype, dev)
    if K.shape != Q.shape:
        raise ValueError("K must have the shape of Q")
    if out is None:
        out = torch.empty((B, H, N, M), dtype=Q.dtype, device=dev)
    _need(out, "out", Q.dtype, dev)
    with torch.cuda.device(dev):
        _check(_lib.la_forward_poly2(_ptr(Q), _ptr(K), _ptr(V), _ptr(out), B, H, N, D, M, _dtype(Q),
                                     1 if causal else 0, _stream_handle(stream)))
    return out


def _decay_args(gamma_head, gates, shape, dev, name):
    if gamma_head is not None and gates is not None:
        raise ValueError(f"give gamma_head or {name}, not both")
    if gamma_head is not None:
        _need(gamma_head, "gamma_head", torch.float32, dev)
        if tuple(gamma_head.shape) != (shape[1],):
            raise ValueError(f"gamma_head must be [H] = {(shape[1],)}")
    if gates is not None:
        _need(gates, name, torch.float32, dev)
        if tuple(gates.shape) != tuple(shape):
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(gates.shape)}")


def la_forward_retention(Q, K, V, gamma_head=None, gates=None, out=None, S_init=None,
                         return_state=False, stream=None):
    """Linear attention with decay: S_t = gamma_t S_{t-1} + k_t v_t^T, Out_t = S_t^T q_t.

    gamma_head [H] (RetNet), gates [B,H,N] (gated retention) or neither (decay 1).
    Returns Out, or (Out, S_final) with return_state."""
    B, H, N, D, M = _dims(Q, V)
    dev = Q.device
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _need(t, n, Q.dtype, dev)
    if K.shape != Q.shape:
        raise ValueError("K must have the shape of Q")
    _decay_args(gamma_head, gates, (B, H, N), dev, "gates")
    if out is None:
        out = torch.empty((B, H, N, M), dtype=Q.dtype, device=dev)
    _need(out, "out", Q.dtype, dev)
    if S_init is not None:
        _need(S_init, "S_init", torch.float32, dev)
    S_f = torch.empty((B, H, D, M), dtype=torch.float32, device=dev) if return_state else None
    with torch.cuda.device(dev):
        _check(_lib.la_forward_retention(_ptr(Q), _ptr(K), _ptr(V), _ptr(out), B, H, N, D, M,
                                         _dtype(Q), _ptr(gamma_head), _ptr(gates), _ptr(S_init),
                                         _ptr(S_f), _stream_handle(stream)))
    return (out, S_f) if return_state else out


def la_retention_decode_step(q, k, v, S, gamma_head=None, gate=None, out=None, stream=None):
    """One retention step: S = gamma S + k v^T (in place), returns out = S^T q [B,H,M] fp32."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q/k must be [B,H,D] and v [B,H,M]")
    B, H, D = q.shape
    M = v.shape[2]
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(S, "S", torch.float32, dev)
    if tuple(S.shape) != (B, H, D, M):
        raise ValueError("S must be [B,H,D,M]")
    _decay_args(gamma_head, gate, (B, H), dev, "gate")
    if out is None:
        out = torch.empty((B, H, M), dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev)
    with torch.cuda.device(dev):
        _check(_lib.la_retention_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma_head), _ptr(gate),
                                             _ptr(S), _ptr(out), B, H, D, M, _dtype(q),
                                             _stream_handle(stream)))
    return out


def la_softmax_decode_step(q, k, v, K_cache, V_cache, T, out=None, stream=None):
    """Softmax attention decode step with a KV cache (the comparator of la_decode_step).

    Writes k, v into row T of K_cache [B,H,T_max,D] / V_cache [B,H,T_max,M] and
    returns out [B,H,M] fp32 = softmax(q K^T / sqrt(D)) V over rows 0..T."""
    if q.dim() != 3 or v.dim() != 3 or K_cache.dim() != 4 or V_cache.dim() != 4:
        raise ValueError("q, k [B,H,D], v [B,H,M], caches [B,H,T_max,D] / [B,H,T_max,M]")
    B, H, D = q.shape
    M = v.shape[2]
    T_max = K_cache.shape[2]
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (K_cache, "K_cache"), (V_cache, "V_cache")):
        _need(t, n, q.dtype, dev)
    if tuple(K_cache.shape) != (B, H, T_max, D) or tuple(V_cache.shape) != (B, H, T_max, M):
        raise ValueError("cache shapes do not match q and v")
    if out is None:
        out = torch.empty((B, H, M), dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev)
    with torch.cuda.device(dev):
        _check(_lib.la_softmax_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(K_cache), _ptr(V_cache),
                                           int(T), T_max, _ptr(out), B, H, D, M, _dtype(q),
                                           _stream_handle(stream)))
    return out


_FORMS = {"decay": _native.LA_GATE_DECAY, "logit": _native.LA_GATE_LOGIT}


def _shaped(t, name, shape, dtype, dev):
    """Refuses t unless it is a contiguous tensor of this shape and dtype on CUDA device `dev`.

    The entry points below are short calls, so what passes is decided by the cheapest
    tests; the message is made up only for what does not."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and dev >= 0 and t.is_contiguous()):
        return
    _need(t, name, dtype, torch.device("cuda", dev) if dev >= 0 else None)
    raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


# The C calls' sizes are 32 bits wide, and ctypes would cut larger ones.  Only sizes that memory
# has room for are looked at: not the pools', whose rows take 64 bytes and more.
_INT_MAX = 2 ** 31 - 1


def _fits(*tensors):
    """Refuses tensors with a size past 32 bits (called where one has that many elements)."""
    n = max(max(t.shape) for t in tensors)
    if n > _INT_MAX:
        raise ValueError(f"a size of {n} does not fit 32 bits")


def _int(x, name):
    """x as a whole number of 32 bits."""
    if type(x) is int and -_INT_MAX <= x <= _INT_MAX:
        return x
    n = int(x)
    if n != x or not -_INT_MAX <= n <= _INT_MAX:
        raise ValueError(f"{name} must be a whole number of 32 bits, got {x}")
    return n


def _launch(fn, dev, stream, *args):
    """fn(*args, stream handle) with device `dev` current: `stream`, or dev's current stream."""
    if _current_device() == dev:
        s = fn(*args, _raw_stream(dev) if stream is None else int(stream.cuda_stream))
    else:
        with torch.cuda.device(dev):
            s = fn(*args, _raw_stream(dev) if stream is None else int(stream.cuda_stream))
    if s:
        _check(s)


# The raw handle of a device's current stream, and the current device's number, without
# the objects that torch.cuda's functions make for them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: int(torch.cuda.current_stream(dev).cuda_stream))
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _scan_args(A, X, form, seq_starts):
    """(B, N, C, sequences, num_seqs, form code, device) of a gated scan call, its inputs checked."""
    if form not in _FORMS:
        raise ValueError(f"form must be one of {sorted(_FORMS)}, got {form!r}")
    if not isinstance(A, torch.Tensor) or A.dim() != 3:
        raise ValueError("A and X must be [B,N,C]")
    shape, dev = A.shape, A.get_device()
    _shaped(A, "A", shape, A.dtype, dev)
    _shaped(X, "X", shape, A.dtype, dev)
    B, N, C = shape
    if A.numel() > _INT_MAX:
        _fits(A)
    if seq_starts is None:
        return B, N, C, B, 0, _FORMS[form], dev
    if not isinstance(seq_starts, torch.Tensor) or seq_starts.dim() != 1 or seq_starts.numel() < 1:
        raise ValueError("seq_starts must be a tensor [num_seqs + 1]")
    _shaped(seq_starts, "seq_starts", seq_starts.shape, torch.int32, dev)
    if B != 1:
        raise ValueError(f"packed sequences need B == 1, got {B}")
    S = seq_starts.numel() - 1
    return B, N, C, S, S, _FORMS[form], dev


def la_gated_scan_ckpt_floats(B, N, C):
    """fp32 words of the gated scan's checkpoints (la_forward_gated_scan(ckpt=...))."""
    return int(_lib.la_gated_scan_ckpt_floats(_int(B, "B"), _int(N, "N"), _int(C, "C")))


def _bytes(n):
    if n == _native.SIZE_MAX:
        raise LinAttnError(_native.LA_ERR_INVALID_ARG, la_last_error_message())
    return int(n)


def la_gated_scan_workspace_bytes(B, N, C, dtype, backward=False, ckpt_given=False):
    """Scratch bytes of one la_forward_gated_scan or la_backward_gated_scan call."""
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    B, N, C = _int(B, "B"), _int(N, "N"), _int(C, "C")
    return _bytes(_lib.la_gated_scan_workspace_bytes(int(backward), B, N, C, _DT[dtype], int(ckpt_given)))


def la_paged_decode_workspace_bytes(R, Hq, Hkv, D, page_size, max_pages, dtype, num_sms=0):
    """Scratch bytes of one la_paged_decode_step call; num_sms <= 0 asks the current device."""
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    sizes = [_int(x, n) for x, n in ((R, "R"), (Hq, "Hq"), (Hkv, "Hkv"), (D, "D"), (page_size, "page_size"),
                                     (max_pages, "max_pages"))]
    return _bytes(_lib.la_paged_decode_workspace_bytes(*sizes, _DT[dtype], num_sms))


def la_page_map_workspace_bytes(R):
    """Scratch bytes of one la_page_map call over R requests."""
    return _bytes(_lib.la_page_map_workspace_bytes(_int(R, "R")))


def _check_scan_ckpt(c, name, B, N, C, dev):
    n = la_gated_scan_ckpt_floats(B, N, C)
    if not isinstance(c, torch.Tensor) or c.numel() != n:
        raise ValueError(f"{name} must hold la_gated_scan_ckpt_floats(...) = {n} floats")
    _shaped(c, name, c.shape, torch.float32, dev)


def la_forward_gated_scan(A, X, form="decay", out=None, h_init=None, return_state=False, ckpt=None,
                          seq_starts=None, stream=None):
    """Gated recurrence over rows [B,N,C]: h_t = a_t h_{t-1} + x_t ("decay"), or with
    s_t = sigmoid(a_t): h_t = s_t h_{t-1} + (1 - s_t) x_t ("logit").

    seq_starts: optional int32 [S+1] cutting the rows of a B = 1 call into packed
    sequences; h_init, and the final state with return_state, are then [S,C] (else [B,C]),
    fp32.  ckpt: optional fp32 tensor of la_gated_scan_ckpt_floats(B, N, C) elements that
    receives states for la_backward_gated_scan(Ckpt=...).  Returns Out, or (Out, h_final).

    Rows that no packed sequence holds are 0 in an Out that the call allocates, and left as
    they are in `out`."""
    B, N, C, S, num, code, dev = _scan_args(A, X, form, seq_starts)
    dt, fill = A.dtype, int(out is None)
    if out is None:
        out = torch.empty_like(A)
    else:
        _shaped(out, "out", (B, N, C), dt, dev)
    if h_init is not None:
        _shaped(h_init, "h_init", (S, C), torch.float32, dev)
    if ckpt is not None:
        _check_scan_ckpt(ckpt, "ckpt", B, N, C, dev)
    h_f = torch.empty((S, C), dtype=torch.float32, device=A.device) if return_state else None
    _launch(_lib.la_forward_gated_scan_padded, dev, stream, A.data_ptr(), X.data_ptr(), out.data_ptr(), B, N, C,
            _dtype(A), code, _ptr(seq_starts), num, _ptr(h_init), _ptr(h_f), _ptr(ckpt), fill)
    return (out, h_f) if return_state else out


def la_backward_gated_scan(A, X, dOut, form="decay", h_init=None, dh_final=None, return_dh_init=False,
                           Ckpt=None, dA=None, dX=None, seq_starts=None, stream=None):
    """Backward of la_forward_gated_scan; returns (dA, dX) or (dA, dX, dh_init).

    dh_final: optional gradient at the final state; Ckpt: the forward's checkpoints
    (computed by the call when absent).  Rows that no packed sequence holds are 0 in
    gradients that the call allocates, and left as they are in dA and dX given to it."""
    B, N, C, S, num, code, dev = _scan_args(A, X, form, seq_starts)
    dt, fill = A.dtype, (dA is None) + 2 * (dX is None)
    _shaped(dOut, "dOut", (B, N, C), dt, dev)
    if dA is None:
        dA = torch.empty_like(A)
    else:
        _shaped(dA, "dA", (B, N, C), dt, dev)
    if dX is None:
        dX = torch.empty_like(X)
    else:
        _shaped(dX, "dX", (B, N, C), dt, dev)
    if h_init is not None:
        _shaped(h_init, "h_init", (S, C), torch.float32, dev)
    if dh_final is not None:
        _shaped(dh_final, "dh_final", (S, C), torch.float32, dev)
    if Ckpt is not None:
        _check_scan_ckpt(Ckpt, "Ckpt", B, N, C, dev)
    dh = torch.empty((S, C), dtype=torch.float32, device=A.device) if return_dh_init else None
    _launch(_lib.la_backward_gated_scan_padded, dev, stream, A.data_ptr(), X.data_ptr(), dOut.data_ptr(),
            dA.data_ptr(), dX.data_ptr(), B, N, C, _dtype(A), code, _ptr(seq_starts), num, _ptr(h_init),
            _ptr(dh_final), _ptr(dh), _ptr(Ckpt), fill)
    return (dA, dX, dh) if return_dh_init else (dA, dX)


def la_gated_scan_decode_step(a, x, h, form="decay", out=None, stream=None):
    """One token of the gated recurrence: updates h [B,C] fp32 in place, returns out [B,C]."""
    if form not in _FORMS:
        raise ValueError(f"form must be one of {sorted(_FORMS)}, got {form!r}")
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a and x must be [B,C]")
    shape, dt, dev = a.shape, a.dtype, a.get_device()
    if a.numel() > _INT_MAX:
        _fits(a)
    _shaped(a, "a", shape, dt, dev)
    _shaped(x, "x", shape, dt, dev)
    _shaped(h, "h", shape, torch.float32, dev)
    if out is None:
        out = torch.empty_like(a)
    else:
        _shaped(out, "out", shape, dt, dev)
    _launch(_lib.la_gated_scan_decode_step, dev, stream, a.data_ptr(), x.data_ptr(), h.data_ptr(),
            out.data_ptr(), shape[0], shape[1], _dtype(a), _FORMS[form])
    return out


def la_page_map(cached_lens, new_lens, free_pages, block_table, page_size, num_pages, slot_map,
                seq_starts=None, counts=None, stream=None):
    """Block table and slot map of a step from request lengths (all int32, on the GPU).

    Pages that the new positions open are taken from free_pages in the order of the requests
    and written into block_table [R,W]; slot_map [max_tokens] receives the new positions'
    slots (-1 behind the last), seq_starts [R+1] their row ranges, counts [2] the new
    positions and the pages wanted.  Returns (slot_map, seq_starts, counts)."""
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [R, max_pages]")
    i32, dev = torch.int32, block_table.get_device()
    _shaped(block_table, "block_table", block_table.shape, i32, dev)
    R, W = block_table.shape
    _shaped(cached_lens, "cached_lens", (R,), i32, dev)
    _shaped(new_lens, "new_lens", (R,), i32, dev)
    for t, n in ((free_pages, "free_pages"), (slot_map, "slot_map")):
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            raise ValueError(f"{n} must be a tensor of one dimension")
        _shaped(t, n, t.shape, i32, dev)
    if block_table.numel() + free_pages.numel() + slot_map.numel() > _INT_MAX:
        _fits(block_table, free_pages, slot_map)
    if seq_starts is None:
        seq_starts = torch.empty(R + 1, dtype=i32, device=block_table.device)
    else:
        _shaped(seq_starts, "seq_starts", (R + 1,), i32, dev)
    if counts is None:
        counts = torch.empty(2, dtype=i32, device=block_table.device)
    else:
        _shaped(counts, "counts", (2,), i32, dev)
    _launch(_lib.la_page_map, dev, stream, cached_lens.data_ptr(), new_lens.data_ptr(), R,
            free_pages.data_ptr(), free_pages.shape[0], _int(page_size, "page_size"), _int(num_pages, "num_pages"),
            block_table.data_ptr(), W, slot_map.data_ptr(), slot_map.shape[0], seq_starts.data_ptr(),
            counts.data_ptr())
    return slot_map, seq_starts, counts


def _pools(K_pages, V_pages):
    """(num_pages, Hkv, page_size, D, device) of the pools, checked."""
    if not isinstance(K_pages, torch.Tensor) or K_pages.dim() != 4:
        raise ValueError("K_pages and V_pages must be [num_pages, Hkv, page_size, D]")
    shape, dev = K_pages.shape, K_pages.get_device()
    _shaped(K_pages, "K_pages", shape, K_pages.dtype, dev)
    _shaped(V_pages, "V_pages", shape, K_pages.dtype, dev)
    return (*shape, dev)


def la_paged_append(k, v, K_pages, V_pages, slot_map, stream=None):
    """Writes rows k, v [T,Hkv,D] into the slots slot_map [T] (int32; -1 skips a row) of the
    pools K_pages, V_pages [num_pages,Hkv,page_size,D]."""
    P, Hkv, page, D, dev = _pools(K_pages, V_pages)
    dt = K_pages.dtype
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k and v must be [T, Hkv, D]")
    T = k.shape[0]
    _shaped(k, "k", (T, Hkv, D), dt, dev)
    _shaped(v, "v", (T, Hkv, D), dt, dev)
    _shaped(slot_map, "slot_map", (T,), torch.int32, dev)
    _launch(_lib.la_paged_append, dev, stream, k.data_ptr(), v.data_ptr(), K_pages.data_ptr(),
            V_pages.data_ptr(), slot_map.data_ptr(), T, Hkv, D, P, page, _dtype(K_pages))


def la_paged_decode_step(q, k, v, K_pages, V_pages, block_table, cached_lens, window=0, scale=None,
                         out=None, return_lse=False, stream=None, lse=None):
    """Softmax attention decode step over a paged KV cache, one request per row.

    Appends k, v [R,Hkv,D] at position cached_lens[r] of each request (None, None: appends
    nothing) and returns out [R,Hq,D] fp32 = softmax(scale q K^T) V over the request's last
    `window` positions (0: all), with return_lse also the log of the sum [R,Hq] fp32 (in `lse` if
    given).  Rows with a negative length (no request) are left as they are in an out or lse given
    to the call; in one that it allocates they are 0 and -infinity.  scale None: 1 / sqrt(D)."""
    P, Hkv, page, D, dev = _pools(K_pages, V_pages)
    dt = K_pages.dtype
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [R, Hq, D]")
    R, Hq = q.shape[:2]
    _shaped(q, "q", (R, Hq, D), dt, dev)
    if (k is None) != (v is None):
        raise ValueError("give both k and v, or neither")
    if k is not None:
        _shaped(k, "k", (R, Hkv, D), dt, dev)
        _shaped(v, "v", (R, Hkv, D), dt, dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError(f"block_table must be [R, max_pages] with R = {R}")
    _shaped(block_table, "block_table", block_table.shape, torch.int32, dev)
    if block_table.numel() > _INT_MAX:
        _fits(block_table)
    _shaped(cached_lens, "cached_lens", (R,), torch.int32, dev)
    if scale is None:
        scale = 0.0
    elif ctypes.c_float(float(scale)).value == 0.0:  # the C call's 0 means the default
        raise ValueError("scale must not be 0 in fp32")
    fill = 0
    if out is None:
        out = torch.empty((R, Hq, D), dtype=torch.float32, device=q.device)
        fill = 1
    else:
        _shaped(out, "out", (R, Hq, D), torch.float32, dev)
    if lse is not None:
        _shaped(lse, "lse", (R, Hq), torch.float32, dev)
    elif return_lse:
        lse = torch.empty((R, Hq), dtype=torch.float32, device=q.device)
        fill |= 2
    _launch(_lib.la_paged_decode_step_padded, dev, stream, q.data_ptr(), _ptr(k), _ptr(v), K_pages.data_ptr(),
            V_pages.data_ptr(), block_table.data_ptr(), cached_lens.data_ptr(), out.data_ptr(), _ptr(lse), R,
            Hq, Hkv, D, P, page, block_table.shape[1], _int(window, "window"), float(scale), _dtype(K_pages), fill)
    return (out, lse) if return_lse else out


def la_check_device_status(stream=None):
    _check(_lib.la_check_device_status(_stream_handle(stream)))


def la_selftest_expired_waits(stream=None):
    """Launch a block whose bounded device waits expire (tests the error-word path).

    The next la_check_device_status() raises LinAttnError with LA_ERR_TIMEOUT.
    """
    _check(_lib.la_selftest_expired_waits(_stream_handle(stream)))


def la_kernel_launch_count() -> int:
    return int(_lib.la_kernel_launch_count())


def la_status_string(status: int) -> str:
    return _lib.la_status_string(int(status)).decode()


def la_last_error_message() -> str:
    return (_lib.la_last_error_message() or b"").decode()
