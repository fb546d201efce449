"""Refusals of the rotary calls and of the prefill, on the host: no call here reaches a kernel."""
import ctypes

import pytest
import torch

import linear_attention_02_gb300 as la
from linear_attention_02_gb300 import _native

lib = _native.lib
FAKE = 0x10000  # aligned, never dereferenced
INV, UNS, OK = _native.LA_ERR_INVALID_ARG, _native.LA_ERR_UNSUPPORTED, _native.LA_OK


def _msg():
    return lib.la_last_error_message().decode()


def _strides(*x):
    return (ctypes.c_int64 * len(x))(*x)


def _rot(fn, extra=(), q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, B=2, N=8, Hq=4, Hk=2, D=64, st=None, pos=None, rows=0,
         first=0, fr=FAKE, rot=64, mag=1.0, lay=0, dt=1, fill=0, wq=None, wk=None, eps=1e-6, dwq=None, dwk=None, g=FAKE):
    tail = (B, N, Hq, Hk, D, st, pos, rows, first, fr, rot, mag, lay)
    if fn == "plain":
        return lib.la_forward_rotary(q, k, qo, ko, *tail, dt, fill, None)
    if fn == "back":
        return lib.la_backward_rotary(q, k, qo, ko, *tail, dt, fill, None)
    if fn == "norm":
        return lib.la_forward_norm_rotary(q, k, wq, wk, qo, ko, *tail, eps, dt, fill, None)
    return lib.la_backward_norm_rotary(q, k, g, g, wq, wk, qo, ko, dwq, dwk, *tail, eps, dt, fill, None)


@pytest.mark.parametrize("fn", ["plain", "back", "norm", "normback"])
def test_rotary_refusals(fn):
    call = lambda **kw: _rot(fn, **kw)  # noqa: E731
    assert call(q=None) == INV and "is NULL" in _msg()
    assert call(ko=None) == INV and call(fr=None) == INV and "freqs" in _msg()
    assert call(q=FAKE + 1) == INV and "aligned" in _msg()
    assert call(q=FAKE + 2, dt=0) == INV and call(fr=FAKE + 4) == INV
    for kw in ({"B": -1}, {"N": -1}, {"Hq": -1}, {"Hk": -1}):
        assert call(**kw) == INV and "negative size" in _msg()
    assert call(D=48) == UNS and call(D=256) == UNS and call(dt=2) == UNS and call(lay=2) == UNS
    for rot in (0, 1, 63, 66, -2):
        assert call(rot=rot) == INV and "rot=" in _msg()
    assert call(mag=float("nan")) == INV and call(mag=float("inf")) == INV
    assert call(pos=FAKE, rows=0) == INV and call(pos=FAKE, rows=3) == INV and call(rows=1) == INV
    assert call(pos=FAKE + 2, rows=1) == INV and "positions" in _msg()
    assert call(pos=FAKE, rows=1, first=1) == INV and call(first=-1) == INV and call(first=(1 << 31) - 4) == INV
    assert call(fill=4) == INV and call(fill=-1) == INV
    assert call(N=1 << 30) == INV and "too large" in _msg()
    assert call(B=1 << 15, N=1 << 15) == INV and call(Hq=1 << 25) == INV
    n = 18 if fn == "normback" else 12
    assert call(st=_strides(*([1 << 40] + [64] * (n - 1)))) == INV and "stride" in _msg()
    # nothing to do: no device call
    assert call(N=0, q=None) == OK and call(Hq=0, Hk=0, q=None, k=None) == OK


@pytest.mark.parametrize("fn", ["norm", "normback"])
def test_norm_refusals(fn):
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert _rot(fn, eps=eps) == INV and "eps" in _msg()
    assert _rot(fn, wq=FAKE + 2) == INV and "weight" in _msg()
    if fn == "normback":
        assert _rot(fn, dwk=FAKE + 1) == INV and "dk_weight" in _msg()
        assert _rot(fn, g=None) == INV and "dq_out is NULL" in _msg()


def _pre(q=FAKE, K=FAKE, V=FAKE, bt=FAKE, ln=FAKE, ss=FAKE, out=FAKE, lse=None, T=9, R=2, Hq=8, Hkv=2, D=64, P=4,
         page=16, W=3, win=0, scale=0.0, dt=1, fill=0):
    return lib.la_paged_prefill(q, K, V, bt, ln, ss, out, lse, T, R, Hq, Hkv, D, P, page, W, win, scale, dt, fill, None)


def test_prefill_refusals():
    assert _pre(D=96) == UNS and _pre(dt=9) == UNS and _pre(page=17) == UNS and _pre(page=2048) == UNS
    assert _pre(Hq=7) == INV and "not a multiple" in _msg()
    assert _pre(Hkv=0) == INV
    for kw in ({"T": -1}, {"R": -1}, {"Hq": -1}, {"Hkv": -1}, {"W": -1}, {"win": -1}):
        assert _pre(**kw) == INV and "negative size" in _msg()
    for s in (float("nan"), float("inf"), 3e38):
        assert _pre(scale=s) == INV and "scale" in _msg()
    assert _pre(q=FAKE + 2) == INV and _pre(out=None) == INV and _pre(K=None) == INV and _pre(V=FAKE + 8) == INV
    assert _pre(bt=None) == INV and _pre(ln=None) == INV and _pre(ss=FAKE + 1) == INV and "seq_starts" in _msg()
    assert _pre(lse=FAKE + 2) == INV and _pre(fill=2) == INV and "lse is NULL" in _msg()
    assert _pre(fill=4) == INV
    assert _pre(P=1 << 27) == INV and _pre(W=1 << 27) == INV and _pre(R=1 << 20) == INV
    assert _pre(T=1 << 29) == INV and "too large" in _msg()
    assert _pre(T=0, q=None) == OK and _pre(Hq=0, Hkv=0, q=None) == OK and _pre(R=0, q=None) == OK


def test_binding_refusals():
    a, f = torch.zeros(4, 2, 64), torch.zeros(32, dtype=torch.int64)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: la.la_forward_rotary(a, a, f), lambda: la.la_backward_rotary(a, None, f),
                 lambda: la.la_forward_norm_rotary(a, a, None, None, f),
                 lambda: la.la_backward_norm_rotary(a, a, a, a, None, None, f)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="layout"):
        la.la_forward_rotary(a, a, f, layout="pairs")
    with pytest.raises(ValueError, match=r"\[B,H,N,D\]"):
        la.la_forward_rotary(None, None, f)
    with pytest.raises(ValueError, match=r"\[B,H,N,D\]"):
        la.la_forward_rotary(a[0], a[0], f)
    with pytest.raises(ValueError, match="scaling"):
        la.la_rotary_frequencies(64, scaling="yes", device="cpu")
    with pytest.raises(la.LinAttnError, match="rot"):
        la.la_rotary_frequencies(63, device="cpu")
    with pytest.raises(ValueError, match="K_pages"):
        la.la_paged_prefill(a, a, a, i, i, i)
    freqs, mag = la.la_rotary_frequencies(64, device="cpu")
    assert freqs.dtype == torch.int64 and freqs.shape == (32,) and mag == 1.0


def test_prefill_workspace():
    f = lib.la_paged_prefill_workspace_bytes
    # bf16: 152 blocks; two partial tiles each of 256 rows of D sums, a maximum and a sum, and two descriptors of 16 bytes
    for D in (32, 64, 128):
        assert f(D, 1, 152) == 152 * 2 * (256 * (4 * D + 8) + 16)
    # fp32: tiles of 128 rows, two blocks an SM up to D = 64
    assert f(64, 0, 152) == 304 * 2 * (128 * (4 * 64 + 8) + 16) and f(128, 0, 152) == 152 * 2 * (128 * (4 * 128 + 8) + 16)
    assert f(48, 1, 152) == _native.SIZE_MAX and f(64, 2, 152) == _native.SIZE_MAX


def test_norm_workspace():
    f = lib.la_norm_rotary_workspace_bytes
    assert f(2, 100, 8, 2, 64, 152) == 2 * 4 * 2 * 152 * 64  # rows of 64 sums, two blocks an SM for each side at most
    assert f(0, 100, 8, 2, 64, 152) == 0 and f(2, 100, 0, 0, 64, 152) == 0
    assert f(2, 100, 8, 2, 48, 152) == _native.SIZE_MAX and f(-1, 100, 8, 2, 64, 152) == _native.SIZE_MAX
