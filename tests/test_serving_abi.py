"""Refusals of the gated scan's and the paged cache's entry points, on the host:
no call here reaches a kernel."""
import pytest
import torch

import linear_attention_02_gb300 as la
from linear_attention_02_gb300 import _native

lib = _native.lib
FAKE = 0x10000  # aligned, never dereferenced
INV, UNS, OK = _native.LA_ERR_INVALID_ARG, _native.LA_ERR_UNSUPPORTED, _native.LA_OK


def _msg():
    return lib.la_last_error_message().decode()


def _fwd(A=FAKE, X=FAKE, O=FAKE, B=1, N=8, C=4, dt=0, form=0, st=None, ns=0, hi=None, hf=None, ck=None):
    return lib.la_forward_gated_scan(A, X, O, B, N, C, dt, form, st, ns, hi, hf, ck, None)


def _bwd(A=FAKE, X=FAKE, G=FAKE, dA=FAKE, dX=FAKE, B=1, N=8, C=4, dt=0, form=0, st=None, ns=0, hi=None,
         df=None, d0=None, ck=None):
    return lib.la_backward_gated_scan(A, X, G, dA, dX, B, N, C, dt, form, st, ns, hi, df, d0, ck, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_scan_refusals(call):
    assert call(A=None) == INV and "A is NULL" in _msg()
    assert call(X=FAKE + 8) == INV and "X is not 16-byte aligned" in _msg()
    assert call(N=-1) == INV and call(B=-1) == INV and call(C=-3) == INV
    assert call(dt=2) == UNS and "dtype" in _msg()
    assert call(form=2) == UNS and "gate form" in _msg()
    assert call(B=2, st=FAKE, ns=2) == INV and "B == 1" in _msg()
    assert call(ns=2) == INV and "without seq_starts" in _msg()
    assert call(st=FAKE, ns=-1) == INV
    assert call(st=FAKE + 2, ns=1) == INV and "seq_starts" in _msg()
    assert call(hi=FAKE + 4) == INV and "h_init" in _msg()
    assert call(ck=FAKE + 4) == INV and "Ckpt" in _msg()
    assert call(B=1 << 20, N=1 << 20, C=4) == INV and "too large" in _msg()
    assert call(B=1, N=(1 << 31) - 1, C=1) == INV and "too large" in _msg()
    assert call(st=FAKE, ns=1 << 30, C=1) == INV and "too large" in _msg()
    # nothing to do and no state asked for: no device call
    for kw in ({"B": 0}, {"N": 0}, {"C": 0}, {"st": FAKE, "ns": 0}):
        assert call(A=None, X=None, **kw) == OK


def test_scan_step_refusals():
    f = lib.la_gated_scan_decode_step
    assert f(FAKE, FAKE, None, FAKE, 2, 8, 0, 0, None) == INV and "h is NULL" in _msg()
    assert f(FAKE, FAKE, FAKE, FAKE + 4, 2, 8, 0, 0, None) == INV
    assert f(FAKE, FAKE, FAKE, FAKE, -2, 8, 0, 0, None) == INV
    assert f(FAKE, FAKE, FAKE, FAKE, 2, 8, 5, 0, None) == UNS
    assert f(FAKE, FAKE, FAKE, FAKE, 2, 8, 0, 7, None) == UNS
    assert f(None, None, None, None, 0, 8, 0, 0, None) == OK


def test_scan_checkpoint_size():
    assert lib.la_gated_scan_ckpt_floats(2, 1, 5) == 10
    assert lib.la_gated_scan_ckpt_floats(3, 257, 64) == 3 * 3 * 64
    assert lib.la_gated_scan_ckpt_floats(0, 257, 64) == 0


def _map(c=FAKE, n=FAKE, R=2, fp=FAKE, nf=3, page=16, P=10, bt=FAKE, W=4, sm=FAKE, T=5, ss=FAKE, ct=FAKE):
    return lib.la_page_map(c, n, R, fp, nf, page, P, bt, W, sm, T, ss, ct, None)


def test_page_map_refusals():
    for page in (0, -16, 3, 24, 2048):
        assert _map(page=page) == UNS and "page_size" in _msg()
    assert _map(P=-1) == INV and _map(P=1 << 27) == INV and "2^31" in _msg()
    assert _map(W=1 << 27) == INV
    assert _map(R=-1) == INV and _map(T=-1) == INV and _map(nf=-1) == INV and _map(W=-1) == INV
    assert _map(c=None) == INV and "cached_lens is NULL" in _msg()
    assert _map(ss=None) == INV and _map(ct=None) == INV and _map(sm=FAKE + 2) == INV
    assert _map(bt=None) == INV and _map(fp=None) == INV
    assert _map(R=(1 << 31) - 1) == INV and "2^30" in _msg()
    assert lib.la_page_map_workspace_bytes((1 << 31) - 1) == _native.SIZE_MAX


def _app(k=FAKE, v=FAKE, K=FAKE, V=FAKE, sm=FAKE, T=3, Hkv=2, D=64, P=4, page=16, dt=1):
    return lib.la_paged_append(k, v, K, V, sm, T, Hkv, D, P, page, dt, None)


def test_append_refusals():
    assert _app(D=48) == UNS and _app(dt=3) == UNS and _app(page=12) == UNS
    assert _app(T=-1) == INV and _app(Hkv=-1) == INV
    assert _app(k=FAKE + 4) == INV and "k is not 16-byte" in _msg()
    assert _app(K=None) == INV and _app(sm=None) == INV
    assert _app(T=1, Hkv=1 << 30, D=32, P=1, page=1) == INV and "too large" in _msg()
    assert _app(T=0, k=None) == OK and _app(Hkv=0, k=None) == OK


def _dec(q=FAKE, k=FAKE, v=FAKE, K=FAKE, V=FAKE, bt=FAKE, ln=FAKE, out=FAKE, lse=None, R=2, Hq=8, Hkv=2, D=64,
         P=4, page=16, W=3, win=0, scale=0.0, dt=1):
    return lib.la_paged_decode_step(q, k, v, K, V, bt, ln, out, lse, R, Hq, Hkv, D, P, page, W, win, scale, dt, None)


def test_paged_decode_refusals():
    assert _dec(D=96) == UNS and _dec(dt=9) == UNS and _dec(page=17) == UNS
    assert _dec(Hq=7) == INV and "not a multiple" in _msg()
    assert _dec(Hkv=0) == INV
    assert _dec(k=None) == INV and "both" in _msg()
    assert _dec(win=-1) == INV and _dec(R=-1) == INV
    assert _dec(scale=float("nan")) == INV and _dec(scale=float("inf")) == INV
    assert _dec(q=FAKE + 2) == INV and _dec(k=FAKE + 8) == INV and _dec(lse=FAKE + 1) == INV
    assert _dec(bt=None) == INV and _dec(ln=None) == INV and _dec(out=None) == INV
    assert _dec(P=1 << 27) == INV and _dec(W=1 << 27, page=16) == INV
    assert _dec(R=0, q=None) == OK and _dec(Hq=0, Hkv=0, q=None) == OK


def test_status_string():
    assert lib.la_status_string(5) == b"LA_ERR_BAD_INDEX"


def test_binding_refuses_host_tensors_and_shapes():
    a = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_forward_gated_scan(a, a)
    with pytest.raises(ValueError, match="form"):
        la.la_forward_gated_scan(a, a, form="sigmoid")
    with pytest.raises(ValueError, match=r"\[B,N,C\]"):
        la.la_backward_gated_scan(a[0], a[0], a[0])
    with pytest.raises(ValueError, match=r"\[B,C\]"):
        la.la_gated_scan_decode_step(a, a, a)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table"):
        la.la_page_map(i, i, i, i, 16, 4, i)
    with pytest.raises(ValueError, match="K_pages"):
        la.la_paged_append(a, a, a, a, i)
    with pytest.raises(ValueError, match="K_pages"):
        la.la_paged_decode_step(a, None, None, a, a, i, i)


def test_workspace_bytes():
    f = lib.la_gated_scan_workspace_bytes
    # 257 rows: 3 tiles; A and B (and the end states without checkpoints) of 2 x 3 x 64 words, 4 words of ticket
    states = 2 * 3 * 64
    assert f(0, 2, 257, 64, 0, 1) == 4 * (4 + 2 * states)
    assert f(0, 2, 257, 64, 1, 0) == 4 * (4 + 3 * states)
    assert f(1, 2, 257, 64, 1, 1) == 4 * (4 + 3 * states)
    # backward without checkpoints: the states, and the larger of its two passes on top
    assert f(1, 2, 257, 64, 0, 0) == 4 * states + 4 * (4 + 3 * states)
    assert f(1, 2, 128, 64, 0, 0) == 0 and f(0, 0, 257, 64, 0, 0) == 0
    assert f(0, -1, 257, 64, 0, 0) == _native.SIZE_MAX
    g = lib.la_paged_decode_workspace_bytes
    # bf16, D = 64: 3 blocks an SM x 4 warps = 12 x 152 warps, one range each (2 x 8 columns of 5 + 2 steps at
    # most are fewer than 16 a warp): 2 partial results of 4 heads x 68 words, 16 bytes of descriptor, 16 bytes
    w = 12 * 152
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert g(2, 32, 8, 64, 16, 5, 1, 152) == up(4 * w * 2 * 4 * 68) + 16 * w + 16
    # long tables: up to four ranges a warp
    assert g(200, 32, 8, 64, 16, 5000, 1, 152) == up(4 * 4 * w * 2 * 4 * 68) + 16 * 4 * w + 16
    assert g(2, 32, 8, 48, 16, 5, 1, 152) == _native.SIZE_MAX and g(2, 30, 8, 64, 16, 5, 1, 152) == _native.SIZE_MAX
    assert lib.la_page_map_workspace_bytes(4096) == 0 and lib.la_page_map_workspace_bytes(5000) == 8 * 5001
    assert lib.la_page_map_workspace_bytes(-1) == _native.SIZE_MAX
