"""Rotary calls without a token: the positions are an array without an element then, whose address may be NULL."""
import pytest
import torch

from test_rotary_abi import FAKE, INV, OK, _rot


@pytest.mark.parametrize("fn", ["plain", "back", "norm", "normback"])
def test_no_token_needs_no_positions(fn):
    none = {"q": None, "k": None, "qo": None, "ko": None, "pos": None}
    assert _rot(fn, N=0, rows=1, **none) == OK
    assert _rot(fn, N=0, rows=2, **none) == OK and _rot(fn, B=0, rows=0, **none) == OK and _rot(fn, B=0, rows=1, **none) == OK
    assert _rot(fn, N=0, pos=FAKE, rows=1, q=None) == OK
    assert _rot(fn, N=0, rows=3, **none) == INV and _rot(fn, N=0, rows=-1, **none) == INV  # neither 0, 1 nor B
    assert _rot(fn, rows=1) == INV and _rot(fn, rows=2) == INV and _rot(fn, pos=FAKE, rows=0) == INV  # with tokens as before
    assert _rot(fn, pos=FAKE, rows=0, N=0) == INV


@pytest.mark.gpu
@pytest.mark.parametrize("shape,positions", [((0, 4, 64), (0,)), ((2, 4, 0, 64), (0,)), ((2, 4, 0, 64), (2, 0)),
                                             ((0, 4, 7, 64), (0, 7)), ((0, 4, 7, 64), (7,))])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_empty_calls_with_positions(shape, positions, dt):
    import linear_attention_02_gb300 as la
    freqs, _ = la.la_rotary_frequencies(64)
    x = torch.zeros(shape, device="cuda", dtype=dt)
    pos = torch.zeros(positions, device="cuda", dtype=torch.int32)
    w = torch.ones(64, device="cuda")
    for q, k in (la.la_forward_rotary(x, x, freqs, positions=pos), la.la_backward_rotary(x, x, freqs, positions=pos),
                 la.la_forward_norm_rotary(x, x, w, w, freqs, positions=pos)):
        assert q.shape == x.shape and k.shape == x.shape and q.dtype == dt
    dq, dk, dwq, dwk = la.la_backward_norm_rotary(x, x, x, x, w, w, freqs, positions=pos)
    assert dq.shape == x.shape and dk.shape == x.shape
    assert float(dwq.abs().max()) == 0 and float(dwk.abs().max()) == 0
    la.la_check_device_status()
