"""GPU tests of the gated scan's logit form at logits from -20 to 20, element by element.

Tolerances.  With e = e^-z, s = 1 / (1 + e) and 1 - s = e s, computed in fp32: the exponent
z log2 e takes two roundings (of the constant and of the product), 2^-23 |z| relative in e; the
power is within 2^-22.5 of itself, the sum, the reciprocal (one unit) and the product take
2^-24 + 2^-23 + 2^-24 more: the smaller of s and 1 - s is within r(z) = (|z| + 6) 2^-23 of
itself, the larger one (one less the smaller) within (1 + (|z| + 6) min(1, e, 1/e)) 2^-23,
which r(z) covers too.  A gradient has up to four more roundings of 2^-24: g(z) = (|z| + 8) 2^-23.
A state moves by min(s, 1 - s) times the difference of state and input, then is rounded:
g(z) min(s, 1 - s) (|h| + |x|) + 2^-24 |h'| a row.  Over rows these add up as the gates carry
them on.  bf16 results are rounded once more, by 2^-8 of their value.
"""
import numpy as np
import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


def _la():
    import linear_attention_02_gb300 as la
    return la


def _g(z):
    return (np.abs(z) + 8) * 2.0 ** -23


def _inputs(B, N, C, dt, seed, low=-20.0, high=20.0):
    g = torch.Generator().manual_seed(seed)
    x = {"A": (torch.rand(B, N, C, generator=g) * (high - low) + low).to(DT[dt]),
         "X": torch.randn(B, N, C, generator=g).to(DT[dt]), "G": torch.randn(B, N, C, generator=g).to(DT[dt]),
         "h0": torch.randn(B, C, generator=g), "dh": torch.randn(B, C, generator=g)}
    return x, {k: v.cuda() for k, v in x.items()}, {k: v.double().numpy() for k, v in x.items()}


def _near(got, want, bound, dt="f32"):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= bound + HALF[dt] * (np.abs(want) + bound))
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {(np.abs(got - want) / np.maximum(bound, 1e-300)).max():.3g} bounds"


def _state_bounds(p, prev, out):
    """Bound of every row's state, row by row."""
    s, c = ref._gates(p["A"], "logit")
    e = np.zeros_like(p["h0"])
    bound = np.zeros_like(out)
    for t in range(out.shape[1]):
        # a run of rows is also kept as a product of decays, each factor rounded once more
        e = s[:, t] * (1 + 2.0 ** -23) * e + _g(p["A"][:, t]) * np.minimum(s, c)[:, t] * (
            np.abs(prev[:, t]) + np.abs(p["X"][:, t])) + 2.0 ** -23 * s[:, t] * np.abs(prev[:, t]) + 2.0 ** -23 * np.abs(out[:, t])
        bound[:, t] = e
    return bound


def _check(B, N, C, dt, seed, low=-20.0, high=20.0, packed=False):
    la = _la()
    x, d, p = _inputs(B, N, C, dt, seed, low, high)
    S, st, starts = B, None, None
    shape = (B, N, C)
    if packed:  # the batch's sequences one after the other
        shape, starts = (1, B * N, C), [i * N for i in range(B + 1)]
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    A, X, G = (d[n].reshape(shape) for n in ("A", "X", "G"))
    out, hf = la.la_forward_gated_scan(A, X, form="logit", h_init=d["h0"], seq_starts=st, return_state=True)
    dA, dX, d0 = la.la_backward_gated_scan(A, X, G, form="logit", h_init=d["h0"], dh_final=d["dh"], seq_starts=st,
                                           return_dh_init=True)
    la.la_check_device_status()
    out, dA, dX = (t.reshape(B, N, C) for t in (out, dA, dX))
    s, c = ref._gates(p["A"], "logit")
    want, wf, prev = ref.gated_scan_forward(x["A"], x["X"], "logit", x["h0"])
    eh = _state_bounds(p, prev, want)
    _near(out, want, eh, dt)
    _near(hf, wf, eh[:, -1])
    wA, wX, w0 = ref.gated_scan_backward(x["A"], x["X"], x["G"], "logit", x["h0"], x["dh"])
    # the whole gradient's size and error at every row, from the last one up
    big, err = np.abs(p["dh"]), np.zeros_like(p["dh"])
    bX, bA = np.zeros_like(wX), np.zeros_like(wA)
    ep = np.concatenate([np.zeros((B, 1, C)), eh[:, :-1]], 1)  # of the state before the row
    for t in range(N - 1, -1, -1):
        tot = np.abs(p["G"][:, t]) + big
        e = err + 2.0 ** -24 * tot
        r = _g(p["A"][:, t])
        bX[:, t] = c[:, t] * (e + r * tot)
        diff = np.abs(prev[:, t] - p["X"][:, t])
        bA[:, t] = s[:, t] * c[:, t] * ((e + r * tot) * diff + tot * ep[:, t])
        big, err = s[:, t] * tot, s[:, t] * (e + r * tot)
    _near(dX, wX, bX, dt)
    _near(dA, wA, bA, dt)
    _near(d0, w0, err)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B,N,C", [(70, 1, 256), (70, 1, 33), (3, 2, 72), (2, 700, 72), (2, 300, 41), (4, 600, 304)])
def test_logits_from_minus_20_to_20(B, N, C, packed, dt):
    _check(B, N, C, dt, B + N + C, packed=packed)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("low,high", [(5.0, 9.0), (12.0, 20.0), (-20.0, -8.0)])
def test_long_memory_and_closed_gates(low, high, packed, dt):
    _check(2, 1500, 40, dt, 7, low, high, packed)


def test_channels_of_long_memory_take_in_their_input():
    # logit 17 or 18: 1 - s is below half a unit of s, yet 5000 rows of it add up
    la = _la()
    for z in (17.0, 18.0):
        A = torch.full((1, 5000, 64), z, device="cuda")
        X = torch.ones_like(A)
        h = la.la_forward_gated_scan(A, X, form="logit", return_state=True)[1]
        s = 1 / (1 + np.exp(-z))
        want = 1 - s ** 5000
        # every row adds a like amount, rounded as it is added to at most the end's value
        tol = (z + 8) * 2.0 ** -23 * want + 5000 * 2.0 ** -24 * want
        assert float((h.double().cpu() - want).abs().max()) <= tol
        dA, dX = la.la_backward_gated_scan(A, X, X, form="logit")
        assert bool((dX > 0).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,C", [(64, 100), (5, 33), (1, 8)])
def test_single_token_step(B, C, dt):
    la = _la()
    x, d, p = _inputs(B, 1, C, dt, B)
    h = d["h0"].clone()
    out = la.la_gated_scan_decode_step(d["A"][:, 0].contiguous(), d["X"][:, 0].contiguous(), h, form="logit")
    want, _, prev = ref.gated_scan_forward(x["A"], x["X"], "logit", x["h0"])
    bound = _state_bounds(p, prev, want)[:, 0]
    _near(h, want[:, 0], bound)
    _near(out, want[:, 0], bound, dt)


def test_gates_at_infinity_are_open_or_closed():
    la = _la()
    inf = float("inf")
    A = torch.tensor([inf, -inf, 1e30, -1e30, 200.0, -200.0, 90.0, -90.0], device="cuda").repeat(1, 260, 1)
    X = torch.full_like(A, 3.0)
    h0 = torch.full((1, 8), 5.0, device="cuda")
    out, h = la.la_forward_gated_scan(A, X, form="logit", h_init=h0, return_state=True)
    want = torch.tensor([5.0, 3.0] * 4, device="cuda")
    assert torch.equal(out, want.expand_as(out)) and torch.equal(h[0], want)
    dA, dX, d0 = la.la_backward_gated_scan(A, X, X, form="logit", h_init=h0, return_dh_init=True)
    assert not bool(dA[..., :6].any())
    assert not bool(dX[..., [0, 2, 4]].any()) and torch.equal(dX[..., 1::2], X[..., 1::2])
    assert d0[0, ::2].tolist() == [780.0] * 4 and not bool(d0[0, [1, 3, 5]].any())
    hs = h0.clone()
    la.la_gated_scan_decode_step(A[:, 0].contiguous(), X[:, 0].contiguous(), hs, form="logit")
    assert torch.equal(hs[0], want)
