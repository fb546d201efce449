"""GPU tests of the gated scan over many tiles: states and gradients that live for
thousands of rows, on both sides of the look-back window's choice.

Where the decays are 1 and the values small whole numbers, every sum is a whole
number below 2^24 and exact in fp32 in any order: those tests ask for equality.

With gates near 1 (1 - s of 1e-4 to 4e-3) a state is the sum of about a thousand rows,
eight tiles and more.  Its error is bounded row by row: with H the sum of the sizes of all
that is in it, a row adds up to 2^-23 H for the product and the sum, 2^-23 s H for a
factor of the tiles' products of decays, and in the logit form r (1 - s) (H + |x|) with
r = (|z| + 8) 2^-23 for the gate; all of it decays as the state does.  Gradients likewise,
from the last row up.  bf16 results are rounded once more, by 2^-8 of their value.
"""
import numpy as np
import pytest
import torch

from oracle import serving as ref

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}
U = 2.0 ** -23

pytestmark = pytest.mark.gpu


def _la():
    import linear_attention_02_gb300 as la
    return la


def _whole(B, N, C, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-4, 5, (B, N, C), generator=g).float()


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()


PACKED_SUMS = [
    (96, [2000]), (40, [1, 4, 124, 128, 3, 1000, 0, 257, 640]), (33, [4] * 60 + [900, 5]),
    (1001, [129, 0, 1500]), (1104, [700, 3, 900]), (2, [8] * 100),
]


@pytest.mark.parametrize("case", range(len(PACKED_SUMS)))
def test_packed_sums_reach_over_every_row_of_a_sequence(case):
    # decay 1: prefix sums forward, suffix sums backward, cut at the borders and nowhere else
    la = _la()
    C, lens = PACKED_SUMS[case]
    starts = _starts(lens)
    N = starts[-1] + 7
    X, G = _whole(1, N, C, case), _whole(1, N, C, 100 + case)
    S = len(lens)
    h0, dh = _whole(1, S, C, 200)[0], _whole(1, S, C, 300)[0]
    want, wX, wA = torch.zeros(N, C), torch.zeros(N, C), torch.zeros(N, C)
    wf, w0 = h0.clone(), dh.clone()
    for i, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        if a == b:
            continue
        h = h0[i] + X[0, a:b].cumsum(0)
        g = dh[i] + G[0, a:b].flip(0).cumsum(0).flip(0)
        want[a:b], wX[a:b], wf[i], w0[i] = h, g, h[-1], g[0]
        wA[a:b] = g * torch.cat([h0[i][None], h[:-1]])
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    A, Xd, Gd = torch.ones(1, N, C, device="cuda"), X.cuda(), G.cuda()
    for _ in range(3):
        out, dA, dX = (torch.zeros(1, N, C, device="cuda") for _ in range(3))
        _, hf = la.la_forward_gated_scan(A, Xd, seq_starts=st, h_init=h0.cuda(), out=out, return_state=True)
        _, _, d0 = la.la_backward_gated_scan(A, Xd, Gd, seq_starts=st, h_init=h0.cuda(), dh_final=dh.cuda(),
                                             return_dh_init=True, dA=dA, dX=dX)
        la.la_check_device_status()
        for got, exp in ((out[0], want), (hf, wf), (dX[0], wX), (d0, w0)):
            assert torch.equal(got.cpu(), exp)
        # dA: one rounding of the product of two exact whole numbers
        assert bool(((dA[0].cpu().double() - wA.double()).abs() <= 2.0 ** -24 * wA.double().abs()).all())


def _near(got, want, bound, dt="f32"):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= bound + HALF[dt] * (np.abs(want) + bound))
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {(np.abs(got - want) / np.maximum(bound, 1e-300)).max():.3g} bounds"


def _gates_near_one(B, N, C, dt, form, g):
    if form == "logit":
        return (torch.rand(B, N, C, generator=g) * 3.5 + 5.5).to(DT[dt])
    if dt == "bf16":  # the largest decay below 1 that bf16 has, one time in ten
        return torch.where(torch.rand(B, N, C, generator=g) < 0.1, 1 - 2.0 ** -8, 1.0).to(DT[dt])
    return 1 - (torch.rand(B, N, C, generator=g) * 9e-4 + 1e-4)


def _expect(p, form, seqs):
    """Wanted results and their bounds, sequence by sequence (batch row, first row, end)."""
    s, c = ref._gates(p["A"], form)
    r = (np.abs(p["A"]) + 8) * U * c if form == "logit" else np.zeros_like(s)  # error of a gate
    X, G = p["X"], p["G"]
    out, dA, dX, eo, eA, eX = (np.zeros(X.shape) for _ in range(6))
    fin, d0, ef, e0 = (np.zeros(p["h0"].shape) for _ in range(4))
    for i, (b, t0, t1) in enumerate(seqs):
        h, H, e = p["h0"][i], np.abs(p["h0"][i]), np.zeros_like(p["h0"][i])
        prev, sizes, errs = [], [], []
        for t in range(t0, t1):
            prev.append(h), sizes.append(H), errs.append(e)
            x = X[b, t]
            e = s[b, t] * e * (1 + U) + U * s[b, t] * H + r[b, t] * (H + np.abs(x))
            h, H = s[b, t] * h + c[b, t] * x, s[b, t] * H + np.abs(c[b, t] * x)
            e = e + U * H
            out[b, t], eo[b, t] = h, e
        fin[i], ef[i] = h, e
        y, Y, e = p["dh"][i], np.abs(p["dh"][i]), np.zeros_like(p["dh"][i])
        for t in range(t1 - 1, t0 - 1, -1):
            g, Q = G[b, t] + y, np.abs(G[b, t]) + Y
            e = e + U * Q
            dX[b, t] = c[b, t] * g
            eX[b, t] = c[b, t] * e + r[b, t] * Q + U * c[b, t] * Q
            ph, pH, pe = prev[t - t0], sizes[t - t0], errs[t - t0]
            if form == "logit":
                dA[b, t] = s[b, t] * c[b, t] * g * (ph - X[b, t])
                eA[b, t] = s[b, t] * ((c[b, t] * (e + 4 * U * Q) + r[b, t] * Q) * (pH + np.abs(X[b, t])) + c[b, t] * Q * pe)
            else:
                dA[b, t] = g * ph
                eA[b, t] = (e + U * Q) * pH + Q * pe
            e = s[b, t] * e * (1 + U) + 2 * U * s[b, t] * Q + r[b, t] * Q
            y, Y = s[b, t] * g, s[b, t] * Q
        d0[i], e0[i] = y, e
    return (out, fin, dA, dX, d0), (eo, ef, eA, eX, e0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["decay", "logit"])
@pytest.mark.parametrize("ckpt", [True, False])
@pytest.mark.parametrize("B,N,C,lens", [
    (1, 3000, 96, None), (2, 2600, 41, None), (1, 2700, 1104, None), (1, 2700, 1101, None), (3, 2570, 512, None),
    (1, 3010, 96, [2600, 0, 100, 300]), (1, 3000, 41, [2999]), (1, 2800, 1104, [7, 2700, 80]), (1, 2800, 1101, [2650, 129]),
])
def test_states_and_gradients_that_live_for_many_tiles(B, N, C, lens, ckpt, form, dt):
    la = _la()
    g = torch.Generator().manual_seed(N + C)
    S = B if lens is None else len(lens)
    x = {"A": _gates_near_one(B, N, C, dt, form, g), "X": torch.randn(B, N, C, generator=g).to(DT[dt]),
         "G": torch.randn(B, N, C, generator=g).to(DT[dt]), "h0": 20 * torch.randn(S, C, generator=g),
         "dh": 20 * torch.randn(S, C, generator=g)}
    d, p = {k: v.cuda() for k, v in x.items()}, {k: v.double().numpy() for k, v in x.items()}
    starts = None if lens is None else _starts(lens)
    st = None if lens is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    ck = torch.empty(la.la_gated_scan_ckpt_floats(B, N, C), device="cuda") if ckpt else None
    kw = dict(form=form, h_init=d["h0"], seq_starts=st)
    out, fin = la.la_forward_gated_scan(d["A"], d["X"], return_state=True, ckpt=ck, **kw)
    dA, dX, d0 = la.la_backward_gated_scan(d["A"], d["X"], d["G"], dh_final=d["dh"], return_dh_init=True, Ckpt=ck, **kw)
    la.la_check_device_status()
    want, bound = _expect(p, form, ref._sequences(B, N, starts))
    for got, w, e, t in zip((out, fin, dA, dX, d0), want, bound, (dt, "f32", dt, dt, "f32")):
        _near(got, w, e, t)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,lens", [(9000, 1104, None), (9000, 1101, None), (9000, 1104, [4000, 3, 4900]), (20000, 16, None)])
def test_results_do_not_depend_on_the_run(N, C, lens, dt):
    la = _la()
    g = torch.Generator(device="cuda").manual_seed(C)
    A = (torch.rand(1, N, C, generator=g, device="cuda") * 4 + 4).to(DT[dt])
    X, G = (torch.randn(1, N, C, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
    st = None if lens is None else torch.tensor(_starts(lens), dtype=torch.int32, device="cuda")

    def once():
        o, f = la.la_forward_gated_scan(A, X, form="logit", seq_starts=st, return_state=True)
        return (o, f) + la.la_backward_gated_scan(A, X, G, form="logit", seq_starts=st, return_dh_init=True)

    first = once()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


@pytest.mark.parametrize("backward,given", [(False, False), (False, True), (True, True), (True, False)])
def test_scratch_of_a_large_call_is_what_is_reported(backward, given):
    # tens of MB, against which the pool's rounding to 2 MB an allocation is small
    la = _la()
    B, N, C = 4, 65536, 1024
    A = torch.full((B, N, C), 0.5, dtype=torch.bfloat16, device="cuda")
    X, out, dA, dX = (torch.zeros_like(A) for _ in range(4))
    ck = torch.zeros(la.la_gated_scan_ckpt_floats(B, N, C), device="cuda") if given else None

    def call():
        if backward:
            la.la_backward_gated_scan(A, X, X, dA=dA, dX=dX, Ckpt=ck)
        else:
            la.la_forward_gated_scan(A, X, out=out, ckpt=ck)

    want = la.la_gated_scan_workspace_bytes(B, N, C, torch.bfloat16, backward=backward, ckpt_given=given)
    states = 4 * B * (N // 128) * C  # (A, B) of each tile, its end state unless checkpoints hold it; the states
    assert want == 16 + states * (2 if given and not backward else 4 if backward and not given else 3)
    call()
    torch.cuda.synchronize()
    la.la_scratch_peak_bytes(reset=True)
    call()
    torch.cuda.synchronize()
    slack = 2 * (2 << 20)
    assert slack < want / 4 and want <= la.la_scratch_peak_bytes() <= want + slack


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["decay", "logit"])
@pytest.mark.parametrize("B,N,C,lens", [(2, 700, 41, None), (1, 2700, 1104, None), (1, 384, 64, None),
                                        (1, 900, 96, [128, 100, 300, 372]), (1, 900, 33, [1, 0, 800])])
def test_checkpoints_are_the_states_at_every_128th_row(B, N, C, lens, form, dt):
    la = _la()
    g = torch.Generator().manual_seed(N)
    A, X = _gates_near_one(B, N, C, dt, form, g), torch.randn(B, N, C, generator=g).to(DT[dt])
    starts = None if lens is None else _starts(lens)
    S = B if lens is None else len(lens)
    h0, z = torch.randn(S, C, generator=g), np.zeros((S, C))
    p = {"A": A.double().numpy(), "X": X.double().numpy(), "G": np.zeros((B, N, C)), "h0": h0.double().numpy(), "dh": z}
    ck = torch.empty(la.la_gated_scan_ckpt_floats(B, N, C), device="cuda")
    la.la_forward_gated_scan(A.cuda(), X.cuda(), form=form, h_init=h0.cuda(), ckpt=ck,
                             seq_starts=None if lens is None else torch.tensor(starts, dtype=torch.int32, device="cuda"))
    want, bound = _expect(p, form, ref._sequences(B, N, starts))
    last = N if lens is None else starts[-1]
    rows = [t for t in range(127, N - 1, 128) if t < last]
    _near(ck.view(B, -(-N // 128), C)[:, :len(rows)], want[0][:, rows], bound[0][:, rows])
