"""GPU tests of the gated scan over many tiles: states and gradients that live for
thousands of rows, on both sides of the look-back window's choice.

Where the decays are 1 and the values small whole numbers, every sum is a whole
number below 2^24 and exact in fp32 in any order: those tests ask for equality.
"""
import numpy as np
import pytest
import torch

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
