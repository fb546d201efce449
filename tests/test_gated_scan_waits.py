"""The gated scan's look-back gives up on a state that never comes, reports it, and ends."""
import pytest
import torch

from linear_attention_02_gb300 import _native
from oracle import serving as ref

pytestmark = pytest.mark.gpu


def _timed_out(la):
    with pytest.raises(la.LinAttnError) as e:
        la.la_check_device_status()
    assert e.value.status == _native.LA_ERR_TIMEOUT and "0x2" in str(e.value)
    la.la_check_device_status()  # the check cleared the word


@pytest.mark.parametrize("C", [64, 1104])  # the 16-tile window and the 4-tile one
@pytest.mark.parametrize("unit", [0, 5])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("given", [True, False])
def test_a_withheld_state_is_reported(C, unit, packed, given):
    # 40 tiles a chain; (test hook) tile `unit` publishes nothing, the tiles behind it give up
    # after 2000 polls.  The other batch row's channels do not wait for it.
    import linear_attention_02_gb300 as la
    la.la_check_device_status()
    B, N = (1, 10240) if packed else (2, 5120)
    g = torch.Generator().manual_seed(C)
    A = (torch.rand(B, N, C, generator=g) * 0.15 + 0.85)
    X, G = (torch.randn(B, N, C, generator=g) for _ in range(2))
    Ad, Xd, Gd = A.cuda(), X.cuda(), G.cuda()
    kw = {"seq_starts": torch.tensor([0, 5000, 10240], dtype=torch.int32, device="cuda")} if packed else {}
    ck = torch.empty(la.la_gated_scan_ckpt_floats(B, N, C), device="cuda")
    good = la.la_forward_gated_scan(Ad, Xd, ckpt=ck, **kw)
    goodA, goodX = la.la_backward_gated_scan(Ad, Xd, Gd, Ckpt=ck, **kw)
    la.la_check_device_status()
    want = ref.gated_scan_forward(A[:, :300], X[:, :300])[0]
    assert float((good[:, :300].cpu().double() - torch.from_numpy(want)).abs().max()) <= 1.5e-5 * abs(want).max()
    spare = torch.empty_like(ck)
    assert _native.lib.la_debug_withhold_publication(unit, 2000) == _native.LA_OK
    out = la.la_forward_gated_scan(Ad, Xd, ckpt=spare if given else None, **kw)
    _timed_out(la)
    if not packed:
        assert torch.equal(out[1], good[1])
    assert _native.lib.la_debug_withhold_publication(unit, 2000) == _native.LA_OK
    dA, dX = la.la_backward_gated_scan(Ad, Xd, Gd, Ckpt=ck if given else None, **kw)
    _timed_out(la)
    if not packed:
        assert torch.equal(dA[1], goodA[1]) and torch.equal(dX[1], goodX[1])
    # the device computes on as before
    assert torch.equal(la.la_forward_gated_scan(Ad, Xd, **kw), good)
    dA, dX = la.la_backward_gated_scan(Ad, Xd, Gd, **kw)
    assert torch.equal(dA, goodA) and torch.equal(dX, goodX)
    la.la_check_device_status()
