"""The bf16 prefill's waits give up on queries that never come, report it, and end."""
import pytest
import torch

from linear_attention_02_gb300 import _native

pytestmark = pytest.mark.gpu


def _timed_out(la):
    with pytest.raises(la.LinAttnError) as e:
        la.la_check_device_status()
    assert e.value.status == _native.LA_ERR_TIMEOUT and "0x1" in str(e.value)
    la.la_check_device_status()  # the check cleared the word


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (8, 2, 128), (3, 1, 32), (6, 2, 128)])  # even and odd rings, both queries' ways
@pytest.mark.parametrize("page", [4, 16])                                                   # both pages' ways
@pytest.mark.parametrize("R,cached,new", [(1500, 0, 100), (40, 6000, 20)])                  # whole tiles, cut ones
@pytest.mark.parametrize("unit", [0, 7])
def test_queries_that_do_not_come(Hq, Hkv, D, page, R, cached, new, unit):
    # (test hook) block `unit` gets no queries: its wait for them gives up after 20000 polls, and all others with it
    import linear_attention_02_gb300 as la
    la.la_check_device_status()
    W = -(-(cached + new) // page)
    g = torch.Generator(device="cuda").manual_seed(D)
    q, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16()
               for s in ((R * new, Hq, D), (R * W, Hkv, page, D), (R * W, Hkv, page, D)))
    table = torch.randperm(R * W, generator=g, device="cuda").to(torch.int32).view(R, W)
    lens = torch.full((R,), cached, dtype=torch.int32, device="cuda")
    starts = torch.arange(R + 1, device="cuda", dtype=torch.int32) * new
    run = lambda: la.la_paged_prefill(q, K, V, table, lens, starts)  # noqa: E731
    good = run()
    la.la_check_device_status()
    assert _native.lib.la_debug_withhold_publication(unit, 20000) == _native.LA_OK
    out = run()
    _timed_out(la)
    if R > 100:  # tiles of the last requests are other blocks'
        assert torch.equal(out[len(out) // 2:], good[len(out) // 2:])
    # the device computes on as before
    for _ in range(3):
        assert torch.equal(run(), good)
    la.la_check_device_status()
