"""Rows of a padded call that no sequence or request holds: defined in outputs that the
call allocates, left as they are in the caller's."""
import pytest
import torch

from linear_attention_02_gb300 import _native

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")


def _la():
    import linear_attention_02_gb300 as la
    return la


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _dirty(*shapes):
    """Leaves NaN in the memory that the allocator hands out next for these (shape, dtype)s."""
    torch.cuda.synchronize()
    ts = [torch.full(s, NAN, dtype=d, device="cuda") for s, d in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del ts


def test_refusals_of_the_padded_calls():
    lib, F, INV = _native.lib, 0x10000, _native.LA_ERR_INVALID_ARG
    msg = lambda: lib.la_last_error_message().decode()  # noqa: E731
    for fill in (-1, 2):
        assert lib.la_forward_gated_scan_padded(F, F, F, 1, 8, 4, 0, 0, F, 1, None, None, None, fill, None) == INV
        assert "fill" in msg()
    for fill in (-1, 4):
        assert lib.la_backward_gated_scan_padded(F, F, F, F, F, 1, 8, 4, 0, 0, F, 1, None, None, None, None, fill, None) == INV
        assert lib.la_paged_decode_step_padded(F, F, F, F, F, F, F, F, None, 2, 8, 2, 64, 4, 16, 3, 0, 0.0, 1, fill, None) == INV
        assert "fill" in msg()
    assert lib.la_paged_decode_step_padded(F, F, F, F, F, F, F, F, None, 2, 8, 2, 64, 4, 16, 3, 0, 0.0, 1, 2, None) == INV
    assert "lse is NULL" in msg()
    assert lib.la_forward_gated_scan_padded(None, F, F, 1, 8, 4, 0, 0, F, 0, None, None, None, 1, None) == INV
    assert lib.la_forward_gated_scan_padded(None, None, None, 1, 8, 4, 0, 0, F, 0, None, None, None, 0, None) == _native.LA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["decay", "logit"])
@pytest.mark.parametrize("N,C,starts", [(300, 64, [0, 100, 100, 250]), (300, 33, [0, 1]), (700, 1104, [0, 129, 513]),
                                        (700, 1101, [0, 600, 640]), (5, 8, [0, 0]), (140, 40, [3, 70]), (9, 16, [0])])
def test_scan_rows_of_no_sequence(N, C, starts, form, dt):
    la = _la()
    g = torch.Generator().manual_seed(N + C)
    A, X, G = ((torch.rand(1, N, C, generator=g) * 0.2 + 0.8).to(DT[dt]).cuda() for _ in range(3))
    lo, hi = starts[0], starts[-1]
    none = [r for r in range(N) if not lo <= r < hi]
    held = slice(lo, hi)
    for t in (A, X, G):
        t[0, none] = NAN
    st, S = _i32(starts), len(starts) - 1
    h0 = torch.randn(S, C, generator=g).cuda()
    kw = dict(form=form, seq_starts=st, h_init=h0)
    given = [torch.full((1, N, C), 7.25, dtype=DT[dt], device="cuda") for _ in range(3)]
    la.la_forward_gated_scan(A, X, out=given[0], **kw)
    la.la_backward_gated_scan(A, X, G, dA=given[1], dX=given[2], **kw)
    shape = ((1, N, C), DT[dt])
    _dirty(shape)
    out = la.la_forward_gated_scan(A, X, **kw)
    _dirty(shape)
    dA, dX = la.la_backward_gated_scan(A, X, G, **kw)
    for mine, theirs in zip((out, dA, dX), given):
        assert not bool(mine[0, none].any()) and bool((theirs[0, none] == 7.25).all())
        assert torch.equal(mine[0, held], theirs[0, held]) and bool(torch.isfinite(mine).all())
    # one of the two given: it keeps its rows, the other's are 0
    for i, name in enumerate(("dA", "dX")):
        buf = torch.full((1, N, C), 7.25, dtype=DT[dt], device="cuda")
        _dirty(shape)
        got = la.la_backward_gated_scan(A, X, G, **{name: buf}, **kw)
        assert torch.equal(got[i], given[1 + i]) and torch.equal(got[1 - i], (dA, dX)[1 - i])
    la.la_check_device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,lens", [(8, 2, 64, [-1, 40, -7, 0, 300, -1]), (20, 1, 128, [-1] * 5),
                                           (3, 3, 32, [(i * 37) % 90 - 20 for i in range(1500)]), (4, 4, 64, [9000, -1, 3])])
def test_decode_rows_without_a_request(Hq, Hkv, D, lens, dt):
    la = _la()
    g = torch.Generator().manual_seed(D)
    R, page = len(lens), 16
    need = [max(n, 0) // page + 1 for n in lens]
    W, P, at, table = max(need), sum(need), 0, []
    for n in need:
        table.append(list(range(at, at + n)) + [-1] * (W - n))
        at += n
    q, k, v = (torch.randn(R, h, D, generator=g).to(DT[dt]).cuda() for h in (Hq, Hkv, Hkv))
    K, V = (torch.randn(P, Hkv, page, D, generator=g).to(DT[dt]).cuda() for _ in range(2))
    none = [r for r, n in enumerate(lens) if n < 0]
    held = [r for r, n in enumerate(lens) if n >= 0]
    args = (q, k, v, K, V, _i32(table), _i32(lens))
    o, l = torch.full((R, Hq, D), 7.25, device="cuda"), torch.full((R, Hq), 7.25, device="cuda")
    got = la.la_paged_decode_step(*args, out=o, lse=l, return_lse=True)
    assert got[0] is o and got[1] is l
    _dirty(((R, Hq, D), torch.float32), ((R, Hq), torch.float32))
    out, lse = la.la_paged_decode_step(*args, return_lse=True)
    assert not bool(out[none].any()) and bool(torch.isneginf(lse[none]).all())
    assert bool((o[none] == 7.25).all()) and bool((l[none] == 7.25).all())
    assert torch.equal(out[held], o[held]) and torch.equal(lse[held], l[held])
    # each of the two given alone
    o2, l2 = torch.full_like(o, 7.25), torch.full_like(l, 7.25)
    _dirty(((R, Hq), torch.float32))
    assert torch.equal(la.la_paged_decode_step(*args, out=o2, return_lse=True)[1], lse) and torch.equal(o2, o)
    _dirty(((R, Hq, D), torch.float32))
    assert torch.equal(la.la_paged_decode_step(*args, lse=l2), out) and torch.equal(l2, l)
    la.la_check_device_status()


@pytest.mark.gpu
def test_lse_is_checked():
    la = _la()
    q = torch.zeros(1, 4, 64, device="cuda")
    K = torch.zeros(2, 4, 16, 64, device="cuda")
    with pytest.raises(ValueError, match="lse"):
        la.la_paged_decode_step(q, None, None, K, K, _i32([[0]]), _i32([3]), lse=torch.zeros(1, 5, device="cuda"))
