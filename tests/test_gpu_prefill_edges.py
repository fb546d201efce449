"""Edges of the prefill over the paged cache: rows of no request, starts that go back, values that are not
finite in cut tiles and in segments that follow one another, the largest finite values, a pool without pages.
Tolerances are test_gpu_paged_prefill.py's."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import serving as ref
from test_gpu_paged_prefill import DT, HALF, _case, _check, _i32, _la, _score_error

pytestmark = pytest.mark.gpu


def _filled(d, table, cached, starts, fill=3):
    """(out, lse) of the C call with `fill`, on outputs that hold 9.5."""
    from linear_attention_02_gb300 import _native
    (T, Hq, D), (P, Hkv, page, _) = d["q"].shape, d["K"].shape
    R, W = table.shape
    out, lse = torch.full_like(d["q"], 9.5), torch.full((T, Hq), 9.5, device="cuda")
    dt = _native.LA_DTYPE_BF16 if out.dtype == torch.bfloat16 else _native.LA_DTYPE_F32
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert _native.lib.la_paged_prefill(d["q"].data_ptr(), d["K"].data_ptr(), d["V"].data_ptr(), table.data_ptr(),
                                        cached.data_ptr(), starts.data_ptr(), out.data_ptr(), lse.data_ptr(), T, R, Hq,
                                        Hkv, D, P, page, W, 0, 0.0, dt, fill, s) == _native.LA_OK
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("before,tail", [(1, 0), (5, 6), (200, 1)])
def test_rows_before_the_first_request(before, tail, dt):
    cached, new = [20, -1, 7], [9, 3, 40]
    x, table, starts = _case(4, 2, 64, 16, cached, new, dt, tail=before + tail)
    starts = [before + s for s in starts]
    out, lse = _check(x, table, cached, starts, 64, dt)
    d = {n: t.cuda() for n, t in x.items()}
    own = torch.zeros(len(x["q"]), dtype=torch.bool)
    own[starts[0]:starts[1]], own[starts[2]:starts[3]] = True, True
    o2, l2 = _filled(d, _i32(table), _i32(cached), _i32(starts))
    assert torch.equal(o2[own], out[own]) and torch.equal(l2[own], lse[own])
    assert bool((o2[~own] == 0).all()) and bool(torch.isneginf(l2[~own]).all())
    o1, l1 = _filled(d, _i32(table), _i32(cached), _i32(starts), fill=1)
    assert torch.equal(o1, o2) and bool((l1[~own] == 9.5).all())
    _la().la_check_device_status()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R", [3, 40, 5000])
@pytest.mark.parametrize("length", [0, -1])
def test_starts_that_go_back_leave_no_row_undefined(length, R, dt):
    # back and forth over all rows: reported, no request done, and every row cleared once, however many requests
    la = _la()
    T = 59
    x, _, _ = _case(4, 2, 64, 16, [0], [T], dt)
    d = {n: t.cuda() for n, t in x.items()}
    table = torch.zeros((R, 8), dtype=torch.int32, device="cuda")
    starts = ([0, T] * R)[:R] + [3]  # the last row that a request names is not the last of all
    out, lse = _filled(d, table, _i32([length] * R), _i32(starts))
    with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
        la.la_check_device_status()
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    out, lse = _filled(d, table, _i32([length] * R), _i32(starts), fill=0)
    assert bool((out == 9.5).all()) and bool((lse == 9.5).all())
    with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
        la.la_check_device_status()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("far", [-40.0, -math.inf])
@pytest.mark.parametrize("early", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,new", [(1, 1, 64, 1), (8, 1, 128, 3), (2, 2, 32, 40)])
def test_an_infinite_value_of_weight_0_in_a_cut_tile(Hq, Hkv, D, new, early, far, dt):
    # One half's keys score so far below the others that their weights are 0 in fp32: by the definition
    # and in an uncut tile 0 times an infinity is NaN, and so it is where another block had that half.
    la = _la()
    page, cached, at, col = 16, 6000, 100 if early else 5000, 5
    x, table, starts = _case(Hq, Hkv, D, page, [cached], [new], dt)
    x["q"][:, :, 0] = 40.0
    n = cached + new
    pages, offs = np.array(table[0])[np.arange(n) // page], np.arange(n) % page
    low = torch.tensor((np.arange(n) < 3000) == early)
    k0 = torch.where(low, torch.tensor(far), torch.tensor(40.0)).to(DT[dt])
    x["K"][pages, :, offs, 0] = k0[:, None]
    d = {m: t.cuda() for m, t in x.items()}
    args = (_i32(table), _i32([cached]), _i32(starts))
    want, wl = la.la_paged_prefill(d["q"], d["K"], d["V"], *args, return_lse=True)
    assert bool(torch.isfinite(want).all())
    rest = [c for c in range(D) if c != col]
    for what in (math.inf, -math.inf, math.nan):
        V = d["V"].clone()
        V[table[0][at // page], :, at % page, col] = what
        got, gl = la.la_paged_prefill(d["q"], d["K"], V, *args, return_lse=True)
        assert not bool(torch.isfinite(got[..., col]).any()), what
        assert torch.equal(got[..., rest], want[..., rest]) and torch.equal(gl, wl)
    la.la_check_device_status()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_values_replaced_elsewhere_do_not_change_an_infinity_that_all_rows_see(dt):
    # many requests a block; position 0 is seen by every row, position 11 by the later ones only
    la = _la()
    R, new, H, D, page = 1500, 150, 2, 64, 16
    W = -(-new // page)
    g = torch.Generator().manual_seed(7)
    q, K, V = (torch.randn(s, generator=g).to(DT[dt]).cuda() for s in ((R * new, H, D), (R * W, H, page, D), (R * W, H, page, D)))
    table = torch.randperm(R * W, generator=g).to(torch.int32).cuda().view(R, W)
    lens, starts = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.arange(R + 1, device="cuda", dtype=torch.int32) * new
    run = lambda: la.la_paged_prefill(q, K, V, table, lens, starts).view(R, new, H, D)  # noqa: E731
    V[table[:, 0].long(), :, 0, 3] = math.inf
    want = run()
    assert not bool(torch.isfinite(want[..., 3]).any())
    hit = torch.arange(0, R, 7, device="cuda")
    V[table[hit, 0].long(), :, 11, 9] = math.nan
    touched = torch.zeros((R, new, H, D), dtype=torch.bool, device="cuda")
    touched[hit, 11:, :, 9] = True
    bits = lambda t: t[~touched].view(torch.int16 if dt == "bf16" else torch.int32)  # noqa: E731  NaN equals NaN here
    for _ in range(3):
        got = run()
        assert torch.equal(bits(got), bits(want))
        assert bool(torch.isnan(got[touched]).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_the_largest_finite_values(D, dt):
    cached, new = [3, 0], [40, 200]
    x, table, starts = _case(4, 2, D, 16, cached, new, dt)
    top = torch.finfo(DT[dt]).max
    g = torch.Generator().manual_seed(D)
    near = torch.rand(x["V"].shape, generator=g, dtype=torch.float64) * 2.0 ** -11  # on both sides of 2^-12 below the largest
    sign = torch.where(torch.rand(x["V"].shape, generator=g) < 0.5, -1.0, 1.0)
    y = dict(x, V=((1 - near) * top * sign).to(DT[dt]))
    assert bool(torch.isfinite(y["V"]).all()) and bool((y["V"].abs() == top).any())
    _check(y, table, cached, starts, D, dt, window=1)  # each row sees its own value only
    # one such value beside ordinary ones, in whole and in partly seen tiles: no sum passes it
    y = dict(x, V=x["V"].clone())
    for r in range(2):
        y["V"][table[r][0], :, 0] = (sign * top)[table[r][0], :, 0].to(DT[dt])
    y["K"] = x["K"].clone()
    for r in range(2):
        y["K"][table[r][0], :, 0] = 0  # its score is 0: a weight of at most the largest
    _check(y, table, cached, starts, D, dt)
    _la().la_check_device_status()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("page", [4, 16])
def test_a_pool_without_pages(page, dt):
    la = _la()
    x, _, _ = _case(4, 2, 64, page, [20, 0], [9, 150], dt)
    q, K = x["q"].cuda(), torch.empty((0, 2, page, 64), device="cuda", dtype=DT[dt])
    table = torch.zeros((2, 64), dtype=torch.int32, device="cuda")
    out, lse = la.la_paged_prefill(q, K, K.clone(), table, _i32([20, 0]), _i32([0, 9, 159]), return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
        la.la_check_device_status()


@pytest.mark.parametrize("D", [32, 64, 128])
def test_fp32_scores_do_not_lose_bits_with_the_heads_length(D):
    # Rows that see one key, so lse is the score, a sum of D products of one sign.  Parts of 32 products are 12 sums on the matrix
    # unit, each cut off by half a unit of the last place (2^-23) in the mean, of i / 12 of the part at the i-th: 3.25 x 2^-23.
    # The operands' terms are off by 2^-21 of a product at most, by 2^-23 in the mean, and what follows rounds
    # three times, by 2^-24 each.  (In one chain of 48 sums: 12.25 x 2^-23.)
    la = _la()
    T = 700
    g = torch.Generator().manual_seed(D)
    q, K = (torch.rand(s, generator=g) * 0.2 + 0.9 for s in ((T, 2, D), (T, 1, 8, D)))
    i32 = lambda n: torch.arange(n, dtype=torch.int32, device="cuda")  # noqa: E731
    _, lse = la.la_paged_prefill(q.cuda(), K.cuda(), K.cuda(), i32(T).view(T, 1), 0 * i32(T), i32(T + 1), return_lse=True)
    want = torch.einsum("thd,td->th", q.double(), K[:, 0, 0].double()) / math.sqrt(D)
    off = float(((lse.cpu().double() - want) / want).abs().mean())
    assert off <= (3.25 + 1 + 1.5) * 2.0 ** -23
