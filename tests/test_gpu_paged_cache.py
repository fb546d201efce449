"""GPU parity of the paged key-value cache (page map, append, decode step)
against its fp64 plain form, through the C ABI.

The map and the append are exact.  The decode step's tolerance: a score is a
sum of D fp32 products, off by at most (D + 4) 2^-24 of scale sum |q k| (the 4:
scaling and base change); a weight is off by that much relative to itself, twice
(in the sum above and below the fraction), and every weight, product and sum of
the output takes a few roundings of 2^-24 more, with the longest fp32 sums here
a few hundred terms that grow by blocks: 64 x 2^-23 in all, of the largest value.
"""
import math

import numpy as np
import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _la():
    import linear_attention_02_gb300 as la
    return la


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- page map

def _map_case(R, page, max_cached, max_new, spare, seed, W_more=2):
    r = np.random.RandomState(seed)
    cached, new = r.randint(0, max_cached + 1, R), r.randint(0, max_new + 1, R)
    W = -(-(max_cached + max_new) // page) + W_more
    need = -(-(cached + new) // page)
    P = int(need.sum()) + spare
    order = r.permutation(P)
    table, at = np.full((R, W), -1), 0
    for i in range(R):
        n = -(-int(cached[i]) // page)
        table[i, :n] = order[at:at + n]
        at += n
    return cached.tolist(), new.tolist(), order[at:].tolist(), table, P


def _run_map(cached, new, free, table, page, P, T):
    la = _la()
    t, slots = _i32(table), torch.full((T,), 123, dtype=torch.int32, device="cuda")
    _, starts, counts = la.la_page_map(_i32(cached), _i32(new), _i32(free), t, page, P, slots)
    return [x.cpu().numpy() for x in (t, slots, starts, counts)]


@pytest.mark.parametrize("R,page,mc,mn,T_more", [
    (1, 1, 5, 3, 0), (1, 16, 0, 1, 3), (3, 4, 9, 6, 2), (64, 16, 4095, 1, 0), (33, 8, 100, 300, 500),
    (300, 64, 50, 40, 7), (1500, 16, 40, 3, 11), (5000, 2, 3, 2, 0), (2, 1024, 5000, 9000, 1), (17, 32, 0, 0, 4)])
def test_page_map(R, page, mc, mn, T_more):
    la = _la()
    cached, new, free, table, P = _map_case(R, page, mc, mn, 3, R + page)
    T = sum(new) + T_more
    want = ref.page_map(cached, new, free, table, page, P, T)
    got = _run_map(cached, new, free, table, page, P, T)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)
    la.la_check_device_status()


def test_page_map_reports_what_does_not_fit():
    la = _la()
    cases = [
        dict(cached=[0, 3], new=[9, 5], free=[1, 2], table=[[-1] * 4, [0, -1, -1, -1]], page=4, P=5, T=20),  # no page left
        dict(cached=[0], new=[9], free=[1, 2, 3], table=[[-1, -1]], page=4, P=5, T=9),       # past the table row
        dict(cached=[99], new=[2], free=[1], table=[[0, 1]], page=4, P=5, T=2),              # held length past it too
        dict(cached=[-3, 2], new=[2, -7], free=[1], table=[[-1, -1], [2, -1]], page=4, P=5, T=3),
        dict(cached=[2], new=[3], free=[1], table=[[-1, -1]], page=4, P=5, T=3),             # the page held is none
        dict(cached=[2], new=[3], free=[7], table=[[0, -1]], page=4, P=5, T=3),              # free page out of range
        dict(cached=[0, 0], new=[4, 4], free=[1, 2], table=[[-1], [-1]], page=4, P=5, T=6),  # slot map too short
    ]
    for c in cases:
        want = ref.page_map(c["cached"], c["new"], c["free"], c["table"], c["page"], c["P"], c["T"])
        assert want[4]
        got = _run_map(c["cached"], c["new"], c["free"], c["table"], c["page"], c["P"], c["T"])
        for g, w in zip(got, want):
            np.testing.assert_array_equal(g, w)
        with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
            la.la_check_device_status()
        la.la_check_device_status()  # cleared


@pytest.mark.parametrize("R", [7, 4500])
def test_page_map_of_a_padded_batch(R):
    # rows without a request (negative cached length, nothing new) change nothing and are not reported
    la = _la()
    cached, new, free, table, P = _map_case(R, 4, 9, 3, 2, R)
    for r in range(0, R, 3):
        cached[r], new[r] = -1 - r, 0
    T = sum(new) + 5
    want = ref.page_map(cached, new, free, table, 4, P, T)
    assert not want[4]
    for g, w in zip(_run_map(cached, new, free, table, 4, P, T), want):
        np.testing.assert_array_equal(g, w)
    la.la_check_device_status()


def test_page_map_without_requests():
    la = _la()
    slots = torch.full((5,), 3, dtype=torch.int32, device="cuda")
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    _, starts, counts = la.la_page_map(e, e, e, e.view(0, 4), 16, 0, slots)
    assert slots.tolist() == [-1] * 5 and starts.tolist() == [0] and counts.tolist() == [0, 0]


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 32, 1), (5, 3, 64, 4), (300, 2, 128, 16), (77, 8, 64, 64), (9, 1, 32, 1024)])
def test_append(T, Hkv, D, page, dt):
    la = _la()
    g = torch.Generator().manual_seed(T)
    P = -(-T // page) + 2
    k, v = (torch.randn(T, Hkv, D, generator=g).to(DT[dt]) for _ in range(2))
    K, V = (torch.randn(P, Hkv, page, D, generator=g).to(DT[dt]) for _ in range(2))
    slots = torch.randperm(P * page, generator=g)[:T].to(torch.int32)
    slots[::5] = -1
    wK, wV = ref.paged_append(k, v, K, V, slots.tolist())
    Kg, Vg = K.cuda(), V.cuda()
    la.la_paged_append(k.cuda(), v.cuda(), Kg, Vg, slots.cuda())
    la.la_check_device_status()
    assert np.array_equal(Kg.double().cpu().numpy(), wK) and np.array_equal(Vg.double().cpu().numpy(), wV)


def test_append_reports_bad_slots():
    la = _la()
    k = torch.ones(3, 1, 32, device="cuda")
    K, V = torch.zeros(2, 1, 4, 32, device="cuda"), torch.zeros(2, 1, 4, 32, device="cuda")
    la.la_paged_append(k, k, K, V, _i32([8, -2, 7]))
    with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
        la.la_check_device_status()
    assert float(K.sum()) == 32 and bool((K[1, 0, 3] == 1).all())


# ---------------------------------------------------------------- decode

def _decode_case(R, Hq, Hkv, D, page, lens, append, dt, seed=1, spare=2):
    g = torch.Generator().manual_seed(seed)
    need = [-(-(max(n, 0) + append) // page) for n in lens]
    P, W = sum(need) + spare, max(need + [1]) + 1
    order, table, at = torch.randperm(P, generator=g).tolist(), [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (W - n))
        at += n
    x = {n: torch.randn(s, generator=g).to(DT[dt]) for n, s in
         (("q", (R, Hq, D)), ("k", (R, Hkv, D)), ("v", (R, Hkv, D)), ("K", (P, Hkv, page, D)), ("V", (P, Hkv, page, D)))}
    return x, table


def _bounds(x, D, scale=None):
    big = max(float(x["K"].abs().max()), float(x["k"].abs().max()))
    kn = max(float(x["K"].float().norm(dim=-1).max()), float(x["k"].float().norm(dim=-1).max()))
    qn = float(x["q"].float().norm(dim=-1).max())
    s = (1 / math.sqrt(D) if scale is None else abs(scale)) * min(qn * kn, D * big * float(x["q"].abs().max()))
    vb = max(float(x["V"].abs().max()), float(x["v"].abs().max()))
    err = (D + 4) * 2.0 ** -24 * s
    return (2 * err + 64 * 2.0 ** -23) * vb, err + 64 * 2.0 ** -23 * 8


def _check_decode(x, table, lens, D, append=True, window=0, scale=None, pad=()):
    la = _la()
    d = {n: t.cuda() for n, t in x.items()}
    out = torch.full(x["q"].shape, 9.5, device="cuda")
    k, v = (d["k"], d["v"]) if append else (None, None)
    _, lse = la.la_paged_decode_step(d["q"], k, v, d["K"], d["V"], _i32(table), _i32(lens), window=window, scale=scale,
                                     out=out, return_lse=True)
    la.la_check_device_status()
    wo, wl = ref.paged_decode(x["q"], x["k"] if append else None, x["v"] if append else None, x["K"], x["V"], table,
                              lens, window, scale)
    own = np.array([n >= 0 for n in lens])
    to, tl = _bounds(x, D, scale)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(got[~own] == 9.5)
    assert np.abs(got[own] - wo[own]).max(initial=0) <= to
    fin = np.isfinite(wl)
    assert np.array_equal(np.isneginf(gl[own]), np.isneginf(wl[own]))
    assert np.abs(gl[own & True][fin[own]] - wl[own][fin[own]]).max(initial=0) <= tl
    # the new rows are in the cache and nothing else has changed
    wK, wV = x["K"].clone(), x["V"].clone()
    if append:
        page = x["K"].shape[2]
        for r, n in enumerate(lens):
            if n >= 0:
                wK[table[r][n // page], :, n % page], wV[table[r][n // page], :, n % page] = x["k"][r], x["v"][r]
    assert torch.equal(d["K"].cpu(), wK) and torch.equal(d["V"].cpu(), wV)


SHAPES = [  # Hq, Hkv, D, page, lens
    (1, 1, 32, 1, [0, 1, 2, 5]), (4, 4, 64, 16, [0, 15, 16, 17, 300]), (8, 2, 128, 8, [7, 8, 9, 1000]),
    (6, 2, 64, 32, [31, 32, 33, 64, 65]), (16, 1, 128, 16, [100, 511]), (20, 1, 64, 16, [77, 200]),
    (40, 2, 32, 64, [63, 128]), (12, 4, 32, 4, [3, 50, 333]), (5, 5, 128, 256, [255, 256, 600]),
    (14, 2, 64, 1024, [1023, 1024, 1500]), (33, 1, 128, 2, [40])]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("append", [True, False])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_paged_decode(case, append, dt):
    Hq, Hkv, D, page, lens = SHAPES[case]
    x, table = _decode_case(len(lens), Hq, Hkv, D, page, lens, append, dt, seed=case)
    _check_decode(x, table, lens, D, append)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 5000])
def test_paged_decode_window(window, dt):
    lens = [0, 1, 15, 16, 47, 99, 100, 101, 700]
    for append in (True, False):
        x, table = _decode_case(len(lens), 4, 2, 64, 16, lens, append, dt, seed=window)
        _check_decode(x, table, lens, 64, append, window=window)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 8), (128, 16, 2), (32, 4, 1)])
def test_paged_decode_long(D, Hq, Hkv, dt):
    # one long context beside short ones: the split over the length and its join
    lens = [20000, 3, 0, 4097, -1, 129]
    x, table = _decode_case(len(lens), Hq, Hkv, D, 16, lens, True, dt, seed=D)
    _check_decode(x, table, lens, D)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_paged_decode_padded_rows_and_scale(dt):
    lens = [-1, 40, -5, 0, -1]
    x, table = _decode_case(len(lens), 4, 2, 64, 16, lens, True, dt, seed=3)
    _check_decode(x, table, lens, 64)
    _check_decode(x, table, lens, 64, scale=0.02)
    _check_decode(x, table, lens, 64, scale=-0.3)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_paged_decode_many_requests(dt):
    lens = [(i * 37) % 90 for i in range(1100)]
    x, table = _decode_case(len(lens), 4, 2, 32, 8, lens, True, dt, seed=4)
    _check_decode(x, table, lens, 32)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_paged_decode_large_scores(dt):
    # scores of several hundred: the running maximum keeps every exponential in range
    lens = [200, 1000]
    x, table = _decode_case(2, 4, 2, 64, 16, lens, True, dt, seed=5)
    x["q"] = x["q"] * 8
    x["K"] = x["K"] * 8
    _check_decode(x, table, lens, 64)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_paged_decode_ignores_what_is_not_the_requests(dt):
    # NaN behind a request's length, on pages of nobody and in unused table entries changes nothing
    la = _la()
    lens = [5, 30, 0, 64]
    x, table = _decode_case(4, 8, 2, 64, 16, lens, True, dt, seed=6)
    d = {n: t.cuda() for n, t in x.items()}
    out = la.la_paged_decode_step(d["q"], d["k"], d["v"], d["K"].clone(), d["V"].clone(), _i32(table), _i32(lens))
    K, V = torch.full_like(d["K"], float("nan")), torch.full_like(d["V"], float("inf"))
    for r, n in enumerate(lens):
        for p in range(n):
            K[table[r][p // 16], :, p % 16] = d["K"][table[r][p // 16], :, p % 16]
            V[table[r][p // 16], :, p % 16] = d["V"][table[r][p // 16], :, p % 16]
    got = la.la_paged_decode_step(d["q"], d["k"], d["v"], K, V, _i32(table), _i32(lens))
    assert torch.equal(got, out)


def test_paged_decode_infinite_scores():
    # keys of -infinity scores count nothing; with all of them the row is NaN, as in the formula
    la = _la()
    x, table = _decode_case(2, 2, 2, 32, 16, [40, 40], False, "f32", seed=7)
    x["q"][:] = x["q"].abs() + 0.1
    x["K"][:] = x["K"].abs()
    for p in range(35):
        x["K"][table[0][p // 16], :, p % 16] = float("-inf")
    d = {n: t.cuda() for n, t in x.items()}
    out, lse = la.la_paged_decode_step(d["q"], None, None, d["K"], d["V"], _i32(table), _i32([40, 40]), return_lse=True)
    K5 = torch.stack([x["K"][table[0][p // 16], :, p % 16] for p in range(35, 40)], 1).double()
    V5 = torch.stack([x["V"][table[0][p // 16], :, p % 16] for p in range(35, 40)], 1).double()
    s = torch.einsum("hd,hnd->hn", x["q"][0].double(), K5) / math.sqrt(32)
    want = torch.einsum("hn,hnd->hd", torch.softmax(s, 1), V5)
    assert float((out[0].cpu().double() - want).abs().max()) <= 1e-4
    assert float((lse[0].cpu().double() - torch.logsumexp(s, 1)).abs().max()) <= 1e-4


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_paged_decode_reports_bad_pages_and_lengths(dt):
    # pages outside the pool and lengths past the table: skipped and reported
    la = _la()
    lens = [40, 40, 30]
    x, table = _decode_case(3, 4, 2, 64, 16, lens, True, dt, seed=8)
    table[0][1] = x["K"].shape[0] + 5
    table[1][0] = -7
    wo, _ = ref.paged_decode(x["q"], x["k"], x["v"], x["K"], x["V"], table, lens)
    d = {n: t.cuda() for n, t in x.items()}
    out = la.la_paged_decode_step(d["q"], d["k"], d["v"], d["K"], d["V"], _i32(table), _i32(lens))
    with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
        la.la_check_device_status()
    assert np.abs(out.double().cpu().numpy() - wo).max() <= _bounds(x, 64)[0]
    # a length past the table: its row cannot be appended, the others are right
    lens2 = [len(table[0]) * 16, 30, 2 ** 31 - 1]
    table[0][1], table[1][0] = table[2][0], table[2][0]
    tb = [[max(i, 0) for i in t] for t in table]
    K0 = d["K"].clone()
    la.la_paged_decode_step(d["q"], d["k"], d["v"], d["K"], d["V"], _i32(tb), _i32(lens2))
    with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
        la.la_check_device_status()
    K0[tb[1][1], :, 14] = d["k"][1]
    assert torch.equal(d["K"], K0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_paged_decode_results_do_not_depend_on_the_run(dt):
    la = _la()
    lens = [5000, 17, 900, 3000]
    x, table = _decode_case(4, 8, 2, 64, 16, lens, True, dt, seed=9)
    d = {n: t.cuda() for n, t in x.items()}
    args = (d["q"], d["k"], d["v"], d["K"], d["V"], _i32(table), _i32(lens))
    first = la.la_paged_decode_step(*args)
    for _ in range(5):
        assert torch.equal(la.la_paged_decode_step(*args), first)


def test_paged_decode_equals_the_contiguous_step():
    # the same cache as pages and as rows: la_softmax_decode_step's result
    la = _la()
    R, H, D, page, T = 3, 4, 64, 16, 200
    g = torch.Generator().manual_seed(10)
    Kc, Vc = (torch.randn(R, H, 208, D, generator=g).bfloat16().cuda() for _ in range(2))
    q, k, v = (torch.randn(R, H, D, generator=g).bfloat16().cuda() for _ in range(3))
    table = torch.arange(R * 13, dtype=torch.int32, device="cuda").view(R, 13)
    K = Kc.view(R, H, 13, page, D).transpose(1, 2).reshape(R * 13, H, page, D).contiguous()
    V = Vc.view(R, H, 13, page, D).transpose(1, 2).reshape(R * 13, H, page, D).contiguous()
    got = la.la_paged_decode_step(q, k, v, K, V, table, _i32([T] * R))
    want = la.la_softmax_decode_step(q, k, v, Kc, Vc, T)
    assert float((got - want).abs().max()) <= 1e-4
    back = K.view(R, 13, H, page, D).transpose(1, 2).reshape(R, H, 208, D)
    assert torch.equal(back, Kc)


def test_paged_decode_joins_parts_by_lse():
    # outputs over two parts of a context, joined by their logs of sums, are the whole's
    la = _la()
    x, table = _decode_case(1, 4, 2, 64, 16, [320], False, "f32", seed=11)
    d = {n: t.cuda() for n, t in x.items()}
    whole, lw = la.la_paged_decode_step(d["q"], None, None, d["K"], d["V"], _i32(table), _i32([320]), return_lse=True)
    o1, l1 = la.la_paged_decode_step(d["q"], None, None, d["K"], d["V"], _i32(table), _i32([192]), return_lse=True)
    o2, l2 = la.la_paged_decode_step(d["q"], None, None, d["K"], d["V"], _i32([table[0][12:]]), _i32([128]), return_lse=True)
    l = torch.logaddexp(l1, l2)
    o = o1 * (l1 - l).exp()[..., None] + o2 * (l2 - l).exp()[..., None]
    to, tl = _bounds(x, 64)
    assert float((o - whole).abs().max()) <= 4 * to and float((l - lw).abs().max()) <= 4 * tl


def test_paged_decode_streams_and_graphs():
    la = _la()
    lens = [3000, 5, 64, 700]
    x, table = _decode_case(4, 8, 2, 64, 16, lens, False, "bf16", seed=12)
    d = {n: t.cuda() for n, t in x.items()}
    tb, ln = _i32(table), _i32(lens)
    args = (d["q"], None, None, d["K"], d["V"], tb, ln)
    want = la.la_paged_decode_step(*args)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(la.la_paged_decode_step(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)
    o = [torch.empty_like(want) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, t in zip(graphs, o):
        with torch.cuda.graph(g):
            la.la_paged_decode_step(*args, out=t)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o[0], want) and torch.equal(o[1], want)
    # the replay follows the lengths and tables as they are then
    ln.copy_(_i32([64, 3, 17, 900 - 200]))
    short = la.la_paged_decode_step(*args)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o[0], short) and torch.equal(o[1], short)


def test_paged_decode_offsets_past_32_bits():
    # a pool of 2.3e9 elements a side; a request on its last pages
    la = _la()
    P, Hkv, page, D = 280_000, 2, 64, 64
    K = torch.zeros(P, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    g = torch.Generator().manual_seed(13)
    n, pages = 150, [P - 1, P - 3, P - 2]
    k, v = (torch.randn(n, Hkv, D, generator=g).bfloat16() for _ in range(2))
    slots = torch.tensor([pages[p // page] * page + p % page for p in range(n)], dtype=torch.int32)
    la.la_paged_append(k.cuda(), v.cuda(), K, V, slots.cuda())
    q = torch.randn(1, 4, D, generator=g).bfloat16()
    out = la.la_paged_decode_step(q.cuda(), None, None, K, V, _i32([pages]), _i32([n]))
    la.la_check_device_status()
    Ks, Vs = k.double().transpose(0, 1), v.double().transpose(0, 1)
    s = torch.einsum("hgd,hnd->hgn", q[0].double().view(2, 2, D), Ks) / 8
    want = torch.einsum("hgn,hnd->hgd", torch.softmax(s, 2), Vs).reshape(4, D)
    assert float((out[0].cpu().double() - want).abs().max()) <= 1e-4


def test_paged_wrapper_refusals():
    la = _la()
    K = torch.zeros(4, 2, 16, 64, device="cuda")
    q, k = torch.zeros(1, 4, 64, device="cuda"), torch.zeros(1, 2, 64, device="cuda")
    tb, ln = _i32([[0, 1]]), _i32([3])
    for bad, match in (((q, k, None, K, K, tb, ln), "neither"), ((q, k, k, K, K[:3], tb, ln), "V_pages"),
                       ((q.bfloat16(), k, k, K, K, tb, ln), "dtype"), ((q, k, k, K, K, tb.long(), ln), "block_table"),
                       ((q, k, k, K, K, tb[0], ln), "block_table"), ((q, k, k, K, K, tb, _i32([3, 4])), "cached_lens"),
                       ((q, k[:, :1].contiguous(), k, K, K, tb, ln), "k must be")):
        with pytest.raises(ValueError, match=match):
            la.la_paged_decode_step(*bad)
    for scale in (0, 1e-60):  # the second is 0 in fp32
        with pytest.raises(ValueError, match="scale"):
            la.la_paged_decode_step(q, k, k, K, K, tb, ln, scale=scale)
    with pytest.raises(la.LinAttnError, match="INVALID_ARG"):
        la.la_paged_decode_step(q, k, k, K, K, tb, ln, window=-2)
    with pytest.raises(la.LinAttnError, match="UNSUPPORTED"):
        P = torch.zeros(4, 2, 12, 64, device="cuda")
        la.la_paged_decode_step(q, k, k, P, P, tb, ln)
    with pytest.raises(la.LinAttnError, match="INVALID_ARG"):
        la.la_paged_decode_step(torch.zeros(1, 3, 64, device="cuda"), k, k, K, K, tb, ln)


# ---------------------------------------------------------------- all of them together

@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_serving_run(dt):
    """A ragged batch through a recurrent layer and a softmax layer: the page map cuts the packed
    prompt rows for the scan and places their keys and values, then tokens are decoded one by one
    with the map of each step, the scan's step and the paged step."""
    la = _la()
    R, Hq, Hkv, D, page, P, W, steps = 5, 4, 2, 32, 8, 64, 12, 10
    C = Hkv * D
    prompt = [13, 1, 0, 40, 8]
    g = torch.Generator().manual_seed(20)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DT[dt])  # noqa: E731
    free = torch.randperm(P, generator=g).to(torch.int32)
    K, V = (torch.zeros(P, Hkv, page, D, dtype=DT[dt], device="cuda") for _ in range(2))
    table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    cached, taken = _i32([0] * R), 0
    rows = sum(prompt) + 6  # a padded row axis
    a, x = rnd(1, rows, C) + 2, rnd(1, rows, C)
    k, v = rnd(rows, Hkv, D), rnd(rows, Hkv, D)
    slots = torch.empty(rows, dtype=torch.int32, device="cuda")
    new = _i32(prompt)
    _, starts, counts = la.la_page_map(cached, new, free.cuda(), table, page, P, slots)
    _, h = la.la_forward_gated_scan(a.cuda(), x.cuda(), form="logit", seq_starts=starts, return_state=True)
    la.la_paged_append(k.cuda(), v.cuda(), K, V, slots)
    taken += int(counts[1])
    cached = cached + new
    off = np.concatenate([[0], np.cumsum(prompt)])
    hist = [(a[0, off[r]:off[r + 1]], x[0, off[r]:off[r + 1]], k[off[r]:off[r + 1]], v[off[r]:off[r + 1]]) for r in range(R)]
    one = _i32([1] * R)
    slots1 = torch.empty(R, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        q, k1, v1, a1, x1 = rnd(R, Hq, D), rnd(R, Hkv, D), rnd(R, Hkv, D), rnd(R, C) + 2, rnd(R, C)
        _, _, counts = la.la_page_map(cached, one, free[taken:].cuda(), table, page, P, slots1)
        y = la.la_gated_scan_decode_step(a1.cuda(), x1.cuda(), h, form="logit")
        out = la.la_paged_decode_step(q.cuda(), k1.cuda(), v1.cuda(), K, V, table, cached)
        la.la_check_device_status()
        # the step wrote its row where the map says
        s = slots1.tolist()
        for r in range(R):
            assert torch.equal(K[s[r] // page, :, s[r] % page].cpu(), k1[r])
        taken += int(counts[1])
        cached = cached + one
        for r in range(R):
            A, X, kk, vv = (torch.cat([o, n[None]]) for o, n in zip(hist[r], (a1[r], x1[r], k1[r], v1[r])))
            hist[r] = (A, X, kk, vv)
            _, wh, _ = ref.gated_scan_forward(A[None], X[None], "logit")
            assert np.abs(h[r].double().cpu().numpy() - wh[0]).max() <= 1.5e-5 * max(4.0, np.abs(wh).max())
            half = 2.0 ** -8 if dt == "bf16" else 0.0
            assert np.all(np.abs(y[r].double().cpu().numpy() - wh[0]) <= half * np.abs(wh[0]) + 6e-5)
            w, _ = ref.paged_decode(q[r:r + 1], None, None, kk.double().transpose(0, 1)[None], vv.double().transpose(0, 1)[None],
                                    [[0]], [kk.shape[0]])
            assert np.abs(out[r].double().cpu().numpy() - w[0]).max() <= 1e-4


# ---------------------------------------------------------------- many ranges, many columns, scratch

def _exact_on_gpu(d, table, lens, window=0):
    """fp64 outputs and logs of sums without a new row, one request at a time on the GPU."""
    q, K, V = d["q"], d["K"], d["V"]
    R, Hq, D = q.shape
    Hkv, page = K.shape[1], K.shape[2]
    out = torch.zeros(R, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        if n == 0:
            continue
        pages = torch.tensor(table[r][:-(-n // page)], device="cuda")
        k = K[pages].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :n]
        v = V[pages].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :n]
        s = torch.einsum("hgd,hnd->hgn", q[r].double().view(Hkv, -1, D), k) / math.sqrt(D)
        out[r] = torch.einsum("hgn,hnd->hgd", torch.softmax(s, 2), v).reshape(Hq, D)
        lse[r] = torch.logsumexp(s, 2).reshape(Hq)
    return out, lse


@pytest.mark.parametrize("dt,R,Hq,Hkv,D,page,most", [
    ("bf16", 64, 16, 16, 32, 16, 4100),   # four ranges a warp
    ("bf16", 40, 64, 8, 64, 32, 4000),    # eight query heads a key head
    ("bf16", 24, 64, 4, 128, 16, 6000),   # sixteen
    ("f32", 30, 24, 8, 64, 64, 5000),     # three, fp32
    ("f32", 20, 48, 4, 128, 16, 4000),    # twelve, fp32
    ("bf16", 4000, 4, 4, 32, 16, 40),     # more columns than ranges
    ("f32", 9000, 2, 2, 32, 8, 12),       # likewise, pages shorter than a step
])
def test_paged_decode_over_many_ranges(dt, R, Hq, Hkv, D, page, most):
    la = _la()
    lens = [(i * 7919) % (most + 1) for i in range(R)]
    g = torch.Generator(device="cuda").manual_seed(R)
    need = [-(-n // page) for n in lens]
    P, W = sum(need) + 1, max(need) + 1
    order, table, at = np.random.RandomState(R).permutation(P).tolist(), [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (W - n))
        at += n
    d = {n: torch.randn(s, generator=g, device="cuda").to(DT[dt]) for n, s in
         (("q", (R, Hq, D)), ("K", (P, Hkv, page, D)), ("V", (P, Hkv, page, D)))}
    out, lse = la.la_paged_decode_step(d["q"], None, None, d["K"], d["V"], _i32(table), _i32(lens), return_lse=True)
    la.la_check_device_status()
    wo, wl = _exact_on_gpu(d, table, lens)
    x = {"q": d["q"], "K": d["K"], "V": d["V"], "k": d["K"][0], "v": d["V"][0]}
    to, tl = _bounds(x, D)
    assert float((out.double() - wo).abs().max()) <= to
    some = torch.isfinite(wl)
    assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
    assert float((lse.double() - wl)[some].abs().max()) <= tl


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_paged_decode_scratch_matches_report(dt):
    la = _la()
    for Hq, Hkv, D, page, lens in ((8, 2, 64, 16, [300, 5]), (32, 2, 128, 32, [9000, 20000, 1])):
        x, table = _decode_case(len(lens), Hq, Hkv, D, page, lens, False, dt)
        d = {n: t.cuda() for n, t in x.items()}
        tb, ln = _i32(table), _i32(lens)
        want = la.la_paged_decode_workspace_bytes(len(lens), Hq, Hkv, D, page, tb.shape[1], DT[dt])
        torch.cuda.synchronize()
        la.la_scratch_peak_bytes(reset=True)
        la.la_paged_decode_step(d["q"], None, None, d["K"], d["V"], tb, ln)
        torch.cuda.synchronize()
        assert want <= la.la_scratch_peak_bytes() <= want + (2 << 20)


@pytest.mark.parametrize("dt,Hq,Hkv", [("bf16", 2, 2), ("bf16", 12, 1), ("f32", 12, 1), ("f32", 20, 1)])
def test_paged_decode_non_finite_keys_stay_where_they_are(dt, Hq, Hkv):
    # keys of infinite negative scores count nothing; a NaN key makes its own request NaN and no other
    la = _la()
    lens = [40, 40, 70]
    x, table = _decode_case(3, Hq, Hkv, 32, 16, lens, False, dt, seed=31)
    x["q"][:] = x["q"].abs() + 0.1
    x["K"][:] = x["K"].abs()
    tol, _ = _bounds(x, 32)
    clean = la.la_paged_decode_step(x["q"].cuda(), None, None, x["K"].cuda(), x["V"].cuda(), _i32(table), _i32(lens))
    for p in range(35):
        x["K"][table[0][p // 16], :, p % 16] = float("-inf")
    x["K"][table[1][0], :, 3] = float("nan")
    out = la.la_paged_decode_step(x["q"].cuda(), None, None, x["K"].cuda(), x["V"].cuda(), _i32(table), _i32(lens))
    K5 = torch.stack([x["K"][table[0][p // 16], :, p % 16] for p in range(35, 40)], 1).double()
    V5 = torch.stack([x["V"][table[0][p // 16], :, p % 16] for p in range(35, 40)], 1).double()
    s = torch.einsum("hgd,hnd->hgn", x["q"][0].double().view(Hkv, -1, 32), K5) / math.sqrt(32)
    want = torch.einsum("hgn,hnd->hgd", torch.softmax(s, 2), V5).reshape(Hq, 32)
    assert float((out[0].cpu().double() - want).abs().max()) <= tol
    assert bool(torch.isnan(out[1]).all())
    assert torch.equal(out[2], clean[2])
