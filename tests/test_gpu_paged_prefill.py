"""GPU parity of the attention of a chunk of new tokens over the paged cache, against its fp64 plain form.

Tolerances.  A score is a sum of D products, off by at most (D + 4) 2^-24 of scale sum |q k| (the 4: scaling
and base change); a weight is off by that much relative to itself, and by the same in the sum below the
fraction; the exponentials, sums and products add 64 x 2^-23 in all.  bf16: a weight is rounded to
bf16 before it meets its value, by 2^-8 of itself, so an output by 2^-8 of the weighted mean of |v|, and the
output is rounded once more.
"""
import math

import numpy as np
import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _la():
    import linear_attention_02_gb300 as la
    return la


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(Hq, Hkv, D, page, cached, new, dt, seed=1, tail=0, spare=2):
    """Inputs, the pages of each request in a shuffled pool."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(max(c, 0) + n) // page) for c, n in zip(cached, new)]
    P, W = sum(need) + spare, max(need + [1]) + 1
    order, table, at = torch.randperm(P, generator=g).tolist(), [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (W - n))
        at += n
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    T = starts[-1] + tail
    x = {n: torch.randn(s, generator=g).to(DT[dt]) for n, s in
         (("q", (T, Hq, D)), ("K", (P, Hkv, page, D)), ("V", (P, Hkv, page, D)))}
    return x, table, starts


def _score_error(x, D, scale):
    s = 1 / math.sqrt(D) if scale is None else abs(scale)
    return (D + 4) * 2.0 ** -24 * s * float(x["q"].float().norm(dim=-1).max()) * float(x["K"].float().norm(dim=-1).max())


def _check(x, table, cached, starts, D, dt, window=0, scale=None, clean=None):
    """clean: what the plain form reads where the call's pages hold what no row may see."""
    la = _la()
    d = {n: t.cuda() for n, t in x.items()}
    out = torch.full(x["q"].shape, 9.5, device="cuda", dtype=DT[dt])
    lse = torch.full(x["q"].shape[:2], 9.5, device="cuda")
    got, gl = la.la_paged_prefill(d["q"], d["K"], d["V"], _i32(table), _i32(cached), _i32(starts), window=window, scale=scale,
                                  out=out, lse=lse, return_lse=True)
    assert got is out and gl is lse
    x = clean or x
    wo, wl, size = ref.paged_prefill(x["q"], x["K"], x["V"], table, cached, starts, window, scale)
    err = _score_error(x, D, scale)
    own = ~np.isnan(wl)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(got[~own] == 9.5) and np.all(gl[~own] == 9.5)
    tol = (2 * err + 64 * 2.0 ** -23 + (HALF[dt] if dt == "bf16" else 0)) * size + HALF[dt] * np.abs(wo)
    worst = (np.abs(got - wo) - tol * 1.01)[own]
    assert np.all(worst <= 0), f"{(worst > 0).sum()} of {worst.size} off, by {np.abs(got - wo)[own].max():.3g}"
    fin = np.isfinite(wl[own])
    assert np.array_equal(np.isneginf(gl[own]), ~fin)
    assert np.abs(gl[own][fin] - wl[own][fin]).max(initial=0) <= err + 64 * 2.0 ** -23 * 8
    return out, lse


SHAPES = [  # Hq, Hkv, D, page, cached, new
    (1, 1, 32, 1, [0, 3, 9], [1, 2, 5]), (2, 1, 32, 2, [0, 31], [33, 7]), (4, 4, 64, 4, [5], [70]),
    (4, 4, 64, 16, [0, 15, 16, 17], [1, 1, 16, 40]), (8, 2, 128, 8, [7, 130], [9, 60]), (6, 2, 64, 32, [31, 0, 400], [3, 100, 1]),
    (12, 2, 128, 64, [200, 64], [50, 11]), (16, 1, 128, 16, [100, 511], [17, 2]), (20, 1, 64, 16, [77], [20]),
    (2, 2, 64, 128, [300], [270]), (3, 1, 128, 1024, [1000, 0], [90, 2]), (1, 1, 64, 16, [0], [600]),
    (130, 1, 32, 16, [40], [3]), (8, 8, 128, 256, [0, 0, 0], [0, 129, 0])]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page,cached,new", SHAPES)
def test_prefill(Hq, Hkv, D, page, cached, new, dt):
    x, table, starts = _case(Hq, Hkv, D, page, cached, new, dt, tail=3)
    _check(x, table, cached, starts, D, dt)
    _la().la_check_device_status()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 129, 100000])
def test_window(window, dt):
    cached, new = [0, 50, 300, 127], [40, 1, 140, 3]
    x, table, starts = _case(4, 2, 64, 16, cached, new, dt, seed=window)
    _check(x, table, cached, starts, 64, dt, window=window)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, -0.3, 4.0, 1e-20])
def test_scale(scale, dt):
    cached, new = [20, 0], [30, 130]
    x, table, starts = _case(4, 2, 64, 16, cached, new, dt)
    _check(x, table, cached, starts, 64, dt, scale=scale)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,cached,new", [(8, 1, 128, [5000, 900, 0], [2, 4, 1]), (4, 4, 64, [6000], [1]),
                                                 (16, 2, 32, [3000] * 3, [5, 9, 33])])
def test_few_rows_over_long_contexts(Hq, Hkv, D, cached, new, dt):
    x, table, starts = _case(Hq, Hkv, D, 16, cached, new, dt)
    _check(x, table, cached, starts, D, dt)


def test_many_requests():
    r = np.random.RandomState(1)
    cached, new = r.randint(0, 60, 700).tolist(), r.randint(0, 4, 700).tolist()
    x, table, starts = _case(2, 1, 32, 16, cached, new, "bf16")
    _check(x, table, cached, starts, 32, "bf16")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_what_no_row_sees_may_be_anything(what, dt):
    # pages' ends behind the last position, positions before the window, pages of no request
    page, D, cached, new, window = 16, 64, [30, 0, 200], [21, 5, 100], 40
    x, table, starts = _case(4, 2, D, page, cached, new, dt)
    bad = {n: t.clone() for n, t in x.items()}
    held = np.zeros((x["K"].shape[0], page), bool)
    for r, (c, n) in enumerate(zip(cached, new)):
        for p in range(max(0, c - window + 1) if n else c, c + n):
            held[table[r][p // page], p % page] = True
    free = torch.tensor(~held)
    for n in ("K", "V"):
        bad[n].permute(0, 2, 1, 3)[free] = what
    _check(bad, table, cached, starts, D, dt, window=window, clean=x)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,cached,new,at", [(2, 2, 10, 300, 200), (8, 1, 500, 40, 520), (1, 1, 0, 700, 640)])
def test_a_later_tokens_values_do_not_reach_earlier_rows(Hq, Hkv, cached, new, at, dt):
    # position `at` holds what is not finite: rows before it stay as they are, rows that see it do not
    page, D = 16, 64
    x, table, starts = _case(Hq, Hkv, D, page, [cached], [new], dt)
    want, wl = _check(x, table, [cached], starts, D, dt)
    la = _la()
    for n, what in (("V", math.inf), ("V", math.nan), ("K", math.nan), ("K", math.inf)):
        y = {k: t.clone().cuda() for k, t in x.items()}
        y[n][table[0][at // page], :, at % page, 5] = what
        for window in (0, 50):
            out, lse = la.la_paged_prefill(y["q"], y["K"], y["V"], _i32(table), _i32([cached]), _i32(starts), window=window, return_lse=True)
            ref_o, ref_l = (want, wl) if window == 0 else la.la_paged_prefill(
                x["q"].cuda(), x["K"].cuda(), x["V"].cuda(), _i32(table), _i32([cached]), _i32(starts), window=window, return_lse=True)
            pos = cached + torch.arange(new, device="cuda")
            sees = (pos >= at) & ((pos < at + window) if window else (pos >= 0))
            assert torch.equal(out[~sees], ref_o[~sees]) and torch.equal(lse[~sees], ref_l[~sees]), (n, what, window)
            if n == "V":
                assert not bool(torch.isfinite(out[sees][..., 5]).any()), (n, what, window)
                rest = [c for c in range(D) if c != 5]
                assert torch.equal(out[sees][..., rest], ref_o[sees][..., rest]) and torch.equal(lse[sees], ref_l[sees])
            elif math.isnan(what):
                assert bool(torch.isnan(out[sees]).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("new", [20, 150])
def test_values_that_are_not_finite_in_some_of_many_requests(new, dt):
    # many tiles a block, a few of them with a NaN that only the request's later rows see
    la = _la()
    R, H, D, page, at = 2000, 2, 64, 16, 11
    W = -(-new // page)
    g = torch.Generator().manual_seed(5)
    q, K, V = (torch.randn(s, generator=g).to(DT[dt]).cuda() for s in ((R * new, H, D), (R * W, H, page, D), (R * W, H, page, D)))
    table = torch.randperm(R * W, generator=g).to(torch.int32).cuda().view(R, W)
    lens, starts = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.arange(R + 1, device="cuda", dtype=torch.int32) * new
    want = la.la_paged_prefill(q, K, V, table, lens, starts).view(R, new, H, D)
    hit = torch.arange(0, R, 7, device="cuda")
    V[table[hit, 0].long(), :, at, 9] = math.nan
    got = la.la_paged_prefill(q, K, V, table, lens, starts).view(R, new, H, D)
    sees = torch.zeros((R, new, H, D), dtype=torch.bool, device="cuda")
    sees[hit, at:, :, 9] = True
    assert torch.equal(torch.isnan(got), sees)
    assert torch.equal(got[~sees], want[~sees])


def test_rows_of_no_request():
    la = _la()
    cached, new = [5, -1, 9, -7], [3, 4, 0, 2]
    x, table, starts = _case(4, 2, 64, 16, cached, new, "bf16", tail=6)
    out, lse = _check(x, table, cached, starts, 64, "bf16")
    d = {n: t.cuda() for n, t in x.items()}
    o2, l2 = la.la_paged_prefill(d["q"], d["K"], d["V"], _i32(table), _i32(cached), _i32(starts), return_lse=True)
    own = torch.zeros(len(x["q"]), dtype=torch.bool)
    own[:3] = True
    assert torch.equal(o2[own], out[own]) and torch.equal(l2[own], lse[own])
    assert bool((o2[~own] == 0).all()) and bool(torch.isneginf(l2[~own]).all())
    # no request at all
    e = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    o3 = la.la_paged_prefill(d["q"], d["K"], d["V"], e, e.view(0), _i32([0]))
    assert bool((o3 == 0).all())
    la.la_check_device_status()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bad_pages_lengths_and_starts_are_reported(dt):
    la = _la()
    cached, new = [40, 10, 0], [30, 20, 9]
    x, table, starts = _case(4, 2, 64, 16, cached, new, dt)
    table[0][1], table[1][0], table[2][0] = -1, 9999, -5  # request 1 keeps one page of two, request 2 none
    _check(x, table, cached, starts, 64, dt)
    with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
        la.la_check_device_status()
    d = {n: t.cuda() for n, t in x.items()}
    x2, table2, _ = _case(4, 2, 64, 16, cached, new, dt)
    for c, st in ((cached, [0, 30, 20, 59]), (cached, [-4, 30, 50, 59]), (cached, [0, 30, 50, 1000]),
                  ([2 ** 31 - 1, 10, 0], starts), ([10 ** 6, 10, 0], starts), (cached, [0, 2 ** 31 - 1, 5, 59])):
        la.la_paged_prefill(d["q"], d["K"], d["V"], _i32(table2), _i32(c), _i32(st))
        with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
            la.la_check_device_status()
    la.la_check_device_status()
    # starts that go back and forth, and would name more rows than there are: no request is done
    R, T = 40, 59
    t3 = torch.zeros((R, 8), dtype=torch.int32, device="cuda")
    keep = torch.full_like(d["q"][:T], 9.5)
    la.la_paged_prefill(d["q"][:T].contiguous(), d["K"], d["V"], t3, _i32([0] * R), _i32([0, T] * (R // 2) + [0]), out=keep)
    with pytest.raises(la.LinAttnError, match="BAD_INDEX"):
        la.la_check_device_status()
    assert bool((keep == 9.5).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_infinite_keys_and_queries(dt):
    # a score of -infinity is a weight of 0, one of +infinity no number; other rows do not notice
    la = _la()
    D, cached, new = 64, 20, 90
    x, table, starts = _case(2, 1, D, 16, [cached], [new], dt)
    x["q"][:, :, 7] = 1.0
    for what in (-math.inf, math.inf):
        y = {n: t.clone() for n, t in x.items()}
        y["K"][table[0][2], 0, 5, 7] = what  # position 37
        _, _, _ = d = tuple(y[n].cuda() for n in ("q", "K", "V"))
        out, lse = la.la_paged_prefill(*d, _i32(table), _i32([cached]), _i32(starts), return_lse=True)
        with np.errstate(invalid="ignore"):
            wo, wl, size = ref.paged_prefill(y["q"], y["K"], y["V"], table, [cached], starts)
        err = _score_error(x, D, None)
        tol = (2 * err + 64 * 2.0 ** -23 + (HALF[dt] if dt == "bf16" else 0)) * size + HALF[dt] * np.abs(wo)
        got = out.double().cpu().numpy()
        assert np.array_equal(np.isfinite(got), np.isfinite(wo))
        fin = np.isfinite(wo)
        assert np.all(np.abs(got - wo)[fin] <= 1.01 * tol[fin])
        if what > 0:
            assert not np.isfinite(got[37 - cached:]).any() and np.isfinite(got[:37 - cached]).all()


def test_serving_run():
    """Prompts in chunks through page map, norm and rotation, append and prefill; then single tokens by the decode step;
    against one pass over the whole sequences."""
    la = _la()
    torch.manual_seed(3)
    R, Hq, Hkv, D, page, P = 3, 8, 2, 64, 16, 40
    total = [150, 37, 90]
    free = torch.randperm(P).to(torch.int32).cuda()
    table = torch.full((R, 12), -1, dtype=torch.int32, device="cuda")
    K, V = (torch.zeros(P, Hkv, page, D, device="cuda") for _ in range(2))
    q, k, v = (torch.randn(sum(total), h, D, device="cuda") for h in (Hq, Hkv, Hkv))
    wq, wk = torch.rand(D, device="cuda") + 0.5, torch.rand(D, device="cuda") + 0.5
    freqs, mag = la.la_rotary_frequencies(D)
    first = [0, total[0], total[0] + total[1]]
    done, used, outs = [0] * R, 0, [[] for _ in range(R)]
    for step in ([70, 37, 0], [79, 0, 89], [1, 0, 1]):
        rows = torch.cat([torch.arange(f + d, f + d + n) for f, d, n in zip(first, done, step)]).cuda()
        pos = torch.cat([torch.arange(d, d + n) for d, n in zip(done, step)]).to(torch.int32).cuda()
        slots = torch.empty(len(rows), dtype=torch.int32, device="cuda")
        _, starts, counts = la.la_page_map(_i32(done), _i32(step), free[used:].contiguous(), table, page, P, slots)
        qr, kr = la.la_forward_norm_rotary(q[rows], k[rows], wq, wk, freqs, positions=pos, magnitude=mag)
        if max(step) > 1:
            la.la_paged_append(kr, v[rows].contiguous(), K, V, slots)
            o = la.la_paged_prefill(qr, K, V, table, _i32(done), starts)
        else:  # the last token of requests 0 and 2; request 1 is a row without a request
            lens = _i32([done[0], -1, done[2]])
            pad = lambda t: torch.stack([t[0], torch.zeros_like(t[0]), t[1]])  # noqa: E731
            o = la.la_paged_decode_step(pad(qr), pad(kr), pad(v[rows]), K, V, table, lens)
            o = torch.stack([o[0], o[2]])
        used += int(counts[1])
        at = 0
        for r, n in enumerate(step):
            outs[r].append(o[at:at + n])
            at, done[r] = at + n, done[r] + n
    la.la_check_device_status()
    assert done == total
    fn = freqs.cpu().numpy()
    for r in range(R):
        s = slice(first[r], first[r] + total[r])
        a = ref.rotary_angles(fn, np.arange(total[r]))[:, None]
        qq = ref.norm_rotary(q[s], wq.double().cpu().numpy(), a)
        kk = ref.norm_rotary(k[s], wk.double().cpu().numpy(), a)
        pool = lambda t: np.ascontiguousarray(np.asarray(t)[:, :, None, :])  # noqa: E731  pages of one position
        wo, _, size = ref.paged_prefill(qq, pool(kk), pool(v[s].double().cpu().numpy()), [list(range(total[r]))], [0], [0, total[r]])
        got = torch.cat(outs[r]).double().cpu().numpy()
        # scores move by (D / 2 + 12) u of the norms' product on each side beside the products' own rounding
        sc = np.linalg.norm(qq, axis=-1).max() * np.linalg.norm(kk, axis=-1).max() / math.sqrt(D)
        tol = (2 * sc * (2 * (D / 2 + 12) * math.sqrt(2) + D + 4) * 2.0 ** -24 + 64 * 2.0 ** -23) * size
        assert np.all(np.abs(got - wo) <= tol + 2.0 ** -24)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_requests_that_share_pages(dt):
    # a common beginning held once, and a page that one table names twice
    cached, new, page, D = [32, 32, 40], [9, 150, 3], 16, 64
    x, table, starts = _case(4, 2, D, page, cached, new, dt)
    for r in (1, 2):
        table[r][:2] = table[0][:2]
    table[2][1] = table[2][0]
    _check(x, table, cached, starts, D, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_calls_at_once_on_two_streams(dt):
    la = _la()
    cases = []
    for seed, cached, new in ((1, [900, 0, 300], [40, 500, 1]), (2, [0] * 40, [70] * 40)):
        x, table, starts = _case(8, 2, 64, 16, cached, new, dt, seed=seed)
        cases.append((*(x[n].cuda() for n in "qKV"), _i32(table), _i32(cached), _i32(starts)))
    want = [la.la_paged_prefill(*c) for c in cases]
    streams, got = [torch.cuda.Stream() for _ in cases], [[], []]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, c, g in zip(streams, cases, got):
            with torch.cuda.stream(s):
                g.append(la.la_paged_prefill(*c))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, o) for o in g)
    la.la_check_device_status()


def test_other_stream_and_captured_graphs_follow_the_lengths():
    la = _la()
    cached, new = [40, 10, 70], [30, 20, 9]
    x, table, starts = _case(4, 2, 64, 16, [90, 60, 80], [40, 40, 40], "bf16")
    d = {n: t.cuda() for n, t in x.items()}
    tb, cl, st = _i32(table), _i32(cached), _i32([0, 30, 50, 59])
    args = (d["q"], d["K"], d["V"], tb, cl, st)
    want = la.la_paged_prefill(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = la.la_paged_prefill(*args)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(la.la_paged_prefill(*args))
        graphs.append(gr)
    for c, n in (([5, 0, 100], [40, 0, 3]), ([90, 60, 80], [40, 40, 40])):
        cl.copy_(_i32(c))
        st.copy_(_i32(np.concatenate([[0], np.cumsum(n)]).tolist()))
        want = la.la_paged_prefill(*args)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scratch(dt):
    la = _la()
    from linear_attention_02_gb300 import _native
    cached, new = [300, 20], [100, 30]
    x, table, starts = _case(8, 2, 128, 16, cached, new, dt)
    d = {n: t.cuda() for n, t in x.items()}
    for _ in range(2):
        _native.lib.la_scratch_peak_bytes(1)
        la.la_paged_prefill(d["q"], d["K"], d["V"], _i32(table), _i32(cached), _i32(starts))
        torch.cuda.synchronize()
    want = la.la_paged_prefill_workspace_bytes(128, DT[dt])
    assert want <= _native.lib.la_scratch_peak_bytes(1) <= want + (2 << 20)


def test_repeatable():
    la = _la()
    cached, new = [3000, 900, 0, 77], [100, 300, 500, 1]
    x, table, starts = _case(8, 2, 128, 16, cached, new, "bf16")
    d = {n: t.cuda() for n, t in x.items()}
    runs = [la.la_paged_prefill(d["q"], d["K"], d["V"], _i32(table), _i32(cached), _i32(starts), return_lse=True) for _ in range(4)]
    for o, l in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(l, runs[0][1])
