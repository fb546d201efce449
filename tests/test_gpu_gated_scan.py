"""GPU parity of the gated scan (forward, backward, single-token step) against
its fp64 plain form, through the C ABI.

Tolerances.  A row's state takes three fp32 roundings of at most 2^-24 of the
largest state (input product, decay product, sum), the sigmoid and its
complement a few more (8 x 2^-24 in all), and an error lives as long as the
gates carry it: with these gates (0.85 to 1, or sigmoid of N(2, 1.5)) the sum of
the products of decays stays below 32, so a state is within
32 * 8 * 2^-24 = 1.5e-5 of the largest one.  A gradient dA is a product of two
such values, each within 1.5e-5 of its largest: 3e-5 of the product of the
largest two, plus its own roundings, 4e-5.  bf16 results are rounded once more,
by at most 2^-8 of their own value.
"""
import numpy as np
import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STATE, GRAD = 1.5e-5, 4e-5
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


def _la():
    import linear_attention_02_gb300 as la
    return la


def _inputs(B, N, C, dt, form, seed, S=None):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(B, N, C, generator=g) * 1.5 + 2 if form == "logit" else \
        torch.rand(B, N, C, generator=g) * 0.15 + 0.85
    S = B if S is None else S
    x = {"A": a.to(DT[dt]), "X": torch.randn(B, N, C, generator=g).to(DT[dt]),
         "G": torch.randn(B, N, C, generator=g).to(DT[dt]), "h0": torch.randn(S, C, generator=g),
         "dh": torch.randn(S, C, generator=g)}
    return x, {k: v.cuda() for k, v in x.items()}


def _close(got, want, dt, scale, tol):
    got = got.double().cpu().numpy()
    bound = HALF[dt] * np.abs(want) + tol * scale
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) - bound):.3e}"


def _check_all(B, N, C, dt, form, starts=None, state=True, ckpt=True, seed=1):
    la = _la()
    S = None if starts is None else len(starts) - 1
    x, d = _inputs(B, N, C, dt, form, seed, S)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    h0, dh = (x["h0"], x["dh"]) if state else (None, None)
    kw = dict(form=form, seq_starts=st, h_init=d["h0"] if state else None)
    mark = 7.25  # exact in bf16: what no sequence owns keeps it
    out, dA, dX = (torch.full((B, N, C), mark, dtype=DT[dt], device="cuda") for _ in range(3))
    ck = torch.full((la.la_gated_scan_ckpt_floats(B, N, C),), float("nan"), device="cuda") if ckpt else None
    _, final = la.la_forward_gated_scan(d["A"], d["X"], out=out, return_state=True, ckpt=ck, **kw)
    _, _, d0 = la.la_backward_gated_scan(d["A"], d["X"], d["G"], dh_final=d["dh"] if state else None,
                                         return_dh_init=True, Ckpt=ck, dA=dA, dX=dX, **kw)
    la.la_check_device_status()
    want, wfinal, prev = ref.gated_scan_forward(x["A"], x["X"], form, h0, starts)
    wA, wX, w0 = ref.gated_scan_backward(x["A"], x["X"], x["G"], form, h0, dh, starts)
    own = ~np.isnan(want)
    for t in (out, dA, dX):
        assert bool((t.cpu()[torch.from_numpy(~own)] == mark).all())
        t[torch.from_numpy(~own).cuda()] = 0
    z = lambda a: np.where(own, a, 0.0)  # noqa: E731
    big = max(np.abs(z(want)).max(), np.abs(z(prev)).max(), 1.0)
    _close(out, z(want), dt, big, STATE)
    _close(final, wfinal, "f32", max(big, np.abs(wfinal).max()), STATE)
    s, c = ref._gates(x["A"], form)
    G = np.abs(z(wX) / np.where(c > 0, c, 1)).max()
    _close(dX, z(wX), dt, G, STATE)
    _close(dA, z(wA), dt, G * (big + (np.abs(x["X"].double().numpy()).max() if form == "logit" else 0)), GRAD)
    _close(d0, w0, "f32", max(G, np.abs(w0).max()), STATE)


SHAPES = [(1, 1, 1), (2, 3, 5), (1, 255, 64), (1, 256, 64), (2, 257, 72), (3, 513, 33), (1, 1000, 130),
          (2, 64, 1000), (1, 3001, 8), (4, 1, 96), (1, 777, 257), (5, 31, 256)]


@pytest.mark.parametrize("form", ["decay", "logit"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_scan(shape, dt, form):
    _check_all(*shape, dt, form)


@pytest.mark.parametrize("form", ["decay", "logit"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("state,ckpt", [(False, True), (True, False), (False, False)])
def test_scan_without_state_or_checkpoints(dt, form, state, ckpt):
    _check_all(2, 700, 72, dt, form, state=state, ckpt=ckpt)
    _check_all(1, 700, 33, dt, form, starts=[0, 300, 300, 650], state=state, ckpt=ckpt)


PACKED = [
    (1, 1, [0, 1]),                                   # one row
    (10, 5, [0, 0, 0, 10, 10]),                       # empty sequences before and behind
    (600, 64, [0, 1, 2, 3, 255, 256, 257, 258, 512, 513, 590]),  # at tile borders, rows behind the last
    (1030, 72, [0, 1030]),
    (1030, 33, [0, 0, 1024, 1024, 1024, 1029]),
    (2000, 136, [0, 700, 701, 1999, 2000, 2000]),
    (520, 8, list(range(0, 521, 1))),                 # every row its own sequence
    (300, 16, [0, 0, 0]),                             # no row belongs to a sequence
]


@pytest.mark.parametrize("form", ["decay", "logit"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(PACKED)))
def test_scan_packed(case, dt, form):
    N, C, starts = PACKED[case]
    _check_all(1, N, C, dt, form, starts=starts, seed=case)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scan_empty_calls_hand_the_state_on(dt):
    la = _la()
    a = torch.zeros(2, 0, 8, dtype=DT[dt], device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    assert torch.equal(la.la_forward_gated_scan(a, a, h_init=h0, return_state=True)[1], h0)
    assert not la.la_forward_gated_scan(a, a, return_state=True)[1].any()
    assert torch.equal(la.la_backward_gated_scan(a, a, a, dh_final=h0, return_dh_init=True)[2], h0)
    st = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert torch.equal(la.la_forward_gated_scan(a[:1], a[:1], h_init=h0, return_state=True, seq_starts=st)[1], h0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scan_sequences_and_padding_do_not_leak(dt):
    # a sequence of NaN and infinities, and such rows behind the last sequence, change nothing else
    la = _la()
    N, C, starts = 900, 72, [0, 200, 500, 600, 850]
    x, d = _inputs(1, N, C, dt, "decay", 5, 4)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")

    def both(A, X, G):
        o, f = la.la_forward_gated_scan(A, X, seq_starts=st, return_state=True, h_init=d["h0"],
                                        out=torch.zeros_like(A))
        dA, dX, d0 = la.la_backward_gated_scan(A, X, G, seq_starts=st, h_init=d["h0"], dh_final=d["dh"],
                                               return_dh_init=True, dA=torch.zeros_like(A), dX=torch.zeros_like(A))
        return o, f, dA, dX, d0

    clean = both(d["A"], d["X"], d["G"])
    A, X, G = (d[n].clone() for n in ("A", "X", "G"))
    X[0, 210:490] = float("nan")
    G[0, 210:490] = float("inf")
    A[0, 300:310] = float("nan")
    for t in (A, X, G):
        t[0, 850:] = float("nan")
    dirty = both(A, X, G)
    keep = [0, 2, 3]
    for c, q in zip(clean, dirty):
        if c.dim() == 3:
            for r in (slice(0, 200), slice(500, 900)):
                assert torch.equal(c[:, r], q[:, r])
        else:
            assert torch.equal(c[keep], q[keep])
    assert torch.isnan(dirty[0][0, 211:500]).all()


@pytest.mark.parametrize("form", ["decay", "logit"])
def test_scan_gradient_against_differences(form):
    # the kernel's gradient along a direction against central differences of the fp64 form
    la = _la()
    B, N, C = 2, 300, 24
    x, d = _inputs(B, N, C, "f32", form, 9)
    ck = torch.empty(la.la_gated_scan_ckpt_floats(B, N, C), device="cuda")
    la.la_forward_gated_scan(d["A"], d["X"], form=form, h_init=d["h0"], ckpt=ck)
    got = la.la_backward_gated_scan(d["A"], d["X"], d["G"], form=form, h_init=d["h0"], dh_final=d["dh"],
                                    return_dh_init=True, Ckpt=ck)
    p = {k: v.double().numpy() for k, v in x.items()}

    def loss(A, X, h0):
        o, f, _ = ref.gated_scan_forward(A, X, form, h0)
        return (o * p["G"]).sum() + (f * p["dh"]).sum()

    r = np.random.RandomState(0)
    e = 1e-6
    for i, n in enumerate(("A", "X", "h0")):
        u = r.choice([-1.0, 1.0], p[n].shape) * np.sign(got[i].double().cpu().numpy())
        u = np.abs(u) * np.sign(got[i].double().cpu().numpy())  # a direction in which the terms add up
        hi, lo = dict(p), dict(p)
        hi[n], lo[n] = p[n] + e * u, p[n] - e * u
        num = (loss(hi["A"], hi["X"], hi["h0"]) - loss(lo["A"], lo["X"], lo["h0"])) / (2 * e)
        # sum of |gradient|: fp32 error 4e-5 of it, differences off by e^2 times third derivatives
        assert abs(num - (got[i].double().cpu().numpy() * u).sum()) <= 1e-4 * abs(num)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["decay", "logit"])
@pytest.mark.parametrize("B,C", [(1, 1), (3, 33), (7, 64), (256, 1024), (5, 1000)])
def test_scan_step(B, C, dt, form):
    la = _la()
    x, d = _inputs(1, B, C, dt, form, 3, B)
    h = d["h0"].clone()
    out = la.la_gated_scan_decode_step(d["A"][0], d["X"][0], h, form=form)
    s, c = ref._gates(x["A"][0], form)
    want = s * x["h0"].double().numpy() + c * x["X"][0].double().numpy()
    _close(h, want, "f32", max(np.abs(want).max(), 4.0), 8 * 2.0 ** -24)
    _close(out, want, dt, max(np.abs(want).max(), 4.0), 8 * 2.0 ** -24)


def test_scan_extreme_logits():
    # sigmoid at +-100 and infinities is 1 or 0 without NaN; the gradient's s (1 - s) is 0
    la = _la()
    z = torch.tensor([100.0, -100.0, float("inf"), float("-inf"), 0.0, 30.0, -30.0, 88.8]).view(1, 1, 8)
    A = z.expand(1, 300, 8).contiguous().cuda()
    X = torch.ones(1, 300, 8, device="cuda") * 3
    out, h = la.la_forward_gated_scan(A, X, form="logit", h_init=torch.ones(1, 8, device="cuda"), return_state=True)
    assert bool(torch.isfinite(out).all())
    assert out[0, -1, [0, 2]].tolist() == [1.0, 1.0] and out[0, -1, [1, 3]].tolist() == [3.0, 3.0]
    dA, dX = la.la_backward_gated_scan(A, X, torch.ones_like(X), form="logit")
    assert bool(torch.isfinite(dA).all()) and bool(torch.isfinite(dX).all())


def test_scan_decay_one_sums_and_zero_forgets():
    la = _la()
    N, C = 1500, 40
    X = torch.randint(-8, 9, (1, N, C), device="cuda").float()
    one = la.la_forward_gated_scan(torch.ones_like(X), X)
    assert torch.equal(one, X.cumsum(1))  # whole numbers below 2^24: exact in any order
    assert torch.equal(la.la_forward_gated_scan(torch.zeros_like(X), X), X)
    minus = la.la_forward_gated_scan(-torch.ones_like(X), X)
    sign = torch.ones(N, device="cuda")
    sign[1::2] = -1
    assert torch.equal(minus, (X * sign.view(1, N, 1)).cumsum(1) * sign.view(1, N, 1))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scan_results_do_not_depend_on_the_run(dt):
    la = _la()
    x, d = _inputs(2, 9000, 64, dt, "decay", 11)

    def once():
        o, f = la.la_forward_gated_scan(d["A"], d["X"], return_state=True)
        return (o, f) + la.la_backward_gated_scan(d["A"], d["X"], d["G"], return_dh_init=True)

    first = once()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


def test_scan_splits_where_the_state_is_handed_on():
    la = _la()
    x, d = _inputs(2, 1200, 72, "f32", "logit", 12)
    whole, hw = la.la_forward_gated_scan(d["A"], d["X"], form="logit", return_state=True)
    h, parts = None, []
    for t0, t1 in ((0, 1), (1, 400), (400, 1199), (1199, 1200)):
        o, h = la.la_forward_gated_scan(d["A"][:, t0:t1].contiguous(), d["X"][:, t0:t1].contiguous(), form="logit",
                                        h_init=h, return_state=True)
        parts.append(o)
    big = float(whole.abs().max())
    assert float((torch.cat(parts, 1) - whole).abs().max()) <= 2 * STATE * big
    assert float((h - hw).abs().max()) <= 2 * STATE * big
    # and the single-token step goes on from a prefix
    _, h = la.la_forward_gated_scan(d["A"][:, :1000].contiguous(), d["X"][:, :1000].contiguous(), form="logit",
                                    return_state=True)
    for t in range(1000, 1020):
        o = la.la_gated_scan_decode_step(d["A"][:, t].contiguous(), d["X"][:, t].contiguous(), h, form="logit")
        assert float((o - whole[:, t]).abs().max()) <= 2 * STATE * big


def test_scan_streams_and_graphs():
    la = _la()
    x, d = _inputs(1, 4000, 256, "bf16", "decay", 13)
    ck = torch.empty(la.la_gated_scan_ckpt_floats(1, 4000, 256), device="cuda")
    out, h = la.la_forward_gated_scan(d["A"], d["X"], return_state=True, ckpt=ck)
    dA, dX = la.la_backward_gated_scan(d["A"], d["X"], d["G"], Ckpt=ck)
    torch.cuda.synchronize()
    # two calls at once on two streams
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(la.la_forward_gated_scan(d["A"], d["X"]))
                got.append(la.la_backward_gated_scan(d["A"], d["X"], d["G"])[0])
    torch.cuda.synchronize()
    for i, t in enumerate(got):
        assert torch.equal(t, out if i % 2 == 0 else dA)
    # captured twice, replayed in turn and again, with new inputs in place
    o1, o2, g1 = torch.empty_like(out), torch.empty_like(out), torch.empty_like(dA)
    A2, X2 = d["A"].clone(), d["X"].clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        la.la_forward_gated_scan(A2, X2, out=o1)
        la.la_backward_gated_scan(A2, X2, d["G"], dA=g1, dX=torch.empty_like(dX))
    with torch.cuda.graph(graphs[1]):
        la.la_forward_gated_scan(A2, X2, out=o2)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, out) and torch.equal(o2, out) and torch.equal(g1, dA)
    X2.mul_(2)  # the recurrence is linear: twice the input, twice the state (an exact scaling)
    graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, out * 2) and torch.equal(o2, out * 2)
    la.la_check_device_status()


def test_scan_offsets_past_32_bits():
    # 1.1 million rows x 2048 channels: 2.25e9 elements.  Decay 1/2: a row is its last 40 inputs
    la = _la()
    N, C = 1_100_000, 2048
    A = torch.full((1, N, C), 0.5, dtype=torch.bfloat16, device="cuda")
    X = torch.zeros((1, N, C), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(200, C, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    X[0, -200:] = tail.cuda()
    G = torch.zeros_like(X)
    G[0, -1] = 1
    out = la.la_forward_gated_scan(A, X)
    want, _, prev = ref.gated_scan_forward(A[:, -200:], tail[None])
    _close(out[:, -200:], want, "bf16", np.abs(want).max(), STATE)
    assert not bool(out[:, 1_000_000:-200].any())
    del out
    dA, dX = la.la_backward_gated_scan(A, X, G)
    wA, wX, _ = ref.gated_scan_backward(A[:, -200:], tail[None], G[:, -200:])
    _close(dX[:, -200:], wX, "bf16", 1.0, STATE)
    _close(dA[:, -200:], wA, "bf16", np.abs(prev).max(), GRAD)


def test_scan_wrapper_refusals():
    la = _la()
    a = torch.zeros(2, 4, 8, device="cuda")
    with pytest.raises(ValueError, match="X must be"):
        la.la_forward_gated_scan(a, a[:, :2].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        la.la_forward_gated_scan(a.transpose(0, 1), a.transpose(0, 1))
    with pytest.raises(ValueError, match="dtype"):
        la.la_forward_gated_scan(a, a.bfloat16())
    with pytest.raises(ValueError, match="unsupported dtype"):
        la.la_forward_gated_scan(a.half(), a.half())
    with pytest.raises(ValueError, match="h_init"):
        la.la_forward_gated_scan(a, a, h_init=torch.zeros(1, 8, device="cuda"))
    st = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="B == 1"):
        la.la_forward_gated_scan(a, a, seq_starts=st)
    with pytest.raises(ValueError, match="seq_starts"):
        la.la_forward_gated_scan(a[:1], a[:1], seq_starts=st.long())
    with pytest.raises(ValueError, match="Ckpt"):
        la.la_backward_gated_scan(a, a, a, Ckpt=torch.zeros(3, device="cuda"))
    with pytest.raises(la.LinAttnError, match="INVALID_ARG"):  # rows not 16-byte aligned
        b = torch.zeros(33, device="cuda")[1:].view(1, 4, 8)
        la.la_forward_gated_scan(b, b)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scan_starts_outside_the_rows_are_cut(dt):
    la = _la()
    x, d = _inputs(1, 300, 40, dt, "decay", 21, 3)
    bad = torch.tensor([-5, 100, 2 ** 31 - 1, 10 ** 9], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 100, 300, 300], dtype=torch.int32, device="cuda")
    a = la.la_forward_gated_scan(d["A"], d["X"], h_init=d["h0"], seq_starts=bad, return_state=True)
    b = la.la_forward_gated_scan(d["A"], d["X"], h_init=d["h0"], seq_starts=good, return_state=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    a = la.la_backward_gated_scan(d["A"], d["X"], d["G"], h_init=d["h0"], seq_starts=bad, return_dh_init=True)
    b = la.la_backward_gated_scan(d["A"], d["X"], d["G"], h_init=d["h0"], seq_starts=good, return_dh_init=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scan_many_packed_sequences(dt):
    # 5000 sequences of 0 to 3 rows: borders found among many, several in each row group
    lens = [(i * 7) % 4 for i in range(5000)]
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    _check_all(1, starts[-1] + 9, 24, dt, "decay", starts=starts, seed=22)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [100, 1000])
def test_scan_scratch_matches_report(dt, N):
    la = _la()
    B, C = 2, 136
    x, d = _inputs(B, N, C, dt, "logit", 23)
    ck = torch.empty(la.la_gated_scan_ckpt_floats(B, N, C), device="cuda")
    calls = [(False, False, lambda: la.la_forward_gated_scan(d["A"], d["X"], form="logit")),
             (False, True, lambda: la.la_forward_gated_scan(d["A"], d["X"], form="logit", ckpt=ck)),
             (True, True, lambda: la.la_backward_gated_scan(d["A"], d["X"], d["G"], form="logit", Ckpt=ck)),
             (True, False, lambda: la.la_backward_gated_scan(d["A"], d["X"], d["G"], form="logit"))]
    for backward, given, call in calls:
        want = la.la_gated_scan_workspace_bytes(B, N, C, DT[dt], backward=backward, ckpt_given=given)
        assert (want == 0) == (N == 100)  # one tile: no chain, no scratch
        torch.cuda.synchronize()
        la.la_scratch_peak_bytes(reset=True)
        call()
        torch.cuda.synchronize()
        assert want <= la.la_scratch_peak_bytes() <= want + 2 * (2 << 20)
