"""GPU parity of the rotary positions, and of the norm before them, against their fp64 plain forms.

Tolerances, u = 2^-24.  An angle is an fp32 number within an eighth of a turn, off by half a unit of itself
(pi / 4 u at most) and by 2^-33 turns; its sine and cosine are off by 2 units in the last place at most (2 u,
values below 1); the magnitude, a product and the sum take u each:
    turned: 6 u magnitude (|x0| + |x1|).
A sum of D squares is off by at most D u of itself (all terms positive), so 1 / sqrt by D / 2 u and by the
rounding of mean, sum with eps, root and quotient (4 u); two products more: n is off by (D / 2 + 6) u of itself.
The gradient: each of the steps of r (h - a mean(a h)), a = x r, by the same rules; a sum over rows adds
the roundings of its longest chain of additions, below 400 here.  Outputs in bf16 are rounded once, by 2^-8.
"""
import math

import numpy as np
import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24


def _la():
    import linear_attention_02_gb300 as la
    return la


def _near(got, want, bound, dt):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= bound + HALF[dt] * (np.abs(want) + bound) + 1e-38)
    assert not bad.any(), f"{bad.sum()} of {bad.size}: off by {np.abs(got - want)[bad].max():.3g} at bound {bound[bad].min():.3g}"


def _abs_rotary(x, angles, layout, mag):
    """magnitude (|x0| + |x1|) of the turned elements, 0 of the others."""
    n = angles.shape[-1]
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y = np.zeros_like(x)
    y[..., a] = y[..., b] = mag * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y


def _angles(freqs, pos, shape, packed):
    """Angles that broadcast against rows [B,H,N,D] or [N,H,D]."""
    a = ref.rotary_angles(freqs.cpu().numpy().astype(np.int64), pos)  # [N, P] or [B, N, P]
    if packed:
        return a[:, None]
    return a[None, None] if a.ndim == 2 else a[:, None]


def _rand(shape, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dt])


SHAPES = [  # B (0: packed), N, Hq, Hk, D, rot
    (0, 1, 1, 1, 32, 32), (0, 5, 3, 1, 64, 64), (0, 300, 16, 4, 64, 64), (0, 7, 32, 4, 128, 128), (1, 1, 1, 1, 128, 2),
    (2, 33, 2, 2, 64, 32), (3, 129, 4, 2, 32, 16), (2, 500, 3, 1, 128, 64), (0, 77, 5, 5, 64, 20), (2, 19, 2, 1, 128, 126),
    (0, 1000, 8, 1, 32, 2), (0, 50, 3, 2, 64, 24), (2, 21, 2, 2, 128, 40)]


def _positions(kind, B, N, seed):
    r = np.random.RandomState(seed)
    if kind == "none":
        return None, np.arange(N) + 11
    if kind == "far":
        p = r.randint(0, 2 ** 31 - 1, N)
        p[0] = 2 ** 31 - 1
    elif kind == "rows":
        p = r.randint(0, 5000, (max(B, 1), N))
    else:
        p = r.randint(0, 5000, N)
    return torch.tensor(p.astype(np.int32)).cuda(), p


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,Hq,Hk,D,rot", SHAPES)
def test_rotary(B, N, Hq, Hk, D, rot, dt, layout):
    la = _la()
    packed = B == 0
    qs, ks = ((N, Hq, D), (N, Hk, D)) if packed else ((B, Hq, N, D), (B, Hk, N, D))
    q, k = _rand(qs, dt, N), _rand(ks, dt, N + 1)
    for kind in ("none", "far", "near") + (() if packed else ("rows",)):
        freqs, mag = la.la_rotary_frequencies(rot, scaling="by_parts" if kind == "far" else "none", factor=8.0, original_len=4096)
        pos, pn = _positions(kind, B, N, 5)
        kw = dict(positions=pos, layout=layout, magnitude=mag, first_position=11 if pos is None else 0)
        a = _angles(freqs, pn, qs, packed)
        m = np.float32(mag).astype(np.float64)
        got = la.la_forward_rotary(q.cuda(), k.cuda(), freqs, **kw)
        back = la.la_backward_rotary(q.cuda(), k.cuda(), freqs, **kw)
        for x, y, z in zip((q, k), got, back):
            x64 = x.double().numpy()
            tol = 6 * U * _abs_rotary(x64, a, layout, m)
            _near(y, ref.rotary(x64, a, layout, m), tol, dt)
            _near(z, ref.rotary(x64, -a, layout, m), tol, dt)
    la.la_check_device_status()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,rot", [(32, 8), (64, 20), (64, 32), (128, 2), (128, 40), (128, 62)])
def test_what_does_not_turn_is_kept(D, rot, dt, layout):
    # every element of the rest as it was, whatever lies beside it; the turned part does not notice
    la = _la()
    N, H = 19, 3
    x = _rand((N, H, D), dt, 7).cuda()
    freqs, mag = la.la_rotary_frequencies(rot, scaling="by_parts", factor=4.0, original_len=512)
    want, _ = la.la_forward_rotary(x, None, freqs, layout=layout, magnitude=mag)
    for what in (math.inf, -math.inf, math.nan, -0.0):
        y = x.clone()
        for n in range(N):
            y[n, :, rot + (5 * n) % (D - rot)] = what
        for f in (la.la_forward_rotary, la.la_backward_rotary):
            got, _ = f(y, None, freqs, layout=layout, magnitude=mag)
            a, b = got[..., rot:], y[..., rot:]  # a NaN stays one, in whichever of its bits
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0, math.inf, -math.inf), b.nan_to_num(0.0, math.inf, -math.inf))
            assert torch.equal(torch.signbit(a)[~a.isnan()], torch.signbit(b)[~b.isnan()])
        got, _ = la.la_forward_rotary(y, None, freqs, layout=layout, magnitude=mag)
        assert torch.equal(got[..., :rot], want[..., :rot])


def _norm_bounds(x, dy, w, a, layout, mag, eps):
    """(bound of y, bound of dx, bound of dw) of _abs values, by the rules above."""
    D = x.shape[-1]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = np.abs(x * r * w)
    e_r = (D / 2 + 4) * U
    by = (D / 2 + 12) * U * _abs_rotary(n, a, layout, mag)
    rest = _abs_rotary(n, a, layout, mag) == 0
    by[rest] = ((D / 2 + 6) * U * n)[rest]
    if dy is None:
        return by, None, None
    g = np.abs(ref.rotary(dy, -a, layout, mag))
    e_g = 6 * U * _abs_rotary(dy, a, layout, mag)
    u, h = np.abs(x * r), g * np.abs(w)
    e_u, e_h = (e_r + U) * u, e_g * np.abs(w) + U * h
    mean = np.abs((ref.rotary(dy, -a, layout, mag) * w * x * r).mean(-1, keepdims=True))
    e_m = (u * e_h + h * e_u + (D + 2) * U * u * h).mean(-1, keepdims=True) + U * mean
    inner = np.abs(ref.rotary(dy, -a, layout, mag) * w - x * r * (ref.rotary(dy, -a, layout, mag) * w * x * r).mean(-1, keepdims=True))
    bx = r * (e_h + u * e_m + e_u * mean + 2 * U * (h + u * mean)) + (e_r + U) * r * inner
    bw = (g * e_u + u * e_g + 401 * U * g * u).reshape(-1, D).sum(0)
    return by, bx * 1.01, bw * 1.01  # products of two errors


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,Hq,Hk,D,rot", SHAPES)
def test_norm_rotary(B, N, Hq, Hk, D, rot, dt, layout):
    la = _la()
    packed = B == 0
    qs, ks = ((N, Hq, D), (N, Hk, D)) if packed else ((B, Hq, N, D), (B, Hk, N, D))
    x = [_rand(qs, dt, N, 3.0), _rand(ks, dt, N + 1, 0.01)]
    g = [_rand(qs, dt, N + 2), _rand(ks, dt, N + 3)]
    x[0].view(-1, D)[0] = 0  # a row without anything
    w = [_rand((D,), "f32", 4), None]
    freqs, mag = la.la_rotary_frequencies(rot)
    pos, pn = _positions("near", B, N, 6)
    eps = 1e-5
    kw = dict(positions=pos, layout=layout, magnitude=1.25, eps=eps)
    wc = [None if t is None else t.cuda() for t in w]
    a = _angles(freqs, pn, qs, packed)
    y = la.la_forward_norm_rotary(x[0].cuda(), x[1].cuda(), *wc, freqs, **kw)
    *dx, dwq, dwk = la.la_backward_norm_rotary(x[0].cuda(), x[1].cuda(), g[0].cuda(), g[1].cuda(), *wc, freqs, **kw)
    la.la_check_device_status()
    e32 = float(np.float32(eps))
    for i, dw in enumerate((dwq, dwk)):
        x64, g64, w64 = x[i].double().numpy(), g[i].double().numpy(), 1.0 if w[i] is None else w[i].double().numpy()
        by, bx, bw = _norm_bounds(x64, g64, w64, a, layout, 1.25, e32)
        _near(y[i], ref.norm_rotary(x64, w64, a, layout, 1.25, e32), by, dt)
        wx, ww = ref.norm_rotary_backward(x64, g64, w64, a, layout, 1.25, e32)
        _near(dx[i], wx, bx, dt)
        _near(dw, ww, bw, "f32")


def test_norm_gradient_by_differences():
    # along one direction of inputs and weights: the loss sum(G y) of the fp64 plain form
    la = _la()
    q, k, G, H = (_rand((2, 2, 9, 32), "f32", s) for s in range(4))
    wq, wk = _rand((32,), "f32", 8), _rand((32,), "f32", 9)
    freqs, _ = la.la_rotary_frequencies(16)
    got = la.la_backward_norm_rotary(*(t.cuda() for t in (q, k, G, H, wq, wk)), freqs)
    a = _angles(freqs, np.arange(9), None, False)
    r = np.random.RandomState(1)
    for x, g, w, dx, dw in ((q, G, wq, got[0], got[2]), (k, H, wk, got[1], got[3])):
        x, g, w = x.double().numpy(), g.double().numpy(), w.double().numpy()
        vx, vw, h = r.randn(*x.shape), r.randn(32), 1e-5
        f = lambda s: (g * ref.norm_rotary(x + s * vx, w + s * vw, a)).sum()  # noqa: E731
        want = (f(h) - f(-h)) / (2 * h)
        mine = (dx.double().cpu().numpy() * vx).sum() + (dw.double().cpu().numpy() * vw).sum()
        scale = np.abs(dx.double().cpu().numpy() * vx).sum() + np.abs(dw.double().cpu().numpy() * vw).sum()
        # each gradient element is within 200 u of its size (the bounds above at D = 32), the quotient within h^2 of its terms
        assert abs(want - mine) <= (200 * U + 1e-8) * scale


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strided_rows_and_in_place(dt):
    la = _la()
    N, Hq, Hk, D = 37, 6, 2, 64
    freqs, _ = la.la_rotary_frequencies(D)
    x = _rand((N, (Hq + 2 * Hk) * D + 5), dt, 1).cuda()
    w = _rand((D,), "f32", 2).cuda()
    # rows in pieces and rows in single elements add up their squares in another order: each is within the
    # bound above of the plain form, with |n| <= sqrt(D) max |w|, and rounded once
    apart = 2 * (D / 2 + 12) * U * 2 * math.sqrt(D) * float(w.abs().max())
    for off in (0, 1, 8):  # whole pieces or single elements
        rows = x[:, off:off + (Hq + 2 * Hk) * D - (0 if off < 8 else D)]
        q, k = rows[:, :Hq * D].view(N, Hq, D), rows[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D)
        dense = [q.contiguous(), k.contiguous()]
        want = la.la_forward_norm_rotary(*dense, w, w, freqs)
        got = la.la_forward_norm_rotary(q, k, w, w, freqs)
        for a, b in zip(got, want):
            assert float((a.float() - b.float()).abs().max()) <= apart + 2 * HALF[dt] * float(b.float().abs().max())
        # in place, in the joint projection: the values behind are left alone
        y = x.clone()
        r2 = y[:, off:off + rows.shape[1]]
        q2, k2 = r2[:, :Hq * D].view(N, Hq, D), r2[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D)
        la.la_forward_norm_rotary(q2, k2, w, w, freqs, q_out=q2, k_out=k2)
        assert torch.equal(q2, got[0]) and torch.equal(k2, got[1])
        rest = torch.ones(x.shape[1], dtype=torch.bool)
        rest[off:off + (Hq + Hk) * D] = False
        assert torch.equal(y[:, rest], x[:, rest])
    # [B,N,H,D] memory as [B,H,N,D], heads of a gradient broadcast by a zero stride, and one batch row's stride
    q4 = _rand((2, 19, 4, D), dt, 3).cuda().transpose(1, 2)
    g4 = _rand((2, 1, 19, D), dt, 4).cuda().expand(2, 4, 19, D)
    a = la.la_backward_norm_rotary(q4, None, g4, None, w, None, freqs)
    b = la.la_backward_norm_rotary(q4.contiguous(), None, g4.contiguous(), None, w, None, freqs)
    assert torch.equal(a[0], b[0]) and a[1] is None and a[3] is None
    # the rows are summed up in the order of memory: the same terms, of 2 x 4 x 19 rows, |a| <= sqrt(D), each
    # sum within 400 u of its terms' sizes
    assert float((a[2] - b[2]).abs().max()) <= 2 * 400 * U * 152 * 2 * float(g4.abs().max()) * math.sqrt(D)
    with pytest.raises(ValueError, match="overlap"):
        la.la_forward_rotary(q4, None, freqs, q_out=g4)
    with pytest.raises(ValueError, match="adjacent"):
        la.la_forward_rotary(x[:, :128:2].unsqueeze(1), None, freqs)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_without_a_token(dt):
    la = _la()
    N, Hq, Hk, D = 50, 4, 2, 64
    q, k, g = _rand((N, Hq, D), dt, 1).cuda(), _rand((N, Hk, D), dt, 2).cuda(), _rand((N, Hq, D), dt, 3).cuda()
    gk = _rand((N, Hk, D), dt, 4).cuda()
    w = _rand((D,), "f32", 5).cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    pad = torch.zeros(N, dtype=torch.bool, device="cuda")
    pad[3], pad[40:] = True, True
    pos[pad] = -1
    freqs, _ = la.la_rotary_frequencies(D)
    live = ~pad
    want = la.la_backward_norm_rotary(q[live], k[live], g[live], gk[live], w, w, freqs, positions=pos[live].contiguous())
    q[pad], g[pad] = math.nan, math.inf  # nothing of these rows counts
    got = la.la_backward_norm_rotary(q, k, g, gk, w, w, freqs, positions=pos)
    assert torch.equal(got[0][live], want[0]) and torch.equal(got[1][live], want[1])
    for i in (2, 3):
        assert float((got[i] - want[i]).abs().max()) <= 400 * U * N * Hq * 6 and bool(torch.isfinite(got[i]).all())
    assert bool((got[0][pad] == 0).all())
    bad = torch.full((D,), math.nan, device="cuda")
    y, _ = la.la_forward_norm_rotary(q, k, bad, w, freqs, positions=pos)
    assert bool((y[pad] == 0).all())
    keep = torch.full_like(q, 9.5)
    out, _ = la.la_forward_rotary(q, k, freqs, positions=pos, q_out=keep)
    assert out is keep and bool((keep[pad] == 9.5).all()) and bool(torch.isfinite(keep[live]).all())


def test_empty_calls_and_single_sides():
    la = _la()
    freqs, _ = la.la_rotary_frequencies(64)
    e = torch.zeros(0, 4, 64, device="cuda")
    q, k = la.la_forward_rotary(e, e, freqs)
    assert q.shape == e.shape and k.shape == e.shape
    *_, dwq, dwk = la.la_backward_norm_rotary(e, e, e, e, None, None, freqs)
    assert float(dwq.abs().max()) == 0 and float(dwk.abs().max()) == 0
    x = _rand((3, 2, 64), "f32", 1).cuda()
    a, none = la.la_forward_rotary(x, None, freqs, first_position=5)
    none2, b = la.la_forward_rotary(None, x, freqs, first_position=5)
    assert none is None and none2 is None and torch.equal(a, b)


def test_weights_gradient_over_many_rows_is_repeatable():
    la = _la()
    x, g = _rand((4, 8, 3000, 64), "bf16", 1).cuda(), _rand((4, 8, 3000, 64), "bf16", 2).cuda()
    w = _rand((64,), "f32", 3).cuda()
    freqs, _ = la.la_rotary_frequencies(64)
    runs = [la.la_backward_norm_rotary(x, x, g, g, w, w, freqs) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))
    xd = x.double()
    a = torch.arange(3000, device="cuda").double()[:, None] * torch.tensor(ref.rotary_theta(64)[0], device="cuda")
    gd, c, s = g.double(), torch.cos(a), torch.sin(a)
    turned = torch.cat([gd[..., :32] * c + gd[..., 32:] * s, gd[..., 32:] * c - gd[..., :32] * s], -1)
    terms = turned * xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + 1e-6)
    want, size = terms.sum((0, 1, 2)), terms.abs().sum((0, 1, 2))
    # a side's rows over 152 blocks of 64: ten a thread (below 40 however they are dealt out); then 64, 5 and 5 additions:
    # within 128 u, and 50 u a term
    for dw in runs[0][2:]:
        assert bool(((dw.double() - want).abs() <= 178 * U * size).all())


def test_other_stream_and_captured_graph():
    la = _la()
    x = _rand((100, 8, 64), "bf16", 1).cuda()
    k = _rand((100, 2, 64), "bf16", 2).cuda()
    w = _rand((64,), "f32", 3).cuda()
    freqs, _ = la.la_rotary_frequencies(64)
    want = la.la_backward_norm_rotary(x, k, x, k, w, w, freqs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = la.la_backward_norm_rotary(x, k, x, k, w, w, freqs)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(la.la_backward_norm_rotary(x, k, x, k, w, w, freqs))
        graphs.append(gr)
    x2 = _rand((100, 8, 64), "bf16", 7).cuda()
    x.copy_(x2)
    want = la.la_backward_norm_rotary(x, k, x, k, w, w, freqs)
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_scratch_of_the_weights_gradient():
    la = _la()
    x = _rand((2000, 8, 128), "bf16", 1).cuda()
    freqs, _ = la.la_rotary_frequencies(128)
    la.la_backward_norm_rotary(x, x, x, x, None, None, freqs)
    torch.cuda.synchronize()
    from linear_attention_02_gb300 import _native
    _native.lib.la_scratch_peak_bytes(1)
    la.la_backward_norm_rotary(x, x, x, x, None, None, freqs)
    torch.cuda.synchronize()
    want = la.la_norm_rotary_workspace_bytes(1, 2000, 8, 8, 128)
    assert want <= _native.lib.la_scratch_peak_bytes(1) <= want + (2 << 20)
