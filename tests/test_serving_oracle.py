"""Pins of the fp64 plain forms of the gated scan and the paged cache
(oracle/serving.py): hand-derived values, torch autograd, central differences
and closed forms."""
import numpy as np
import torch

from oracle import serving as ref


def test_scan_hand_values():
    # decay: h = 0.5 * 2 + 1 = 2, then 0.25 * 2 - 1 = -0.5
    out, final, prev = ref.gated_scan_forward([[[0.5], [0.25]]], [[[1.0], [-1.0]]], "decay", [[2.0]])
    assert out.ravel().tolist() == [2.0, -0.5] and final.ravel().tolist() == [-0.5]
    assert prev.ravel().tolist() == [2.0, 2.0]
    # logit 0: s = 1/2, h = (0 + 4) / 2 = 2, then (2 + 6) / 2 = 4
    out, _, _ = ref.gated_scan_forward([[[0.0], [0.0]]], [[[4.0], [6.0]]], "logit")
    assert out.ravel().tolist() == [2.0, 4.0]
    # backward of the first: g2 = 1, g1 = 1 + 0.25; da = g * h_prev; dh0 = 0.5 g1
    dA, dX, d0 = ref.gated_scan_backward([[[0.5], [0.25]]], [[[1.0], [-1.0]]], [[[1.0], [1.0]]], "decay",
                                         [[2.0]])
    assert dX.ravel().tolist() == [1.25, 1.0] and dA.ravel().tolist() == [2.5, 2.0]
    assert d0.ravel().tolist() == [0.625]


def _torch_scan(a, x, form, h0, starts):
    s, c = (a, 1.0) if form == "decay" else (torch.sigmoid(a), torch.sigmoid(-a))
    b = c * x
    outs, finals = [], []
    seqs = [(i, 0, a.shape[1]) for i in range(a.shape[0])] if starts is None else \
        [(0, starts[i], starts[i + 1]) for i in range(len(starts) - 1)]
    for i, (r, t0, t1) in enumerate(seqs):
        h = h0[i]
        for t in range(t0, t1):
            h = s[r, t] * h + b[r, t]
            outs.append(h)
        finals.append(h)
    return torch.stack(outs), torch.stack(finals)


def test_scan_backward_matches_autograd_and_differences():
    g = torch.Generator().manual_seed(1)
    for form in ("decay", "logit"):
        for B, N, C, starts in ((2, 7, 3, None), (1, 9, 2, [0, 4, 4, 9])):
            S = B if starts is None else len(starts) - 1
            a = torch.rand(B, N, C, generator=g, dtype=torch.float64).requires_grad_()
            x = torch.randn(B, N, C, generator=g, dtype=torch.float64).requires_grad_()
            h0 = torch.randn(S, C, generator=g, dtype=torch.float64).requires_grad_()
            G = torch.randn(B, N, C, generator=g, dtype=torch.float64)
            dh = torch.randn(S, C, generator=g, dtype=torch.float64)
            o, f = _torch_scan(a, x, form, h0, starts)
            ((o * G.reshape(-1, C)).sum() + (f * dh).sum()).backward()
            out, final, _ = ref.gated_scan_forward(a, x, form, h0, starts)
            dA, dX, d0 = ref.gated_scan_backward(a, x, G, form, h0, dh, starts)
            np.testing.assert_allclose(out.reshape(-1, C), o.detach(), rtol=1e-12, atol=1e-12)
            np.testing.assert_allclose(final, f.detach(), rtol=1e-12, atol=1e-12)
            for got, want in ((dA, a.grad), (dX, x.grad), (d0, h0.grad)):
                np.testing.assert_allclose(got, want, rtol=1e-10, atol=1e-12)

            def loss(da, dx):
                o, f, _ = ref.gated_scan_forward(a.detach().numpy() + da, x.detach().numpy() + dx, form, h0, starts)
                return (o * G.numpy()).sum() + (f * dh.numpy()).sum()

            u = torch.randn(B, N, C, generator=g, dtype=torch.float64).numpy()
            e = 1e-5
            np.testing.assert_allclose((loss(e * u, 0) - loss(-e * u, 0)) / (2 * e), (dA * u).sum(), rtol=1e-6)
            np.testing.assert_allclose((loss(0, e * u) - loss(0, -e * u)) / (2 * e), (dX * u).sum(), rtol=1e-6)


def test_scan_constant_decay_is_geometric():
    out, _, _ = ref.gated_scan_forward(np.full((1, 30, 1), 0.5), np.ones((1, 30, 1)))
    np.testing.assert_allclose(out.ravel(), 2 * (1 - 0.5 ** np.arange(1, 31)), rtol=1e-14)


def test_page_map_hand_values():
    # page 4: request 0 holds 3 of page 9 and gets 3 (one more page), request 1 gets none, request 2 opens two
    table, slots, starts, counts, bad = ref.page_map([3, 4, 0], [3, 0, 5], [7, 2, 5], [[9, -1], [1, -1], [-1, -1]],
                                                     4, 10, 10)
    assert table.tolist() == [[9, 7], [1, -1], [2, 5]] and not bad
    assert slots.tolist() == [39, 28, 29, 8, 9, 10, 11, 20, -1, -1]
    assert starts.tolist() == [0, 3, 3, 8] and counts.tolist() == [8, 3]
    # the free list ends: entry and slots -1
    table, slots, _, counts, bad = ref.page_map([0], [5], [7], [[-1, -1]], 4, 10, 5)
    assert table.tolist() == [[7, -1]] and slots.tolist() == [28, 29, 30, 31, -1] and bad
    assert counts.tolist() == [5, 2]


def test_page_map_rows_without_a_request():
    table, slots, starts, counts, bad = ref.page_map([4, -1, 0], [1, 0, 1], [7, 2], [[9, -1], [5, 5], [-1, -1]], 4, 10, 3)
    assert table.tolist() == [[9, 7], [5, 5], [2, -1]] and not bad
    assert slots.tolist() == [28, 8, -1] and starts.tolist() == [0, 1, 1, 2] and counts.tolist() == [2, 2]
    assert ref.page_map([-1], [1], [7], [[-1]], 4, 10, 1)[4]


def test_paged_decode_against_softmax():
    g = np.random.RandomState(2)
    P, Hkv, page, D, Hq = 6, 2, 4, 8, 4
    K, V = g.randn(P, Hkv, page, D), g.randn(P, Hkv, page, D)
    q, k, v = g.randn(2, Hq, D), g.randn(2, Hkv, D), g.randn(2, Hkv, D)
    table, lens = [[3, 0, 5], [1, -1, -1]], [9, 0]
    out, lse = ref.paged_decode(q, k, v, K, V, table, lens)
    flatK = np.concatenate([K[i] for i in table[0]], axis=1)[:, :9]
    flatV = np.concatenate([V[i] for i in table[0]], axis=1)[:, :9]
    for h in range(Hq):
        ks, vs = np.vstack([flatK[h // 2], k[0, h // 2]]), np.vstack([flatV[h // 2], v[0, h // 2]])
        x = torch.tensor(ks @ q[0, h] / np.sqrt(D))
        np.testing.assert_allclose(out[0, h], torch.softmax(x, 0).numpy() @ vs, rtol=1e-12)
        np.testing.assert_allclose(lse[0, h], float(torch.logsumexp(x, 0)), rtol=1e-12)
        np.testing.assert_allclose(out[1, h], v[1, h // 2], rtol=1e-12)  # only its own row
    # a window of one position is the new row alone; no position: zeros and -infinity
    np.testing.assert_allclose(ref.paged_decode(q, k, v, K, V, table, lens, window=1)[0][0, 3], v[0, 1])
    out, lse = ref.paged_decode(q, None, None, K, V, table, [0, -1])
    assert not out[0].any() and np.all(np.isneginf(lse[0])) and np.isnan(out[1]).all()


def test_append_places_rows():
    K = np.zeros((3, 1, 2, 1))
    k = np.arange(1.0, 4.0).reshape(3, 1, 1)
    K2, _ = ref.paged_append(k, k, K, K, [5, -1, 0])
    assert K2.ravel().tolist() == [3, 0, 0, 0, 0, 1]
