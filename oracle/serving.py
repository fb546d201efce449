"""fp64 plain forms of the gated scan, of the paged key-value cache and of the rotary positions.

Written from the definitions, one row, position or request at a time, on numpy
arrays; used by the tests only.  Packed sequences are given by `starts`
(starts[i] .. starts[i+1] - 1 are sequence i's rows of a one-row batch).
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


def _gates(A, form):
    """(decay, factor on x) of every element."""
    A = _f64(A)
    if form == "decay":
        return A, np.ones_like(A)
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-A)), 1 / (1 + np.exp(A))


def _sequences(B, N, starts):
    """(batch row, first row, end) of every sequence."""
    if starts is None:
        return [(b, 0, N) for b in range(B)]
    return [(0, int(starts[i]), int(starts[i + 1])) for i in range(len(starts) - 1)]


def gated_scan_forward(A, X, form="decay", h_init=None, starts=None):
    """(Out, h_final, h_prev): h_prev[t] is the state before row t.  Rows of no sequence are NaN."""
    s, c = _gates(A, form)
    X, h_init = _f64(X), _f64(h_init)
    B, N, C = X.shape
    seqs = _sequences(B, N, starts)
    out, prev = np.full((B, N, C), np.nan), np.full((B, N, C), np.nan)
    final = np.zeros((len(seqs), C))
    for i, (b, t0, t1) in enumerate(seqs):
        h = np.zeros(C) if h_init is None else h_init[i].copy()
        for t in range(t0, t1):
            prev[b, t] = h
            h = s[b, t] * h + c[b, t] * X[b, t]
            out[b, t] = h
        final[i] = h
    return out, final, prev


def gated_scan_backward(A, X, dOut, form="decay", h_init=None, dh_final=None, starts=None):
    """(dA, dX, dh_init); rows of no sequence are NaN."""
    _, _, prev = gated_scan_forward(A, X, form, h_init, starts)
    s, c = _gates(A, form)
    X, dOut, dh_final = _f64(X), _f64(dOut), _f64(dh_final)
    B, N, C = X.shape
    seqs = _sequences(B, N, starts)
    dA, dX = np.full((B, N, C), np.nan), np.full((B, N, C), np.nan)
    d0 = np.zeros((len(seqs), C))
    for i, (b, t0, t1) in enumerate(seqs):
        carry = np.zeros(C) if dh_final is None else dh_final[i].copy()
        for t in range(t1 - 1, t0 - 1, -1):
            g = dOut[b, t] + carry
            dX[b, t] = c[b, t] * g
            dA[b, t] = g * prev[b, t] if form == "decay" else s[b, t] * c[b, t] * g * (prev[b, t] - X[b, t])
            carry = s[b, t] * g
        d0[i] = carry
    return dA, dX, d0


def page_map(cached, new, free, table, page, num_pages, max_tokens):
    """(table, slots, starts, counts, bad): la_page_map on lists of whole numbers."""
    table = np.array(table, dtype=np.int64)
    W = table.shape[1]
    slots, starts, used, bad = [], [0], 0, False
    for r, (have, more) in enumerate(zip(cached, new)):
        bad |= more < 0 or (have < 0 and more > 0) or have + more > W * page
        have, more = min(max(have, 0), W * page), max(more, 0)
        for p in range(have, have + more):
            if p >= W * page:
                slots.append(-1)
                continue
            if p % page == 0:
                i = free[used] if used < len(free) else -1
                ok = 0 <= i < num_pages
                bad |= not ok
                table[r, p // page] = i if ok else -1
                used += 1
            i = int(table[r, p // page])
            ok = 0 <= i < num_pages
            bad |= not ok
            slots.append(i * page + p % page if ok else -1)
        starts.append(len(slots))
    counts = [len(slots), used]
    bad |= len(slots) > max_tokens
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return table, np.array(slots), np.array(starts), np.array(counts), bool(bad)


def paged_append(k, v, K, V, slots):
    """The pools (copies) with row t of k, v in slot slots[t]."""
    K, V, k, v = _f64(K).copy(), _f64(V).copy(), _f64(k), _f64(v)
    page = K.shape[2]
    for t, s in enumerate(slots):
        if 0 <= s < K.shape[0] * page:
            K[s // page, :, s % page], V[s // page, :, s % page] = k[t], v[t]
    return K, V


def paged_decode(q, k, v, K, V, table, lens, window=0, scale=None):
    """(out, lse) over the pools as they are before the step; rows with a negative length are NaN.
    Positions on a page outside the pool are left out."""
    q, K, V = _f64(q), _f64(K), _f64(V)
    k, v = _f64(k), _f64(v)
    R, Hq, D = q.shape
    P, Hkv, page, _ = K.shape
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, lse = np.full((R, Hq, D), np.nan), np.full((R, Hq), np.nan)
    for r in range(R):
        n = int(lens[r])
        if n < 0:
            continue
        n = min(n, len(table[r]) * page)
        total = n + (k is not None)
        first = max(0, total - window) if window else 0
        at = [(int(table[r][p // page]), p % page) for p in range(first, min(n, total))]
        at = [(i, o) for i, o in at if 0 <= i < P]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            ks = [K[i, g, o] for i, o in at] + ([k[r, g]] if k is not None else [])
            vs = [V[i, g, o] for i, o in at] + ([v[r, g]] if k is not None else [])
            if not ks:
                out[r, h], lse[r, h] = 0, -np.inf
                continue
            x = scale * (np.array(ks) @ q[r, h])
            m = x.max()
            w = np.exp(x - m)
            out[r, h] = w @ np.array(vs) / w.sum()
            lse[r, h] = m + np.log(w.sum())
    return out, lse


def paged_prefill(q, K, V, table, lens, starts, window=0, scale=None):
    """(out, lse, size): size is the weighted mean of |v| of every output; rows of no request are NaN.
    Positions on a page outside the pool are left out."""
    q, K, V = _f64(q), _f64(K), _f64(V)
    T, Hq, D = q.shape
    P, Hkv, page, _ = K.shape
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, size, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    for r in range(len(lens)):
        if int(lens[r]) < 0:
            continue
        a, b = int(starts[r]), int(starts[r + 1])
        for t in range(a, b):
            pos = int(lens[r]) + t - a
            first = max(0, pos - window + 1) if window else 0
            at = [(int(table[r][p // page]), p % page) for p in range(first, min(pos + 1, len(table[r]) * page))]
            at = [(i, o) for i, o in at if 0 <= i < P]
            if not at:
                out[t], size[t], lse[t] = 0, 0, -np.inf
                continue
            i, o = np.array(at).T
            k, v = K[i, :, o], V[i, :, o]  # [positions, Hkv, D]
            for h in range(Hq):
                g = h // (Hq // Hkv)
                x = scale * (k[:, g] @ q[t, h])
                m = x.max()
                w = np.exp(x - m)
                out[t, h], size[t, h] = w @ v[:, g] / w.sum(), w @ np.abs(v[:, g]) / w.sum()
                lse[t, h] = m + np.log(w.sum())
    return out, lse, size


def rotary_theta(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(angles a position [rot / 2], magnitude)."""
    i = np.arange(rot // 2)
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    theta = np.array([float(base) ** (-2.0 * j / rot) for j in i])
    if scaling == "linear":
        theta = theta / factor
    if scaling == "by_parts":
        g = np.clip((original_len * theta / (2 * np.pi) - beta_slow) / (beta_fast - beta_slow), 0, 1)
        theta = theta * (g + (1 - g) / factor)
    return theta, 1 + 0.1 * np.log(factor) if scaling == "by_parts" else 1.0


def rotary_angles(freqs, positions):
    """Angles [.., rot / 2] of whole-number positions, from frequencies in 2^-64 turns: whole numbers, so exact
    until the last step."""
    f = [int(x) % (1 << 64) for x in freqs]
    pos = np.asarray(positions)
    a = [[2 * np.pi * ((int(p) * u % (1 << 64)) / 2.0 ** 64) for u in f] for p in pos.reshape(-1)]
    return np.array(a).reshape(*pos.shape, len(f))


def rotary(x, angles, layout="half", magnitude=1.0):
    """Rows [.., D] turned by angles [.., rot / 2] that broadcast against them."""
    x = _f64(x)
    n = angles.shape[-1]
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y = x.copy()
    c, s = magnitude * np.cos(angles), magnitude * np.sin(angles)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def norm_rotary(x, w, angles, layout="half", magnitude=1.0, eps=1e-6):
    x = _f64(x)
    w = 1.0 if w is None else _f64(w)
    return rotary(x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w, angles, layout, magnitude)


def norm_rotary_backward(x, dy, w, angles, layout="half", magnitude=1.0, eps=1e-6):
    """(dx, dw)."""
    x, w = _f64(x), 1.0 if w is None else _f64(w)
    g = rotary(dy, -angles, layout, magnitude)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u, h = x * r, g * w
    return r * (h - u * (u * h).mean(-1, keepdims=True)), (g * u).reshape(-1, x.shape[-1]).sum(0)
