"""Measured cases of the gated scan and of the paged key-value cache.

Operators:
  scan         gated linear recurrence over packed or batched rows: forward, forward + backward
  scan_step    its single-token form
  page_map     block table, slot map and sequence starts from request lengths
  append       rows of keys and values into the pages of the cache, by slot
  paged        attention of one new token over the paged cache

With `own` false, run() computes the plain form: elementary torch operations in 32 bits, rounded once
at the end; with `own` true it makes the library's calls.  exact() follows the definitions in 64 bits,
one token or one request at a time.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_ES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of 256 sequences, 16 heads x 64 channels: the decode workload's batch
        {"name": "scan_step_256x1024_bf16", "op": "scan_step", "B": 256, "C": 1024, "dtype": "bf16",
         "form": "logit"},
        # training step of a recurrent layer: the training workload's rows (B 4, N 8192, 16 x 64 channels)
        {"name": "scan_train_bf16", "op": "scan", "B": 4, "N": 8192, "C": 1024, "dtype": "bf16",
         "form": "logit", "backward": True, "seqs": 0, "pad": 0},
        # the long-sequence workload's rows (N 65536, 16 x 128 channels), forward with its final state
        {"name": "scan_long_bf16", "op": "scan", "B": 1, "N": 65536, "C": 2048, "dtype": "bf16",
         "form": "decay", "backward": False, "seqs": 0, "pad": 0},
        # ragged documents packed into one row axis, an odd channel count, rows behind the last one
        {"name": "scan_packed_train_f32", "op": "scan", "B": 1, "N": 5003, "C": 1001, "dtype": "f32",
         "form": "decay", "backward": True, "seqs": 17, "pad": 77},
        # one decode step's bookkeeping for a small batch: latency
        {"name": "page_map_step_64", "op": "page_map", "R": 64, "page": 16, "max_cached": 4095,
         "max_new": 1, "pad": 0},
        # a large admission: prompts of up to 2048 tokens beside running requests
        {"name": "page_map_prefill_512", "op": "page_map", "R": 512, "page": 16, "max_cached": 2048,
         "max_new": 2048, "pad": 1000},
        # a short prompt's keys and values into the cache
        {"name": "append_300x8x128_f32", "op": "append", "T": 300, "Hkv": 8, "D": 128, "page": 16,
         "dtype": "f32"},
        # prefill of the decode workload's prompts (16 heads x 64), 64 prompts of 2048 tokens at once
        {"name": "append_131072x16x64_bf16", "op": "append", "T": 131072, "Hkv": 16, "D": 64, "page": 16,
         "dtype": "bf16"},
        # a few requests with short contexts: latency
        {"name": "paged_small_bf16", "op": "paged", "R": 4, "Hq": 16, "Hkv": 4, "D": 64, "page": 16,
         "min_len": 5, "max_len": 299, "window": 0, "append": True, "dtype": "bf16"},
        # the decode workload (256 sequences x 16 heads, 4096 positions), one key head per query head
        {"name": "paged_256x16_4096_bf16", "op": "paged", "R": 256, "Hq": 16, "Hkv": 16, "D": 64,
         "page": 16, "min_len": 4095, "max_len": 4095, "window": 0, "append": True, "dtype": "bf16"},
        # a few long contexts with shared key heads: the split over the length carries the parallelism
        {"name": "paged_long_gqa_bf16", "op": "paged", "R": 6, "Hq": 32, "Hkv": 4, "D": 128, "page": 64,
         "min_len": 9000, "max_len": 65535, "window": 0, "append": True, "dtype": "bf16"},
        # ragged fp32 batch, two query heads to a key head, a sliding window
        {"name": "paged_ragged_window_f32", "op": "paged", "R": 48, "Hq": 16, "Hkv": 8, "D": 64, "page": 32,
         "min_len": 0, "max_len": 8000, "window": 4096, "append": False, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "scan_step", "page_map", "append", "paged", "paged", "paged"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "scan_step":
        return {"op": op, "B": _log(rng, 1, 1024), "C": _log(rng, 16, 4096), "dtype": dtype,
                "form": rng.choice(["decay", "logit"])}
    if op == "scan":
        C = _log(rng, 16, 2048)
        if rng.random() < 0.6:
            C = max(64, C // 64 * 64)
        backward = rng.random() < 0.6
        seqs = rng.choice([0, 0, _log(rng, 2, 100)])
        most = 32_000_000 // C
        N = _log(rng, 1, min(65536, most)) if not seqs else _log(rng, 200, min(40000, most))
        B = 1 if seqs else min(_log(rng, 1, 16), max(1, most // N))
        return {"op": op, "B": B, "N": N, "C": C, "dtype": dtype, "form": rng.choice(["decay", "logit"]),
                "backward": backward, "seqs": seqs, "pad": rng.choice([0, rng.randint(1, 99)]) if seqs else 0}
    if op == "page_map":
        return {"op": op, "R": _log(rng, 1, 512), "page": rng.choice([8, 16, 32, 64]),
                "max_cached": rng.choice([0, _log(rng, 1, 4096)]), "max_new": _log(rng, 1, 2048),
                "pad": rng.choice([0, rng.randint(1, 999)])}
    D = rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        return {"op": op, "T": _log(rng, 1, 65536), "Hkv": Hkv, "D": D, "page": rng.choice([8, 16, 32, 64, 128]),
                "dtype": dtype}
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    R = _log(rng, 1, 256)
    most = max(2, min(65535, 500_000_000 // (R * Hkv * D)))
    max_len = _log(rng, 1, most)
    append = rng.random() < 0.7
    return {"op": op, "R": R, "Hq": group * Hkv, "Hkv": Hkv, "D": D, "page": rng.choice([8, 16, 32, 64, 128]),
            "min_len": rng.choice([0, max_len, rng.randint(0, max_len)]), "max_len": max_len,
            "window": rng.choice([0, 0, _log(rng, 1, 5000)]), "append": append, "dtype": dtype}


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced, whatever the seed (their order is the seed's)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _seq_lens(case):
    """Lengths of the packed sequences: they sum to N - pad, from empty to twice the mean."""
    S, total = case["seqs"], case["N"] - case["pad"]
    w = _spread(0, 1000, S) if S > 1 else [1]
    lens = [total * x // sum(w) for x in w]
    lens[-1] += total - sum(lens)
    return lens


# ------------------------------------------------------------------ inputs

def _shuffled(values, seed):
    return np.random.RandomState(seed % (1 << 31)).permutation(np.array(values, dtype=np.int64)).astype(np.int32)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case}

    def randn(*shape, dtype, scale=1.0, shift=0.0):
        return torch.randn(shape, generator=g, device=dev).mul_(scale).add_(shift).to(dtype)

    def gates(*shape, dtype):
        if case["form"] == "logit":  # sigmoid about 0.5 to 0.99
            return randn(*shape, dtype=dtype, scale=1.5, shift=2.0)
        return torch.rand(shape, generator=g, device=dev).mul_(0.15).add_(0.85).to(dtype)

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    op = case["op"]
    if op == "scan_step":
        dt = _DT[case["dtype"]]
        s["a"] = gates(case["B"], case["C"], dtype=dt)
        s["x"] = randn(case["B"], case["C"], dtype=dt)
        s["h"] = randn(case["B"], case["C"], dtype=torch.float32)  # the pass moves it on by a token
    elif op == "scan":
        dt, B, N, C = _DT[case["dtype"]], case["B"], case["N"], case["C"]
        s["a"] = gates(B, N, C, dtype=dt)
        s["x"] = randn(B, N, C, dtype=dt)
        s["starts"], S = None, B
        if case["seqs"]:
            S = case["seqs"]
            s["starts"] = ints(np.concatenate([[0], np.cumsum(_shuffled(_seq_lens(case), seed))]).astype(np.int32))
        s["h0"] = randn(S, C, dtype=torch.float32)
        s["out"] = torch.zeros((B, N, C), dtype=dt, device=dev)
        if case["backward"]:
            s["g"] = randn(B, N, C, dtype=dt)
            s["dh"] = randn(S, C, dtype=torch.float32)
            s["da"], s["dx"] = torch.zeros_like(s["a"]), torch.zeros_like(s["x"])
    elif op == "page_map":
        R, page = case["R"], case["page"]
        cached = _shuffled(_spread(0, case["max_cached"], R), seed)
        new = _shuffled(_spread(min(1, case["max_new"]), case["max_new"], R), seed + 1)
        old = -(-cached // page)
        need = -(-(cached + new) // page)
        W = -(-(case["max_cached"] + case["max_new"]) // page) + 3
        P = int(need.sum()) + 61
        order = np.random.RandomState((seed + 2) % (1 << 31)).permutation(P).astype(np.int32)
        table = np.full((R, W), -1, np.int32)
        at = 0
        for r in range(R):
            table[r, :old[r]] = order[at:at + old[r]]
            at += old[r]
        s["cached"], s["new"], s["free"] = ints(cached), ints(new), ints(order[at:])
        s["table"] = ints(table)
        s["pages"], s["tokens"] = P, int(new.sum()) + case["pad"]
        s["slots"] = torch.empty(s["tokens"], dtype=torch.int32, device=dev)
        s["starts"] = torch.empty(R + 1, dtype=torch.int32, device=dev)
        s["counts"] = torch.empty(2, dtype=torch.int32, device=dev)
    elif op == "append":
        dt, T, H, D, page = _DT[case["dtype"]], case["T"], case["Hkv"], case["D"], case["page"]
        P = -(-T // page) + 3
        s["k"], s["v"] = randn(T, H, D, dtype=dt), randn(T, H, D, dtype=dt)
        s["K"], s["V"] = randn(P, H, page, D, dtype=dt), randn(P, H, page, D, dtype=dt)
        order = np.random.RandomState(seed % (1 << 31)).permutation(P)[:-(-T // page)]
        i = np.arange(T)
        s["slots"] = ints((order[i // page] * page + i % page).astype(np.int32))
    else:
        dt, R, Hkv, D, page = _DT[case["dtype"]], case["R"], case["Hkv"], case["D"], case["page"]
        lens = _shuffled(_spread(case["min_len"], case["max_len"], R), seed)
        need = -(-(lens + (1 if case["append"] else 0)) // page)
        W, P = int(max(need.max(), 1)) + 2, int(need.sum()) + 3
        order = np.random.RandomState((seed + 1) % (1 << 31)).permutation(P).astype(np.int32)
        table = np.full((R, W), -1, np.int32)
        at = 0
        for r in range(R):
            table[r, :need[r]] = order[at:at + need[r]]
            at += need[r]
        s["lens"], s["table"] = ints(lens), ints(table)
        s["q"] = randn(R, case["Hq"], D, dtype=dt)
        s["k"], s["v"] = randn(R, Hkv, D, dtype=dt), randn(R, Hkv, D, dtype=dt)
        s["K"], s["V"] = randn(P, Hkv, page, D, dtype=dt), randn(P, Hkv, page, D, dtype=dt)
    return s


# ------------------------------------------------------------------ plain forms

def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from a zero state, by doubling the reach of each row."""
    n, d = a.shape[1], 1
    while d < n:
        h = b.clone()
        h[:, d:] += a[:, d:] * b[:, :-d]
        b = h
        if 2 * d < n:
            p = a.clone()
            p[:, d:] *= a[:, :-d]
            a = p
        d *= 2
    return b


def _plain_scan(s):
    c = s["case"]
    B, N, C, dt = c["B"], c["N"], c["C"], _DT[c["dtype"]]
    a, x = s["a"].float(), s["x"].float()
    if c["form"] == "logit":
        a = 1 / (1 + torch.exp(-a))
        b = (1 - a) * x
    else:
        b = x
    rows = torch.arange(N, device=a.device)
    if s["starts"] is None:
        first = (rows == 0).view(1, N, 1)
        last = (rows == N - 1).view(1, N, 1)
        valid = None
        h0 = s["h0"].view(B, 1, C)
        begin, end = torch.zeros(1, dtype=torch.long, device=a.device), torch.full((1,), N - 1, device=a.device)
    else:
        starts = s["starts"].long()
        S = starts.numel() - 1
        seq = (torch.searchsorted(starts, rows, right=True) - 1).clamp_(0, S - 1)
        first = (rows == starts[seq]).view(1, N, 1)
        last = (rows == starts[seq + 1] - 1).view(1, N, 1)
        valid = (rows < starts[-1]).view(1, N, 1)
        h0 = s["h0"][seq].view(1, N, C)
        begin, end = starts[:-1], starts[1:] - 1
        some = (starts[1:] > starts[:-1]).view(S, 1)
    zero = torch.zeros((), device=a.device)
    keep = torch.where(first, zero, a)
    h = _doubling(keep, b + torch.where(first, a * h0, zero))
    out = h if valid is None else torch.where(valid, h, s["out"].float())
    if s["starts"] is None:
        final = h[:, -1]
    else:
        final = torch.where(some, h[0, end.clamp(min=0)], s["h0"])
    got = {"out": out.to(dt), "final": final.clone()}
    if not c["backward"]:
        return got
    g = s["g"].float()
    dh = s["dh"].view(B, 1, C) if s["starts"] is None else s["dh"][seq].view(1, N, C)
    g = g + torch.where(last, dh, zero)
    nxt = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1)
    if s["starts"] is not None:
        nxt = torch.where(last, zero, nxt)
    G = _doubling(nxt.flip(1), g.flip(1)).flip(1)
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    prev = torch.where(first, h0.expand_as(h), prev)
    if c["form"] == "logit":
        da, dx = a * (1 - a) * G * (prev - x), (1 - a) * G
    else:
        da, dx = G * prev, G
    if s["starts"] is None:
        d0 = a[:, 0] * G[:, 0]
    else:
        da = torch.where(valid, da, s["da"].float())
        dx = torch.where(valid, dx, s["dx"].float())
        at = begin.clamp(max=N - 1)
        d0 = torch.where(some, a[0, at] * G[0, at], s["dh"])
    got.update(da=da.to(dt), dx=dx.to(dt), d0=d0)
    return got


def _plain_scan_step(s):
    a, x = s["a"].float(), s["x"].float()
    if s["case"]["form"] == "logit":
        a = 1 / (1 + torch.exp(-a))
        x = (1 - a) * x
    s["h"].mul_(a).add_(x)
    return {"out": s["h"].to(s["x"].dtype), "h": s["h"]}


def _plain_page_map(s):
    c, page = s["case"], s["case"]["page"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    old, need = (cached + page - 1) // page, (cached + new + page - 1) // page
    starts = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    taken = (need - old).cumsum(0)
    cols = torch.arange(table.shape[1], device=table.device).view(1, -1)
    fresh = (cols >= old.view(-1, 1)) & (cols < need.view(-1, 1))
    at = (taken - (need - old)).view(-1, 1) + cols - old.view(-1, 1)
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    rows = torch.arange(s["tokens"], device=table.device)
    req = (torch.searchsorted(starts, rows, right=True) - 1).clamp_(0, c["R"] - 1)
    pos = cached[req] + rows - starts[req]
    col = (pos // page).clamp(0, table.shape[1] - 1)
    slots = torch.where(rows < starts[-1], table[req, col].long() * page + pos % page, -1)
    counts = torch.stack([starts[-1], taken[-1]])
    return {"table": table, "slots": slots.to(torch.int32), "starts": starts.to(torch.int32),
            "counts": counts.to(torch.int32)}


def _plain_append(s):
    page, slots = s["case"]["page"], s["slots"].long()
    s["K"][slots // page, :, slots % page] = s["k"]
    s["V"][slots // page, :, slots % page] = s["v"]
    return {"K": s["K"], "V": s["V"]}


def _plain_paged(s):
    c = s["case"]
    R, Hq, Hkv, D, page = c["R"], c["Hq"], c["Hkv"], c["D"], c["page"]
    lens = s["lens"].long()
    total = lens
    if c["append"]:
        at = torch.gather(s["table"].long(), 1, (lens // page).view(R, 1)).view(R)
        s["K"][at, :, lens % page] = s["k"]
        s["V"][at, :, lens % page] = s["v"]
        total = lens + 1
    idx = s["table"].long().clamp(min=0)
    L = idx.shape[1] * page
    K = s["K"][idx].transpose(1, 2).reshape(R, Hkv, L, D).float()
    S = torch.matmul(s["q"].float().view(R, Hkv, Hq // Hkv, D), K.transpose(2, 3)) / math.sqrt(D)
    del K
    pos = torch.arange(L, device=S.device).view(1, 1, 1, L)
    end = total.view(R, 1, 1, 1)
    seen = pos < end
    if c["window"]:
        seen = seen & (pos >= end - c["window"])
    S = torch.where(seen, S, torch.full((), -math.inf, device=S.device))
    m = S.amax(3, keepdim=True)
    e = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
    del S
    V = s["V"][idx].transpose(1, 2).reshape(R, Hkv, L, D).float()
    V = torch.where(seen.view(R, 1, L, 1), V, torch.zeros((), device=V.device))
    t = e.sum(3, keepdim=True)
    out = torch.matmul(e, V) / torch.where(t > 0, t, torch.ones_like(t))
    lse = (m + torch.log(t)).view(R, Hq)
    return {"out": out.reshape(R, Hq, D), "lse": lse, "K": s["K"], "V": s["V"]}


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "scan":
            return _plain_scan(s)
        if op == "scan_step":
            return _plain_scan_step(s)
        if op == "page_map":
            return _plain_page_map(s)
        if op == "append":
            return _plain_append(s)
        return _plain_paged(s)
    import linear_attention_02_gb300 as la
    if op == "scan_step":
        out = la.la_gated_scan_decode_step(s["a"], s["x"], s["h"], form=c["form"])
        return {"out": out, "h": s["h"]}
    if op == "scan":
        S = c["seqs"] if c["seqs"] else c["B"]
        if not c["backward"]:
            out, final = la.la_forward_gated_scan(s["a"], s["x"], form=c["form"], h_init=s["h0"],
                                                  seq_starts=s["starts"], out=s["out"], return_state=True)
            return {"out": out, "final": final}
        ckpt = torch.empty(la.la_gated_scan_ckpt_floats(c["B"], c["N"], c["C"]), dtype=torch.float32,
                           device=s["a"].device)
        out, final = la.la_forward_gated_scan(s["a"], s["x"], form=c["form"], h_init=s["h0"],
                                              seq_starts=s["starts"], out=s["out"], return_state=True,
                                              ckpt=ckpt)
        da, dx, d0 = la.la_backward_gated_scan(s["a"], s["x"], s["g"], form=c["form"], h_init=s["h0"],
                                               dh_final=s["dh"], return_dh_init=True, Ckpt=ckpt,
                                               seq_starts=s["starts"], dA=s["da"], dX=s["dx"])
        return {"out": out, "final": final, "da": da, "dx": dx, "d0": d0}
    if op == "page_map":
        la.la_page_map(s["cached"], s["new"], s["free"], s["table"], c["page"], s["pages"], s["slots"],
                       s["starts"], s["counts"])
        return {"table": s["table"], "slots": s["slots"], "starts": s["starts"], "counts": s["counts"]}
    if op == "append":
        la.la_paged_append(s["k"], s["v"], s["K"], s["V"], s["slots"])
        return {"K": s["K"], "V": s["V"]}
    k, v = (s["k"], s["v"]) if c["append"] else (None, None)
    out, lse = la.la_paged_decode_step(s["q"], k, v, s["K"], s["V"], s["table"], s["lens"],
                                       window=c["window"], return_lse=True)
    return {"out": out, "lse": lse, "K": s["K"], "V": s["V"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "scan_step":
        n = c["B"] * c["C"]
        return {"bytes": n * (3 * _ES[c["dtype"]] + 8), "flops": 2 * n}
    if op == "scan":
        S = c["seqs"] if c["seqs"] else c["B"]
        n = (c["B"] * c["N"] - c["pad"]) * c["C"]
        streams = 3 + (5 if c["backward"] else 0)
        states = S * c["C"] * 4 * (2 + (3 if c["backward"] else 0))
        return {"bytes": n * streams * _ES[c["dtype"]] + states, "flops": n * (2 + (8 if c["backward"] else 0))}
    if op == "page_map":
        new = _spread(min(1, c["max_new"]), c["max_new"], c["R"])
        cached = _spread(0, c["max_cached"], c["R"])
        pages = sum(-(-(a + b) // c["page"]) + (-a // c["page"]) for a, b in zip(cached, new))
        return {"bytes": 4 * (3 * c["R"] + 2 * max(0, pages) + sum(new) + c["pad"]), "flops": 0}
    if op == "append":
        return {"bytes": c["T"] * (4 * c["Hkv"] * c["D"] * _ES[c["dtype"]] + 4), "flops": 0}
    more = 1 if c["append"] else 0
    seen = 0
    for n in _spread(c["min_len"], c["max_len"], c["R"]):
        seen += min(n + more, c["window"]) if c["window"] else n + more
    es = _ES[c["dtype"]]
    rows = c["R"] * c["Hq"]
    return {"bytes": seen * 2 * c["Hkv"] * c["D"] * es + rows * (c["D"] * (es + 4) + 4)
            + more * c["R"] * 4 * c["Hkv"] * c["D"] * es - more * c["R"] * 2 * c["Hkv"] * c["D"] * es,
            "flops": seen * c["Hq"] * c["D"] * 4}


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    s, c, f = prepare(case, seed), case, torch.float64
    op = c["op"]
    if op == "scan_step":
        a, x, h = s["a"].to(f), s["x"].to(f), s["h"].to(f)
        h = torch.sigmoid(a) * h + torch.sigmoid(-a) * x if c["form"] == "logit" else a * h + x
        return {"out": h, "h": h}
    if op == "scan":
        return _exact_scan(s)
    if op == "page_map":
        return _exact_page_map(s)
    if op == "append":
        page = c["page"]
        for i, slot in enumerate(s["slots"].tolist()):
            s["K"][slot // page, :, slot % page] = s["k"][i]
            s["V"][slot // page, :, slot % page] = s["v"][i]
        return {"K": s["K"], "V": s["V"]}
    return _exact_paged(s)


def _exact_scan(s):
    c, f = s["case"], torch.float64
    B, N = c["B"], c["N"]
    a, x = s["a"].to(f), s["x"].to(f)
    logit = c["form"] == "logit"
    sg, co = (torch.sigmoid(a), torch.sigmoid(-a)) if logit else (a, None)
    b = co * x if logit else x
    # (batch row or 0, first token, one past the last, state) of every sequence
    if s["starts"] is None:
        seqs = [(slice(0, B), 0, N, slice(0, B))]
    else:
        st = s["starts"].tolist()
        seqs = [(slice(0, 1), st[i], st[i + 1], slice(i, i + 1)) for i in range(len(st) - 1)]
    out, final = s["out"].to(f), s["h0"].to(f).clone()
    for rows, t0, t1, st in seqs:
        h = s["h0"][st].to(f)
        for t in range(t0, t1):
            h = torch.addcmul(b[rows, t], sg[rows, t], h)
            out[rows, t] = h
        final[st] = h
    got = {"out": out, "final": final}
    if not c["backward"]:
        return got
    g = s["g"].to(f)
    G, prev, d0 = torch.zeros_like(g), torch.zeros_like(g), s["dh"].to(f).clone()
    da, dx = s["da"].to(f), s["dx"].to(f)
    for rows, t0, t1, st in seqs:
        carry = s["dh"][st].to(f)
        for t in range(t1 - 1, t0 - 1, -1):
            tot = g[rows, t] + carry
            G[rows, t] = tot
            carry = sg[rows, t] * tot
        d0[st] = carry
        if t1 > t0:
            prev[rows, t0] = s["h0"][st].to(f)
            prev[rows, t0 + 1:t1] = out[rows, t0:t1 - 1]
            r = (rows, slice(t0, t1))
            da[r] = sg[r] * co[r] * G[r] * (prev[r] - x[r]) if logit else G[r] * prev[r]
            dx[r] = co[r] * G[r] if logit else G[r]
    got.update(da=da, dx=dx, d0=d0)
    return got


def _exact_page_map(s):
    page = s["case"]["page"]
    cached, new, free = s["cached"].tolist(), s["new"].tolist(), s["free"].tolist()
    table, slots, starts, used = s["table"].cpu().numpy().copy(), [], [0], 0
    for r, (have, more) in enumerate(zip(cached, new)):
        for p in range(have, have + more):
            if p % page == 0:  # the position opens a page
                table[r, p // page] = free[used]
                used += 1
            slots.append(int(table[r, p // page]) * page + p % page)
        starts.append(len(slots))
    counts = np.array([len(slots), used], np.int32)
    slots += [-1] * (s["tokens"] - len(slots))
    return {"table": table, "slots": np.array(slots, np.int32), "starts": np.array(starts, np.int32),
            "counts": counts}


def _exact_paged(s):
    c, f = s["case"], torch.float64
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    out = torch.zeros((c["R"], Hq, D), dtype=f, device=s["q"].device)
    lse = torch.full((c["R"], Hq), -math.inf, dtype=f, device=s["q"].device)
    for r, n in enumerate(lens):
        if c["append"]:
            s["K"][table[r][n // page], :, n % page] = s["k"][r]
            s["V"][table[r][n // page], :, n % page] = s["v"][r]
            n += 1
        n0 = max(0, n - c["window"]) if c["window"] else 0
        if n == n0:
            continue
        pages = torch.tensor(table[r][n0 // page:(n - 1) // page + 1], device=out.device)
        cut = slice(n0 - n0 // page * page, n - n0 // page * page)
        K = s["K"][pages].to(f).transpose(0, 1).reshape(Hkv, -1, D)[:, cut]
        V = s["V"][pages].to(f).transpose(0, 1).reshape(Hkv, -1, D)[:, cut]
        q = s["q"][r].to(f).view(Hkv, Hq // Hkv, D)
        x = torch.einsum("hgd,hnd->hgn", q, K) / math.sqrt(D)
        out[r] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, 2), V).reshape(Hq, D)
        lse[r] = torch.logsumexp(x, 2).reshape(Hq)
    return {"out": out, "lse": lse, "K": s["K"], "V": s["V"]}
