"""Measured cases of the rotary positions, of the norms with the rotation in the same pass, and of
the attention of a chunk of new tokens over the paged key-value cache.

Operators:
  rotary       positions of queries and keys as rotations: forward, forward + backward
  norm_rotary  root-mean-square norm of every query and key head, then the rotation: the same
  prefill      softmax attention of each request's new tokens over its pages

With `own` false, run() computes the plain form: elementary torch operations in 32 bits (angles in 64),
rounded once at the end; with `own` true it makes the library's calls.  exact() follows the definitions
in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_ES = {"f32": 4, "bf16": 2}
_EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of 256 sequences with shared key heads: the step before a decode step, latency
        {"name": "rotary_step_256x16x64_bf16", "op": "rotary", "B": 0, "N": 256, "Hq": 16, "Hk": 4, "D": 64,
         "rot": 64, "layout": "half", "scaling": "none", "factor": 1.0, "max_pos": 4095, "fused": True,
         "backward": False, "dtype": "bf16"},
        # the training workload's queries and keys (B 4, H 16, N 8192, D 64), forward and backward
        {"name": "rotary_train_bf16", "op": "rotary", "B": 4, "N": 8192, "Hq": 16, "Hk": 16, "D": 64,
         "rot": 64, "layout": "half", "scaling": "none", "factor": 1.0, "max_pos": 8191, "fused": False,
         "backward": True, "dtype": "bf16"},
        # packed rows at far positions, a part of the head, frequencies scaled by parts for a long context
        {"name": "rotary_far_part_f32", "op": "rotary", "B": 0, "N": 5003, "Hq": 12, "Hk": 4, "D": 64,
         "rot": 20, "layout": "interleaved", "scaling": "by_parts", "factor": 32.0, "max_pos": 1000000,
         "fused": False, "backward": True, "dtype": "f32"},
        # a few requests' next tokens
        {"name": "norm_rotary_step_4x32x128_bf16", "op": "norm_rotary", "B": 0, "N": 4, "Hq": 32, "Hk": 4,
         "D": 128, "rot": 128, "layout": "half", "scaling": "none", "factor": 1.0, "max_pos": 65535,
         "fused": True, "backward": False, "dtype": "bf16"},
        # the training workload's queries and keys with learned norms: gradients of inputs and weights
        {"name": "norm_rotary_train_bf16", "op": "norm_rotary", "B": 4, "N": 8192, "Hq": 16, "Hk": 16, "D": 64,
         "rot": 64, "layout": "half", "scaling": "none", "factor": 1.0, "max_pos": 8191, "fused": False,
         "backward": True, "dtype": "bf16"},
        # prompts packed into one row axis, cut out of a joint projection: prefill of long contexts
        {"name": "norm_rotary_prompt_65536x32x128_bf16", "op": "norm_rotary", "B": 0, "N": 65536, "Hq": 32,
         "Hk": 4, "D": 128, "rot": 128, "layout": "half", "scaling": "base", "factor": 8.0,
         "max_pos": 131071, "fused": True, "backward": False, "dtype": "bf16"},
        # ragged fp32 rows, half of the head rotated in adjacent pairs
        {"name": "norm_rotary_part_train_f32", "op": "norm_rotary", "B": 0, "N": 3001, "Hq": 24, "Hk": 8,
         "D": 128, "rot": 64, "layout": "interleaved", "scaling": "linear", "factor": 4.0, "max_pos": 16383,
         "fused": True, "backward": True, "dtype": "f32"},
        # a few short prompts beside short contexts: latency
        {"name": "prefill_small_bf16", "op": "prefill", "R": 4, "Hq": 16, "Hkv": 4, "D": 64, "page": 16,
         "min_new": 3, "max_new": 48, "min_cached": 0, "max_cached": 200, "window": 0, "pad": 0, "dtype": "bf16"},
        # prefill of the decode workload's prompts (16 heads x 64), 32 prompts of 2048 tokens
        {"name": "prefill_32x2048x16x64_bf16", "op": "prefill", "R": 32, "Hq": 16, "Hkv": 16, "D": 64, "page": 16,
         "min_new": 2048, "max_new": 2048, "min_cached": 0, "max_cached": 0, "window": 0, "pad": 0,
         "dtype": "bf16"},
        # chunks of long prompts over what is already cached, shared key heads
        {"name": "prefill_long_chunk_bf16", "op": "prefill", "R": 2, "Hq": 32, "Hkv": 4, "D": 128, "page": 64,
         "min_new": 2000, "max_new": 2048, "min_cached": 30000, "max_cached": 63000, "window": 0, "pad": 48,
         "dtype": "bf16"},
        # a few drafted tokens of many requests checked at once: read-bound, split over the length
        {"name": "prefill_draft_48_bf16", "op": "prefill", "R": 48, "Hq": 32, "Hkv": 4, "D": 128, "page": 16,
         "min_new": 1, "max_new": 8, "min_cached": 500, "max_cached": 16000, "window": 0, "pad": 0,
         "dtype": "bf16"},
        # ragged fp32 prompts, two query heads to a key head, a sliding window
        {"name": "prefill_ragged_window_f32", "op": "prefill", "R": 13, "Hq": 16, "Hkv": 8, "D": 64, "page": 32,
         "min_new": 0, "max_new": 700, "min_cached": 0, "max_cached": 3000, "window": 1000, "pad": 5,
         "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "norm_rotary", "norm_rotary", "prefill", "prefill", "prefill", "prefill"])
    dtype = rng.choice(["f32", "bf16"])
    D = rng.choice([32, 64, 128])
    if op != "prefill":
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 3, 4, 8])
        B = rng.choice([0, 0, _log(rng, 1, 16)])
        most = 100_000_000 // ((Hq + Hk) * D * max(B, 1))
        return {"op": op, "B": B, "N": _log(rng, 1, max(1, min(65536, most))), "Hq": Hq, "Hk": Hk, "D": D,
                "rot": rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "by_parts"]),
                "factor": rng.choice([1.5, 4.0, 32.0]), "max_pos": _log(rng, 1, 1 << 20),
                "fused": B == 0 and rng.random() < 0.5, "backward": rng.random() < 0.6, "dtype": dtype}
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 6, 8, 16])
    R = _log(rng, 1, 64)
    max_new = _log(rng, 1, max(1, min(4096, 80_000_000 // (R * Hkv * G * D))))
    cells = 1e12 / (R * max_new * Hkv * G * D * 4)      # positions that the pass's products leave room for
    max_cached = rng.choice([0, _log(rng, 1, int(max(2, min(65535, cells - max_new, 2.5e8 / (R * Hkv * D)))))])
    return {"op": op, "R": R, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "page": rng.choice([8, 16, 32, 64, 128]),
            "min_new": rng.choice([0, 1, max_new]) if max_new > 1 else 1, "max_new": max_new,
            "min_cached": rng.choice([0, max_cached]), "max_cached": max_cached,
            "window": rng.choice([0, 0, _log(rng, 1, 5000)]), "pad": rng.choice([0, rng.randint(1, 99)]),
            "dtype": dtype}


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced, whatever the seed (their order is the seed's)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


# ------------------------------------------------------------------ inputs

def _shuffled(values, seed):
    return np.random.RandomState(seed % (1 << 31)).permutation(np.array(values, dtype=np.int64)).astype(np.int32)


def _scaling(c):
    """Arguments of the frequencies: the original length that "by_parts" refers to is a power of two."""
    return {"base": 10000.0, "scaling": c["scaling"], "factor": c["factor"], "original_len": 4096,
            "beta_fast": 32.0, "beta_slow": 1.0}


def prepare(case, seed):
    dev, c = "cuda", case
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": c}
    dt = _DT[c["dtype"]]

    def randn(*shape, dtype=dt, scale=1.0, shift=0.0):
        return torch.randn(shape, generator=g, device=dev).mul_(scale).add_(shift).to(dtype)

    if c["op"] == "prefill":
        R, Hkv, D, page = c["R"], c["Hkv"], c["D"], c["page"]
        new = _shuffled(_spread(c["min_new"], c["max_new"], R), seed)
        cached = _shuffled(_spread(c["min_cached"], c["max_cached"], R), seed + 1)
        need = -(-(cached + new) // page)
        W, P = int(max(need.max(), 1)) + 2, int(need.sum()) + 3
        order = np.random.RandomState((seed + 2) % (1 << 31)).permutation(P).astype(np.int32)
        table, at = np.full((R, W), -1, np.int32), 0
        for r in range(R):
            table[r, :need[r]] = order[at:at + need[r]]
            at += need[r]
        s["new"], s["had"] = new.tolist(), cached.tolist()  # the host's copy, as a scheduler has it
        s["table"], s["cached"] = torch.from_numpy(table).to(dev), torch.from_numpy(cached).to(dev)
        s["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev)
        T = int(new.sum()) + c["pad"]
        s["q"] = randn(T, c["Hq"], D)
        s["K"], s["V"] = randn(P, Hkv, page, D), randn(P, Hkv, page, D)
        s["out"] = torch.zeros((T, c["Hq"], D), dtype=dt, device=dev)
        s["lse"] = torch.zeros((T, c["Hq"]), dtype=torch.float32, device=dev)
        return s

    B, N, Hq, Hk, D = c["B"], c["N"], c["Hq"], c["Hk"], c["D"]
    if B == 0:  # packed rows [N][H][D], each request's positions counted on from where it stood
        if c["fused"]:  # queries and keys as columns of a joint projection with values behind them
            x = randn(N, (Hq + 2 * Hk) * D)
            s["q"] = x[:, :Hq * D].view(N, Hq, D)
            s["k"] = x[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D)
        else:
            s["q"], s["k"] = randn(N, Hq, D), randn(N, Hk, D)
        r = np.random.RandomState(seed % (1 << 31))
        run = max(1, min(N, 1024))
        first = r.randint(0, c["max_pos"] + 1, -(-N // run))
        pos = np.minimum(first[np.arange(N) // run] + np.arange(N) % run, c["max_pos"])
        s["pos"] = torch.from_numpy(pos.astype(np.int32)).to(dev)
    else:       # rows [B][H][N][D] of a training step, positions from 0
        s["q"], s["k"], s["pos"] = randn(B, Hq, N, D), randn(B, Hk, N, D), None
    if c["backward"]:
        s["gq"], s["gk"] = randn(*s["q"].shape), randn(*s["k"].shape)
    if c["op"] == "norm_rotary":
        s["wq"], s["wk"] = (randn(D, dtype=torch.float32, scale=0.1, shift=1.0) for _ in range(2))
    if own:
        import linear_attention_02_gb300 as la
        s["freqs"], s["mag"] = la.la_rotary_frequencies(c["rot"], device=dev, **_scaling(c))
    else:
        s["freqs"], s["mag"] = _frequencies(c, dev)
    return s


# ------------------------------------------------------------------ plain forms

def _frequencies(c, dev):
    """Angles a position in 64 bits, and the factor on the rotated elements."""
    a, rot, f = _scaling(c), c["rot"], c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    theta, mag = a["base"] ** (-2 * i / rot), 1.0
    if c["scaling"] == "linear":
        theta = theta / f
    elif c["scaling"] == "base":
        theta = (a["base"] * f ** (rot / (rot - 2) if rot > 2 else 1.0)) ** (-2 * i / rot)
    elif c["scaling"] == "by_parts":
        turns = a["original_len"] * theta / (2 * math.pi)
        keep = ((turns - a["beta_slow"]) / (a["beta_fast"] - a["beta_slow"])).clamp(0, 1)
        theta, mag = theta * keep + theta / f * (1 - keep), 0.1 * math.log(f) + 1
    return theta, mag


def _cos_sin(s, x):
    """Factors of a rotation for x [.., N, H, D] or [B, H, N, D]."""
    N = s["case"]["N"]
    pos = torch.arange(N, device=x.device) if s["pos"] is None else s["pos"]
    a = pos.double().view(N, 1) * s["freqs"]
    a = a.view(N, 1, -1) if x.dim() == 3 else a.view(1, 1, N, -1)
    return torch.cos(a).float() * s["mag"], torch.sin(a).float() * s["mag"]


def _turn(x, cos, sin, c):
    """The rotation of x in 32 bits."""
    rot = c["rot"]
    out = x.clone()
    if c["layout"] == "half":
        a, b = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        a, b = slice(0, rot, 2), slice(1, rot, 2)
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., a] * sin + x[..., b] * cos
    return out


def _plain_rotary(s):
    c, got = s["case"], {}
    for n in ("q", "k"):
        x = s[n]
        cos, sin = _cos_sin(s, x)
        y = x.float()
        if c["op"] == "norm_rotary":
            w = s["w" + n]
            r = torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS)
            y = y * r * w
        got[n] = _turn(y, cos, sin, c).to(x.dtype)
        if c["backward"]:
            g = _turn(s["g" + n].float(), cos, -sin, c)
            if c["op"] == "norm_rotary":
                xf = x.float()
                h = g * w
                got["dw" + n] = (g * xf * r).double().sum(tuple(range(x.dim() - 1))).float()
                g = r * h - xf * (r * r * r) * (xf * h).mean(-1, keepdim=True)
            got["d" + n] = g.to(x.dtype)
    return got


def _plain_prefill(s):
    c = s["case"]
    Hq, Hkv, D, page, win = c["Hq"], c["Hkv"], c["D"], c["page"], c["window"]
    G, row = Hq // Hkv, 0
    for r, (n, had) in enumerate(zip(s["new"], s["had"])):
        if n == 0:
            continue
        first = max(0, had - win + 1) if win else 0     # what the first new token sees
        p0, total = first // page, had + n
        idx = s["table"][r, p0:-(-total // page)].long()
        K = s["K"][idx].transpose(0, 1).reshape(Hkv, -1, D)[:, :total - p0 * page].float()
        V = s["V"][idx].transpose(0, 1).reshape(Hkv, -1, D)[:, :total - p0 * page].float()
        L = K.shape[1]
        q = s["q"][row:row + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3)  # [Hkv, G, n, D]
        at = torch.arange(had, had + n, device=q.device).view(n, 1)
        pos = torch.arange(p0 * page, total, device=q.device).view(1, L)
        seen = pos <= at
        if win:
            seen = seen & (pos > at - win)
        each = max(1, min(Hkv, 1_500_000_000 // (G * n * L)))  # key heads at once, by memory
        for h in range(0, Hkv, each):
            x = torch.matmul(q[h:h + each].reshape(-1, G * n, D), K[h:h + each].transpose(1, 2))
            x = x.view(-1, G, n, L).div_(math.sqrt(D))
            x = torch.where(seen, x, torch.full((), -math.inf, device=x.device))
            m = x.amax(3, keepdim=True)
            x = torch.exp(x.sub_(m))
            t = x.sum(3, keepdim=True)
            o = torch.matmul(x.view(-1, G * n, L), V[h:h + each]).view(-1, G, n, D) / t
            b = slice(h * G, (h + o.shape[0]) * G)
            s["out"][row:row + n, b] = o.permute(2, 0, 1, 3).reshape(n, -1, D).to(s["out"].dtype)
            s["lse"][row:row + n, b] = (m + torch.log(t)).permute(2, 0, 1, 3).reshape(n, -1)
        row += n
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_prefill(s) if c["op"] == "prefill" else _plain_rotary(s)
    import linear_attention_02_gb300 as la
    if c["op"] == "prefill":
        out, lse = la.la_paged_prefill(s["q"], s["K"], s["V"], s["table"], s["cached"], s["starts"],
                                       window=c["window"], out=s["out"], lse=s["lse"], return_lse=True)
        return {"out": out, "lse": lse}
    kw = {"positions": s["pos"], "layout": c["layout"], "magnitude": s["mag"]}
    if c["op"] == "rotary":
        q, k = la.la_forward_rotary(s["q"], s["k"], s["freqs"], **kw)
        got = {"q": q, "k": k}
        if c["backward"]:
            got["dq"], got["dk"] = la.la_backward_rotary(s["gq"], s["gk"], s["freqs"], **kw)
        return got
    q, k = la.la_forward_norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["freqs"], eps=_EPS, **kw)
    got = {"q": q, "k": k}
    if c["backward"]:
        got["dq"], got["dk"], got["dwq"], got["dwk"] = la.la_backward_norm_rotary(
            s["q"], s["k"], s["gq"], s["gk"], s["wq"], s["wk"], s["freqs"], eps=_EPS, **kw)
    return got


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, es = case, _ES[case["dtype"]]
    if c["op"] != "prefill":
        tokens = max(c["B"], 1) * c["N"]
        n = tokens * (c["Hq"] + c["Hk"]) * c["D"]
        norm = c["op"] == "norm_rotary"
        streams, flops = 2, 3 + (4 if norm else 0)
        if c["backward"]:  # the norm's backward reads its input again
            streams += 3 if norm else 2
            flops += 3 + (9 if norm else 0)
        return {"bytes": n * streams * es + (4 * tokens if c["B"] == 0 else 0), "flops": n * flops}
    # every pairing of lengths has the same sums but for the order of the seed: pairs in the mean
    new, had = _spread(c["min_new"], c["max_new"], c["R"]), _spread(c["min_cached"], c["max_cached"], c["R"])
    pairs = keys = 0.0
    for n in new:
        for h in had:
            w = c["window"] or h + n
            full = max(0, min(n, h + n - w))  # tokens that see the whole window
            part = n - full
            pairs += full * w + part * h + part * (part + 1) / 2 if n else 0
            keys += min(h + n, w + n - 1) if n else 0
    pairs, keys, T = pairs / c["R"], keys / c["R"], sum(new)
    return {"bytes": int(keys * 2 * c["Hkv"] * c["D"] * es + T * c["Hq"] * (2 * c["D"] * es + 4)),
            "flops": int(pairs * c["Hq"] * c["D"] * 4)}


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    s, c, f = prepare(case, seed), case, torch.float64
    if c["op"] == "prefill":
        return _exact_prefill(s)
    rot, N, dev = c["rot"], c["N"], s["q"].device
    sc = _scaling(c)
    theta, mag = [], 1.0
    for i in range(rot // 2):
        base = sc["base"]
        if c["scaling"] == "base":
            base *= math.pow(c["factor"], rot / (rot - 2) if rot > 2 else 1.0)
        t = math.exp(-2 * i / rot * math.log(base))
        if c["scaling"] == "linear":
            t /= c["factor"]
        elif c["scaling"] == "by_parts":
            turns = sc["original_len"] * t / (2 * math.pi)
            ramp = (turns - sc["beta_slow"]) / (sc["beta_fast"] - sc["beta_slow"])
            ramp = min(1.0, max(0.0, ramp))
            t = (1 - ramp) * (t / c["factor"]) + ramp * t
        theta.append(t)
    if c["scaling"] == "by_parts":
        mag = 1 + 0.1 * math.log(c["factor"])
    pos = torch.arange(N, device=dev) if s["pos"] is None else s["pos"]
    angle = torch.outer(pos.to(f), torch.tensor(theta, dtype=f, device=dev))
    z = torch.polar(torch.full_like(angle, mag), angle)
    got = {}

    def pairs(x):  # [..., rot] to complex pairs
        x = x.view(*x.shape[:-1], 2, rot // 2).transpose(-1, -2) if c["layout"] == "half" else \
            x.view(*x.shape[:-1], rot // 2, 2)
        return torch.view_as_complex(x.contiguous())

    def turned(x, w):
        head = torch.view_as_real(pairs(x[..., :rot].contiguous()) * w)
        head = head.transpose(-1, -2) if c["layout"] == "half" else head
        return torch.cat([head.reshape(*x.shape[:-1], rot), x[..., rot:]], -1)

    for n in ("q", "k"):
        x = s[n].to(f)
        zz = z.view(N, 1, -1) if x.dim() == 3 else z.view(1, 1, N, -1)
        if c["op"] == "rotary":
            got[n] = turned(x, zz)
            if c["backward"]:
                got["d" + n] = turned(s["g" + n].to(f), zz.conj())
            continue
        w = s["w" + n].to(f)
        size = torch.sqrt(x.square().sum(-1, keepdim=True) / c["D"] + _EPS)
        got[n] = turned(x / size * w, zz)
        if c["backward"]:
            g = turned(s["g" + n].to(f), zz.conj())
            unit = x / size
            got["dw" + n] = torch.einsum("rd,rd->d", g.reshape(-1, c["D"]), unit.reshape(-1, c["D"]))
            h = g * w
            got["d" + n] = (h - unit * (unit * h).sum(-1, keepdim=True) / c["D"]) / size
    return got


def _exact_prefill(s):
    c, f = s["case"], torch.float64
    if work(c)["flops"] > 6e12:
        return None
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    out, lse = s["out"].to(f), s["lse"].to(f)
    row = 0
    for r, (n, had) in enumerate(zip(s["new"], s["had"])):
        pages = s["table"][r, :-(-(had + n) // page)].long()
        for t0 in range(0, n, 256):  # 256 of its tokens at once
            t1 = min(n, t0 + 256)
            q = s["q"][row + t0:row + t1].to(f)
            lo = max(0, had + t0 + 1 - c["window"]) if c["window"] else 0
            hi = had + t1
            pg = pages[lo // page:(hi - 1) // page + 1]
            cut = slice(lo % page, lo % page + hi - lo)
            at = torch.arange(had + t0, had + t1, device=q.device)[:, None]
            pos = torch.arange(lo, hi, device=q.device)[None]
            hide = (pos > at) | (pos <= at - c["window"] if c["window"] else pos < 0)
            for h in range(Hq):
                g = h // (Hq // Hkv)
                K, V = s["K"][pg, g].to(f).reshape(-1, D)[cut], s["V"][pg, g].to(f).reshape(-1, D)[cut]
                x = (q[:, h] @ K.T / math.sqrt(D)).masked_fill_(hide, -math.inf)
                out[row + t0:row + t1, h] = torch.softmax(x, 1) @ V
                lse[row + t0:row + t1, h] = torch.logsumexp(x, 1)
        row += n
    return {"out": out, "lse": lse}
