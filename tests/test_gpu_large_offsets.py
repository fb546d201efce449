"""Rotary calls and the prefill where offsets pass 2^31 elements: the far rows and pages give what they give alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _la():
    import linear_attention_02_gb300 as la
    return la


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [True, False])
def test_rotary_rows(packed, dt):
    la = _la()
    H, D, few = 32, 128, 37
    N = 2 ** 31 // (H * D) + few
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.zeros((N, H, D) if packed else (1, H, N, D), device="cuda", dtype=DT[dt])
    far = (lambda t: t[-few:]) if packed else (lambda t: t[:, :, -few:])
    for part in (far(q), q[:few] if packed else q[:, :, :few]):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    assert q.numel() > 2 ** 31
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    freqs, _ = la.la_rotary_frequencies(D)
    x, first = far(q).clone(), N - few
    want = la.la_forward_rotary(x, None, freqs, first_position=first)[0]
    wn = la.la_forward_norm_rotary(x, None, w, None, freqs, first_position=first)[0]
    wd, _, wdw, _ = la.la_backward_norm_rotary(x, None, x, None, w, None, freqs, first_position=first)
    assert torch.equal(far(la.la_forward_rotary(q, None, freqs)[0]), want)
    assert torch.equal(far(la.la_forward_norm_rotary(q, None, w, None, freqs)[0]), wn)
    dq, _, dw, _ = la.la_backward_norm_rotary(q, None, q, None, w, None, freqs)
    assert torch.equal(far(dq), wd)
    near = q[:few] if packed else q[:, :, :few].contiguous()
    sums = wdw + la.la_backward_norm_rotary(near, None, near, None, w, None, freqs)[2]  # rows of zeros add nothing
    # |g| of a pair is at most |x0| + |x1|, u = x r; n terms in any order are off by n 2^-24 of their absolute sum, a
    # term itself by its 16 or so roundings
    size = 0
    for t in (x, near):
        t = t.double()
        u = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)
        size = size + ((t.abs() + t.abs().roll(D // 2, -1)) * u.abs()).reshape(-1, D).sum(0)
    assert bool(((dw - sums).double().abs() <= (2 * few * H + 16) * 2.0 ** -24 * size).all())
    la.la_forward_rotary(q, None, freqs, q_out=q)
    assert torch.equal(far(q), want)
    la.la_check_device_status()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("page", [4, 64])
def test_prefill_pages(page, dt):
    la = _la()
    Hq, Hkv, D, cached, new = 16, 8, 128, [300, 40], [20, 150]
    need = [-(-(c + n) // page) for c, n in zip(cached, new)]
    n = sum(need)
    P = 2 ** 31 // (Hkv * page * D) + 2 * n
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dt])  # noqa: E731
    q, Ks, Vs = rand(sum(new), Hq, D), rand(n, Hkv, page, D), rand(n, Hkv, page, D)
    K, V = (torch.zeros((P, Hkv, page, D), device="cuda", dtype=DT[dt]) for _ in range(2))
    K[P - n:], V[P - n:] = Ks, Vs
    W = max(need)
    table = torch.full((2, W), -1, dtype=torch.int32)
    table[0, :need[0]], table[1, :need[1]] = torch.arange(need[0]), torch.arange(need[0], n)
    far = torch.where(table >= 0, table + P - n, table).cuda()
    lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
    want = la.la_paged_prefill(q, Ks, Vs, table.cuda(), lens, starts, return_lse=True)
    got = la.la_paged_prefill(q, K, V, far, lens, starts, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    la.la_check_device_status()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_prefill_rows(dt):
    # one token of very many requests, over a common beginning
    la = _la()
    Hq, Hkv, D, page, few = 32, 4, 128, 16, 50
    R = 2 ** 31 // (Hq * D) + few
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dt])  # noqa: E731
    K, V = rand(2, Hkv, page, D), rand(2, Hkv, page, D)
    q = torch.zeros((R + 3, Hq, D), device="cuda", dtype=DT[dt])
    q[-few - 3:] = rand(few + 3, Hq, D)
    i32 = lambda n: torch.ones(n, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda").repeat(R, 1)
    starts = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    out, lse = la.la_paged_prefill(q, K, V, table, 20 * i32(R), starts, return_lse=True)
    want, wl = la.la_paged_prefill(q[-few - 3:].clone(), K, V, table[:few], 20 * i32(few), starts[:few + 1], return_lse=True)
    assert torch.equal(out[-few - 3:], want) and torch.equal(lse[-few - 3:], wl)
    assert bool((out[-3:] == 0).all()) and bool(torch.isneginf(lse[-3:]).all())
    la.la_check_device_status()
