"""GPU tests of what the paged decode step keeps of its values.

A request that sees one position has a weight of exactly 1 there, so its output is that
position's value row, bit for bit, in either storage type.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _la():
    import linear_attention_02_gb300 as la
    return la


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _values(g, shape, dt):
    """Normal numbers of every size, random in all bits, with the largest and some whole ones among them."""
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-60, 61, shape, generator=g).float())
    x.view(-1)[::7] = torch.randn(x.numel(), generator=g)[::7]
    x.view(-1)[::31] = torch.finfo(DT[dt]).max
    x.view(-1)[::37] = torch.finfo(DT[dt]).min
    x.view(-1)[::41] = 3.0
    x.view(-1)[::43] = 0.0
    return x.to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["append", "cached", "window"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(2, 2, 64, 16), (8, 1, 32, 16), (16, 1, 128, 16), (24, 2, 64, 4), (40, 1, 128, 32),
                                           (12, 12, 128, 64), (36, 3, 32, 8)])
def test_one_position_gives_its_value_row(Hq, Hkv, D, page, how, dt):
    la = _la()
    g = torch.Generator().manual_seed(Hq + D)
    R, W = 9, 128 // page + 1
    P = R * W
    table = torch.randperm(P, generator=g).view(R, W)
    q = torch.randn(R, Hq, D, generator=g).to(DT[dt])
    k, K = torch.randn(R, Hkv, D, generator=g).to(DT[dt]), torch.randn(P, Hkv, page, D, generator=g).to(DT[dt])
    v, V = _values(g, (R, Hkv, D), dt), _values(g, (P, Hkv, page, D), dt)
    lens = {"append": [0] * R, "cached": [1] * R, "window": [1, 2, 15, 16, 17, 40, 63, 64, 100]}[how]
    new = (k.cuda(), v.cuda()) if how == "append" else (None, None)
    out, lse = la.la_paged_decode_step(q.cuda(), *new, K.cuda(), V.cuda(), _i32(table.tolist()), _i32(lens),
                                       window=1 if how == "window" else 0, return_lse=True)
    la.la_check_device_status()
    for r, n in enumerate(lens):
        if how == "append":
            krow, row = k[r], v[r]
        else:
            at = (table[r, (n - 1) // page], slice(None), (n - 1) % page)
            krow, row = K[at], V[at]
        assert torch.equal(out[r].cpu(), row.float().repeat_interleave(Hq // Hkv, 0))
        s = (q[r].double() * krow.double().repeat_interleave(Hq // Hkv, 0)).sum(1) / D ** 0.5
        # a score: D products and their sums, the scale and the change of base, there and back
        size = (q[r].double() * krow.double().repeat_interleave(Hq // Hkv, 0)).abs().sum(1) / D ** 0.5
        assert bool(((lse[r].cpu().double() - s).abs() <= (D + 8) * 2.0 ** -24 * size).all())


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (24, 2, 64), (4, 4, 128), (16, 1, 128), (3, 1, 32)])
def test_a_position_that_takes_all_the_weight(Hq, Hkv, D):
    # among many positions, one whose score is so far above the others' that their weights are 0: its
    # value row to 2^-22 (two terms of 11 bits, the second rounded) and a unit's 2^-23 for the sum of the two
    la = _la()
    g = torch.Generator().manual_seed(D)
    n, page = 77, 16
    W = -(-n // page)
    V = torch.randn(W, Hkv, page, D, generator=g)
    K = torch.zeros(W, Hkv, page, D)
    K[2, :, 5, 0] = 1000.0
    q = torch.zeros(1, Hq, D)
    q[..., 0] = D ** 0.5
    out = la.la_paged_decode_step(q.cuda(), None, None, K.cuda(), V.cuda(), _i32([list(range(W))]), _i32([n]))[0].cpu()
    want = V[2, :, 5].repeat_interleave(Hq // Hkv, 0).double()
    err = (out.double() - want) / want.abs()
    assert float(err.abs().max()) <= 2.0 ** -22 + 2.0 ** -23
    assert bool((err > 0).any()) and bool((err < 0).any())  # to either side


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (24, 2, 64), (4, 4, 128), (16, 1, 128)])
def test_few_positions_of_one_value(Hq, Hkv, D):
    # up to 32 positions with one and the same value row and equal scores: every weight is 1, the sum of n rows
    # is exact for n a power of two, and so is its n-th part
    la = _la()
    g = torch.Generator().manual_seed(D)
    lens, page = [1, 2, 4, 8, 16, 32], 16
    R, W = len(lens), 2
    row = torch.randn(R, Hkv, D, generator=g)
    row = (row.view(torch.int32) & ~31).view(torch.float32)  # five bits of room, so that partial sums are exact too
    V = row.view(R, 1, Hkv, 1, D).expand(R, W, Hkv, page, D).reshape(R * W, Hkv, page, D).contiguous()
    K = torch.randn(R * W, Hkv, page, D, generator=g)
    q = torch.zeros(R, Hq, D)
    out = la.la_paged_decode_step(q.cuda(), None, None, K.cuda(), V.cuda(), _i32(torch.arange(R * W).view(R, W).tolist()), _i32(lens))
    assert torch.equal(out.cpu(), row.repeat_interleave(Hq // Hkv, 1))
