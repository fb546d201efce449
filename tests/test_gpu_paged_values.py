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
