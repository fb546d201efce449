"""Sizes that the C calls cannot hold are refused, not cut to 32 bits."""
import pytest
import torch

import linear_attention_02_gb300 as la
from linear_attention_02_gb300 import _native

BIG = 2 ** 32 + 8


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bad", [BIG, 2 ** 31, -2 ** 32 + 5, 2.5])
def test_numbers_past_32_bits(bad):
    for call in (lambda: la.la_gated_scan_ckpt_floats(1, bad, 1),
                 lambda: la.la_gated_scan_workspace_bytes(1, bad, 1, torch.float32),
                 lambda: la.la_paged_decode_workspace_bytes(2, 8, 2, 64, 16, bad, torch.float32, num_sms=152),
                 lambda: la.la_page_map_workspace_bytes(bad)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [BIG, 2 ** 32 + 16, 2 ** 31, 0.5])
def test_arguments_past_32_bits(bad):
    q = torch.zeros(1, 4, 64, device="cuda")
    K = torch.zeros(2, 4, 16, 64, device="cuda")
    with pytest.raises(ValueError, match="window"):
        la.la_paged_decode_step(q, None, None, K, K, _i32([[0]]), _i32([3]), window=bad)
    slots = _i32([0] * 4)
    with pytest.raises(ValueError, match="page_size"):
        la.la_page_map(_i32([0]), _i32([1]), _i32([0]), _i32([[-1]]), bad, 1, slots)
    with pytest.raises(ValueError, match="num_pages"):
        la.la_page_map(_i32([0]), _i32([1]), _i32([0]), _i32([[-1]]), 16, bad, slots)


@pytest.mark.gpu
def test_tensors_past_32_bits():
    a = torch.empty(1, BIG, 1, dtype=torch.bfloat16, device="cuda")  # never launched on
    with pytest.raises(ValueError, match="32 bits"):
        la.la_forward_gated_scan(a, a)
    with pytest.raises(ValueError, match="32 bits"):
        la.la_backward_gated_scan(a, a, a)
    with pytest.raises(ValueError, match="32 bits"):
        la.la_gated_scan_decode_step(a[0], a[0], torch.empty(0, device="cuda"))


FAKE = 0x10000  # aligned, never dereferenced


def _dec(k=FAKE, v=FAKE, R=2, Hq=8, Hkv=2, D=64, scale=0.0):
    return _native.lib.la_paged_decode_step(FAKE, k, v, FAKE, FAKE, FAKE, FAKE, FAKE, None, R, Hq, Hkv, D, 4, 16, 3, 0,
                                            scale, 1, None)


def _msg():
    return _native.lib.la_last_error_message().decode()


def test_scale_past_fp32_in_base_2():
    # scores are scaled by scale log2 e: infinite in fp32 from 2.36e38 up, and infinity times a score of 0 is NaN
    for scale in (2.4e38, -3e38):
        assert _dec(scale=scale) == _native.LA_ERR_INVALID_ARG and "scale" in _msg()


def test_new_rows_without_query_heads():
    # nothing would be attended, but the rows were not appended either
    assert _dec(Hq=0) == _native.LA_ERR_INVALID_ARG and "query heads" in _msg()
    assert _dec(Hq=0, k=None, v=None) == _native.LA_OK and _dec(Hq=0, R=0) == _native.LA_OK
    assert _dec(Hq=0, Hkv=0) == _native.LA_OK


def test_workspace_of_sizes_that_the_call_refuses():
    f = _native.lib.la_paged_decode_workspace_bytes
    assert _dec(R=1 << 20, Hq=64, Hkv=64) == _native.LA_ERR_INVALID_ARG and "too large" in _msg()
    assert f(1 << 20, 64, 64, 64, 16, 4, 1, 152) == _native.SIZE_MAX and "too large" in _msg()
    _dec(scale=float("inf"))
    assert _native.lib.la_page_map_workspace_bytes(1 << 30) == _native.SIZE_MAX and "R=" in _msg()
