"""Sizes whose products pass 64 bits are refused like those that pass the limits (no GPU)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import int4_quantized_flashattention_b200 as ra
    if torch.cuda.is_available():
        pytest.skip("fake pointers: host-only check")
    return ra


GOOD = 0x10000
INVALID, CUDA = 1, 3


@pytest.mark.parametrize("B,H,Nq", [(1 << 16, 1 << 30, 1 << 24), (1 << 20, 1 << 30, 1 << 30), (1 << 15, 1 << 30, 1 << 24),
                                    (1 << 15, 1 << 28, 1 << 14), (3, 1 << 30, 1 << 24)])
def test_attention_over_the_cache(ra, B, H, Nq):
    c = ra._block._Kv4Cache(9, 16, 2, 128, GOOD, GOOD, GOOD, GOOD)
    a = ra._block._Kv4Attn(B, H, Nq, 4, 64, 0, 0.1)
    assert ra.lib().ra_attn_kv4_workspace_bytes(C.byref(c), C.byref(a)) == 0
    assert ra.lib().ra_attn_kv4(C.byref(c), C.byref(a), GOOD, GOOD, GOOD, None, GOOD, 1 << 60, GOOD, None, None) == INVALID


@pytest.mark.parametrize("B,H,Nq", [(1 << 22, 1 << 30, 1 << 20), (1 << 20, 1 << 28, 1 << 24)])
def test_cross_attention(ra, B, H, Nq):
    p = ra._block._CrossProblem(B, H, H, Nq, 7, 128, 0.1)
    D = 128
    # strides that keep rows apart where they fit 64 bits at all
    far = ra._block.Strides(1 << 37, 1 << 37, D)
    small = ra._block.Strides(H * Nq * D if H * Nq * D < 1 << 37 else 1 << 37, Nq * D if Nq * D < 1 << 37 else 1 << 37, D)
    for st in (far, small):
        assert ra.lib().ra_attn_cross(C.byref(p), GOOD, C.byref(st), GOOD, C.byref(st), GOOD, C.byref(st), None, GOOD,
                                      C.byref(st), None, None) == INVALID


def test_cache_of_many_pages(ra):
    c = ra._block._Kv4Cache((1 << 31) - 1, 1 << 30, 32767, 128, GOOD, GOOD, GOOD, GOOD)
    st = ra._block.Strides(1280, 640, 128)
    assert ra.lib().ra_kv4_append(C.byref(c), 1, 2, 5, GOOD, C.byref(st), GOOD, C.byref(st), GOOD, 4, GOOD, None,
                                  None) == INVALID
