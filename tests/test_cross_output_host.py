"""Output rows of the cross attention that share memory are refused (no GPU: checks come before a launch)."""
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


def _call(ra, ost, B=2, H=4, Nq=9, D=128):
    p = ra._block._CrossProblem(B, H, H, Nq, 7, D, 0.1)
    st = [C.byref(ra._block.Strides(*x)) for x in ((H * Nq * D, Nq * D, D), (H * 7 * D, 7 * D, D), ost)]
    return ra.lib().ra_attn_cross(C.byref(p), GOOD, st[0], GOOD, st[1], GOOD, st[1], None, GOOD, st[2], None, None)


@pytest.mark.parametrize("ost", [(4608, 128, 128), (128, 128, 128), (1152, 1152, 128), (4608, 1144, 128),
                                 (4600, 1152, 128), (512, 128, 504), (4608, 128, 504), (1024, 4608, 128), (128, 1152, 256),
                                 (4616, 1160, 128)])   # 3 x 1160 + 8 x 128 + 128 = 4632
def test_rows_that_share_memory_are_refused(ra, ost):
    assert _call(ra, ost) == INVALID


@pytest.mark.parametrize("ost", [(4608, 1152, 128), (4608, 128, 512), (128, 256, 1024), (1152, 2304, 128), (10000, 2000, 136),
                                 (13824, 384, 1536), (4632, 1160, 128)])
def test_other_orders_and_gaps_are_not(ra, ost):
    assert _call(ra, ost) == CUDA


def test_extents_of_one_do_not_count(ra):
    assert _call(ra, (0, 1152, 128), B=1) == CUDA
    assert _call(ra, (1152, 128, 128), H=1) == CUDA
    assert _call(ra, (512, 128, 128), Nq=1) == CUDA
    assert _call(ra, (0, 0, 0), B=1, H=1, Nq=1) == CUDA
    assert _call(ra, (128, 128, 0), Nq=1) == INVALID
