"""Queries, keys and values that are not finite give NaN where the formulas do, in every form of the attention, and
rows without keys still give zeros."""
import math

import pytest
import torch

from tests import block_gpu as bg
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import int4_quantized_flashattention_b200 as ra
    gu.device()
    return ra


@pytest.fixture()
def gen():
    return torch.Generator(device="cuda").manual_seed(12)


def _spoil(q, how):
    """Row (H - 1, Nq - 1) of every batch entry."""
    if how == "all nan":
        q[:, -1, -1] = math.nan
    else:
        q[:, -1, -1, 5] = {"nan": math.nan, "inf": math.inf, "-inf": -math.inf}[how]
    bad = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    bad[:, -1, -1] = True
    return bad


def _check(out, lse, bad, empty, how):
    nan = torch.isnan(out)
    assert bool((nan.all(-1) == (bad & ~empty)).all()) and bool((nan.any(-1) == (bad & ~empty)).all())
    wrong = lse[bad & ~empty]
    assert not bool(torch.isfinite(wrong).any())
    if "nan" in how:
        assert bool(torch.isnan(wrong).all())
    assert bool((out[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())
    assert bool(torch.isfinite(lse[~bad & ~empty]).all())


@pytest.mark.parametrize("how", ["nan", "all nan", "inf", "-inf"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq,length", [(1, 77), (1, 9000), (4, 77), (4, 9000), (40, 77), (40, 9000)])
def test_cache_attention(ra, gen, how, D, Nq, length):
    """Few rows (8 and 16 a CTA) and tiles, keys in one part and in several; the second sequence is empty."""
    B, H, Hk = 2, 4, 1 if Nq < 40 else 2
    k, v = bg.rand(gen, B, Hk, length, D), bg.rand(gen, B, Hk, length, D)
    c, table, lens_t = bg.filled(ra, gen, [length, 0], 64, k, v)
    assert (ra.attn_kv4_workspace_bytes(c, B, H, Nq, length) > 0) == (length == 9000)
    q = bg.rand(gen, B, H, Nq, D, dtype=torch.bfloat16)
    bad = _spoil(q, how)
    lse = torch.empty(B, H, Nq, device="cuda")
    out = ra.attn_kv4(c, q, table, lens_t, max_len=length, lse=lse)
    assert ra.sync_status() == 0
    empty = torch.zeros_like(bad)
    empty[1] = True
    _check(out, lse, bad, empty, how)


@pytest.mark.parametrize("how", ["nan", "all nan", "inf", "-inf"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(1, 1), (130, 77), (300, 300)])
def test_cross_attention(ra, gen, how, D, Nq, Nk):
    B, H = 2, 3
    q = bg.rand(gen, B, H, Nq, D, dtype=torch.bfloat16)
    k, v = (bg.rand(gen, B, H, Nk, D, dtype=torch.bfloat16) for _ in range(2))
    bad = _spoil(q, how)
    lse = torch.empty(B, H, Nq, device="cuda")
    lens = torch.tensor([Nk, 0], device="cuda", dtype=torch.int32)
    out = ra.attn_cross(q, k, v, lens, lse=lse)
    assert ra.sync_status() == 0
    empty = torch.zeros_like(bad)
    empty[1] = True
    _check(out, lse, bad, empty, how)


def test_cross_attention_keys_and_values(ra, gen):
    """A NaN key spoils every row of its head, a NaN value the channel it lies in; other heads stay."""
    q, k, v = (bg.rand(gen, 1, 3, 140, 64, dtype=torch.bfloat16) for _ in range(3))
    k[0, 0, 70, 3] = math.nan
    v[0, 1, 139, 9] = math.nan
    lse = torch.empty(1, 3, 140, device="cuda")
    out = ra.attn_cross(q, k, v, lse=lse)
    assert ra.sync_status() == 0
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[0, 0] = True
    want[0, 1, :, 9] = True
    assert torch.equal(nan, want)
    assert bool(torch.isnan(lse[0, 0]).all()) and bool(torch.isfinite(lse[0, 1:]).all())


@pytest.mark.parametrize("Nq", [1, 4, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [50, 6000])
def test_rows_whose_scores_are_all_minus_infinity(ra, gen, Nq, D, length):
    """0 / 0, not the zeros of a row without keys; in one part of the keys and in several."""
    k, v = torch.ones(1, 1, length, D, device="cuda"), bg.rand(gen, 1, 1, length, D)
    c, table, lens_t = bg.filled(ra, gen, [length], 32, k, v)
    q = torch.zeros(1, 4, Nq, D, device="cuda", dtype=torch.bfloat16)
    q[:, :, :, 0] = -math.inf
    q[:, 1, :, 0] = 1.0
    lse = torch.empty(1, 4, Nq, device="cuda")
    out = ra.attn_kv4(c, q, table, lens_t, lse=lse)
    assert ra.sync_status() == 0
    assert bool(torch.isnan(out[:, [0, 2, 3]]).all()) and not bool(torch.isfinite(lse[:, [0, 2, 3]]).any())
    assert bool(torch.isfinite(out[:, 1]).all()) and bool(torch.isfinite(lse[:, 1]).all())
