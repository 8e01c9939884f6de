"""What the bounds of the cache's attention notice (CPU): mistakes planted in the 64-bit reference."""
import math

import pytest
import torch

from tests import block_bounds as bb


def _case(n=9, D=64, H=4, rows=40):
    g = torch.Generator().manual_seed(3)
    q = torch.randn(H, rows, D, generator=g).to(torch.bfloat16)
    codes = [torch.randint(-7, 8, (H, n, D), generator=g).double() for _ in range(2)]
    scales = [0.1 + 0.2 * torch.rand(H, n, generator=g).double() for _ in range(2)]
    return q, (codes[0], scales[0]), (codes[1], scales[1]), torch.full((rows,), n)


@pytest.mark.parametrize("form", ["rows", "tiles"])
def test_p_in_bf16_is_noticed_and_p_in_f16_is_not(form):
    q, k, v, ends = _case()
    ref, lse, bound, bound_lse = bb.cache_attention(q, k, v, ends, 0.125, form)
    for kind, fits in ((torch.float16, True), (torch.bfloat16, False)):
        got = bb.cache_attention(q, k, v, ends, 0.125, form, p_round=kind)[0].to(torch.bfloat16)
        assert bool(((got.double() - ref).abs() <= bound).all()) == fits


@pytest.mark.parametrize("D", [64, 128])
def test_sums_that_lose_bits_are_noticed_in_the_log_sum(D):
    """Nine keys, whole numbers as products, large ones that cancel: fp32 sums of q c are exact; sums of q (c + 8), with
    8 q taken off again, are not."""
    n, small = 9, D // 2
    g = torch.Generator().manual_seed(4)
    c = torch.randint(-7, 8, (1, n, D), generator=g).double()
    c[..., small:] = 2 * torch.randint(0, 2, (1, n, D // 2), generator=g) - 1
    c[..., small + 1::2] = -c[..., small::2]
    q = torch.randint(1, 16, (1, 5, D), generator=g).double()
    q[..., small:] = 2.0 ** 17 * 1.5
    ones = torch.ones(1, n, dtype=torch.float64)
    scale = 2.0 ** -10
    _, lse, _, bound = bb.cache_attention(q, (c, ones), (c, ones), torch.full((5,), n), scale, "rows", exact_sums=True)
    for offset, fits in ((0.0, True), (8.0, False)):
        s = torch.zeros(5, n)
        for d in range(D):
            s += (q[0, :, d:d + 1] * (c[0, :, d] + offset)).float()
        s = s.double() - offset * q[0].sum(1, keepdim=True)
        assert bool(((torch.logsumexp(s * scale, 1) - lse[0]).abs() <= bound[0]).all()) == fits
    assert float(bound.max()) < 3e-6


def test_masked_and_empty_rows():
    q, k, v, _ = _case(rows=3)
    v = (v[0], v[1].clone())
    v[1][:, 4] = math.nan
    out, lse, _, _ = bb.cache_attention(q, k, v, torch.tensor([0, 4, 5]), 0.125, "rows")
    assert bool((out[:, 0] == 0).all()) and bool((lse[:, 0] == -math.inf).all())
    assert bool(torch.isfinite(out[:, 1]).all()) and bool(torch.isnan(out[:, 2]).all())
    assert bool(torch.isfinite(lse[:, 1:]).all())
