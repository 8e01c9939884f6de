"""Scores far beyond fp32's whole numbers: finite inputs, so a finite result (the weights of the largest score)."""
import math

import pytest
import torch

from tests import block_bounds as bb
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
    return torch.Generator(device="cuda").manual_seed(16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq", [(8, 1, 1), (16, 1, 1), (3, 1, 5)])
def test_rows_of_all_sizes_together(ra, gen, D, H, Hk, Nq):
    """Rows of one key head from 2^-30 to 2^30, over a short and a split cache: each within its own bound."""
    lens = [9, 6000]
    k, v = bg.rand(gen, 2, Hk, 6000, D), bg.rand(gen, 2, Hk, 6000, D)
    c, table, lens_t = bg.filled(ra, gen, lens, 64, k, v)
    q = bg.rand(gen, 2, H, Nq, D)
    r = torch.arange(H * Nq, device="cuda", dtype=torch.float32).reshape(1, H, Nq, 1)
    q = (q * 2.0 ** (r * 60 / max(1, H * Nq - 1) - 30)).to(torch.bfloat16)
    bb.check_cache_attention(ra, c, table, lens_t, q)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq", [1, 3, 16, 40, 300])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 24, 2.0 ** 40, 2.0 ** 90])
def test_cache_attention(ra, gen, D, Nq, size):
    """Both signs of the scores: rows whose largest one is far below zero too."""
    lens = [300, 5000, 1]
    k, v = bg.rand(gen, 3, 1, 5000, D), bg.rand(gen, 3, 1, 5000, D)
    k[..., 0] = 3.0
    c, table, lens_t = bg.filled(ra, gen, lens, 64, k, v)
    q = bg.rand(gen, 3, 1, Nq, D)
    q[:, :, ::3, 0] = -60.0
    bb.check_cache_attention(ra, c, table, lens_t, (q * size).to(torch.bfloat16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 5, 2.0 ** 12, 2.0 ** 16, 2.0 ** 20, 2.0 ** 40])
def test_cross_attention(ra, gen, D, size):
    """Keys and queries of this size each.  A score may be off by delta of its size, so that where the two largest are
    nearer the row lies between their values: the output stays within what the values of the row span, and the
    log-sum-exp within delta of the largest score."""
    B, H, Nq, Nk = 1, 2, 150, 200
    q = (bg.rand(gen, B, H, Nq, D) * size).to(torch.bfloat16)
    k = (bg.rand(gen, B, H, Nk, D) * size).to(torch.bfloat16)
    k[..., 0] = 2 * size
    q[:, :, ::3, 0] = -40 * size
    v = bg.rand(gen, B, H, Nk, D, dtype=torch.bfloat16)
    lse = torch.empty(B, H, Nq, device="cuda")
    out = ra.attn_cross(q, k, v, lse=lse)
    assert ra.sync_status() == 0
    scale = float(torch.tensor(D ** -0.5))
    s = q.double() @ k.double().transpose(-1, -2) * scale
    delta = (D + 8) * bb.F32 * scale * (q.double().abs() @ k.double().abs().transpose(-1, -2)).amax(-1)
    want = torch.logsumexp(s, -1)
    assert bool(((lse - want).abs() <= 2 * delta + 2.0 ** -18 + 8 * bb.F32 * want.abs()).all())
    assert bool(torch.isfinite(out).all())
    # the keys that may be the largest
    near = s >= s.amax(-1, keepdim=True) - 2 * delta[..., None] - 30.0
    vv = v.double()[:, :, None].expand(B, H, Nq, Nk, D)
    lo = torch.where(near[..., None], vv, math.inf).amin(3)
    hi = torch.where(near[..., None], vv, -math.inf).amax(3)
    slack = 2.0 ** -6 * vv.abs().amax()
    assert bool((out.double() >= lo - slack).all() and (out.double() <= hi + slack).all())
