"""A row of the cache's attention does not depend on the other rows that are worked on beside it."""
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
    return torch.Generator(device="cuda").manual_seed(11)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq", [(4, 2, 1), (8, 1, 1), (2, 1, 4), (8, 2, 4), (2, 1, 8), (4, 2, 40)])
@pytest.mark.parametrize("big", [2.0 ** 40, 2.0 ** 100, 2.0 ** -60, math.inf, -math.inf, math.nan])
def test_rows_beside_large_and_small_and_non_finite_ones(ra, gen, D, H, Hk, Nq, big):
    """One row of every batch entry is scaled by `big` (or, for what is not finite, holds it once); all others are
    ordinary rows and have to come out as if it were not there."""
    B, lens = 2, [70, 333]
    k, v = bg.rand(gen, B, Hk, 333, D), bg.rand(gen, B, Hk, 333, D)
    c, table, lens_t = bg.filled(ra, gen, lens, 32, k, v)
    q = bg.rand(gen, B, H, Nq, D, dtype=torch.bfloat16)
    odd = torch.zeros(H, Nq, dtype=torch.bool)
    odd[H - 1, Nq // 2] = True
    if math.isfinite(big):
        q[:, H - 1, Nq // 2] *= big
    else:
        q[:, H - 1, Nq // 2, 3] = big
    odd = odd.cuda()
    lse = torch.empty(B, H, Nq, device="cuda")
    out = ra.attn_kv4(c, q, table, lens_t, lse=lse)
    assert ra.sync_status() == 0
    for b in range(B):
        kk, vv = bb.codes_of(c, table, b, lens[b])
        ref, rl, bo, bl = bb.cache_attention(q[b], kk, vv, torch.full((Nq,), lens[b], device="cuda"), D ** -0.5,
                                             bb.form_of(H, Hk, Nq))
        bb.assert_close(out[b][~odd], ref[~odd], bo[~odd], ("out", b))
        bb.assert_close(lse[b][~odd], rl[~odd], bl[~odd], ("lse", b))
