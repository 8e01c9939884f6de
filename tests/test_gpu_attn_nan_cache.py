"""Keys and values of the cache that are not finite spoil the attention rows that see them, and those alone."""
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
    return torch.Generator(device="cuda").manual_seed(13)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq", [1, 4, 40])
@pytest.mark.parametrize("length,at", [(64, 3), (64, 63), (77, 70), (5000, 4990), (5000, 100)])
def test_attention_sees_it(ra, gen, D, Nq, length, at):
    """One bad key in one head, one bad value in another, in the middle and in the last step of the keys: the key
    spoils output and log-sum-exp, the value the output, and the third head stays."""
    H = Hk = 3
    H *= 4 if Nq == 4 else 1
    k, v = bg.rand(gen, 1, Hk, length, D), bg.rand(gen, 1, Hk, length, D)
    k[0, 0, at, 7] = math.nan
    v[0, 1, at, 0] = -math.inf
    c, table, lens_t = bg.filled(ra, gen, [length], 16, k, v)
    q = bg.rand(gen, 1, H, Nq, D, dtype=torch.bfloat16)
    out, lse = bb.check_cache_attention(ra, c, table, lens_t, q)
    g = H // Hk
    assert bool(torch.isnan(out[0, :2 * g]).all()) and bool(torch.isnan(lse[0, :g]).all())
    assert bool(torch.isfinite(lse[0, g:]).all()) and bool(torch.isfinite(out[0, 2 * g:]).all())


@pytest.mark.parametrize("Nq", [1, 40])
def test_attention_over_bad_rows_only(ra, gen, Nq):
    k = torch.full((1, 2, 5, 64), math.nan, device="cuda")
    c, table, lens_t = bg.filled(ra, gen, [5], 16, k, k)
    q = bg.rand(gen, 1, 2, Nq, 64, dtype=torch.bfloat16)
    lse = torch.empty(1, 2, Nq, device="cuda")
    out = ra.attn_kv4(c, q, table, lens_t, lse=lse)
    assert ra.sync_status() == 0
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
