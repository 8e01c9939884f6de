"""What is not finite stays visible in the 4-bit cache: a row of keys or values that holds a NaN or an infinity is
stored with a NaN scale and reads back as NaN."""
import math

import pytest
import torch

from tests import block_bounds as bb
from tests import block_gpu as bg
from tests import block_ref as br
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk", [1, 2, 3, 5])
def test_append_and_read(ra, gen, dtype, D, Hk):
    """Every place of a row and every kind of value, beside rows that stay exact."""
    B, T, page = 2, 2 * D + 9, 32
    k, v = bg.rand(gen, B, Hk, T, D), bg.rand(gen, B, Hk, T, D)
    for x in (k, v):
        for t in range(0, 2 * D, 2):                          # every other token, all channels in turn
            x[t // 2 % B, t // 4 % Hk, t, t // 2] = (math.nan, math.inf, -math.inf)[t // 2 % 3]
        x[1, Hk - 1, T - 1] = math.nan
        x[1, 0, T - 3] = math.inf
        x[0, 0, T - 5, 0], x[0, 0, T - 5, D - 1] = math.inf, math.nan
    k, v = k.to(dtype), v.to(dtype)
    c, table, lens_t = bg.filled(ra, gen, [T, T], page, k, v)
    got = ra.kv4_read(c, table, None, T, dtype=torch.float32)
    got16 = ra.kv4_read(c, table, None, T)
    assert ra.sync_status() == 0
    for b in range(B):
        for x, (codes, scale), y, y16 in zip((k, v), bb.codes_of(c, table, b, T), got, got16):
            bad = ~torch.isfinite(x[b].double()).all(-1)
            assert bool(bad.any()) and bool((~bad).any())
            assert bool(torch.isnan(scale[bad]).all())
            assert bool(torch.isnan(y[b][bad]).all()) and bool(torch.isnan(y16[b][bad]).all())
            rc, rs = br.quantise(x[b][~bad])
            assert torch.equal(codes[~bad], rc) and torch.equal(scale[~bad].float(), rs[..., 0])
            assert torch.equal(y[b][~bad], rc.float() * rs)
