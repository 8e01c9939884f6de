"""Keys that a row may not see do not reach it, whatever they hold: NaN, infinities' NaN, or values of any size."""
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
    return torch.Generator(device="cuda").manual_seed(14)


SHAPES = [(4, 4, 3, 9), (2, 1, 4, 33), (1, 1, 8, 40), (2, 1, 8, 64), (16, 1, 1, 50), (1, 1, 16, 5000), (2, 1, 16, 5000),
          (1, 1, 16, 16), (2, 1, 40, 70), (1, 1, 100, 100), (1, 1, 300, 4000), (2, 1, 33, 33)]


def _inputs(ra, gen, H, Hk, Nq, length, D, spoil):
    """Two sequences; of the newest Nq tokens the ones in the second half are spoiled."""
    lens = [length, max(Nq, length - 5)]
    k, v = bg.rand(gen, 2, Hk, length, D), bg.rand(gen, 2, Hk, length, D)
    for b, n in enumerate(lens):
        spoil(k[b], v[b], n - max(1, Nq // 2), n)
    return bg.filled(ra, gen, lens, 16, k, v), bg.rand(gen, 2, H, Nq, D, dtype=torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq,length", SHAPES)
@pytest.mark.parametrize("what", ["k", "v", "both"])
def test_nan_of_later_tokens(ra, gen, H, Hk, Nq, length, D, what):
    def spoil(k, v, lo, hi):
        if what != "v":
            k[:, lo:hi, 1] = math.nan
        if what != "k":
            v[:, lo:hi, 2] = math.inf
    (c, table, lens), q = _inputs(ra, gen, H, Hk, Nq, length, D, spoil)
    out, _ = bb.check_cache_attention(ra, c, table, lens, q, causal=True)
    if Nq > 1:
        assert bool(torch.isfinite(out[:, :, 0]).all()) and bool(torch.isnan(out[:, :, -1]).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq,length", SHAPES)
@pytest.mark.parametrize("size", [2.0 ** 24, 1e12, 1e35, 1e-12])
def test_sizes_of_later_tokens(ra, gen, H, Hk, Nq, length, D, size):
    """Values of the later tokens many times larger or smaller than what the earlier rows see (keys too, within what
    scores hold)."""
    def spoil(k, v, lo, hi):
        v[:, lo:hi] *= size
        v[:, lo:hi:3] *= 0.01
        k[:, lo:hi] *= 3.0
    (c, table, lens), q = _inputs(ra, gen, H, Hk, Nq, length, D, spoil)
    bb.check_cache_attention(ra, c, table, lens, q, causal=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq", [1, 4, 40])
def test_values_of_all_sizes(ra, gen, D, Nq):
    """Without a mask: value scales from 2^-30 to 2^30 of their neighbours', in mixed order."""
    length = 700
    k, v = bg.rand(gen, 2, 1, length, D), bg.rand(gen, 2, 1, length, D)
    v *= 2.0 ** torch.empty(2, 1, length, 1, device="cuda").uniform_(-30, 30, generator=gen)
    c, table, lens = bg.filled(ra, gen, [length, 31], 32, k, v)
    bb.check_cache_attention(ra, c, table, lens, bg.rand(gen, 2, 4, Nq, D, dtype=torch.bfloat16))


def test_nan_behind_the_end(ra, gen):
    """Slots behind a sequence's end hold NaN scales and rows of all ones (make_cache): both forms, all page sizes."""
    for page in (16, 32, 64, 128):
        for n in (1, 15, 17, 33, 100):
            k, v = bg.rand(gen, 1, 2, n, 64), bg.rand(gen, 1, 2, n, 64)
            c, table, lens = bg.filled(ra, gen, [n], page, k, v)
            for Nq in (1, 6, 40):
                q = bg.rand(gen, 1, 2, Nq, 64, dtype=torch.bfloat16)
                bb.check_cache_attention(ra, c, table, lens, q, causal=True)
                bb.check_cache_attention(ra, c, table, lens, q)
