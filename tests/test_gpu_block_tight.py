"""The cache's attention within the bounds of its own arithmetic (tests/block_bounds.py): P in f16, sums that lose
nothing, padded batches over split keys, and a stream of frames over what the cache really holds."""
import math

import pytest
import torch

from tests import block_bounds as bb
from tests import block_gpu as bg
from tests import block_ref as br
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
SEG = {64: (24, 20, 20), 128: (44, 42, 42)}


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import int4_quantized_flashattention_b200 as ra
    gu.device()
    return ra


@pytest.fixture()
def gen():
    return torch.Generator(device="cuda").manual_seed(15)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq,lens", [(16, 8, 1, [9, 2, 1]), (8, 1, 1, [9, 40]), (8, 1, 2, [9, 33]),
                                          (4, 1, 4, [9, 700]), (4, 2, 40, [9, 90]), (4, 4, 200, [9, 300]),
                                          (2, 2, 1, [12000]), (2, 1, 8, [12000]), (1, 1, 60, [12000])])
def test_bounds(ra, gen, causal, D, H, Hk, Nq, lens):
    """Few keys, where a rounding of P shows, and many."""
    T = max(lens)
    k, v = bg.rand(gen, len(lens), Hk, T, D), bg.rand(gen, len(lens), Hk, T, D)
    c, table, lens_t = bg.filled(ra, gen, lens, 64, k, v)
    q = bg.rand(gen, len(lens), H, Nq, D, dtype=torch.bfloat16)
    bb.check_cache_attention(ra, c, table, lens_t, q, causal=causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Nq,n", [(1, 1, 9), (8, 1, 9), (2, 8, 9), (1, 40, 9), (8, 1, 300), (1, 130, 300)])
def test_sums_of_large_products_that_cancel(ra, gen, D, H, Nq, n):
    """Whole numbers whose products' magnitudes stay below 2^24, so that a sum in fp32 is exact in any order; the
    large ones cancel and the scores are small.  A form of the codes with an offset (code + 8, taken off again
    afterwards) passes 2^24 and is off by whole units, a thousandth each here."""
    small = D // 2
    k = torch.zeros(1, 1, n, D, device="cuda")
    k[..., small:] = (2 * torch.randint(0, 2, (1, 1, n, D // 2), generator=gen, device="cuda") - 1).float()
    k[..., small + 1::2] = -k[..., small::2]                  # cancels: pairs of large channels
    k[..., :small] = torch.randint(-7, 8, (1, 1, n, small), generator=gen, device="cuda").float()
    k[..., 0] = 7                                             # scale 1: the codes are the values
    v = bg.rand(gen, 1, 1, n, D)
    c, table, lens_t = bg.filled(ra, gen, [n], 32, k, v)
    assert torch.equal(bb.codes_of(c, table, 0, n)[0][0][0], k[0, 0].double())
    q = torch.zeros(1, H, Nq, D, device="cuda")
    big = 2.0 ** 17
    q[..., small::2] = big * (1 + torch.randint(0, 2, (1, H, Nq, D // 4), generator=gen, device="cuda").float() / 2)
    q[..., small + 1::2] = q[..., small::2]
    q[..., :small] = torch.randint(1, 16, (1, H, Nq, small), generator=gen, device="cuda").float()
    qb = q.to(torch.bfloat16)
    assert torch.equal(qb.float(), q) and float((q.abs().amax() * D / 2) + 16 * 7 * D / 2) < 2.0 ** 24
    bb.check_cache_attention(ra, c, table, lens_t, qb, scale=2.0 ** -10, exact_sums=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq,qlens", [(4, 2, 3, [3, 1, 0, 2]), (8, 2, 4, [1, 4, 3, 0]), (2, 2, 13, [5, 0, 13, 1]),
                                           (4, 2, 50, [50, 17, 0, 1]), (1, 1, 300, [129, 300, 0, 256])])
def test_padded_batches_over_split_keys(ra, gen, D, H, Hk, Nq, qlens):
    """q_lens with keys in several parts: rows behind them keep what they held, NaN queries there do no harm."""
    lens = [9000, 40, 3, 0]
    k, v = bg.rand(gen, 4, Hk, 9000, D), bg.rand(gen, 4, Hk, 9000, D)
    c, table, lens_t = bg.filled(ra, gen, lens, 64, k, v)
    assert ra.attn_kv4_workspace_bytes(c, 4, H, Nq, 9000) > 0
    q = bg.rand(gen, 4, H, Nq, D, dtype=torch.bfloat16)
    for b, n in enumerate(qlens):
        q[b, :, n:] = math.nan
    for causal in (False, True):
        bb.check_cache_attention(ra, c, table, lens_t, q, qlens=qlens, causal=causal, max_len=9000)


@pytest.mark.parametrize("n,rot", [(1, 0), (24, 2), (96, 1)])
def test_stream_of_frames(ra, gen, n, rot):
    """Frame after frame: keys and values in the cache as the rule stores them, attention over what is stored, cross
    attention of its result; the replay of a captured step gives the same bits."""
    B, H, D, steps, page = 2, 4, 128, 4, 16
    grid = (steps * max(1, n // 4), 2 if n > 1 else 1, 2 if n > 1 else 1)
    p = ra.Problem.make(B, H, D, SEG[D], grid, N=n, rot=rot)
    rope = ra.rope_table(p)
    w = 1 + 0.1 * bg.rand(gen, D)
    c, table = bg.make_cache(ra, gen, B, -(-n * steps // page), page, H, D)
    tk, tv = (bg.rand(gen, B, H, 33, D, dtype=torch.bfloat16) for _ in range(2))
    x = torch.empty(B, n, 3, H, D, device="cuda", dtype=torch.bfloat16)
    pos = torch.empty(n, 3, device="cuda", dtype=torch.int32)
    start, seq = (torch.zeros(B, device="cuda", dtype=torch.int32) for _ in range(2))
    i = torch.arange(n * steps, device="cuda", dtype=torch.int32)
    every = torch.stack((i // (grid[1] * grid[2]), i // grid[2] % grid[1], i % grid[2]), 1)

    def step():
        q, k = ra.qk_norm_rope(p, x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2), rope, pos, q_weight=w,
                               k_weight=w)
        ra.kv4_append(c, k, x[:, :, 2].transpose(1, 2), table, start)
        a = ra.attn_kv4(c, q, table, seq, max_len=table.shape[1] * page)
        return q, k, a, ra.attn_cross(a, tk, tv)
    graph = None
    for s in range(steps):
        x.copy_(bg.rand(gen, B, n, 3, H, D, dtype=torch.bfloat16))
        pos.copy_(every[s * n:(s + 1) * n])
        start.fill_(s * n)
        seq.fill_((s + 1) * n)
        if s == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                captured = step()
        q, k, a, o = step()
        assert ra.sync_status() == 0
        if graph is not None:
            for t in captured:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(t, u) for t, u in zip(captured, (q, k, a, o)))
        for b in range(B):
            kc, vc = bb.codes_of(c, table, b, (s + 1) * n)
            for (codes, scale), new in ((kc, k[b]), (vc, x[b, :, 2].transpose(0, 1))):
                rc, rs = br.quantise(new)
                assert torch.equal(codes[:, s * n:], rc) and torch.equal(scale[:, s * n:].float(), rs[..., 0])
            ends = torch.full((n,), (s + 1) * n, device="cuda")
            ref, _, bound, _ = bb.cache_attention(q[b], kc, vc, ends, float(torch.tensor(D ** -0.5)), bb.form_of(H, H, n))
            bb.assert_close(a[b], ref, bound, ("cache", s, b))
            ref, _, bound, _ = br.attention(a[b], tk[b], tv[b], torch.full((n,), 33, device="cuda"),
                                            float(torch.tensor(D ** -0.5)))
            bb.assert_close(o[b], ref, bound, ("cross", s, b))
