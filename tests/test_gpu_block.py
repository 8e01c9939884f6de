"""GPU tests of the operators around the attention against 64-bit references (tests/block_ref.py, which derives the
bounds): norm + RoPE + rotation, the 4-bit cache, attention over it, cross attention, and a block of them together."""
import math

import pytest
import torch

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
    yield ra
    torch.cuda.synchronize()


@pytest.fixture()
def gen():
    return torch.Generator(device="cuda").manual_seed(7)


def _rand(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def _positions(grid, n):
    i = torch.arange(n, device="cuda", dtype=torch.int32) + (grid[0] * grid[1] * grid[2] - n)
    return torch.stack((i // (grid[1] * grid[2]), i // grid[2] % grid[1], i % grid[2]), 1).contiguous()


# ------------------------------------------------------------------ norm + RoPE

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("rot", [0, 1, 2, 3, None])
@pytest.mark.parametrize("B,H,Hk,D,grid,n", [(1, 1, 1, 128, (3, 1, 1), 1), (2, 5, 3, 64, (3, 7, 5), 103),
                                             (1, 9, 9, 128, (2, 9, 11), 197)])
def test_norm_rope(ra, gen, dtype, layer, rot, B, H, Hk, D, grid, n):
    p = ra.Problem.make(B, H, D, SEG[D], grid, N=n, rot=rot or 0)
    # token-major projections and a dense tensor, with outlier channels and a zero row
    q = _rand(gen, B, n, H, D)
    q[..., 1::7] *= 20
    q = q.to(dtype).transpose(1, 2)
    k = _rand(gen, B, Hk, n, D, dtype=dtype)
    k[0, 0, 0] = 0
    w = [1 + 0.3 * _rand(gen, D) for _ in range(2)]
    b = [0.2 * _rand(gen, D), None]
    pos = None if rot is None else _positions(grid, n)
    table = None if rot is None else ra.rope_table(p)
    eps = 1e-6
    qo, ko = ra.qk_norm_rope(p, q, k, table, pos, q_weight=w[0], k_weight=w[1], q_bias=b[0], k_bias=b[1],
                             norm=ra.NORM_LAYER if layer else ra.NORM_RMS, eps=eps)
    assert ra.sync_status() == 0
    for x, o, ww, bb in ((q, qo, w[0], b[0]), (k, ko, w[1], b[1])):
        ref = br.norm_rope(x, ww, bb, layer, eps, pos, SEG[D], 10000.0, rot or 0)
        br.assert_within(o, ref, br.norm_rope_bound(ref))


def test_norm_rope_one_tensor_and_no_weights(ra, gen):
    p = ra.Problem.make(2, 3, 64, SEG[64], (2, 4, 4), rot=0)
    x = _rand(gen, 2, 3, 32, 64, dtype=torch.bfloat16)
    pos, table = _positions((2, 4, 4), 32), ra.rope_table(p)
    q1, none = ra.qk_norm_rope(p, x, None, table, pos)
    none2, k1 = ra.qk_norm_rope(p, None, x, table, pos)
    assert none is None and none2 is None and torch.equal(q1, k1)
    ref = br.norm_rope(x, None, None, False, 1e-6, pos, SEG[64], 10000.0, 0)
    br.assert_within(q1, ref, br.norm_rope_bound(ref))
    assert ra.sync_status() == 0


def test_norm_rope_many_heads_and_tokens(ra, gen):
    """Head groups of eight that do not divide the heads, two batches, in a fused projection's strides."""
    B, H, Hk, D, grid = 2, 21, 10, 128, (4, 20, 31)
    n = 4 * 20 * 31
    p = ra.Problem.make(B, H, D, SEG[D], grid, rot=1)
    x = _rand(gen, B, n, H + 2 * Hk, D, dtype=torch.bfloat16)
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    pos, table = _positions(grid, n), ra.rope_table(p)
    qo, ko = ra.qk_norm_rope(p, q, k, table, pos)
    for t, o in ((q, qo), (k, ko)):
        ref = br.norm_rope(t, None, None, False, 1e-6, pos, SEG[D], 10000.0, 1)
        br.assert_within(o, ref, br.norm_rope_bound(ref))
    assert ra.sync_status() == 0


def test_norm_rope_matches_rope_bf16_on_unit_rows(ra, gen):
    """Rows of norm sqrt(D) with eps 0 pass the norm unchanged up to rounding: RoPE as ra_rope_bf16 applies it."""
    p = ra.Problem.make(1, 2, 128, SEG[128], (3, 4, 5), rot=0)
    x = torch.sign(_rand(gen, 1, 2, 60, 128)).to(torch.bfloat16)   # +-1: norm exactly sqrt(D)
    pos = _positions((3, 4, 5), 60)
    a, b = ra.rope_bf16(p, x, x, pos)
    c, d = ra.qk_norm_rope(p, x, x, ra.rope_table(p), pos, eps=0.0)
    assert (a.float() - c.float()).abs().max() <= 2 ** -7 * 1.5 and torch.equal(c, d) and torch.equal(a, b)


def test_norm_rope_reports_positions_outside_the_grid(ra, gen):
    p = ra.Problem.make(1, 2, 64, SEG[64], (2, 2, 2), rot=0)
    x = _rand(gen, 1, 2, 8, 64, dtype=torch.bfloat16)
    pos = _positions((2, 2, 2), 8)
    pos[3, 1] = 2
    ra.qk_norm_rope(p, x, x, ra.rope_table(p), pos)
    assert ra.sync_status() == 1
    assert ra.sync_status() == 0


# ------------------------------------------------------------------ the cache

def _make_cache(ra, gen, B, pages_each, page, Hk, D, fill=True):
    """A cache whose unused slots hold codes of all ones and NaN scales, and a shuffled block table."""
    n = B * pages_each + 2
    c = ra.KV4Cache.empty(n, page, Hk, D)
    table = torch.randperm(n, generator=gen, device="cuda")[:B * pages_each].reshape(B, pages_each).to(torch.int32)
    for codes, scale in ((c.k4, c.sk), (c.v4, c.sv)):
        codes.fill_(255)
        scale.fill_(math.nan)
    return c, table.contiguous()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hk,D,T,page,starts,counts", [
    (1, 1, 128, 1, 16, None, None), (3, 5, 64, 37, 32, (0, 31, 90), (37, 0, 11)),
    (2, 9, 128, 133, 64, (63, 5), None), (2, 3, 64, 200, 128, (1, 127), (200, 129))])
def test_append_and_read(ra, gen, dtype, B, Hk, D, T, page, starts, counts):
    each = -(-(max(starts or [0]) + T) // page)
    c, table = _make_cache(ra, gen, B, each, page, Hk, D)
    before = [t.clone() for t in (c.k4, c.sk, c.v4, c.sv)]
    k = _rand(gen, B, T, Hk, D, dtype=dtype).transpose(1, 2)
    v = (_rand(gen, B, Hk, T, D) * 10).to(dtype)
    v[..., ::9] *= 30
    k[0, 0, 0], v[0, 0, 0] = 0, 1e-39      # a zero row, and one below the smallest scale
    dev_i = lambda x: None if x is None else torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    start, n = dev_i(starts), dev_i(counts)
    ra.kv4_append(c, k, v, table, start, n)
    sentinel = 77.0
    back = ra.kv4_read(c, table, start, T, n, out=(torch.full((B, Hk, T, D), sentinel, device="cuda"),
                                                   torch.full((B, Hk, T, D), sentinel, device="cuda")))
    back16 = ra.kv4_read(c, table, start, T, n, dtype=torch.bfloat16)
    assert ra.sync_status() == 0
    written = torch.zeros(c.num_pages, Hk, page, dtype=torch.bool, device="cuda")
    for b in range(B):
        cnt = T if counts is None else counts[b]
        at = torch.arange(cnt, device="cuda") + (0 if starts is None else starts[b])
        pg, slot = table[b].long()[at // page], at % page
        written[pg, :, slot] = True
        for x, codes, scale, y, y16 in ((k, c.k4, c.sk, back[0], back16[0]), (v, c.v4, c.sv, back[1], back16[1])):
            rc, rs = br.quantise(x[b, :, :cnt])
            assert torch.equal(br.unpack(codes[pg, :, slot]).transpose(0, 1), rc.long())
            assert torch.equal(scale[pg, :, slot].transpose(0, 1)[..., None], rs)
            exact = (rc.float() * rs)
            assert torch.equal(y[b, :, :cnt], exact)
            assert torch.equal(y16[b, :, :cnt], exact.to(torch.bfloat16))
            assert bool((y[b, :, cnt:] == sentinel).all())
    # nothing else in the cache moved
    for old, new in zip(before, (c.k4, c.sk, c.v4, c.sv)):
        m = ~written
        assert torch.equal(old[m].view(torch.uint8), new[m].view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hk,D", [(1, 64), (1, 128), (2, 64), (2, 128), (3, 64), (4, 128), (6, 128)])
@pytest.mark.parametrize("T,starts,counts", [(1, (0, 17), None), (301, (5, 128), (301, 66)), (130, (63, 0), (0, 129))])
def test_append_and_read_few_heads(ra, gen, dtype, Hk, D, T, starts, counts):
    """A thread works on several tokens where there are fewer heads than rows at a time; a bad page among them is
    left out alone."""
    B, page = 2, 16
    each = -(-(max(starts) + T) // page)
    c, table = _make_cache(ra, gen, B, each, page, Hk, D)
    bad_page = (starts[0] + T // 2) // page
    table[0, bad_page] = c.num_pages                       # of the first sequence
    before = [t.clone() for t in (c.k4, c.sk, c.v4, c.sv)]
    k = _rand(gen, B, T, Hk, D, dtype=dtype).transpose(1, 2)
    v = (_rand(gen, B, Hk, T, D) * torch.rand(B, Hk, T, 1, device="cuda", generator=gen) * 9).to(dtype)
    start = torch.tensor(starts, device="cuda", dtype=torch.int32)
    n = None if counts is None else torch.tensor(counts, device="cuda", dtype=torch.int32)
    out = tuple(torch.full((B, Hk, T, D), 77.0, device="cuda") for _ in range(2))
    ra.kv4_append(c, k, v, table, start, n)
    ra.kv4_read(c, table, start, T, n, out=out)
    written = torch.zeros(c.num_pages, Hk, page, dtype=torch.bool, device="cuda")
    reported = 0
    for b in range(B):
        cnt = T if counts is None else counts[b]
        i = torch.arange(T, device="cuda")
        at = i + starts[b]
        pg, slot = table[b].long()[at // page], at % page
        good = (i < cnt) & (pg < c.num_pages)
        reported |= int(bool(((i < cnt) & ~good).any()))
        written[pg[good], :, slot[good]] = True
        for x, codes, scale, y in ((k, c.k4, c.sk, out[0]), (v, c.v4, c.sv, out[1])):
            rc, rs = br.quantise(x[b][:, good])
            assert torch.equal(br.unpack(codes[pg[good], :, slot[good]]).transpose(0, 1), rc.long())
            assert torch.equal(scale[pg[good], :, slot[good]].transpose(0, 1)[..., None], rs)
            assert torch.equal(y[b][:, good], rc.float() * rs)
            assert bool((y[b][:, ~good] == 77.0).all())
    for old, now in zip(before, (c.k4, c.sk, c.v4, c.sv)):
        assert torch.equal(old[~written].view(torch.uint8), now[~written].view(torch.uint8))
    assert ra.sync_status() == reported


def test_append_refuses_bad_places(ra, gen):
    """Pages outside the cache, positions past the table, negative starts and counts: reported, nothing written."""
    for table, start, n in (([[0, 9]], [16], None), ([[0, -1]], [16], None), ([[0, 1]], [31], None),
                            ([[0, 1]], [-1], None), ([[0, 1]], [0], [3]), ([[0, 1]], [0], [-1])):
        c = ra.KV4Cache.empty(4, 16, 2, 64)
        x = _rand(gen, 1, 2, 2, 64, dtype=torch.bfloat16)
        i32 = lambda y: None if y is None else torch.tensor(y, device="cuda", dtype=torch.int32)  # noqa: E731
        ra.kv4_append(c, x, x, i32(table), i32(start), i32(n))
        assert ra.sync_status() == 1
        assert int(c.k4.max()) == 0 or start == [31]   # start 31: its first token still has a place
        assert ra.sync_status() == 0


# ------------------------------------------------------------------ attention over the cache

def _filled(ra, gen, lens, page, Hk, D, extra=0, outliers=True):
    B = len(lens)
    each = max(1, -(-max(lens) // page)) + extra
    c, table = _make_cache(ra, gen, B, each, page, Hk, D)
    T = max(max(lens), 1)
    k = _rand(gen, B, Hk, T, D)
    if outliers:
        k[..., ::5] *= 6
    v = _rand(gen, B, Hk, T, D)
    lens_t = torch.tensor(lens, device="cuda", dtype=torch.int32)
    ra.kv4_append(c, k, v, table, None, lens_t)
    return c, table, lens_t


def _check_kv4(ra, c, table, lens, q, qlens=None, causal=False, scale=None, **kw):
    B, H, Nq, D = q.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full_like(q, 55.0)
    lse = torch.full((B, H, Nq), 55.0, device="cuda")
    ql_t = None if qlens is None else torch.tensor(qlens, device="cuda", dtype=torch.int32)
    ra.attn_kv4(c, q, table, lens, q_lens=ql_t, causal=causal, scale=scale, out=out, lse=lse, **kw)
    assert ra.sync_status() == 0
    for b in range(B):
        n = int(lens[b])
        ql = Nq if qlens is None else qlens[b]
        k, v = br.cached(c, table, b, n)
        i = torch.arange(ql, device="cuda")
        ends = n - ql + i + 1 if causal else torch.full_like(i, n)
        ref, rl, bo, bl = br.attention(q[b, :, :ql], k, v, ends, float(torch.tensor(scale, dtype=torch.float32)))
        br.assert_within(out[b, :, :ql], ref, bo, ("out", b))
        br.assert_within(lse[b, :, :ql], rl, bl, ("lse", b))
        assert bool((out[b, :, ql:] == 55.0).all()) and bool((lse[b, :, ql:] == 55.0).all())
    return out, lse


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hk,D,Nq,page,lens", [
    (1, 1, 128, 1, 16, [1]), (1, 1, 64, 1, 16, [33]),
    (8, 8, 128, 1, 64, [0, 31, 64, 65, 700]), (8, 2, 64, 1, 32, [17, 0, 129]),
    (16, 2, 128, 1, 128, [500, 128, 3]), (6, 2, 128, 3, 16, [2, 0, 49, 95]), (12, 3, 64, 4, 64, [5, 4, 3, 321]),
    (3, 3, 128, 16, 32, [40, 16, 7, 200])])
def test_attn_few_rows(ra, gen, H, Hk, D, Nq, page, lens, causal):
    c, table, lens_t = _filled(ra, gen, lens, page, Hk, D)
    q = _rand(gen, len(lens), H, Nq, D, dtype=torch.bfloat16)
    _check_kv4(ra, c, table, lens_t, q, causal=causal)


@pytest.mark.parametrize("causal", [False, True])
def test_attn_few_rows_split(ra, gen, causal):
    """A long cache split over many CTAs, and short sequences in the same call (parts without keys)."""
    lens = [9000, 1, 0, 4097]
    c, table, lens_t = _filled(ra, gen, lens, 64, 2, 128)
    q = _rand(gen, 4, 4, 2, 128, dtype=torch.bfloat16)
    assert ra.attn_kv4_workspace_bytes(c, 4, 4, 2, 9000) > 0
    _check_kv4(ra, c, table, lens_t, q, causal=causal)
    # a plan for shorter sequences than there are still covers every key
    _check_kv4(ra, c, table, lens_t, q, causal=causal, max_len=100)
    _check_kv4(ra, c, table, lens_t, q, causal=causal, max_len=3000)


@pytest.mark.parametrize("Nq,qlens", [(3, [3, 1, 0]), (50, [50, 17, 0])])
def test_attn_padded_queries(ra, gen, Nq, qlens):
    """Padded batches: rows behind q_lens keep what they held, NaN queries there do no harm."""
    c, table, lens_t = _filled(ra, gen, [70, 200, 33], 32, 2, 64)
    q = _rand(gen, 3, 4, Nq, 64, dtype=torch.bfloat16)
    for b, n in enumerate(qlens):
        q[b, :, n:] = math.nan
    for causal in (False, True):
        _check_kv4(ra, c, table, lens_t, q, qlens=qlens, causal=causal)


def test_attn_sharp_and_scaled(ra, gen):
    """Nearly one-hot rows, growing scores (the reference maximum moves) and another scale, few and many rows."""
    c, table, lens_t = _filled(ra, gen, [3000, 1500], 64, 2, 128)
    for Nq in (1, 40):
        q = _rand(gen, 2, 4, Nq, 128, dtype=torch.bfloat16) * 8
        _check_kv4(ra, c, table, lens_t, q)
        _check_kv4(ra, c, table, lens_t, q, scale=0.01)
    k = torch.linspace(0.1, 30, 2000, device="cuda")[None, None, :, None].expand(1, 2, 2000, 128).contiguous()
    c, table = _make_cache(ra, gen, 1, 32, 64, 2, 128)
    ra.kv4_append(c, k, _rand(gen, 1, 2, 2000, 128), table)
    lens_t = torch.tensor([2000], device="cuda", dtype=torch.int32)
    for Nq in (1, 40):
        _check_kv4(ra, c, table, lens_t, torch.ones(1, 4, Nq, 128, device="cuda", dtype=torch.bfloat16))


@pytest.mark.parametrize("Nq", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_scales_of_many_sizes(ra, gen, Nq, D):
    """Keys and values whose rows differ by factors of up to 10^6, zero rows, and a cache that begins with tiny
    values: the running exponent of the value scales moves many times."""
    n = 1500
    c, table = _make_cache(ra, gen, 2, 24, 64, 2, D)
    k, v = _rand(gen, 2, 2, n, D), _rand(gen, 2, 2, n, D)
    size = 10.0 ** torch.empty(2, 2, n, 1, device="cuda").uniform_(-3, 3, generator=gen)
    size[0, 0] = 10.0 ** torch.linspace(-3, 3, n, device="cuda")[:, None]
    v *= size
    v[:, :, 5:40] = 0
    k[:, :, 9:12] = 0
    k *= 10.0 ** torch.empty(2, 2, n, 1, device="cuda").uniform_(-1.5, 0.5, generator=gen)
    ra.kv4_append(c, k, v, table)
    q = _rand(gen, 2, 4, Nq, D, dtype=torch.bfloat16)
    q[:, 1] *= 1e-3
    q[:, 2, :, :] = 0
    _check_kv4(ra, c, table, torch.tensor([n, 33], device="cuda", dtype=torch.int32), q)
    _check_kv4(ra, c, table, torch.tensor([n, 1001], device="cuda", dtype=torch.int32), q, causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hk,D,Nq,page,lens", [
    (1, 1, 128, 17, 16, [1]), (2, 2, 64, 33, 16, [33, 0, 127]), (4, 2, 128, 64, 64, [128, 129, 64]),
    (3, 3, 128, 127, 32, [500, 90]), (6, 2, 64, 100, 128, [300, 0, 700]), (2, 1, 128, 300, 64, [301, 2000]),
    (1, 1, 64, 1025, 32, [1500])])
def test_attn_many_rows(ra, gen, H, Hk, D, Nq, page, lens, causal):
    c, table, lens_t = _filled(ra, gen, lens, page, Hk, D)
    q = _rand(gen, len(lens), H, Nq, D, dtype=torch.bfloat16)
    _check_kv4(ra, c, table, lens_t, q, causal=causal)


def test_attn_many_rows_split(ra, gen):
    lens = [9000, 5, 0]
    c, table, lens_t = _filled(ra, gen, lens, 64, 2, 128)
    q = _rand(gen, 3, 2, 40, 128, dtype=torch.bfloat16)
    assert ra.attn_kv4_workspace_bytes(c, 3, 2, 40, 9000) > 0
    for causal in (False, True):
        _check_kv4(ra, c, table, lens_t, q, causal=causal)


def test_attn_many_sequences(ra, gen):
    """More sequence-head pairs than a grid dimension of 65535 holds, one token each."""
    B, Hk, D = 9000, 8, 64
    c = ra.KV4Cache.empty(B, 16, Hk, D)
    table = torch.randperm(B, generator=gen, device="cuda")[:, None].to(torch.int32).contiguous()
    k, v = _rand(gen, B, Hk, 16, D, dtype=torch.bfloat16), _rand(gen, B, Hk, 16, D, dtype=torch.bfloat16)
    lens = torch.randint(0, 17, (B,), generator=gen, device="cuda").to(torch.int32)
    ra.kv4_append(c, k, v, table, None, lens)
    q = _rand(gen, B, Hk, 1, D, dtype=torch.bfloat16)
    out = ra.attn_kv4(c, q, table, lens)
    assert ra.sync_status() == 0
    for b in (0, 1, 4095, 8190, 8191, 8192, 8999):   # on both sides of pair 65535
        n = int(lens[b])
        kk, vv = br.cached(c, table, b, n)
        ref, _, bound, _ = br.attention(q[b], kk, vv, torch.full((1,), n, device="cuda"),
                                        float(torch.tensor(D ** -0.5, dtype=torch.float32)))
        br.assert_within(out[b], ref, bound, b)


def test_attn_reports_bad_lengths_and_pages(ra, gen):
    for Nq in (1, 40):
        q = _rand(gen, 1, 2, Nq, 64, dtype=torch.bfloat16)
        c, table, lens_t = _filled(ra, gen, [64], 32, 2, 64)
        for lens, qlens, tb in (([65], None, table), ([-1], None, table), ([64], [Nq + 1], table),
                                ([64], None, torch.full_like(table, c.num_pages)), ([64], None, table * 0 - 1)):
            i32 = lambda y: None if y is None else torch.tensor(y, device="cuda", dtype=torch.int32)  # noqa: E731
            ra.attn_kv4(c, q, tb, i32(lens), q_lens=i32(qlens))
            assert ra.sync_status() == 1
        assert ra.sync_status() == 0


# ------------------------------------------------------------------ cross attention

def _check_cross(ra, q, k, v, lens=None, scale=None, out=None):
    B, H, Nq, D = q.shape
    Nk = k.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    lse = torch.full((B, H, Nq), 55.0, device="cuda")
    lens_t = None if lens is None else torch.tensor(lens, device="cuda", dtype=torch.int32)
    got = ra.attn_cross(q, k, v, lens_t, scale=scale, out=out, lse=lse)
    assert ra.sync_status() == 0
    for b in range(B):
        ends = torch.full((Nq,), Nk if lens is None else lens[b], device="cuda")
        ref, rl, bo, bl = br.attention(q[b], k[b], v[b], ends, float(torch.tensor(scale, dtype=torch.float32)))
        br.assert_within(got[b], ref, bo, ("out", b))
        br.assert_within(lse[b], rl, bl, ("lse", b))


@pytest.mark.parametrize("B,H,Hk,D,Nq,Nk,lens", [
    (1, 1, 1, 128, 1, 1, None), (1, 2, 2, 64, 128, 128, None), (2, 3, 3, 128, 129, 77, [77, 5]),
    (2, 4, 2, 64, 300, 257, [0, 130]), (1, 3, 1, 128, 513, 512, None), (3, 2, 2, 128, 77, 700, [128, 699, 1])])
def test_cross_shapes(ra, gen, B, H, Hk, D, Nq, Nk, lens):
    q = _rand(gen, B, H, Nq, D, dtype=torch.bfloat16)
    k, v = _rand(gen, B, Hk, Nk, D, dtype=torch.bfloat16), _rand(gen, B, Hk, Nk, D, dtype=torch.bfloat16)
    _check_cross(ra, q, k, v, lens)
    _check_cross(ra, q * 8, k, v, lens, scale=0.2)


def test_cross_token_major_and_nan_padding(ra, gen):
    """Views of fused projections, an output of token-major order, NaN and infinities behind the last key."""
    B, H, D, Nq, Nk = 2, 5, 128, 400, 300
    qkv = _rand(gen, B, Nq, 3, H, D, dtype=torch.bfloat16)
    kv = _rand(gen, B, Nk, 2, H, D, dtype=torch.bfloat16)
    lens = [131, 300]
    kv[0, 131:, 0] = math.nan
    kv[0, 131:215, 1] = math.nan
    kv[0, 215:, 1] = math.inf
    buf = torch.full((B, Nq, 2, H, D), 9.0, device="cuda", dtype=torch.bfloat16)
    _check_cross(ra, qkv[:, :, 1].transpose(1, 2), kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2), lens,
                 out=buf[:, :, 0].transpose(1, 2))
    assert bool((buf[:, :, 1] == 9.0).all())


def test_cross_many_items(ra, gen):
    """More items than SMs: every CTA goes through several, with batch entries of no keys among them."""
    B, H, D, Nq, Nk = 4, 20, 64, 1100, 150
    q = _rand(gen, B, H, Nq, D, dtype=torch.bfloat16)
    k, v = _rand(gen, B, H, Nk, D, dtype=torch.bfloat16), _rand(gen, B, H, Nk, D, dtype=torch.bfloat16)
    _check_cross(ra, q, k, v, [150, 0, 64, 129])


def test_cross_reports_bad_lengths(ra, gen):
    x = _rand(gen, 1, 2, 40, 64, dtype=torch.bfloat16)
    for n in (41, -1):
        ra.attn_cross(x, x, x, torch.tensor([n], device="cuda", dtype=torch.int32))
        assert ra.sync_status() == 1
    assert ra.sync_status() == 0


def test_cross_agrees_with_the_bf16_fallback(ra, gen):
    """Equal lengths: the same attention as ra_attn_bf16_fallback."""
    p = ra.Problem.make(1, 2, 128, SEG[128], (1, 20, 30))
    q, k, v = (_rand(gen, 1, 2, 600, 128, dtype=torch.bfloat16) for _ in range(3))
    a, b = ra.attn_bf16_fallback(p, q, k, v), ra.attn_cross(q, k, v)
    assert (a.float() - b.float()).norm() <= 5e-3 * a.float().norm()


# ------------------------------------------------------------------ use

def test_results_do_not_vary(ra, gen):
    """No atomics in the sums: the same call gives the same bits."""
    c, table, lens_t = _filled(ra, gen, [5000, 900], 64, 2, 128)
    for Nq in (1, 60):
        q = _rand(gen, 2, 8, Nq, 128, dtype=torch.bfloat16)
        first = ra.attn_kv4(c, q, table, lens_t)
        for _ in range(5):
            assert torch.equal(first, ra.attn_kv4(c, q, table, lens_t))


def _step(ra, p, table_r, pos, x, c, table, start, seq, text_k, text_v, w):
    """One block's attention: norms and RoPE, the cache, attention over it, and cross attention of the result."""
    B, n, H, D = p.B, p.N, p.H, p.D
    q, k = ra.qk_norm_rope(p, x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2), table_r, pos, q_weight=w,
                           k_weight=w)
    ra.kv4_append(c, k, x[:, :, 2].transpose(1, 2), table, start)
    a = ra.attn_kv4(c, q, table, seq, max_len=table.shape[1] * c.page_size)
    return ra.attn_cross(a, text_k, text_v)


@pytest.mark.parametrize("n,rot", [(1, 0), (24, 2), (96, 1)])
def test_streaming_block(ra, gen, n, rot):
    """Frame after frame through a block: each step against 64-bit attention over everything so far, with a graph
    replaying the later steps."""
    B, H, D, grid = 2, 4, 128, (n if n == 1 else 4, 1 if n == 1 else 4, 1 if n == 1 else n // 4)
    steps = 4
    grid = (steps * max(1, n // 4), 2 if n > 1 else 1, 2 if n > 1 else 1)
    p = ra.Problem.make(B, H, D, SEG[D], grid, N=n, rot=rot)
    table_r = ra.rope_table(p)
    w = 1 + 0.1 * _rand(gen, D)
    page = 16
    c, table = _make_cache(ra, gen, B, -(-n * steps // page), page, H, D)
    tk, tv = (_rand(gen, B, H, 33, D, dtype=torch.bfloat16) for _ in range(2))
    x = torch.empty(B, n, 3, H, D, device="cuda", dtype=torch.bfloat16)
    pos = torch.empty(n, 3, device="cuda", dtype=torch.int32)
    start, seq = (torch.zeros(B, device="cuda", dtype=torch.int32) for _ in range(2))
    allpos = _positions(grid, grid[0] * grid[1] * grid[2])
    kept, graph = [], None
    for s in range(steps):
        x.copy_(_rand(gen, B, n, 3, H, D, dtype=torch.bfloat16))
        pos.copy_(allpos[s * n:(s + 1) * n])
        start.fill_(s * n)
        seq.fill_((s + 1) * n)
        if s == 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = _step(ra, p, table_r, pos, x, c, table, start, seq, tk, tv, w)
        if graph is not None:
            graph.replay()
        else:
            out = _step(ra, p, table_r, pos, x, c, table, start, seq, tk, tv, w)
        assert ra.sync_status() == 0
        rows = [br.norm_rope(x[:, :, i].transpose(1, 2), w, None, False, 1e-6, pos, SEG[D], 10000.0, rot)
                for i in range(2)]
        kept.append((rows[1], x[:, :, 2].transpose(1, 2).double()))
        for b in range(B):
            k = torch.cat([t[0][b] for t in kept], 1)
            v = torch.cat([t[1][b] for t in kept], 1)
            ends = torch.full((n,), (s + 1) * n, device="cuda")
            # against exact attention: 4-bit keys and values, so only loosely
            a = br.attention(rows[0][b], k, v, ends, D ** -0.5)[0]
            ref = br.attention(a, tk[b], tv[b], torch.full((n,), 33, device="cuda"), D ** -0.5)[0]
            assert torch.nn.functional.cosine_similarity(out[b].double().flatten(), ref.flatten(), 0) > 0.98


def test_caches_and_tensors_past_32_bits(ra, gen):
    """Pages and rows whose offsets pass 2^32 bytes and 2^31 elements."""
    Hk, D, page, pages = 8, 128, 128, 72000             # 4.7 GB of codes for keys, and for values
    c = ra.KV4Cache(*(torch.empty(pages, Hk, page, *((D // 2,) if codes else ()), device="cuda",
                                  dtype=torch.uint8 if codes else torch.float32) for codes in (1, 0, 1, 0)))
    table = torch.tensor([[pages - 1, 3, pages - 2]], device="cuda", dtype=torch.int32)
    k, v = _rand(gen, 1, Hk, 300, D), _rand(gen, 1, Hk, 300, D)
    ra.kv4_append(c, k, v, table)
    lens = torch.tensor([300], device="cuda", dtype=torch.int32)
    for Nq in (1, 20):
        _check_kv4(ra, c, table, lens, _rand(gen, 1, Hk, Nq, D, dtype=torch.bfloat16))
    del c
    torch.cuda.empty_cache()
    buf = torch.empty(3 * 10 ** 9, device="cuda", dtype=torch.bfloat16)
    far = lambda n: buf.as_strided((2, 2, n, D), (2_500_000_000, 300 * D, D, 1))  # noqa: E731
    q, out = far(200), torch.empty(2, 2, 200, D, device="cuda", dtype=torch.bfloat16)
    q.copy_(_rand(gen, 2, 2, 200, D, dtype=torch.bfloat16))
    _check_cross(ra, q, q, q, out=out)
    p = ra.Problem.make(2, 2, D, SEG[D], (2, 10, 10), rot=0)
    got, _ = ra.qk_norm_rope(p, q, None, ra.rope_table(p), _positions((2, 10, 10), 200))
    assert torch.equal(got, ra.qk_norm_rope(p, q.contiguous(), None, ra.rope_table(p), _positions((2, 10, 10), 200))[0])
    k2 = q.contiguous()
    ra.attn_cross(k2, k2, k2, out=q)
    assert torch.equal(q, ra.attn_cross(k2, k2, k2))


def test_graph_replays_on_changed_inputs(ra, gen):
    """A captured call with split keys (two launches, the second begun early) replays on what its tensors then hold."""
    c, table, lens_t = _filled(ra, gen, [9000], 64, 2, 128)
    for Nq in (1, 40):
        q = _rand(gen, 1, 4, Nq, 128, dtype=torch.bfloat16)
        assert ra.attn_kv4_workspace_bytes(c, 1, 4, Nq, 9000) > 0
        ra.attn_kv4(c, q, table, lens_t)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ra.attn_kv4(c, q, table, lens_t)
        for n in (9000, 17, 0, 5000):
            q.copy_(_rand(gen, 1, 4, Nq, 128, dtype=torch.bfloat16))
            lens_t.fill_(n)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ra.attn_kv4(c, q, table, lens_t))
        lens_t.fill_(9000)
    assert ra.sync_status() == 0


def test_other_streams(ra, gen):
    """Two streams at once, each with its own workspace, and a stream given by handle: the results of one stream."""
    c, table, lens_t = _filled(ra, gen, [6000], 64, 2, 128)
    qs = [_rand(gen, 1, 4, n, 128, dtype=torch.bfloat16) for n in (1, 60)]
    want = [ra.attn_kv4(c, q, table, lens_t) for q in qs]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a = ra.attn_kv4(c, qs[0], table, lens_t, stream=s1)
        b = ra.attn_kv4(c, qs[1], table, lens_t, stream=s2.cuda_stream)
        d = ra.attn_cross(qs[1], qs[1], qs[1], stream=s1)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(d, ra.attn_cross(qs[1], qs[1], qs[1]))
    assert ra.sync_status() == 0


def _chain(ra, c, table, src, work, q_rows, steps, fence):
    """Steps in which every call reads what the one before wrote and the next one overwrites it; `fence` runs between."""
    B, Hk, _, D = src.shape
    seen = []
    for i in range(steps):
        work.copy_(src[:, :, i:i + 1])                                        # torch before, over the last call's input
        fence()
        start = torch.full((B,), i, dtype=torch.int32, device="cuda")
        ra.kv4_append(c, work, work, table, start=start)
        fence()
        work.zero_()
        fence()
        k, v = ra.kv4_read(c, table, None, i + 1)
        fence()
        q = k[:, :, -1:].expand(B, Hk, q_rows, D).contiguous()
        lens_t = start + 1
        fence()
        o = ra.attn_kv4(c, q, table, lens_t)
        fence()
        x = ra.attn_cross(o, k, v, out=q)                                     # over the queries of the call before
        fence()
        y, _ = ra.qk_norm_rope(ra.Problem.make(B, Hk, D, SEG[D], (1, 1, 1), N=q_rows, rot=0), x, None, None, None)
        fence()
        seen += [k.clone(), o, x.clone(), y]
    return seen


@pytest.mark.parametrize("q_rows", [1, 40])
def test_calls_in_a_row_keep_the_order_of_the_stream(ra, gen, q_rows):
    """Kernels start before the one ahead has ended: without a wait between the calls, on the stream and captured,
    each still sees all of what came before, and nothing of what comes after."""
    B, Hk, D, steps = 2, 3, 128, 24
    src = _rand(gen, B, Hk, steps, D, dtype=torch.bfloat16)
    table = torch.randperm(B * 2, generator=gen, device="cuda").to(torch.int32).reshape(B, 2).contiguous()
    c = ra.KV4Cache.empty(B * 2, 16, Hk, D)
    work = torch.empty_like(src[:, :, :1])
    args = (ra, c, table, src, work, q_rows, steps)
    want = _chain(*args, torch.cuda.synchronize)
    for t in (c.k4, c.sk, c.v4, c.sv):
        t.zero_()
    for _ in range(3):
        got = _chain(*args, lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _chain(*args, lambda: None)
    for _ in range(2):
        for t in (c.k4, c.sk, c.v4, c.sv):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ra.sync_status() == 0


def test_captured_over_two_streams(ra, gen):
    """A captured call that waits for two streams at once, and one that two streams wait for."""
    x = _rand(gen, 1, 2, 70, 64, dtype=torch.bfloat16)
    a, b, src = torch.empty_like(x), torch.empty_like(x), x.clone()
    side = torch.cuda.Stream()

    def calls():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            b.copy_(src)
            k = ra.attn_cross(b, b, b)
        a.copy_(src)
        here.wait_stream(side)
        o = ra.attn_cross(a, k, b)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            p = ra.attn_cross(o, o, b)
        r = ra.attn_cross(o, k, o)
        here.wait_stream(side)
        return k, o, p, r
    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls()
    for _ in range(3):
        a.zero_(), b.zero_()
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, w) for u, w in zip(got, want))
    assert ra.sync_status() == 0


def test_threads(ra, gen):
    """Calls from several threads at once, each on its own stream: the results of one thread."""
    from concurrent.futures import ThreadPoolExecutor
    c, table, lens_t = _filled(ra, gen, [3000, 1], 64, 2, 128)
    qs = [_rand(gen, 2, 4, n, 128, dtype=torch.bfloat16) for n in (1, 5, 60, 130)]
    want = [ra.attn_kv4(c, q, table, lens_t, causal=True) for q in qs]
    cross = [ra.attn_cross(q, q, q) for q in qs]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [(ra.attn_kv4(c, qs[i], table, lens_t, causal=True), ra.attn_cross(qs[i], qs[i], qs[i]))
                   for _ in range(50)]
            torch.cuda.current_stream().synchronize()
        return all(torch.equal(a, want[i]) and torch.equal(b, cross[i]) for a, b in got)
    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(4)))
    assert ra.sync_status() == 0


def test_wrappers_refuse(ra, gen):
    x = _rand(gen, 1, 2, 5, 64, dtype=torch.bfloat16)
    c, table, lens_t = _filled(ra, gen, [20], 16, 2, 64)
    with pytest.raises(ValueError):
        ra.attn_cross(x, x.float(), x)
    with pytest.raises(ValueError):
        ra.attn_cross(x, x, x[:, :1])
    with pytest.raises(ValueError):
        ra.attn_cross(x.transpose(2, 3), x, x)
    with pytest.raises(ra.RaError):
        ra.attn_cross(x.expand(2, 2, 5, 64), x.expand(2, 2, 5, 64), x.expand(2, 2, 5, 64))
    with pytest.raises(ValueError):
        ra.attn_kv4(c, x.half(), table, lens_t)
    with pytest.raises(ValueError):
        ra.attn_kv4(c, x, table.long(), lens_t)
    with pytest.raises(ValueError):
        ra.attn_kv4(c, x, table, lens_t.cpu())
    with pytest.raises(ValueError):
        ra.attn_kv4(c, x[..., :32], table, lens_t)
    with pytest.raises(ValueError):
        ra.kv4_append(c, x[:, :1], x[:, :1], table)
    with pytest.raises(ValueError):
        ra.kv4_append(c, x.half(), x.half(), table)
    p = ra.Problem.make(1, 2, 64, SEG[64], (5, 1, 1))
    with pytest.raises(ra.RaError):
        ra.qk_norm_rope(p, x, x, ra.rope_table(p)[:3], _positions((5, 1, 1), 5))
    with pytest.raises(ra.RaError):
        ra.qk_norm_rope(p, x, x, ra.rope_table(p), None)
    assert ra.sync_status() == 0
