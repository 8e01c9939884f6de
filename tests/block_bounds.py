"""64-bit reference of the attention over the 4-bit cache, straight from codes and scales, non-finite ones among them,
and the error bounds that the arithmetic of each of its two kernels allows.

Half steps relative to the value: fp32 2^-24, f16 2^-11, bf16 2^-8.  For a row that sees n keys, with z the scores in
powers of two below the row's reference maximum and p = 2^z:

  * S: q (bf16) and the codes are exact in what the products take, so S = sum of D exact products, added in fp32, then
    times the key's scale, the softmax scale and log2(e), each rounded: |dS| <= delta = (D + 8) 2^-24 scale sum|q k|.
    Where all products are whole numbers whose magnitudes add up to less than 2^24, the sum is exact in any order and
    delta is 6 * 2^-24 |S| (three roundings of factors, one of the product, one of the difference; one to spare).
  * p: 2^z by the hardware's approximation, 2^-22 relative, and the rounding of z, 2^-24 |z| (p |z| ln 2 < 0.37).
  * The sum of p: additions of non-negative terms, 2^-24 each; one with a zero (a key that is not there) is exact, so
    at most n - 1, and on the way of a term at most n / 8 within a lane and 48 more (lanes, warps, parts, weights).
  * The log: log2 of the sum, at most 16 n, by a function of one unit in the last place, 2^-23 of its value (times ln 2);
    three roundings of the result.
  * Output: the terms p v, where p (times the value's scale in the few-row kernel) is rounded to f16, 2^-11; in the
    128-row tiles the value's scale and its product with the code too, 2^-11 each.  p times scale is held relative to
    the largest value scale that the row has seen (a power of two not below it, so at most twice it), times 2^11; what
    is a subnormal f16 there is off by 2^-25, so by 2^-36 of the power of two and 7 for the code: 2^-35 of the largest
    |v| that scale can hold, a key.  The row's sum is at least 1, because a key has the reference maximum itself.  The
    tiles' values below 2^-14 are subnormal in the same way, weighted with p, whose sum is 1: 2^-34 covers both.
  * The output is rounded to bf16 once.
"""
from __future__ import annotations

import math

import torch

from tests import block_ref as br

F32, F16, BF16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8
LN2 = math.log(2)
P_ROUNDINGS = {"rows": 1, "tiles": 3}


def codes_of(cache, table, b, n):
    """((codes, scales) of the keys, the same of the values) of a sequence's first n tokens: [Hk, n, D], [Hk, n]."""
    pages = table[b].long()[:-(-n // cache.page_size)]
    got = []
    for codes, scale in ((cache.k4, cache.sk), (cache.v4, cache.sv)):
        got.append((br.unpack(codes[pages]).double().transpose(0, 1).flatten(1, 2)[:, :n],
                    scale[pages].double().transpose(0, 1).flatten(1, 2)[:, :n]))
    return got


def cache_attention(q, k, v, ends, scale, form, exact_sums=False, p_round=None):
    """q [H, n, D]; k and v as from codes_of; row i sees the keys below ends[i] and nothing of the others.
    A row that sees a score or a value that is not finite is NaN there.  Returns out, lse and their bounds.  p_round:
    a type that P is rounded to (mistakes planted here show what the bounds notice)."""
    (ck, sk), (cv, sv) = k, v
    H, n, D = q.shape
    g, m = H // ck.shape[0], ck.shape[1]
    dev = q.device
    out = torch.zeros(H, n, D, dtype=torch.float64, device=dev)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=dev)
    bound, bound_lse = torch.zeros_like(out), torch.zeros_like(lse)
    ends = ends.clamp(0, m)
    live = torch.arange(m, device=dev)[None] < ends[:, None]
    some = ends > 0
    if m == 0 or not bool(some.any()):
        return out, lse, bound, bound_lse
    for h in range(H):
        kk = ck[h // g] * sk[h // g][:, None]
        good_v = torch.isfinite(sv[h // g])
        vs = torch.where(good_v, sv[h // g], 0.0)
        vv = cv[h // g] * vs[:, None]
        qq = q[h].double()
        s = torch.where(live, qq @ kk.T * scale, -math.inf)
        p = torch.softmax(s, 1)
        p = torch.where(live, p, 0.0) if p_round is None else torch.where(live, p, 0.0).to(p_round).double()
        o = p @ vv
        o = torch.where(((live & ~good_v).any(1))[:, None], math.nan, o)
        size = torch.where(live, qq.abs() @ kk.abs().T * scale, 0.0).amax(1)
        top = torch.where(live, s.abs(), 0.0).amax(1)
        delta = 6 * F32 * top if exact_sums else (D + 8) * F32 * size
        most = 7 * torch.where(live, vs.abs(), 0.0).amax(1)
        lost = p @ vv.abs()
        out[h], lse[h] = torch.where(some[:, None], o, 0.0), torch.where(some, torch.logsumexp(s, 1), -math.inf)
        rel = P_ROUNDINGS[form] * F16 + 2 * delta + 2.0 ** -20 + (m + 16) * F32
        bound[h] = (BF16 * o.abs() + rel[:, None] * (1 + 2 * BF16) * lost + (2.0 ** -34 * m * most)[:, None])
        adds = torch.minimum(ends - 1, ends // 8 + 48).clamp_min(0)
        bound_lse[h] = (delta + 2.0 ** -22 + (1 + adds) * F32 + LN2 * 2 * F32 * (torch.log2(ends.clamp_min(1).double()) + 4)
                        + 3 * F32 * torch.where(torch.isfinite(lse[h]), lse[h].abs(), 0.0))
    return out, lse, bound, bound_lse


def assert_close(got, ref, bound, what=""):
    """Within the bound where the reference is finite, the same infinity or NaN elsewhere."""
    got = got.double()
    bad = ~torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), (what, "NaN", int(torch.isnan(got).sum()), int(torch.isnan(ref).sum()))
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), (what, "infinities")
    d = torch.where(bad, 0.0, (got - ref).abs())
    b = torch.where(bad, 1.0, bound)
    assert bool((d <= b + 1e-30).all()), (what, float((d - b).max()), float(d.max()), float((d / (b + 1e-30)).max()))


def form_of(H, Hk, Nq):
    return "rows" if H // Hk * Nq <= 16 else "tiles"


def check_cache_attention(ra, c, table, lens, q, qlens=None, causal=False, scale=None, exact_sums=False, **kw):
    """Runs ra.attn_kv4 and checks output, log-sum-exp, and that the rows behind q_lens keep what they held."""
    B, H, Nq, D = q.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full_like(q, 55.0)
    lse = torch.full((B, H, Nq), 55.0, device=q.device)
    ql_t = None if qlens is None else torch.tensor(qlens, device=q.device, dtype=torch.int32)
    ra.attn_kv4(c, q, table, lens, q_lens=ql_t, causal=causal, scale=scale, out=out, lse=lse, **kw)
    assert ra.sync_status() == 0
    form = form_of(H, c.Hk, Nq)
    for b in range(B):
        n, ql = int(lens[b]), Nq if qlens is None else qlens[b]
        k, v = codes_of(c, table, b, n)
        i = torch.arange(ql, device=q.device)
        ends = n - ql + i + 1 if causal else torch.full_like(i, n)
        ref, rl, bo, bl = cache_attention(q[b, :, :ql], k, v, ends, float(torch.tensor(scale, dtype=torch.float32)),
                                          form, exact_sums)
        assert_close(out[b, :, :ql], ref, bo, ("out", b))
        assert_close(lse[b, :, :ql], rl, bl, ("lse", b))
        assert bool((out[b, :, ql:] == 55.0).all()) and bool((lse[b, :, ql:] == 55.0).all())
    return out, lse
