"""64-bit references of the operators around the attention, from their definitions, and the error bounds that the
kernels' arithmetic allows.  Torch in double precision, on whatever device the inputs are."""
from __future__ import annotations

import math

import torch

U32, UB16 = 2.0 ** -24, 2.0 ** -8   # half steps of fp32 and bf16, relative to the value


def rotation(rot, seg):
    """R as a D x D matrix (row vectors x R): 0 none, 1 adjacent pairs, 2 pairs i, i + Dj/2, 3 the whole row."""
    D = sum(seg)
    r = math.sqrt(0.5)
    if rot == 0:
        return torch.eye(D, dtype=torch.float64)
    if rot == 3:
        m = torch.ones(1, 1, dtype=torch.float64)
        while len(m) < D:
            m = torch.kron(torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64), m)
        return m / math.sqrt(D)
    m = torch.zeros(D, D, dtype=torch.float64)
    o = 0
    for s in seg:
        for i in range(s // 2):
            u, w = (o + 2 * i, o + 2 * i + 1) if rot == 1 else (o + i, o + i + s // 2)
            m[u, o + 2 * i] = m[w, o + 2 * i] = m[u, o + 2 * i + 1] = r
            m[w, o + 2 * i + 1] = -r
        o += s
    return m


def norm_rope(x, weight, bias, layer, eps, pos, seg, theta, rot):
    """norm(x) w + b, RoPE pairs, rotation: x [B, H, N, D] -> float64.  pos None: the norm alone."""
    x = x.double()
    if layer:
        x = x - x.mean(-1, keepdim=True)
    x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    x = x * (1.0 if weight is None else weight.double()) + (0.0 if bias is None else bias.double())
    if pos is None:
        return x
    ang = torch.cat([pos[:, j:j + 1].double() * theta ** (-2.0 * torch.arange(s // 2, dtype=torch.float64,
                                                                             device=x.device) / s)
                     for j, s in enumerate(seg)], 1)
    c, s = ang.cos(), ang.sin()
    x0, x1 = x[..., 0::2], x[..., 1::2]
    x = torch.stack((x0 * c - x1 * s, x0 * s + x1 * c), -1).flatten(-2)
    return x @ rotation(rot, seg).to(x.device)


def norm_rope_bound(ref):
    """One rounding to bf16; before it fp32: the sum of squares (a tree over D <= 128 and two roundings more), the
    scaled value, the table, the pair products and up to seven butterflies with a scaling each add at most a few half
    steps of the row's 2-norm to a channel: 32 covers their sum."""
    return UB16 * ref.abs() + 32 * U32 * ref.square().sum(-1, keepdim=True).sqrt()


def quantise(x):
    """(codes, scale) of the symmetric INT4 rule: s = fl(amax / 7), code = rint(x * fl(7 / amax)), exact product."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    amax = torch.where(amax < 2.0 ** -125, torch.zeros_like(amax), amax)
    inv = torch.where(amax > 0, 7.0 / amax, torch.zeros_like(amax)).float().double()
    return (x * inv).round(), (amax / 7.0).float()


def unpack(codes4):
    """Packed bytes -> int64 codes, element 2t in the low nibble."""
    c = codes4.to(torch.int64)
    c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    return (c ^ 8) - 8


def cached(cache, table, b, n):
    """Keys and values of sequence b's first n tokens, [Hk, n, D] float64."""
    pages = table[b].long()
    out = []
    for codes, scale in ((cache.k4, cache.sk), (cache.v4, cache.sv)):
        c = unpack(codes[pages[:-(-n // cache.page_size)]]).double()
        v = c * scale[pages[:-(-n // cache.page_size)]].double()[..., None]
        out.append(v.transpose(0, 1).flatten(1, 2)[:, :n])
    return out


def attention(q, k, v, ends, scale):
    """Rows q [H, n, D] over keys [Hk, m, D]; row i sees keys below ends[i].  Returns out, lse and the elementwise
    error bounds of both:
      * S has D products and the key's scale in fp32: |dS| <= delta = (D + 8) u32 scale sum_d |q_d k_d| (its largest);
      * P = exp(S - m): relative error delta, plus 2^-18 for the exponential, the lazily moved reference and sums;
      * P is rounded to bf16 once in cross attention, the output once more.  (Both forms over the cache round to f16
        instead, 2^-11, in the tiles the value's scale and its product with the code too: this bound is wider than
        they need, block_bounds.py has theirs.  What is subnormal there adds an absolute part of 2^-36 * 2 * s_max *
        |code| <= 2^-35 max|v| per key, divided by the row's sum, which is at least 1 because a key has the reference
        maximum itself.)"""
    H, n, D = q.shape
    g = H // k.shape[0]
    out = torch.zeros(H, n, D, dtype=torch.float64, device=q.device)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=q.device)
    bound, bound_lse = torch.zeros_like(out), torch.zeros_like(lse)
    ends = ends.clamp(0, k.shape[1])
    some = ends > 0
    if not bool(some.any()):
        return out, lse, bound, bound_lse
    m = int(ends.max())
    live = (torch.arange(m, device=q.device)[None] < ends[:, None])[some]
    for h in range(H):
        kk, vv, qq = k[h // g, :m].double(), v[h // g, :m].double(), q[h][some].double()
        live_v = torch.where(torch.isfinite(vv), vv, torch.zeros_like(vv))
        live_k = torch.where(torch.isfinite(kk), kk, torch.zeros_like(kk))
        s = (qq @ live_k.T * scale).masked_fill(~live, -math.inf)
        delta = (D + 8) * U32 * scale * (qq.abs() @ live_k.abs().T).masked_fill(~live, 0.0).amax(1, keepdim=True)
        p = torch.softmax(s, 1)
        o = p @ live_v
        out[h, some], lse[h, some] = o, torch.logsumexp(s, 1)
        bound[h, some] = (UB16 * o.abs() + (UB16 + 2 * delta + 2.0 ** -18) * (1 + UB16) * (p @ live_v.abs())
                          + 2.0 ** -35 * m * live_v.abs().max())
        bound_lse[h, some] = (delta[:, 0] + 2.0 ** -18 + 4 * U32 * lse[h, some].abs())
    return out, lse, bound, bound_lse


def assert_within(got, ref, bound, what=""):
    got = got.double()
    if ref.numel() == 0:
        return
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), what
    d = (got - ref).abs().masked_fill(inf, 0.0)
    worst = (d - bound.masked_fill(inf, 0.0)).max()
    assert bool((d <= bound.masked_fill(inf, 1.0) + 1e-30).all()), (what, float(worst), float(d.max()))
