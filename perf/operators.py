"""The operators around the attention of a video transformer block, as measured cases.

  norm_rope   norm of every head's query and key row, 3D RoPE and the RoPE-aware rotation, in one pass
  kv4_update  new keys and values quantised into a paged 4-bit cache, and read back from it
  attn_kv4    attention of new queries over the paged 4-bit cache
  attn_cross  attention of the video tokens over an encoder's states

`run` computes them from elementary torch operations in 32 bits, or, with `own`, through the package.
"""
import math

import torch

own = False

NONE, INTERLEAVED, HALF, FULL = 0, 1, 2, 3
THETA, EPS = 10000.0, 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The step of one new token (B sequences) of an autoregressive model: latency only.
        dict(name="norm_rope one token", op="norm_rope", B=4, H=16, Hk=4, D=128, f=33, h=1, w=1, n=1, norm="rms",
             rot=NONE, dtype="bf16", fused=True),
        # One latent frame in fp32 with a LayerNorm and the half rotation, D = 64, odd token count.
        dict(name="norm_rope frame fp32", op="norm_rope", B=2, H=24, Hk=24, D=64, f=3, h=29, w=53, n=1537,
             norm="layer", rot=HALF, dtype="f32", fused=False),
        # All tokens of a 480p clip (Wan-like: 21 x 30 x 52, 40 heads), projections in token-major order.
        dict(name="norm_rope clip", op="norm_rope", B=1, H=40, Hk=40, D=128, f=21, h=30, w=52, n=32760, norm="rms",
             rot=INTERLEAVED, dtype="bf16", fused=True),
        # A batch of streams, one new token each.
        dict(name="kv4_update tokens", op="kv4_update", B=32, Hk=8, D=128, new=1, start=8190, page=16, ragged=False,
             dtype="bf16"),
        # Three latent frames of the 480p clip enter the cache.
        dict(name="kv4_update frames", op="kv4_update", B=1, Hk=40, D=128, new=4680, start=9361, page=64, ragged=False,
             dtype="bf16"),
        # One stream, one new token, shared key heads: the smallest call.
        dict(name="attn_kv4 short", op="attn_kv4", B=1, H=16, Hk=4, D=128, new=1, len=333, page=16, causal=False,
             ragged=False),
        # A padded batch of short prompts of a D = 64 model, causal, some sequences empty.
        dict(name="attn_kv4 ragged", op="attn_kv4", B=7, H=24, Hk=8, D=64, new=5, len=777, page=32, causal=True,
             ragged=True),
        # A batch of streams, one token each, long caches: bandwidth.
        dict(name="attn_kv4 tokens", op="attn_kv4", B=16, H=40, Hk=40, D=128, new=1, len=8191, page=64, causal=False,
             ragged=False),
        # The next latent frame (30 x 52 tokens) over the cache of a whole 480p clip: tensor cores.
        dict(name="attn_kv4 frame", op="attn_kv4", B=1, H=40, Hk=40, D=128, new=1560, len=32760, page=64, causal=False,
             ragged=False),
        # A small block over a short caption.
        dict(name="attn_cross small", op="attn_cross", B=1, H=2, Hk=2, D=128, nq=256, nk=77, ragged=False, fused=False),
        # A batch of captions of different lengths (one is empty), D = 64.
        dict(name="attn_cross ragged", op="attn_cross", B=3, H=24, Hk=24, D=64, nq=4161, nk=257, ragged=True,
             fused=True),
        # All tokens of the 480p clip over 512 text tokens, every tensor in token-major order.
        dict(name="attn_cross clip", op="attn_cross", B=1, H=40, Hk=40, D=128, nq=32760, nk=512, ragged=False,
             fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes spread over the logarithm of their range, the batch shrunk to the largest listed cost."""
    op = rng.choice(["norm_rope", "kv4_update", "attn_kv4", "attn_cross"])
    D = rng.choice([64, 128])
    hk, g = rng.choice([(1, 1), (2, 8), (4, 4), (8, 3), (8, 1), (16, 2), (24, 1), (40, 1)])
    B = _log(rng, 1, 16)
    if op == "norm_rope":
        f, h, w = _log(rng, 1, 24), _log(rng, 1, 64), _log(rng, 1, 64)
        n = min(max(1, f * h * w - rng.randint(0, 3)), 32760)
        B = max(1, min(B, 32760 * 40 // (n * hk * g)))
        return dict(op=op, B=B, H=hk * g, Hk=hk, D=D, f=f, h=h, w=w, n=n, norm=rng.choice(["rms", "layer"]),
                    rot=rng.choice([NONE, INTERLEAVED, HALF, FULL]), dtype=rng.choice(["bf16", "f32"]),
                    fused=rng.random() < 0.5)
    page, ragged = rng.choice([16, 32, 64, 128]), rng.random() < 0.5
    if op == "kv4_update":
        new = _log(rng, 1, 4680)
        B = max(1, min(B, 4680 * 40 // (new * hk)))
        return dict(op=op, B=B, Hk=hk, D=D, new=new, start=rng.randint(0, 9361), page=page, ragged=ragged,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "attn_kv4":
        new = 1 if rng.random() < 0.4 else _log(rng, 1, 1560)
        length = max(new, _log(rng, 1, 32760))
        B = max(1, min(B, 40 * 1560 * 32760 // (hk * g * new * length), 16 * 40 * 8191 // (hk * length)))
        return dict(op=op, B=B, H=hk * g, Hk=hk, D=D, new=new, len=length, page=page, causal=rng.random() < 0.5,
                    ragged=ragged)
    nq, nk = _log(rng, 1, 32760), _log(rng, 1, 1024)
    B = max(1, min(B, 40 * 32760 * 512 // (hk * g * nq * nk)))
    return dict(op=op, B=B, H=hk * g, Hk=hk, D=D, nq=nq, nk=nk, ragged=ragged, fused=rng.random() < 0.5)


def _lengths(case, most):
    """The sequences' lengths: all `most`, or spread below it, the first one empty."""
    B = case["B"]
    if not case["ragged"]:
        return [most] * B
    return [0 if b == 0 and B > 1 else max(1, most * (b + 1) // B - b) for b in range(B)]


def _segments(D):
    return (24, 20, 20) if D == 64 else (44, 42, 42)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    op, B, D = case["op"], case["B"], case["D"]
    st = dict(case=case)

    def rows(heads, n, fused, unit=True):
        """Projections of one kind, [B, heads, n, D]: dense, or a view of token-major order.  Every fourth
        channel of the first half is an outlier; with `unit` each row has a root mean square of one."""
        x = normal(B, n, heads, D) if fused else normal(B, heads, n, D)
        x[..., 0:D // 2:4] *= 8.0
        if unit:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True))
        x = x.to(dt)
        return x.transpose(1, 2) if fused else x

    if op == "norm_rope":
        n, grid = case["n"], (case["f"], case["h"], case["w"])
        st["q"], st["k"] = rows(case["H"], n, case["fused"], False), rows(case["Hk"], n, case["fused"], False)
        last = grid[0] * grid[1] * grid[2] - n  # the newest n tokens of the clip
        i = torch.arange(last, last + n, device=dev, dtype=torch.int32)
        st["pos"] = torch.stack((i // (grid[1] * grid[2]), i // grid[2] % grid[1], i % grid[2]), 1).contiguous()
        st["w"] = [1.0 + 0.2 * normal(D) for _ in range(2)]
        st["b"] = [0.1 * normal(D) for _ in range(2)] if case["norm"] == "layer" else [None, None]
        # cos and sin of every axis position, and the same with the interleaved 2x2 rotation in it, as a program keeps them
        ang = [torch.arange(grid[j], device=dev, dtype=torch.float64)[:, None]
               * THETA ** (-2.0 * torch.arange(s // 2, device=dev, dtype=torch.float64) / s) for j, s in enumerate(_segments(D))]
        st["angle"] = ang
        scale = 1.0
        cs = [(a.cos(), a.sin()) for a in ang]
        if case["rot"] == INTERLEAVED:
            scale = math.sqrt(0.5)
            cs = [((c + s) * scale, (c - s) * scale) for c, s in cs]
        st["table"] = torch.cat([torch.stack(p, -1).reshape(-1, 2) for p in cs]).float().contiguous()
        st["cossin"] = [torch.cat([f(a)[st["pos"][:, j].long()] for j, a in enumerate(ang)], 1).float() for f in (torch.cos, torch.sin)]
        return st

    if op == "attn_cross":
        st["q"] = rows(case["H"], case["nq"], case["fused"])
        st["k"], st["v"] = rows(case["Hk"], case["nk"], case["fused"]), rows(case["Hk"], case["nk"], case["fused"])
        st["lens"] = torch.tensor(_lengths(case, case["nk"]), device=dev, dtype=torch.int32) if case["ragged"] else None
        if case["ragged"]:  # what lies behind a caption's end is not defined
            dead = torch.arange(case["nk"], device=dev)[None, :] >= st["lens"][:, None]
            for t in (st["k"], st["v"]):
                t.masked_fill_(dead[:, None, :, None], float("nan"))
        return st

    # a paged cache; the pages of the sequences are spread over it at random
    page = case["page"]
    most = case["len"] if op == "attn_kv4" else case["start"] + case["new"]
    each = -(-most // page)
    pages = B * each + 3
    st["table"] = torch.randperm(pages, generator=gen, device=dev)[:B * each].reshape(B, each).to(torch.int32).contiguous()
    st["cache"] = []
    for _ in range(2):
        if op == "attn_kv4":
            x = normal(pages, case["Hk"], page, D)
            x[..., 0:D // 2:4] *= 4.0
            amax = x.abs().amax(-1)
            codes = torch.round(x * (7.0 / amax)[..., None]).to(torch.int32) & 15
            st["cache"] += [(codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8).contiguous(), (amax / 7.0).contiguous()]
        else:
            st["cache"] += [torch.zeros(pages, case["Hk"], page, D // 2, dtype=torch.uint8, device=dev),
                            torch.zeros(pages, case["Hk"], page, device=dev)]
    if op == "attn_kv4":
        st["q"] = rows(case["H"], case["new"], False)
        st["lens"] = torch.tensor(_lengths(case, case["len"]), device=dev, dtype=torch.int32)
        st["max_len"] = case["len"]
    else:
        st["k"], st["v"] = rows(case["Hk"], case["new"], True), rows(case["Hk"], case["new"], True, False)
        starts = [case["start"]] * B if not case["ragged"] else [case["start"] * b // B for b in range(B)]
        st["start"] = torch.tensor(starts, device=dev, dtype=torch.int32)
    return st


# ------------------------------------------------------------------ the operators

def run(st):
    case = st["case"]
    return globals()["_own_" + case["op"] if own else "_plain_" + case["op"]](st, case)


def _package():  # imported where `own` is true only
    import int4_quantized_flashattention_b200 as ra
    return ra


def _own_norm_rope(st, case):
    ra = _package()
    p = st.get("problem")
    if p is None:
        p = st["problem"] = ra.Problem.make(case["B"], case["H"], case["D"], _segments(case["D"]),
                                            (case["f"], case["h"], case["w"]), N=case["n"], theta=THETA, rot=case["rot"])
    return ra.qk_norm_rope(p, st["q"], st["k"], st["table"], st["pos"], q_weight=st["w"][0], k_weight=st["w"][1],
                           q_bias=st["b"][0], k_bias=st["b"][1],
                           norm=ra.NORM_RMS if case["norm"] == "rms" else ra.NORM_LAYER, eps=EPS)


def _own_kv4_update(st, case):
    ra = _package()
    cache = ra.KV4Cache(*st["cache"])
    ra.kv4_append(cache, st["k"], st["v"], st["table"], st["start"])
    return ra.kv4_read(cache, st["table"], st["start"], case["new"], dtype=torch.float32)


def _own_attn_kv4(st, case):
    ra = _package()
    q = st["q"]
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    out = ra.attn_kv4(ra.KV4Cache(*st["cache"]), q, st["table"], st["lens"], causal=case["causal"],
                      max_len=st["max_len"], lse=lse)
    return out, lse


def _own_attn_cross(st, case):
    ra = _package()
    q = st["q"]
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    out = ra.attn_cross(q, st["k"], st["v"], st["lens"], out=torch.empty_like(q), lse=lse)
    return out, lse


def _hadamard(x):
    """The last axis times the Sylvester Hadamard matrix over the root of its length (at most 256)."""
    n = x.shape[-1]
    i = torch.arange(n, device=x.device)
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> s) & 1 for s in range(8)) & 1
    return x @ ((1 - 2 * odd).to(x.dtype) / math.sqrt(n))


def _rotate(x, rot, seg):
    """The RoPE-aware rotation of rows that carry their positions."""
    r = math.sqrt(0.5)
    if rot == INTERLEAVED:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack(((a + b) * r, (a - b) * r), -1).flatten(-2)
    if rot == HALF:
        parts = [t.unflatten(-1, (2, -1)) for t in x.split(seg, -1)]
        return torch.cat([torch.stack(((t[..., 0, :] + t[..., 1, :]) * r, (t[..., 0, :] - t[..., 1, :]) * r), -1).flatten(-2) for t in parts], -1)
    return _hadamard(x) if rot == FULL else x


def _plain_norm_rope(st, case):
    c, s = st["cossin"]
    outs = []
    for x, w, b in zip((st["q"], st["k"]), st["w"], st["b"]):
        x = x.float()
        if case["norm"] == "layer":
            x = x - x.mean(-1, keepdim=True)
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        if b is not None:
            x = x + b
        x0, x1 = x[..., 0::2], x[..., 1::2]
        x = torch.stack((x0 * c - x1 * s, x0 * s + x1 * c), -1).flatten(-2)
        outs.append(_rotate(x, case["rot"], _segments(case["D"])).to(torch.bfloat16).contiguous())
    return tuple(outs)


def _plain_kv4_update(st, case):
    outs = []
    for x in (st["k"], st["v"]):
        x = x.float()
        amax = x.abs().amax(-1, keepdim=True).double()  # correctly rounded quotients and exact products: codes next to a border
        codes = torch.round(x.double() * (7.0 / amax).float().double())
        outs.append((codes.float() * (amax / 7.0).float()).contiguous())
    return tuple(outs)


def _cached(st, case, dtype):
    """Keys and values of the sequences in their order, [B, Hk, length, D]."""
    k4, sk, v4, sv = st["cache"]
    n = st["max_len"]
    got = []
    for codes, scale in ((k4, sk), (v4, sv)):
        c = codes[st["table"].long()].transpose(1, 2).flatten(2, 3)[:, :, :n].to(torch.int16)
        sc = scale[st["table"].long()].transpose(1, 2).flatten(2, 3)[:, :, :n]
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
        got.append(((c ^ 8) - 8).to(dtype) * sc[..., None].to(dtype))
    return got


def _attend(q, k, v, dead, dtype):
    """softmax(q k^T / sqrt(D)) v where `dead` is false, zero for a row that has nothing; with the log of its sums."""
    B, H, n, D = q.shape
    q = q.to(dtype).unflatten(1, (k.shape[1], -1))
    s = (q.flatten(2, 3) @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).unflatten(2, (-1, n))
    if dead is not None:
        s = s.masked_fill_(dead, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    s = s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    out = (s.flatten(2, 3) @ v).unflatten(2, (-1, n)) / torch.where(total > 0, total, torch.ones_like(total))
    return out.flatten(1, 2), (m + total.log()).squeeze(-1).flatten(1, 2)


def _dead_kv4(st, case):
    """True where a query of the newest `new` positions may not look."""
    j = torch.arange(st["max_len"], device=st["lens"].device)
    last = st["lens"][:, None].expand(-1, case["new"]) - 1
    if case["causal"]:
        last = last - case["new"] + 1 + torch.arange(case["new"], device=j.device)
    return (j[None, None, :] > last[:, :, None])[:, None, None]


def _plain_attn_kv4(st, case):
    k, v = _cached(st, case, torch.float32)
    dead = _dead_kv4(st, case) if case["causal"] or case["ragged"] else None
    out, lse = _attend(st["q"], k, v, dead, torch.float32)
    return out.to(torch.bfloat16), lse


def _plain_attn_cross(st, case):
    dead, k, v = None, st["k"].float(), st["v"].float()
    if st["lens"] is not None:
        dead = torch.arange(case["nk"], device=k.device)[None, :] >= st["lens"][:, None]
        v = v.masked_fill(dead[:, None, :, None], 0.0)
        dead = dead[:, None, None, None, :]
    out, lse = _attend(st["q"], k, v, dead, torch.float32)
    return out.to(torch.bfloat16), lse


# ------------------------------------------------------------------ work and 64-bit values

def work(case):
    op, B, D, Hk = case["op"], case["B"], case["D"], case["Hk"]
    size = 4 if case.get("dtype") == "f32" else 2
    if op == "norm_rope":
        rows = B * (case["H"] + Hk) * case["n"]
        table = 8 * sum(g * s // 2 for g, s in zip((case["f"], case["h"], case["w"]), _segments(D)))
        return dict(bytes=rows * D * (size + 2) + 12 * case["n"] + table, flops=rows * D * 10)
    if op == "kv4_update":
        rows = 2 * B * Hk * case["new"]  # read once, 4-bit rows written and read, 32-bit values written
        return dict(bytes=rows * (D * size + 2 * (D // 2 + 4) + 4 * D), flops=rows * D * 6)
    if op == "attn_kv4":
        lens, n = _lengths(case, case["len"]), case["new"]
        if case["causal"]:
            pairs = sum(sum(max(0, x - n + 1 + i) for i in range(n)) for x in lens)
        else:
            pairs = n * sum(lens)
        nbytes = B * case["H"] * n * (4 * D + 4) + sum(lens) * Hk * (D + 8) + 4 * B * -(-case["len"] // case["page"])
        return dict(bytes=nbytes, flops=4 * pairs * case["H"] * D)
    lens = _lengths(case, case["nk"])
    nbytes = B * case["H"] * case["nq"] * (4 * D + 4) + sum(lens) * Hk * 4 * D
    return dict(bytes=nbytes, flops=4 * case["nq"] * sum(lens) * case["H"] * D)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        seg = _segments(case["D"])
        phi = torch.cat([a[st["pos"][:, j].long()] for j, a in enumerate(st["angle"])], 1)  # [n, D/2], 64 bits
        turn = torch.complex(phi.cos(), phi.sin())
        outs = []
        for x, w, b in zip((st["q"], st["k"]), st["w"], st["b"]):
            got = torch.empty(x.shape, dtype=torch.float64, device=x.device)
            for i in range(x.shape[0]):
                for h in range(x.shape[1]):
                    r = x[i, h].double()
                    if case["norm"] == "layer":
                        r = (r - r.mean(1, keepdim=True)) / (r.var(1, unbiased=False, keepdim=True) + EPS).sqrt()
                    else:
                        r = r / (r.pow(2).mean(1, keepdim=True) + EPS).sqrt()
                    r = r * w.double() + (0.0 if b is None else b.double())
                    z = torch.view_as_complex(r.reshape(-1, case["D"] // 2, 2).contiguous()) * turn
                    got[i, h] = torch.view_as_real(z).reshape(-1, case["D"]) @ _rotation_matrix(case["rot"], seg, x.device)
            outs.append(got)
        return tuple(outs)
    if op == "kv4_update":
        outs = []
        for x in (st["k"], st["v"]):
            x = x.double()
            top = x.abs().max(-1, keepdim=True).values
            outs.append((x * (7.0 / top).float().double()).round() * (top / 7.0).float().double())
        return tuple(outs)
    if op == "attn_kv4":
        k, v = _cached(st, case, torch.float64)
        first = st["lens"].tolist()
        ends = [[x - case["new"] + 1 + i if case["causal"] else x for i in range(case["new"])] for x in first]
    else:
        k, v = st["k"].double(), st["v"].double()
        n = case["nq"]
        ends = [[x] * n for x in _lengths(case, case["nk"])]
    q = st["q"]
    group = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], float("-inf"), dtype=torch.float64, device=q.device)
    for b in range(q.shape[0]):
        end = torch.tensor(ends[b], device=q.device).clamp_min(0)
        most = int(end.max())
        if most == 0:
            continue
        live = torch.arange(most, device=q.device)[None, :] < end[:, None]
        some = end > 0
        for h in range(q.shape[1]):
            s = q[b, h].double() @ k[b, h // group, :most].T / math.sqrt(case["D"])
            s = torch.where(live, s, torch.full_like(s, float("-inf")))[some]
            lse[b, h, some] = torch.logsumexp(s, 1)
            out[b, h, some] = torch.softmax(s, 1) @ v[b, h // group, :most]
    return out, lse


def _rotation_matrix(rot, seg, device):
    """The rotation as a D x D matrix that rows are multiplied with."""
    D = sum(seg)
    m = torch.eye(D, dtype=torch.float64, device=device)
    r = math.sqrt(0.5)
    if rot == FULL:
        m = torch.ones(1, 1, dtype=torch.float64, device=device)
        while m.shape[0] < D:
            m = torch.cat((torch.cat((m, m), 1), torch.cat((m, -m), 1)), 0) * r
    elif rot in (HALF, INTERLEAVED):
        m = torch.zeros_like(m)
        o = 0
        for s in seg:
            for i in range(s // 2):
                u, v = (o + i, o + i + s // 2) if rot == HALF else (o + 2 * i, o + 2 * i + 1)
                m[u, o + 2 * i] = m[v, o + 2 * i] = m[u, o + 2 * i + 1] = r
                m[v, o + 2 * i + 1] = -r
            o += s
    return m
