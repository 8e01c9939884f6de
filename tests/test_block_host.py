"""Host-side validation of the operators around the attention (no GPU): every
refusal comes before a launch.  Fake pointers stand for device memory; checks
that would reach a launch run only where no GPU is visible."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import int4_quantized_flashattention_b200 as ra
    ra.lib()
    return ra


GOOD, BAD16, BAD4 = 0x10000, 0x10008, 0x10002
INVALID, UNSUPPORTED, CUDA = 1, 2, 3


def _problem(ra, **kw):
    args = dict(B=2, H=4, D=128, seg=(44, 42, 42), grid=(3, 5, 7), rot=0)
    args.update(kw)
    return ra.Problem.make(args.pop("B"), args.pop("H"), args.pop("D"), args.pop("seg"), args.pop("grid"), **args)


def _st(ra, b, h, n):
    return ra._block.Strides(b, h, n)


def _norm(ra, p=None, Hk=4, norm=0, eps=1e-6, dt=1, q=GOOD, qst=None, k=GOOD, kst=None, qw=GOOD, kw=GOOD, qb=None,
          kb=None, pos=GOOD, table=GOOD, tb=1 << 20, qo=GOOD, ko=GOOD):
    p = p or _problem(ra)
    dense = _st(ra, 4 * 105 * 128, 105 * 128, 128)
    return ra.lib().ra_qk_norm_rope(C.byref(p), Hk, norm, eps, dt, q, C.byref(qst or dense), k, C.byref(kst or dense),
                                    qw, kw, qb, kb, pos, table, tb, qo, ko, None)


def _reaches_launch(rc):
    assert rc == CUDA, rc


@pytest.mark.parametrize("kw", [
    dict(Hk=0), dict(norm=2), dict(norm=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(dt=2), dict(q=BAD16),
    dict(k=BAD16), dict(q=None), dict(qo=None), dict(ko=None), dict(k=None), dict(pos=None), dict(table=None),
    dict(table=BAD16), dict(tb=2543), dict(pos=BAD4), dict(qw=BAD4), dict(qo=BAD16), dict(q=None, qo=None, k=None, ko=None),
    dict(Hk=1 << 20)])
def test_norm_rope_refusals(ra, kw):
    assert _norm(ra, **kw) in (INVALID, UNSUPPORTED)


@pytest.mark.parametrize("st", [(4, 128, 4), (0, 13440, 128), (53760, 0, 128), (53760, 13440, 0), (53760, 13440, -128),
                                (53760, 13440, 129), (1 << 40, 13440, 128)])
def test_norm_rope_refuses_strides(ra, st):
    assert _norm(ra, qst=_st(ra, *st)) == INVALID
    assert _norm(ra, kst=_st(ra, *st)) == INVALID


def test_norm_rope_refuses_bad_problems(ra):
    for field, value in (("D", 96), ("N", 0), ("rot", 4), ("B", 0)):
        p = _problem(ra)
        setattr(p, field, value)
        assert _norm(ra, p=p) == INVALID


def test_stride_of_an_extent_of_one_is_not_looked_at(ra):
    if torch.cuda.is_available():
        pytest.skip("reaches a launch with fake pointers; host-only check")
    p = _problem(ra, B=1, H=1)
    _reaches_launch(_norm(ra, p=p, Hk=1, qst=_st(ra, 3, 0, 128), kst=_st(ra, -1, 7, 128)))


def test_rope_table_bytes(ra):
    p = _problem(ra)
    assert ra.lib().ra_rope_table_bytes(C.byref(p)) == 8 * (3 * 22 + 5 * 21 + 7 * 21)
    assert ra.lib().ra_rope_table(C.byref(p), GOOD, 8, None) == INVALID
    assert ra.lib().ra_rope_table(C.byref(p), None, 1 << 20, None) == INVALID
    p.D = 96
    assert ra.lib().ra_rope_table_bytes(C.byref(p)) == 0


def _cache(ra, num_pages=9, page=16, Hk=2, D=128, k4=GOOD, sk=GOOD, v4=GOOD, sv=GOOD):
    return ra._block._Kv4Cache(num_pages, page, Hk, D, k4, sk, v4, sv)


BAD_CACHES = [dict(num_pages=0), dict(page=8), dict(page=48), dict(page=256), dict(Hk=0), dict(D=96), dict(k4=None),
              dict(sk=BAD16), dict(v4=BAD16), dict(sv=None)]


def _append(ra, c, dt=1, B=2, T=5, k=GOOD, kst=(1280, 640, 128), v=GOOD, vst=(1280, 640, 128), table=GOOD, pages=4,
            start=GOOD, n=None):
    return ra.lib().ra_kv4_append(C.byref(c), dt, B, T, k, C.byref(_st(ra, *kst)), v, C.byref(_st(ra, *vst)), table,
                                  pages, start, n, None)


def _read(ra, c, dt=0, B=2, T=5, table=GOOD, pages=4, start=GOOD, n=None, k=GOOD, v=GOOD):
    return ra.lib().ra_kv4_read(C.byref(c), dt, B, T, table, pages, start, n, k, v, None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_cache_refusals(ra, kw):
    c = _cache(ra, **kw)
    assert _append(ra, c) == INVALID
    assert _read(ra, c) == INVALID
    assert _attn(ra, c=c) == INVALID


@pytest.mark.parametrize("kw", [dict(dt=3), dict(B=0), dict(B=70000), dict(T=0), dict(table=None), dict(table=BAD4),
                                dict(pages=0), dict(pages=1 << 30), dict(start=BAD4), dict(n=BAD4), dict(k=BAD16),
                                dict(v=None)])
def test_append_and_read_refusals(ra, kw):
    assert _append(ra, _cache(ra), **kw) == INVALID
    assert _read(ra, _cache(ra), **kw) == INVALID


def test_append_refuses_strides(ra):
    for st in ((1280, 640, 0), (1280, 641, 128), (-8, 640, 128)):
        assert _append(ra, _cache(ra), kst=st) == INVALID
        assert _append(ra, _cache(ra), vst=st) == INVALID
    assert _append(ra, _cache(ra), dt=0, kst=(1280, 640, 130)) == INVALID


def _attn(ra, c=None, B=2, H=4, Nq=1, pages=4, max_len=64, causal=0, scale=0.1, q=GOOD, table=GOOD, lens=GOOD,
          qlens=None, ws=None, ws_bytes=0, out=GOOD, lse=None):
    c = c or _cache(ra)
    a = ra._block._Kv4Attn(B, H, Nq, pages, max_len, causal, scale)
    return ra.lib().ra_attn_kv4(C.byref(c), C.byref(a), q, table, lens, qlens, ws, ws_bytes, out, lse, None)


@pytest.mark.parametrize("kw", [dict(B=0), dict(H=3), dict(H=0), dict(Nq=0), dict(pages=0), dict(max_len=-1),
                                dict(causal=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                                dict(q=BAD16), dict(table=None), dict(lens=None), dict(lens=BAD4), dict(qlens=BAD4),
                                dict(out=BAD16), dict(lse=BAD4), dict(B=70000)])
def test_attn_kv4_refusals(ra, kw):
    assert _attn(ra, **kw) == INVALID


def test_attn_kv4_workspace(ra):
    c = _cache(ra, num_pages=4000)
    a = ra._block._Kv4Attn(1, 4, 1, 2000, 32000, 0, 0.1)
    need = ra.lib().ra_attn_kv4_workspace_bytes(C.byref(c), C.byref(a))
    assert need > 0 and need % (4 * 129 * 4) == 0   # parts x rows x (D + 1) floats
    kw = dict(c=c, B=1, pages=2000, max_len=32000)
    assert _attn(ra, **kw) == INVALID                                    # no workspace
    assert _attn(ra, **kw, ws=GOOD, ws_bytes=need - 1) == INVALID
    assert _attn(ra, **kw, ws=BAD16, ws_bytes=need) == INVALID
    a.max_len = 16                                                       # short: one part, none needed
    assert ra.lib().ra_attn_kv4_workspace_bytes(C.byref(c), C.byref(a)) == 0
    if not torch.cuda.is_available():
        _reaches_launch(_attn(ra, **kw, ws=GOOD, ws_bytes=need))


def _cross(ra, B=2, H=4, Hk=2, Nq=9, Nk=7, D=128, scale=0.1, q=GOOD, k=GOOD, v=GOOD, out=GOOD, lens=None, lse=None,
           qst=(4608, 1152, 128), kst=(1792, 896, 128), vst=(1792, 896, 128), ost=(4608, 1152, 128)):
    p = ra._block._CrossProblem(B, H, Hk, Nq, Nk, D, scale)
    s = [C.byref(_st(ra, *x)) for x in (qst, kst, vst, ost)]
    return ra.lib().ra_attn_cross(C.byref(p), q, s[0], k, s[1], v, s[2], lens, out, s[3], lse, None)


@pytest.mark.parametrize("kw", [dict(B=0), dict(H=3), dict(Hk=0), dict(Nq=0), dict(Nk=0), dict(D=80), dict(scale=0.0),
                                dict(scale=float("nan")), dict(q=None), dict(k=BAD16), dict(v=BAD16), dict(out=None),
                                dict(lens=BAD4), dict(lse=BAD4), dict(qst=(4608, 1152, 0)), dict(kst=(1792, 0, 128)),
                                dict(vst=(1792, 896, 132)), dict(ost=(0, 1152, 128)), dict(ost=(4608, 1152, 64)), dict(ost=(4608, 120, 512)),
                                dict(Nq=(1 << 24) + 1)])
def test_attn_cross_refusals(ra, kw):
    assert _cross(ra, **kw) == INVALID


def test_python_wrappers_refuse_host_tensors_and_shapes(ra):
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ra.attn_cross(x, x, x)
    with pytest.raises(ValueError):
        ra.KV4Cache.empty(4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        ra.qk_norm_rope(_problem(ra), None, None, None, None)
    with pytest.raises(ValueError):
        ra.qk_norm_rope(_problem(ra), x, None, None, None)


def test_binding_refuses_what_is_not_a_tensor_or_structure(ra):
    """The compiled binding's own checks: no argument reaches a C entry unchecked."""
    bind = ra._block._bind()
    p, x = _problem(ra), torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    for bad in (None, 3, "q", [x]):
        with pytest.raises(ValueError):
            ra.attn_cross(bad, x, x)
        with pytest.raises(ValueError):
            ra.KV4Cache(bad, x, x, x)
    with pytest.raises(ValueError):
        ra.qk_norm_rope(p, 5, None, None, None)
    with pytest.raises(ValueError):                       # a structure of another size
        bind.kv4_append(b"short", 0, x, x, x, None, None)
    with pytest.raises(TypeError):                        # no buffer at all
        bind.kv4_append(None, 0, x, x, x, None, None)
    for name in ("qk_norm_rope", "kv4_cache", "kv4_append", "kv4_read", "attn_kv4", "attn_cross"):
        with pytest.raises(TypeError):
            getattr(bind, name)()
        with pytest.raises(TypeError):
            getattr(bind, name)(*[x] * 20)
