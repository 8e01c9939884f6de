"""The operators around the attention: norm + RoPE, the 4-bit key/value cache, attention over it and cross attention.
Their tensors may live on any one CUDA device: a call runs on that device, on `stream` or the device's current stream,
and buffers made here are allocated in that stream's order.  The checks and the call of the C entry of the same name
are in csrc/ra_bind.cpp (module _bind).
"""
from __future__ import annotations

import contextlib
import ctypes as C
from typing import Optional, Tuple

import torch

from . import Problem, RaError, _check, lib

NORM_RMS, NORM_LAYER = 0, 1                   # ra_norm_mode


class Strides(C.Structure):
    """ra_strides: element strides of a [B, H, N, D] tensor with contiguous channels."""
    _fields_ = [("b", C.c_int64), ("h", C.c_int64), ("n", C.c_int64)]


class _Kv4Cache(C.Structure):
    """ra_kv4_cache."""
    _fields_ = [("num_pages", C.c_int), ("page_size", C.c_int), ("Hk", C.c_int), ("D", C.c_int),
                ("k4", C.c_void_p), ("sk", C.c_void_p), ("v4", C.c_void_p), ("sv", C.c_void_p)]


class _Kv4Attn(C.Structure):
    """ra_kv4_attn."""
    _fields_ = [("B", C.c_int), ("H", C.c_int), ("Nq", C.c_int), ("max_pages", C.c_int), ("max_len", C.c_int),
                ("causal", C.c_int), ("scale", C.c_float)]


class _CrossProblem(C.Structure):
    """ra_cross_problem."""
    _fields_ = [("B", C.c_int), ("H", C.c_int), ("Hk", C.c_int), ("Nq", C.c_int), ("Nk", C.c_int), ("D", C.c_int),
                ("scale", C.c_float)]


def declare(L) -> None:
    """Argument types of the entry points of this module."""
    P, vp, sz, i = C.POINTER(Problem), C.c_void_p, C.c_size_t, C.c_int
    L.ra_rope_table_bytes.restype = sz
    L.ra_rope_table_bytes.argtypes = [P]
    L.ra_rope_table.argtypes = [P, vp, sz, vp]
    L.ra_qk_norm_rope.argtypes = [P, i, i, C.c_float, i] + [vp] * 10 + [sz] + [vp] * 3
    L.ra_kv4_append.argtypes = [vp, i, i, i] + [vp] * 5 + [i] + [vp] * 3
    L.ra_kv4_read.argtypes = [vp, i, i, i, vp, i] + [vp] * 5
    L.ra_attn_kv4_workspace_bytes.restype = sz
    L.ra_attn_kv4_workspace_bytes.argtypes = [vp, vp]
    L.ra_attn_kv4.argtypes = [vp] * 7 + [sz] + [vp] * 3
    L.ra_attn_cross.argtypes = [vp] * 11
    for name in ("ra_rope_table", "ra_qk_norm_rope", "ra_kv4_append", "ra_kv4_read", "ra_attn_kv4", "ra_attn_cross"):
        getattr(L, name).restype = i


_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_ext = None


def _bind():
    """The compiled binding; loads it, and libra.so with it, on first use."""
    global _ext
    if _ext is None:
        lib()
        try:
            from . import _bind as ext
        except ImportError as e:
            raise RuntimeError("the compiled binding is missing: build it with __graft_entry__.build()") from e
        ext.set_errors(RaError, torch.OutOfMemoryError)
        _ext = ext
    return _ext


@contextlib.contextmanager
def _on(idx: int, stream):
    """Device `idx` as the current device and `stream` (a stream or its handle), if given, as the current stream."""
    with torch.cuda.device(idx):
        if stream is None:
            yield
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=idx)
            with torch.cuda.stream(stream):
                yield


def _run(fn: str, idx: int, stream, *args):
    """The binding's `fn` on a stream of device `idx`."""
    if idx < 0:
        raise ValueError("the tensors must be on a CUDA device")
    with _on(idx, stream):
        return getattr(_bind(), fn)(*args)


def rope_table(p: Problem, device="cuda", stream=None) -> torch.Tensor:
    """ra_rope_table: the RoPE table of p (grid, seg, theta, rot), fp32 [entries, 2]; build it once and keep it."""
    n = int(lib().ra_rope_table_bytes(C.byref(p)))
    if n == 0:
        raise ValueError("invalid problem")
    if torch.device(device).type != "cuda":
        raise ValueError("device must be a CUDA device")
    idx = torch.empty(0, device=device).get_device()
    with _on(idx, stream):
        t = torch.empty(n // 8, 2, dtype=_F32, device="cuda")
        st = torch.cuda.current_stream().cuda_stream
        _check("ra_rope_table", lib().ra_rope_table(C.byref(p), t.data_ptr(), n, st))
    return t


def qk_norm_rope(p: Problem, q: Optional[torch.Tensor], k: Optional[torch.Tensor], table: Optional[torch.Tensor],
                 pos: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, q_bias: Optional[torch.Tensor] = None,
                 k_bias: Optional[torch.Tensor] = None, norm: int = NORM_RMS, eps: float = 1e-6,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """ra_qk_norm_rope: per-head norm of q [B, H, N, D] and k [B, Hk, N, D] (any strides with contiguous channels,
    e.g. token-major projections seen as x.view(B, N, H, D).transpose(1, 2)), 3D RoPE and the rotation p.rot.
    Returns dense bf16 (q_out, k_out); q or k may be None.  table and pos None: the norm alone."""
    args = (p, q, k, table, pos, q_weight, k_weight, q_bias, k_bias, norm, eps, q_out, k_out)
    if stream is not None:
        some = q if q is not None else k
        return _run("qk_norm_rope", -1 if some is None else some.get_device(), stream, *args)
    return (_ext or _bind()).qk_norm_rope(*args)


class KV4Cache:
    """A paged 4-bit key/value cache (ra_kv4_cache): codes k4, v4 [num_pages, Hk, page_size, D/2] uint8 and scales
    sk, sv [num_pages, Hk, page_size] fp32.  Only a handle: the tensors are the caller's, kept alive by it.  They
    cannot be exchanged for others, and every call looks at them as they then are."""

    __slots__ = ("_tensors", "_index")

    def __init__(self, k4: torch.Tensor, sk: torch.Tensor, v4: torch.Tensor, sv: torch.Tensor):
        (_ext or _bind()).kv4_cache(k4, sk, v4, sv)  # checks them
        self._tensors, self._index = (k4, sk, v4, sv), k4.get_device()

    k4 = property(lambda self: self._tensors[0])
    sk = property(lambda self: self._tensors[1])
    v4 = property(lambda self: self._tensors[2])
    sv = property(lambda self: self._tensors[3])
    index = property(lambda self: self._index, doc="Index of the CUDA device.")
    num_pages = property(lambda self: self.k4.shape[0])
    Hk = property(lambda self: self.k4.shape[1])
    page_size = property(lambda self: self.k4.shape[2])
    D = property(lambda self: 2 * self.k4.shape[3])

    @classmethod
    def empty(cls, num_pages: int, page_size: int, Hk: int, D: int, device="cuda") -> "KV4Cache":
        """A cache of zeros."""
        def codes():
            return torch.zeros(num_pages, Hk, page_size, D // 2, dtype=_U8, device=device)

        def scales():
            return torch.zeros(num_pages, Hk, page_size, dtype=_F32, device=device)
        return cls(codes(), scales(), codes(), scales())


def kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
               start: Optional[torch.Tensor] = None, n_new: Optional[torch.Tensor] = None, stream=None) -> None:
    """ra_kv4_append: quantises k, v [B, Hk, T, D] (any strides with contiguous channels) into the cache at
    positions start[b] + 0 .. n_new[b] - 1 of each sequence."""
    if stream is not None:
        return _run("kv4_append", cache._index, stream, cache._tensors, cache._index, k, v, block_table, start,
                    n_new)
    return (_ext or _bind()).kv4_append(cache._tensors, cache._index, k, v, block_table, start, n_new)


def kv4_read(cache: KV4Cache, block_table: torch.Tensor, start: Optional[torch.Tensor], T: int,
             n: Optional[torch.Tensor] = None, dtype: torch.dtype = _BF16,
             out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """ra_kv4_read: tokens start[b] .. start[b] + n[b] - 1 as code * scale in dense k, v [B, Hk, T, D]; rows at and
    past n[b] are left as they were."""
    if dtype is not _BF16 and dtype is not _F32:
        raise ValueError("dtype must be bfloat16 or float32")
    k, v = (None, None) if out is None else out
    if (k is None) != (v is None):
        raise ValueError("out must hold both tensors")
    args = (cache._tensors, cache._index, block_table, start, T, n, dtype is _F32, k, v)
    if stream is not None:
        return _run("kv4_read", cache._index, stream, *args)
    return (_ext or _bind()).kv4_read(*args)


def attn_kv4_workspace_bytes(cache: KV4Cache, B: int, H: int, Nq: int, max_len: int) -> int:
    """Bytes of workspace attn_kv4 needs for queries [B, H, Nq, D] and sequences of up to max_len keys."""
    a = _Kv4Attn(B, H, Nq, 1, max_len, 0, 1.0)
    return int(lib().ra_attn_kv4_workspace_bytes(_bind().kv4_cache(*cache._tensors), C.byref(a)))


def attn_kv4(cache: KV4Cache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
             q_lens: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None,
             max_len: Optional[int] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ra_attn_kv4: attention of q [B, H, Nq, D] bf16 over the cache; returns out [B, H, Nq, D] bf16.  max_len is a
    bound on seq_lens that the split of the keys is planned for (the block table's reach by default)."""
    args = (cache._tensors, cache._index, q, block_table, seq_lens, q_lens, causal, scale, max_len, out, lse, workspace)
    if stream is not None:
        return _run("attn_kv4", cache._index, stream, *args)
    return (_ext or _bind()).attn_kv4(*args)


def attn_cross(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_lens: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ra_attn_cross: attention of q [B, H, Nq, D] to an encoder's k, v [B, Hk, Nk, D], bf16 with any strides that
    keep the channels contiguous; keys at and past kv_lens[b] take no part.  Returns out, dense unless given."""
    if stream is not None:
        return _run("attn_cross", q.get_device(), stream, q, k, v, kv_lens, scale, out, lse)
    return (_ext or _bind()).attn_cross(q, k, v, kv_lens, scale, out, lse)
