"""Binding of the operators around the attention: norm + RoPE, the 4-bit key/value cache, attention over it and
cross attention.  Their tensors may live on any one CUDA device: a call runs on that device, on `stream` or the
device's current stream, and buffers made here are allocated in that stream's order.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
from typing import Optional, Tuple

import torch

from . import Problem, _check, lib

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


# The wrappers are most of a small call's time, so they ask for as little as they can: the raw handle of the current
# stream and the current device's index come from torch's C module, without the objects around them.
_raw_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice
_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
_DT = {_F32: 0, _BF16: 1}                     # ra_dtype


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


def _bad(t, dtype, shape, idx, name: str):
    return ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA device {idx}, got "
                      f"{t.dtype}, {tuple(t.shape)}, strides {t.stride()} on {t.device}")


def _arg(t: Optional[torch.Tensor], dtype, shape, idx: int, name: str) -> Optional[int]:
    """Address of a contiguous tensor of the given dtype and shape on device `idx`; None for None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == idx and t.is_contiguous():
        return t.data_ptr()
    raise _bad(t, dtype, shape, idx, name)


def _view(t: torch.Tensor, dtype, shape, idx: int, name: str):
    """Address and Strides reference of a [B, H, N, D] tensor with contiguous channels."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == idx:
        b, h, n, d = t.stride()
        if d == 1:
            return t.data_ptr(), C.byref(Strides(b, h, n))
        raise ValueError(f"{name} must have contiguous channels, got strides {t.stride()}")
    raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on CUDA device {idx}, got {t.dtype}, "
                     f"{tuple(t.shape)} on {t.device}")


def _dense(B: int, H: int, N: int, D: int, dtype, dev) -> torch.Tensor:
    """A new dense [B, H, N, D] tensor (empty_strided takes two thirds of empty's time)."""
    return torch.empty_strided((B, H, N, D), (H * N * D, N * D, D, 1), dtype=dtype, device=dev)


def _cuda4(t: torch.Tensor, name: str) -> int:
    if t.dim() != 4 or not t.is_cuda:
        raise ValueError(f"{name} must be a four-dimensional CUDA tensor")
    return t.get_device()


def _dtype(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise ValueError("inputs must be bfloat16 or float32") from None


def rope_table(p: Problem, device="cuda", stream=None) -> torch.Tensor:
    """ra_rope_table: the RoPE table of p (grid, seg, theta, rot), fp32 [entries, 2]; build it once and keep it."""
    n = int(lib().ra_rope_table_bytes(C.byref(p)))
    if n == 0:
        raise ValueError("invalid problem")
    idx = torch.empty(0, device=device).get_device()
    with _on(idx, stream):
        t = torch.empty(n // 8, 2, dtype=_F32, device="cuda")
        _check("ra_rope_table", lib().ra_rope_table(C.byref(p), t.data_ptr(), n, _raw_stream(idx)))
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
    some = q if q is not None else k
    if some is None:
        raise ValueError("q or k must be given")
    idx = _cuda4(some, "q" if q is not None else "k")
    if stream is not None or idx != _device():
        with _on(idx, stream):
            return qk_norm_rope(p, q, k, table, pos, q_weight, k_weight, q_bias, k_bias, norm, eps, q_out, k_out)
    B, H, N, D = p.B, p.H, p.N, p.D
    dt = some.dtype
    Hk = H
    qp = qs = qo = kp = ks = ko = None
    if q is not None:
        shape = (B, H, N, D)
        qp, qs = _view(q, dt, shape, idx, "q")
        if q_out is None:
            q_out = _dense(B, H, N, D, _BF16, q.device)
            qo = q_out.data_ptr()
        else:
            qo = _arg(q_out, _BF16, shape, idx, "q_out")
    else:
        q_out = None
    if k is not None:
        Hk = k.shape[1] if k.dim() == 4 else H
        shape = (B, Hk, N, D)
        kp, ks = _view(k, dt, shape, idx, "k")
        if k_out is None:
            k_out = _dense(B, Hk, N, D, _BF16, k.device)
            ko = k_out.data_ptr()
        else:
            ko = _arg(k_out, _BF16, shape, idx, "k_out")
    else:
        k_out = None
    w = (D,)
    rc = lib().ra_qk_norm_rope(
        C.byref(p), Hk, norm, eps, _dtype(some), qp, qs, kp, ks, _arg(q_weight, _F32, w, idx, "q_weight"),
        _arg(k_weight, _F32, w, idx, "k_weight"), _arg(q_bias, _F32, w, idx, "q_bias"),
        _arg(k_bias, _F32, w, idx, "k_bias"), _arg(pos, _I32, (N, 3), idx, "pos"),
        None if table is None else _arg(table, _F32, (len(table), 2), idx, "table"),
        0 if table is None else 8 * len(table), qo, ko, _raw_stream(idx))
    if rc:
        _check("ra_qk_norm_rope", rc)
    return q_out, k_out


class KV4Cache:
    """A paged 4-bit key/value cache (ra_kv4_cache): codes k4, v4 [num_pages, Hk, page_size, D/2] uint8 and scales
    sk, sv [num_pages, Hk, page_size] fp32.  Only a handle: the tensors are the caller's, kept alive by it."""

    def __init__(self, k4: torch.Tensor, sk: torch.Tensor, v4: torch.Tensor, sv: torch.Tensor):
        idx = _cuda4(k4, "k4")
        codes = k4.shape
        n, hk, page, half = codes
        scales = codes[:3]
        self.k4, self.sk, self.v4, self.sv, self.index = k4, sk, v4, sv, idx
        self.num_pages, self.Hk, self.page_size, self.D = n, hk, page, 2 * half
        self._c = _Kv4Cache(n, page, hk, 2 * half, _arg(k4, _U8, codes, idx, "k4"), _arg(sk, _F32, scales, idx, "sk"),
                            _arg(v4, _U8, codes, idx, "v4"), _arg(sv, _F32, scales, idx, "sv"))
        self._ref = C.byref(self._c)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, Hk: int, D: int, device="cuda") -> "KV4Cache":
        """A cache of zeros."""
        def codes():
            return torch.zeros(num_pages, Hk, page_size, D // 2, dtype=_U8, device=device)

        def scales():
            return torch.zeros(num_pages, Hk, page_size, dtype=_F32, device=device)
        return cls(codes(), scales(), codes(), scales())


def _table(cache: KV4Cache, t: torch.Tensor, B: int) -> int:
    if t.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    return _arg(t, _I32, (B, t.shape[1]), cache.index, "block_table")


def kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
               start: Optional[torch.Tensor] = None, n_new: Optional[torch.Tensor] = None, stream=None) -> None:
    """ra_kv4_append: quantises k, v [B, Hk, T, D] (any strides with contiguous channels) into the cache at
    positions start[b] + 0 .. n_new[b] - 1 of each sequence."""
    idx = cache.index
    if stream is not None or idx != _device():
        with _on(idx, stream):
            return kv4_append(cache, k, v, block_table, start, n_new)
    _cuda4(k, "k")
    B, T, dt = k.shape[0], k.shape[2], k.dtype
    shape = (B, cache.Hk, T, cache.D)
    kp, ks = _view(k, dt, shape, idx, "k")
    vp, vs = _view(v, dt, shape, idx, "v")
    b = (B,)
    rc = lib().ra_kv4_append(cache._ref, _dtype(k), B, T, kp, ks, vp, vs, _table(cache, block_table, B),
                             block_table.shape[1], _arg(start, _I32, b, idx, "start"),
                             _arg(n_new, _I32, b, idx, "n_new"), _raw_stream(idx))
    if rc:
        _check("ra_kv4_append", rc)


def kv4_read(cache: KV4Cache, block_table: torch.Tensor, start: Optional[torch.Tensor], T: int,
             n: Optional[torch.Tensor] = None, dtype: torch.dtype = _BF16,
             out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """ra_kv4_read: tokens start[b] .. start[b] + n[b] - 1 as code * scale in dense k, v [B, Hk, T, D]; rows at and
    past n[b] are left as they were."""
    idx = cache.index
    if stream is not None or idx != _device():
        with _on(idx, stream):
            return kv4_read(cache, block_table, start, T, n, dtype, out)
    B = block_table.shape[0]
    shape = (B, cache.Hk, T, cache.D)
    if out is None:
        dev = cache.k4.device
        k, v = _dense(*shape, dtype, dev), _dense(*shape, dtype, dev)
    else:
        k, v = out
    b = (B,)
    rc = lib().ra_kv4_read(cache._ref, _dtype(k), B, T, _table(cache, block_table, B), block_table.shape[1],
                           _arg(start, _I32, b, idx, "start"), _arg(n, _I32, b, idx, "n"),
                           _arg(k, k.dtype, shape, idx, "k"), _arg(v, k.dtype, shape, idx, "v"), _raw_stream(idx))
    if rc:
        _check("ra_kv4_read", rc)
    return k, v


def _scale(scale: Optional[float], D: int) -> float:
    return 1.0 / math.sqrt(D) if scale is None else float(scale)


def attn_kv4_workspace_bytes(cache: KV4Cache, B: int, H: int, Nq: int, max_len: int) -> int:
    """Bytes of workspace attn_kv4 needs for queries [B, H, Nq, D] and sequences of up to max_len keys."""
    a = _Kv4Attn(B, H, Nq, 1, max_len, 0, 1.0)
    return int(lib().ra_attn_kv4_workspace_bytes(cache._ref, C.byref(a)))


def attn_kv4(cache: KV4Cache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
             q_lens: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None,
             max_len: Optional[int] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ra_attn_kv4: attention of q [B, H, Nq, D] bf16 over the cache; returns out [B, H, Nq, D] bf16.  max_len is a
    bound on seq_lens that the split of the keys is planned for (the block table's reach by default)."""
    idx = _cuda4(q, "q")
    if stream is not None or idx != _device():
        with _on(idx, stream):
            return attn_kv4(cache, q, block_table, seq_lens, q_lens, causal, scale, max_len, out, lse, workspace)
    shape = q.shape
    B, H, Nq, D = shape
    if idx != cache.index or D != cache.D:
        raise ValueError(f"q must have {cache.D} channels and be on CUDA device {cache.index}, got {D} on {idx}")
    table = _table(cache, block_table, B)
    pages = block_table.shape[1]
    a = C.byref(_Kv4Attn(B, H, Nq, pages, pages * cache.page_size if max_len is None else max_len,
                         1 if causal else 0, _scale(scale, D)))
    L = lib()
    if out is None:
        out = _dense(B, H, Nq, D, _BF16, q.device)
        op = out.data_ptr()
    else:
        op = _arg(out, _BF16, shape, idx, "out")
    wp = None
    if workspace is None:
        need = L.ra_attn_kv4_workspace_bytes(cache._ref, a)
        if need:
            workspace = torch.empty(need, dtype=_U8, device=q.device)
            wp = workspace.data_ptr()
    else:
        need = workspace.numel()
        wp = _arg(workspace, _U8, (need,), idx, "workspace")
    b = (B,)
    rc = L.ra_attn_kv4(cache._ref, a, _arg(q, _BF16, shape, idx, "q"), table, _arg(seq_lens, _I32, b, idx, "seq_lens"),
                       _arg(q_lens, _I32, b, idx, "q_lens"), wp, need, op, _arg(lse, _F32, shape[:3], idx, "lse"),
                       _raw_stream(idx))
    if rc:
        _check("ra_attn_kv4", rc)
    return out


def attn_cross(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_lens: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ra_attn_cross: attention of q [B, H, Nq, D] to an encoder's k, v [B, Hk, Nk, D], bf16 with any strides that
    keep the channels contiguous; keys at and past kv_lens[b] take no part.  Returns out, dense unless given."""
    idx = _cuda4(q, "q")
    if stream is not None or idx != _device():
        with _on(idx, stream):
            return attn_cross(q, k, v, kv_lens, scale, out, lse)
    _cuda4(k, "k")
    shape = q.shape
    B, H, Nq, D = shape
    Hk, Nk = k.shape[1], k.shape[2]
    kshape = (B, Hk, Nk, D)
    qp, qs = _view(q, _BF16, shape, idx, "q")
    kp, ks = _view(k, _BF16, kshape, idx, "k")
    vp, vs = _view(v, _BF16, kshape, idx, "v")
    if out is None:
        out = _dense(B, H, Nq, D, _BF16, q.device)
    op, os_ = _view(out, _BF16, shape, idx, "out")
    rc = lib().ra_attn_cross(C.byref(_CrossProblem(B, H, Hk, Nq, Nk, D, _scale(scale, D))), qp, qs, kp, ks, vp, vs,
                             _arg(kv_lens, _I32, (B,), idx, "kv_lens"), op, os_,
                             _arg(lse, _F32, shape[:3], idx, "lse"), _raw_stream(idx))
    if rc:
        _check("ra_attn_cross", rc)
    return out
