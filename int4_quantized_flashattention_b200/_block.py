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

from . import Problem, _check, _in_dtype, lib

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
    L.ra_qk_norm_rope.argtypes = [P, i, i, C.c_float, i] + [vp] * 13
    L.ra_kv4_append.argtypes = [vp, i, i, i] + [vp] * 5 + [i] + [vp] * 3
    L.ra_kv4_read.argtypes = [vp, i, i, i, vp, i] + [vp] * 5
    L.ra_attn_kv4_workspace_bytes.restype = sz
    L.ra_attn_kv4_workspace_bytes.argtypes = [vp, vp]
    L.ra_attn_kv4.argtypes = [vp] * 7 + [sz] + [vp] * 3
    L.ra_attn_cross.argtypes = [vp] * 11
    for name in ("ra_rope_table", "ra_qk_norm_rope", "ra_kv4_append", "ra_kv4_read", "ra_attn_kv4", "ra_attn_cross"):
        getattr(L, name).restype = i


_SAME = contextlib.nullcontext()


def _on(dev: torch.device, stream):
    """Context in which `dev` is the current device and `stream`, if given, the current stream."""
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        return torch.cuda.stream(stream)
    return _SAME if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _current() -> int:
    return torch.cuda.current_stream().cuda_stream


def _arg(t: Optional[torch.Tensor], dtype, shape, dev, name: str) -> Optional[int]:
    """Address of a contiguous tensor of the given dtype and shape on `dev`; None for None."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, got "
                         f"{t.dtype}, {tuple(t.shape)}, strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _view(t: torch.Tensor, dtype, shape, dev, name: str):
    """Address and Strides of a [B, H, N, D] tensor with contiguous channels."""
    if t.dtype != dtype or t.shape != shape or t.device != dev:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {dev}, got {t.dtype}, "
                         f"{tuple(t.shape)} on {t.device}")
    b, h, n, d = t.stride()
    if d != 1:
        raise ValueError(f"{name} must have contiguous channels, got strides {t.stride()}")
    return t.data_ptr(), Strides(b, h, n)


def _cuda4(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda or t.dim() != 4:
        raise ValueError(f"{name} must be a four-dimensional CUDA tensor")
    return t.device


def rope_table(p: Problem, device="cuda", stream=None) -> torch.Tensor:
    """ra_rope_table: the RoPE table of p (grid, seg, theta, rot), fp32 [entries, 2]; build it once and keep it."""
    n = int(lib().ra_rope_table_bytes(C.byref(p)))
    if n == 0:
        raise ValueError("invalid problem")
    dev = torch.empty(0, device=device).device
    with _on(dev, stream):
        t = torch.empty(n // 8, 2, dtype=torch.float32, device=dev)
        _check("ra_rope_table", lib().ra_rope_table(C.byref(p), t.data_ptr(), n, _current()))
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
    dev, dt = _cuda4(some, "q" if q is not None else "k"), some.dtype
    L, D = lib(), p.D
    Hk = k.shape[1] if k is not None and k.dim() == 4 else p.H
    qs, ks = (p.B, p.H, p.N, D), (p.B, Hk, p.N, D)
    qp = qst = kp = kst = None
    if q is not None:
        qp, qst = _view(q, dt, qs, dev, "q")
        qst = C.byref(qst)
    if k is not None:
        kp, kst = _view(k, dt, ks, dev, "k")
        kst = C.byref(kst)
    if table is not None and 8 * table.shape[0] < L.ra_rope_table_bytes(C.byref(p)):
        raise ValueError("table is shorter than the RoPE table of p")
    f32, bf16 = torch.float32, torch.bfloat16
    with _on(dev, stream):
        if q is None:
            q_out = None
        elif q_out is None:
            q_out = torch.empty(qs, dtype=bf16, device=dev)
        if k is None:
            k_out = None
        elif k_out is None:
            k_out = torch.empty(ks, dtype=bf16, device=dev)
        _check("ra_qk_norm_rope", L.ra_qk_norm_rope(
            C.byref(p), Hk, norm, eps, _in_dtype(some), qp, qst, kp, kst,
            _arg(q_weight, f32, (D,), dev, "q_weight"), _arg(k_weight, f32, (D,), dev, "k_weight"),
            _arg(q_bias, f32, (D,), dev, "q_bias"), _arg(k_bias, f32, (D,), dev, "k_bias"),
            _arg(pos, torch.int32, (p.N, 3), dev, "pos"),
            None if table is None else _arg(table, f32, (table.shape[0], 2), dev, "table"),
            _arg(q_out, bf16, qs, dev, "q_out"), _arg(k_out, bf16, ks, dev, "k_out"), _current()))
    return q_out, k_out


class KV4Cache:
    """A paged 4-bit key/value cache (ra_kv4_cache): codes k4, v4 [num_pages, Hk, page_size, D/2] uint8 and scales
    sk, sv [num_pages, Hk, page_size] fp32.  Only a handle: the tensors are the caller's, kept alive by it."""

    def __init__(self, k4: torch.Tensor, sk: torch.Tensor, v4: torch.Tensor, sv: torch.Tensor):
        dev = _cuda4(k4, "k4")
        n, hk, page, half = k4.shape
        self.k4, self.sk, self.v4, self.sv, self.device = k4, sk, v4, sv, dev
        self.num_pages, self.Hk, self.page_size, self.D = n, hk, page, 2 * half
        codes, scales = (n, hk, page, half), (n, hk, page)
        self._c = _Kv4Cache(n, page, hk, 2 * half, _arg(k4, torch.uint8, codes, dev, "k4"),
                            _arg(sk, torch.float32, scales, dev, "sk"), _arg(v4, torch.uint8, codes, dev, "v4"),
                            _arg(sv, torch.float32, scales, dev, "sv"))
        self._ref = C.byref(self._c)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, Hk: int, D: int, device="cuda") -> "KV4Cache":
        """A cache of zeros."""
        def codes():
            return torch.zeros(num_pages, Hk, page_size, D // 2, dtype=torch.uint8, device=device)

        def scales():
            return torch.zeros(num_pages, Hk, page_size, dtype=torch.float32, device=device)
        return cls(codes(), scales(), codes(), scales())


def _table(cache: KV4Cache, t: torch.Tensor, B: int) -> int:
    if t.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    return _arg(t, torch.int32, (B, t.shape[1]), cache.device, "block_table")


def kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
               start: Optional[torch.Tensor] = None, n_new: Optional[torch.Tensor] = None, stream=None) -> None:
    """ra_kv4_append: quantises k, v [B, Hk, T, D] (any strides with contiguous channels) into the cache at
    positions start[b] + 0 .. n_new[b] - 1 of each sequence."""
    dev = cache.device
    _cuda4(k, "k")
    B, T = k.shape[0], k.shape[2]
    shape = (B, cache.Hk, T, cache.D)
    kp, ks = _view(k, k.dtype, shape, dev, "k")
    vp, vs = _view(v, k.dtype, shape, dev, "v")
    with _on(dev, stream):
        _check("ra_kv4_append", lib().ra_kv4_append(
            cache._ref, _in_dtype(k), B, T, kp, C.byref(ks), vp, C.byref(vs), _table(cache, block_table, B),
            block_table.shape[1], _arg(start, torch.int32, (B,), dev, "start"),
            _arg(n_new, torch.int32, (B,), dev, "n_new"), _current()))


def kv4_read(cache: KV4Cache, block_table: torch.Tensor, start: Optional[torch.Tensor], T: int,
             n: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
             out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """ra_kv4_read: tokens start[b] .. start[b] + n[b] - 1 as code * scale in dense k, v [B, Hk, T, D]; rows at and
    past n[b] are left as they were."""
    dev, B = cache.device, block_table.shape[0]
    shape = (B, cache.Hk, T, cache.D)
    with _on(dev, stream):
        if out is None:
            out = (torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev))
        k, v = out
        _check("ra_kv4_read", lib().ra_kv4_read(
            cache._ref, _in_dtype(k), B, T, _table(cache, block_table, B), block_table.shape[1],
            _arg(start, torch.int32, (B,), dev, "start"), _arg(n, torch.int32, (B,), dev, "n"),
            _arg(k, k.dtype, shape, dev, "k"), _arg(v, k.dtype, shape, dev, "v"), _current()))
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
    dev = _cuda4(q, "q")
    shape = q.shape
    B, H, Nq, D = shape
    if dev != cache.device or D != cache.D:
        raise ValueError(f"q must have {cache.D} channels and be on {cache.device}, got {D} on {dev}")
    table = _table(cache, block_table, B)
    pages = block_table.shape[1]
    a = C.byref(_Kv4Attn(B, H, Nq, pages, pages * cache.page_size if max_len is None else max_len,
                         1 if causal else 0, _scale(scale, D)))
    L = lib()
    with _on(dev, stream):
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        if workspace is None:
            need = L.ra_attn_kv4_workspace_bytes(cache._ref, a)
            wp = None
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
                wp = workspace.data_ptr()
        else:
            need = workspace.numel()
            wp = _arg(workspace, torch.uint8, (need,), dev, "workspace")
        _check("ra_attn_kv4", L.ra_attn_kv4(
            cache._ref, a, _arg(q, torch.bfloat16, shape, dev, "q"), table,
            _arg(seq_lens, torch.int32, (B,), dev, "seq_lens"), _arg(q_lens, torch.int32, (B,), dev, "q_lens"),
            wp, need, _arg(out, torch.bfloat16, shape, dev, "out"),
            _arg(lse, torch.float32, (B, H, Nq), dev, "lse"), _current()))
    return out


def attn_cross(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_lens: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ra_attn_cross: attention of q [B, H, Nq, D] to an encoder's k, v [B, Hk, Nk, D], bf16 with any strides that
    keep the channels contiguous; keys at and past kv_lens[b] take no part.  Returns out, dense unless given."""
    dev = _cuda4(q, "q")
    _cuda4(k, "k")
    bf16, shape = torch.bfloat16, q.shape
    B, H, Nq, D = shape
    Hk, Nk = k.shape[1], k.shape[2]
    qp, qs = _view(q, bf16, shape, dev, "q")
    kp, ks = _view(k, bf16, (B, Hk, Nk, D), dev, "k")
    vp, vs = _view(v, bf16, (B, Hk, Nk, D), dev, "v")
    with _on(dev, stream):
        if out is None:
            out = torch.empty(shape, dtype=bf16, device=dev)
        op, os_ = _view(out, bf16, shape, dev, "out")
        _check("ra_attn_cross", lib().ra_attn_cross(
            C.byref(_CrossProblem(B, H, Hk, Nq, Nk, D, _scale(scale, D))), qp, C.byref(qs), kp, C.byref(ks), vp,
            C.byref(vs), _arg(kv_lens, torch.int32, (B,), dev, "kv_lens"), op, C.byref(os_),
            _arg(lse, torch.float32, (B, H, Nq), dev, "lse"), _current()))
    return out
