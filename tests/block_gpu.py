"""Helpers of the GPU tests of the 4-bit cache."""
from __future__ import annotations

import math

import torch


def rand(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def make_cache(ra, gen, B, pages_each, page, Hk, D):
    """A cache whose unused slots hold codes of all ones and NaN scales, and a shuffled block table."""
    n = B * pages_each + 2
    c = ra.KV4Cache.empty(n, page, Hk, D)
    table = torch.randperm(n, generator=gen, device="cuda")[:B * pages_each].reshape(B, pages_each).to(torch.int32)
    for codes, scale in ((c.k4, c.sk), (c.v4, c.sv)):
        codes.fill_(255)
        scale.fill_(math.nan)
    return c, table.contiguous()


def filled(ra, gen, lens, page, k, v):
    """The first lens[b] tokens of k, v [B, Hk, T, D] in a cache: (cache, table, lengths)."""
    B, Hk, T, D = k.shape
    c, table = make_cache(ra, gen, B, max(1, -(-max(lens) // page)), page, Hk, D)
    lens_t = torch.tensor(lens, device="cuda", dtype=torch.int32)
    ra.kv4_append(c, k, v, table, None, lens_t)
    return c, table, lens_t
