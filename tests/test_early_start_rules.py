"""Source rules of kernels that start before the one ahead of them has ended (no GPU): each waits for it, and none
reads through the read-only path, which is for memory that nothing writes from the kernel's start on."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_quantized_flashattention_b200",
                    "csrc")


def _sources():
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as h:
            text = re.sub(r"//[^\n]*", "", h.read())
        yield f, text


EARLY = {f: t for f, t in _sources() if f.endswith(".cu") and "launch_early(" in t}


def test_there_are_such_kernels():
    assert set(EARLY) == {"ra_kv4.cu", "ra_attn_tiles.cu", "ra_norm_rope.cu"}
    assert not any("<<<" in t for t in EARLY.values())


def test_each_kernel_waits():
    for f, t in EARLY.items():
        assert t.count("__global__") == len(re.findall(r"\bgrid_wait\(\);", t)), f


def test_no_read_only_loads():
    shared = [t for f, t in _sources() if f in ("ra_kv4.cuh", "ra_tmem_row.cuh", "ra_block.h")]
    for t in list(EARLY.values()) + shared:
        assert "__ldg(" not in t and "ld.global.nc" not in t and "__restrict__" not in t


def test_shared_loads_take_the_ordinary_form():
    for f, t in EARLY.items():
        assert len(re.findall(r"\bload_raw8<kBf16, false>\(", t)) == len(re.findall(r"\bload_raw8<", t)), f
        assert len(re.findall(r"\brope_coef8p<false>\(", t)) == len(re.findall(r"\brope_coef8p\b", t)), f
