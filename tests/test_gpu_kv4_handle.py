"""A KV4Cache is its four tensors, as they are at the time of a call."""
import pytest
import torch

from tests import block_gpu as bg
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import int4_quantized_flashattention_b200 as ra
    gu.device()
    return ra


@pytest.mark.parametrize("name", ["k4", "sk", "v4", "sv", "index", "num_pages", "Hk", "page_size", "D"])
def test_fields_are_read_only(ra, name):
    c = ra.KV4Cache.empty(4, 16, 2, 64)
    with pytest.raises(AttributeError):
        setattr(c, name, getattr(c, name))


def test_tensors_moved_to_other_memory(ra):
    """In-place changes of storage and shape between calls: the new memory is written and read, or the call refused."""
    gen = torch.Generator(device="cuda").manual_seed(17)
    c = ra.KV4Cache.empty(4, 16, 2, 64)
    table = torch.tensor([[2, 1]], device="cuda", dtype=torch.int32)
    k, v = bg.rand(gen, 1, 2, 20, 64), bg.rand(gen, 1, 2, 20, 64)
    ra.kv4_append(c, k, v, table)
    first = ra.kv4_read(c, table, None, 20)
    old = [t.detach().clone() for t in (c.k4, c.sk, c.v4, c.sv)]
    keep = [torch.zeros(6, *t.shape[1:], dtype=t.dtype, device="cuda") for t in old]
    held = [t.untyped_storage() for t in (c.k4, c.sk, c.v4, c.sv)]   # the old memory stays allocated
    for t, new in zip((c.k4, c.sk, c.v4, c.sv), keep):
        t.set_(new)
    assert c.num_pages == 6
    assert all(bool((x == 0).all()) for x in ra.kv4_read(c, table, None, 20))
    ra.kv4_append(c, 2 * k, v, table)
    again = ra.kv4_read(c, table, None, 20)
    assert torch.equal(again[0], 2 * first[0]) and torch.equal(again[1], first[1])
    for s, t in zip(held, old):                                      # untouched
        assert torch.equal(torch.empty(0, dtype=t.dtype, device="cuda").set_(s).view(t.shape), t)
    q = bg.rand(gen, 1, 2, 1, 64, dtype=torch.bfloat16)
    lens = torch.tensor([20], device="cuda", dtype=torch.int32)
    assert torch.equal(ra.attn_kv4(c, q, table, lens), ra.attn_kv4(ra.KV4Cache(*keep), q, table, lens))
    c.sk.set_(keep[1][:5])                                           # no longer one cache
    for call in (lambda: ra.kv4_append(c, k, v, table), lambda: ra.kv4_read(c, table, None, 20),
                 lambda: ra.attn_kv4(c, q, table, lens), lambda: ra.attn_kv4_workspace_bytes(c, 1, 2, 1, 20)):
        with pytest.raises(ValueError):
            call()
    assert ra.sync_status() == 0
