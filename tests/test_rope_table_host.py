"""The RoPE table is made on a CUDA device or not at all (no GPU)."""
import pytest
import torch


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), "meta"])
def test_other_devices_are_refused(device):
    """Asked for one on the CPU it gave one on the current CUDA device."""
    import __graft_entry__
    __graft_entry__.build()
    import int4_quantized_flashattention_b200 as ra
    p = ra.Problem.make(1, 2, 64, (24, 20, 20), (2, 3, 4))
    with pytest.raises(ValueError):
        ra.rope_table(p, device=device)
