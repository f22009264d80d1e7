"""What the binding of the calls for blocks, shared prefixes and pages took and should not have (no GPU needed)."""
import pytest
import torch

import sparse_attention_row_gb300 as sar


@pytest.fixture
def dec():
    """A decoder whose device is that of CPU tensors, without a library call."""
    d = object.__new__(sar.PagedDecoder)
    d.device, d._dev = -1, "cpu"
    return d


@pytest.mark.parametrize("make", [lambda: torch.zeros(64).unfold(0, 8, 4), lambda: torch.zeros(8, 16).unfold(0, 3, 2), lambda: torch.zeros(64).as_strided((4, 3, 4), (4, 16, 2)),
                                  lambda: torch.zeros(64).as_strided((5, 4), (1, 2))])
def test_caches_whose_pages_overlap_are_refused(dec, make):
    with pytest.raises(ValueError, match="do not overlap"):
        dec.page_caches([make()])


@pytest.mark.parametrize("make", [lambda: torch.zeros(16, 4, 8).transpose(0, 1), lambda: torch.zeros(64).as_strided((4, 8), (1, 4)), lambda: torch.zeros(64).unfold(0, 8, 8),
                                  lambda: torch.zeros(3, 16, 8)[:, :, 2:6].permute(1, 0, 2)])
def test_caches_whose_pages_lie_among_one_another_are_not(dec, make):
    t = make()
    c = sar.TopkPageCache.from_buffer_copy(dec._page_cache(t))
    assert (c.num_blocks, c.block_stride) == (t.shape[0], t.stride(0) * 4)


def test_caches_of_another_device_are_refused(dec):
    kept = dec.page_caches([torch.zeros(4, 8)])
    other = object.__new__(sar.PagedDecoder)
    other.device, other._dev = 1, torch.device("cuda", 1)
    with pytest.raises(ValueError, match="device -1"):
        other.copy_pages(kept, sar.PageCopies(torch.zeros(1).int(), torch.zeros(1).int()))
