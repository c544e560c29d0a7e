"""What one test leaves in torch's allocator is no part of the next."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BIG = 1 << 32


def test_that_leaves_a_large_segment():
    torch.empty(BIG, dtype=torch.uint8, device="cuda")
    assert torch.cuda.memory_reserved() >= BIG


def test_next_one_has_no_part_of_it():
    """A tensor of a few MB (one of over 1 MB is cut out of what is cached) lives in a small segment,
    and a limit at what is reserved leaves no room for a larger one."""
    held = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.empty_cache()
    reserved, total = torch.cuda.memory_reserved(), torch.cuda.get_device_properties(0).total_memory
    assert reserved < BIG
    try:
        torch.cuda.set_per_process_memory_fraction(reserved / total)
        with pytest.raises(torch.OutOfMemoryError):
            torch.empty(BIG // 2, dtype=torch.uint8, device="cuda")
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert held.numel() == 4 << 20
