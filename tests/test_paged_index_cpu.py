"""What the paged layer takes for rows, pages, offsets and lengths, and the sizes that the
paged decode refuses (on the host, before anything is launched)."""
import ctypes as C

import numpy as np
import pytest
import torch

from long_context_decoding_eta_b200 import _lib as L
from long_context_decoding_eta_b200.paged import _index_tensor

CPU = torch.device("cpu")


@pytest.mark.parametrize("x", [
    [True, False], [0, True], [1.0], [0.5], ["1"], [None], np.array([True, False]), np.array([1.0]),
    [torch.tensor(True)], [torch.tensor(1.0)], torch.tensor([True, False]), torch.tensor([1.0]),
    torch.tensor([1.0], dtype=torch.bfloat16), torch.tensor([1j]), [1 << 31], [-(1 << 31) - 1]])
def test_refused(x):
    with pytest.raises(ValueError):
        _index_tensor(x, CPU)


@pytest.mark.parametrize("x", [
    [3, 0, -1], (3, 0, -1), np.array([3, 0, -1]), [np.int64(3), torch.tensor(0), -1],
    range(3, -4, -3), *(torch.tensor([3, 0, -1], dtype=t)
                        for t in (torch.int32, torch.int64, torch.int16, torch.int8)),
    torch.tensor([[3, 9], [0, 9], [-1, 9]], dtype=torch.int32)[:, 0]])
def test_taken(x):
    t = _index_tensor(x, CPU)
    want = list(x) if isinstance(x, range) else [3, 0, -1]
    assert t.dtype is torch.int32 and t.is_contiguous() and t.tolist() == want


def test_empty_and_passed_through():
    assert _index_tensor([], CPU).tolist() == []
    t = torch.arange(4, dtype=torch.int32)
    assert _index_tensor(t, CPU) is t


def test_wide_numbers_do_not_wrap():
    x = torch.tensor([1 << 32, (1 << 32) + 1, -(1 << 32), 7])
    assert _index_tensor(x, CPU).tolist() == [2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31, 7]


@pytest.mark.parametrize("B,code", [(8192, 2), (4096, 2), (4095, 3)])
def test_paged_decode_refuses_more_blocks_than_32_bits_count(B, code):
    """Rows that share pages can have 2^30 and more blocks in all; just below, the call
    goes on to its next check (a missing workspace)."""
    dims, fake = L.Dims.of(B, 8, 4, 64, 64, 65536 * 64), C.c_void_p(4096)
    assert L.lib().eta_paged_decode(C.byref(dims), 13, fake, None, fake, fake, fake, fake, None,
                                    None, 0.0, 0.0, 0, None, None, 0, fake, fake, None, 0, None,
                                    None) == code
