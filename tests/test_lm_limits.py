"""The binding and the refusals of the language-model operators without a GPU, at
the arguments where they are easily taken for others."""
import pytest
import torch

import ring_all_reduce_ar_amd as ar


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.uint8, torch.bool])
def test_a_tensor_of_one_integer_is_a_buffer(dtype):
    """Its address counts, wherever it stands among addresses."""
    x = torch.ones(1, dtype=dtype)
    assert list(ar._ptrs([16, x])) == [16, x.data_ptr()]
    assert list(ar._ptrs([16, 32, x, 64])) == [16, 32, x.data_ptr(), 64]
    assert list(ar._ptrs((x, 16))) == [x.data_ptr(), 16]


def test_addresses_beyond_64_bits_and_below_zero():
    """As ctypes takes them one by one."""
    for bad in ([16, 1 << 64], [16, -1]):
        assert list(ar._ptrs(bad)) == [16, bad[1] & ((1 << 64) - 1) or None]


def test_numbers_that_are_no_addresses():
    class Five:
        def __index__(self):
            return 5

    for bad in ([16, Five()], [16, 2.0], [16, "32"], [16, None]):
        with pytest.raises(TypeError):
            ar._ptrs(bad)
