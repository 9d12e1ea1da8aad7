"""Rows that lie on one another, as an expanded tensor's, are refused: read as
dense ones they would pass its end."""
import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_lm_host import host_comm


@pytest.mark.parametrize("x", [torch.zeros(1, 16).expand(8, 16), torch.zeros(1, 1).expand(8, 16), torch.zeros(16).expand(8, 16)])
def test_lists_of_matrices(x):
    dense = [torch.zeros(8, 16) for _ in range(3)]
    with pytest.raises(ValueError):
        ar._matrices([x, x], 0)
    with pytest.raises(ValueError):
        ar._matrices([dense[0], x], 0)
    with pytest.raises(ValueError):
        ar.ar_orthogonalize(host_comm(), [x], dense[:1], 8, 16, "f32", stream=0)
    with pytest.raises(ValueError):
        ar.ar_muon_update(host_comm(), [x], dense[:1], dense[:1], dense[1:2], dense[1:2], 8, 16, "f32", stream=0)


def test_one_row_has_no_pitch():
    x = torch.zeros(16).expand(1, 16)
    assert list(ar._matrices([x, x], 0)[0]) == [x.data_ptr()] * 2
