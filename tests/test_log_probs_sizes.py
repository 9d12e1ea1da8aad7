"""The workspace of the log probabilities' gradient does not depend on `top`."""
import pytest

import ring_all_reduce_ar_amd as ar


@pytest.mark.parametrize("top", [-1, 1, 64, 65, 1000])
def test_top_is_not_looked_at(top):
    for size in ((10, 1000, 64, "bf16"), (300, 50_000, 512, "f32"), (10, 1 << 25, 8, "f16")):
        want = ar.ar_linear_log_probs_workspace_bytes(*size, backward=True)
        assert ar.ar_linear_log_probs_workspace_bytes(*size, top=top, backward=True) == want > 0
