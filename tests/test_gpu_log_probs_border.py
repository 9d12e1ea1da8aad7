"""Alternatives on both sides of the number of tokens from which one wave finds
those of a token rather than eight."""
import pytest

from test_gpu_lm import comms  # noqa: F401
from test_gpu_log_probs import check_top

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [255, 256, 257, 400, 512, 513])
@pytest.mark.parametrize("vocab,width,top,dtype", [(999, 64, 5, "bf16"), (4099, 72, 20, "f16"), (9000, 64, 64, "bf16"),
                                                   (700, 33, 9, "f32")])
def test_alternatives(comms, n, vocab, width, top, dtype):  # noqa: F811
    check_top(comms, n, vocab, width, dtype, top)
