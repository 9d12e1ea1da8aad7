"""The cross entropy of fp32 operands in bf16 pieces: more than 64 tokens, and
more than 512 tiles of 64 tokens by 64 rows of the vocabulary (below that fp32
matrix instructions take the call)."""
import pytest
import torch

from test_gpu_lm import check_loss, comms  # noqa: F401

pytestmark = pytest.mark.gpu


def in_pieces(n, vocab):
    return n > 64 and -(-n // 64) * -(-vocab // 64) > 512


@pytest.mark.parametrize("n,vocab,width", [
    (700, 6001, 131),    # rows on 4 bytes; scalar stores of the gradients
    (130, 12_001, 770),  # rows on 8 bytes
    (129, 16_385, 33),   # one token, one row and one column over a tile
    (257, 7169, 129),
    (128, 16_640, 256),  # whole tiles
    (65, 16_500, 1),
    (1000, 2050, 513),
])
def test_widths(comms, n, vocab, width):  # noqa: F811
    assert in_pieces(n, vocab)
    check_loss(comms, n, vocab, width, "f32", 80)


@pytest.mark.parametrize("pitch,offset", [(5, 1), (2, 2), (4, 0), (3, 0), (64, 4), (1, 3)])
@pytest.mark.parametrize("width", [128, 77])
def test_strided_rows(comms, pitch, offset, width):  # noqa: F811
    """Rows on 4, 8 and 16 bytes, with NaN between them."""
    assert in_pieces(130, 12_000)
    check_loss(comms, 130, 12_000, width, "f32", 81, pitch=pitch, offset=offset, index="i32")


@pytest.mark.parametrize("n,vocab,width", [
    (4200, 600, 72), (2500, 1500, 130),  # parts of the tokens; the model's columns as rows of the second operand
    (4200, 600, 200),                    # as rows of the first
    (65, 33_001, 40), (70, 70_000, 36),  # parts of the vocabulary
    (200, 9000, 250),
])
def test_split_sums(comms, n, vocab, width):  # noqa: F811
    assert in_pieces(n, vocab)
    check_loss(comms, n, vocab, width, "f32", 82)


@pytest.mark.parametrize("n,vocab,width", [(1021, 8003, 770), (5000, 30_007, 100)])
def test_several_pieces_of_the_vocabulary(comms, n, vocab, width):  # noqa: F811
    """More than one GiB of buffers in the second, odd sizes in both."""
    assert in_pieces(n, vocab)
    check_loss(comms, n, vocab, width, "f32", 83, pitch=5, offset=1)


@pytest.mark.parametrize("ignored", [0.0, 0.9, 1.0])
def test_ignored_tokens(comms, ignored):  # noqa: F811
    assert in_pieces(150, 12_000)
    check_loss(comms, 150, 12_000, 61, "f32", 84, ignored=ignored)
