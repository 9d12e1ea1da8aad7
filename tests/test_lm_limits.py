"""The binding and the refusals of the language-model operators without a GPU, at
the arguments where they are easily taken for others."""
import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_lm_host import BAD, at, host_comm, refused


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


# ---------------------------------------------------------------------------
# overlaps
# ---------------------------------------------------------------------------
WS = 1 << 44  # host_comm's workspace


def passes(fn, *args, **kw):
    """Past every check of its arguments: the call gets as far as HIP."""
    with pytest.raises(ar.ArError) as e:
        fn(*args, **kw, stream=0)
    assert e.value.code == ar.AR_ERR_HIP, str(e.value)


@pytest.mark.parametrize("layout", ["replicated", "sharded", "reduce"])
def test_the_norm_overlaps_nothing(layout):
    def call(check, norm_out, send=(at(0), at(1)), recv=(at(2), at(3))):
        fn, kw = (ar.ar_all_reduce_clip, {}) if layout == "reduce" else (ar.ar_clip_grads, {"layout": layout})
        check(fn, host_comm(2), list(send), list(recv), [8], 1.0, norm_out, "f32", **kw)

    def refuse(fn, *args, **kw):
        refused(BAD, fn, *args, **kw)

    for inside in (at(0), at(0) + 28, at(2), at(3) + 28, WS, WS + ar.ar_clip_workspace_bytes() - 4):
        call(refuse, inside)
    if not torch.cuda.is_available():  # made-up addresses are not for a GPU
        for beside in (at(0) - 4, at(0) + 32, at(3) + 32, WS - 4, WS + ar.ar_clip_workspace_bytes(), None):
            call(passes, beside)
        if layout == "replicated":  # not read
            call(passes, at(1))
        else:
            call(refuse, at(1))


@pytest.mark.parametrize("layout", ["replicated", "sharded"])
def test_a_norm_alone_overlaps_nothing(layout):
    def call(check, grads, norm_out):
        check(ar.ar_grad_norm, host_comm(2), grads, [8], norm_out, "f32", layout=layout)

    def refuse(fn, *args, **kw):
        refused(BAD, fn, *args, **kw)

    call(refuse, [WS, at(1)], at(4))
    call(refuse, [WS + ar.ar_clip_workspace_bytes() - 4, at(1)], at(4))
    call(refuse, [at(0), at(1)], at(0) + 4)
    call(refuse, [at(0), at(1)], WS + 8)
    if layout == "sharded":
        call(refuse, [at(0), WS], at(4))
        call(refuse, [at(0), at(1)], at(1))
    if not torch.cuda.is_available():
        call(passes, [at(0), at(1)], at(0) + 32)
        call(passes, [at(0), at(0) + 16], at(4))  # what is only read may be read twice
        call(passes, [at(0), at(0)], at(4))
        call(passes, [WS - 32, WS + ar.ar_clip_workspace_bytes()], at(4))
        if layout == "replicated":  # rank 1's are not read
            call(passes, [at(0), WS], at(4))
            call(passes, [at(0), at(1)], at(1))
