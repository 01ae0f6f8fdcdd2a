"""The binding's C++ module beside its Python forms: the same keys apart, the same structs, and its refusals."""
import struct

import pytest
import torch

import chunked_recurrence_gb300 as crg
from chunked_recurrence_gb300 import paged

native = pytest.mark.skipif(paged._marshal is None, reason="gdn_marshal is not built")


def test_lays_tell_layouts_apart():
    x = torch.zeros(4, 6, 8)
    others = [x[:, :5], x[:, ::2], x.transpose(0, 1), x.double(), x.to("meta"), x[0], None]
    keys = [paged._lays(t) for t in [x, *others]]
    assert len(set(keys)) == len(keys)
    assert paged._lays(x) == paged._lays(torch.ones(4, 6, 8))  # values and addresses are no part of it
    assert paged._lays(x, None) != paged._lays(None, x)
    assert paged._lays(x, x) != paged._lays(x)


def test_like():
    x = torch.zeros(4, 6, 8, dtype=torch.bfloat16, requires_grad=True)[:, ::2]
    y, z = paged._like(x, 3, False), paged._like(x, 2, True)
    assert y.shape == x.shape and y.dtype == x.dtype and y.is_contiguous() and not y.requires_grad
    assert z.shape == x.shape[:2] and z.dtype == torch.float32


def test_pack():
    x, tail = torch.zeros(3), b"\x01\x02\x03\x04"
    at = paged._pack(b"", x, None)
    assert at == struct.pack("2P", x.data_ptr(), 0)
    assert paged._pack(tail, x) == struct.pack("P", x.data_ptr()) + tail
    assert len(paged._pack(tail, at)) == struct.calcsize("P") + 4


@native
def test_refusals():
    x = torch.zeros(2, 2)
    for bad in (lambda: paged._lays(3), lambda: paged._like(3, 1, False), lambda: paged._pack(3, x),
                lambda: paged._pack(b"", "x")):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: paged._like(x, 3, False), lambda: paged._like(x, -1, False), lambda: paged._lays(*[x] * 257),
                lambda: paged._lays(torch.zeros([1] * 9))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        paged._entry("gdn_rope")(None)


@native
def test_entry_converts_like_the_library():
    # no tensors: refused by the library with the same status either way
    assert paged._entry("gdn_pages_copy")(None, None, 1, 4, None, None, 0, 0) == \
        crg.load().gdn_pages_copy(None, None, 1, 4, None, None, 0, 0) != 0
    with pytest.raises(OverflowError):
        paged._entry("gdn_pages_copy")(None, None, 1 << 40, 4, None, None, 0, 0)


def test_the_module_is_this_interpreters():
    """Its name carries the interpreter's tag, so that another Python does not load it."""
    import sysconfig
    from chunked_recurrence_gb300 import build
    assert build.MARSHAL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and "cpython" in build.MARSHAL
    assert paged._marshal is None or paged._marshal.__file__ == build.MARSHAL


def test_a_module_that_was_built_loads():
    import os
    from chunked_recurrence_gb300 import build
    if not os.path.exists(build.MARSHAL):
        pytest.skip("gdn_marshal is not built")
    assert paged._marshal is not None
