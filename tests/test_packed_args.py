"""The packed argument structs of the binding have the layout of their ctypes
mirrors (which name the fields of include/salad.h)."""
import ctypes

import pytest

import sparse_linear_hybrid_top_b200 as salad


def _flatten(x):
    if isinstance(x, ctypes.Structure):
        for name, _ in x._fields_:
            yield from _flatten(getattr(x, name))
    elif isinstance(x, ctypes.Array):
        yield from x
    else:
        yield x


@pytest.mark.parametrize("fmt,mirror", [(salad._PACK_ROPE, salad.RopeArgs), (salad._PACK_APPEND, salad.CacheAppendArgs),
                                        (salad._PACK_ATTN, salad.CacheAttnArgs)])
def test_packed_layout(fmt, mirror):
    n = len(list(_flatten(mirror())))
    values = list(range(1, n + 1))
    packed = fmt.pack(*values)
    assert len(packed) == ctypes.sizeof(mirror)
    assert [int(v) for v in _flatten(mirror.from_buffer_copy(packed))] == values


def test_numbers_that_do_not_fit_are_refused():
    with pytest.raises(ValueError):
        salad._pack(salad._PACK_ROPE, "salad_rope", *[1 << 40] * len(list(_flatten(salad.RopeArgs()))))
