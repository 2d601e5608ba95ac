"""The 8-bit cache's entry points without layers, sequences or a cache that could be: errors, on the host."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


@pytest.mark.parametrize("field,code", [("num_blocks", -2), ("block_size", -2), ("num_kv_heads", -2), ("head_dim", -2)])
def test_copies_of_no_layers_look_at_the_descriptor(B, field, code):
    """Tables alone may be remapped; the sizes that bound their entries count all the same."""
    fine = dict(num_blocks=64, block_size=16, num_kv_heads=2, head_dim=64)

    def calls(d):
        yield B.lib().paged_kv_compact_q8(None, 0, None, None, 0, None, 0, 0, None, ctypes.byref(d), None)
        yield B.lib().paged_kv_copy_blocks_q8(None, 0, None, None, 0, ctypes.byref(d), None)

    assert list(calls(B.pkv_cache_desc(**fine))) == [0, 0]
    for value in (0, -1):
        assert list(calls(B.pkv_cache_desc(**dict(fine, **{field: value})))) == [code, code], value
    assert list(calls(B.pkv_cache_desc(**dict(fine, head_dim=96)))) == [-3, -3]
    assert list(calls(B.pkv_cache_desc(0, 0, 0, 0))) == [-2, -2]
