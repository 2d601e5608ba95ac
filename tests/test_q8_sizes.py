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


def test_few_queries_need_no_room_for_the_contexts(B):
    """The prefill's workspace by its call: drafts' goes by the sequences alone, a chunk's by its rows."""
    size = B.paged_prefill_q8_workspace_size_for
    drafts = size(256 * 5, 5, 256, 24, 8, 128, 32768)
    assert 0 < drafts < 32 << 20 and drafts == size(256, 1, 256, 24, 8, 128, 131072)
    assert size(4 * 2000, 2000, 4, 24, 8, 128, 6000) >= 4 * 6000 * 8 * 128 * 4
    for n, new, hq, hkv, d, longest in ((2, 4, 8, 2, 64, 100), (8, 5, 32, 8, 64, 2000), (4, 2048, 24, 8, 128, 8000),
                                        (3, 33, 5, 1, 64, 40), (64, 32, 8, 8, 64, 4000)):
        assert 0 < size(n * new, new, n, hq, hkv, d, longest) <= B.paged_prefill_q8_workspace_size(n, hkv, d, 16, longest)
    # over 2^31 rows of heads
    assert B.paged_prefill_q8_workspace_size(1024, 8, 64, 16, 1 << 18) == 0
    assert 0 < size(1024 * 2, 2, 1024, 8, 8, 64, 1 << 18) < 32 << 20
    # chunks: 8 GB of rows at a time, or one context's
    assert 7 << 30 < size(1024 * 40, 40, 1024, 8, 8, 64, 1 << 18) <= 8 << 30
    assert 8 << 30 <= size(2 * 40, 40, 2, 8, 8, 64, 1 << 22) < (8 << 30) + (1 << 20) and size(40, 40, 1, 8, 8, 64, 1 << 29) == 0
    for bad in ((0, 1, 1, 1, 1, 64, 9), (1, 0, 1, 1, 1, 64, 9), (1, 1, 0, 1, 1, 64, 9), (1, 1, 1, 0, 1, 64, 9), (1, 1, 1, 1, 0, 64, 9),
                (1, 1, 1, 1, 1, 96, 9), (1, 10, 1, 1, 1, 64, 9), (1, 1, 1, 9, 1, 64, 9), (1, 1, 1, 3, 2, 64, 9)):
        assert size(*bad) == 0


def test_a_chunk_is_refused_without_its_rows(B):
    """Workspaces one byte short, both ways; a context of over 2^31 rows where queries are not few."""
    fake = ctypes.c_void_p(1 << 20)  # (never dereferenced: each of these calls is refused)
    cache, desc = B.pkv_q8_cache(fake, fake, fake, fake, 0), B.pkv_cache_desc(64, 16, 2, 64)

    def call(new, n, most, size):
        return B.lib().paged_prefill_attention_q8(fake, fake, new * n, ctypes.byref(cache), fake, most // 16 + 1, fake, most, fake,
                                                  new, n, 8, ctypes.byref(desc), 0.1, fake, size, None)

    for new, n, most in ((4, 2, 100), (5, 256, 32768), (70, 1, 4000), (70, 1, 1 << 22)):
        assert call(new, n, most, B.paged_prefill_q8_workspace_size_for(new * n, new, n, 8, 2, 64, most) - 1) == -4
    assert call(70, 3, 4000, B.paged_prefill_q8_workspace_size_for(70, 70, 1, 8, 2, 64, 4000) - 1) == -4  # not one sequence's
    assert call(40, 3, 1 << 30, 1 << 40) == -3
