"""paged_decode_shared_prefix_attention at the ends of what it takes."""

import ctypes

import pytest

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced by the host checks


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


@pytest.mark.parametrize("prefix,suffix", [(2**29 + 1, 16), (2**31 - 1, 16), (16, 2**29 + 1),
                                           (2**31 - 1, 2**31 - 1)])
def test_lengths_past_the_cuts_are_refused(B, prefix, suffix):
    """A prefix is cut into at most 2^29 keys a row: over 2^29 tokens, more rows were counted than
    the workspace held."""
    rc = B.lib().paged_decode_shared_prefix_attention(
        FAKE, FAKE, FAKE, FAKE, FAKE, 2**25, FAKE, FAKE, FAKE, 1, prefix, suffix, 2, 8,
        ctypes.byref(B.pkv_cache_desc(64, 256, 2, 64)), 0.125, FAKE, 2**62, None)
    assert rc == -3 and "2^29" in B.pkv_last_error()
    assert B.paged_decode_shared_prefix_workspace_size(2, 8, 2, 64, 1, prefix, suffix) == 0


@pytest.mark.parametrize("seqs,hkv", [(1, 1), (400, 1), (3, 8)])
def test_longest_lengths_have_room_for_their_rows(B, seqs, hkv):
    # at least one row for the prefix and one for the own keys of each query head
    n = B.paged_decode_shared_prefix_workspace_size(seqs, hkv, hkv, 64, 1, 2**29, 2**29)
    assert n >= 2 * seqs * hkv * 65 * 4
