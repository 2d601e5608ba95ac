"""The workspace of paged_decode_shared_prefix_attention: sized once, by the largest sizes."""

import random

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


HEADS = [(24, 8, 128), (32, 8, 64), (8, 1, 64), (1, 1, 128), (32, 32, 128), (7, 1, 128), (20, 4, 64)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_smaller_calls_need_no_more(B, hq, hkv, d):
    size = B.paged_decode_shared_prefix_workspace_size
    rng = random.Random(hq * 1000 + hkv)

    def log(lo, hi):
        return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))

    for _ in range(1500):
        n, groups, prefix, suffix = log(1, 1500), log(1, 300), log(1, 200_000), log(1, 50_000)
        most = size(n, hq, hkv, d, groups, prefix, suffix)
        less = [rng.choice([x, log(1, x), max(1, x - 1)]) for x in (n, groups, prefix, suffix)]
        less[1] = rng.choice([less[1], 0])
        assert 0 < size(less[0], hq, hkv, d, *less[1:]) <= most, (n, groups, prefix, suffix, less)


def test_a_sequence_leaves(B):
    size = B.paged_decode_shared_prefix_workspace_size
    assert size(15, 24, 8, 128, 1, 8192, 1024) <= size(16, 24, 8, 128, 1, 8192, 1024)
    assert size(64, 24, 8, 128, 1, 512, 512) <= size(64, 24, 8, 128, 1, 1024, 1024)


def test_size_is_in_proportion(B):
    """No more than 1/8 of the keys that it lets be cut (their K and V bytes), and 32 MB."""
    size = B.paged_decode_shared_prefix_workspace_size
    for hq, hkv, d in HEADS:
        for n, prefix, suffix in ((16, 2048, 512), (64, 8192, 1024), (256, 1000, 131072), (1000, 100, 8192)):
            own = n * hkv * d * 4 * (prefix + suffix)
            assert size(n, hq, hkv, d, 4, prefix, suffix) <= own / 8 + (32 << 20)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_one_workspace_as_sequences_leave(B, mode):
    """A batch that shrinks to nothing, shared, plain and by size, in the workspace made for all."""
    g = torch.Generator(device="cuda").manual_seed(4)
    n, hq, hkv, d, bs, prefix, own = 16, 24, 8, 128, 16, 8192, 64
    sh = prefix // bs
    tables = torch.empty(n, sh + own // bs, dtype=torch.int32, device="cuda")
    tables[:, :sh] = torch.arange(sh, device="cuda")
    tables[:, sh:] = sh + torch.arange(n * own // bs, device="cuda").view(n, -1)
    nb = sh + n * own // bs
    k, v = (torch.randn(nb, hkv, bs, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([prefix + 1 + 4 * b for b in range(n)], dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.paged_decode_shared_prefix_workspace_size(n, hq, hkv, d, 1, prefix, 1024),
                     dtype=torch.uint8, device="cuda")
    before = B.pkv_set_shared_prefix(mode)
    try:
        for left in range(n, 0, -1):
            want = torch.empty_like(q[:left])
            B.paged_decode_attention(want, q[:left], k, v, tables[:left], lens[:left], prefix + own, 0.09)
            for max_suffix in (1024, own):
                out = torch.full_like(want, 9.0)
                B.paged_decode_shared_prefix_attention(
                    out, q[:left], k, v, tables[:left], lens[:left],
                    torch.tensor([0, left], dtype=torch.int32, device="cuda"),
                    torch.tensor([prefix], dtype=torch.int32, device="cuda"), prefix, max_suffix, 0.09,
                    workspace=ws)
                # Both outputs are rounded (2^-8 of each value at most), and the prefix's weights
                # are: v is independent of the roundings, so that sum p_t d_t v_t with |d_t| <= 2^-8
                # is as long as 2^-8 of sum p_t v_t, not of the sum of |p_t v_t|.
                err = (out.double() - want.double()).norm() / want.double().norm()
                assert err <= 3 * 2.0 ** -8, (left, max_suffix, err.item())
    finally:
        B.pkv_set_shared_prefix(before)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_never_is_the_plain_decode_past_the_table(B):
    """Bounds whose sum passes the tables: the call is cut to what they hold, where the plain
    decode takes 19 parts and not the 18 of the sum; it is the plain decode all the same."""
    n, d, bs, blocks = 24, 64, 8, 1161
    cap = blocks * bs  # 9288
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = (torch.randn(n * blocks, 1, bs, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, 1, d, generator=g, device="cuda").to(torch.bfloat16)
    tables = torch.randperm(n * blocks, generator=g, device="cuda").to(torch.int32).view(n, blocks)
    lens = torch.randint(1, cap + 1, (n,), generator=g, device="cuda").to(torch.int32)
    lens[0] = cap
    want, out = torch.empty_like(q), torch.empty_like(q)
    B.paged_decode_attention(want, q, k, v, tables, lens, cap, 0.125)
    ws = torch.zeros(B.paged_decode_shared_prefix_workspace_size(n, 1, 1, d, n, cap, 512),
                     dtype=torch.uint8, device="cuda")
    before = B.pkv_set_shared_prefix(B.SHARED_NEVER)
    try:
        B.paged_decode_shared_prefix_attention(
            out, q, k, v, tables, lens, torch.arange(n + 1, dtype=torch.int32, device="cuda"),
            torch.full((n,), cap, dtype=torch.int32, device="cuda"), cap, 512, 0.125, workspace=ws)
    finally:
        B.pkv_set_shared_prefix(before)
    assert torch.equal(out, want) and B.pkv_device_errors() == 0
