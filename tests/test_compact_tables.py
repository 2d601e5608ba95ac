"""paged_kv_compact's table rewrite where few pages move: large tables, odd sizes, and what it costs."""

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


def plan(layers, nb, hkv, bs, d, moves, rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(layers, nb, hkv, bs, d, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(layers, nb, hkv, bs, d, generator=g, device="cuda").to(torch.bfloat16)
    perm = torch.randperm(nb, generator=g, device="cuda")
    pairs = torch.stack((perm[:moves], perm[nb - moves:]), 1).to(torch.int32).contiguous()
    block_map = torch.arange(nb, device="cuda", dtype=torch.int32)
    block_map[pairs[:, 0].long()] = pairs[:, 1]
    tables = perm[torch.randint(0, nb - moves, (rows, cols), generator=g, device="cuda")].to(torch.int32)
    tables[torch.rand(rows, cols, generator=g, device="cuda") < 0.2] = -1
    return k, v, pairs, tables, block_map


# one page of one chunk; pages of several chunks; more page CTAs than table CTAs; tables past
# one pass of the grid (4096 CTAs of 256 entries); single entries
@pytest.mark.gpu
@pytest.mark.parametrize("layers,nb,hkv,bs,d,moves,rows,cols", [
    (1, 9, 1, 8, 64, 1, 256, 512), (3, 40, 8, 16, 128, 2, 333, 77), (2, 300, 2, 16, 64, 120, 3, 5),
    (1, 5, 1, 8, 8, 2, 1100, 1024), (70, 7, 1, 16, 64, 3, 64, 999), (1, 4, 1, 8, 64, 1, 1, 1)])
def test_few_moves_large_tables(B, layers, nb, hkv, bs, d, moves, rows, cols):
    k, v, pairs, tables, block_map = plan(layers, nb, hkv, bs, d, moves, rows, cols, 7)
    want_k, want_v = k.clone(), v.clone()
    src, dst = pairs[:, 0].long(), pairs[:, 1].long()
    want_k[:, dst], want_v[:, dst] = k[:, src], v[:, src]
    want = torch.where(tables >= 0, block_map[tables.clamp(min=0).long()], tables)
    for _ in range(2):  # the same plan again changes nothing more
        B.paged_kv_compact(k, v, pairs, tables, block_map)
        assert torch.equal(tables, want)
        assert torch.equal(k, want_k) and torch.equal(v, want_v)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_one_move_costs_no_serial_walk(B):
    """The tables' rewrite takes the CTAs that the tables need, however few pages move: as long
    with one move as with none (131072 entries behind a single CTA are 512 dependent rounds)."""
    k, v, pairs, tables, block_map = plan(1, 9, 1, 8, 64, 1, 256, 512, 3)

    def us(moves):
        times = []
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            for _ in range(4):
                B.paged_kv_compact(k, v, moves, tables, block_map)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 250)
        return min(times)

    assert us(pairs) < 3 * us(pairs[:0]) + 20
