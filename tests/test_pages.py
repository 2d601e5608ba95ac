"""Page copies, forks with copy-on-write, truncation and compaction.

The host side (pkv_bm_*) runs on the CPU against a plain model; the device side
(paged_kv_copy_blocks, paged_kv_compact) moves bytes, so every comparison is bit-exact.
"""

import ctypes
import random

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced by the host checks


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


# ------------------------------------------------------------------ host side

class Tokens:
    """What every slot of the pool should hold: a fork copies, a write overwrites."""

    def __init__(self, bm):
        self.bm, self.pool, self.seqs = bm, {}, {}

    def apply_copies(self, pairs, rows):
        bs = self.bm.block_size
        for (a, b), n in zip(pairs.tolist(), rows.tolist()):
            for t in range(n):
                self.pool[b * bs + t] = self.pool[a * bs + t]

    def check(self):
        ids = sorted(self.seqs)
        bs = self.bm.block_size
        maxb = max([1] + [-(-len(self.seqs[s]) // bs) for s in ids])
        tables, lens = self.bm.block_tables(ids, maxb)
        held = {}
        for i, s in enumerate(ids):
            want = self.seqs[s]
            assert int(lens[i]) == len(want)
            row = tables[i].tolist()
            n = -(-len(want) // bs)
            assert all(x == -1 for x in row[n:])
            for blk in row[:n]:
                held[blk] = held.get(blk, 0) + 1
            got = [self.pool[row[t // bs] * bs + t % bs] for t in range(len(want))]
            assert got == want, f"sequence {s} reads another's tokens"
        for blk in range(self.bm.num_blocks):
            assert self.bm.ref_count(blk) == held.get(blk, 0)
        assert self.bm.num_free_blocks == self.bm.num_blocks - len(held)


@pytest.mark.parametrize("seed", range(8))
def test_forks_copy_on_write_truncate_and_compact(B, seed):
    """Random admissions, forks, appends, truncations, frees and compactions: every
    sequence reads back exactly the tokens it was given, whoever shares its blocks."""
    rng = random.Random(seed)
    nb, bs = rng.choice([(12, 4), (30, 2), (9, 8), (24, 1)])
    bm = B.BlockManager(nb, bs)
    t = Tokens(bm)
    stamp = 0
    for step in range(250):
        op, ids = rng.random(), sorted(t.seqs)
        try:
            if op < 0.15 or not ids:
                n = rng.randint(0, 2 * bs)
                bm.add_sequence(1000 + step, n)
                tables, _ = bm.block_tables([1000 + step], max(1, n))
                t.seqs[1000 + step] = []
                for p in range(n):
                    stamp += 1
                    t.pool[int(tables[0, p // bs]) * bs + p % bs] = stamp
                    t.seqs[1000 + step].append(stamp)
            elif op < 0.35:
                s = rng.choice(ids)
                bm.fork(s, 1000 + step)
                t.seqs[1000 + step] = list(t.seqs[s])
            elif op < 0.75:
                who = [rng.choice(ids) for _ in range(rng.randint(1, 4))]
                slots, pairs, rows = bm.append_slots_cow(who)
                assert len(set(pairs[:, 1].tolist())) == len(pairs)
                assert not set(pairs[:, 0].tolist()) & set(pairs[:, 1].tolist())
                t.apply_copies(pairs, rows)
                for s, slot in zip(who, slots.tolist()):
                    stamp += 1
                    t.pool[slot] = stamp
                    t.seqs[s].append(stamp)
            elif op < 0.83:
                s = rng.choice(ids)
                n = rng.randint(0, len(t.seqs[s]))
                bm.truncate(s, n)
                del t.seqs[s][n:]
            elif op < 0.93:
                s = rng.choice(ids)
                bm.free_sequence(s)
                del t.seqs[s]
            elif op < 0.97:
                moves, block_map = bm.compact()
                used = bm.num_blocks - bm.num_free_blocks
                src, dst = moves[:, 0].tolist(), moves[:, 1].tolist()
                assert all(x >= used for x in src) and all(x < used for x in dst)
                want = list(range(nb))
                for a, b in zip(src, dst):
                    want[a] = b
                    for o in range(bs):
                        if a * bs + o in t.pool:
                            t.pool[b * bs + o] = t.pool[a * bs + o]
                assert block_map.tolist() == want
            else:
                s = bm.preempt_lifo()
                assert s == max(t.seqs)  # ids grow with admission
                del t.seqs[s]
        except B.PkvError as e:
            assert e.code == -8  # the pool was full: nothing changed
        t.check()


def test_block_manager_refusals(B):
    bm = B.BlockManager(4, 4)
    bm.add_sequence(1, 6)
    bm.fork(1, 2)
    with pytest.raises(B.PkvError, match="append_slots_cow") as e:
        bm.append_slots([2])  # would write into the block it shares with 1
    assert e.value.code == -3
    assert bm.ref_count(0) == 2 and bm.num_free_blocks == 2
    for call, code in ((lambda: bm.fork(7, 8), -2), (lambda: bm.fork(1, 2), -2),
                       (lambda: bm.truncate(1, 7), -2), (lambda: bm.truncate(1, -1), -2),
                       (lambda: bm.truncate(9, 0), -2), (lambda: bm.ref_count(4), -2),
                       (lambda: bm.ref_count(-1), -2), (lambda: bm.append_slots_cow([5]), -2)):
        with pytest.raises(B.PkvError) as e:
            call()
        assert e.value.code == code
    # all or nothing: three copies wanted (1, 2 and 3 share; the last one keeps it), 2 free
    bm.fork(1, 3)
    bm.fork(1, 4)
    with pytest.raises(B.PkvError) as e:
        bm.append_slots_cow([1, 2, 3, 4])
    assert e.value.code == -8 and bm.num_free_blocks == 2 and bm.ref_count(1) == 4
    slots, pairs, rows = bm.append_slots_cow([1, 2])
    assert rows.tolist() == [2, 2] and pairs[:, 0].tolist() == [1, 1] and bm.ref_count(1) == 2
    # a plan that does not fit its array changes nothing and says what it needs
    bm = B.BlockManager(4, 1)
    bm.add_sequence(1, 2)
    bm.add_sequence(2, 2)
    bm.free_sequence(1)
    n = ctypes.c_int64(0)
    m = (ctypes.c_int32 * 4)()
    assert B.lib().pkv_bm_compact(bm._h, None, 0, ctypes.byref(n), m) == -8 and n.value == 2
    assert bm.block_tables([2], 2)[0].tolist() == [[2, 3]]
    moves, _ = bm.compact()
    assert sorted(moves[:, 0].tolist()) == [2, 3] and bm.block_tables([2], 2)[0].tolist() == [[0, 1]]


def test_page_argument_errors(B):
    lib = B.lib()
    arr = (ctypes.c_void_p * 2)(1 << 20, 1 << 21)
    odd = (ctypes.c_void_p * 2)(1 << 20, (1 << 20) + 8)
    hole = (ctypes.c_void_p * 2)(1 << 20, None)

    def copy(k=arr, v=arr, n=2, pairs=FAKE, rows=None, m=3, d=(64, 16, 2, 64)):
        return lib.paged_kv_copy_blocks(k, v, n, pairs, rows, m, ctypes.byref(B.pkv_cache_desc(*d)), None)

    assert copy(k=None) == -1 and copy(v=hole) == -1 and copy(pairs=None) == -1
    assert copy(v=odd) == -5 and copy(pairs=ctypes.c_void_p((1 << 20) + 4)) == -5
    assert copy(rows=ctypes.c_void_p((1 << 20) + 2)) == -5
    assert copy(n=-1) == -2 and copy(m=-1) == -2 and copy(d=(0, 16, 2, 64)) == -2
    assert copy(d=(64, 16, 2, 60)) == -3 and "head_dim" in B.pkv_last_error()
    assert copy(d=(1 << 31, 16, 2, 64)) == -3
    assert copy(d=(64, 1 << 20, 1 << 20, 64)) == -3
    assert copy(m=1 << 40) == -3
    assert copy(m=0, pairs=None) == 0 and copy(n=0, k=None, v=None) == 0  # nothing to do
    assert lib.paged_kv_copy_blocks(arr, arr, 2, FAKE, None, 3, None, None) == -1

    def compact(moves=FAKE, m=3, tables=FAKE, seqs=2, cols=4, bmap=FAKE):
        return lib.paged_kv_compact(arr, arr, 2, moves, m, tables, seqs, cols, bmap,
                                    ctypes.byref(B.pkv_cache_desc(64, 16, 2, 64)), None)

    assert compact(tables=None) == -1 and compact(bmap=None) == -1 and compact(moves=None) == -1
    assert compact(seqs=-1) == -2 and compact(cols=-1) == -2 and compact(seqs=1 << 32) == -3
    assert compact(tables=ctypes.c_void_p((1 << 20) + 2)) == -5
    assert compact(m=0, moves=None, seqs=0, tables=None, bmap=None) == 0


def test_binding_refuses_tensors_of_another_device(B, monkeypatch):
    class Fake:  # what the check looks at
        def __init__(self, index):
            self.device = torch.device("cuda", index)

        def get_device(self):
            return self.device.index

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    B._one_device(Fake(0), a=Fake(0), b=None)
    with pytest.raises(ValueError, match="current device"):
        B._one_device(Fake(1))
    with pytest.raises(ValueError, match="expected cuda:0"):
        B._one_device(Fake(0), a=Fake(1))


# ------------------------------------------------------------------ device side

def bits(t):
    return t.view(torch.int16)


def pool(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-32768, 32768, shape, generator=g, device="cuda", dtype=torch.int32)
    return x.to(torch.int16).view(torch.bfloat16)  # every bit pattern, NaN among them


def reference(x, pairs, rows):
    """x [L, NB, Hkv, BS, D] after the copies, all reads before all writes."""
    old, new = bits(x).clone(), bits(x).clone()
    for (a, b), n in zip(pairs.tolist(), rows):
        new[:, b, :, :n] = old[:, a, :, :n]
    return new


@pytest.mark.gpu
@pytest.mark.parametrize("layers,nb,hkv,bs,d,n,partial", [
    (1, 2, 1, 1, 8, 1, False),        # the smallest page: one vector
    (1, 40, 3, 5, 24, 17, True),      # nothing a power of two
    (2, 64, 8, 16, 64, 20, True),
    (3, 50, 8, 16, 128, 25, False),
    (1, 30, 2, 256, 128, 11, True),
    (130, 12, 2, 8, 80, 5, True),     # three launches
    (1, 9, 7, 33, 40, 4, False),      # a page that ends inside a CTA's chunk
])
def test_copy_blocks(B, layers, nb, hkv, bs, d, n, partial):
    k, v = pool((layers, nb, hkv, bs, d), 1), pool((layers, nb, hkv, bs, d), 2)
    rng = random.Random(n)
    ids = rng.sample(range(nb), nb)
    dst, rest = ids[:n], ids[n:]
    src = [rng.choice(rest) for _ in range(n)]  # the same source more than once
    rows = [rng.randint(0, bs) for _ in range(n)] if partial else [bs] * n
    pairs = torch.tensor(list(zip(src, dst)), dtype=torch.int32)
    want_k, want_v = reference(k, pairs, rows), reference(v, pairs, rows)
    B.pkv_device_errors()
    B.paged_kv_copy_blocks(k, v, pairs.cuda(),
                           torch.tensor(rows, dtype=torch.int32).cuda() if partial else None)
    assert torch.equal(bits(k), want_k) and torch.equal(bits(v), want_v)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_copy_blocks_list_of_layers_and_one_layer(B):
    ks, vs = [pool((20, 2, 16, 64), i) for i in range(3)], [pool((20, 2, 16, 64), 9 + i) for i in range(3)]
    pairs = torch.tensor([[3, 4], [3, 19], [0, 7]], dtype=torch.int32)
    want = [reference(x[None], pairs, [16] * 3)[0] for x in ks + vs]
    B.paged_kv_copy_blocks(ks, vs, pairs.cuda())
    assert all(torch.equal(bits(x), w) for x, w in zip(ks + vs, want))
    x, y = pool((20, 2, 16, 64), 30), pool((20, 2, 16, 64), 31)
    want = [reference(t[None], pairs, [16] * 3)[0] for t in (x, y)]
    B.paged_kv_copy_blocks(x, y, pairs.cuda())
    assert torch.equal(bits(x), want[0]) and torch.equal(bits(y), want[1])


@pytest.mark.gpu
def test_nothing_to_do(B):
    k = torch.randn(8, 2, 16, 64, device="cuda").to(torch.bfloat16)
    was, none = k.clone(), torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    B.paged_kv_copy_blocks(k, k, none)
    B.paged_kv_copy_blocks(k, k, none, none[:, 0].contiguous())
    B.paged_kv_compact(k, k, none)
    B.paged_kv_compact(k, k, none, torch.zeros(0, 4, dtype=torch.int32, device="cuda"),
                       torch.arange(8, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(k, was) and B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_copy_blocks_skips_bad_pairs_and_clamps_rows(B):
    """Blocks outside the pool are skipped and flagged, bad row counts clamped and flagged,
    and src == dst does nothing; the good pairs of the same call are copied."""
    k, v = pool((2, 10, 2, 8, 64), 5), pool((2, 10, 2, 8, 64), 6)
    B.pkv_device_errors()
    pairs = torch.tensor([[0, 5], [1, 10], [-1, 6], [2, -3], [10, 7], [3, 3], [4, 8]], dtype=torch.int32)
    good = torch.tensor([[0, 5], [4, 8]], dtype=torch.int32)
    wk, wv = reference(k, good, [8, 8]), reference(v, good, [8, 8])
    B.paged_kv_copy_blocks(k, v, pairs.cuda())
    assert torch.equal(bits(k), wk) and torch.equal(bits(v), wv)
    assert B.pkv_device_errors() == 1
    pairs = torch.tensor([[0, 5], [1, 6], [2, 7]], dtype=torch.int32)
    wk, wv = reference(k, pairs, [0, 8, 3]), reference(v, pairs, [0, 8, 3])
    B.paged_kv_copy_blocks(k, v, pairs.cuda(), torch.tensor([-2, 9, 3], dtype=torch.int32).cuda())
    assert torch.equal(bits(k), wk) and torch.equal(bits(v), wv)
    assert B.pkv_device_errors() == 4


@pytest.mark.gpu
def test_copy_blocks_past_4_gb(B):
    """Offsets past 32 bits: the last pages of a pool of 4.6 GB."""
    k = torch.zeros(1, 70000, 8, 32, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[:, 69998], v[:, 69998] = pool((8, 32, 128), 1), pool((8, 32, 128), 2)
    B.paged_kv_copy_blocks(k, v, torch.tensor([[69998, 69999], [69998, 1]], dtype=torch.int32).cuda())
    for x in (k, v):
        assert torch.equal(bits(x[0, 69999]), bits(x[0, 69998])) and torch.equal(bits(x[0, 1]), bits(x[0, 69998]))
        assert int((x[0, 2:69998] != 0).sum()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("layers,nb,hkv,bs,d,seqs,cols", [
    (1, 64, 2, 16, 64, 5, 9), (3, 200, 1, 8, 80, 64, 33), (70, 20, 2, 4, 8, 1, 1)])
def test_compact_moves_pages_and_tables(B, layers, nb, hkv, bs, d, seqs, cols):
    """A plan of the block manager applied on the device, twice (the second changes nothing)."""
    rng = random.Random(nb)
    bm = B.BlockManager(nb, bs)
    ids = list(range(min(seqs * 3, nb)))
    for s in ids:
        bm.add_sequence(s, rng.randint(0, bs * max(1, nb // len(ids))))
    for s in rng.sample(ids, len(ids) // 2):
        bm.free_sequence(s)
        ids.remove(s)
    ids = ids[:seqs]
    tables, lens = bm.block_tables(ids, max(cols, nb))
    moves, block_map = bm.compact()
    assert len(moves) > 0
    after, _ = bm.block_tables(ids, max(cols, nb))
    k, v = pool((layers, nb, hkv, bs, d), 3), pool((layers, nb, hkv, bs, d), 4)
    wk, wv = reference(k, moves, [bs] * len(moves)), reference(v, moves, [bs] * len(moves))
    B.pkv_device_errors()
    t = tables.cuda()
    for _ in range(2):
        B.paged_kv_compact(k, v, moves.cuda(), t, block_map.cuda())
        assert torch.equal(t.cpu(), after)
        assert torch.equal(bits(k), wk) and torch.equal(bits(v), wv)
    # tables alone, and pages alone
    t = tables.cuda()
    B.paged_kv_compact(k, v, moves[:0].cuda(), t, block_map.cuda())
    assert torch.equal(t.cpu(), after)
    B.paged_kv_compact(k, v, moves.cuda())
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_compact_leaves_bad_entries(B):
    k, v = pool((1, 8, 1, 8, 64), 1), pool((1, 8, 1, 8, 64), 2)
    t = torch.tensor([[7, -1, 9, 3], [5, 2, -8, 7]], dtype=torch.int32).cuda()
    block_map = torch.tensor([0, 1, 2, 44, 4, -1, 6, 0], dtype=torch.int32).cuda()
    B.pkv_device_errors()
    B.paged_kv_compact(k, v, torch.tensor([[7, 0]], dtype=torch.int32).cuda(), t, block_map)
    assert t.cpu().tolist() == [[0, -1, 9, 3], [5, 2, -8, 0]]
    assert torch.equal(bits(k[0, 0]), bits(k[0, 7]))
    assert B.pkv_device_errors() == 1


@pytest.mark.gpu
def test_copy_blocks_in_a_graph_on_its_stream(B):
    """Captured on a side stream and replayed with other pairs in the same tensor."""
    k, v = pool((2, 30, 2, 16, 64), 7), pool((2, 30, 2, 16, 64), 8)
    pairs = torch.tensor([[0, 20], [1, 21]], dtype=torch.int32).cuda()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        B.paged_kv_copy_blocks(k, v, pairs)
    torch.cuda.synchronize()
    for new in ([[5, 22], [6, 23]], [[22, 24], [23, 25]]):
        pairs.copy_(torch.tensor(new, dtype=torch.int32))
        want = reference(k, torch.tensor(new), [16, 16])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(k), want)
