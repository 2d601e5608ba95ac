"""The 8-bit cache's quantising write, with and without rotary embedding, and its reading back:
codes and scales bit for bit as defined, every other byte of the pools as it was."""

import math

import pytest
import torch

import q8_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    binding.pkv_device_errors(clear=True)
    return binding


class Batch:
    """Sequences of `lens` tokens in shuffled pages of a pool with spare pages."""

    def __init__(self, lens, dtype, hkv=2, d=64, bs=16, seed=0):
        self.gen = torch.Generator().manual_seed(seed)
        self.lens, self.bs, self.hkv, self.d, self.dtype = list(lens), bs, hkv, d, dtype
        need = sum(-(-n // bs) for n in lens)
        self.nb = need + 3
        perm = torch.randperm(self.nb, generator=self.gen).tolist()
        width = max(1, max(-(-n // bs) for n in lens)) + 1
        self.tables = []
        for n in lens:
            m = -(-n // bs)
            self.tables.append(perm[:m] + [-1] * (width - m))
            perm = perm[m:]
        self.k, self.v, self.ks, self.vs = R.pools(self.nb, hkv, bs, d, dtype, self.gen, DEV)
        self.bt = torch.tensor(self.tables, dtype=torch.int32, device=DEV)
        self.cl = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def cache(self):
        return self.k, self.v, self.ks, self.vs

    def copies(self):
        return [t.clone() for t in self.cache()]

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen).to(torch.bfloat16).to(DEV)


def starts(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)


def same(a, b, what):
    a, b = R.bits(a), R.bits(b)
    if a.dtype is torch.float32:
        a, b = a.view(torch.int32), b.view(torch.int32)
    assert torch.equal(a, b), f"{what}: {int((a != b).sum())} of {a.numel()} differ"


def check_write(b, new, k, v, before):
    want = before
    at = 0
    for s, n in enumerate(new):
        R.write(want[0], want[2], k[at:at + n], b.tables[s], b.lens[s] - n)
        R.write(want[1], want[3], v[at:at + n], b.tables[s], b.lens[s] - n)
        at += n
    for x, y, what in zip(b.cache(), want, ("k codes", "v codes", "k scales", "v scales")):
        same(x, y, what)


SHAPES = [
    # lens, new tokens, kv heads, head_dim, block size
    ([1], [1], 1, 64, 8),
    ([16, 17, 31, 32, 33], [1, 1, 1, 1, 1], 3, 64, 16),
    ([40, 0, 5, 100], [40, 0, 5, 3], 2, 128, 16),
    ([300, 299, 17], [300, 43, 1], 2, 64, 32),
    ([513, 70], [257, 70], 1, 128, 256),
    ([600], [599], 2, 128, 128),
    ([9, 1000], [2, 990], 5, 64, 8),
    ([65, 64, 130], [64, 64, 129], 2, 128, 64),
]


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("lens,new,hkv,d,bs", SHAPES)
def test_write_codes_and_scales(B, dtype, lens, new, hkv, d, bs):
    b = Batch(lens, dtype, hkv, d, bs, seed=1)
    t = sum(new)
    k, v = b.randn(t, hkv, d), b.randn(t, hkv, d) * 3
    before = b.copies()
    B.paged_kv_write_q8(k, v, *b.cache(), b.bt, b.cl, starts(new), max(new))
    check_write(b, new, k, v, before)
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
def test_pages_grow_token_by_token(B, dtype):
    """40 steps of one token: scales grow within a page (rows rounded anew) and begin again."""
    lens = [3, 20, 60, 0]
    b = Batch([n + 40 for n in lens[:3]] + [0], dtype, 2, 64, 16, seed=2)
    want = b.copies()
    for step in range(40):
        now = [n + step + 1 for n in lens[:3]] + [0]
        cl = torch.tensor(now, dtype=torch.int32, device=DEV)
        k, v = b.randn(4, 2, 64) * (1 + step % 7), b.randn(4, 2, 64)
        B.paged_kv_write_q8(k, v, *b.cache(), b.bt, cl)
        for s, n in enumerate(now[:3]):
            R.write(want[0], want[2], k[s:s + 1], b.tables[s], n - 1)
            R.write(want[1], want[3], v[s:s + 1], b.tables[s], n - 1)
    for x, y, what in zip(b.cache(), want, ("k codes", "v codes", "k scales", "v scales")):
        same(x, y, what)
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
def test_write_from_slices_of_a_projection(B, dtype):
    lens, new = [50, 21], [30, 2]
    b = Batch(lens, dtype, 2, 128, 16, seed=3)
    x = b.randn(32, 7, 128)
    k, v = x[:, 3:5], x[:, 5:7]
    before = b.copies()
    B.paged_kv_write_q8(k, v, *b.cache(), b.bt, b.cl, starts(new), 30)
    check_write(b, new, k, v, before)
    out = torch.full((32, 6, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    B.paged_kv_read_q8(out[:, 0:2], out[:, 4:6], *b.cache(), b.bt, b.cl, starts(new), 30)
    for s, (n, m, at) in enumerate(((30, 50, 0), (2, 21, 30))):
        for codes, scale, lo in ((b.k, b.ks, 0), (b.v, b.vs, 4)):
            want = R.values(codes, scale, b.tables[s], m - n, m).to(torch.bfloat16)
            assert torch.equal(out[at:at + n, lo:lo + 2], want)
    assert bool((out[:, 2:4] == 7).all())


@pytest.mark.parametrize("dtype", R.KINDS)
def test_values_at_the_edges(B, dtype):
    """Zeros, a page of zeros that grows, the smallest and largest numbers, infinities and NaN."""
    rows = torch.zeros(64, 1, 64)
    rows[17, 0, 5] = 1.0                    # zeros, then one value: page 1
    rows[32:48] = torch.randn(16, 1, 64, generator=torch.Generator().manual_seed(4)) * 1e-38
    rows[48:64] = torch.randn(16, 1, 64, generator=torch.Generator().manual_seed(5)) * 1e37
    rows = rows.to(torch.bfloat16)
    rows[48, 0, 0] = 3.3895e38              # the largest bf16
    rows[33, 0, 1] = 1e-40                  # not a normal number
    rows = rows.to(DEV)
    b = Batch([64], dtype, 1, 64, 16, seed=6)
    for lo, hi in ((0, 5), (5, 17), (17, 18), (18, 33), (33, 64)):
        before = b.copies()
        cl = torch.tensor([hi], dtype=torch.int32, device=DEV)
        k = rows[lo:hi]
        B.paged_kv_write_q8(k, -k, *b.cache(), b.bt, cl, starts([hi - lo]), hi - lo)
        R.write(before[0], before[2], k, b.tables[0], lo)
        R.write(before[1], before[3], -k, b.tables[0], lo)
        for x, y, what in zip(b.cache(), before, ("k codes", "v codes", "k scales", "v scales")):
            same(x, y, f"{what} {lo}..{hi}")
    assert bool(torch.isfinite(b.ks[b.tables[0][:4]]).all())
    # what is not finite makes its page NaN (this head of it), until the page begins again
    for bad in (math.inf, -math.inf, math.nan):
        k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=DEV)
        k[0, 0, 63] = bad
        cl = torch.tensor([62], dtype=torch.int32, device=DEV)
        B.paged_kv_write_q8(k, torch.ones_like(k), *b.cache(), b.bt, cl)
        assert math.isnan(b.ks[b.tables[0][3], 0]) and math.isfinite(b.vs[b.tables[0][3], 0])
        ko, vo = (torch.zeros(64, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        B.paged_kv_read_q8(ko, vo, *b.cache(), b.bt, b.cl, starts([64]), 64)
        assert bool(ko[48:].isnan().all()) and bool(ko[:48].isfinite().all()) and bool(vo.isfinite().all())
        k[0, 0, 63] = 2.0
        B.paged_kv_write_q8(k, k, *b.cache(), b.bt, torch.tensor([63], dtype=torch.int32, device=DEV))
        assert math.isnan(b.ks[b.tables[0][3], 0])
        B.paged_kv_write_q8(rows[48:64], rows[48:64], *b.cache(), b.bt, b.cl, starts([16]), 16)
        assert math.isfinite(b.ks[b.tables[0][3], 0])
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("dtype,d,r,hq,given", [
    (torch.int8, 64, 64, 4, False), (torch.float8_e4m3fn, 128, 32, 6, True), (torch.int8, 128, 128, 1, True),
    (torch.float8_e4m3fn, 64, 16, 3, False),
])
def test_rotary_write(B, neox, dtype, d, r, hq, given):
    lens, new, hkv = [70, 33, 0, 16], [70, 1, 0, 5], 2
    b = Batch(lens, dtype, hkv, d, 16, seed=7)
    t = sum(new)
    x = b.randn(t, hq + 2 * hkv, d)
    q, k, v = x.split([hq, hkv, hkv], dim=1)
    pos = torch.cat([torch.arange(m - n, m) for m, n in zip(lens, new)])
    if given:
        pos = (pos * 7 + 3) % 90
    freq = 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    ang = torch.arange(90, dtype=torch.float64)[:, None] * freq
    table = torch.cat((ang.cos(), ang.sin()), 1).float().to(DEV)
    pos = pos.to(DEV)
    before = b.copies()
    q_out = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)
    kw = dict(rotary_dim=r, neox_style=neox, positions=pos if given else None)
    want_q, want_k = R.rotate(q, table, pos, r, neox), R.rotate(k, table, pos, r, neox)
    B.paged_kv_write_rope_q8(k, v, table, *b.cache(), b.bt, b.cl, starts(new), max(new), q=q, q_out=q_out, **kw)
    check_write(b, new, want_k, v, before)
    assert torch.equal(q_out, want_q)
    B.paged_kv_write_rope_q8(k, v, table, *b.cache(), b.bt, b.cl, starts(new), max(new), q=q, **kw)  # in place
    assert torch.equal(x[:, :hq], want_q)
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("lens,back,hkv,d,bs", [
    ([300], [300], 8, 64, 16), ([5, 0, 1000, 77], [5, 0, 1000, 77], 2, 128, 32),
    ([40, 513], [3, 200], 1, 128, 256), ([9, 8], [9, 1], 3, 64, 8),
])
def test_reading_back(B, dtype, lens, back, hkv, d, bs):
    b = Batch(lens, dtype, hkv, d, bs, seed=8)
    t = sum(back)
    ko = torch.full((t + 2, hkv, d), 5.0, dtype=torch.bfloat16, device=DEV)
    vo = ko.clone()
    B.paged_kv_read_q8(ko, vo, *b.cache(), b.bt, b.cl, starts(back), max(back))
    at = 0
    for s, n in enumerate(back):
        for got, codes, scale in ((ko, b.k, b.ks), (vo, b.v, b.vs)):
            want = R.values(codes, scale, b.tables[s], lens[s] - n, lens[s]).to(torch.bfloat16)
            assert torch.equal(got[at:at + n], want)
        at += n
    assert bool((ko[t:] == 5).all()) and bool((vo[t:] == 5).all())  # rows of no sequence
    assert B.pkv_device_errors() == 0


def test_bad_lengths_and_pages_are_skipped(B):
    """Flagged, nothing written outside what the call names, the other sequences complete."""
    CL, ID = 4, 1
    b = Batch([20, 20, 20], torch.int8, 1, 64, 16, seed=9)
    k = b.randn(6, 1, 64)
    for cl, st, most, flag in (
            ([20, -1, 20], [0, 2, 4, 6], 2, CL), ([20, 1, 20], [0, 2, 4, 6], 2, CL),      # n > L
            ([20, 1000, 20], [0, 2, 4, 6], 2, CL), ([20, 20, 20], [0, 2, 6, 8], 2, CL),   # n > max, rows out
            ([20, 20, 20], [0, 2, 1, 3], 2, CL)):                                         # decreasing
        before = b.copies()
        c = torch.tensor(cl, dtype=torch.int32, device=DEV)
        s = torch.tensor(st, dtype=torch.int32, device=DEV)
        B.paged_kv_write_q8(k, k, *b.cache(), b.bt, c, s, most)
        assert B.pkv_device_errors() == flag
        for i in range(3):
            n = st[i + 1] - st[i]
            if 0 <= n <= most and n <= cl[i] <= 48 and st[i + 1] <= 6:
                R.write(before[0], before[2], k[st[i]:st[i + 1]], b.tables[i], cl[i] - n)
                R.write(before[1], before[3], k[st[i]:st[i + 1]], b.tables[i], cl[i] - n)
        for x, y in zip(b.cache(), before):
            same(x, y, "pools")
        out = torch.zeros(6, 1, 64, dtype=torch.bfloat16, device=DEV)
        B.paged_kv_read_q8(out, out.clone(), *b.cache(), b.bt, c, s, most)
        assert B.pkv_device_errors() == flag
    bt = b.bt.clone()
    bt[1, 1] = b.nb
    before = b.copies()
    B.paged_kv_write_q8(k[:3], k[:3], *b.cache(), bt, b.cl)
    assert B.pkv_device_errors() == ID
    for i in (0, 2):
        R.write(before[0], before[2], k[i:i + 1], b.tables[i], 19)
        R.write(before[1], before[3], k[i:i + 1], b.tables[i], 19)
    for x, y in zip(b.cache(), before):
        same(x, y, "pools")


def test_positions_out_of_range(B):
    b = Batch([20, 20], torch.int8, 1, 64, 16, seed=10)
    x = b.randn(2, 3, 64)
    table = torch.ones(10, 64, device=DEV)
    before = b.copies()
    q_out = torch.full((2, 1, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    pos = torch.tensor([10, -1], device=DEV)
    B.paged_kv_write_rope_q8(x[:, 1:2], x[:, 2:], table, *b.cache(), b.bt, b.cl, q=x[:, :1], q_out=q_out,
                             positions=pos)
    assert B.pkv_device_errors() == 16
    assert bool((q_out == 9).all())
    same(b.k, before[0], "k codes")
    same(b.ks, before[2], "k scales")
    for i in range(2):
        R.write(before[1], before[3], x[i:i + 1, 2:], b.tables[i], 19)
    same(b.v, before[1], "v codes")


def test_nothing_to_do(B):
    b = Batch([20], torch.int8, 1, 64, 16, seed=11)
    before = b.copies()
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    B.paged_kv_write_q8(none, none, *b.cache(), b.bt, b.cl, starts([0]), 0)
    B.paged_kv_write_q8(none, none, *b.cache(), b.bt[:0], b.cl[:0])
    B.paged_kv_read_q8(none, none, *b.cache(), b.bt, b.cl, starts([0]), 4)
    for x, y in zip(b.cache(), before):
        same(x, y, "pools")
    assert B.pkv_device_errors() == 0


def test_pages_past_4_gb(B):
    """A pool of more than 2^32 codes: the last pages are written and read at their own places."""
    nb, hkv, bs, d = 33000, 8, 256, 64   # 4.3e9 codes each for K and V
    k, v = (torch.empty(nb, hkv, bs, d, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(nb, hkv, device=DEV) for _ in range(2))
    x = torch.randn(300, hkv, d, generator=torch.Generator().manual_seed(12)).to(torch.bfloat16).to(DEV)
    table = [[nb - 1, nb - 2]]
    bt = torch.tensor(table, dtype=torch.int32, device=DEV)
    cl = torch.tensor([300], dtype=torch.int32, device=DEV)
    B.paged_kv_write_q8(x, -x, k, v, ks, vs, bt, cl, starts([300]), 300)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    B.paged_kv_read_q8(ko, vo, k, v, ks, vs, bt, cl, starts([300]), 300)
    assert torch.equal(ko, -vo)
    top = x.float().abs().amax()
    assert float((ko.float() - x.float()).abs().max()) <= float(top) / 127 / 2 + 2.0 ** -8 * float(top)
    assert bool((ks[:nb - 2] == 0).all()) and B.pkv_device_errors() == 0
    q = torch.randn(1, hkv, d, generator=torch.Generator().manual_seed(13)).to(torch.bfloat16).to(DEV)
    out = torch.empty_like(q)
    B.paged_decode_attention_q8(out, q, k, v, ks, vs, bt, cl, 300, 0.125)
    want, mag = R.attention(q, R.values(k, ks, table[0], 0, 300), R.values(v, vs, table[0], 0, 300), 0.125)
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag).all())


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("layers,form", [(1, "one"), (3, "stacked"), (70, "list")])
def test_pages_are_copied_with_their_scales(B, dtype, layers, form):
    gen = torch.Generator().manual_seed(14)
    pools = [R.pools(20, 2, 16, 64, dtype, gen, DEV) for _ in range(layers)]
    want = [[t.clone() for t in p] for p in pools]
    pairs = [(3, 10), (3, 11), (4, 12), (5, 5), (6, 13), (7, 14)]
    rows = [16, 5, 0, 3, 1, 16]
    for p in want:
        for (s, t), n in zip(pairs, rows):
            if s != t and n:
                for codes, scale in ((p[0], p[2]), (p[1], p[3])):
                    R.bits(codes)[t, :, :n] = R.bits(codes)[s, :, :n]
                    scale[t] = scale[s]
    given = [list(x) for x in zip(*pools)]
    if form == "one":
        args = [x[0] for x in given]
    elif form == "stacked":
        args = [torch.stack([R.bits(t) for t in x]).view(x[0].dtype) for x in given]
    else:
        args = given
    bp = torch.tensor(pairs, dtype=torch.int32, device=DEV)
    B.paged_kv_copy_blocks_q8(*args, bp, torch.tensor(rows, dtype=torch.int32, device=DEV))
    for l in range(layers):
        for i in range(4):
            same(args[i] if form == "one" else args[i][l], want[l][i], f"layer {l}")
    assert B.pkv_device_errors() == 0
    # a compaction: two pages into free ones, the tables after them
    table = torch.tensor([[3, 19, -1], [18, 4, 5]], dtype=torch.int32, device=DEV)
    bmap = torch.arange(20, dtype=torch.int32, device=DEV)
    bmap[19], bmap[18] = 0, 1
    B.paged_kv_compact_q8(*args, torch.tensor([[19, 0], [18, 1]], dtype=torch.int32, device=DEV), table, bmap)
    assert table.tolist() == [[3, 0, -1], [1, 4, 5]]
    for l in range(layers):
        for i in range(4):
            x = args[i] if form == "one" else args[i][l]
            want[l][i][0], want[l][i][1] = R.bits(want[l][i])[19].view(x.dtype), R.bits(want[l][i])[18].view(x.dtype)
            same(x, want[l][i], f"layer {l}")
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
def test_forks_write_into_copies(B, dtype):
    """The block manager's forks over an 8-bit cache: a prompt written, forked, each fork's next tokens
    into its own copy of the last page; every sequence reads what writing it alone would give."""
    n, hkv, d, bs, nb, steps = 37, 2, 64, 16, 40, 3
    gen = torch.Generator().manual_seed(15)
    k, v, ks, vs = R.pools(nb, hkv, bs, d, dtype, gen, DEV)
    prompt = torch.randn(2, n, hkv, d, generator=gen).to(torch.bfloat16).to(DEV)
    bm = B.BlockManager(nb, bs)
    bm.add_sequence(0, n)
    bt, cl = bm.block_tables([0], 5)
    B.paged_kv_write_q8(prompt[0], prompt[1], k, v, ks, vs, bt.to(DEV), cl.to(DEV), starts([n]), n)
    for child in (1, 2, 3):
        bm.fork(0, child)
    new = torch.randn(2, steps, 4, hkv, d, generator=gen).to(torch.bfloat16).to(DEV) * 2
    for s in range(steps):
        _, pairs, rows = bm.append_slots_cow(range(4))
        if pairs.shape[0]:
            B.paged_kv_copy_blocks_q8(k, v, ks, vs, pairs.to(DEV), rows.to(DEV))
        bt, cl = bm.block_tables(list(range(4)), 5)
        B.paged_kv_write_q8(new[0, s], new[1, s], k, v, ks, vs, bt.to(DEV), cl.to(DEV))
    tables = bt.tolist()
    for seq in range(4):
        alone = [t.clone().zero_() if t.dtype is torch.float32 else torch.zeros_like(R.bits(t)).view(t.dtype)
                 for t in (k, v, ks, vs)]
        for i, (codes, scale, mine, my_scale) in enumerate(((alone[0], alone[2], k, ks), (alone[1], alone[3], v, vs))):
            R.write(codes, scale, prompt[i], tables[seq], 0)
            for s in range(steps):
                R.write(codes, scale, new[i, s, seq][None], tables[seq], n + s)
            got = R.values(mine, my_scale, tables[seq], 0, n + steps)
            assert torch.equal(got, R.values(codes, scale, tables[seq], 0, n + steps)), f"sequence {seq}"
    assert B.pkv_device_errors() == 0
