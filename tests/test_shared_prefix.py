"""paged_decode_shared_prefix_attention against a plain float64 implementation.

The allowed difference of an output o = sum p_t v_t, with A = sum p_t |v_t|: rounding it to
bf16 moves it by at most 2^-8 |o|; the prefix's weights enter the product with V as bf16,
each off by at most 2^-8 of itself, and are divided by the sum of the weights (of the
rounded ones at head_dim 64, of the unrounded ones at 128), so that half moves by at most 2 * 2^-8 of its A (the tail's weights keep 16 bits); fp32
scores, the hardware exp2 and the fp32 merge add less than 2^-12 A.
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


@pytest.fixture(autouse=True)
def always_shared(B):
    """The shared path at every size; test_modes_agree takes the others."""
    before = B.pkv_set_shared_prefix(B.SHARED_ALWAYS)
    yield
    B.pkv_set_shared_prefix(before)


def make(groups, prefixes, suffixes, hq, hkv, d, bs, seed, lead=0, tail=0, poison=True):
    """`groups`: sizes; one prefix each; one suffix per sequence.  `lead`/`tail` sequences of
    no group come before and after (their suffix is their whole context).  Slots that no
    sequence reads hold NaN."""
    rng = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lead + sum(groups) + tail
    assert len(suffixes) == n
    start = [lead]
    for s in groups:
        start.append(start[-1] + s)
    lens, rows = [], []
    shared = [p // bs for p in prefixes]
    need = 0
    for b in range(n):
        grp = next((i for i in range(len(groups)) if start[i] <= b < start[i + 1]), None)
        lens.append(suffixes[b] + (prefixes[grp] if grp is not None else 0))
        rows.append(grp)
    blocks = [-(-x // bs) for x in lens]
    nb = sum(shared) + sum(max(0, blocks[b] - (shared[rows[b]] if rows[b] is not None else 0))
                           for b in range(n)) + 3
    ids = rng.sample(range(nb), nb)
    common = [[ids.pop() for _ in range(s)] for s in shared]
    maxb = max(blocks + shared + [1]) + 1
    tables = torch.full((n, maxb), -1, dtype=torch.int32)
    for b in range(n):
        pre = common[rows[b]] if rows[b] is not None else []
        row = pre + [ids.pop() for _ in range(max(0, blocks[b] - len(pre)))]
        tables[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    k = torch.randn(nb, hkv, bs, d, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(nb, hkv, bs, d, generator=g, device="cuda").to(torch.bfloat16)
    if poison:
        live = torch.zeros(nb, bs, dtype=torch.bool)
        for i, s in enumerate(common):
            live[s] = True
        for b in range(n):
            for t in range(0, lens[b], bs):
                live[int(tables[b, t // bs]), :min(bs, lens[b] - t)] = True
        dead = ~live.cuda()
        k.masked_fill_(dead[:, None, :, None], float("nan"))
        v.masked_fill_(dead[:, None, :, None], float("nan"))
    q = torch.randn(n, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    longest = max(lens[b] - (shared[rows[b]] * bs if rows[b] is not None else 0) for b in range(n))
    return dict(q=q, k=k, v=v, tables=tables.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                start=torch.tensor(start, dtype=torch.int32).cuda(),
                prefix=torch.tensor(prefixes, dtype=torch.int32).cuda(),
                max_prefix=max(prefixes + [0]), max_suffix=max(longest, 0))


def reference(c, scale, lens=None):
    q, bs, d = c["q"], c["k"].shape[2], c["q"].shape[2]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    amp = torch.zeros_like(o)
    grp = q.shape[1] // c["k"].shape[1]
    for b, n in enumerate((c["lens"] if lens is None else lens).tolist()):
        if n == 0:
            continue
        at = c["tables"][b, :-(-n // bs)].long()
        for h in range(c["k"].shape[1]):
            kk = c["k"][at, h].reshape(-1, d)[:n].double()
            vv = c["v"][at, h].reshape(-1, d)[:n].double()
            p = torch.softmax(q[b, h * grp:(h + 1) * grp].double() @ kk.T * scale, -1)
            o[b, h * grp:(h + 1) * grp], amp[b, h * grp:(h + 1) * grp] = p @ vv, p @ vv.abs()
    return o, amp


def call(B, c, scale, ws=None, out=None):
    out = torch.full_like(c["q"], 3.0) if out is None else out
    B.paged_decode_shared_prefix_attention(out, c["q"], c["k"], c["v"], c["tables"], c["lens"],
                                           c["start"], c["prefix"], c["max_prefix"],
                                           c["max_suffix"], scale, workspace=ws)
    return out


def workspace(B, c):
    return torch.zeros(B.paged_decode_shared_prefix_workspace_size(
        c["q"].shape[0], c["q"].shape[1], c["k"].shape[1], c["q"].shape[2], c["prefix"].shape[0],
        c["max_prefix"], c["max_suffix"]), dtype=torch.uint8, device="cuda")


def check(out, o, amp, what=""):
    err = (out.double() - o).abs()
    bound = 2.0 ** -8 * o.abs() + (2.0 ** -7 + 2.0 ** -12) * amp + 1e-30
    assert bool((err <= bound).all()), f"{what}: {(err / bound).max().item():.3f} of the bound"


CASES = [
    # groups, prefixes, suffixes, hq, hkv, d, bs, lead, tail
    ([1], [64], [1], 1, 1, 64, 16, 0, 0),
    ([3], [512], [1, 40, 64], 32, 8, 64, 16, 0, 0),
    ([2], [100], [0, 5], 8, 2, 128, 8, 0, 0),                   # a prefix that ends inside a page
    ([40], [700], list(range(40)), 24, 8, 128, 32, 0, 0),       # group 3, 120 rows
    ([43], [1300], [7] * 43, 24, 8, 128, 16, 0, 0),             # 129 rows: a tile of one row
    ([5, 1, 9], [300, 0, 129], [3] * 15, 32, 4, 64, 16, 0, 0),  # a group without a prefix
    ([4, 4], [256, 31], [10] * 8, 8, 8, 64, 32, 0, 0),          # less than a page is not shared
    ([6], [640], [20] * 11, 16, 2, 64, 64, 3, 2),               # sequences of no group around it
    ([2] * 40, [48] * 40, [1] * 80, 4, 2, 128, 16, 0, 0),       # more groups than a warp has lanes
    ([3], [2048], [5000, 1, 1500], 24, 8, 128, 32, 0, 0),       # tails in several partitions
    ([2], [513], [1100, 900], 8, 1, 64, 256, 0, 0),
    ([17], [4096], [1] * 17, 6, 6, 128, 16, 0, 0),              # group 1
    ([], [], [70, 0, 9], 8, 2, 64, 16, 3, 0),                   # no group at all
]


@pytest.mark.gpu
@pytest.mark.parametrize("groups,prefixes,suffixes,hq,hkv,d,bs,lead,tail", CASES)
def test_matches_reference(B, groups, prefixes, suffixes, hq, hkv, d, bs, lead, tail):
    c = make(groups, prefixes, suffixes, hq, hkv, d, bs, 7 + len(suffixes), lead, tail)
    o, amp = reference(c, d ** -0.5)
    B.pkv_device_errors()
    ws = workspace(B, c)
    for _ in range(2):  # the workspace is left ready
        check(call(B, c, d ** -0.5, ws), o, amp, f"{groups} {prefixes}")
    check(call(B, c, d ** -0.5), o, amp)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (128, 32)])
def test_many_blocks_per_split(B, d, bs):
    """More groups than the prefix needs splits: every tile CTA walks dozens of key blocks of
    scattered pages, and its two tiles run apart."""
    rng = random.Random(d + bs)
    c = make([2] * 24, [rng.randint(2500, 6500) for _ in range(24)], [3] * 48, 24, 8, d, bs, 13,
             poison=False)
    o, amp = reference(c, d ** -0.5)
    ws = workspace(B, c)
    B.pkv_device_errors()
    for _ in range(4):
        check(call(B, c, d ** -0.5, ws), o, amp)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,hkv,d,bs,most", [(50, 8, 128, 16, 900), (170, 4, 128, 32, 700),
                                             (170, 4, 64, 16, 900), (36, 8, 128, 16, 300)])
def test_many_tails(B, n, hkv, d, bs, most):
    """More own parts than fit on the GPU at once, and (the last) just fewer; own lengths from
    none to many ring stages, with and without the sort by length."""
    rng = random.Random(n + d)
    suffixes = [rng.choice([0, 1, 63, 64, 65, 129, rng.randint(0, most), most]) for _ in range(n)]
    c = make([n // 2, n - n // 2], [600, 350], suffixes, 2 * hkv, hkv, d, bs, n, poison=False)
    o, amp = reference(c, d ** -0.5)
    ws = workspace(B, c)
    B.pkv_device_errors()
    for _ in range(3):
        check(call(B, c, d ** -0.5, ws), o, amp)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,scale", [(64, 1.0), (128, 1.0), (128, -0.5), (64, 0.0)])
def test_wide_scores(B, d, scale):
    """Scores of tens, whose maxima jump from block to block and from prefix to tail."""
    c = make([9], [900], [50] * 9, 6, 2, d, 16, 5)
    c["k"] = (c["k"].float() * (30 / d) ** 0.5).to(torch.bfloat16)
    check(call(B, c, scale), *reference(c, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_contexts_shorter_than_the_prefix(B, d):
    """Padded sequences (length 0) give zeros; a context that ends inside the prefix sees its
    own tokens only."""
    c = make([9], [800], [33] * 9, 8, 2, d, 16, 3)
    c["lens"][1:8] = torch.tensor([0, 1, 127, 128, 300, 799, 800], dtype=torch.int32)
    o, amp = reference(c, 0.125)
    B.pkv_device_errors()
    out = call(B, c, 0.125)
    check(out, o, amp)
    assert bool((out[1] == 0).all()) and B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [0, 1])
@pytest.mark.parametrize("n", [0, 2])
def test_nothing_to_do(B, n, groups):
    """No sequences; sequences without keys (zeros)."""
    q = torch.ones(n, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(8, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    c = dict(q=q, k=k, v=k, tables=torch.zeros(n, 4, dtype=torch.int32, device="cuda"),
             lens=torch.zeros(n, dtype=torch.int32, device="cuda"),
             start=torch.zeros(groups + 1, dtype=torch.int32, device="cuda"),
             prefix=torch.zeros(groups, dtype=torch.int32, device="cuda"), max_prefix=0, max_suffix=64)
    assert bool((call(B, c, 0.1) == 0).all()) and B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_modes_agree(B):
    """Shared, plain and by size, in turn on one workspace."""
    c = make([20, 4], [1000, 2500], list(range(24)), 32, 8, 64, 16, 1)
    o, amp = reference(c, 0.125)
    ws = workspace(B, c)
    B.pkv_device_errors()
    for mode in (B.SHARED_ALWAYS, B.SHARED_NEVER, B.SHARED_AUTO, B.SHARED_ALWAYS, B.SHARED_NEVER):
        B.pkv_set_shared_prefix(mode)
        check(call(B, c, 0.125, ws), o, amp, f"mode {mode}")
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_pages_past_4_gb(B):
    c = make([5], [700], [40] * 5, 16, 8, 128, 16, 6, poison=False)
    o, amp = reference(c, 0.09)
    nb, off = 135000, 135000 - c["k"].shape[0]  # 32 KB a page and head set
    for x in ("k", "v"):
        pool = torch.empty(nb, *c[x].shape[1:], dtype=torch.bfloat16, device="cuda")
        pool[off:] = c[x]
        c[x] = pool
    c["tables"] = torch.where(c["tables"] >= 0, c["tables"] + off, c["tables"])
    B.pkv_device_errors()
    check(call(B, c, 0.09), o, amp)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_two_calls_at_once(B):
    """Two streams, each with a workspace of its own, beside each other."""
    sets = [make([30, 9], [2100, 900], [64] * 39, 16, 4, 64, 16, 3),
            make([12], [3000], list(range(0, 600, 50)), 24, 8, 128, 32, 4)]
    refs = [reference(c, 0.1) for c in sets]
    spaces = [workspace(B, c) for c in sets]
    outs = [[torch.empty_like(c["q"]) for _ in range(6)] for c in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        for j, c in enumerate(sets):
            with torch.cuda.stream(streams[j]):
                call(B, c, 0.1, spaces[j], outs[j][i])
    torch.cuda.synchronize()
    for out, ref in zip(outs, refs):
        for x in out:
            check(x, *ref)


@pytest.mark.gpu
def test_workspace_of_its_own_on_a_given_stream(B):
    """stream= without a workspace while the current stream is busy and freed memory is not
    zero: the workspace is made in the given stream's order."""
    c = make([20], [2000], [70] * 20, 16, 4, 64, 16, 9, poison=False)
    o, amp = reference(c, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        dirty = torch.full((workspace(B, c).numel(),), 255, dtype=torch.uint8, device="cuda")
        del dirty
        out = torch.empty_like(c["q"])
        torch.cuda.current_stream().synchronize()
        torch.cuda._sleep(20_000_000)  # about 10 ms
        B.paged_decode_shared_prefix_attention(out, c["q"], c["k"], c["v"], c["tables"], c["lens"],
                                               c["start"], c["prefix"], c["max_prefix"],
                                               c["max_suffix"], 0.1, stream=side)
        side.synchronize()
        check(out, o, amp)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_one_workspace_for_many_sizes(B):
    """Calls of other batch sizes, heads and lengths, eager and as captured graphs, in turn on
    one workspace, shared and plain."""
    cs = [make([20, 4], [1000, 2500], list(range(24)), 32, 8, 64, 16, 1, poison=False),
          make([3], [300], [5, 0, 400], 8, 2, 128, 16, 2, poison=False),
          make([60, 30], [700, 900], [k % 7 * 90 for k in range(90)], 16, 8, 128, 32, 3, poison=False),
          make([2, 2, 2], [64, 0, 200], [1500, 2, 3, 4, 900, 6], 6, 1, 64, 16, 4, poison=False)]
    refs = [reference(c, 0.1) for c in cs]
    ws = max((workspace(B, c) for c in cs), key=lambda w: w.numel())
    outs, graphs = [torch.empty_like(c["q"]) for c in cs], []
    for mode in (B.SHARED_ALWAYS, B.SHARED_NEVER):
        B.pkv_set_shared_prefix(mode)
        for i, c in enumerate(cs):
            check(call(B, c, 0.1, ws), *refs[i], f"mode {mode}, {i}")
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(B, c, 0.1, ws, outs[i])
            graphs.append((i, g))
    rng = random.Random(7)
    for _ in range(4):
        for i, g in rng.sample(graphs, len(graphs)):
            outs[i].fill_(5.0)
            g.replay()
            check(outs[i], *refs[i], f"graph {i}")
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_equals_plain_decode(B):
    c = make([20, 4], [1000, 2500], list(range(24)), 32, 8, 64, 16, 1)
    a, b = call(B, c, 0.125), torch.empty_like(c["q"])
    B.paged_decode_attention(b, c["q"], c["k"], c["v"], c["tables"], c["lens"],
                             int(c["lens"].max()), 0.125)
    o, amp = reference(c, 0.125)
    check(a, o, amp)
    check(b, o, amp)


@pytest.mark.gpu
def test_graph_replay_and_streams(B):
    """One captured call, replayed as the contexts grow and shrink; on a side stream too."""
    c = make([12], [1024], [200] * 12, 24, 8, 128, 16, 2, poison=False)
    ws, out = workspace(B, c), torch.empty_like(c["q"])
    call(B, c, 0.09, ws, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(B, c, 0.09, ws, out)
    full = c["lens"].clone()
    for cut in (0, 150, 199, 1000, 7):
        c["lens"].copy_(full - cut)
        g.replay()
        torch.cuda.synchronize()
        check(out, *reference(c, 0.09), f"cut {cut}")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(B, c, 0.09, ws, out)
    s.synchronize()
    check(out, *reference(c, 0.09))


@pytest.mark.gpu
def test_bad_values_are_flagged(B):
    c = make([4], [256], [10] * 4, 8, 2, 64, 16, 4, poison=False)
    o, amp = reference(c, 0.125)

    def flags(**change):
        B.pkv_device_errors()
        out = call(B, {**c, **change}, 0.125)
        return B.pkv_device_errors(), out

    i32 = dict(dtype=torch.int32, device="cuda")
    assert flags()[0] == 0
    assert flags(prefix=torch.tensor([257], **i32), max_prefix=256)[0] == 4
    assert flags(prefix=torch.tensor([-1], **i32), max_suffix=266)[0] == 4
    assert flags(start=torch.tensor([0, 5], **i32))[0] == 4
    assert flags(start=torch.tensor([-2, 4], **i32))[0] == 4
    assert flags(max_suffix=9)[0] == 4
    assert flags(lens=torch.tensor([-1, 266, 266, 266], **i32))[0] == 4
    t = c["tables"].clone()
    t[0, 3] = 10 ** 6  # a page of the prefix, and one of a tail
    assert flags(tables=t)[0] == 1
    t = c["tables"].clone()
    t[2, 16] = -7
    f, out = flags(tables=t)
    assert f == 1
    check(out[[0, 1, 3]], o[[0, 1, 3]], amp[[0, 1, 3]])
    assert flags()[0] == 0  # and the next call is clean


@pytest.mark.gpu
def test_prompt_fork_decode_copy_on_write_compact(B):
    """The set as a server uses it: a packed prompt, its pages, forks, decode steps that share
    them with copy-on-write, a fork that leaves, a compaction, and on."""
    hq, hkv, d, bs, n0 = 8, 2, 64, 16, 150
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    bm = B.BlockManager(64, bs)
    kc, vc = torch.zeros(64, hkv, bs, d, dtype=torch.bfloat16, device="cuda"), \
        torch.zeros(64, hkv, bs, d, dtype=torch.bfloat16, device="cuda")
    bm.add_sequence(99, 40)  # something that leaves later: the pool gets holes
    bm.add_sequence(0, 0)
    q, k, v = rand(n0, hq + 2 * hkv, d).split([hq, hkv, hkv], dim=1)
    out = torch.empty(n0, hq, d, dtype=torch.bfloat16, device="cuda")
    B.prompt_attention(out, q, k, v, torch.tensor([0, n0], dtype=torch.int32, device="cuda"), n0, 0.125)
    B.paged_kv_write(k.contiguous(), v.contiguous(), bm.append_slots([0] * n0).cuda(), kc, vc)
    ids = [0]
    for child in range(1, 7):
        bm.fork(0, child)
        ids.append(child)
    hist = {s: (list(k.unbind(0)), list(v.unbind(0))) for s in ids}
    B.pkv_device_errors()
    for step in range(30):
        if step == 12:
            bm.free_sequence(3)
            ids.remove(3)
            bm.free_sequence(99)
        if step == 15:
            tables, _ = bm.block_tables(ids, 16)
            moves, block_map = bm.compact()
            assert len(moves) > 0
            dev = tables.cuda()
            B.paged_kv_compact(kc, vc, moves.cuda(), dev, block_map.cuda())
            assert torch.equal(dev.cpu(), bm.block_tables(ids, 16)[0])
        nq, nk, nv = rand(len(ids), hq, d), rand(len(ids), hkv, d), rand(len(ids), hkv, d)
        slots, pairs, rows = bm.append_slots_cow(ids)
        assert len(pairs) == (6 if step == 0 else 0)  # the last holder writes in place
        B.paged_kv_copy_blocks(kc, vc, pairs.cuda(), rows.cuda())
        B.paged_kv_write(nk, nv, slots.cuda(), kc, vc)
        tables, lens = bm.block_tables(ids, 16)
        o = torch.empty_like(nq)
        B.paged_decode_shared_prefix_attention(
            o, nq, kc, vc, tables.cuda(), lens.cuda(),
            torch.tensor([0, len(ids)], dtype=torch.int32, device="cuda"),
            torch.tensor([n0], dtype=torch.int32, device="cuda"), n0, 64, 0.125)
        for i, s in enumerate(ids):
            hist[s][0].append(nk[i])
            hist[s][1].append(nv[i])
            kk, vv = (torch.stack(x).double() for x in hist[s])
            for h in range(hq):
                p = torch.softmax(kk[:, h // 4] @ nq[i, h].double() * 0.125, 0)
                check(o[i, h], p @ vv[:, h // 4], p @ vv[:, h // 4].abs(), f"step {step} sequence {s}")
    assert B.pkv_device_errors() == 0


def test_argument_errors(B):
    lib = B.lib()

    def run(out=FAKE, start=FAKE, prefix=FAKE, groups=1, mp=64, ms=40, n=2, hq=8, d=64, bs=16, hkv=2,
            ws=None, nbytes=0):
        return lib.paged_decode_shared_prefix_attention(
            out, FAKE, FAKE, FAKE, FAKE, 8, FAKE, start, prefix, groups, mp, ms, n, hq,
            ctypes.byref(B.pkv_cache_desc(64, bs, hkv, d)), 0.125, ws, nbytes, None)

    assert run(d=96) == -3 and run(bs=12) == -3 and run(hkv=1, hq=16) == -3
    assert run(hq=7) == -2 and run(mp=129) == -2 and run(ms=129) == -2  # over the table
    assert run(mp=-1) == -2 and run(ms=-1) == -2 and run(groups=-1) == -2
    assert run(out=None) == -1 and run(start=None) == -1 and run(prefix=None) == -1
    assert run(out=ctypes.c_void_p((1 << 20) + 2)) == -5
    assert run(n=0) == 0


def test_unknown_mode(B):
    assert B.lib().pkv_set_shared_prefix(3) == -3 and B.lib().pkv_set_shared_prefix(-1) == -3
    with pytest.raises(B.PkvError):
        B.pkv_set_shared_prefix(7)


def test_workspace_size(B):
    size = B.paged_decode_shared_prefix_workspace_size
    assert size(0, 8, 2, 64, 1, 100, 100) == 0 and size(2, 8, 2, 96, 1, 100, 100) == 0
    assert size(2, 8, 2, 64, -1, 100, 100) == 0 and size(2, 8, 2, 64, 1, -1, 100) == 0
    # at least a counter per (sequence, kv head) and two prefix rows and a tail row per head
    assert size(4, 32, 8, 128, 1, 1000, 50) >= 4 * 8 * 4 + 3 * 4 * 32 * 129 * 4
    assert size(4, 32, 8, 128, 0, 0, 50) > 0
