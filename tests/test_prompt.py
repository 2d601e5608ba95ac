"""prompt_attention against a plain float64 implementation.

The allowed difference of an output o = sum p_t v_t, with A = sum p_t |v_t|: rounding it to
bf16 moves it by at most 2^-8 |o|; the weights enter the product as bf16, each off by at
most 2^-8 of itself, and are divided by the sum of the weights (of the rounded ones at
head_dim 64, of the unrounded ones at 128), so the quotient moves by at most 2 * 2^-8 A; fp32 scores of 128 products and the hardware exp2 add less than
2^-12 A (128 * 2^-24 of |scale q k| <= 30 in the exponent, plus 2^-22 per weight).
"""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced by the host checks


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


def make(lens, hq, hkv, d, fused, seed, lead=0, tail=0):
    """Packed q, k, v (slices of one projection when fused) with `lead` and `tail` rows that
    belong to no sequence, and query_start."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = lead + sum(lens) + tail
    if fused:
        x = torch.randn(t, hq + 2 * hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = x.split([hq, hkv, hkv], dim=1)
    else:
        q, k, v = (torch.randn(t, h, d, generator=g, device="cuda").to(torch.bfloat16)
                   for h in (hq, hkv, hkv))
    start = [lead]
    for n in lens:
        start.append(start[-1] + n)
    return q, k, v, torch.tensor(start, dtype=torch.int32)


def reference(q, k, v, start, scale):
    """(o, A) of every row in float64; rows of no sequence are zero."""
    t, hq, d = q.shape
    grp = hq // k.shape[1]
    o = torch.zeros(t, hq, d, dtype=torch.float64, device=q.device)
    amp = torch.zeros_like(o)
    for a, z in zip(start[:-1].tolist(), start[1:].tolist()):
        n = z - a
        if n == 0:
            continue
        mask = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        for h in range(hq):
            x = q[a:z, h].double() @ k[a:z, h // grp].double().T * scale
            p = torch.softmax(torch.where(mask, x, -float("inf")), -1)
            vv = v[a:z, h // grp].double()
            o[a:z, h], amp[a:z, h] = p @ vv, p @ vv.abs()
    return o, amp


def check(out, o, amp, what=""):
    err = (out.double() - o).abs()
    bound = 2.0 ** -8 * o.abs() + (2.0 ** -7 + 2.0 ** -12) * amp + 1e-30
    assert bool((err <= bound).all()), f"{what}: {(err / bound).max().item():.3f} of the bound"


CASES = [
    # lens, hq, hkv, d, fused
    ([1], 1, 1, 64, False),
    ([1, 0, 2, 0], 8, 2, 128, True),
    ([31, 32, 33], 8, 8, 64, True),               # group 1
    ([127, 128, 129, 1], 4, 4, 128, False),       # block borders at group 1
    ([42, 43, 85, 86, 300], 24, 8, 128, True),    # group 3: tiles end inside a token
    ([64, 0, 1, 257, 500], 32, 8, 64, True),
    ([700, 3], 32, 4, 128, False),                # group 8
    ([100, 29], 32, 1, 64, True),                 # one kv head, group 32
    ([5, 260], 10, 2, 128, True),                 # group 5
    ([1100], 3, 1, 64, False),
    ([1] * 70 + [130] * 3, 4, 2, 64, False),      # more sequences than a warp has lanes
    ([60, 7, 131], 128, 1, 64, True),             # a token fills a tile
    ([40, 129], 100, 1, 128, False),              # tiles of one token and 28 empty rows
    ([50, 3], 65, 1, 64, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,hq,hkv,d,fused", CASES)
def test_matches_reference(B, lens, hq, hkv, d, fused):
    q, k, v, start = make(lens, hq, hkv, d, fused, seed=sum(lens) + hq, lead=3, tail=2)
    out = torch.full((q.shape[0], hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    B.pkv_device_errors()
    B.prompt_attention(out, q, k, v, start.cuda(), max(lens), d ** -0.5)
    assert B.pkv_device_errors() == 0
    o, amp = reference(q, k, v, start, d ** -0.5)
    a, z = int(start[0]), int(start[-1])
    check(out[a:z], o[a:z], amp[a:z], f"{lens}")
    assert bool((out[:a] == 7).all()) and bool((out[z:] == 7).all())  # rows of no sequence


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(24, 8, 128), (8, 8, 64), (10, 2, 128), (16, 2, 64)])
def test_many_items_per_cta(B, hq, hkv, d):
    """Far more tiles than SMs: every CTA goes through many items, of sequences of all sizes
    (none, one token, tiles whose halves end in the same block and in different ones)."""
    g = torch.Generator().manual_seed(hq + d)
    lens = torch.randint(0, 420, (150,), generator=g).tolist() + [1, 0, 127, 128, 129, 2000]
    q, k, v, start = make(lens, hq, hkv, d, True, seed=d)
    out = torch.empty(q.shape[0], hq, d, dtype=torch.bfloat16, device="cuda")
    o, amp = reference(q, k, v, start, d ** -0.5)
    B.pkv_device_errors()
    for _ in range(3):
        out.fill_(9.0)
        B.prompt_attention(out, q, k, v, start.cuda(), max(lens), d ** -0.5)
        check(out, o, amp)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_short_sequences(B, d):
    """Hundreds of sequences of a few tokens or none: a CTA's items lie far apart in the list,
    and the grid holds many more pieces than there are."""
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(-20, 30, (1100,), generator=g).clamp(min=0).tolist() + [0] * 200 + [50]
    q, k, v, start = make(lens, 8, 2, d, True, seed=d)
    out = torch.empty(q.shape[0], 8, d, dtype=torch.bfloat16, device="cuda")
    o, amp = reference(q, k, v, start, d ** -0.5)
    B.pkv_device_errors()
    B.prompt_attention(out, q, k, v, start.cuda(), max(lens), d ** -0.5)
    check(out, o, amp)
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rows_past_4_gb(B, d):
    """Token strides of 8 MB: the last rows lie past 2^31 elements and 2^32 bytes."""
    step, lens = 1 << 22, [200, 370]
    q, k, v, start = make(lens, 4, 2, d, False, seed=8)
    base = torch.empty(4, sum(lens) * step, dtype=torch.bfloat16, device="cuda")
    far = []
    for x, t in zip((q, k, v, q), base):
        y = t.as_strided((x.shape[0], x.shape[1], d), (step, d, 1))
        far.append(y.copy_(x))
    B.prompt_attention(far[3], far[0], far[1], far[2], start.cuda(), 370, d ** -0.5)
    check(far[3], *reference(q, k, v, start, d ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_long_prompt(B, d):
    """One prompt of 100003 tokens, compared at rows of its start, its middle and its end."""
    n = 100003
    q, k, v, start = make([n], 6, 2, d, True, seed=d)
    out = torch.empty(n, 6, d, dtype=torch.bfloat16, device="cuda")
    B.pkv_device_errors()
    B.prompt_attention(out, q, k, v, start.cuda(), n, 2 * d ** -0.5)
    assert B.pkv_device_errors() == 0
    for i in (0, 1, 127, 128, 50000, 65535, 65536, 99999, n - 1):
        for h in range(6):
            kk, vv = k[:i + 1, h // 3].double(), v[:i + 1, h // 3].double()
            p = torch.softmax(kk @ q[i, h].double() * (2 * d ** -0.5), 0)
            check(out[i, h], p @ vv, p @ vv.abs(), f"row {i}")


@pytest.mark.gpu
def test_two_calls_at_once(B):
    """Two streams' calls beside each other, many times over."""
    sets = [make([700, 90, 1300], 12, 4, 128, True, seed=1), make([33] * 60, 8, 2, 64, False, seed=2)]
    refs = [reference(*x, 0.1) for x in sets]
    starts = [x[3].cuda() for x in sets]
    outs = [[torch.empty_like(x[0]) for _ in range(6)] for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        for j, (q, k, v, start) in enumerate(sets):
            with torch.cuda.stream(streams[j]):
                B.prompt_attention(outs[j][i], q, k, v, starts[j], 1300, 0.1)
    torch.cuda.synchronize()
    for out, ref in zip(outs, refs):
        for x in out:
            check(x, *ref)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1.0, -0.7, 0.0])
def test_wide_scores(B, d, scale):
    """Scores of tens, whose maxima jump from block to block; a negative and a zero scale."""
    lens = [400, 130, 257]
    q, k, v, start = make(lens, 6, 2, d, False, seed=d)
    q, k = (q.float() * 0.6).to(torch.bfloat16), (k.float() * (30 / d) ** 0.5).to(torch.bfloat16)
    out = torch.empty_like(q)
    B.prompt_attention(out, q, k, v, start.cuda(), 400, scale)
    o, amp = reference(q, k, v, start, scale)
    check(out, o, amp, f"scale {scale}")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rising_maxima(B, d):
    """Keys that grow along the sequence: the reference max moves at many blocks."""
    n = 900
    q, k, v, start = make([n], 4, 1, d, False, seed=5)
    q = q.abs()
    k = (k.float().abs() * torch.linspace(0.1, 2.0, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    out = torch.empty_like(q)
    B.prompt_attention(out, q, k, v, start.cuda(), n, 0.3)
    o, amp = reference(q, k, v, start, 0.3)
    check(out, o, amp)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_do_not_leak(B, bad):
    """NaN and infinity in the rows of other sequences, of no sequence, and in the keys after
    a query stay out of a sequence's rows."""
    lens = [50, 140, 61]
    q, k, v, start = make(lens, 8, 2, 128, True, seed=9, lead=2, tail=3)
    a, z = int(start[1]), int(start[2])
    o, amp = reference(q, k, v, start, 0.1)
    for x in (q, k, v):
        x[:a] = bad
        x[z:] = bad
    k[a + 100:z] = bad  # seen by the last 40 queries alone
    out = torch.empty_like(q)
    B.prompt_attention(out, q, k, v, start.cuda(), 140, 0.1)
    check(out[a:a + 100], o[a:a + 100], amp[a:a + 100])


@pytest.mark.gpu
def test_strides_streams_and_graphs(B):
    """Strided outputs, a side stream, and a captured call replayed with other lengths."""
    hq, hkv, d = 6, 2, 64
    q, k, v, start = make([200, 120], hq, hkv, d, True, seed=3)
    big = torch.zeros(320, hq + 3, d, dtype=torch.bfloat16, device="cuda")
    out, dev = big[:, 1:1 + hq], start.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.prompt_attention(out, q, k, v, dev, 320, 0.125)
    s.synchronize()
    check(out, *reference(q, k, v, start, 0.125))
    assert bool((big[:, 0] == 0).all()) and bool((big[:, 1 + hq:] == 0).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.prompt_attention(out, q, k, v, dev, 320, 0.125)
    for cut in ([0, 1, 320], [0, 320, 320]):
        now = torch.tensor(cut, dtype=torch.int32)
        dev.copy_(now)
        g.replay()
        torch.cuda.synchronize()
        check(out, *reference(q, k, v, now, 0.125))


@pytest.mark.gpu
@pytest.mark.parametrize("seqs", [0, 3])
def test_nothing_to_do(B, seqs):
    q, k = (torch.zeros(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    start = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    B.prompt_attention(torch.empty_like(q), q, k, k, start, 5, 0.1)
    torch.cuda.synchronize()
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
def test_bad_starts_are_flagged(B):
    """Sequences that are too long, run backwards or leave the tensors are cut and flagged;
    the others are computed."""
    q, k, v, _ = make([300], 4, 2, 64, False, seed=1)
    good = torch.tensor([0, 100], dtype=torch.int32)
    o, amp = reference(q, k, v, good, 0.125)
    out = torch.zeros_like(q)
    for start, longest in (([0, 100, 400], 300), ([0, 100, 50], 300), ([0, 100, 300], 150),
                           ([-5, 100], 300)):
        B.pkv_device_errors()
        B.prompt_attention(out, q, k, v, torch.tensor(start, dtype=torch.int32).cuda(), longest, 0.125)
        assert B.pkv_device_errors() == 4
        check(out[:100], o[:100], amp[:100])


@pytest.mark.gpu
def test_same_rows_as_paged_prefill(B):
    """A prompt attended packed, then written into pages and attended there."""
    lens, hq, hkv, d, bs = [37, 200, 5], 8, 2, 64, 16
    q, k, v, start = make(lens, hq, hkv, d, False, seed=11)
    bm = B.BlockManager(64, bs)
    kc = torch.zeros(64, hkv, bs, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    for i in range(3):
        bm.add_sequence(i, 0)
    slots = torch.cat([bm.append_slots([i] * n) for i, n in enumerate(lens)])
    B.paged_kv_write(k, v, slots.cuda(), kc, vc)
    tables, ctx = bm.block_tables([0, 1, 2], 13)
    a, b = torch.empty_like(q), torch.empty_like(q)
    B.prompt_attention(a, q, k, v, start.cuda(), 200, 0.125)
    B.paged_prefill_attention(b, q, kc, vc, tables.cuda(), ctx.cuda(), 200, start.cuda(), 200, 0.125)
    o, amp = reference(q, k, v, start, 0.125)
    check(a, o, amp)
    check(b, o, amp)


def test_argument_errors(B):
    lib = B.lib()

    def call(out=FAKE, q=FAKE, start=FAKE, st=(512, 512, 128, 128), t=100, longest=50, n=2, hq=8,
             hkv=2, d=64):
        return lib.prompt_attention(out, q, FAKE, FAKE, *st, start, t, longest, n, hq, hkv, d, 0.1, None)

    assert call(d=96) == -3 and "head_dim" in B.pkv_last_error()
    assert call(hq=258, st=(1 << 15, 1 << 15, 128, 128)) == -3 and "group" in B.pkv_last_error()
    assert call(hq=7) == -2 and call(hkv=0) == -2 and call(n=-1) == -2 and call(t=-1) == -2
    assert call(longest=-1) == -2
    assert call(st=(512, 504, 128, 128)) == -2                 # shorter than a token
    assert call(st=(512, 516, 128, 128)) == -5                 # rows off the 16-byte grid
    assert call(st=(512, 1 << 39, 128, 128)) == -3
    assert call(t=1 << 31) == -3
    assert call(out=None) == -1 and call(start=None) == -1
    assert call(q=ctypes.c_void_p((1 << 20) + 8)) == -5
    assert call(start=ctypes.c_void_p((1 << 20) + 2)) == -5
    assert call(n=0) == 0 and call(t=0) == 0 and call(longest=0) == 0  # nothing to do


def test_binding_refusals(B):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    s = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.prompt_attention(x, x, x, x, s, 4, 0.1)
    with pytest.raises(TypeError, match="expected torch.bfloat16"):
        B.prompt_attention(x.float(), x, x, x, s, 4, 0.1)
    with pytest.raises(ValueError, match=r"\[T, heads, D\]"):
        B.prompt_attention(x, x, x[:3], x, s, 4, 0.1)
