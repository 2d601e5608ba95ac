"""The 8-bit cache's attention at the ends of its ranges.

Tolerances as in test_q8_attention.py: 2^-8 |out| + 2^-10 sum p |v|, and n 2^-35 of the largest |v|;
where a chunk may go either way, or its queries are aimed at single keys, chunk_ref's.
"""

import math

import pytest
import torch

import q8_ref as R
from test_q8_attention import check, decode, decode_ref, poison
from test_q8_cache import DEV, Batch, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    binding.pkv_device_errors(clear=True)
    return binding


def prefill(B, b, q, new, scale, **kw):
    out = torch.full_like(q, 77.0)
    B.paged_prefill_attention_q8(out, q, *b.cache(), b.bt, b.cl, max(b.lens), starts(new), max(new), scale, **kw)
    return out


def prefill_ref(b, q, new, scale):
    """As decode_ref, of each sequence's newest tokens."""
    out, mag = (torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    at = 0
    for s, (m, n) in enumerate(zip(b.lens, new)):
        if m and n:
            k, v = (R.values(c, sc, b.tables[s], 0, m, torch.float64) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
            seen = torch.arange(m, device=DEV)[None, :] <= torch.arange(m - n, m, device=DEV)[:, None]
            out[at:at + n], mag[at:at + n] = R.attention(q[at:at + n], k, v, scale, seen)
            top = b.vs[b.tables[s][:-(-m // b.bs)]].nan_to_num().amax(0).double() * R.TOP[b.dtype]
            mag[at:at + n] += m * 2.0 ** -25 * top.repeat_interleave(q.shape[1] // b.hkv)[:, None]
        at += n
    return out, mag


# Entries of one query in kernels of two tiles of rows: 8 heads a kv head and 3 or 5 drafts (entries of 2
# and 1), fewer drafts than the batch's most.
ONE_QUERY = [
    ([100, 37, 201], [3, 3, 3], 8, 1), ([77, 300], [5, 5], 16, 2), ([45, 131, 260], [1, 5, 4], 4, 2),
    ([333, 50, 1000], [1, 5, 4], 8, 2), ([129, 31, 5000, 7], [1, 1, 8, 7], 2, 2),
]


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,hq,hkv", ONE_QUERY)
def test_few_queries_of_any_scale(B, dtype, d, lens, new, hq, hkv):
    """A scale of 0, below 0, and one whose product with a row's power of two is 0."""
    b = Batch(lens, dtype, hkv, d, 16, seed=80)
    q = b.randn(sum(new), hq, d)
    for scale in (0.0, -0.125, 0.125):
        check(prefill(B, b, q, new, scale), *prefill_ref(b, q, new, scale), f"scale {scale}")
        check(decode(B, b, q[:len(lens)], scale), *decode_ref(b, q[:len(lens)], scale), f"decode, scale {scale}")
    q = torch.zeros_like(q)
    check(prefill(B, b, q, new, 1e-30), *prefill_ref(b, q, new, 1e-30), "queries of zeros")
    assert B.pkv_device_errors() == 0


def chunk_ref(b, q, new, scale, codes=False):
    """Output and bound of chunks.  Scores off by up to e_t move the output by at most sum p (exp(e) - 1)
    |v - out| / sum p exp(-e).

    Through fp16 rows, K's and V's codes and the weights are each off by 2^-11 of themselves at most, K and V
    by 2^-25 of their unit (the head's largest scale) where that is more, a weight by 2^-25 of 2^-7 of the
    largest; the scores' fp32 sums are an eighth of K's rounding.  Over the codes as they are, scores are D / 16
    fp32 sums and a few roundings, each of 2^-23 of sum |q| |k|, |k| being up to 255 scales in int8 (codes are
    taken as c + 128), and weights off by 2^-11 of themselves or by 2^-35 of the largest."""
    out, bound = (torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    at, g = 0, q.shape[1] // b.hkv
    for s, (m, n) in enumerate(zip(b.lens, new)):
        if m and n:
            pages = b.tables[s][:-(-m // b.bs)]
            ku, vu = (x[pages].nan_to_num().amax(0).double() for x in (b.ks, b.vs))
            k, v = (R.values(c, sc, b.tables[s], 0, m, torch.float64) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
            for lo in range(0, n, 64):
                rows = slice(at + lo, at + min(n, lo + 64))
                own = torch.arange(m - n + lo, m - n + min(n, lo + 64), device=DEV)
                unseen = torch.arange(m, device=DEV)[None, :] > own[:, None]
                for h in range(q.shape[1]):
                    x, kk, vv = q[rows, h].double(), k[:, h // g], v[:, h // g]
                    p = torch.softmax((x @ kk.T * scale).masked_fill(unseen, -math.inf), -1)
                    o, mag, large = p @ vv, p @ vv.abs(), x.abs().sum(1, keepdim=True)
                    if codes:
                        of = large * 255 * ku[h // g] if b.dtype is torch.int8 else x.abs() @ kk.abs().T
                        e, weights, least = (b.d // 16 + 4) * 2.0 ** -23 * of, 5 * 2.0 ** -13, m * 2.0 ** -35 * R.TOP[b.dtype]
                    else:
                        e = 9 * 2.0 ** -14 * (x.abs() @ kk.abs().T) + 2.0 ** -25 * ku[h // g] * large
                        weights, least = 5 * 2.0 ** -12, m * 2.0 ** -32 * R.TOP[b.dtype] + 2.0 ** -25
                    e = (e * abs(scale)).expand_as(p)
                    apart = (vv[None] - o[:, None]).abs_()
                    moved = torch.bmm((p * torch.expm1(e))[:, None], apart)[:, 0] / (p * torch.exp(-e)).sum(1, keepdim=True)
                    out[rows, h] = o
                    bound[rows, h] = 2.0 ** -8 * o.abs() + weights * mag + moved + least * vu[h // g]
        at += n
    return out, bound


def check_chunk(got, want, bound, what=""):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((got.double() - want).abs().max()):.3e}"


# The same values times a power of two.
RANGE = [([1], 2, 1), ([300, 129, 0, 17], 4, 2), ([20000, 31], 8, 1), ([100] * 40, 3, 3)]


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,hq,hkv", RANGE)
def test_values_near_the_ends_of_the_range(B, dtype, d, lens, hq, hkv):
    """V up to 1.7e38 and down to where the output is hardly a normal number, and pages of all the largest
    value that bf16 has: decode, drafts, chunks."""
    b = Batch(lens, dtype, hkv, d, 16, seed=81)
    q, scale = b.randn(len(lens), hq, d), 2 * d ** -0.5
    few, many = [min(n, 3) for n in lens], [min(n, 70) for n in lens]
    q3, q70 = b.randn(sum(few), hq, d), b.randn(sum(many), hq, d)
    plain = b.vs.clone()
    for e in (125, 118, -110):
        b.vs.copy_(plain * 2.0 ** e)
        check(decode(B, b, q, scale), *decode_ref(b, q, scale), f"decode, 2^{e}")
        check(prefill(B, b, q3, few, scale), *prefill_ref(b, q3, few, scale), f"drafts, 2^{e}")
        check_chunk(prefill(B, b, q70, many, scale), *chunk_ref(b, q70, many, scale), f"chunk, 2^{e}")
    largest = torch.finfo(torch.bfloat16).max
    R.bits(b.v)[:] = R.bits(torch.full((1,), R.TOP[dtype], device=DEV).to(dtype))[0]
    b.vs.fill_(largest / R.TOP[dtype])
    for out in (decode(B, b, q, scale)[b.cl > 0], prefill(B, b, q3, few, scale), prefill(B, b, q70, many, scale)):
        assert bool((out.double() >= largest * (1 - 2.0 ** -7)).all()) and bool(out.isfinite().all())
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_queries_near_the_end_of_the_range(B, dtype, d):
    """q up to 2^127 over keys as small, and the other way round: the scores are ordinary."""
    b = Batch([300, 1, 77], dtype, 2, d, 16, seed=82)
    q, new = b.randn(3, 16, d), [5, 1, 5]
    q5, plain = b.randn(11, 16, d), b.ks.clone()
    for e in (118, 110, -110, -118):
        k = 2.0 ** -e if e > 0 else 2.0 ** (-e - 3)
        b.ks.copy_(plain * k)
        qq, qq5 = ((x.float() * 2.0 ** e).to(torch.bfloat16) for x in (q, q5))
        scale = 0.1 if e > 0 else 0.8
        check(decode(B, b, qq, scale), *decode_ref(b, qq, scale), f"decode, 2^{e}")
        check(prefill(B, b, qq5, new, scale), *prefill_ref(b, qq5, new, scale), f"drafts, 2^{e}")
    # the largest exponents: q from 2^124 on, keys of 2^-124, one chosen by its sign
    b.ks.fill_(2.0 ** -125)
    R.bits(b.k)[:] = R.bits(torch.full((1,), 2.0, device=DEV).to(dtype))[0]
    for s, n in enumerate(b.lens):
        page, row = b.tables[s][(n // 2) // 16], (n // 2) % 16
        b.k[page, :, row] = b.k[page, :, row].float().neg().to(dtype)
    for sign in (1.0, -1.0):
        q1 = torch.zeros(3, 16, d, dtype=torch.bfloat16, device=DEV)
        q1[:, :, 3] = sign * 2.0 ** 127  # scores of 8 either way
        check(decode(B, b, q1, 1.0), *decode_ref(b, q1, 1.0), "decode, one value")
        check(prefill(B, b, q1, [1, 1, 1], 1.0), *prefill_ref(b, q1, [1, 1, 1], 1.0), "drafts, one value")
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
def test_drafts_over_room_for_long_contexts(B, dtype):
    """Tables and max_context_len for far longer contexts than the sequences have so far: a workspace that has no
    room for those, exactly as large as the call says, and none."""
    lens, new, hq, hkv, d, longest = [300, 17, 0, 129] * 16, [5, 3, 0, 1] * 16, 8, 8, 64, 1 << 22
    b = Batch(lens, dtype, hkv, d, 256, seed=85)
    wide = torch.full((len(lens), longest // 256), -1, dtype=torch.int32, device=DEV)
    wide[:, :b.bt.shape[1]] = b.bt
    q = b.randn(sum(new), hq, d)
    assert B.paged_prefill_q8_workspace_size(len(lens), hkv, d, 256, longest) == 0  # (2^31 rows of heads)
    size = B.paged_prefill_q8_workspace_size_for(sum(new), 5, len(lens), hq, hkv, d, longest)
    assert 0 < size < 32 << 20
    ws = torch.full((size + 4096,), 7, dtype=torch.uint8, device=DEV)
    want, mag = prefill_ref(b, q, new, 0.125)
    for kw in ({"workspace": ws[:size]}, {}):
        out = torch.full_like(q, 77.0)
        B.paged_prefill_attention_q8(out, q, *b.cache(), wide, b.cl, longest, starts(new), 5, 0.125, **kw)
        check(out, want, mag, str(list(kw)))
    assert bool((ws[size:] == 7).all())
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("new", [[90, 0, 130, 0], [0, 70, 0, 0]])
def test_sequences_without_queries_are_not_looked_at(B, dtype, new):
    """A chunk's call over a batch some of whose sequences have no queries, and tables that mean nothing:
    no flag, and nothing read back for them."""
    b = Batch([300, 250, 200, 40], dtype, 2, 64, 16, seed=86)
    q = b.randn(sum(new), 4, 64)
    want, bound = chunk_ref(b, q, new, 0.125)
    bt, cl = b.bt.clone(), b.cl.clone()
    for s, n in enumerate(new):
        if n == 0:
            bt[s], cl[s] = b.nb + 1000, 288 if s < 3 else 0
    size = B.paged_prefill_q8_workspace_size_for(sum(new), max(new), 4, 4, 2, 64, 300)
    ws = torch.full((size,), 7, dtype=torch.uint8, device=DEV)
    out = torch.full_like(q, 77.0)
    B.paged_prefill_attention_q8(out, q, *b.cache(), bt, cl, 300, starts(new), max(new), 0.125, workspace=ws)
    check_chunk(out, want, bound)
    assert B.pkv_device_errors() == 0
    rows = ws[:4 * 300 * 2 * 64 * 2].view(4, -1)  # K's, of each sequence
    for s, n in enumerate(new):
        assert bool((rows[s] == 7).all()) == (n == 0), f"sequence {s}"


AIMS = [
    # context lengths, new tokens, q heads, kv heads, block size: drafts, then chunks
    ([700, 30, 5000, 131], [5, 5, 5, 3], 8, 2, 16), ([9000, 257], [31, 8], 3, 1, 32), ([2, 129, 300], [2, 1, 8], 16, 2, 8),
    ([700, 130, 3000], [150, 130, 300], 6, 2, 16), ([1000, 256, 1], [129, 256, 1], 8, 1, 256),
]


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,hq,hkv,bs", AIMS)
def test_chunks_aimed_at_single_keys(B, dtype, d, lens, new, hq, hkv, bs):
    """Every query aimed at one key, whose value is then the output: its own, the one before, those at the
    borders of pages and of blocks of 128, any; and at the next one and the last, which it must not see."""
    b = Batch(lens, dtype, hkv, d, bs, seed=83)
    gen = torch.Generator().manual_seed(84)
    own = torch.cat([torch.arange(m - n, m) for m, n in zip(lens, new)])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(new)])
    last = torch.tensor(lens)[seq] - 1
    k = [R.values(b.k, b.ks, b.tables[s], 0, m) for s, m in enumerate(lens)]
    v = [R.values(b.v, b.vs, b.tables[s], 0, m, torch.float64) for s, m in enumerate(lens)]
    aims = [("own", own), ("before", own - 1), ("next", own + 1), ("last", last)]
    aims += [(f"key {t}", torch.full_like(own, t)) for t in (0, bs - 1, bs, 127, 128)]
    aims += [("back 128", own - 128), ("back to a block", own // 128 * 128)]
    aims += [("any", (torch.rand(len(own), generator=gen) * (own + 1)).long()) for _ in range(4)]
    for what, at in aims:
        at = torch.minimum(at.clamp(min=0), last)
        aim = torch.stack([k[s][t] for s, t in zip(seq.tolist(), at.tolist())])
        aimed = torch.stack([v[s][t] for s, t in zip(seq.tolist(), at.tolist())])
        q = (aim * 6.0).repeat_interleave(hq // hkv, 1).to(torch.bfloat16)
        out = prefill(B, b, q, new, 1.0)
        want, bound = chunk_ref(b, q, new, 1.0, codes=max(new) <= 32)  # few queries are rows of the decode kernel
        check_chunk(out, want, bound, what)
        off = (want - aimed.repeat_interleave(hq // hkv, 1)).abs().amax((1, 2))
        seen = (at <= own).to(DEV)
        assert bool((off[seen] < 0.05).all()) and bool((off[~seen] > 0.5).all())  # a lost or an extra key would show
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("lens,new,hq,hkv,d,bs", [
    ([300, 90, 0, 555, 128, 40, 200], [130, 1, 0, 300, 0, 40, 77], 4, 2, 64, 16), ([1000, 129], [100, 129], 3, 1, 128, 32),
])
def test_chunks_in_groups_of_sequences(B, dtype, lens, new, hq, hkv, d, bs):
    """Workspaces for all sequences and for ever fewer, down to one: the same bits, and nothing behind them."""
    b = Batch(lens, dtype, hkv, d, bs, seed=87)
    poison(b)
    q = b.randn(sum(new) + 3, hq, d)
    full = B.paged_prefill_q8_workspace_size_for(sum(new) + 3, max(new), len(lens), hq, hkv, d, max(lens))
    one = B.paged_prefill_q8_workspace_size_for(max(new), max(new), 1, hq, hkv, d, max(lens))
    assert full >= len(lens) * (one - 4096)
    want, bound = chunk_ref(b, q[:sum(new)], new, 0.125)
    first = None
    for size in [full] + [one * n for n in range(len(lens), 0, -1)]:
        ws = torch.full((size + 4096,), 0xff, dtype=torch.uint8, device=DEV)
        out = prefill(B, b, q, new, 0.125, workspace=ws[:size])
        if first is None:
            first = out
            check_chunk(out[:sum(new)], want, bound)
        assert torch.equal(out, first), f"{size} of {full} bytes"
        assert bool((ws[size:] == 0xff).all()) and bool((out[sum(new):] == 77).all())
    assert B.pkv_device_errors() == 0
    # sequences whose rows overlap are cut and flagged, in whatever group
    start = starts(new)
    start[2] = 0
    first = None
    for size in (full, 2 * one, one):
        out = torch.full_like(q, 77.0)
        B.paged_prefill_attention_q8(out, q, *b.cache(), b.bt, b.cl, max(lens), start, sum(new), 0.125,
                                     workspace=torch.empty(max(size, one), dtype=torch.uint8, device=DEV))
        assert B.pkv_device_errors() == 4 and bool(out[:sum(new)].isfinite().all())
        first = out if first is None else first
        assert torch.equal(out, first)
    with pytest.raises(B.PkvError, match="workspace"):
        prefill(B, b, q, new, 0.125, workspace=torch.empty(one - 1, dtype=torch.uint8, device=DEV))
