"""Attention over the 8-bit cache against fp64 on the same codes.

Tolerance: the output's rounding to bf16 is at most 2^-8 of it; a weight's rounding to fp16 at most
2^-11 of the weight, so 2^-11 of sum p |v|; the scores' fp32 sums (at most 128 exact products and
a few roundings of 2^-24 each, on scores up to some tens) and the exponential move each weight by
less than 2^-12.  Together 2^-8 |out| + 2^-10 sum p |v|.  A small weight has an absolute step
instead: weights are held in fp16, the largest of them (times its page's V scale over the largest) at
2^10 or more, and fp16's steps below 2^-14 are 2^-24, so off by 2^-25 2^-10 = 2^-35 of the largest |v|
of the context's codes, for each key.
"""

import math

import pytest
import torch

import q8_ref as R
from test_q8_cache import DEV, Batch, same, starts

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


def poison(b):
    """NaN in all that no sequence owns: other pages' scales, and (e4m3) rows past the contexts."""
    owned = {p for t in b.tables for p in t if p >= 0}
    for p in range(b.nb):
        if p not in owned:
            b.ks[p] = b.vs[p] = math.nan
    fill = 0x7f if b.dtype is torch.float8_e4m3fn else 0x80
    for s, n in enumerate(b.lens):
        if n % b.bs:
            for codes in (b.k, b.v):
                R.bits(codes)[b.tables[s][n // b.bs], :, n % b.bs:] = fill


def check(got, want, mag, what=""):
    err = (got.double() - want).abs()
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {err.max():.3e}"


def decode_ref(b, q, scale):
    out, mag = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for s, n in enumerate(b.lens):
        k, v = (R.values(c, sc, b.tables[s], 0, n, torch.float64) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
        o, m = R.attention(q[s:s + 1], k, v, scale)
        out[s:s + 1], mag[s:s + 1] = o, m
        if n:  # 2^-10 of this is n 2^-35 of the largest |v| that the head's scales can hold
            top = b.vs[b.tables[s][:-(-n // b.bs)]].nan_to_num().amax(0).double() * R.TOP[b.dtype]
            mag[s] += n * 2.0 ** -25 * top.repeat_interleave(q.shape[1] // b.hkv)[:, None]
    return out, mag


def decode(B, b, q, scale, **kw):
    out = torch.full_like(q, 77.0)
    B.paged_decode_attention_q8(out, q, *b.cache(), b.bt, b.cl, max(max(b.lens), 1), scale, **kw)
    return out


DECODE = [
    # lens, q heads, kv heads, head_dim, block size
    ([1], 1, 1, 64, 8),
    ([128], 32, 8, 64, 16),
    ([127, 128, 129, 0, 1, 255, 256, 257], 6, 2, 128, 16),
    ([15, 16, 17, 31, 32, 33, 8, 9], 8, 1, 64, 8),
    ([0, 0, 0], 4, 2, 64, 16),
    ([700, 1, 2048, 0, 333], 14, 2, 128, 32),
    ([3000], 8, 8, 64, 64),
    ([5000, 4100, 300], 24, 8, 128, 16),
    ([1000, 513], 10, 2, 128, 256),
    ([777, 130], 3, 1, 64, 128),
    ([100] * 200, 4, 4, 64, 16),
    (list(range(0, 600, 2)), 6, 2, 64, 16),
]


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("lens,hq,hkv,d,bs", DECODE)
def test_decode(B, dtype, lens, hq, hkv, d, bs):
    b = Batch(lens, dtype, hkv, d, bs, seed=20)
    poison(b)
    q = b.randn(len(lens), hq, d)
    out = decode(B, b, q, d ** -0.5)
    check(out, *decode_ref(b, q, d ** -0.5))
    assert B.pkv_device_errors() == 0
    assert torch.equal(out, decode(B, b, q, d ** -0.5))  # the same bits every time


@pytest.mark.parametrize("dtype,hq,hkv,d,bs,n", [
    (torch.int8, 1, 1, 64, 16, 120000), (torch.float8_e4m3fn, 8, 1, 128, 32, 100003),
    (torch.int8, 4, 2, 128, 64, 40001),
])
def test_one_long_context(B, dtype, hq, hkv, d, bs, n):
    """One context over every CTA of the GPU; a key that draws the query sits in each region."""
    b = Batch([n], dtype, hkv, d, bs, seed=21)
    poison(b)
    q = b.randn(1, hq, d)
    check(decode(B, b, q, d ** -0.5), *decode_ref(b, q, d ** -0.5))
    # a query aimed at one key: the output is that key's value, wherever it lies
    for t in (0, 1, 127, 128, n // 3, n // 2 + 5, n - 129, n - 2, n - 1):
        k = R.values(b.k, b.ks, b.tables[0], t, t + 1)[0]  # [Hkv, D]
        aim = (k * 6.0).repeat_interleave(hq // hkv, 0)[None].to(torch.bfloat16)
        want, mag = decode_ref(b, aim, 1.0)
        check(decode(B, b, aim, 1.0), want, mag, f"key {t}")
        v = R.values(b.v, b.vs, b.tables[0], t, t + 1, torch.float64)[0].repeat_interleave(hq // hkv, 0)
        assert float((want[0] - v).abs().max()) < 1e-3  # the aim is good: a lost key would show
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype,d,share,cut", [
    (torch.int8, 64, 10, 329), (torch.float8_e4m3fn, 64, 10, 489), (torch.int8, 128, 10, 325),
])
def test_a_share_of_two_long_contexts(B, dtype, d, share, cut):
    """The first context (of 33 or 49 shares) ends in the share that the second begins in."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    groups = 3 if d == 64 else 2
    lens = [(cut - 1) * 128, (share * groups * sms - cut - 1) * 128]
    b = Batch(lens, dtype, 1, d, 128, seed=30)
    q = b.randn(2, 1, d)
    ws = torch.zeros(B.paged_decode_q8_workspace_size(2, 1, 1, d, max(lens)), dtype=torch.uint8, device=DEV)
    outs = [decode(B, b, q, 2 * d ** -0.5, workspace=ws) for _ in range(40)]
    check(outs[0], *decode_ref(b, q, 2 * d ** -0.5))
    for o in outs[1:]:
        same(o, outs[0], "the same bits every time")
    assert not ws[:8192].any()
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_scales_far_apart(B, dtype, d):
    """Pages whose V scales differ by up to 2^40, and K scales by 2^6."""
    b = Batch([400, 400, 37], dtype, 2, d, 16, seed=22)
    gen = torch.Generator().manual_seed(23)
    b.vs *= torch.exp2(torch.randint(-20, 21, b.vs.shape, generator=gen).float()).to(DEV)
    b.ks *= torch.exp2(torch.randint(-5, 2, b.ks.shape, generator=gen).float()).to(DEV)
    b.vs[b.tables[1][3]] = 0.0
    b.ks[b.tables[1][4]] = 0.0
    q = b.randn(3, 8, d)
    check(decode(B, b, q, d ** -0.5), *decode_ref(b, q, d ** -0.5))


@pytest.mark.parametrize("dtype", R.KINDS)
def test_queries_of_any_size(B, dtype):
    """Rows of q between 2^-100 and 2^100 (the scale undoes them), with small values beside large."""
    b = Batch([200] * 6, dtype, 1, 128, 16, seed=24)
    q = b.randn(6, 2, 128)
    base, mag = decode_ref(b, q, 128 ** -0.5)
    for e in (-100, -30, 30, 100):
        qq = (q.float() * 2.0 ** e).to(torch.bfloat16)
        got = decode(B, b, qq, 128 ** -0.5 * 2.0 ** -e)
        check(got, base, mag, f"2^{e}")
    q[0] = 0
    q[1, 0, :] = 0
    q[1, 0, 7] = 2.0 ** -130  # not a normal number
    check(decode(B, b, q, 128 ** -0.5), *decode_ref(b, q, 128 ** -0.5), "zeros")


def test_long_tails_keep_their_weight(B):
    """One key with a large score and 30000 equal ones far below it: their sum still counts."""
    for dtype in R.KINDS:
        b = Batch([30001], dtype, 1, 64, 16, seed=25)
        R.bits(b.k).zero_()
        b.k[b.tables[0][0], 0, 0, 0] = 100
        b.ks.fill_(1.0)
        b.vs.fill_(0.01)
        R.bits(b.v)[:] = R.bits(torch.full((1,), 64.0, device=DEV).to(dtype))[0]
        b.v[b.tables[0][0], 0, 0] = -64.0 if dtype is not torch.int8 else -64
        q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=DEV)
        q[0, 0, 0] = 1.0
        for gap in (2.0, 8.0, 12.0, 14.0):  # in powers of e
            want, mag = decode_ref(b, q, gap / 100)
            check(decode(B, b, q, gap / 100), want, mag, f"gap {gap}")


@pytest.mark.parametrize("dtype", R.KINDS)
def test_not_finite(B, dtype):
    """A page of scale NaN makes its (sequence, kv head) NaN and nothing else; a query's NaN its row."""
    b = Batch([300, 40, 2000], dtype, 2, 64, 16, seed=26)
    q = b.randn(3, 4, 64)
    want, mag = decode_ref(b, q, 0.125)
    b.vs[b.tables[0][18], 1] = math.nan
    b.ks[b.tables[2][100], 0] = math.nan
    q[1, 2, 9] = math.nan
    out = decode(B, b, q, 0.125)
    nan = torch.zeros(3, 4, dtype=torch.bool)
    nan[0, 2:] = nan[2, :2] = nan[1, 2] = True
    assert torch.equal(out.isnan().all(-1).cpu(), nan) and torch.equal(out.isnan().any(-1).cpu(), nan)
    keep = ~nan.to(DEV)
    check(out[keep], want[keep], mag[keep])
    if dtype is torch.float8_e4m3fn:  # a NaN code within the context
        b = Batch([300, 300], dtype, 2, 64, 16, seed=27)
        R.bits(b.v)[b.tables[1][5], 0, 3, 11] = 0x7f
        q = b.randn(2, 4, 64)
        out = decode(B, b, q, 0.125)
        nan = torch.zeros(2, 4, 64, dtype=torch.bool, device=DEV)
        nan[1, :2, 11] = True
        assert torch.equal(out.isnan(), nan)


def test_bad_values_are_flagged(B):
    b = Batch([100, 100, 100], torch.int8, 1, 64, 16, seed=28)
    q = b.randn(3, 2, 64)
    want, mag = decode_ref(b, q, 0.125)
    b.cl[0] = -5
    b.cl[2] = 1 << 30
    out = torch.empty_like(q)
    B.paged_decode_attention_q8(out, q, *b.cache(), b.bt, b.cl, 100, 0.125)
    assert B.pkv_device_errors() == 4
    assert bool((out[0] == 0).all())
    check(out[1:], want[1:], mag[1:])  # the third's length is cut to max_context_len
    b.cl[:] = 100
    b.bt[1, 2] = b.nb + 7
    b.bt[1, 3] = -2
    B.paged_decode_attention_q8(out, q, *b.cache(), b.bt, b.cl, 100, 0.125)
    assert B.pkv_device_errors() == 1
    check(out[::2], want[::2], mag[::2])
    assert bool(out.isfinite().all())


def test_one_workspace_for_calls_of_any_sizes(B):
    batches = [Batch([5000, 10], torch.int8, 2, 64, 16, seed=30), Batch([300] * 100, torch.float8_e4m3fn, 4, 128, 16, seed=31),
               Batch([1], torch.int8, 1, 64, 8, seed=32), Batch([20000], torch.float8_e4m3fn, 1, 128, 32, seed=33)]
    need = max(B.paged_decode_q8_workspace_size(len(b.lens), 2 * b.hkv, b.hkv, b.d, max(b.lens)) for b in batches)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for b in batches:
            q = b.randn(len(b.lens), 2 * b.hkv, b.d)
            check(decode(B, b, q, 0.1, workspace=ws), *decode_ref(b, q, 0.1))
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("d,hq,hkv,bs", [(64, 8, 2, 16), (128, 3, 3, 32)])
def test_steps(B, dtype, d, hq, hkv, bs):
    """Steps of a batch, as a model's layer runs them: the write, then attention over what it wrote."""
    lens = [0, 15, 16, 200, 1300]
    b = Batch([n + 20 for n in lens], dtype, hkv, d, bs, seed=40)
    want_cache = b.copies()
    ws = torch.zeros(B.paged_decode_q8_workspace_size(5, hq, hkv, d, 1400), dtype=torch.uint8, device=DEV)
    for step in range(20):
        b.lens = [n + step + 1 for n in lens]
        b.cl = torch.tensor(b.lens, dtype=torch.int32, device=DEV)
        x = b.randn(5, hq + 2 * hkv, d)
        q, k, v = x[:, :hq].contiguous(), x[:, hq:hq + hkv], x[:, hq + hkv:]
        out = torch.empty_like(q)
        B.paged_decode_step_q8(out, q, k, v, *b.cache(), b.bt, b.cl, max(b.lens), d ** -0.5, workspace=ws)
        for s, n in enumerate(b.lens):
            R.write(want_cache[0], want_cache[2], k[s:s + 1], b.tables[s], n - 1)
            R.write(want_cache[1], want_cache[3], v[s:s + 1], b.tables[s], n - 1)
        for got, w, what in zip(b.cache(), want_cache, ("k codes", "v codes", "k scales", "v scales")):
            same(got, w, f"{what}, step {step}")
        check(out, *decode_ref(b, q, d ** -0.5), f"step {step}")
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("neox", [True, False])
def test_rotary_steps(B, neox):
    dtype, d, hq, hkv, bs, r = torch.float8_e4m3fn, 128, 6, 2, 16, 64
    lens = [30, 700, 0]
    b = Batch([n + 6 for n in lens], dtype, hkv, d, bs, seed=41)
    ang = torch.arange(800, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    table = torch.cat((ang.cos(), ang.sin()), 1).float().to(DEV)
    want_cache = b.copies()
    for step in range(6):
        b.lens = [n + step + 1 for n in lens]
        b.cl = torch.tensor(b.lens, dtype=torch.int32, device=DEV)
        pos = torch.tensor([n - 1 for n in b.lens], device=DEV)
        x = b.randn(3, hq + 2 * hkv, d)
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        wq, wk = R.rotate(q, table, pos, r, neox), R.rotate(k, table, pos, r, neox)
        out, q_out = (torch.empty(3, hq, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        B.paged_decode_step_rope_q8(out, q, k, v, table, *b.cache(), b.bt, b.cl, max(b.lens), d ** -0.5,
                                    q_out=q_out, rotary_dim=r, neox_style=neox)
        for s, n in enumerate(b.lens):
            R.write(want_cache[0], want_cache[2], wk[s:s + 1], b.tables[s], n - 1)
            R.write(want_cache[1], want_cache[3], v[s:s + 1], b.tables[s], n - 1)
        for got, w in zip(b.cache(), want_cache):
            same(got, w, "cache")
        assert torch.equal(q_out, wq)
        check(out, *decode_ref(b, wq, d ** -0.5))
    assert B.pkv_device_errors() == 0


def check_prefill(got, q, k, want, mag, scale):
    """K, V and the weights are fp16 here, each off by 2^-11 of itself at most (values below 2^-14 of
    the largest scale's unit by 2^-25 of it): the weights' and V's are 2^-10 sum p |v| together, K's
    move a score by 2^-11 sum |q k| scale, and so a normalised weight by twice that of itself."""
    if not k.shape[0]:
        return
    g = q.shape[1] // k.shape[1]
    top = max(float((q[:, h].double().abs() @ k[:, h // g].abs().T).max()) for h in range(q.shape[1])) * abs(scale)
    err = (got.double() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -10 * top) * mag + 2.0 ** -24 * mag.max()).all()), float(err.max())


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("lens,new,hq,hkv,d,bs", [
    ([100, 37, 0, 300], [5, 1, 0, 300], 4, 2, 64, 16), ([1000, 700], [130, 257], 6, 2, 128, 32),
    ([50], [50], 8, 1, 128, 8), ([600, 256], [3, 256], 3, 3, 64, 256),
    ([1], [1], 1, 1, 64, 8), ([129, 128, 127, 257], [1, 128, 2, 129], 5, 1, 128, 16),
    ([3000], [700], 4, 4, 64, 64), ([2000] * 20, [64] * 20, 8, 2, 128, 16),
    ([700, 30, 5000, 6], [5, 5, 5, 5], 8, 2, 64, 16), ([9000], [32], 3, 1, 128, 32), ([300] * 50, [1, 2, 3, 4, 5] * 10, 4, 4, 128, 8),
])
def test_prefill(B, dtype, lens, new, hq, hkv, d, bs):
    b = Batch(lens, dtype, hkv, d, bs, seed=50)
    poison(b)
    t = sum(new)
    q = b.randn(t, hq, d)
    out = torch.full_like(q, 77.0)
    ws = torch.full((B.paged_prefill_q8_workspace_size(len(lens), hkv, d, bs, max(lens)),), 0xff, dtype=torch.uint8,
                    device=DEV)  # bf16 NaN all over
    B.paged_prefill_attention_q8(out, q, *b.cache(), b.bt, b.cl, max(lens), starts(new), max(new), d ** -0.5,
                                 workspace=ws)
    at = 0
    for s, (m, n) in enumerate(zip(lens, new)):
        k, v = (R.values(c, sc, b.tables[s], 0, m, torch.float64) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
        seen = torch.arange(m, device=DEV)[None, :] <= torch.arange(m - n, m, device=DEV)[:, None]
        want, mag = R.attention(q[at:at + n], k, v, d ** -0.5, seen)
        check_prefill(out[at:at + n], q[at:at + n], k, want, mag, d ** -0.5)
        at += n
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (6, 2), (4, 1), (10, 2), (7, 1), (8, 1)])
@pytest.mark.parametrize("lens,new", [
    ([2, 9, 131, 0, 257, 5000, 128, 40], [2, 9, 7, 0, 8, 6, 1, 3]),       # a page's and a chunk's border between queries
    ([130, 300, 16, 9000], [17, 32, 16, 31]),
    ([260] * 40, [3, 4] * 20),
])
def test_few_queries(B, dtype, d, hq, hkv, lens, new):
    """Entries of 1 to 16 rows, whole and in part filled, whose queries end in different chunks."""
    test_prefill(B, dtype, lens, new, hq, hkv, d, 16)


@pytest.mark.parametrize("new", [[4, 5], [150, 170]])  # as rows of the decode, and on the tiles
def test_prefill_of_hard_values(B, new):
    """Queries of any size, a scale below 0, pages of scales far apart and of zeros."""
    for dtype in R.KINDS:
        b = Batch([300, 200], dtype, 2, 64, 16, seed=51)
        gen = torch.Generator().manual_seed(52)
        b.vs *= torch.exp2(torch.randint(-6, 7, b.vs.shape, generator=gen).float()).to(DEV)
        b.ks *= torch.exp2(torch.randint(-3, 2, b.ks.shape, generator=gen).float()).to(DEV)
        b.ks[b.tables[0][2]] = b.vs[b.tables[0][3]] = 0.0
        b.ks[b.tables[1]] = 0.0  # all of a context's keys are zeros
        poison(b)
        base = b.randn(sum(new), 4, 64)
        for e, scale in ((0, 0.125), (0, -0.125), (60, 0.125 * 2.0 ** -60), (-90, 0.125 * 2.0 ** 90)):
            q = (base.float() * 2.0 ** e).to(torch.bfloat16)
            out = torch.empty_like(q)
            B.paged_prefill_attention_q8(out, q, *b.cache(), b.bt, b.cl, 300, starts(new), max(new), scale)
            for s, (lo, hi) in enumerate(((0, new[0]), (new[0], sum(new)))):
                m, n = b.lens[s], hi - lo
                k, v = (R.values(c, sc, b.tables[s], 0, m, torch.float64) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
                seen = torch.arange(m, device=DEV)[None, :] <= torch.arange(m - n, m, device=DEV)[:, None]
                want, mag = R.attention(q[lo:hi], k, v, scale, seen)
                check_prefill(out[lo:hi], q[lo:hi], k, want, mag, scale)
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("new", [20, 220])  # as rows of the decode, and on the tiles
def test_prefill_not_finite(B, dtype, new):
    """A page of scale NaN makes the queries NaN that see it and no others; a query's NaN its row."""
    lens, bs = [300, 250, 900], 16
    b = Batch(lens, dtype, 2, 64, bs, seed=53)
    q = b.randn(3 * new, 4, 64)
    start = starts([new] * 3)
    marks = [(0, b.vs, 1, lens[0] - 9), (1, b.ks, 0, lens[1] - 17), (2, b.vs, 0, 40)]  # sequence, scales, kv head, key
    nan = torch.zeros(3 * new, 4, dtype=torch.bool)
    for s, scales, g, key in marks:
        page = key // bs
        scales[b.tables[s][page], g] = math.nan
        if dtype is torch.float8_e4m3fn:  # as the write leaves it
            R.bits(b.v if scales is b.vs else b.k)[b.tables[s][page], g, 3:] = 0x7f
        first = max(page * bs - (lens[s] - new), 0)  # the query at the page's first token sees it
        nan[s * new + first:(s + 1) * new, 2 * g:2 * g + 2] = True
    q[2 * new + 5, 3, 9] = math.nan
    nan[2 * new + 5, 3] = True
    out = torch.full_like(q, 77.0)
    B.paged_prefill_attention_q8(out, q, *b.cache(), b.bt, b.cl, max(lens), start, new, 0.125)
    assert torch.equal(out.isnan().all(-1).cpu(), nan) and torch.equal(out.isnan().any(-1).cpu(), nan)
    for s, n in enumerate(lens):
        k, v = (R.values(c, sc, b.tables[s], 0, n, torch.float64).nan_to_num(0.0) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
        rows = slice(s * new, (s + 1) * new)
        seen = torch.arange(n, device=DEV)[None, :] <= torch.arange(n - new, n, device=DEV)[:, None]
        want, mag = R.attention(q[rows].nan_to_num(0.0), k, v, 0.125, seen)
        keep = ~nan[rows].to(DEV)
        top = max(float((q[rows, h].double().nan_to_num(0.0).abs() @ k[:, h // 2].abs().T).max()) for h in range(4)) * 0.125
        err = (out[rows].double() - want).abs()[keep]  # as check_prefill
        assert bool((err <= (2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -10 * top) * mag)[keep] + 2.0 ** -24 * mag.max()).all())
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("n", [4, 40])
def test_prefill_lengths_that_do_not_fit(B, n):
    b = Batch([100, 100, 100], torch.int8, 1, 64, 16, seed=53)
    q = b.randn(3 * n, 2, 64)
    b.cl[0] = 2          # of n queries, all but two lie before the first token
    b.cl[2] = 1 << 30    # cut to max_context_len
    out = torch.full((3 * n + 2, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    B.paged_prefill_attention_q8(out[:3 * n], q, *b.cache(), b.bt, b.cl, 100, starts([n, n, n]), n, 0.125)
    assert B.pkv_device_errors() == 4
    assert bool((out[:n - 2] == 0).all()) and bool((out[3 * n:] == 9).all())
    for s, (lo, m) in enumerate(((n - 2, 2), (n, 100), (2 * n, 100))):
        k, v = (R.values(c, sc, b.tables[s], 0, m, torch.float64) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
        x = (s + 1) * n - lo
        seen = torch.arange(m, device=DEV)[None, :] <= torch.arange(m - x, m, device=DEV)[:, None]
        want, mag = R.attention(q[lo:lo + x], k, v, 0.125, seen)
        check_prefill(out[lo:lo + x], q[lo:lo + x], k, want, mag, 0.125)


def test_prefill_leaves_rows_of_no_sequence(B):
    """Rows between and behind the sequences', empty contexts among them, both ways."""
    for n in (3, 60):
        b = Batch([200, 0, 90], torch.float8_e4m3fn, 2, 128, 16, seed=54)
        q = b.randn(2 * n + 7, 4, 128)
        out = torch.full_like(q, 5.0)
        st = torch.tensor([2, 2 + n, 2 + n, 2 + 2 * n], dtype=torch.int32, device=DEV)
        B.paged_prefill_attention_q8(out, q, *b.cache(), b.bt, b.cl, 200, st, n, 0.1)
        assert bool((out[:2] == 5).all()) and bool((out[2 + 2 * n:] == 5).all())
        for s, (lo, m) in enumerate(((2, 200), (0, 0), (2 + n, 90))):
            if m:
                k, v = (R.values(c, sc, b.tables[s], 0, m, torch.float64) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
                seen = torch.arange(m, device=DEV)[None, :] <= torch.arange(m - n, m, device=DEV)[:, None]
                want, mag = R.attention(q[lo:lo + n], k, v, 0.1, seen)
                check_prefill(out[lo:lo + n], q[lo:lo + n], k, want, mag, 0.1)
        assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("seqs,rows", [(1, 3000), (3, 97)])
def test_prefill_of_a_padded_batch(B, seqs, rows):
    """More packed rows than the sequences could have: the others stay, and so does what lies behind the
    workspace."""
    lens, hq, hkv, d = [40, 9, 300][:seqs], 2, 1, 64
    b = Batch(lens, torch.int8, hkv, d, 16, seed=31)
    q = b.randn(rows, hq, d)
    start = starts([4] * seqs)
    size = B.paged_prefill_q8_workspace_size(seqs, hkv, d, 16, max(lens))
    ws = torch.full((size + (1 << 16),), 7, dtype=torch.uint8, device=DEV)
    out = torch.full_like(q, 77.0)
    B.paged_prefill_attention_q8(out, q, *b.cache(), b.bt, b.cl, max(lens), start, 4, d ** -0.5, workspace=ws[:size])
    assert (out[4 * seqs:] == 77).all() and (ws[size:] == 7).all()
    for s, n in enumerate(lens):
        k, v = (R.values(c, sc, b.tables[s], 0, n, torch.float64) for c, sc in ((b.k, b.ks), (b.v, b.vs)))
        for i in range(4):
            at = n - 3 + i
            want, mag = R.attention(q[4 * s + i:4 * s + i + 1], k[:at], v[:at], d ** -0.5)
            check(out[4 * s + i:4 * s + i + 1], want, mag, f"sequence {s}, query {i}")
    assert B.pkv_device_errors() == 0


def test_streams_and_graphs(B):
    """A step captured once and replayed on other inputs; another stream with a workspace of its own."""
    dtype, d, hq, hkv = torch.int8, 64, 8, 2
    b = Batch([200, 900], dtype, hkv, d, 16, seed=60)
    ws = torch.zeros(B.paged_decode_q8_workspace_size(2, hq, hkv, d, 900), dtype=torch.uint8, device=DEV)
    q, k, v = b.randn(2, hq, d), b.randn(2, hkv, d), b.randn(2, hkv, d)
    out = torch.empty_like(q)

    def step():
        B.paged_decode_step_q8(out, q, k, v, *b.cache(), b.bt, b.cl, 900, 0.125, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    side = torch.cuda.Stream()
    b2 = Batch([3000, 64], torch.float8_e4m3fn, hkv, 128, 16, seed=61)
    q2 = b2.randn(2, hq, 128)
    want2 = decode_ref(b2, q2, 0.1)
    for i in range(5):
        for t, s in ((q, 1.0), (k, 1.0 + i), (v, 2.0)):
            t.copy_(b.randn(*t.shape) * s)
        before = b.copies()
        torch.cuda.synchronize()
        g.replay()
        out2 = torch.empty_like(q2)
        with torch.cuda.stream(side):
            pass
        B.paged_decode_attention_q8(out2, q2, *b2.cache(), b2.bt, b2.cl, 3000, 0.1, stream=side)
        torch.cuda.synchronize()
        for s, n in enumerate(b.lens):
            R.write(before[0], before[2], k[s:s + 1], b.tables[s], n - 1)
            R.write(before[1], before[3], v[s:s + 1], b.tables[s], n - 1)
        for got, w in zip(b.cache(), before):
            same(got, w, "cache")
        check(out, *decode_ref(b, q, 0.125), f"replay {i}")
        check(out2, *want2, "side stream")
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("k_at,v_at", [(0, 1 << 20), (1 << 20, 0), (0, (1 << 20) + 16), ((1 << 20) + 48, 0), (0, 0)])
@pytest.mark.parametrize("dtype,d", [(torch.int8, 64), (torch.float8_e4m3fn, 128)])
def test_pools_anywhere_in_memory(B, dtype, d, k_at, v_at):
    """V's pool behind K's, before it, not a whole number of 128-byte rows away, and K's itself."""
    b = Batch([130, 1, 300], dtype, 2, d, 16, seed=62)
    room = torch.zeros((1 << 20) + 64 + b.k.numel(), dtype=torch.uint8, device=DEV)
    assert b.k.numel() <= 1 << 20
    old = (b.k, b.v)
    b.k, b.v = (room[at:at + x.numel()].view(x.dtype).view(x.shape) for x, at in zip(old, (k_at, v_at)))
    R.bits(b.k).copy_(R.bits(old[0]))
    if k_at != v_at:
        R.bits(b.v).copy_(R.bits(old[1]))
    q = b.randn(3, 6, d)
    check(decode(B, b, q, 0.1), *decode_ref(b, q, 0.1))
    assert B.pkv_device_errors() == 0


def test_many_sequences(B):
    """More sequences than the GPU has threads in a CTA's scan, some empty, some long."""
    gen = torch.Generator().manual_seed(63)
    lens = [0 if x < 0.2 else (200 if x > 0.98 else int(1 + 40 * x)) for x in torch.rand(7000, generator=gen).tolist()]
    b = Batch(lens, torch.int8, 1, 64, 8, seed=64)
    q = b.randn(7000, 2, 64)
    out = decode(B, b, q, 0.125)
    # (two heads of one kv head, so all sequences of one length at once)
    for n in sorted(set(lens)):
        at = [s for s, m in enumerate(lens) if m == n]
        if n == 0:
            assert not out[at].any()
            continue
        rows = torch.tensor([b.tables[s][:-(-n // 8)] for s in at], device=DEV)
        k, v = ((x[rows].double() * s[rows][..., None, None].double()).permute(0, 2, 1, 3, 4).reshape(len(at), -1, 64)[:, :n]
                for x, s in ((b.k, b.ks), (b.v, b.vs)))
        p = torch.softmax(q[at].double() @ k.transpose(1, 2) * 0.125, -1)
        check(out[at], p @ v, p @ v.abs(), f"length {n}")
    assert B.pkv_device_errors() == 0


def test_two_graphs_share_a_workspace(B):
    """A decode of a batch and a chunk of another, captured, replayed in turns on one workspace each kind."""
    b1, b2 = Batch([4000, 77], torch.int8, 2, 64, 16, seed=65), Batch([900] * 30, torch.float8_e4m3fn, 2, 64, 16, seed=66)
    q1, q2 = b1.randn(2, 4, 64), b2.randn(30, 4, 64)
    ws = torch.zeros(B.paged_decode_q8_workspace_size(30, 4, 2, 64, 4000), dtype=torch.uint8, device=DEV)
    chunk = torch.empty(max(B.paged_prefill_q8_workspace_size(2, 2, 64, 16, 4000),
                            B.paged_prefill_q8_workspace_size(30, 2, 64, 16, 900)), dtype=torch.uint8, device=DEV)
    o1, o2, c1, c2 = (torch.empty_like(x) for x in (q1, q2, q1, q2))
    s1, s2 = starts([1, 1]), starts([1] * 30)

    def one():
        decode_into(o1, q1, b1)
        B.paged_prefill_attention_q8(c1, q1, *b1.cache(), b1.bt, b1.cl, 4000, s1, 1, 0.125, workspace=chunk)

    def two():
        decode_into(o2, q2, b2)
        B.paged_prefill_attention_q8(c2, q2, *b2.cache(), b2.bt, b2.cl, 900, s2, 1, 0.125, workspace=chunk)

    def decode_into(out, q, b):
        B.paged_decode_attention_q8(out, q, *b.cache(), b.bt, b.cl, max(b.lens), 0.125, workspace=ws)

    graphs = []
    for f in (one, two):
        f()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    w1, w2 = decode_ref(b1, q1, 0.125), decode_ref(b2, q2, 0.125)
    for i in (0, 1, 1, 0, 1):
        for t in (o1, o2, c1, c2):
            t.fill_(77)
        graphs[i].replay()
        torch.cuda.synchronize()
        for out in ((o1, c1), (o2, c2))[i]:
            check(out, *(w1, w2)[i], f"graph {i}")
    assert B.pkv_device_errors() == 0


def test_behind_other_work(B):
    """Calls right behind what makes their inputs: kernels, copies and fills of the same stream, another
    stream's end; one after another and as a graph with a fork and a join."""
    b = Batch([500, 33, 900], torch.int8, 2, 64, 16, seed=68)
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    new = [b.randn(3, 6 + 4, 64) for _ in range(4)]
    big = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    x, src = torch.zeros_like(new[0]), torch.zeros_like(new[0])
    cl, bt, chunk = torch.zeros_like(b.cl), torch.zeros_like(b.bt), starts([1, 1, 1])
    q, k, v = x.split([6, 2, 2], dim=1)
    qc = torch.empty(3, 6, 64, dtype=torch.bfloat16, device=DEV)
    kr, vr = (torch.empty(3, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = torch.zeros(B.paged_decode_q8_workspace_size(3, 6, 2, 64, 900), dtype=torch.uint8, device=DEV)
    cws = torch.empty(B.paged_prefill_q8_workspace_size(3, 2, 64, 16, 900), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(qc) for _ in range(3)]
    cache = b.cache()

    def work():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            big.fill_(1)
            cl.copy_(b.cl)              # (late, behind the fill)
            bt.copy_(b.bt)
        x.copy_(src)
        qc.copy_(q)
        here.wait_stream(side)
        B.paged_decode_step_q8(outs[0], qc, k, v, *cache, bt, cl, 900, 0.125, workspace=ws)
        big.zero_()
        outs[1].fill_(3)
        B.paged_decode_attention_q8(outs[1], qc, *cache, bt, cl, 900, 0.125, workspace=ws)
        B.paged_prefill_attention_q8(outs[2], qc, *cache, bt, cl, 900, chunk, 1, 0.125, workspace=cws)
        big.zero_()
        B.paged_kv_read_q8(kr, vr, *cache, bt, cl, chunk, 1)
        qc.zero_()
        x.zero_()
        cl.zero_()
        bt.fill_(-1)

    def checked(i, run):
        want = b.copies()
        src.copy_(new[i])
        for s, n in enumerate(b.lens):
            R.write(want[0], want[2], new[i][s:s + 1, 6:8], b.tables[s], n - 1)
            R.write(want[1], want[3], new[i][s:s + 1, 8:], b.tables[s], n - 1)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        for got, w in zip(cache, want):
            same(got, w, "cache")
        for o in outs:
            check(o, *decode_ref(b, new[i][:, :6], 0.125), f"run {i}")
        for s, n in enumerate(b.lens):
            for got, c, sc in ((kr, b.k, b.ks), (vr, b.v, b.vs)):
                assert torch.equal(got[s], R.values(c, sc, b.tables[s], n - 1, n)[0].to(torch.bfloat16))

    with torch.cuda.stream(main):
        checked(0, work)
        checked(1, work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        work()
    checked(2, graph.replay)
    checked(3, graph.replay)
    assert B.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 32)])
def test_prompts_chunks_drafts_forks_and_steps(B, dtype, d, bs):
    """A serving loop over the 8-bit cache with the block manager: prompts, their next chunks, drafts
    checked and partly taken back, forks, rotated steps, compaction, the contexts handed on as bf16."""
    hq, hkv, nb, scale, r = 6, 2, 60, d ** -0.5, 32
    gen = torch.Generator().manual_seed(67)
    k, v, ks, vs = R.pools(nb, hkv, bs, d, dtype, gen, DEV)
    cache = (k, v, ks, vs)
    model = [t.clone() for t in cache]  # what R.write makes of the same calls
    ang = torch.arange(400, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    table = torch.cat((ang.cos(), ang.sin()), 1).float().to(DEV)
    bm = B.BlockManager(nb, bs)
    lens = {}

    def run(seqs, counts, attend):
        """The next counts[i] tokens of seqs[i]: appended, rotated and written, attended to."""
        rows = []
        for s, n in zip(seqs, counts):
            if s not in lens:
                bm.add_sequence(s, n)
                lens[s] = n
            else:
                for _ in range(n):
                    _, pairs, copied = bm.append_slots_cow([s])
                    if pairs.shape[0]:
                        B.paged_kv_copy_blocks_q8(*cache, pairs.to(DEV), copied.to(DEV))
                        for (a, z), m in zip(pairs.tolist(), copied.tolist()):
                            for i in range(4):
                                x = R.bits(model[i])
                                if i < 2:
                                    x[z, :, :m] = x[a, :, :m]
                                else:
                                    x[z] = x[a]
                lens[s] += n
            rows.append(range(lens[s] - n, lens[s]))
        bt, cl = (t.to(DEV) for t in bm.block_tables(list(seqs), 16))
        x = torch.randn(sum(counts), hq + 2 * hkv, d, generator=gen).to(torch.bfloat16).to(DEV)
        q, kn, vn = x.split([hq, hkv, hkv], dim=1)
        pos = torch.tensor([p for x in rows for p in x], device=DEV)
        wq, wk = R.rotate(q, table, pos, r, True), R.rotate(kn, table, pos, r, True)
        at = 0
        for s, n in zip(seqs, counts):
            tab = bt[list(seqs).index(s)].tolist()
            R.write(model[0], model[2], wk[at:at + n], tab, lens[s] - n)
            R.write(model[1], model[3], vn[at:at + n], tab, lens[s] - n)
            at += n
        out, q_out = (torch.empty(sum(counts), hq, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        longest = max(lens[s] for s in seqs)
        if attend == "step":
            B.paged_decode_step_rope_q8(out, q, kn, vn, table, *cache, bt, cl, longest, scale, q_out=q_out, rotary_dim=r)
        else:
            B.paged_kv_write_rope_q8(kn, vn, table, *cache, bt, cl, starts(counts), max(counts), q=q, q_out=q_out, rotary_dim=r)
            B.paged_prefill_attention_q8(out, q_out, *cache, bt, cl, longest, starts(counts), max(counts), scale)
        assert torch.equal(q_out, wq)
        at = 0
        for i, (s, n) in enumerate(zip(seqs, counts)):
            kk, vv = (R.values(c, sc, bt[i].tolist(), 0, lens[s], torch.float64) for c, sc in ((k, ks), (v, vs)))
            for got, c, sc in ((kk, model[0], model[2]), (vv, model[1], model[3])):
                assert torch.equal(got, R.values(c, sc, bt[i].tolist(), 0, lens[s], torch.float64)), f"sequence {s}"
            seen = torch.arange(lens[s], device=DEV)[None, :] <= torch.arange(lens[s] - n, lens[s], device=DEV)[:, None]
            want, mag = R.attention(wq[at:at + n], kk, vv, scale, seen)
            check_prefill(out[at:at + n], wq[at:at + n], kk, want, mag, scale)
            at += n
        return bt, cl

    run((0, 1, 2), (70, 33, 100), "chunk")     # prompts
    run((0, 2), (130, 1), "chunk")             # a prompt's next chunk beside a sequence's one token
    run((0, 1, 2), (5, 5, 5), "chunk")         # drafts, of which two are right
    for s in (0, 1, 2):
        bm.truncate(s, lens[s] - 3)
        lens[s] -= 3
    for child in (3, 4):
        bm.fork(0, child)
        lens[child] = lens[0]
    for _ in range(3):
        bt, cl = run((0, 1, 2, 3, 4), (1,) * 5, "step")
    before = [R.values(c, sc, bt[i].tolist(), 0, lens[s], torch.float32) for i, s in enumerate(range(5)) for c, sc in ((k, ks), (v, vs))]
    bm.free_sequence(1)
    moves, bmap = bm.compact()
    B.paged_kv_compact_q8(*cache, moves.to(DEV), bt, bmap.to(DEV))
    left = [0, 2, 3, 4]
    bt2, cl2 = (t.to(DEV) for t in bm.block_tables(left, 16))
    total = sum(lens[s] for s in left)
    k_out, v_out = (torch.empty(total, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    B.paged_kv_read_q8(k_out, v_out, *cache, bt2, cl2, starts([lens[s] for s in left]), max(lens.values()))
    at = 0
    for s in left:
        for got, want in ((k_out, before[2 * s]), (v_out, before[2 * s + 1])):
            assert torch.equal(got[at:at + lens[s]], want.to(torch.bfloat16)), f"sequence {s}"
        at += lens[s]
    assert B.pkv_device_errors() == 0
