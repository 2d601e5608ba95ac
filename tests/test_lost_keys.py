"""prompt_attention and paged_decode_shared_prefix_attention: no key is lost or counted twice.

With thousands of keys of like weight a single one, or a whole block of them, weighs less than
the roundings' worst case.  Here every query row is a multiple of one key of its context, its
target, so that this key weighs far more than the others; the targets lie at the borders of
blocks, pages, splits and parts, and anywhere else.

A row's error in the Euclidean norm over its dims, rounding by rounding and by the triangle
inequality, with A = sum p_t |v_t|: the output to bf16 at most 2^-8 |o|; the weights to bf16 at
most 2^-8 A, and once more where the row's sum is of the rounded ones; fp32 scores, the
hardware exp2, fp32 sums and merges under 2^-12 A.  A key of weight p that is left out moves the
row by about p |v_t|, and p is 0.05 at least for the targets (checked).

Over a whole call of independent normal v, the roundings add up as independent errors do: a
value rounded to bf16 is off by 2^-8 / sqrt(3) * 0.735 of itself in the mean square (over
significands spread evenly on the logarithm), the weights' and the output's together by
sqrt(2) * 0.00166 = 0.0023 of |o|, which leaves 0.004 far outside of chance for thousands of rows.
"""

import math
import random

import pytest
import torch

LOST = 0.05


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


def row_errors(out, o, amp):
    """Each row's error over its bound: o and out [..., d], amp = sum p |v| [...]."""
    o = o.double()
    return (out.double() - o).norm(dim=-1) / (2.0**-8 * o.norm(dim=-1) + (2.0**-7 + 2.0**-12) * amp)


def attend(q, k, v, scale, seen=None):
    """(o, sum p |v|, p) of q [r, d] over k, v [n, d] in 64 bits; seen [r, n] or None."""
    x = q.double() @ k.double().T * scale
    if seen is not None:
        x = x.masked_fill(~seen, float("-inf"))
    p = torch.softmax(x, -1)
    return p @ v.double(), p @ v.double().norm(dim=-1), p


def targets(rng, n, count):
    """`count` key positions of [0, n): borders of 16, 64 and 128 keys, the ends, and any."""
    out = []
    for _ in range(count):
        step = rng.choice([16, 64, 128, 128, 256])
        at = rng.choice([0, n - 1, rng.randrange(n), rng.randrange(0, n, step), rng.randrange(0, n, step) - 1])
        out.append(min(max(at, 0), n - 1))
    return out


def aimed(keys, n):
    """Queries [..., d] whose score against their key, at scale d^-0.5, passes by 2 the logarithm
    of the n keys' number; the other keys' scores are normal about 0."""
    x = keys.float()
    return ((math.log(n + 1) + 2) * x.shape[-1] ** 0.5 * x / (x * x).sum(-1, keepdim=True)).to(torch.bfloat16)


def test_the_bound_sees_a_lost_key():
    """On the CPU, weights and outputs rounded as the kernels': inside the bound; without the
    target, or with it twice, or without its block: outside."""
    g = torch.Generator().manual_seed(1)
    rng = random.Random(1)
    for d, n in ((64, 700), (128, 4096), (128, 20000)):
        k, v = (torch.randn(n, d, generator=g).to(torch.bfloat16) for _ in range(2))
        at = targets(rng, n, 24)
        q = aimed(k[at], n)
        o, amp, p = attend(q, k, v, d**-0.5)
        assert p[range(24), at].min() > LOST

        def output(p):
            pb = p.float().to(torch.bfloat16).double()
            return (pb @ v.double() / p.sum(-1, keepdim=True)).float().to(torch.bfloat16)

        x = torch.exp(q.double() @ k.double().T * d**-0.5)
        assert (row_errors(output(x), o, amp) <= 1).all()
        for change in (0.0, 2.0):
            y = x.clone()
            y[range(24), at] *= change
            assert (row_errors(output(y), o, amp) > 1).all()
        y = x.clone()
        for r, t in enumerate(at):
            y[r, t // 128 * 128:t // 128 * 128 + 128] = 0
        assert (row_errors(output(y), o, amp) > 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,hkv,grp", [([3001], 2, 3), ([1], 4, 1), ([129, 1, 700, 64, 2049], 2, 4),
                                          ([255, 256, 257, 511, 513], 1, 7), ([5000], 1, 128)])
def test_prompt(B, d, lens, hkv, grp):
    g = torch.Generator(device="cuda").manual_seed(d + len(lens))
    rng = random.Random(d + sum(lens))
    t, hq = sum(lens), hkv * grp
    k, v = (torch.randn(t, hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    start = [sum(lens[:i]) for i in range(len(lens) + 1)]
    at = torch.zeros(t, hq, dtype=torch.long)
    for s, n in zip(start, lens):
        for i in range(n):
            at[s + i] = torch.tensor([s + x for x in targets(rng, i + 1, hq)])
    at = at.cuda()
    heads = torch.arange(hq, device="cuda") // grp
    q = aimed(k[at, heads[None, :]], max(lens))
    out = torch.full_like(q, 3.0)
    B.prompt_attention(out, q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), max(lens), d**-0.5)
    least = 1.0
    for s, n in zip(start, lens):
        for h in range(hkv):
            for a in range(0, n, max(1, 2048 // grp)):
                z = min(n, a + max(1, 2048 // grp))
                rows = q[s + a:s + z, h * grp:(h + 1) * grp].reshape(-1, d)
                i = torch.arange(a, z, device="cuda").repeat_interleave(grp)
                seen = torch.arange(z, device="cuda")[None, :] <= i[:, None]
                o, amp, p = attend(rows, k[s:s + z, h], v[s:s + z, h], d**-0.5, seen)
                got = out[s + a:s + z, h * grp:(h + 1) * grp].reshape(-1, d)
                worst = row_errors(got, o, amp).max().item()
                assert worst <= 1, f"sequence at {s}, rows {a}.., head {h}: {worst}"
                hit = at[s + a:s + z, h * grp:(h + 1) * grp].reshape(-1) - s
                least = min(least, p[torch.arange(len(hit), device="cuda"), hit].min().item())
    assert least > LOST and B.pkv_device_errors() == 0


def batch(groups, prefixes, owns, hq, hkv, d, bs, seed):
    """Pages, tables and lengths of groups of sequences behind shared prefixes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    start = [sum(groups[:i]) for i in range(len(groups) + 1)]
    lens, rows, nb = [], [], 0
    for i, size in enumerate(groups):
        sh = prefixes[i] // bs
        common = list(range(nb, nb + sh))
        nb += sh
        for _ in range(size):
            n = prefixes[i] + owns[len(lens)]
            own = -(-n // bs) - sh
            rows.append(common + list(range(nb, nb + own)))
            nb += own
            lens.append(n)
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    tables = torch.full((len(lens), max(map(len, rows))), -1, dtype=torch.int32)
    for b, r in enumerate(rows):
        tables[b, :len(r)] = perm[r]
    k, v = (torch.randn(nb, hkv, bs, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    whole = [prefixes[i] // bs * bs for i in range(len(groups)) for _ in range(groups[i])]
    return dict(k=k, v=v, tables=tables.cuda(), lens=lens, start=torch.tensor(start, **i32), n=len(lens),
                prefix=torch.tensor(prefixes, **i32), max_prefix=max(prefixes),
                max_suffix=max(n - w for n, w in zip(lens, whole)))


def decode(B, c, q, scale, mode):
    out = torch.full_like(q, 3.0)
    before = B.pkv_set_shared_prefix(mode)
    try:
        B.paged_decode_shared_prefix_attention(
            out, q, c["k"], c["v"], c["tables"], torch.tensor(c["lens"], dtype=torch.int32, device="cuda"),
            c["start"], c["prefix"], c["max_prefix"], c["max_suffix"], scale)
    finally:
        B.pkv_set_shared_prefix(before)
    return out


def gathered(c, b, h):
    n, bs, d = c["lens"][b], c["k"].shape[2], c["k"].shape[3]
    at = c["tables"][b, :-(-n // bs)].long()
    return (x[at, h].reshape(-1, d)[:n] for x in (c["k"], c["v"]))


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("groups,prefixes,own,hq,hkv,d,bs", [
    ([17], [4096], 1, 24, 8, 128, 16), ([64], [8192], 200, 24, 8, 128, 16), ([64], [8200], 300, 32, 8, 64, 32),
    ([1] * 70, [150] * 70, 3, 8, 1, 64, 8), ([2] * 300, [100] * 300, 40, 4, 2, 128, 16),
    ([3, 50, 1, 11], [60000, 1000, 0, 129], 700, 8, 2, 64, 64)])
def test_shared_prefix(B, mode, groups, prefixes, own, hq, hkv, d, bs):
    rng = random.Random(len(groups))
    owns = [own if k % 3 == 0 else rng.randint(1, own) for k in range(sum(groups))]
    c = batch(groups, prefixes, owns, hq, hkv, d, bs, 5)
    grp, n = hq // hkv, max(c["lens"])
    for seed in range(2):
        q, at = torch.empty(c["n"], hq, d, dtype=torch.bfloat16, device="cuda"), []
        for b in range(c["n"]):
            ctx = c["lens"][b]
            t = targets(rng, ctx, hq)
            for h in range(0, hq, 2):  # half of them among the own keys
                t[h] = ctx - 1 - rng.randrange(owns[b])
            at.append(t)
            page = c["tables"][b, [x // bs for x in t]].long()
            keys = c["k"][page, torch.arange(hq, device="cuda") // grp, torch.tensor(t, device="cuda") % bs]
            q[b] = aimed(keys, n)
        out = decode(B, c, q, d**-0.5, mode)
        for b in range(c["n"]):
            for h in range(hkv):
                kk, vv = gathered(c, b, h)
                o, amp, p = attend(q[b, h * grp:(h + 1) * grp], kk, vv, d**-0.5)
                worst = row_errors(out[b, h * grp:(h + 1) * grp], o, amp).max().item()
                assert worst <= 1, f"seed {seed}, sequence {b}, kv head {h}: {worst}"
                hit = at[b][h * grp:(h + 1) * grp]
                assert p[range(grp), hit].min() > LOST
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_errors_over_a_call(B, d):
    """Normal q, k, v: the error over the whole call, and over each sequence of it."""
    g = torch.Generator(device="cuda").manual_seed(d)
    hq, hkv, lens = 8, 2, [2048, 700, 1500]
    t = sum(lens)
    q, k, v = (torch.randn(t, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    start, out = [0, 2048, 2748, 4248], torch.empty_like(q)
    B.prompt_attention(out, q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), 2048, d**-0.5)
    o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for s, n in zip(start, lens):
        seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for h in range(hq):
            o[s:s + n, h] = attend(q[s:s + n, h], k[s:s + n, h // 4], v[s:s + n, h // 4], d**-0.5, seen)[0]
    calls = [("prompt", out, o, [slice(s, s + n) for s, n in zip(start, lens)])]
    c = batch([40], [4100], [1 + x % 50 for x in range(40)], hq, hkv, d, 16, 9)
    q = torch.randn(40, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b in range(40):
        for h in range(hkv):
            o[b, 4 * h:4 * h + 4] = attend(q[b, 4 * h:4 * h + 4], *gathered(c, b, h), d**-0.5)[0]
    for mode in (B.SHARED_ALWAYS, B.SHARED_NEVER):
        calls.append((f"shared prefix, mode {mode}", decode(B, c, q, d**-0.5, mode), o,
                      [slice(b, b + 1) for b in range(40)]))
    for name, out, o, parts in calls:
        err = out.double() - o
        assert err.norm() <= 4e-3 * o.norm(), f"{name}: {(err.norm() / o.norm()).item()}"
        for p in parts:  # each of two roundings at its largest
            assert err[p].norm() <= 2.0**-7.5 * o[p].norm(), f"{name}: {(err[p].norm() / o[p].norm()).item()}"
    assert B.pkv_device_errors() == 0
