"""NaN and infinities in k and v: they reach the rows that see their keys, and no others.

Reference in 64 bits, over the keys each row sees.  Where it is finite the output is within
2^-8 |o| + (2^-7 + 2^-12) sum p |v| of it (the output's rounding, the weights', and where it
is of rounded weights their sum's; fp32 elsewhere); where it is not, the output is not either.
"""

import pytest
import torch

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


def reference(q, k, v, scale):
    """(o, sum p |v|) of q [r, d] over k, v [n, d]."""
    p = torch.softmax(q.double() @ k.double().T * scale, -1)
    return p @ v.double(), p @ v.double().abs()


def check(out, o, amp, what=""):
    out, ok = out.double(), o.isfinite()
    assert torch.equal(out.isfinite(), ok), \
        f"{what}: {int((~out.isfinite() & ok).sum())} values hit, {int((out.isfinite() & ~ok).sum())} missed"
    bound = 2.0**-8 * o.abs() + (2.0**-7 + 2.0**-12) * amp + 1e-30
    worst = ((out - o).abs() / bound)[ok].max().item() if bool(ok.any()) else 0.0
    assert worst <= 1, f"{what}: {worst} of the bound"


def spoil(x, at, d, seed):
    """Some dims of rows x[at] (pairs of row and head) become NaN or infinite."""
    g = torch.Generator().manual_seed(seed)
    for n, (t, h) in enumerate(at):
        dims = torch.randperm(d, generator=g)[:1 + n % 5]
        x[t, h, dims.to(x.device)] = [NAN, INF, -INF][n % 3]


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("hq,hkv,d,bs,prefix", [(24, 8, 128, 16, 2048), (8, 8, 64, 32, 1000), (8, 1, 64, 8, 700),
                                                (12, 4, 128, 64, 9000)])
def test_shared_pages(B, mode, hq, hkv, d, bs, prefix):
    """Contexts that end all over the shared prefix, non-finite v at the ends of some and behind,
    shared and plain."""
    g = torch.Generator(device="cuda").manual_seed(d + bs)
    ends = [prefix + 9, 0, 1, 63, 64, 65, prefix // 2, prefix // 2 + 1, prefix - prefix % bs, prefix - 1, 130, prefix + 40]
    ends += [1 + 37 * i % prefix for i in range(30)]
    n, sh = len(ends), prefix // bs
    own = -(-(prefix + 40) // bs) - sh
    k, v = (torch.randn((sh + n * own) * bs, hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    grp = hq // hkv
    spoil(v, [(t % (sh * bs), h) for t, h in ((prefix // 2, 0), (64, hkv - 1), (prefix - 2, hkv // 2), (128, 0),
                                              (prefix // 3, hkv - 1), (bs, 0))], d, 5)
    k[sh * bs - 1, 0, 3] = NAN
    perm = torch.randperm(sh + n * own, generator=g, device="cuda")
    pages = [x.view(-1, bs, hkv, d).transpose(1, 2).contiguous() for x in (k, v)]
    pool = [torch.empty_like(x) for x in pages]
    for p, x in zip(pool, pages):
        p[perm] = x
    rows = [list(range(sh)) + [sh + b * own + j for j in range(own)] for b in range(n)]
    tables = perm[torch.tensor(rows, device="cuda")].to(torch.int32).contiguous()
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(n, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    before = B.pkv_set_shared_prefix(mode)
    try:
        B.paged_decode_shared_prefix_attention(out, q, *pool, tables, torch.tensor(ends, **i32),
                                               torch.tensor([0, n], **i32), torch.tensor([prefix], **i32), prefix,
                                               own * bs, d**-0.5)
    finally:
        B.pkv_set_shared_prefix(before)
    for b, end in enumerate(ends):
        if end == 0:
            assert bool((out[b] == 0).all())
            continue
        at = torch.cat([torch.arange(r * bs, r * bs + bs) for r in rows[b]])[:end].cuda()
        for h in range(hkv):
            o, amp = reference(q[b, h * grp:(h + 1) * grp], k[at, h], v[at, h], d**-0.5)
            check(out[b, h * grp:(h + 1) * grp], o, amp, f"end {end}, kv head {h}")
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,grp", [(2, 1), (2, 3), (1, 5), (2, 8), (1, 128)])
def test_prompts(B, d, hkv, grp):
    """A NaN key makes the rows that see it NaN and changes no bit before it; a NaN in v, the
    rows that see it, and none that many tokens before it, nor of another sequence."""
    g = torch.Generator(device="cuda").manual_seed(d + grp)
    lens, hq = [257, 700, 1, 90], hkv * grp
    start = [sum(lens[:i]) for i in range(len(lens) + 1)]
    q, k, v = (torch.randn(sum(lens), h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))

    def run(k, v):
        out = torch.full_like(q, 3.0)
        B.prompt_attention(out, q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), max(lens), d**-0.5)
        return out

    clean, rows = run(k, v), torch.arange(sum(lens), device="cuda")
    for at in (start[1], start[1] + 127, start[1] + 255, start[1] + 256, start[1] + 300, start[1] + 511, start[2] - 1):
        hit = (rows >= at) & (rows < start[2])
        for which in (0, 1):
            kv = [k.clone(), v.clone()]
            kv[which][at, 0, 11] = NAN
            out = run(*kv)
            free = ~hit if which == 0 else ~hit & ~((rows < at) & (rows >= start[1]) & (rows > at - 128 - 128 // grp))
            assert torch.equal(out[free], clean[free]), at
            assert torch.equal(out[:, grp:], clean[:, grp:])  # the other kv heads
            dims = slice(None) if which == 0 else slice(11, 12)
            assert bool(out[hit][:, :grp, dims].isnan().all()), at
    assert B.pkv_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_minus_infinity(B, mode, d):
    """Keys of score -inf weigh nothing: leading ones, whole blocks and splits, the own keys alone;
    in prompts the rows that see such keys only have no value and are left out."""
    g = torch.Generator(device="cuda").manual_seed(d)
    hq, hkv, bs, prefix, own, n = 8, 2, 16, 1024, 48, 6
    sh, cols = prefix // bs, (prefix + own) // bs
    tables = torch.empty(n, cols, dtype=torch.int32, device="cuda")
    tables[:, :sh] = torch.arange(sh, device="cuda")
    tables[:, sh:] = sh + torch.arange(n * (cols - sh), device="cuda").view(n, -1)
    k, v = (torch.randn(sh + n * (cols - sh), hkv, bs, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    q[:, :, 5] = q[:, :, 5].abs() + 0.25
    i32 = dict(dtype=torch.int32, device="cuda")
    lens = [prefix + 1 + 9 * b for b in range(n)]
    for dead in ([(0, 1)], [(0, 700)], [(128, 256), (prefix, prefix + own)], [(0, prefix)], [(prefix - 300, prefix + own)]):
        kk = k.clone()
        for b in range(n):
            for lo, hi in dead:
                for t in range(lo, hi):
                    kk[tables[b, t // bs].long(), :, t % bs, 5] = -INF
        out = torch.full_like(q, 3.0)
        before = B.pkv_set_shared_prefix(mode)
        try:
            B.paged_decode_shared_prefix_attention(out, q, kk, v, tables, torch.tensor(lens, **i32),
                                                   torch.tensor([0, n], **i32), torch.tensor([prefix], **i32), prefix,
                                                   own, d**-0.5)
        finally:
            B.pkv_set_shared_prefix(before)
        for b in range(n):
            for h in range(hkv):
                x, y = (z[tables[b].long(), h].reshape(-1, d)[:lens[b]] for z in (kk, v))
                o, amp = reference(q[b, 4 * h:4 * h + 4], x, y, d**-0.5)
                check(out[b, 4 * h:4 * h + 4], o, amp, f"{dead}, sequence {b}, kv head {h}")
    t = 600
    q, k, v = (torch.randn(t, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    q[:, :, 5] = q[:, :, 5].abs() + 0.25
    for lo, hi in ((0, 1), (0, 128), (0, 300), (200, 500), (130, 131)):
        kk, out = k.clone(), torch.full_like(q, 3.0)
        kk[lo:hi, :, 5] = -INF
        B.prompt_attention(out, q, kk, v, torch.tensor([0, t], **i32), t, d**-0.5)
        for h in range(hq):
            for i in range(hi if lo == 0 else 0, t, 37):
                o, amp = reference(q[i:i + 1, h], kk[:i + 1, h // 4], v[:i + 1, h // 4], d**-0.5)
                check(out[i:i + 1, h], o, amp, f"prompt {lo}..{hi}, row {i}, head {h}")
    assert B.pkv_device_errors() == 0
