"""paged_decode_attention where keys are not finite: a visible NaN makes its rows NaN, on every
arrangement of the kernels; a score of -inf weighs nothing; what lies past a context is not seen.

Reference in 64 bits.  Allowed: 2^-8 |o| for the output's rounding and 2^-10 sum p |v| (weights
held in 16 bits or more, fp32 sums of at most 2^14 terms).
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


# sequences, kv heads, group, head_dim, longest context, arrangement
SHAPES = [(3, 2, 4, 128, 400, "PARTITIONS"), (3, 2, 3, 128, 3000, "CLUSTER"), (2, 1, 8, 64, 900, "CLUSTER"),
          (3, 2, 4, 64, 9000, "PARTITIONS"), (160, 4, 2, 64, 2000, "PERSISTENT"), (100, 4, 1, 128, 1700, "PERSISTENT")]


def make(n, hkv, grp, d, longest, what, bs=16):
    """Contexts of three kinds (b % 3): clean; keys of score -inf; a NaN among the keys."""
    g = torch.Generator(device="cuda").manual_seed(d + longest)
    cols = -(-longest // bs) + 1
    k, v = (torch.randn(n, cols * bs, hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, hkv * grp, d, generator=g, device="cuda").to(torch.bfloat16)
    q[:, :, 5] = q[:, :, 5].abs() + 0.25  # a key of -inf there scores -inf
    lens = [longest - (37 * b) % min(longest - 1, 700) for b in range(n)]
    for b, m in enumerate(lens):
        k[b, m:], v[b, m:] = NAN, INF
        if b % 3 == 1:
            for lo, hi in what[0]:
                k[b, lo % m:min(hi, m - 1), :, 5] = -INF
            if what[2]:
                k[b, m - 1, :, 5] = -INF
        if b % 3 == 2:
            k[b, what[1] % m, 0, 9] = NAN
    perm = torch.randperm(n * cols, generator=g, device="cuda")
    pools = []
    for x in (k, v):
        pool = torch.empty(n * cols, hkv, bs, d, dtype=torch.bfloat16, device="cuda")
        pool[perm] = x.view(n * cols, bs, hkv, d).transpose(1, 2)
        pools.append(pool)
    return q, k, v, pools, perm.view(n, cols).to(torch.int32).contiguous(), lens


def check(out, q, k, v, lens, grp, scale):
    for b in range(0, len(lens), max(1, len(lens) // 12)):
        m = lens[b]
        for h in range(k.shape[2]):
            x = q[b, h * grp:(h + 1) * grp].double() @ k[b, :m, h].double().T * scale
            p, vv = torch.softmax(x, -1), v[b, :m, h].double()
            o, got = p @ vv, out[b, h * grp:(h + 1) * grp].double()
            assert torch.equal(o.isnan(), got.isnan()), f"sequence {b}, kv head {h}"
            ok = ~o.isnan()
            bound = 2.0**-8 * o.abs() + 2.0**-10 * (p @ vv.abs())
            assert bool(((got - o).abs() <= bound)[ok].all()), f"sequence {b}, kv head {h}"


# (ranges of keys with a score of -inf, the NaN's place, whether the last key scores -inf too)
@pytest.mark.gpu
@pytest.mark.parametrize("what", [([(0, 1)], 0, False), ([(0, 70), (100, 130)], -1, True), ([(0, 640)], 513, False),
                                  ([(512, 100000)], -1, True)])
@pytest.mark.parametrize("n,hkv,grp,d,longest,path", SHAPES)
def test_decode(B, n, hkv, grp, d, longest, path, what):
    if what[0][0] == (0, 640) and longest < 700:
        what = ([(0, 300)], 200, False)
    q, k, v, pools, tables, lens = make(n, hkv, grp, d, longest, what)
    i32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert B.paged_decode_path(n, hkv * grp, hkv, d, longest) == getattr(B, "PATH_" + path)
    for consumer in (B.CONSUMER_TENSOR, B.CONSUMER_FMA):
        before = B.pkv_set_decode_consumer(consumer)
        try:
            out = torch.full_like(q, 3.0)
            B.paged_decode_attention(out, q, *pools, tables, i32, longest, d**-0.5)
            check(out, q, k, v, lens, grp, d**-0.5)
            P = 512
            parts = -(-longest // P)
            o = torch.zeros(n, hkv * grp, parts, d, device="cuda")
            lse = torch.zeros(n, hkv * grp, parts, device="cuda")
            B.paged_decode_split(o, lse, q, *pools, tables, i32, longest, d**-0.5, P)
            out.fill_(3.0)
            B.paged_decode_combine(out, o, lse, i32, longest, P)
            check(out, q, k, v, lens, grp, d**-0.5)
        finally:
            B.pkv_set_decode_consumer(before)
    assert B.pkv_device_errors() == 0
