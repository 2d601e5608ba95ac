"""The rotary write over pages of every size: rows by groups of a warp to a whole CTA, rows that do not fit a
group's registers and are read a second time, positions that have no angles.  Bit for bit."""

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


def angles(n, r):
    ang = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    return torch.cat((ang.cos(), ang.sin()), 1).float().to(DEV)


def write_and_check(B, b, new, k, v, table, r, neox, bad=(), **kw):
    """k rotated and v written; rows `bad` (packed) have no angles: k's are left as they were."""
    t = sum(new)
    pos = torch.cat([torch.arange(m - n, m) for m, n in zip(b.lens, new)]).to(DEV)
    given = pos.clone()
    given[list(bad)] = table.shape[0]
    want = b.copies()
    q = kw.get("q")
    B.paged_kv_write_rope_q8(k, v, table, *b.cache(), b.bt, b.cl, starts(new), max(new), rotary_dim=r, neox_style=neox,
                             positions=given if bad else None, **kw)
    wk = R.rotate(k, table, pos, r, neox)
    wk[list(bad)] = 0
    kept = R.bits(want[0]).clone()
    at = 0
    for s, n in enumerate(new):
        R.write(want[0], want[2], wk[at:at + n], b.tables[s], b.lens[s] - n)
        R.write(want[1], want[3], v[at:at + n], b.tables[s], b.lens[s] - n)
        for i in bad:
            if at <= i < at + n:
                p = b.lens[s] - n + i - at
                page, row = b.tables[s][p // b.bs], p % b.bs
                R.bits(want[0])[page, :, row] = kept[page, :, row]
        at += n
    for x, y, what in zip(b.cache(), want, ("k codes", "v codes", "k scales", "v scales")):
        same(x, y, what)
    if q is not None:
        wq = R.rotate(q, table, pos, r, neox)
        keep = torch.ones(t, dtype=torch.bool)
        keep[list(bad)] = False
        assert torch.equal(kw["q_out"][keep], wq[keep]) and bool((kw["q_out"][~keep] == 9).all())
    assert B.pkv_device_errors() == (16 if bad else 0)


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("bs,d,r,hkv,lens,new", [
    (8, 128, 128, 2, [100, 7, 9], [93, 7, 2]), (32, 128, 64, 3, [200, 33], [200, 1]),
    (64, 128, 128, 2, [500, 64, 65], [437, 64, 1]), (64, 64, 32, 1, [300], [299]),
    (128, 128, 128, 2, [400, 129, 128], [271, 129, 127]), (128, 64, 64, 3, [260], [259]),
    (256, 128, 128, 2, [700, 256, 1, 300], [600, 256, 1, 129]), (256, 128, 16, 1, [513, 255], [513, 250]),
    (256, 64, 64, 2, [600, 257], [600, 200]),
])
def test_rotary_write_of_pages(B, dtype, neox, bs, d, r, hkv, lens, new):
    """Prompts and their next chunks, q rotated beside them; then the same rows larger, so that every page that
    holds rows has them rounded anew."""
    hq = 3 * hkv
    b = Batch(lens, dtype, hkv, d, bs, seed=91)
    table = angles(max(lens), r)
    for grow in (1.0, 5.0):
        x = b.randn(sum(new), hq + 2 * hkv, d) * grow
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        write_and_check(B, b, new, k, v, table, r, neox, q=q, q_out=torch.full_like(q.contiguous(), 9.0))


@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("bs,d", [(16, 128), (128, 128), (256, 128), (256, 64)])
def test_positions_without_angles(B, neox, bs, d):
    """Rows of a long run whose positions are out of range, among them the largest of a page, first and last ones,
    and ones of the rows that are read a second time."""
    lens, new = [2 * bs + 40, bs], [2 * bs + 10, bs]
    b = Batch(lens, torch.float8_e4m3fn, 2, d, bs, seed=92)
    x = b.randn(sum(new), 8, d)
    q, k, v = x.split([4, 2, 2], dim=1)
    bad = [0, 3, bs - 1, 2 * bs + 9, 2 * bs + 10 + bs // 2, sum(new) - 1]
    k[3] *= 40
    write_and_check(B, b, new, k, v, angles(max(lens), d), d, neox, bad, q=q, q_out=torch.full_like(q.contiguous(), 9.0))
