"""How far the 8-bit cache's values may be from the rows that were written, as its pages grow.

A scale s rounds to s / 2 (int8), or to 2^-4 of the value and 2^-10 s where that is more (e4m3). Each growth
of a page's scale to s' rounds the rows that it held again: with an error e so far, to e + s' / 2, or to
(|x| + e) (1 + 2^-4) - |x| and 2^-10 s' more.  fp32 quotients and products are 2^-22 of the value.
"""

import pytest
import torch

import q8_ref as R
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


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("bs", [16, 256])
@pytest.mark.parametrize("step", [1, 3, 1000])
def test_errors_of_pages_that_grow(B, dtype, bs, step):
    """Two sequences whose values rise (most growths) and do not, written `step` tokens at a time: every
    row against the original after every write, within the sum of the roundings that it had."""
    n, hkv, d = 2 * bs + 5, 2, 64
    b = Batch([n, n], dtype, hkv, d, bs, seed=90)
    rise = torch.stack((torch.linspace(0.5, 1.5, n), torch.ones(n))).to(DEV)
    x = (b.randn(2, n, hkv, d).float() * rise[:, :, None, None]).to(torch.bfloat16)
    bound = torch.zeros(2, n, hkv, d, dtype=torch.float64, device=DEV)
    size = x.double().abs()
    growths = 0
    for at in range(0, n, step):
        end = min(at + step, n)
        before = [b.ks[b.tables[s][:-(-n // bs)]].clone() for s in range(2)]
        cl = torch.full((2,), end, dtype=torch.int32, device=DEV)
        k = x[:, at:end].reshape(-1, hkv, d)
        B.paged_kv_write_q8(k, -k, *b.cache(), b.bt, cl, starts([end - at] * 2), end - at)
        for s in range(2):
            now = b.ks[b.tables[s][:-(-n // bs)]]
            for page in range(at // bs, -(-end // bs)):
                lo, first = page * bs, max(page * bs, at)
                last = min(end, lo + bs)
                unit = now[page].double()[None, :, None]
                grew = ((now[page] > before[s][page]) & (first > lo))[None, :, None]
                growths += int(grew.sum())
                for rows, rounded in ((slice(lo, first), grew), (slice(first, last), torch.ones_like(grew))):
                    e, y = bound[s, rows], size[s, rows]
                    if dtype is torch.int8:
                        more = unit / 2
                    else:
                        more = torch.maximum((y + e) / 16, unit / 1024)
                    bound[s, rows] = torch.where(rounded, e + more + 2.0 ** -22 * (y + e), e)
            got = R.values(b.k, b.ks, b.tables[s], 0, end, torch.float64)
            err = (got - x[s, :end].double()).abs()
            assert bool((err <= bound[s, :end]).all()), f"after {end}: {float((err / bound[s, :end]).max())}"
            assert torch.equal(R.values(b.v, b.vs, b.tables[s], 0, end, torch.float64), -got)
    if step >= n:  # every page at once: the bound of a block written at once
        top = R.TOP[dtype]
        for s in range(2):
            for page in range(-(-n // bs)):
                rows = slice(page * bs, min(n, page * bs + bs))
                largest = size[s, rows].amax((0, 2), keepdim=True)
                least = largest / top / 2 if dtype is torch.int8 else torch.maximum(size[s, rows] / 16, largest / top / 1024)
                # (2^-22 of a value, at most 127 scales, is less than 2^-14 of half a scale; and fp32's rounding of the scale)
                assert bool((bound[s, rows] <= least * (1 + 2.0 ** -13)).all())
    else:
        assert growths > 0
    assert B.pkv_device_errors() == 0
