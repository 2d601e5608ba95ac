"""The 8-bit cache's attention at the ends of its ranges.

Tolerances as in test_q8_attention.py: 2^-8 |out| + 2^-10 sum p |v|, and n 2^-35 of the largest |v|.
"""

import pytest
import torch

import q8_ref as R
from test_q8_attention import check, decode, decode_ref
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
