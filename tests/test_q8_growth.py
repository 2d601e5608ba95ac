"""Pages whose scale grows: the rows that they held rounded anew, of every code, by ratios of the scales that put
codes on the borders between two; bit for bit."""

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


@pytest.mark.parametrize("dtype", R.KINDS)
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("d,bs,held,new", [
    (64, 8, 7, 1), (64, 16, 1, 1), (128, 16, 15, 1), (128, 32, 5, 27), (64, 128, 127, 1), (128, 256, 255, 1), (128, 256, 100, 156),
])
def test_every_code_rounded_anew(B, dtype, rope, d, bs, held, new):
    """Ratios of 1.0078 to 2^20, 2 and 3 among them; a page of zeros' scale; one that does not grow."""
    ratios = [1.0078125, 1.25, 1.5, 2.0, 3.0, 4.0, 7.0, 250.0, 2.0 ** 20, 0.5]
    b = Batch([held + new] * (len(ratios) + 1), dtype, 2, d, bs, seed=93)
    n = len(b.lens)
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[codes != 0x80] if dtype is torch.int8 else codes[codes & 0x7f != 0x7f]
    for c in (b.k, b.v):
        at = torch.randint(0, len(codes), c.shape, generator=b.gen)
        flat = at.view(c.shape[0], -1)  # every code at the beginning of each page and kv head, where there is room
        m = min(len(codes), held * d)
        flat.view(c.shape[0], 2, -1)[:, :, :m] = torch.arange(m)
        R.bits(c).copy_(codes[at].to(DEV))
    k, v = b.randn(n * new, 2, d), b.randn(n * new, 2, d)
    top = R.TOP[dtype]
    for s, ratio in enumerate(ratios + [0.0]):
        page = b.tables[s][0]
        for x, scale in ((k, b.ks), (v, b.vs)):
            need = x[s * new:(s + 1) * new].float().abs().amax((0, 2)) / torch.tensor(top, device=DEV)
            scale[page] = need / ratio if ratio else 0.0
    want = b.copies()
    if rope:  # by angles of 0
        table = torch.cat((torch.ones(held + new, d // 2), torch.zeros(held + new, d // 2)), 1).to(DEV)
        B.paged_kv_write_rope_q8(k, v, table, *b.cache(), b.bt, b.cl, starts([new] * n), new)
    else:
        B.paged_kv_write_q8(k, v, *b.cache(), b.bt, b.cl, starts([new] * n), new)
    for s in range(n):
        R.write(want[0], want[2], k[s * new:(s + 1) * new], b.tables[s], held)
        R.write(want[1], want[3], v[s * new:(s + 1) * new], b.tables[s], held)
    for x, y, what in zip(b.cache(), want, ("k codes", "v codes", "k scales", "v scales")):
        same(x, y, what)
    assert B.pkv_device_errors() == 0
