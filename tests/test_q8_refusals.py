"""The 8-bit cache's entry points refuse bad arguments on the host, before any launch."""

import ctypes
import struct

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced by the host checks
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_mapping_gb300 import build

    build.build()
    from paged_kv_decode_mapping_gb300 import binding

    return binding


def q8(B, kind=0, k=FAKE, ks=FAKE):
    return B.pkv_q8_cache(k, FAKE, ks, FAKE, kind)


def desc(B, nb=64, bs=16, hkv=2, d=64):
    return B.pkv_cache_desc(nb, bs, hkv, d)


def both(B, c, d):
    return (ctypes.byref(c) if c is not None else None), (ctypes.byref(d) if d is not None else None)


@pytest.mark.parametrize("name", ["paged_kv_write_q8", "paged_kv_read_q8"])
def test_rows(B, name):
    fn = getattr(B.lib(), name)

    def call(k=FAKE, sk=128, start=FAKE, tokens=6, most=3, tables=FAKE, cols=8, lens=FAKE, seqs=2, c=q8(B), d=desc(B)):
        return fn(k, FAKE, sk, 128, start, tokens, most, tables, cols, lens, seqs, *both(B, c, d), None)

    assert call(c=None) == -1 and call(d=None) == -1
    assert call(c=q8(B, kind=2)) == -3 and "kind" in B.pkv_last_error()
    assert call(d=desc(B, d=96)) == -3 and call(d=desc(B, bs=12)) == -3 and call(d=desc(B, bs=512)) == -3
    assert call(d=desc(B, nb=0)) == -2 and call(d=desc(B, nb=1 << 30)) == -3
    assert call(seqs=-1) == -2 and call(tokens=-1) == -2 and call(most=-1) == -2 and call(cols=0) == -2
    assert call(seqs=70000) == -3
    assert call(start=None) == -2                       # three tokens a sequence, no query_start
    assert call(start=None, most=1, tokens=1) == -2     # fewer rows than sequences
    assert call(sk=120) == -2                           # a stride under a token's heads
    assert call(sk=132) == -5
    assert call(k=None) == -1 and call(tables=None) == -1 and call(lens=None) == -1
    assert call(k=ODD) == -5 and call(c=q8(B, k=ODD)) == -5 and call(c=q8(B, ks=ctypes.c_void_p((1 << 20) + 2))) == -5
    assert call(c=q8(B, ks=None)) == -1
    assert call(lens=ctypes.c_void_p((1 << 20) + 2)) == -5
    assert call(seqs=65535, most=1 << 30, cols=1 << 30, tokens=1 << 40) == -3
    assert call(tokens=0) == 0 and call(most=0) == 0 and call(seqs=0, k=None, c=B.pkv_q8_cache()) == 0


def test_rotary(B):
    def call(q=FAKE, q_out=FAKE, sq=256, hq=4, pos=FAKE, cs=FAKE, most_pos=100, r=32, tokens=6):
        return B.lib().paged_kv_write_rope_q8(FAKE, FAKE, 128, 128, q, q_out, sq, 256, hq, pos, cs, most_pos, r, 1, FAKE,
                                              tokens, 3, FAKE, 8, FAKE, 2, *both(B, q8(B), desc(B)), None)

    assert call(r=24) == -3 and call(r=0) == -3 and call(r=128) == -3
    assert call(most_pos=0) == -2 and call(hq=0) == -2 and call(sq=248) == -2
    assert call(cs=None) == -1 and call(q_out=None) == -1
    assert call(cs=ODD) == -5 and call(q=ODD) == -5 and call(pos=ODD) == -5 and call(sq=260) == -5
    assert call(tokens=0) == 0


def test_decode(B):
    ws = B.paged_decode_q8_workspace_size(2, 8, 2, 64, 100)
    assert ws > 0 and ws == B.paged_decode_q8_workspace_size(900, 8, 2, 64, 100000)  # by the heads alone
    assert B.paged_decode_q8_workspace_size(2, 8, 2, 96, 100) == 0
    assert B.paged_decode_q8_workspace_size(2, 7, 2, 64, 100) == 0
    assert B.paged_decode_q8_workspace_size(2, 18, 2, 64, 100) == 0

    def call(out=FAKE, q=FAKE, c=q8(B), d=desc(B), cols=8, most=100, seqs=2, hq=8, w=FAKE, size=ws, tables=FAKE):
        return B.lib().paged_decode_attention_q8(out, q, ctypes.byref(c) if c else None, tables, cols, FAKE, most, seqs, hq,
                                                 ctypes.byref(d) if d else None, 0.1, w, size, None)

    assert call(c=None) == -1 and call(d=None) == -1 and call(out=None) == -1 and call(q=None) == -1
    assert call(tables=None) == -1
    assert call(hq=7) == -2 and call(hq=18) == -3 and call(most=129) == -2 and call(most=-1) == -2
    assert call(d=desc(B, d=32)) == -3 and call(c=q8(B, kind=7)) == -3
    assert call(w=None) == -4 and call(size=ws - 1) == -4 and "workspace" in B.pkv_last_error()
    assert call(w=ODD) == -5 and call(out=ODD) == -5 and call(q=ODD) == -5
    assert call(seqs=0, out=None, q=None, tables=None, w=None) == 0


def test_steps(B):
    ws = B.paged_decode_q8_workspace_size(2, 8, 2, 64, 100)

    def call(k=FAKE, w=FAKE, rope=False, r=64, q_out=FAKE, d=desc(B)):
        c, d = both(B, q8(B), d)
        if rope:
            return B.lib().paged_decode_step_rope_q8(FAKE, FAKE, 512, q_out, k, FAKE, 128, 128, None, FAKE, 100, r, 1, c, FAKE,
                                                     8, FAKE, 100, 2, 8, d, 0.1, w, ws, None)
        return B.lib().paged_decode_step_q8(FAKE, FAKE, k, FAKE, 128, 128, c, FAKE, 8, FAKE, 100, 2, 8, d, 0.1, w, ws, None)

    for rope in (False, True):
        assert call(k=None, rope=rope) == -1 and call(w=None, rope=rope) == -4 and call(d=None, rope=rope) == -1
    assert call(rope=True, r=8) == -3 and call(rope=True, q_out=None) == -1


def test_prefill(B):
    ws = B.paged_prefill_q8_workspace_size(2, 2, 64, 16, 100)
    assert ws >= 2 * 2 * 100 * 2 * 64 * 2 and B.paged_prefill_q8_workspace_size(2, 2, 80, 16, 100) == 0
    assert B.paged_prefill_q8_workspace_size(65535, 8, 64, 16, 1 << 20) == 0  # over 2^31 rows

    def call(out=FAKE, most=100, start=FAKE, new=4, w=FAKE, size=ws, c=q8(B), queries=8):
        return B.lib().paged_prefill_attention_q8(out, FAKE, queries, ctypes.byref(c), FAKE, 8, FAKE, most, start, new, 2, 8,
                                                  ctypes.byref(desc(B)), 0.1, w, size, None)

    assert call(out=None) == -1 and call(start=None) == -1 and call(new=101) == -2 and call(w=None) == -4
    assert call(size=ws - 1) == -4 and call(w=ODD) == -5 and call(out=ODD) == -5 and call(c=q8(B, kind=3)) == -3
    assert call(queries=-1) == -2
    assert call(new=0) == 0 and call(queries=0) == 0


def test_the_binding_names_what_is_wrong(B):
    bf = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    codes, scale = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2)
    bt, cl = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.paged_kv_write_q8(bf, bf, codes, codes, scale, scale, bt, cl)
    with pytest.raises(ValueError, match=r"\[T, Hkv, D\]"):
        B.paged_kv_write_q8(bf[:, :1], bf, codes, codes, scale, scale, bt, cl)
    with pytest.raises(TypeError, match="bfloat16"):
        B.paged_kv_read_q8(bf.float(), bf.float(), codes, codes, scale, scale, bt, cl)
    with pytest.raises(ValueError, match="CUDA"):
        B.paged_decode_attention_q8(bf, bf, codes, codes, scale, scale, bt, cl, 16, 0.1)
    with pytest.raises(TypeError, match="int8"):
        B._q8_cache(-2, bf, bf, scale, scale, bt, cl)


def test_copies(B):
    one = (B.pkv_q8_cache * 2)(q8(B), q8(B, kind=1))

    def call(caches=one, layers=2, pairs=FAKE, n=3, d=desc(B), tables=FAKE, seqs=2, bmap=FAKE, rows=FAKE):
        return B.lib().paged_kv_compact_q8(ctypes.addressof(caches) if caches is not None else None, layers, pairs, rows, n,
                                           tables, seqs, 4, bmap, ctypes.byref(d) if d else None, None)

    assert call(caches=None) == -1 and call(d=None) == -1 and call(layers=-1) == -2 and call(n=-1) == -2 and call(seqs=-1) == -2
    assert call(pairs=None) == -1 and call(tables=None) == -1 and call(bmap=None) == -1
    assert call(pairs=ODD) == -5 and call(rows=ctypes.c_void_p((1 << 20) + 2)) == -5
    assert call(d=desc(B, d=96)) == -3 and call(n=1 << 40) == -3
    assert call(caches=(B.pkv_q8_cache * 2)(q8(B), q8(B, ks=None))) == -1
    assert call(n=0, seqs=0) == 0 and call(layers=0, seqs=0) == 0
    assert B.lib().paged_kv_copy_blocks_q8(ctypes.addressof(one), 2, FAKE, None, 0, ctypes.byref(desc(B)), None) == 0


def test_the_binding_names_what_is_wrong_with_copies(B):
    codes, scale, pairs = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.paged_kv_copy_blocks_q8(codes, codes, scale, scale, pairs)
    with pytest.raises(ValueError, match="shorter"):
        B.paged_kv_copy_blocks_q8([codes, codes], [codes], [scale] * 2, [scale] * 2, pairs)
    with pytest.raises(ValueError, match="no layers"):
        B.paged_kv_compact_q8([], [], [], [], pairs)
    with pytest.raises(ValueError, match="in front"):
        B.paged_kv_copy_blocks_q8(codes[None], codes, scale, scale, pairs)
    with pytest.raises(TypeError, match="alike"):
        B.paged_kv_copy_blocks_q8(codes, [codes], [scale], [scale], pairs)
    with pytest.raises(TypeError, match="int8"):
        B.paged_kv_compact_q8(codes.float(), codes, scale, scale, pairs)


def test_packed_calls(B):
    """pkv_call_q8 refuses what its calls refuse, and counts that do not fit their types."""
    lead = dict(k=1 << 20, v=1 << 20, ks=1 << 20, vs=1 << 20, kind=1, nb=64, bs=16, hkv=2, d=64, bt=1 << 20, m=8, cl=1 << 20,
                b=2, stream=0)

    def call(what, fmt, *rest, **changed):
        words = struct.pack("14q" + fmt, *dict(lead, **changed).values(), *rest)
        return B.lib().pkv_call_q8(what, words)

    rows = (1 << 20, 1 << 20, 128, 128, 1 << 20, 8, 4)
    decode = (1 << 20, 1 << 20, 100, 8, 0.125, 0, 0)
    assert B.lib().pkv_call_q8(0, None) == -1 and call(7, "7q", *rows) == -3 and call(-1, "7q", *rows) == -3
    for what in (0, 1):
        assert call(what, "7q", *rows, k=0) == -1 and call(what, "7q", *rows, d=96) == -3 and call(what, "7q", *rows, kind=5) == -3
        assert call(what, "7q", *rows, k=(1 << 20) + 4) == -5 and call(what, "7q", *rows, m=0) == -2
        assert call(what, "7q", *rows[:6], 1 << 40) == -2 and call(what, "7q", *rows, b=1 << 33) == -2
        assert call(what, "7q", *rows[:5], 0, 4) == 0
    assert call(3, "4qd2q", *decode) == -4 and call(3, "4qd2q", *decode, b=0) == 0
    assert call(3, "4qd2q", *decode[:3], 9, *decode[4:]) == -2
    assert call(4, "4qd2q3q", *decode, 8, 1 << 20, 4) == -4 and call(4, "4qd2q3q", *decode, 0, 1 << 20, 4) == 0
    assert call(5, "4qd2q4q", *decode, 1 << 20, 1 << 20, 128, 128) == -4
    assert call(6, "4qd2q4q7q", *decode, 1 << 20, 1 << 20, 128, 128, 512, 1 << 20, 0, 1 << 20, 100, 8, 1) == -3
