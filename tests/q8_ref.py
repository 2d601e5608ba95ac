"""The 8-bit cache's definitions in plain torch, for the tests: the quantising write and the
reading back in fp32 with each operation rounded once (bit for bit), attention in fp64.  Divisors
are tensors: by a Python number, torch on the GPU multiplies with its rounded reciprocal."""

import math

import torch

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
KINDS = [torch.int8, torch.float8_e4m3fn]


def encode(x, dtype):
    """Codes of fp32 values in units of the scale."""
    if dtype is torch.int8:
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


def write(codes, scale, rows, table, begin):
    """rows [n, Hkv, D] bf16 go to positions begin .. of the pages `table` (a list); in place."""
    n, bs = rows.shape[0], codes.shape[2]
    top = TOP[codes.dtype]
    for lo in range(begin // bs * bs, begin + n if n else 0, bs):
        hi, first = min(lo + bs, begin + n), max(lo, begin)
        page = table[lo // bs]
        x = rows[first - begin:hi - begin].float()
        for h in range(codes.shape[1]):
            old = scale[page, h].clone() if first > lo else torch.zeros((), device=scale.device)
            xh = x[:, h]
            if not torch.isfinite(xh).all() or torch.isnan(old):
                scale[page, h] = math.nan
                bits(codes)[page, h, first - lo:hi - lo] = bits(encode(xh * math.nan, codes.dtype).nan_to_num()
                                                               if codes.dtype is torch.int8 else
                                                               encode(xh * math.nan, codes.dtype))
                continue
            m = xh.abs().max()
            need = torch.maximum(m / torch.full_like(m, top), torch.full_like(m, 2.0 ** -126)) if m > 0 else torch.zeros_like(m)
            to = torch.maximum(old, need)
            unit = to if to > 0 else torch.ones_like(to)
            if to > old and first > lo:
                held = codes[page, h, :first - lo].float() * old
                bits(codes)[page, h, :first - lo] = bits(encode(held / unit, codes.dtype))
            bits(codes)[page, h, first - lo:hi - lo] = bits(encode(xh / unit, codes.dtype))
            scale[page, h] = to


def values(codes, scale, table, lo, hi, dtype=torch.float32):
    """Positions lo .. hi-1 of the pages `table`: [hi - lo, Hkv, D]."""
    bs = codes.shape[2]
    at = torch.tensor(table[lo // bs:-(-hi // bs)], dtype=torch.long, device=codes.device)
    x = bits(codes)[at].view(codes.dtype).to(dtype) * scale[at].to(dtype)[..., None, None]
    x = x.permute(0, 2, 1, 3).reshape(-1, codes.shape[1], codes.shape[3])
    return x[lo - lo // bs * bs:][:hi - lo]


def rotate(x, cos_sin, pos, r, neox):
    """x [T, H, D] bf16 at positions pos: fp32, each product and sum rounded once, then bf16."""
    y = x.clone()
    h = r // 2
    cos, sin = cos_sin[pos][:, None, :h], cos_sin[pos][:, None, h:]
    a, b = ((x[..., :h], x[..., h:r]) if neox else (x[..., 0:r:2], x[..., 1:r:2]))
    a, b = a.float(), b.float()
    na, nb = (a * cos - b * sin).to(torch.bfloat16), (b * cos + a * sin).to(torch.bfloat16)
    if neox:
        y[..., :h], y[..., h:r] = na, nb
    else:
        y[..., 0:r:2], y[..., 1:r:2] = na, nb
    return y


def attention(q, k, v, scale, seen=None):
    """q [n, Hq, D] over k, v [L, Hkv, D] in fp64; seen [n, L]: which keys a row sees.  Returns the
    output and sum p |v|, what a relative error of the weights multiplies."""
    q, k, v = q.double(), k.double(), v.double()
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    if k.shape[0] == 0:
        return out, mag
    for h in range(hq):
        x = q[:, h] @ k[:, h // g].T * scale
        if seen is not None:
            x = x.masked_fill(~seen, -math.inf)
        p = torch.softmax(x, -1)
        out[:, h] = p @ v[:, h // g]
        mag[:, h] = p @ v[:, h // g].abs()
    return out, mag


def pools(nb, hkv, bs, d, dtype, gen, dev):
    """Codes of normal values with scales as if their largest were about 3.5."""
    out = []
    for _ in range(2):
        x = torch.randn(nb, hkv, bs, d, generator=gen)
        x = x * (36.0 if dtype is torch.int8 else 128.0)
        s = (0.85 + 0.3 * torch.rand(nb, hkv, generator=gen)) * (3.5 / TOP[dtype])
        out += [encode(x, dtype).to(dev), s.to(dev)]
    return out[0], out[2], out[1], out[3]  # k, v, k_scale, v_scale
