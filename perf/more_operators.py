"""Cases of the 8-bit paged cache: its quantising write, its reading back, and the attention over it.

A cache held in 8 bits keeps, beside the codes [num_blocks, Hkv, block_size, D] (int8, or e4m3
floats), one fp32 scale for each block and kv head, [num_blocks, Hkv]; a code stands for
code * scale.  Four operators, each in a plain form (elementary torch operations, 32 bits,
rounded once at the end) and, where ``own`` is true, through the library's binding:

* ``write``   paged_kv_write_q8, paged_kv_write_rope_q8: each sequence's newest tokens
              quantised into its pages; a page whose scale has to grow has the rows that it
              held rounded anew.  The pass reads the rows of the touched pages back;
* ``read``    paged_kv_read_q8: tokens of the cache as bf16 rows, packed;
* ``decode``  paged_decode_attention_q8: one query token per sequence;
* ``prefill`` paged_prefill_attention_q8: causal attention of each sequence's newest tokens.

Lengths and sizes come from the case alone, values from the seed.
"""

import math
import random

import torch

own = False


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the next token of eight chats (latency counts)
        dict(name="write 8 tokens", op="write", kind="int8", seqs=8, hq=32, hkv=8, d=64, bs=16,
             new_lo=1, new_hi=1, past_lo=0, past_hi=2000, rope=0),
        # a continuous-batching step: positions rotated, part of the head, on the way in
        dict(name="write 256 tokens rotated", op="write", kind="e4m3", seqs=256, hq=24, hkv=8, d=128,
             bs=16, new_lo=1, new_hi=1, past_lo=15, past_hi=4000, rope=64),
        # chunks of prompts of many lengths, some behind tokens that are cached already
        dict(name="write 16 ragged", op="write", kind="e4m3", seqs=16, hq=24, hkv=8, d=128, bs=16,
             new_lo=1, new_hi=4096, past_lo=0, past_hi=100, rope=0),
        # one short context handed on as bf16 rows (latency counts)
        dict(name="read 1 x 300", op="read", kind="int8", seqs=1, hkv=8, d=64, bs=16, lo=300, hi=300),
        # the contexts of a batch
        dict(name="read 16 ragged", op="read", kind="e4m3", seqs=16, hkv=8, d=128, bs=32, lo=1, hi=8192),
        # one short chat (latency counts)
        dict(name="decode 1 x 128", op="decode", kind="int8", seqs=1, hq=32, hkv=8, d=64, bs=16,
             lo=128, hi=128),
        # sixteen chats
        dict(name="decode 16 x 2048", op="decode", kind="e4m3", seqs=16, hq=32, hkv=8, d=64, bs=16,
             lo=2048, hi=2048),
        # a batch of many lengths
        dict(name="decode 64 ragged", op="decode", kind="e4m3", seqs=64, hq=24, hkv=8, d=128, bs=16,
             lo=128, hi=4096),
        # a continuous-batching step: most contexts short, some long
        dict(name="decode 256 short and long", op="decode", kind="int8", seqs=256, hq=32, hkv=4, d=64,
             bs=16, lo=16, hi=8192),
        # four long documents
        dict(name="decode 4 x 32768", op="decode", kind="int8", seqs=4, hq=24, hkv=8, d=128, bs=32,
             lo=32768, hi=32768),
        # a few draft tokens of each chat, checked at once
        dict(name="prefill 8 x 5", op="prefill", kind="int8", seqs=8, hq=32, hkv=8, d=64, bs=16,
             new_lo=5, new_hi=5, past_lo=100, past_hi=2000),
        # the next chunks of long prompts
        dict(name="prefill 4 chunks", op="prefill", kind="e4m3", seqs=4, hq=24, hkv=8, d=128, bs=16,
             new_lo=100, new_hi=2048, past_lo=0, past_hi=6000),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "decode", "decode", "decode", "prefill"])
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
    c = dict(op=op, kind=rng.choice(["int8", "e4m3"]), hkv=hkv, d=rng.choice([64, 128]),
             bs=rng.choice([8, 16, 16, 32, 64, 128, 256]))
    if op == "write":
        c.update(hq=hkv * g, rope=rng.choice([0, 0, 16, 32, c["d"]]))
        if rng.random() < 0.5:
            c.update(seqs=_log(rng, 1, 256), new_lo=1, new_hi=1, past_lo=0, past_hi=_log(rng, 1, 4000))
        else:
            c.update(seqs=_log(rng, 1, 16), new_hi=_log(rng, 1, 4096), past_lo=0, past_hi=_log(rng, 1, 200))
            c["new_lo"] = rng.randint(0, c["new_hi"])
    elif op == "read":
        c["seqs"] = _log(rng, 1, 64)
        c["hi"] = _log(rng, 1, min(8192, 16 * 8192 // c["seqs"]))
        c["lo"] = rng.randint(0, c["hi"])
    elif op == "decode":
        c.update(hq=hkv * g, seqs=_log(rng, 1, 256))
        c["hi"] = _log(rng, 1, min(65536, 4 * 32768 * 8 * 128 // (c["seqs"] * hkv * c["d"])))
        c["lo"] = rng.randint(0, c["hi"])
    else:
        c.update(hq=hkv * g, seqs=_log(rng, 1, 8), past_lo=0, past_hi=_log(rng, 1, 6000))
        c["new_hi"] = _log(rng, 1, min(2048, 4 * 2048 // c["seqs"]))
        c["new_lo"] = rng.randint(0, c["new_hi"])
    return c


def _lengths(c):
    """(context lengths, newest tokens among them): of the case alone, the same for every seed."""
    rng = random.Random("%s" % sorted((k, v) for k, v in c.items() if k != "name"))
    if c["op"] in ("read", "decode"):
        if c["lo"] > 0 and c["hi"] > 64 * c["lo"]:  # most short, some long
            lens = [_log(rng, c["lo"], c["hi"]) for _ in range(c["seqs"])]
        else:
            lens = [rng.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
        lens[rng.randrange(c["seqs"])] = c["hi"]
        return lens, lens
    new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    new[rng.randrange(c["seqs"])] = c["new_hi"]
    return [n + rng.randint(c["past_lo"], c["past_hi"]) for n in new], new


# --------------------------------------------------------------------------- inputs

def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32).to(torch.bfloat16)


def _pool(c, nb, gen):
    """Codes of normal values and the scales of pages whose largest value is about 3.5."""
    x = torch.empty((nb, c["hkv"], c["bs"], c["d"]), dtype=torch.bfloat16, device=gen.device)
    x.normal_(generator=gen)
    if c["kind"] == "int8":
        codes, top = x.mul_(36.0).round_().clamp_(-127, 127).to(torch.int8), 127.0
    else:
        codes, top = x.mul_(128.0).clamp_(-448, 448).to(torch.float8_e4m3fn), 448.0
    s = 0.85 + 0.3 * torch.rand((nb, c["hkv"]), generator=gen, device=gen.device)
    return codes, s * (3.5 / top)


def _start(counts, dev):
    return torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device=dev)


def prepare(case, seed):
    c, dev = case, _dev()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    lens, new = _lengths(c)
    bs, seqs = c["bs"], c["seqs"]
    need = sum(-(-n // bs) for n in lens)
    nb = need + need // 4 + 1
    maxb = max(1, max(-(-n // bs) for n in lens))
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(int(seed))).to(torch.int32)
    tables = torch.full((seqs, maxb), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // bs)
        tables[b, :m] = perm[at:at + m]
        at += m
    k, ks = _pool(c, nb, gen)
    v, vs = _pool(c, nb, gen)
    s = dict(op=c["op"], bs=bs, k=k, v=v, ks=ks, vs=vs, tables=tables.to(dev),
             lens=torch.tensor(lens, dtype=torch.int32, device=dev), max_len=max(lens))
    hkv, d = c["hkv"], c["d"]
    bf = dict(dtype=torch.bfloat16, device=dev)
    if c["op"] == "decode":
        q = _randn((seqs, c["hq"], d), gen)
        return dict(s, q=q, out=torch.empty_like(q), scale=d ** -0.5)
    t = sum(new)
    s.update(start=_start(new, dev), max_new=max(new))
    if c["op"] == "read":
        return dict(s, k_out=torch.empty((t, hkv, d), **bf), v_out=torch.empty((t, hkv, d), **bf))
    if c["op"] == "prefill":
        q = _randn((t, c["hq"], d), gen)
        return dict(s, q=q, out=torch.empty_like(q), scale=d ** -0.5)
    # the rows of one projection: q heads, then k heads, then v heads
    q, kn, vn = _randn((t, c["hq"] + 2 * hkv, d), gen).split([c["hq"], hkv, hkv], dim=1)
    # the rows of the touched pages: the new tokens and those that share their first page
    held = [n + ((m - n) % bs if n else 0) for m, n in zip(lens, new)]
    s.update(kn=kn, vn=vn, back=_start(held, dev), max_back=max(held), rope=c["rope"],
             k_out=torch.empty((sum(held), hkv, d), **bf), v_out=torch.empty((sum(held), hkv, d), **bf))
    if c["rope"]:
        r = c["rope"]
        freq = 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device=dev) / r)
        ang = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * freq
        s.update(q=q, q_out=torch.empty((t, c["hq"], d), **bf),
                 cos_sin=torch.cat((ang.cos(), ang.sin()), 1).float())
    return s


# --------------------------------------------------------------------------- one pass

def _rows(codes, scale, tables, m):
    """Pages 0 .. m-1 of every sequence, as values in 32 bits: [B, Hkv, m * bs, D]."""
    _, hkv, bs, d = codes.shape
    at = tables[:, :m].clamp(min=0).long()
    x = codes.view(torch.uint8)[at].view(codes.dtype).float() * scale[at][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(at.shape[0], hkv, m * bs, d)


def _where(start, lens, width):
    """Of each sequence's last start[b + 1] - start[b] tokens: the positions [B, width], and
    whether there is one."""
    n = (start[1:] - start[:-1]).long()
    i = torch.arange(width, device=start.device)[None, :]
    return lens.long()[:, None] - n[:, None] + i, i < n[:, None]


def _back(s, start, width):
    pos, here = _where(start, s["lens"], width)
    at = pos.clamp(min=0)
    page = torch.gather(s["tables"], 1, (at // s["bs"]).clamp(max=s["tables"].shape[1] - 1)).clamp(min=0).long()[here]
    row = (at % s["bs"])[here]
    return tuple((codes.view(torch.uint8)[page, :, row].view(codes.dtype).float()
                  * scale[page][:, :, None]).to(torch.bfloat16)
                 for codes, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])))


def _rotate(x, s, pos):
    """Pairs (e, e + r/2) of the first r coordinates, products and sums in 32 bits."""
    r = s["rope"]
    h = r // 2
    cos, sin = s["cos_sin"][pos][:, None, :h], s["cos_sin"][pos][:, None, h:]
    a, b, rest = x[..., :h].float(), x[..., h:r].float(), x[..., r:].float()
    return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1).to(torch.bfloat16)


def _round(x, dtype):
    """Codes of x, which is in units of the scale."""
    if dtype == torch.int8:
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _plain_write(s):
    bs, lens, tables = s["bs"], s["lens"].long(), s["tables"]
    n = (s["start"][1:] - s["start"][:-1]).long()
    pos, here = _where(s["start"], s["lens"], s["max_new"])
    kn, out = s["kn"], {}
    if s["rope"]:
        kn = _rotate(kn, s, pos[here])
        out["q"] = _rotate(s["q"], s, pos[here])
    first = (lens - n) // bs  # first page touched
    m = (s["max_new"] + bs - 2) // bs + 1
    page = first[:, None] + torch.arange(m, device=lens.device)  # [B, m]
    p = page[:, :, None] * bs + torch.arange(bs, device=lens.device)  # [B, m, bs] positions
    begin = (lens - n)[:, None, None]
    fresh = (p >= begin) & (p < lens[:, None, None])
    held = (p < begin) & (n > 0)[:, None, None]
    live = fresh.any(-1)  # [B, m] pages with a new row
    phys = torch.gather(tables, 1, page.clamp(max=tables.shape[1] - 1)).clamp(min=0).long()[live]
    src = (s["start"][:-1].long()[:, None, None] + p - begin).clamp(0, max(0, kn.shape[0] - 1))[live]
    fresh, held = fresh[live][:, None, :, None], held[live][:, None, :, None]
    for name, codes, scale, x in (("k", s["k"], s["ks"], kn), ("v", s["v"], s["vs"], s["vn"])):
        top = 127.0 if codes.dtype == torch.int8 else 448.0
        rows = torch.where(fresh, x[src].permute(0, 2, 1, 3).float(), 0.0)  # [P, Hkv, bs, D]
        need = rows.abs().amax((2, 3))
        old = torch.where(held.any(2)[..., 0], scale[phys], 0.0)  # a page that begins here has none
        to = torch.maximum(old, torch.where(need > 0, (need / torch.full_like(need, top)).clamp(min=2.0 ** -126), 0.0))
        unit = torch.where(to > 0, to, 1.0)[..., None, None]
        was = codes.view(torch.uint8)[phys].view(codes.dtype)
        again = _round(was.float() * old[..., None, None] / unit, codes.dtype)
        grown = (to > old)[..., None, None] & held
        now = torch.where(fresh, _round(rows / unit, codes.dtype).view(torch.uint8),
                          torch.where(grown, again.view(torch.uint8), was.view(torch.uint8)))
        codes.view(torch.uint8)[phys] = now
        scale[phys] = to
    k, v = _back(s, s["back"], s["max_back"])
    return dict(out, k=k, v=v, k_scale=s["ks"], v_scale=s["vs"])


def _softmax_rows(x):
    """Softmax of the last axis whose masked places hold -inf; a row with none left gives zeros."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    n = e.sum(-1, keepdim=True)
    return e / torch.where(n == 0, 1.0, n)


def _plain_attention(s, q, pos):
    """q [B, n, Hq, D] at positions pos [B, n], each over the positions up to its own."""
    b, n, hq, d = q.shape
    m = -(-max(1, s["max_len"]) // s["bs"])
    kk, vv = _rows(s["k"], s["ks"], s["tables"], m), _rows(s["v"], s["vs"], s["tables"], m)
    hkv, g, w = kk.shape[1], hq // kk.shape[1], kk.shape[2]
    i = torch.arange(w, device=q.device)
    vv = torch.where((i[None, :] < s["lens"][:, None])[:, None, :, None], vv, 0.0)
    x = q.float().view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    x = (torch.matmul(x, kk.transpose(2, 3)) * s["scale"]).view(b, hkv, g, n, w)
    x = x.masked_fill_((i[None, None, :] > pos[:, :, None])[:, None, None], -math.inf)
    x = torch.matmul(_softmax_rows(x).view(b, hkv, g * n, w), vv).view(b, hkv, g, n, d)
    return x.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d).to(torch.bfloat16)


def _plain_prefill(s):
    q = s["q"]
    pos, here = _where(s["start"], s["lens"], s["max_new"])
    i = torch.arange(s["max_new"], device=q.device)
    at = (s["start"][:-1].long()[:, None] + i[None, :]).clamp(max=max(0, q.shape[0] - 1))
    return _plain_attention(s, q[at], pos)[here]


def run(state):
    s = state
    if own:
        from paged_kv_decode_mapping_gb300 import binding as B
        cache = (s["k"], s["v"], s["ks"], s["vs"])
        if s["op"] == "write":
            out = {}
            if s["rope"]:
                B.paged_kv_write_rope_q8(s["kn"], s["vn"], s["cos_sin"], *cache, s["tables"], s["lens"],
                                         s["start"], s["max_new"], q=s["q"], q_out=s["q_out"],
                                         rotary_dim=s["rope"])
                out["q"] = s["q_out"]
            else:
                B.paged_kv_write_q8(s["kn"], s["vn"], *cache, s["tables"], s["lens"], s["start"],
                                    s["max_new"])
            B.paged_kv_read_q8(s["k_out"], s["v_out"], *cache, s["tables"], s["lens"], s["back"],
                               s["max_back"])
            return dict(out, k=s["k_out"], v=s["v_out"], k_scale=s["ks"], v_scale=s["vs"])
        if s["op"] == "read":
            B.paged_kv_read_q8(s["k_out"], s["v_out"], *cache, s["tables"], s["lens"], s["start"],
                               s["max_new"])
            return s["k_out"], s["v_out"]
        hq, hkv, d = s["q"].shape[1], s["k"].shape[1], s["k"].shape[3]
        if s["op"] == "decode":
            if "ws" not in s:  # zeroed once, kept beside the caches for every later step
                s["ws"] = torch.zeros(B.paged_decode_q8_workspace_size(s["q"].shape[0], hq, hkv, d, s["max_len"]),
                                      dtype=torch.uint8, device=s["q"].device)
            B.paged_decode_attention_q8(s["out"], s["q"], *cache, s["tables"], s["lens"], s["max_len"],
                                        s["scale"], workspace=s["ws"])
            return s["out"]
        if "ws" not in s:
            s["ws"] = torch.empty(B.paged_prefill_q8_workspace_size(s["tables"].shape[0], hkv, d, s["bs"], s["max_len"]),
                                  dtype=torch.uint8, device=s["q"].device)
        B.paged_prefill_attention_q8(s["out"], s["q"], *cache, s["tables"], s["lens"], s["max_len"],
                                     s["start"], s["max_new"], s["scale"], workspace=s["ws"])
        return s["out"]
    if s["op"] == "write":
        return _plain_write(s)
    if s["op"] == "read":
        return _back(s, s["start"], s["max_new"])
    if s["op"] == "decode":
        return _plain_attention(s, s["q"][:, None], s["lens"].long()[:, None] - 1)[:, 0]
    return _plain_prefill(s)


# --------------------------------------------------------------------------- floors

def work(case):
    c = case
    lens, new = _lengths(c)
    row = c["hkv"] * c["d"]  # elements of one token's K (or V)
    pages = sum(-(-n // c["bs"]) for n in lens)
    if c["op"] == "write":
        held = sum(n + ((m - n) % c["bs"] if n else 0) for m, n in zip(lens, new))
        b = sum(new) * row * (4 + 2) + held * row * (2 + 4)
        if c["rope"]:
            b += 4 * sum(new) * c["hq"] * c["d"]
        return {"bytes": b, "flops": 0}
    if c["op"] == "read":
        return {"bytes": sum(lens) * row * 6 + pages * (4 + 8 * c["hkv"]), "flops": 0}
    cache = sum(lens) * row * 2 + pages * (4 + 8 * c["hkv"])
    if c["op"] == "decode":
        return {"bytes": cache + 4 * c["seqs"] * c["hq"] * c["d"], "flops": 4 * sum(lens) * c["hq"] * c["d"]}
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for m, n in zip(lens, new))
    return {"bytes": cache + 4 * sum(new) * c["hq"] * c["d"], "flops": 4 * pairs * c["hq"] * c["d"]}


# --------------------------------------------------------------------------- in 64 bits

def _exact_codes(x, kind):
    """The nearest value that 8 bits hold, halves to even."""
    if kind == "int8":
        return torch.round(x).clamp(-127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    lens, new = _lengths(c)
    bs, hkv, d, tables = c["bs"], c["hkv"], c["d"], s["tables"].tolist()
    start = s.get("start", s["lens"]).tolist()
    pools = [[s["k"], s["ks"]], [s["v"], s["vs"]]]

    def held(pool, b, lo, hi):
        """Positions lo .. hi-1 of sequence b, [hi - lo, Hkv, D]."""
        codes, scale = pool
        at = torch.tensor(tables[b][lo // bs:-(-hi // bs)], dtype=torch.long, device=codes.device)
        x = codes.view(torch.uint8)[at].view(codes.dtype).double() * scale[at].double()[..., None, None]
        return x.permute(0, 2, 1, 3).reshape(-1, hkv, d)[lo - lo // bs * bs:][:hi - lo]

    if c["op"] == "read":
        return tuple(torch.cat([held(p, b, 0, n) for b, n in enumerate(lens)]) for p in pools)
    if c["op"] == "write":
        top = 127.0 if c["kind"] == "int8" else 448.0
        kn, vn, out = s["kn"].double(), s["vn"].double(), {}
        if c["rope"]:
            r = c["rope"]
            at = torch.cat([torch.arange(m - n, m) for m, n in zip(lens, new)]).to(kn.device)
            cos, sin = s["cos_sin"].double()[at].unsqueeze(1).split([r // 2, r // 2], -1)

            def turn(x):
                y = x.clone()
                y[..., :r // 2] = x[..., :r // 2] * cos - x[..., r // 2:r] * sin
                y[..., r // 2:r] = x[..., r // 2:r] * cos + x[..., :r // 2] * sin
                return y
            out["q"] = turn(s["q"].double())
            kn = turn(kn).to(torch.bfloat16).double()
        scales = [s["ks"].double(), s["vs"].double()]
        back = [[], []]
        if sum(-(-n // bs) + 1 for n in new) > 6000:
            return None
        for b, (m, n) in enumerate(zip(lens, new)):
            for lo in range((m - n) // bs * bs, m if n else 0, bs):
                hi, first = min(lo + bs, m), max(lo, m - n)
                for i, x in enumerate((kn, vn)):
                    rows = x[start[b] + first - (m - n):start[b] + hi - (m - n)]
                    page = tables[b][lo // bs]
                    old = scales[i][page] if first > lo else torch.zeros_like(scales[i][page])
                    to = torch.maximum(old, rows.abs().amax((0, 2)) / top)
                    unit = torch.where(to > 0, to, 1.0)[:, None]
                    if first > lo:
                        before = held(pools[i], b, lo, first)
                        again = _exact_codes(before / unit, c["kind"]) * unit
                        back[i].append(torch.where((to > old)[:, None], again, before))
                    back[i].append(_exact_codes(rows / unit, c["kind"]) * unit)
                    scales[i][page] = to
        k, v = (torch.cat(x) if x else torch.zeros((0, hkv, d), dtype=torch.float64, device=kn.device)
                for x in back)
        return dict(out, k=k, v=v, k_scale=scales[0], v_scale=scales[1])
    if work(c)["flops"] > 2e12:
        return None
    q = s["q"].double()
    g = c["hq"] // hkv
    out = torch.zeros_like(q)
    for b, (m, n) in enumerate(zip(lens, new)):
        if m == 0:
            continue
        lo, hi = (b, b + 1) if c["op"] == "decode" else (start[b], start[b + 1])
        kk, vv = held(pools[0], b, 0, m), held(pools[1], b, 0, m)
        see = torch.arange(m, device=q.device)[None, :] <= torch.arange(m - (hi - lo), m, device=q.device)[:, None]
        for h in range(c["hq"]):
            x = (q[lo:hi, h] @ kk[:, h // g].T * s["scale"]).masked_fill(~see, -math.inf)
            out[lo:hi, h] = torch.softmax(x, -1) @ vv[:, h // g]
    return out
