"""Cases of the page operators, the shared-prefix decode and the packed prompt attention.

Four operators of the paged KV cache, each in a plain form (elementary torch operations,
32 bits, rounded once at the end) and, where ``own`` is true, through the library's binding:

* ``copy``    paged_kv_copy_blocks: pages copied to other pages of the same pool, all layers
              in one call (the copy-on-write of forked sequences), whole or their first rows;
* ``compact`` paged_kv_compact: pages moved into free pages, and the block tables rewritten;
* ``shared``  paged_decode_shared_prefix_attention: one query token per sequence over the
              paged cache, where the sequences of a group share a long prefix's pages;
* ``prompt``  prompt_attention: causal attention of whole prompts packed one after another,
              K and V straight from the projections (no pages).

Lengths and sizes come from the case alone, values from the seed.
"""

import math
import random

import torch

own = False


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # five forked sequences write their next token: the last, partly filled page of each
        # is copied in all 16 layers (latency counts)
        dict(name="copy 5 last pages", op="copy", layers=16, num_blocks=256, hkv=8, d=64, bs=16,
             pairs=5, partial=True),
        # 256 beams change their parents at once: one full page each, in all 28 layers
        dict(name="copy 256 pages", op="copy", layers=28, num_blocks=1024, hkv=8, d=128, bs=16,
             pairs=256, partial=False),
        # a small pool after a few sequences have left: single layer
        dict(name="compact 61 moves", op="compact", layers=1, num_blocks=2560, hkv=8, d=64, bs=16,
             moves=61, seqs=16, max_blocks=128),
        # a continuous-batching pool after hours: a fifth of its pages move, in four layers
        dict(name="compact 2900 moves", op="compact", layers=4, num_blocks=18000, hkv=4, d=64,
             bs=16, moves=2900, seqs=256, max_blocks=512),
        # three samples of one request behind a short system prompt (latency counts)
        dict(name="shared 3 x 512", op="shared", seqs=3, hq=32, hkv=8, d=64, bs=16, groups=1,
             prefix_lo=512, prefix_hi=512, suffix_lo=1, suffix_hi=64),
        # sixteen chats behind one system prompt
        dict(name="shared 16 x 2048", op="shared", seqs=16, hq=32, hkv=8, d=64, bs=16, groups=1,
             prefix_lo=2048, prefix_hi=2048, suffix_lo=1, suffix_hi=512),
        # 64 questions about one document
        dict(name="shared 64 x 8192", op="shared", seqs=64, hq=24, hkv=8, d=128, bs=16, groups=1,
             prefix_lo=8192, prefix_hi=8192, suffix_lo=1, suffix_hi=1024),
        # several tenants, each with its own system prompt of its own length
        dict(name="shared 6 groups", op="shared", seqs=97, hq=32, hkv=4, d=64, bs=16, groups=6,
             prefix_lo=1000, prefix_hi=4096, suffix_lo=0, suffix_hi=300),
        # parallel samples over a book
        dict(name="shared 16 x 65536", op="shared", seqs=16, hq=24, hkv=8, d=128, bs=32, groups=1,
             prefix_lo=65536, prefix_hi=65536, suffix_lo=1, suffix_hi=256),
        # the first prompt of an idle server (latency counts)
        dict(name="prompt 1 x 100", op="prompt", seqs=1, hq=32, hkv=8, d=64, lo=100, hi=100,
             fused=True),
        # prompts of many lengths packed into one pass, rows of a fused projection
        dict(name="prompt 16 ragged", op="prompt", seqs=16, hq=24, hkv=8, d=128, lo=1, hi=2048,
             fused=True),
        # two long documents
        dict(name="prompt 2 long", op="prompt", seqs=2, hq=24, hkv=8, d=128, lo=5000, hi=8192,
             fused=False),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["copy", "compact", "shared", "shared", "prompt", "prompt"])
    if op in ("copy", "compact"):
        c = dict(op=op, layers=_log(rng, 1, 32), hkv=rng.choice([1, 2, 4, 8]),
                 d=rng.choice([64, 64, 80, 128, 128]), bs=rng.choice([8, 16, 16, 32, 64]))
        page = 2 * c["layers"] * c["hkv"] * c["bs"] * c["d"] * 2
        most = max(1, min(4000, 470_000_000 // page))
        n = _log(rng, 1, most)
        c["num_blocks"] = 2 * n + _log(rng, 1, max(1, n))
        if op == "copy":
            c.update(pairs=n, partial=rng.random() < 0.5)
        else:
            c.update(moves=n, seqs=_log(rng, 1, 256), max_blocks=_log(rng, 1, 512))
        return c
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 128])
    if op == "shared":
        seqs = _log(rng, 1, 128)
        top = max(64, min(65536, 16 * 65536 * 8 * 128 // (seqs * hkv * d)))
        hi = _log(rng, 16, top)
        return dict(op=op, seqs=seqs, hq=hkv * g, hkv=hkv, d=d, bs=rng.choice([8, 16, 32, 64]),
                    groups=_log(rng, 1, max(1, min(8, seqs))), prefix_lo=max(1, hi // 2),
                    prefix_hi=hi, suffix_lo=rng.choice([0, 1]), suffix_hi=_log(rng, 1, 1024))
    seqs = _log(rng, 1, 24)
    top = int(min(8192, math.sqrt(2 * 8192 * 8192 * 24 / (seqs * hkv * g))))
    hi = _log(rng, 1, top)
    return dict(op=op, seqs=seqs, hq=hkv * g, hkv=hkv, d=d, lo=rng.randint(0, hi), hi=hi,
                fused=rng.random() < 0.5)


def _lengths(c):
    """What a case's lengths are: of the case alone (the same for every seed)."""
    rng = random.Random("%s" % sorted((k, v) for k, v in c.items() if k != "name"))
    if c["op"] == "shared":
        cuts = sorted(rng.sample(range(1, c["seqs"]), c["groups"] - 1)) if c["groups"] > 1 else []
        start = [0] + cuts + [c["seqs"]]
        prefix = [rng.randint(c["prefix_lo"], c["prefix_hi"]) for _ in range(c["groups"])]
        suffix = [rng.randint(c["suffix_lo"], c["suffix_hi"]) for _ in range(c["seqs"])]
        return start, prefix, suffix
    lens = [rng.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    lens[rng.randrange(c["seqs"])] = c["hi"]
    return lens


# --------------------------------------------------------------------------- inputs

def _gen(seed, dev):
    return torch.Generator(device=dev).manual_seed(int(seed))


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32).to(torch.bfloat16)


def _pool(c, gen):
    shape = (c["layers"], c["num_blocks"], c["hkv"], c["bs"], c["d"])
    k = torch.empty(shape, dtype=torch.bfloat16, device=gen.device)
    return k.normal_(generator=gen), torch.empty_like(k).normal_(generator=gen)


def prepare(case, seed):
    c, dev = case, _dev()
    gen = _gen(seed, dev)
    if c["op"] == "copy":
        k, v = _pool(c, gen)
        perm = torch.randperm(c["num_blocks"], generator=gen, device=dev)
        n = c["pairs"]
        # destinations are pages of their own; a source may be forked more than once
        src = perm[n:][torch.randint(0, c["num_blocks"] - n, (n,), generator=gen, device=dev)]
        rows = torch.randint(1, c["bs"] + 1, (n,), generator=gen, device=dev).to(torch.int32)
        return dict(op="copy", k=k, v=v, pairs=torch.stack((src, perm[:n]), 1).to(torch.int32).contiguous(),
                    rows=rows if c["partial"] else None)
    if c["op"] == "compact":
        k, v = _pool(c, gen)
        nb, n = c["num_blocks"], c["moves"]
        live = nb - max(n, nb // 5)  # pages in use; below that id, n are free
        low = torch.randperm(live, generator=gen, device=dev)
        high = live + torch.randperm(nb - live, generator=gen, device=dev)
        moves = torch.stack((high[:n], low[:n]), 1).to(torch.int32).contiguous()
        block_map = torch.arange(nb, device=dev, dtype=torch.int32)
        block_map[moves[:, 0].long()] = moves[:, 1]
        used = torch.cat((low[n:], high[:n])).to(torch.int32)
        pick = torch.randint(0, used.numel(), (c["seqs"], c["max_blocks"]), generator=gen, device=dev)
        tables = used[pick]
        nblk = torch.randint(0, c["max_blocks"] + 1, (c["seqs"], 1), generator=gen, device=dev)
        tables[torch.arange(c["max_blocks"], device=dev)[None, :] >= nblk] = -1
        return dict(op="compact", k=k, v=v, moves=moves, block_map=block_map, tables=tables)
    if c["op"] == "shared":
        start, prefix, suffix = _lengths(c)
        bs = c["bs"]
        # a fork shares the whole pages of its prefix and owns a copy of the last, partial one
        lens = [prefix[g] + suffix[b] for g in range(c["groups"]) for b in range(start[g], start[g + 1])]
        own_blocks = [-(-(lens[b] - prefix[g] // bs * bs) // bs)
                      for g in range(c["groups"]) for b in range(start[g], start[g + 1])]
        need = sum(p // bs for p in prefix) + sum(own_blocks)
        nb = need + need // 4 + 1
        perm = torch.randperm(nb, generator=_gen(seed, "cpu")).to(torch.int32)
        maxb = max(1, max(-(-n // bs) for n in lens))
        tables = torch.full((c["seqs"], maxb), -1, dtype=torch.int32)
        at = 0
        for g in range(c["groups"]):
            sh = prefix[g] // bs
            common = perm[at:at + sh]
            at += sh
            for b in range(start[g], start[g + 1]):
                tables[b, :sh] = common
                tables[b, sh:sh + own_blocks[b]] = perm[at:at + own_blocks[b]]
                at += own_blocks[b]
        q = _randn((c["seqs"], c["hq"], c["d"]), gen)
        k = _randn((nb, c["hkv"], bs, c["d"]), gen)
        v = _randn((nb, c["hkv"], bs, c["d"]), gen)
        i32 = dict(dtype=torch.int32, device=dev)
        return dict(op="shared", q=q, k=k, v=v, tables=tables.to(dev), lens=torch.tensor(lens, **i32),
                    group_start=torch.tensor(start, **i32), prefix=torch.tensor(prefix, **i32),
                    max_prefix=max(prefix), max_suffix=max(lens[b] - prefix[g] // bs * bs for g in range(c["groups"]) for b in range(start[g], start[g + 1])),
                    max_len=max(lens), scale=c["d"] ** -0.5, out=torch.empty_like(q))
    lens = _lengths(c)
    start = [sum(lens[:i]) for i in range(len(lens) + 1)]
    t, hq, hkv, d = start[-1], c["hq"], c["hkv"], c["d"]
    if c["fused"]:  # the rows of one projection: q heads, then k heads, then v heads
        q, k, v = _randn((t, hq + 2 * hkv, d), gen).split([hq, hkv, hkv], dim=1)
    else:
        q, k, v = (_randn((t, h, d), gen) for h in (hq, hkv, hkv))
    return dict(op="prompt", q=q, k=k, v=v, start=torch.tensor(start, dtype=torch.int32, device=dev),
                max_len=max(lens), scale=d ** -0.5,
                out=torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev))


# --------------------------------------------------------------------------- one pass

def _plain_copy(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    rows = s["rows"]
    if rows is None:
        s["k"][:, dst] = s["k"][:, src]
        s["v"][:, dst] = s["v"][:, src]
    else:
        keep = torch.arange(s["k"].shape[3], device=rows.device)[None, :] < rows[:, None]
        keep = keep[None, :, None, :, None]
        s["k"][:, dst] = torch.where(keep, s["k"][:, src], s["k"][:, dst])
        s["v"][:, dst] = torch.where(keep, s["v"][:, src], s["v"][:, dst])
    return s["k"], s["v"]


def _plain_compact(s):
    src, dst = s["moves"][:, 0].long(), s["moves"][:, 1].long()
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    t = s["tables"]
    s["tables"].copy_(torch.where(t >= 0, s["block_map"][t.clamp(min=0).long()], t))
    return s["k"], s["v"], s["tables"]


def _softmax_rows(x):
    """Softmax of the last axis whose masked places hold -inf; a row with none left gives zeros."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    n = e.sum(-1, keepdim=True)
    return e / torch.where(n == 0, 1.0, n)


def _plain_shared(s):
    q, k, v = s["q"].float(), s["k"], s["v"]
    b, hq, d = q.shape
    _, hkv, bs, _ = k.shape
    m = -(-s["max_len"] // bs)
    at = s["tables"][:, :m].clamp(min=0).long()
    kk = k[at].permute(0, 2, 1, 3, 4).reshape(b, hkv, m * bs, d).float()
    vv = v[at].permute(0, 2, 1, 3, 4).reshape(b, hkv, m * bs, d).float()
    seen = torch.arange(m * bs, device=q.device)[None, :] < s["lens"][:, None]
    vv = torch.where(seen[:, None, :, None], vv, 0.0)
    x = torch.matmul(q.view(b, hkv, hq // hkv, d), kk.transpose(2, 3)) * s["scale"]
    x = torch.where(seen[:, None, None, :], x, -math.inf)
    return torch.matmul(_softmax_rows(x), vv).reshape(b, hq, d).to(torch.bfloat16)


def _plain_prompt(s):
    q, k, v, start = s["q"], s["k"], s["v"], s["start"].long()
    t, hq, d = q.shape
    hkv, n, b = k.shape[1], s["max_len"], start.numel() - 1
    i = torch.arange(n, device=q.device)
    lens = start[1:] - start[:-1]
    here = i[None, :] < lens[:, None]
    at = (start[:-1, None] + i[None, :]).clamp(max=max(t - 1, 0))
    qq = q[at].float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    kk = k[at].float().permute(0, 2, 3, 1)[:, :, None]
    vv = torch.where(here[:, :, None, None], v[at].float(), 0.0).permute(0, 2, 1, 3)[:, :, None]
    x = torch.matmul(qq, kk) * s["scale"]
    x = x.masked_fill_((i[None, :] > i[:, None]), -math.inf)
    x = torch.matmul(_softmax_rows(x), vv)
    return x.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)[here].to(torch.bfloat16)


def run(state):
    s = state
    if own:
        from paged_kv_decode_mapping_gb300 import binding as B
        if s["op"] == "copy":
            B.paged_kv_copy_blocks(s["k"], s["v"], s["pairs"], num_tokens=s["rows"])
            return s["k"], s["v"]
        if s["op"] == "compact":
            B.paged_kv_compact(s["k"], s["v"], s["moves"], s["tables"], s["block_map"])
            return s["k"], s["v"], s["tables"]
        if s["op"] == "shared":
            if "ws" not in s:  # zeroed once, kept beside the caches for every later step
                s["ws"] = torch.zeros(B.paged_decode_shared_prefix_workspace_size(
                    s["q"].shape[0], s["q"].shape[1], s["k"].shape[1], s["q"].shape[2],
                    s["prefix"].shape[0], s["max_prefix"], s["max_suffix"]),
                    dtype=torch.uint8, device=s["q"].device)
            B.paged_decode_shared_prefix_attention(
                s["out"], s["q"], s["k"], s["v"], s["tables"], s["lens"], s["group_start"],
                s["prefix"], s["max_prefix"], s["max_suffix"], s["scale"], workspace=s["ws"])
            return s["out"]
        B.prompt_attention(s["out"], s["q"], s["k"], s["v"], s["start"], s["max_len"], s["scale"])
        return s["out"]
    return {"copy": _plain_copy, "compact": _plain_compact, "shared": _plain_shared,
            "prompt": _plain_prompt}[s["op"]](s)


# --------------------------------------------------------------------------- floors

def work(case):
    c = case
    if c["op"] == "copy":
        page = 2 * c["layers"] * c["hkv"] * c["bs"] * c["d"] * 2
        part = (c["bs"] + 1) / (2 * c["bs"]) if c["partial"] else 1.0
        return {"bytes": 2 * page * c["pairs"] * part + 8 * c["pairs"], "flops": 0}
    if c["op"] == "compact":
        page = 2 * c["layers"] * c["hkv"] * c["bs"] * c["d"] * 2
        return {"bytes": 2 * page * c["moves"] + 8 * c["moves"] + 4 * c["num_blocks"]
                + 8 * c["seqs"] * c["max_blocks"], "flops": 0}
    if c["op"] == "shared":
        start, prefix, suffix = _lengths(c)
        shared = [p // c["bs"] * c["bs"] for p in prefix]
        tokens = sum(shared) + sum(suffix)
        pairs = sum(suffix)
        for g, p in enumerate(prefix):
            tokens += (p - shared[g]) * (start[g + 1] - start[g])
            pairs += p * (start[g + 1] - start[g])
        return {"bytes": tokens * c["hkv"] * c["d"] * 4 + 4 * c["seqs"] * c["hq"] * c["d"]
                + 4 * tokens // c["bs"], "flops": 4 * pairs * c["hq"] * c["d"]}
    lens = _lengths(c)
    return {"bytes": 2 * sum(lens) * c["d"] * (2 * c["hq"] + 2 * c["hkv"]),
            "flops": 4 * c["hq"] * c["d"] * sum(n * (n + 1) // 2 for n in lens)}


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("copy", "compact"):
        moves = (s["pairs"] if s["op"] == "copy" else s["moves"]).tolist()
        rows = s["rows"].tolist() if s.get("rows") is not None else [case["bs"]] * len(moves)
        k, v = s["k"], s["v"]
        old = k.clone(), v.clone()
        for (a, b), n in zip(moves, rows):
            k[:, b, :, :n] = old[0][:, a, :, :n]
            v[:, b, :, :n] = old[1][:, a, :, :n]
        if s["op"] == "copy":
            return k, v
        to = dict(moves)
        tables = [[to.get(x, x) for x in row] for row in s["tables"].tolist()]
        return k, v, torch.tensor(tables, dtype=torch.int32, device=k.device)
    q = s["q"].double()
    t, hq, d = q.shape
    out = torch.zeros((t, hq, d), dtype=torch.float64, device=q.device)
    g = hq // case["hkv"]
    if s["op"] == "shared":
        for b, n in enumerate(s["lens"].tolist()):
            if n == 0:
                continue
            at = s["tables"][b, :-(-n // case["bs"])].long()
            for h in range(case["hkv"]):
                kk = s["k"][at, h].reshape(-1, d)[:n].double()
                vv = s["v"][at, h].reshape(-1, d)[:n].double()
                x = q[b, h * g:(h + 1) * g] @ kk.T * s["scale"]
                out[b, h * g:(h + 1) * g] = torch.softmax(x, -1) @ vv
        return out
    start = s["start"].tolist()
    if work(case)["flops"] > 8e12:
        return None
    for lo, hi in zip(start[:-1], start[1:]):
        for h in range(hq):
            kk, vv = s["k"][lo:hi, h // g].double(), s["v"][lo:hi, h // g].double()
            for a in range(lo, hi, 2048):
                z = min(a + 2048, hi)
                x = q[a:z, h] @ kk[:z - lo].T * s["scale"]
                i = torch.arange(a - lo, z - lo, device=q.device)
                x[torch.arange(z - lo, device=q.device)[None, :] > i[:, None]] = -math.inf
                out[a:z, h] = torch.softmax(x, -1) @ vv[:z - lo]
    return out
