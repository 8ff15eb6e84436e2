"""Cases of the operators for long contexts with pictures: rotary positions with several axes on the way into a
paged cache, a 4-bit cache (written, read back, attended to), and decode attention with a sliding window and a
few first tokens that stay visible.

The 4-bit cache ("kv4") is one uint8 tensor (num_blocks, h_kv, block_size * (d + d / 8)).  A (block, head) holds
the K codes [block_size][d / 2], the V codes [block_size][d / 2], a scale byte for every 16 elements of every K row
[block_size][d / 16] and those of V.  Byte i of a row's codes has element 2i in its low four bits and 2i + 1 in its
high ones; the 16-byte chunk c of row r is stored at chunk c ^ (r // 2 % 4) for d = 128 and c ^ (r // 4 % 2) for
d = 64.  A code is sign and e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale byte is the upper byte of a binary16 number.
Sixteen elements with the largest magnitude m have the scale m / 6, at most 10240, rounded to the nearest such byte,
and the codes of x / scale, rounded to nearest; ties go to the even byte and code.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
THETA = 500000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one request, three position axes, enters a 16-bit paged cache: the latency of a decode step
        dict(name="axes_1_token", op="append", cache="rows", tokens=1, h_q=32, h_kv=8, d=128, bs=16, type="f16",
             norm=True, rot=128, pairs=False, axes=3, turns=True),
        # the prefill of a long prompt of text and pictures into a 16-bit paged cache, the axes dealt out in turn
        dict(name="axes_prompt", op="append", cache="rows", tokens=16384, h_q=64, h_kv=8, d=128, bs=16, type="bf16",
             norm=True, rot=128, pairs=False, axes=3, turns=True),
        # one decode step of 64 requests entering the 4-bit cache; what was stored is read back
        dict(name="store_64_steps", op="store", seqs=64, new=1, ctx_lo=1024, ctx_hi=16384, all=False, h_q=32, h_kv=8,
             d=128, bs=16, type="bf16", norm=True, rot=128, pairs=False, axes=1, turns=False),
        # chunked prefill of 4 requests with pictures: 2048 new tokens each, then the whole context back in 16 bits
        dict(name="store_chunks", op="store", seqs=4, new=2048, ctx_lo=1000, ctx_hi=6000, all=True, h_q=32, h_kv=8,
             d=128, bs=16, type="bf16", norm=True, rot=128, pairs=False, axes=3, turns=False),
        # a small model's single sequence over its 4-bit cache: latency
        dict(name="decode_4096", op="decode", cache="kv4", seqs=1, lo=4096, hi=4096, tq=1, h_q=8, h_kv=2, d=64, bs=16,
             type="f16", window=0, sinks=0),
        # serving: 64 requests of 1K to 16K tokens
        dict(name="decode_64x16k", op="decode", cache="kv4", seqs=64, lo=1024, hi=16384, tq=1, h_q=32, h_kv=8, d=128,
             bs=16, type="bf16", window=0, sinks=0),
        # verification of 4 speculated tokens over a long, odd context: 32 query rows for each KV head
        dict(name="decode_verify_4", op="decode", cache="kv4", seqs=1, lo=131071, hi=131071, tq=4, h_q=64, h_kv=8,
             d=128, bs=64, type="bf16", window=0, sinks=0),
        # one request with a context of 2^20 tokens
        dict(name="decode_1m", op="decode", cache="kv4", seqs=1, lo=1 << 20, hi=1 << 20, tq=1, h_q=32, h_kv=8, d=128,
             bs=32, type="f16", window=0, sinks=0),
        # one request, far beyond its window: the latency of a layer with a sliding window
        dict(name="window_1", op="decode", cache="rows", seqs=1, lo=100000, hi=100000, tq=1, h_q=32, h_kv=8, d=128,
             bs=16, type="f16", window=1024, sinks=4),
        # serving: 64 requests of 1K to 32K tokens, a window of 4096
        dict(name="window_64x4096", op="decode", cache="rows", seqs=64, lo=1024, hi=32768, tq=1, h_q=32, h_kv=8,
             d=128, bs=16, type="bf16", window=4096, sinks=4),
        # many requests that verify 3 speculated tokens under a short, odd window
        dict(name="window_384_verify_3", op="decode", cache="rows", seqs=384, lo=128, hi=4096, tq=3, h_q=32, h_kv=8,
             d=128, bs=16, type="f16", window=500, sinks=1),
        # 64 long requests under a window, over the 4-bit cache
        dict(name="window_kv4_64x8192", op="decode", cache="kv4", seqs=64, lo=8192, hi=65536, tq=1, h_q=32, h_kv=8,
             d=128, bs=32, type="bf16", window=8192, sinks=64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads = rng.choice([(8, 2), (32, 8), (64, 8), (8, 8), (12, 4), (28, 4), (16, 1), (6, 3)])
    c = dict(op=rng.choice(["append", "store", "decode", "decode", "decode"]), h_q=heads[0], h_kv=heads[1],
             d=rng.choice([64, 128]), bs=rng.choice([8, 16, 32, 64]), type=rng.choice(["f16", "bf16"]))
    if c["op"] != "decode":
        c.update(norm=rng.random() < 0.75, rot=rng.choice([c["d"], c["d"], c["d"] // 2, 16]), pairs=rng.random() < 0.3,
                 turns=rng.random() < 0.5)
    if c["op"] == "append":
        c.update(cache=rng.choice(["rows", "vllm"]), tokens=log(1, 12000), axes=rng.choice([2, 3, 3, 4]))
    elif c["op"] == "store":
        c.update(seqs=log(1, 100), all=rng.random() < 0.5, axes=rng.choice([1, 2, 3]))
        c.update(new=log(1, max(2, 8000 // c["seqs"])), ctx_lo=rng.randrange(0, 100))
        c.update(ctx_hi=c["ctx_lo"] + log(1, max(2, 30000 // c["seqs"])))
    else:
        c.update(cache=rng.choice(["kv4", "rows"]), seqs=log(1, 200))
        c.update(hi=log(1, max(2, min(60000, 600000 // c["seqs"]))))
        c.update(lo=rng.randint(min(c["hi"], 1 + c["hi"] // 50), c["hi"]))
        c.update(tq=rng.choice([1, 1, 1, rng.randint(2, max(2, min(8, 64 * heads[1] // heads[0])))]))
        c.update(lo=max(c["lo"], c["tq"]), hi=max(c["hi"], c["tq"]))
        windowed = c["cache"] == "rows" or rng.random() < 0.4
        c.update(window=log(1, 8192) if windowed else 0, sinks=rng.choice([0, 1, 4, rng.randint(2, 200)]) if windowed else 0)
    return c


def lengths(c):
    """Tokens of each sequence (for "store": before the new ones): the case's own, whatever the seed."""
    r = random.Random("%s %s %s" % (c["op"], c["seqs"], c["h_q"]))
    lo, hi = (c["ctx_lo"], c["ctx_hi"]) if c["op"] == "store" else (c["lo"], c["hi"])
    return [r.randint(lo, hi) for _ in range(c["seqs"])]


def row_bytes(c, cache):
    """Bytes of a token's K and V of one head."""
    return c["d"] + c["d"] // 8 if cache == "kv4" else 4 * c["d"]


def work(c):
    hq, hk, d = c["h_q"], c["h_kv"], c["d"]
    if c["op"] == "append":
        n = c["tokens"]
        return {"bytes": n * ((2 * hq + 4 * hk) * d * 2 + c["rot"] * 4 + 8 + 4 * c["axes"]), "flops": n * (hq + hk) * d * 7}
    lens = lengths(c)
    if c["op"] == "store":
        n = c["seqs"] * c["new"]
        back = sum(lens) + n if c["all"] else n
        return {"bytes": n * ((2 * hq + 2 * hk) * d * 2 + hk * row_bytes(c, "kv4") + c["rot"] * 4 + 8 + 4 * c["axes"])
                + back * hk * (row_bytes(c, "kv4") + 4 * d), "flops": n * (hq + 2 * hk) * d * 7 + back * hk * d * 2}
    w, tq = c["window"], c["tq"]
    # keys that some token of a sequence sees
    n = sum(lens) if w == 0 else sum(min(m, min(c["sinks"], m) + w + tq - 1) for m in lens)
    return {"bytes": n * hk * row_bytes(c, c["cache"]) + c["seqs"] * (tq * hq * d * 4 + 4) + 4 * (n // c["bs"]),
            "flops": 4 * n * tq * hq * d}


# ---------------------------------------------------------------- inputs
def random_kv4(c, blocks, g):
    """A 4-bit cache as one finds it: groups of 16 about normal values of different size."""
    d, bs, hk = c["d"], c["bs"], c["h_kv"]
    cache = torch.randint(0, 256, (blocks, hk, bs * (d + d // 8)), dtype=torch.uint8, device="cuda", generator=g)
    cache[..., bs * d:] = torch.randint(0x2e, 0x36, (blocks, hk, bs * (d // 8)), dtype=torch.uint8, device="cuda",
                                        generator=g)
    return cache


def tables_for(c, lens, g):
    """Block tables over a shuffled pool: (N, most blocks) int32, -1 past a sequence's last block."""
    need = torch.tensor([(n + c["bs"] - 1) // c["bs"] for n in lens])
    most = max(1, int(need.max()))
    used = torch.arange(most)[None, :] < need[:, None]
    total = int(need.sum()) + 3
    t = torch.full((len(lens), most), -1, dtype=torch.int32)
    t[used] = torch.randperm(total, generator=g)[:int(need.sum())].to(torch.int32)
    return t.cuda(), total


def places(n, first, axes, g):
    """Positions (axes, n) of a stretch of text and pictures: in text all axes go on by one; in a picture the first
    axis stands still and the others are its rows and columns."""
    out = np.zeros((axes, n), dtype=np.int64)
    at, pos, picture = 0, first, False
    while at < n:
        if picture and axes > 1:
            h, w = (int(torch.randint(4, 33, (1,), generator=g)) for _ in range(2))
            m = min(h * w, n - at)
            i = np.arange(m)
            grid = [np.zeros(m, np.int64)] + [i // w, i % w, i // w][:axes - 1]
            out[:, at:at + m] = pos + np.stack(grid)
            pos += max(h, w)
        else:
            m = min(int(torch.randint(20, 600, (1,), generator=g)), n - at)
            out[:, at:at + m] = pos + np.arange(m)
            pos += m
        at, picture = at + m, not picture
    return torch.from_numpy(out)


def axis_of_pairs(c):
    """The axis that turns each of the rot/2 pairs: in turn, or a run for each axis."""
    half, a = c["rot"] // 2, c["axes"]
    return torch.arange(half) % a if c["turns"] else torch.arange(half) * a // half


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    dt, hq, hk, d, bs = TYPES[c["type"]], c["h_q"], c["h_kv"], c["d"], c["bs"]
    s = dict(c, dt=dt)
    if c["op"] != "decode":
        if c["op"] == "append":
            n = c["tokens"]
            blocks = (n + bs - 1) // bs + 2
            pos = places(n, int(torch.randint(0, 5000, (1,), generator=gc)), c["axes"], gc)
            order = torch.randperm(blocks, generator=gc)
            at = torch.arange(n)
            slots = order[at // bs] * bs + at % bs
            if c["cache"] == "rows":
                s["k_cache"] = torch.zeros(blocks, bs, hk * d, dtype=dt, device="cuda")
                s["v_cache"] = torch.zeros_like(s["k_cache"])
            else:
                s["k_cache"] = torch.zeros(blocks, hk, d // 8, bs, 8, dtype=dt, device="cuda")
                s["v_cache"] = torch.zeros(blocks, hk, d, bs, dtype=dt, device="cuda")
        else:
            before = torch.tensor(lengths(c))
            lens = before + c["new"]
            t, blocks = tables_for(c, lens.tolist(), gc)
            n = c["seqs"] * c["new"]
            pos = torch.cat([places(c["new"], m, c["axes"], gc) for m in before.tolist()], 1)
            row = (before[:, None] + torch.arange(c["new"])).reshape(-1)
            seq = torch.arange(c["seqs"]).repeat_interleave(c["new"])
            slots = t.cpu()[seq, row // bs].long() * bs + row % bs
            s["cache"] = random_kv4(c, blocks, g)
            s["tables"], s["lens"] = t, lens.to(torch.int32).cuda()
            s["begins"] = None if c["all"] else before.to(torch.int32).cuda()
            s["count"] = int(lens.max()) if c["all"] else c["new"]
            s["k_back"] = torch.zeros(c["seqs"], s["count"], hk * d, dtype=dt, device="cuda")
            s["v_back"] = torch.zeros_like(s["k_back"])
        # the fused projection's output: q, k and v are views of it
        qkv = torch.randn(n, (hq + 2 * hk) * d, device="cuda", generator=g).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
        s["positions"], s["slots"] = pos.to(torch.int32).cuda(), slots.cuda()
        s["pair_axes"] = axis_of_pairs(c).to(torch.uint8).cuda()
        s["q_weight"] = s["k_weight"] = None
        if c["norm"]:
            s["q_weight"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt)
            s["k_weight"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt)
        inv = THETA ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        ang = torch.arange(int(pos.max()) + 1, device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        return s
    lens = lengths(c)
    s["tables"], blocks = tables_for(c, lens, gc)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if c["cache"] == "kv4":
        s["pool"] = random_kv4(c, blocks, g)
    else:
        s["k_pool"] = torch.randn(blocks, bs, hk * d, device="cuda", generator=g, dtype=dt)
        s["v_pool"] = torch.randn(blocks, bs, hk * d, device="cuda", generator=g, dtype=dt)
    s["q"] = torch.randn(c["seqs"], c["tq"], hq * d, device="cuda", generator=g).to(dt)
    return s


# ---------------------------------------------------------------- plain forms
def plain_turn(y, s):
    """Each pair (a, b) turned by its own axis' angle."""
    rot, half = s["rot"], s["rot"] // 2
    i = torch.arange(half, device="cuda")
    row = s["positions"].long()[s["pair_axes"].long()]                     # (pairs, tokens)
    cos, sin = s["cos_sin"][row, i[:, None]].T[:, None], s["cos_sin"][row, i[:, None] + half].T[:, None]
    if s["pairs"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def plain_rows(x, w, s):
    y = x.float().unflatten(-1, (-1, s["d"]))
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    return plain_turn(y, s)


def plain_code_columns(row, d, bs, which):
    """Byte offsets (..., d/2) of a row's codes inside a (block, head); which: 0 K, 1 V."""
    f = row // 2 % 4 if d == 128 else row // 4 % 2
    e = torch.arange(d // 2, device=row.device)
    return which * bs * (d // 2) + row[..., None] * (d // 2) + ((e // 16) ^ f[..., None]) * 16 + e % 16


def plain_scale_columns(row, d, bs, which):
    return bs * d + which * bs * (d // 16) + row[..., None] * (d // 16) + torch.arange(d // 16, device=row.device)


def plain_quantise(y):
    """Code bytes (..., d/2) and scale bytes (..., d/16) of rows (..., d)."""
    x = y.unflatten(-1, (-1, 16))
    scale = (x.abs().amax(-1) / 6).clamp(max=10240).to(torch.float8_e5m2)
    f = scale.float()[..., None]
    z = torch.where(f > 0, x / f, torch.zeros_like(x)).abs()
    code = ((z > 0.25).int() + (z >= 0.75).int() + (z > 1.25).int() + (z >= 1.75).int() + (z > 2.5).int()
            + (z >= 3.5).int() + (z > 5).int() + 8 * torch.signbit(x).int()).flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), scale.view(torch.uint8)


def plain_store(s, y, which):
    d, bs = s["d"], s["bs"]
    blk, row = s["slots"] // bs, s["slots"] % bs
    h = torch.arange(s["h_kv"], device=row.device)
    codes, scales = plain_quantise(y)
    s["cache"][blk[:, None, None], h[None, :, None], plain_code_columns(row, d, bs, which)[:, None, :]] = codes
    s["cache"][blk[:, None, None], h[None, :, None], plain_scale_columns(row, d, bs, which)[:, None, :]] = scales


def plain_held(cache, blk, row, d, bs, which):
    """32-bit values (..., h_kv, d) of the cache rows (blk, row)."""
    h = torch.arange(cache.shape[1], device="cuda")
    codes = cache[blk[..., None, None], h[:, None], plain_code_columns(row, d, bs, which)[..., None, :]]
    scales = cache[blk[..., None, None], h[:, None], plain_scale_columns(row, d, bs, which)[..., None, :]]
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    table = torch.cat([table, -table])
    pair = torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)        # the two values of a byte
    x = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    return (x * scales.view(torch.float8_e5m2).float()[..., None]).flatten(-2)


def plain_back(s, begins, count, which, out):
    """Tokens of every sequence from begins on, in 16 bits; rows behind a sequence's last token stay."""
    tok = begins[:, None].long() + torch.arange(count, device="cuda")
    there = tok < s["lens"][:, None]
    blk = s["tables"].gather(1, (tok // s["bs"]).clamp(max=s["tables"].shape[1] - 1)).clamp(min=0).long()
    x = plain_held(s["cache"], blk, tok % s["bs"], s["d"], s["bs"], which)
    return torch.where(there[..., None], x.flatten(2).to(s["dt"]), out)


def plain_decode(s):
    n, tq, _ = s["q"].shape
    hq, hk, d, bs, w, sinks = s["h_q"], s["h_kv"], s["d"], s["bs"], s["window"], s["sinks"]
    lens = s["lens"].long()
    # token t of the tq newest has the place lens - tq + t and sees the keys up to its own
    place = lens[:, None] - tq + torch.arange(tq, device="cuda")
    most = s["tables"].shape[1] * bs
    if w == 0:
        key = torch.arange(most, device="cuda").expand(n, -1)
    else:     # the first keys, and from the oldest key in the oldest token's window on
        i = torch.arange(min(most, sinks + w + tq - 1), device="cuda")
        start = (place[:, :1] - w + 1).clamp(min=sinks)
        key = torch.where(i < sinks, i, start + i - sinks)
    there = key < lens[:, None]
    blk = s["tables"].gather(1, (key // bs).clamp(max=s["tables"].shape[1] - 1)).clamp(min=0).long()

    def rows(which):
        if s["cache"] == "kv4":
            return plain_held(s["pool"], blk, key % bs, d, bs, which)
        return s["v_pool" if which else "k_pool"][blk, key % bs].float().unflatten(-1, (hk, d))

    q = s["q"].float().view(n, tq, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)
    p = (q @ rows(0).permute(0, 2, 3, 1)).view(n, hk, tq, hq // hk, -1) / math.sqrt(d)
    seen = there[:, None, :] & (key[:, None, :] <= place[..., None])
    if w:
        seen &= (key[:, None, :] > place[..., None] - w) | (key[:, None, :] < sinks)
    p = p.masked_fill(~seen[:, None, :, None, :], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    l = p.sum(-1, keepdim=True)
    o = (p.view(n, hk, tq * (hq // hk), -1) @ rows(1).permute(0, 2, 1, 3)).view(n, hk, tq, hq // hk, d) / l
    return o.permute(0, 2, 1, 3, 4).reshape(n, tq, hq * d).to(s["dt"])


def plain_run(s):
    if s["op"] == "decode":
        return plain_decode(s)
    q = plain_rows(s["q"], s["q_weight"], s).flatten(1).to(s["dt"])
    k, v = plain_rows(s["k"], s["k_weight"], s), s["v"].float().unflatten(-1, (-1, s["d"]))
    if s["op"] == "store":
        plain_store(s, k, 0)
        plain_store(s, v, 1)
        begins = torch.zeros_like(s["lens"]) if s["begins"] is None else s["begins"]
        return (q, plain_back(s, begins, s["count"], 0, s["k_back"]), plain_back(s, begins, s["count"], 1, s["v_back"]))
    bs, d = s["bs"], s["d"]
    blk, row = s["slots"] // bs, s["slots"] % bs
    if s["cache"] == "rows":
        s["k_cache"][blk, row] = k.flatten(1).to(s["dt"])
        s["v_cache"][blk, row] = v.flatten(1).to(s["dt"])
    else:
        s["k_cache"][blk, :, :, row] = k.unflatten(-1, (d // 8, 8)).to(s["dt"])
        s["v_cache"][blk, :, :, row] = v.to(s["dt"])
    return q, s["k_cache"], s["v_cache"]


# ---------------------------------------------------------------- the framework's calls
def own_run(s):
    import decode_attention_03_gb300 as gqa

    if s["op"] == "decode":
        if s["cache"] == "kv4":
            return gqa.gqa_decode_kv4(s["q"], s["pool"], s["tables"], s["lens"], s["h_q"], s["h_kv"], causal=True,
                                      window=s["window"], sinks=s["sinks"])
        return gqa.gqa_decode_window(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["h_q"], s["h_kv"],
                                     causal=True, window=s["window"], sinks=s["sinks"])
    caches = (s["k_cache"], s["v_cache"]) if s["op"] == "append" else (s["cache"],)
    q = gqa.gqa_append(s["q"], s["k"], s["v"], s["h_q"], s["h_kv"], s["slots"], *caches, positions=s["positions"],
                       cos_sin=s["cos_sin"], pair_axes=s["pair_axes"], interleaved=s["pairs"], q_weight=s["q_weight"],
                       k_weight=s["k_weight"], eps=EPS)
    if s["op"] == "append":
        return q, s["k_cache"], s["v_cache"]
    k, v = gqa.gqa_kv4_read(s["cache"], s["tables"], s["lens"], s["d"], begins=s["begins"], k_out=s["k_back"],
                            v_out=s["v_back"])
    return q, k, v


def run(s):
    return own_run(s) if own else plain_run(s)


# ---------------------------------------------------------------- 64 bits, from the definition
def exact_power(k):
    """2^k for whole k, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def exact_scales(byte):
    """The binary16 numbers whose upper byte this is and whose lower byte is 0."""
    b = byte.long()
    e, m = b >> 2 & 31, (b & 3).double() / 4
    return torch.where(e == 0, m * 2.0 ** -14, (1 + m) * exact_power(e - 15))


def exact_held(y):
    """What a row (..., d) of 64-bit values stands for once it is held in four bits."""
    x = y.reshape(*y.shape[:-1], -1, 16)
    want = torch.clamp(x.abs().amax(-1, keepdim=True) / 6, max=10240)
    step = exact_power(torch.frexp(want.clamp(min=2.0 ** -14)).exponent - 3)       # three significant bits
    scale = torch.round(want / step) * step
    z = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    unit = exact_power(torch.frexp(z.abs().clamp(min=1.0)).exponent - 2)           # two, and halves below 1
    code = (torch.round(z / unit) * unit).clamp(-6, 6)
    return (code * scale).reshape(y.shape)


def exact_rows(x, w, s):
    d, half = s["d"], s["rot"] // 2
    y = x.double().reshape(x.shape[0], -1, d)
    if w is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + EPS) * w.double()
    out = y.clone()
    axis = s["pair_axes"].tolist()
    for i in range(half):
        cs = s["cos_sin"][s["positions"][axis[i]].long()].double()
        turn = torch.complex(cs[:, i], cs[:, half + i])[:, None]
        a, b = (2 * i, 2 * i + 1) if s["pairs"] else (i, i + half)
        z = torch.complex(y[..., a], y[..., b]) * turn
        out[..., a], out[..., b] = z.real, z.imag
    return out


def exact_sequence(s, cache, b, first, last):
    """K and V (tokens, h_kv, d) of the tokens first .. last - 1 of sequence b of a 4-bit cache, in 64 bits."""
    d, bs = s["d"], s["bs"]
    j0, j1 = first // bs, (last + bs - 1) // bs
    blocks = cache[s["tables"][b, j0:j1].long()]
    r = torch.arange(bs, device="cuda")
    turn = r // 2 % 4 if d == 128 else r // 4 % 2
    place = torch.arange(d // 32, device="cuda") ^ turn[:, None]
    size = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    got = []
    for w in (0, 1):
        x = blocks[..., w * bs * d // 2:(w + 1) * bs * d // 2].view(-1, s["h_kv"], bs, d // 32, 16)
        x = x.gather(3, place[None, None, :, :, None].expand_as(x)).flatten(3)
        x = torch.stack([x & 15, x >> 4], -1).flatten(3).long()
        x = size[x & 7] * (1 - 2 * (x >> 3))
        at = bs * d + w * bs * d // 16
        scale = exact_scales(blocks[..., at:at + bs * d // 16].view(-1, s["h_kv"], bs, d // 16))
        x = x * scale.repeat_interleave(16, -1)
        got.append(x.transpose(1, 2).flatten(0, 1)[first - j0 * bs:last - j0 * bs])
    return got


def exact_decode(c, s):
    hq, hk, d, bs, tq, w = c["h_q"], c["h_kv"], c["d"], c["bs"], c["tq"], c["window"]
    out = torch.empty(c["seqs"], tq, hq * d, dtype=torch.float64, device="cuda")
    for b in range(c["seqs"]):
        n = int(s["lens"][b])
        start = max(0, n - tq - w + 1) if w else 0
        spans = [(0, n)] if start <= c["sinks"] else [(0, c["sinks"]), (start, n)]
        got, where = [], []
        for lo, hi in spans:
            if hi == lo:
                continue
            where.append(torch.arange(lo, hi, device="cuda"))
            if c["cache"] == "kv4":
                got.append(exact_sequence(s, s["pool"], b, lo, hi))
            else:
                at = s["tables"][b].long()[where[-1] // bs] * bs + where[-1] % bs
                got.append([s[p].flatten(0, 1)[at].double().unflatten(-1, (hk, d)) for p in ("k_pool", "v_pool")])
        k, v = (torch.cat(x) for x in zip(*got))
        where = torch.cat(where)
        age = (n - tq + torch.arange(tq, device="cuda"))[:, None] - where
        hidden = age < 0
        if w:
            hidden |= (age >= w) & (where >= c["sinks"])
        for h in range(hk):
            q = s["q"][b].double().view(tq, hk, hq // hk, d)[:, h]
            x = torch.einsum("tgd,nd->tgn", q, k[:, h]) / math.sqrt(d)
            x[hidden[:, None, :].expand_as(x)] = -math.inf
            out[b].view(tq, hk, hq // hk, d)[:, h] = torch.einsum("tgn,nd->tgd", torch.softmax(x, -1), v[:, h])
    return out


def exact(c, seed):
    s = prepare(c, seed)
    hk, d = c["h_kv"], c["d"]
    if c["op"] == "decode":
        return exact_decode(c, s)
    q = exact_rows(s["q"], s["q_weight"], s).flatten(1)
    k, v = exact_rows(s["k"], s["k_weight"], s), s["v"].double().reshape(-1, hk, d)
    if c["op"] == "append":
        caches = []
        for name, y in (("k_cache", k), ("v_cache", v)):
            at = s["slots"]
            if c["cache"] == "rows":
                out = s[name].double().flatten(0, 1)
                out[at] = y.flatten(1)
            else:  # tokens to the front, written, and back
                x = s[name].double().reshape(s[name].shape[0], hk, -1, c["bs"], 8 if name == "k_cache" else 1)
                flat = x.permute(0, 3, 1, 2, 4).flatten(2).flatten(0, 1)
                flat[at] = y.flatten(1)
                out = flat.view(x.shape[0], c["bs"], hk, x.shape[2], x.shape[4]).permute(0, 2, 3, 1, 4)
            caches.append(out.reshape(s[name].shape))
        return q, caches[0], caches[1]
    back = [torch.zeros(c["seqs"], s["count"], hk * d, dtype=torch.float64, device="cuda") for _ in range(2)]
    held = [exact_held(y).flatten(1).view(c["seqs"], c["new"], -1) for y in (k, v)]
    for b in range(c["seqs"]):
        n = int(s["lens"][b])
        first = 0 if c["all"] else n - c["new"]
        old = exact_sequence(s, s["cache"], b, first, n)
        for w in (0, 1):
            x = old[w].flatten(1)
            x[n - c["new"] - first:] = held[w][b]
            back[w][b, :n - first] = x
    return (q, *back)
