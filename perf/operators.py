"""Cases of the cache operators: filling a paged KV cache (per-head norms, rotation, quantisation),
decode attention over the quantised cache, and reading it back.

The 8-bit cache ("kv8") is one uint8 tensor (num_blocks, h_kv, block_size * (2 * d + 2)).  A (block, head)
holds the K codes [block_size][d] (e4m3), the V codes [block_size][d], one scale exponent per K row and one
per V row (the scale is 2^(e - 127)).  The 16-byte chunk c of row r is stored at chunk c ^ f(r), with
f(r) = r % 8 for d = 128 and (r // 2) % 4 for d = 64.  A row x is held as codes e4m3(x * 2^-k) where k is
the smallest integer with max|x| <= 448 * 2^k.
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
        # one token of one request enters a 16-bit paged cache: the latency of a single decode step
        dict(name="append_1_token", op="append", cache="rows", tokens=1, h_q=32, h_kv=8, d=128, bs=16, type="f16",
             norm=True, rot=128, pairs=False),
        # the prefill of a long prompt into a 16-bit paged cache, 64 query heads
        dict(name="append_prompt", op="append", cache="rows", tokens=16384, h_q=64, h_kv=8, d=128, bs=16,
             type="bf16", norm=True, rot=128, pairs=False),
        # one decode step of 64 requests entering the 8-bit cache; what was stored is read back
        dict(name="store_64_steps", op="store", seqs=64, new=1, ctx_lo=1024, ctx_hi=16384, all=False, h_q=32,
             h_kv=8, d=128, bs=16, type="bf16", norm=True, rot=128, pairs=False),
        # chunked prefill of 4 requests: 2048 new tokens each, then the whole context back for their attention
        dict(name="store_chunks", op="store", seqs=4, new=2048, ctx_lo=1000, ctx_hi=6000, all=True, h_q=32, h_kv=8,
             d=128, bs=16, type="bf16", norm=True, rot=128, pairs=False),
        # a small model's single sequence: latency
        dict(name="decode_4096", op="decode", seqs=1, lo=4096, hi=4096, tq=1, h_q=8, h_kv=2, d=64, bs=16,
             type="f16"),
        # serving: 64 requests of 1K to 16K tokens
        dict(name="decode_64x16k", op="decode", seqs=64, lo=1024, hi=16384, tq=1, h_q=32, h_kv=8, d=128, bs=16,
             type="f16"),
        # serving: many short requests
        dict(name="decode_384x2k", op="decode", seqs=384, lo=128, hi=2048, tq=1, h_q=32, h_kv=8, d=128, bs=16,
             type="bf16"),
        # verification of 4 speculated tokens over a long, odd context: 32 query rows for each KV head
        dict(name="decode_verify_4", op="decode", seqs=1, lo=131071, hi=131071, tq=4, h_q=64, h_kv=8, d=128, bs=64,
             type="bf16"),
        # one request with a context of 2^20 tokens
        dict(name="decode_1m", op="decode", seqs=1, lo=1 << 20, hi=1 << 20, tq=1, h_q=32, h_kv=8, d=128, bs=32,
             type="f16"),
        # a short prompt's cache read back
        dict(name="read_513", op="read", seqs=1, lo=513, hi=513, h_q=8, h_kv=2, d=64, bs=16, type="f16"),
        # the caches of 64 requests read back to 16 bits
        dict(name="read_64x16k", op="read", seqs=64, lo=1024, hi=16384, h_q=32, h_kv=8, d=128, bs=16, type="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads = rng.choice([(8, 2), (32, 8), (64, 8), (8, 8), (12, 4), (28, 4), (16, 1), (6, 3)])
    c = dict(op=rng.choice(["append", "store", "decode", "decode", "read"]), h_q=heads[0], h_kv=heads[1],
             d=rng.choice([64, 128]), bs=rng.choice([8, 16, 32, 64]), type=rng.choice(["f16", "bf16"]))
    if c["op"] in ("append", "store"):
        c.update(norm=rng.random() < 0.75, rot=rng.choice([c["d"], c["d"], c["d"] // 2, 16]), pairs=rng.random() < 0.3)
    if c["op"] == "append":
        c.update(cache=rng.choice(["rows", "vllm"]), tokens=log(1, 12000))
    elif c["op"] == "store":
        c.update(seqs=log(1, 100), all=rng.random() < 0.5)
        c.update(new=log(1, max(2, 8000 // c["seqs"])), ctx_lo=rng.randrange(0, 100))
        c.update(ctx_hi=c["ctx_lo"] + log(1, max(2, 30000 // c["seqs"])))
    else:
        c.update(seqs=log(1, 200))
        c.update(hi=log(1, max(2, min(60000, 600000 // c["seqs"]))))
        c.update(lo=rng.randint(min(c["hi"], 1 + c["hi"] // 50), c["hi"]))
        if c["op"] == "decode":
            c.update(tq=rng.choice([1, 1, 1, rng.randint(2, max(2, min(8, 64 * heads[1] // heads[0])))]))
            c.update(lo=max(c["lo"], c["tq"]), hi=max(c["hi"], c["tq"]))
    return c


def lengths(c):
    """Tokens of each sequence (for "store": before the new ones): the case's own, whatever the seed."""
    r = random.Random("%s %s %s" % (c["op"], c["seqs"], c["h_q"]))
    lo, hi = (c["ctx_lo"], c["ctx_hi"]) if c["op"] == "store" else (c["lo"], c["hi"])
    return [r.randint(lo, hi) for _ in range(c["seqs"])]


def work(c):
    hq, hk, d = c["h_q"], c["h_kv"], c["d"]
    if c["op"] == "append":
        n = c["tokens"]
        return {"bytes": n * ((2 * hq + 4 * hk) * d * 2 + c["rot"] * 4 + 12), "flops": n * (hq + hk) * d * 7}
    lens = lengths(c)
    if c["op"] == "store":
        n = c["seqs"] * c["new"]
        back = sum(lens) + n if c["all"] else n
        return {"bytes": n * ((2 * hq + 2 * hk) * d * 2 + 2 * hk * (d + 1) + c["rot"] * 4 + 12)
                + back * hk * (2 * d + 2 + 4 * d), "flops": n * (hq + 2 * hk) * d * 7 + back * hk * d * 2}
    n = sum(lens)
    if c["op"] == "decode":
        return {"bytes": n * hk * (2 * d + 2) + c["seqs"] * (c["tq"] * hq * d * 4 + 4) + 4 * (n // c["bs"]),
                "flops": 4 * n * c["tq"] * hq * d}
    return {"bytes": n * hk * (2 * d + 2 + 4 * d) + 4 * (n // c["bs"]), "flops": n * hk * d * 2}


# ---------------------------------------------------------------- inputs
def random_cache(c, blocks, g):
    """An 8-bit cache as one finds it: codes of normal values, the scales of rows of different size."""
    d, bs, hk = c["d"], c["bs"], c["h_kv"]
    cache = torch.empty(blocks, hk, bs * (2 * d + 2), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (hk * bs * 2 * d))
    for b in range(0, blocks, step):
        part = cache[b:b + step]
        x = torch.randn(part.shape[0], hk, bs * 2 * d, device="cuda", generator=g)
        part[..., :bs * 2 * d] = x.mul_(96).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[..., bs * 2 * d:] = torch.randint(118, 122, (blocks, hk, 2 * bs), dtype=torch.uint8, device="cuda",
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


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    dt, hq, hk, d, bs = TYPES[c["type"]], c["h_q"], c["h_kv"], c["d"], c["bs"]
    s = dict(c, dt=dt)
    if c["op"] in ("append", "store"):
        if c["op"] == "append":
            n = c["tokens"]
            blocks = (n + bs - 1) // bs + 2
            first = int(torch.randint(0, 5000, (1,), generator=gc))
            pos = torch.arange(first, first + n)
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
            pos = (before[:, None] + torch.arange(c["new"])).reshape(-1)
            seq = torch.arange(c["seqs"]).repeat_interleave(c["new"])
            slots = t.cpu()[seq, pos // bs].long() * bs + pos % bs
            s["cache"] = random_cache(c, blocks, g)
            s["tables"], s["lens"] = t, lens.to(torch.int32).cuda()
            s["begins"] = None if c["all"] else before.to(torch.int32).cuda()
            s["count"] = int(lens.max()) if c["all"] else c["new"]
            s["k_back"] = torch.zeros(c["seqs"], s["count"], hk * d, dtype=dt, device="cuda")
            s["v_back"] = torch.zeros_like(s["k_back"])
        # the fused projection's output: q, k and v are views of it
        qkv = torch.randn(n, (hq + 2 * hk) * d, device="cuda", generator=g).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
        s["positions"], s["slots"] = pos.to(torch.int32).cuda(), slots.cuda()
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
    s["cache"] = random_cache(c, blocks, g)
    if c["op"] == "decode":
        s["q"] = torch.randn(c["seqs"], c["tq"], hq * d, device="cuda", generator=g).to(dt)
    else:
        s["k_back"] = torch.zeros(c["seqs"], max(lens), hk * d, dtype=dt, device="cuda")
        s["v_back"] = torch.zeros_like(s["k_back"])
    return s


# ---------------------------------------------------------------- plain forms
def plain_rotate(y, s):
    rot = s["rot"]
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if s["pairs"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def plain_head_rows(x, w, s):
    y = x.float().unflatten(-1, (-1, s["d"]))
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    return plain_rotate(y, s)


def plain_append(s):
    """q_out, and the 32-bit K and V rows (tokens, h_kv, d) that go into the cache."""
    q = plain_head_rows(s["q"], s["q_weight"], s).flatten(1).to(s["dt"])
    return q, plain_head_rows(s["k"], s["k_weight"], s), s["v"].float().unflatten(-1, (-1, s["d"]))


def plain_columns(row, d, bs, which):
    """Byte offsets (..., d) of a row's elements inside a (block, head); which: 0 K, 1 V."""
    f = row % 8 if d == 128 else row // 2 % 4
    e = torch.arange(d, device=row.device)
    return which * bs * d + row[..., None] * d + ((e // 16) ^ f[..., None]) * 16 + e % 16


def plain_quantise(y):
    m, e = torch.frexp(y.abs().amax(-1))
    k = torch.where(m == 0, -126, (e - 9 + (m > 0.875)).clamp(-126, 127))
    return torch.ldexp(y, -k[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (k + 127).to(torch.uint8)


def plain_store(s, y, which):
    d, bs = s["d"], s["bs"]
    blk, row = s["slots"] // bs, s["slots"] % bs
    h = torch.arange(s["h_kv"], device=row.device)
    codes, exps = plain_quantise(y)
    s["cache"][blk[:, None, None], h[None, :, None], plain_columns(row, d, bs, which)[:, None, :]] = codes
    s["cache"][blk[:, None], h[None, :], 2 * bs * d + which * bs + row[:, None]] = exps


def plain_read(s, begins, count, which):
    """32-bit values (N, count, h_kv, d) of the tokens from begins on, and which of them exist."""
    d, bs = s["d"], s["bs"]
    tok = begins[:, None].long() + torch.arange(count, device="cuda")
    there = tok < s["lens"][:, None]
    blk = s["tables"].gather(1, (tok // bs).clamp(max=s["tables"].shape[1] - 1)).clamp(min=0).long()
    row = tok % bs
    h = torch.arange(s["h_kv"], device="cuda")
    codes = s["cache"][blk[..., None, None], h[:, None], plain_columns(row, d, bs, which)[:, :, None, :]]
    exps = s["cache"][blk[..., None], h, 2 * bs * d + which * bs + row[..., None]]
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), exps[..., None].int() - 127), there


def plain_back(s, begins, count, which, out):
    x, there = plain_read(s, begins, count, which)
    return torch.where(there[..., None], x.flatten(2).to(s["dt"]), out)


def plain_decode(s):
    n, tq, _ = s["q"].shape
    hq, hk, d = s["h_q"], s["h_kv"], s["d"]
    count = s["tables"].shape[1] * s["bs"]
    zero = torch.zeros(n, dtype=torch.int64, device="cuda")
    k, there = plain_read(s, zero, count, 0)
    q = s["q"].float().view(n, tq, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)
    p = (q @ k.permute(0, 2, 3, 1)).view(n, hk, tq, hq // hk, count) / math.sqrt(d)
    del k
    # token t of the tq newest sees the keys up to its own
    last = s["lens"][:, None].long() - tq + torch.arange(tq, device="cuda")
    seen = there[:, None, :] & (torch.arange(count, device="cuda") <= last[..., None])
    p = p.masked_fill(~seen[:, None, :, None, :], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    l = p.sum(-1, keepdim=True)
    v, _ = plain_read(s, zero, count, 1)
    o = (p.view(n, hk, -1, count) @ v.permute(0, 2, 1, 3)).view(n, hk, tq, hq // hk, d) / l
    return o.permute(0, 2, 1, 3, 4).reshape(n, tq, hq * d).to(s["dt"])


def plain_run(s):
    if s["op"] == "append":
        q, k, v = plain_append(s)
        bs, d = s["bs"], s["d"]
        blk, row = s["slots"] // bs, s["slots"] % bs
        if s["cache"] == "rows":
            s["k_cache"][blk, row] = k.flatten(1).to(s["dt"])
            s["v_cache"][blk, row] = v.flatten(1).to(s["dt"])
        else:
            s["k_cache"][blk, :, :, row] = k.unflatten(-1, (d // 8, 8)).to(s["dt"])
            s["v_cache"][blk, :, :, row] = v.to(s["dt"])
        return q, s["k_cache"], s["v_cache"]
    if s["op"] == "store":
        q, k, v = plain_append(s)
        plain_store(s, k, 0)
        plain_store(s, v, 1)
        begins = torch.zeros_like(s["lens"]) if s["begins"] is None else s["begins"]
        return (q, plain_back(s, begins, s["count"], 0, s["k_back"]), plain_back(s, begins, s["count"], 1, s["v_back"]))
    if s["op"] == "decode":
        return plain_decode(s)
    zero = torch.zeros_like(s["lens"])
    count = s["k_back"].shape[1]
    return plain_back(s, zero, count, 0, s["k_back"]), plain_back(s, zero, count, 1, s["v_back"])


# ---------------------------------------------------------------- the framework's calls
def own_run(s):
    import decode_attention_03_gb300 as gqa

    if s["op"] in ("append", "store"):
        caches = (s["k_cache"], s["v_cache"]) if s["op"] == "append" else (s["cache"],)
        q = gqa.gqa_append(s["q"], s["k"], s["v"], s["h_q"], s["h_kv"], s["slots"], *caches, positions=s["positions"],
                           cos_sin=s["cos_sin"], interleaved=s["pairs"], q_weight=s["q_weight"],
                           k_weight=s["k_weight"], eps=EPS)
        if s["op"] == "append":
            return q, s["k_cache"], s["v_cache"]
        k, v = gqa.gqa_kv8_read(s["cache"], s["tables"], s["lens"], s["d"], begins=s["begins"], k_out=s["k_back"],
                                v_out=s["v_back"])
        return q, k, v
    if s["op"] == "decode":
        return gqa.gqa_decode_kv8(s["q"], s["cache"], s["tables"], s["lens"], s["h_q"], s["h_kv"], causal=True)
    return gqa.gqa_kv8_read(s["cache"], s["tables"], s["lens"], s["d"], k_out=s["k_back"], v_out=s["v_back"])


def run(s):
    return own_run(s) if own else plain_run(s)


# ---------------------------------------------------------------- 64 bits, from the definition
def exact_code_values():
    """The value of each of the 256 e4m3 codes."""
    c = np.arange(256)
    sign, e, m = np.where(c >= 128, -1.0, 1.0), c // 8 % 16, c % 8
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    return torch.from_numpy(np.where(c % 128 == 127, np.nan, sign * v)).cuda()


def exact_power(k):
    """2^k for whole k, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def exact_held(y):
    """What a row held in 8 bits stands for: rounded to 4 significant bits (fewer near zero), half to even."""
    top = y.abs().amax(-1, keepdim=True)
    k = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), torch.zeros_like(top))
    k = torch.where(top > 448 * exact_power(k), k + 1, torch.where(top <= 224 * exact_power(k), k - 1, k))
    x = y / exact_power(k)
    step = exact_power(torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(x / step) * step * exact_power(k)


def exact_rows(x, w, s):
    d, rot, half = s["d"], s["rot"], s["rot"] // 2
    y = x.double().reshape(x.shape[0], -1, d)
    if w is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + EPS) * w.double()
    cs = s["cos_sin"].double()[s["positions"].long()]
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["pairs"] else (i, i + half)
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(cs[:, :half], cs[:, half:])[:, None, :]
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact_sequence(s, b, values):
    """K and V (tokens, h_kv, d) of sequence b in 64 bits."""
    d, bs, n = s["d"], s["bs"], int(s["lens"][b])
    blocks = s["cache"][s["tables"][b, :(n + bs - 1) // bs].long()]
    r = torch.arange(bs, device="cuda")
    turn = r % 8 if d == 128 else r // 2 % 4
    place = torch.arange(d // 16, device="cuda") ^ turn[:, None]
    got = []
    for w in (0, 1):
        x = values[blocks[..., w * bs * d:(w + 1) * bs * d].long()].view(-1, s["h_kv"], bs, d // 16, 16)
        x = x.gather(3, place[None, None, :, :, None].expand_as(x)).flatten(3)
        at = 2 * bs * d + w * bs
        x = x * exact_power(blocks[..., at:at + bs].long() - 127)[..., None]
        got.append(x.transpose(1, 2).flatten(0, 1)[:n])
    return got


def exact(c, seed):
    s = prepare(c, seed)
    hq, hk, d = c["h_q"], c["h_kv"], c["d"]
    if c["op"] in ("append", "store"):
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
    values = exact_code_values()
    if c["op"] == "decode":
        out = torch.empty(c["seqs"], c["tq"], hq * d, dtype=torch.float64, device="cuda")
        for b in range(c["seqs"]):
            k, v = exact_sequence(s, b, values)
            n = k.shape[0]
            for h in range(hk):
                q = s["q"][b].double().view(c["tq"], hk, hq // hk, d)[:, h]
                x = torch.einsum("tgd,nd->tgn", q, k[:, h]) / math.sqrt(d)
                last = n - c["tq"] + torch.arange(c["tq"], device="cuda")
                x[(torch.arange(n, device="cuda") > last[:, None])[:, None, :].expand_as(x)] = -math.inf
                o = torch.einsum("tgn,nd->tgd", torch.softmax(x, -1), v[:, h])
                out[b].view(c["tq"], hk, hq // hk, d)[:, h] = o
        return out
    count = s["k_back"].shape[1]
    back = [torch.zeros(c["seqs"], count, hk * d, dtype=torch.float64, device="cuda") for _ in range(2)]
    if c["op"] == "store":
        held = [exact_held(y).flatten(1).view(c["seqs"], c["new"], -1) for y in (k, v)]
    for b in range(c["seqs"]):
        n = int(s["lens"][b])
        old = exact_sequence(s, b, values)
        first = 0 if c["op"] == "read" or c["all"] else int(s["begins"][b])
        for w in (0, 1):
            x = old[w].flatten(1).clone()
            if c["op"] == "store":
                x[n - c["new"]:] = held[w][b]
            back[w][b, :n - first] = x[first:]
    return (q, *back) if c["op"] == "store" else tuple(back)
