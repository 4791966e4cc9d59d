"""Measured cases of the 8-bit latent cache and of sparse decode's own key selection.

Five operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as the library's call:

  write   new tokens' latent rows (RMSNorm, RoPE) into an e4m3 paged cache with
          one power-of-two scale for each block of `scale_block` tokens, and the
          rotation of the queries' rope parts
  gather  the rows of one plan chunk out of that cache as bf16 buffers
  decode  absorbed MLA decode attention over that cache, dense or over listed rows
  scores  the cheap score of every block of keys for every new token:
          max over the block's visible keys j of
          scale_j * sum_h w[t,h] * relu(q[t,h] . k_j)
  select  the best blocks of every new token, as the list of physical cache rows
          that sparse decode takes

Cases hold sizes only; `shape` seeds the ragged lengths, which therefore belong
to the case, while the values come from the seed given to prepare().
"""
import math
import random

import torch

own = False

DEV = "cuda"
R, DN, DR, DV = 512, 128, 64, 128      # latent, nope, rope and value widths
WIDE = R + DR                          # a cache row
DI = 128                               # width of an index key
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decode step's cache write of 64 sequences, a scale for each token.
        dict(name="write_step", op="write", B=64, H=128, new_lo=1, new_hi=1, cache_lo=4096, cache_hi=16384,
             page=128, scale_block=1, shape=1),
        # Prompts of 8 ragged sequences behind cached prefixes, a scale for 64 tokens.
        dict(name="write_prompts", op="write", B=8, H=128, new_lo=256, new_hi=2048, cache_lo=0, cache_hi=8192,
             page=128, scale_block=64, shape=2),
        # A short chunk on small pages.
        dict(name="gather_short", op="gather", B=2, new_lo=16, new_hi=33, cache_lo=0, cache_hi=700,
             page=16, scale_block=1, shape=3),
        # 64 sequences of 8192 cached tokens in one chunk.
        dict(name="gather_64x8192", op="gather", B=64, new_lo=1, new_hi=1, cache_lo=8192, cache_hi=8192,
             page=128, scale_block=64, shape=4),
        # One user, 16 heads, a short context: latency.
        dict(name="decode_one_short", op="decode", B=1, H=16, new_lo=1, new_hi=1, cache_lo=1000, cache_hi=1000,
             page=128, scale_block=1, topk=0, sink=False, shape=5),
        # 32 sequences with 16 heads over long contexts: bound by the cache read.
        dict(name="decode_h16_long", op="decode", B=32, H=16, new_lo=1, new_hi=1, cache_lo=16384, cache_hi=32768,
             page=64, scale_block=64, topk=0, sink=False, shape=6),
        # 64 sequences, 128 heads, 1 or 2 new tokens over 4k to 16k.
        dict(name="decode_h128", op="decode", B=64, H=128, new_lo=1, new_hi=2, cache_lo=4096, cache_hi=16384,
             page=128, scale_block=64, topk=0, sink=False, shape=7),
        # The same contexts through lists of 2048 rows, with attention sinks.
        dict(name="decode_sparse_h128", op="decode", B=64, H=128, new_lo=1, new_hi=1, cache_lo=4096, cache_hi=16384,
             page=128, scale_block=1, topk=2048, sink=True, shape=8),
        # Key scores of a decode step, bf16 index keys, every key its own block.
        dict(name="scores_step", op="scores", B=64, Hi=64, new_lo=1, new_hi=1, cache_lo=4096, cache_hi=16384,
             page=128, block=1, eight=False, shape=9),
        # Block scores of prompt chunks, 8-bit index keys.
        dict(name="scores_chunk", op="scores", B=2, Hi=32, new_lo=400, new_hi=600, cache_lo=6000, cache_hi=9000,
             page=64, block=64, eight=True, shape=10),
        # The 2048 best keys of every sequence of a decode step.
        dict(name="select_step", op="select", B=64, new_lo=1, new_hi=1, cache_lo=4096, cache_hi=16384,
             page=128, block=1, top=2048, local=1, shape=11),
        # The 2048 best keys of one user's two tokens in a context of 128k.
        dict(name="select_one_long", op="select", B=1, new_lo=2, new_hi=2, cache_lo=131000, cache_hi=131000,
             page=64, block=1, top=2048, local=1, shape=12),
    ]


def _spread(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], [0.0, 0.0])
        m[0], m[1] = max(m[0], w["bytes"]), max(m[1], w["flops"])
    op = rng.choice(["write", "gather", "decode", "decode", "decode", "scores", "scores", "select", "select"])
    while True:
        page = rng.choice([16, 24, 64, 64, 100, 128, 128, 256])
        sb = rng.choice([s for s in (1, 1, 4, 8, 32, 64, 128) if page % s == 0])
        lo = _spread(rng, 64, 20000)
        c = dict(op=op, B=_spread(rng, 1, 96), new_lo=1, new_hi=rng.choice([1, 1, 2, 4]), cache_lo=lo,
                 cache_hi=lo + rng.randrange(lo + 1), page=page, shape=rng.randrange(1 << 20))
        if op == "write":
            c.update(H=_spread(rng, 1, 128), scale_block=sb)
            if rng.random() < 0.5:
                c["new_hi"] = _spread(rng, 1, 2048)
        elif op == "gather":
            c.update(scale_block=sb)
        elif op == "decode":
            c.update(H=_spread(rng, 1, 128), scale_block=sb, topk=rng.choice([0, 0, _spread(rng, 1, 4096)]),
                     sink=rng.random() < 0.3)
        elif op == "scores":
            c.update(Hi=rng.choice([1, 8, 24, 32, 64, 64, 128]), block=rng.choice([1, 1, 8, 64, 128]),
                     eight=rng.random() < 0.5)
            if rng.random() < 0.3:
                c.update(B=rng.randrange(1, 4), new_hi=_spread(rng, 1, 400))
        else:
            c.update(block=rng.choice([1, 1, 1, 8, 64]), local=rng.choice([0, 1, 2]))
            c["top"] = max(1 + c["local"], _spread(rng, 4, 2048) // c["block"])
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1] or op in ("gather", "select", "write") and \
                w["bytes"] <= most[op][0]:
            return c


def _lengths(c):
    """(new, cached) tokens of every sequence."""
    rng = random.Random(c["shape"])
    new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    cached = [rng.randint(c["cache_lo"], c["cache_hi"]) for _ in range(c["B"])]
    return new, cached


def work(case):
    c = case
    new, cached = _lengths(c)
    T = sum(new)
    if c["op"] == "write":
        blocks = sum((p + n - 1) // c["scale_block"] - p // c["scale_block"] + 1 for n, p in zip(new, cached))
        return {"bytes": T * (2 * WIDE + WIDE + 4 * DR + 4 * c["H"] * DR) + 4 * R + 4 * blocks,
                "flops": T * (4 * R + 3 * DR * (c["H"] + 1))}
    if c["op"] == "gather":
        rows = T + sum(cached)
        return {"bytes": rows * (WIDE + 2 * WIDE) + 4 * -(-rows // c["scale_block"]), "flops": rows * WIDE}
    if c["op"] == "decode":
        H, rows, pairs, scales = c["H"], 0, 0, 0
        for n, p in zip(new, cached):
            keys = min(c["topk"], n + p) if c["topk"] else n + p
            rows += keys
            scales += keys if c["topk"] else -(-keys // c["scale_block"])
            pairs += n * keys if c["topk"] else n * p + n * (n + 1) // 2
        index = 4 * rows if c["topk"] else 0
        return {"bytes": rows * WIDE + 4 * scales + index + 2 * T * H * (DN + DR + DV) + 2 * H * R * (DN + DV),
                "flops": 2.0 * H * (pairs * (WIDE + R) + T * R * (DN + DV))}
    if c["op"] == "scores":
        e = 1 if c["eight"] else 2
        rows = T + sum(cached)
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, cached))
        stride = -(-max(n + p for n, p in zip(new, cached)) // c["block"])
        return {"bytes": rows * (DI * e + (4 if c["eight"] else 0)) + T * c["Hi"] * (DI * e + 4) + 4 * T * stride,
                "flops": 2.0 * pairs * c["Hi"] * (DI + 1)}
    seen = sum((p + i) // c["block"] + 1 for n, p in zip(new, cached) for i in range(n))
    return {"bytes": 4 * seen + 4 * T * (c["top"] * c["block"] + 1), "flops": seen}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s (2^-60 at least)."""
    m, e = torch.frexp(amax / E4M3_MAX)               # amax / 448 = m 2^e, 0.5 <= m < 1
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).clamp(min=-60)
    return torch.ldexp(torch.ones_like(amax), e)


def _filled_cache(g, rows, sb):
    """Codes and block scales of N(0, 1) latent rows."""
    codes = torch.empty(rows, WIDE, device=DEV, dtype=torch.float8_e4m3fn)
    scales = torch.empty(rows // sb, device=DEV, dtype=torch.float32)
    step = max(sb, (1 << 18) // sb * sb)
    for a in range(0, rows, step):
        x = _normal(g, min(step, rows - a), WIDE)
        s = _scale_of(x.view(-1, sb * WIDE).abs().amax(1))
        scales[a // sb: a // sb + s.numel()] = s
        codes[a: a + x.shape[0]] = (x.view(-1, sb * WIDE) / s[:, None]).view(-1, WIDE).to(torch.float8_e4m3fn)
    return codes, scales


def prepare(case, seed):
    c = dict(case)
    new, cached = _lengths(c)
    B, T, page = c["B"], sum(new), c["page"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    pages = [-(-(n + p) // page) for n, p in zip(new, cached)]
    num_pages, max_pages = sum(pages), max(pages)
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at: at + k]
        at += k
    iro = torch.zeros(B + 1, dtype=torch.int32)
    iro[1:] = torch.tensor(new).cumsum(0)
    st = dict(c=c, B=B, T=T, page=page, num_pages=num_pages, max_pages=max_pages, max_new=max(new),
              max_seq=max(n + p for n, p in zip(new, cached)), total=T + sum(cached), iro=iro.to(DEV),
              cached=torch.tensor(cached, dtype=torch.int32, device=DEV), table=table,
              status=torch.zeros(1, dtype=torch.int32, device=DEV))
    rows = num_pages * page
    if c["op"] == "write":
        st["cache"], st["scales"] = _filled_cache(g, rows, c["scale_block"])
        st["q"] = _normal(g, T, c["H"], DN + DR).to(torch.bfloat16)
        st["latent"] = _normal(g, T, WIDE, std=2.0).to(torch.bfloat16)
        st["gamma"] = 1.0 + _normal(g, R, std=0.1)
        ang = torch.arange(st["max_seq"], device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(DR // 2, device=DEV, dtype=torch.float64) / (DR // 2))
        st["freqs"] = torch.stack([ang.cos(), ang.sin()], -1).reshape(-1, DR).float()
    elif c["op"] == "gather":
        st["cache"], st["scales"] = _filled_cache(g, rows, c["scale_block"])
        n = st["total"]
        ends = torch.tensor([0] + [a + b for a, b in zip(new, cached)]).cumsum(0).to(torch.int32)
        st["bro"], st["co"] = ends.view(1, -1).to(DEV), torch.zeros(1, B, dtype=torch.int32, device=DEV)
        st["bl"] = torch.tensor([n], dtype=torch.int32, device=DEV)
        st["ckv"] = torch.zeros(n, R, dtype=torch.bfloat16, device=DEV)
        st["krope"] = torch.zeros(n, DR, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "decode":
        H = c["H"]
        st["cache"], st["scales"] = _filled_cache(g, rows, c["scale_block"])
        st["q"] = _normal(g, T, H, DN + DR).to(torch.bfloat16)
        st["w_uk"] = _normal(g, H, R, DN, std=R ** -0.5).to(torch.bfloat16)
        st["w_uv"] = _normal(g, H, DV, R, std=R ** -0.5).to(torch.bfloat16)
        st["out"] = torch.zeros(T, H, DV, dtype=torch.bfloat16, device=DEV)
        st["sink"] = _normal(g, B) if c["sink"] else None
        st["list"] = st["count"] = None
        if c["topk"]:
            st["list"] = torch.full((B, c["topk"]), -1, dtype=torch.int32, device=DEV)
            for b in range(B):
                L = new[b] + cached[b]
                k = min(c["topk"], L)
                pos = torch.randperm(L, generator=g, device=DEV)[:k].sort().values
                st["list"][b, :k] = table[b][pos // page] * page + (pos % page).int()
            st["count"] = torch.tensor([min(c["topk"], n + p) for n, p in zip(new, cached)], dtype=torch.int32,
                                       device=DEV)
    elif c["op"] == "scores":
        Hi = c["Hi"]
        q, k = _normal(g, T, Hi, DI), _normal(g, rows, DI)
        st["w"] = _normal(g, T, Hi, std=(Hi * DI) ** -0.5)
        st["key_scales"] = None
        if c["eight"]:
            st["key_scales"] = (k.abs().amax(1) / E4M3_MAX).clamp_(min=1e-12)
            k = k / st["key_scales"][:, None]
        kind = torch.float8_e4m3fn if c["eight"] else torch.bfloat16
        st["iq"], st["keys"] = q.to(kind), k.to(kind)
        st["stride"] = -(-st["max_seq"] // c["block"])
        st["scores"] = torch.zeros(T, st["stride"], device=DEV)
    else:
        st["stride"] = -(-st["max_seq"] // c["block"])
        st["scores"] = _normal(g, T, st["stride"])
        st["width"] = c["top"] * c["block"]
        st["rows"] = torch.zeros(T, st["width"], dtype=torch.int32, device=DEV)
        st["count"] = torch.zeros(T, dtype=torch.int32, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms

def _tokens(s):
    """Sequence and position of every new token."""
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(s["iro"].long(), t, right=True) - 1
    return b, s["cached"].long()[b] + t - s["iro"].long()[b]


def _physical(s, b, pos):
    """Cache row of position `pos` of sequence `b`."""
    return s["table"].long()[b, pos // s["page"]] * s["page"] + pos % s["page"]


def _rotated(x, f):
    re, im, c, d = x[..., 0::2], x[..., 1::2], f[..., 0::2], f[..., 1::2]
    return torch.stack([re * c - im * d, re * d + im * c], -1).flatten(-2)


def _quantised(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_write(s):
    sb = s["c"]["scale_block"]
    b, pos = _tokens(s)
    x = s["latent"].float()
    f = s["freqs"][pos]
    lat, rope = x[:, :R], x[:, R:]
    lat = lat / torch.sqrt(lat.square().mean(1, keepdim=True) + EPS) * s["gamma"]
    x = torch.cat([lat, _rotated(rope, f)], 1)
    row = _physical(s, b, pos)
    block = row // sb
    # The largest value that each touched block gets, and how many rows it had before.
    amax = torch.zeros_like(s["scales"]).scatter_reduce(0, block, x.abs().amax(1), "amax")
    first = torch.full_like(s["scales"], sb, dtype=torch.int64).scatter_reduce(0, block, row % sb, "amin")
    touched = first < sb
    fresh = _scale_of(amax)
    grown = touched & (first > 0) & (fresh > s["scales"])
    if sb > 1:
        cells = torch.nonzero(grown)[:, 0]
        old = s["cache"].view(-1, sb, WIDE)[cells].float()
        again = _quantised(old * (s["scales"][cells] / fresh[cells])[:, None, None])
        keep = torch.arange(sb, device=DEV) < first[cells][:, None]
        old = torch.where(keep[..., None], again.float(), old)
        s["cache"].view(-1, sb, WIDE)[cells] = old.to(torch.float8_e4m3fn)
    s["scales"].copy_(torch.where(touched & ((first == 0) | grown), fresh, s["scales"]))
    s["cache"][row] = _quantised(x / s["scales"][block][:, None])
    s["q"][..., DN:] = _rotated(s["q"][..., DN:].float(), f[:, None]).to(torch.bfloat16)
    return {"cache": s["cache"], "scales": s["scales"], "q": s["q"]}


def _plain_gather(s):
    r = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(s["bro"][0].long(), r, right=True) - 1
    row = _physical(s, b, s["co"][0].long()[b] + r - s["bro"][0].long()[b])
    x = (s["cache"][row].float() * s["scales"][row // s["c"]["scale_block"]][:, None]).to(torch.bfloat16)
    return {"c_kv": x[:, :R].contiguous(), "k_rope": x[:, R:].contiguous()}


def _plain_decode(s):
    c = s["c"]
    B, H, n = s["B"], c["H"], s["max_new"]
    tok, pos = _tokens(s)
    i = torch.arange(s["T"], device=DEV) - s["iro"].long()[tok]
    q = torch.zeros(B, n, H, DN + DR, device=DEV)
    q[tok, i] = s["q"].float()
    full = torch.cat([torch.einsum("bnhd,hkd->bnhk", q[..., :DN], s["w_uk"].float()), q[..., DN:]], -1)
    if s["list"] is not None:
        row = s["list"].long().clamp(min=0)
        L = row.shape[1]
        seen = (torch.arange(L, device=DEV) < s["count"][:, None])[:, None].expand(B, n, L)
    else:
        L = s["max_seq"]
        j = torch.arange(L, device=DEV)
        row = _physical(s, torch.arange(B, device=DEV)[:, None], j.expand(B, L)).clamp(min=0)
        seen = j <= s["cached"].long()[:, None, None] + torch.arange(n, device=DEV)[:, None]
    k = s["cache"][row].float() * s["scales"][row // c["scale_block"]][..., None]
    x = torch.matmul(full.view(B, n * H, WIDE), k.transpose(1, 2)).view(B, n, H, L) * (DN + DR) ** -0.5
    x.masked_fill_(~seen[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"][:, None, None, None])
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    x = torch.exp_(x.sub_(top))
    total = x.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"][:, None, None, None] - top)
    o = torch.matmul(x.view(B, n * H, L), k[..., :R]).view(B, n, H, R) / torch.where(total > 0, total, 1.0)
    return {"out": torch.einsum("bnhk,hdk->bnhd", o, s["w_uv"].float())[tok, i].to(torch.bfloat16)}


def _plain_scores(s):
    c = s["c"]
    B, Hi, n, L, block = s["B"], c["Hi"], s["max_new"], s["max_seq"], c["block"]
    tok, pos = _tokens(s)
    i = torch.arange(s["T"], device=DEV) - s["iro"].long()[tok]
    q, w = torch.zeros(B, n, Hi, DI, device=DEV), torch.zeros(B, n, Hi, device=DEV)
    q[tok, i], w[tok, i] = s["iq"].float(), s["w"]
    j = torch.arange(L, device=DEV)
    row = _physical(s, torch.arange(B, device=DEV)[:, None], j.expand(B, L)).clamp(min=0)
    x = torch.matmul(q.view(B, n * Hi, DI), s["keys"][row].float().transpose(1, 2)).view(B, n, Hi, L)
    x = torch.matmul(w[:, :, None], torch.relu_(x))[:, :, 0]
    if s["key_scales"] is not None:
        x = x * s["key_scales"][row][:, None]
    x = x[tok, i]
    x.masked_fill_(j > pos[:, None], -math.inf)
    full = torch.full((s["T"], s["stride"] * block), -math.inf, device=DEV)
    full[:, :L] = x
    return {"scores": full.view(s["T"], s["stride"], block).amax(-1)}


def _plain_select(s):
    c = s["c"]
    block, top, local = c["block"], c["top"], c["local"]
    tok, pos = _tokens(s)
    j = torch.arange(s["stride"], device=DEV)
    last = (pos // block)[:, None]
    x = torch.where(torch.isnan(s["scores"]), -math.inf, s["scores"])
    x = torch.where((j <= last) & (j > last - local), math.inf, x)
    x = torch.where(j > last, -math.inf, x)
    best = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    n = torch.clamp(last + 1, max=top)
    best = torch.where(torch.arange(best.shape[1], device=DEV) < n, best, s["stride"]).sort(1).values
    p = (best[..., None] * block + torch.arange(block, device=DEV)).flatten(1)
    used = p <= pos[:, None]
    row = _physical(s, tok[:, None], torch.where(used, p, 0))
    rows = torch.full((s["T"], s["width"]), -1, dtype=torch.int32, device=DEV)
    rows[:, :p.shape[1]] = torch.where(used, row, -1).int()
    return {"rows": rows, "count": used.sum(1).int()}


# ------------------------------------------------------------------ the library's calls

def _own_write(s, mla):
    c = s["c"]
    mla.check(mla.mla_latent_cache_write_q8(
        s["cache"], s["scales"], s["q"], s["latent"], s["gamma"], s["freqs"], s["iro"], s["cached"], s["table"],
        s["num_pages"], s["page"], s["max_pages"], c["scale_block"], s["B"], c["H"], s["T"], s["max_seq"], EPS,
        s["status"]))
    return {"cache": s["cache"], "scales": s["scales"], "q": s["q"]}


def _own_gather(s, mla):
    mla.check(mla.mla_gather_latent_q8(
        s["ckv"], s["krope"], s["cache"], s["scales"], s["table"], s["num_pages"], s["page"], s["max_pages"],
        s["c"]["scale_block"], s["bro"], s["co"], s["bl"], 0, s["B"], s["total"], s["status"]))
    return {"c_kv": s["ckv"], "k_rope": s["krope"]}


def _own_decode(s, mla):
    c = s["c"]
    if "ws" not in s:
        keys = min(c["topk"], s["max_seq"]) if c["topk"] else s["max_seq"]
        parts = mla.mla_decode_q8_partitions(s["B"], c["H"], s["max_new"], keys)
        s["bytes"] = mla.mla_decode_q8_workspace_bytes(c["H"], s["T"], parts)
        s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    mla.check(mla.mla_decode_q8(
        s["out"], None, s["q"], s["iro"], s["cached"], s["cache"], s["scales"], s["table"], s["num_pages"], s["page"],
        s["max_pages"], c["scale_block"], s["w_uk"], s["w_uv"], s["B"], c["H"], s["T"], s["max_new"], s["max_seq"], 0,
        (DN + DR) ** -0.5, d_indices=s["list"], indices_stride=c["topk"], topk_lengths=s["count"],
        attn_sink=s["sink"], workspace=s["ws"], workspace_bytes=s["bytes"], d_status=s["status"]))
    return {"out": s["out"]}


def _own_scores(s, mla):
    c = s["c"]
    mla.check(mla.mla_index_scores(
        s["scores"], s["iq"], s["w"], s["keys"], s["key_scales"], s["iro"], s["cached"], s["table"], s["num_pages"],
        s["page"], s["max_pages"], c["block"], s["B"], c["Hi"], s["T"], s["max_new"], s["max_seq"], s["stride"],
        mla.MLA_E4M3 if c["eight"] else mla.MLA_BF16, s["status"]))
    return {"scores": s["scores"]}


def _own_select(s, mla):
    c = s["c"]
    mla.check(mla.mla_index_select(
        s["rows"], s["count"], s["scores"], s["iro"], s["cached"], s["table"], s["num_pages"], s["page"],
        s["max_pages"], c["block"], c["top"], c["local"], s["B"], s["T"], s["max_seq"], s["stride"], s["width"],
        s["status"]))
    return {"rows": s["rows"], "count": s["count"]}


def run(state):
    op = state["c"]["op"]
    if own:
        import mla_prefill_attention_plan_gb300 as mla
        return globals()["_own_" + op](state, mla)
    return globals()["_plain_" + op](state)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence (or token) at a time."""
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s, s["c"], *_lengths(s["c"]))


def _context(s, b, L):
    """Cache rows of the positions 0 .. L-1 of sequence b."""
    j = torch.arange(L, device=DEV)
    return s["table"][b].long()[torch.div(j, s["page"], rounding_mode="floor")] * s["page"] + j.remainder(s["page"])


def _turn(x, f):
    z = torch.view_as_complex(x.reshape(*x.shape[:-1], DR // 2, 2)) * torch.view_as_complex(f.reshape(-1, DR // 2, 2))
    return torch.view_as_real(z).reshape(x.shape)


def _nearest_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even, saturating at 448."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0)))
    e = torch.where(torch.pow(2.0, e) > a, e - 1, e)
    step = torch.pow(2.0, e.clamp(min=-6.0) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_write(s, c, new, cached):
    sb = c["scale_block"]
    x = s["latent"].double()
    lat = x[:, :R] * (x[:, :R].pow(2).sum(1, keepdim=True) / R + EPS).rsqrt() * s["gamma"].double()
    q, scales = s["q"].double(), s["scales"].double()
    cache = s["cache"].to(torch.float64 if s["cache"].numel() < 1 << 28 else torch.float32)
    t = 0
    for b, (n, p) in enumerate(zip(new, cached)):
        f = s["freqs"][p: p + n].double()
        y = torch.cat([lat[t: t + n], _turn(x[t: t + n, R:].contiguous(), f)], 1)
        q[t: t + n, :, DN:] = _turn(q[t: t + n, :, DN:].transpose(0, 1).contiguous(), f).transpose(0, 1)
        row = _context(s, b, p + n)
        if sb == 1:
            scales[row[p:]] = torch.pow(2.0, torch.ceil(torch.log2(y.abs().amax(1) / E4M3_MAX)))
        else:
            for k in range(p // sb, (p + n - 1) // sb + 1):
                lo, hi = max(p, k * sb), min(p + n, (k + 1) * sb)
                m = float(y[lo - p: hi - p].abs().max()) / E4M3_MAX
                up, cell = 2.0 ** math.ceil(math.log2(m)), int(row[lo]) // sb
                was = float(scales[cell])
                if lo > k * sb and up > was:
                    prior = row[k * sb: lo]
                    cache[prior] = _nearest_e4m3(cache[prior].double() * (was / up)).to(cache.dtype)
                if lo == k * sb or up > was:
                    scales[cell] = up
        cache[row[p:]] = _nearest_e4m3(y / scales[row[p:] // sb][:, None]).to(cache.dtype)
        t += n
    return {"cache": cache, "scales": scales, "q": q}


def _exact_gather(s, c, new, cached):
    row = torch.cat([_context(s, b, n + p) for b, (n, p) in enumerate(zip(new, cached))])
    x = s["cache"][row].double() * s["scales"].double()[row // c["scale_block"]].unsqueeze(1)
    return {"c_kv": x[:, :R].contiguous(), "k_rope": x[:, R:].contiguous()}


def _exact_decode(s, c, new, cached):
    out, t = [], 0
    w_uk, w_uv = s["w_uk"].double(), s["w_uv"].double()
    for b, (n, p) in enumerate(zip(new, cached)):
        row = _context(s, b, n + p) if s["list"] is None else s["list"][b, : int(s["count"][b])].long()
        k = s["cache"][row].double() * s["scales"].double()[row // c["scale_block"]].unsqueeze(1)
        q = s["q"][t: t + n].double()
        lat = torch.bmm(q[..., :DN].transpose(0, 1), w_uk.transpose(1, 2)).transpose(0, 1)
        x = torch.cat([lat, q[..., DN:]], -1) @ k.T / math.sqrt(DN + DR)
        if s["list"] is None:
            hidden = torch.arange(n + p, device=DEV)[None] > p + torch.arange(n, device=DEV)[:, None]
            x = x.masked_fill(hidden[:, None], -math.inf)
        if s["sink"] is not None:
            x = torch.cat([x, s["sink"][b].double().expand(n, x.shape[1], 1)], -1)
        pr = torch.softmax(x, -1)[..., : row.numel()]
        out.append(torch.bmm((pr @ k[:, :R]).transpose(0, 1), w_uv.transpose(1, 2)).transpose(0, 1))
        t += n
    return {"out": torch.cat(out)}


def _exact_scores(s, c, new, cached):
    got, t = torch.full((s["T"], s["stride"]), -math.inf, device=DEV, dtype=torch.float64), 0
    for b, (n, p) in enumerate(zip(new, cached)):
        row = _context(s, b, n + p)
        k = s["keys"][row].double()
        if s["key_scales"] is not None:
            k = k * s["key_scales"].double()[row].unsqueeze(1)
        for a in range(0, n, 64):
            z = min(n, a + 64)
            x = (s["iq"][t + a: t + z].double() @ k.T).clamp(min=0) * s["w"][t + a: t + z].double()[..., None]
            x = x.sum(1)
            hidden = torch.arange(n + p, device=DEV)[None] > p + torch.arange(a, z, device=DEV)[:, None]
            x = torch.nn.functional.pad(x.masked_fill(hidden, -math.inf), (0, -(n + p) % c["block"]), value=-math.inf)
            got[t + a: t + z, : x.shape[1] // c["block"]] = x.unflatten(1, (-1, c["block"])).amax(2)
        t += n
    return {"scores": got}


def _exact_select(s, c, new, cached):
    return None                                       # whole numbers: they have to be equal
