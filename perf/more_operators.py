"""Measured cases of chunk attention and of the paged cache's bookkeeping.

Five kinds of work, each in a plain form (elementary torch operations) and as
the library's calls:

  attend   absorbed MLA attention of a chunk of new tokens of every sequence (a
           draft tree to be verified, or consecutive tokens) over the paged bf16
           latent cache: all cached positions are visible, new tokens see each
           other by a bit mask or causally
  keep     the rows of the accepted drafts moved together behind the cached
           context, in every layer of a cache
  fork     sequences continued several times from shared pages: tables and
           reference counts, pages for the next token (a shared page that is
           about to be written gets a copy), and the copies in every layer
  step     pages reserved for new tokens and given back
  compact  half the sequences end, the pool's live pages move to its low end (in
           every layer), new sequences take pages behind them

Cases hold sizes only; `shape` seeds lengths and beam parents, which therefore
belong to the case, while values, trees and page orders come from the seed given
to prepare().
"""
import math
import random

import torch

own = False

DEV = "cuda"
R, DN, DR, DV = 512, 128, 64, 128      # latent, nope, rope and value widths
WIDE = R + DR                          # a cache row

# What a cache row can be: (elements, type) of the bf16 and the 8-bit latent
# cache, of a float32 scale for each token, and of a bf16 index key.
KINDS = {"bf16": (WIDE, torch.bfloat16), "codes": (WIDE, torch.uint8), "scale": (1, torch.float32),
         "index": (128, torch.bfloat16)}
SIZE = {"bf16": 2 * WIDE, "codes": WIDE, "scale": 4, "index": 256}     # bytes of one


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One user verifies a tree of 6 drafts, 16 heads, short context: latency.
        dict(name="attend_one_short", op="attend", B=1, H=16, new_lo=6, new_hi=6, cache_lo=1000, cache_hi=1000,
             page=128, mask="tree", sink=False, shape=21),
        # 32 users' trees of 4 to 16 drafts over long contexts, 16 heads.
        dict(name="attend_tree_h16", op="attend", B=32, H=16, new_lo=4, new_hi=16, cache_lo=8192, cache_hi=32768,
             page=64, mask="tree", sink=False, shape=22),
        # Trees of 8 to 32 drafts, 128 heads, attention sinks.
        dict(name="attend_tree_h128", op="attend", B=16, H=128, new_lo=8, new_hi=32, cache_lo=4096, cache_hi=16384,
             page=128, mask="tree", sink=True, shape=23),
        # The next 64 prompt tokens of one long context, causal, 128 heads.
        dict(name="attend_chunk_long", op="attend", B=1, H=128, new_lo=64, new_hi=64, cache_lo=65536, cache_hi=65536,
             page=64, mask="causal", sink=False, shape=24),
        # Accepted drafts of 16 users in one layer: latency.
        dict(name="keep_step", op="keep", B=16, layers=1, kind="bf16", drafts=8, cache_lo=100, cache_hi=4000,
             page=128, shape=25),
        # Accepted drafts of 128 users in all layers of a model.
        dict(name="keep_layers", op="keep", B=128, layers=24, kind="bf16", drafts=16, cache_lo=0, cache_hi=200,
             page=64, shape=26),
        # A beam search step of 32 beams, one layer.
        dict(name="fork_beams", op="fork", B=32, fan=4, layers=1, kind="bf16", cache_lo=500, cache_hi=4000,
             page=64, shape=27),
        # 16 prompts continued 16 times each, 8 layers: the last pages are copied.
        dict(name="fork_samples", op="fork", B=256, fan=16, layers=8, kind="bf16", cache_lo=200, cache_hi=2000,
             page=128, shape=28),
        # A speculative step's pages of 64 users, on small pages.
        dict(name="step_drafts", op="step", B=64, new_lo=1, new_hi=8, cache_lo=100, cache_hi=4000, page=16, shape=29),
        # 512 prompts come and go in a pool of many small pages.
        dict(name="step_prompts", op="step", B=512, new_lo=200, new_hi=8000, cache_lo=0, cache_hi=0, page=16,
             shape=30),
        # A small pool of one layer is compacted.
        dict(name="compact_small", op="compact", B=16, layers=1, kind="bf16", cache_lo=200, cache_hi=1000, page=64,
             shape=31),
        # The pools of 8 layers: about 1000 pages of each move.
        dict(name="compact_layers", op="compact", B=64, layers=8, kind="bf16", cache_lo=1000, cache_hi=4000, page=64,
             shape=32),
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
    op = rng.choice(["attend", "attend", "attend", "attend", "keep", "fork", "step", "compact"])
    while True:
        page = rng.choice([16, 24, 32, 64, 64, 100, 128, 128, 256])
        c = dict(op=op, page=page, shape=rng.randrange(1 << 20))
        if op == "attend":
            lo = rng.choice([0, _spread(rng, 16, 60000), _spread(rng, 16, 60000), _spread(rng, 16, 60000)])
            n = _spread(rng, 1, 128)
            c.update(B=_spread(rng, 1, 64), H=_spread(rng, 1, 128), new_lo=rng.choice([1, n]), new_hi=n, cache_lo=lo,
                     cache_hi=lo + rng.randrange(lo + 1), mask=rng.choice(["tree", "tree", "causal", "any"]),
                     sink=rng.random() < 0.3)
        elif op == "step":
            lo, n = rng.choice([0, _spread(rng, 16, 4000)]), _spread(rng, 1, 4000)
            c.update(B=_spread(rng, 1, 512), new_lo=rng.choice([0, 1, n]), new_hi=n, cache_lo=lo,
                     cache_hi=lo + rng.randrange(lo + 1))
        else:
            lo = _spread(rng, 16, 2000)
            c.update(B=_spread(rng, 2, 256), layers=_spread(rng, 1, 24),
                     kind=rng.choice(["bf16", "bf16", "codes", "scale", "index"]), cache_lo=lo,
                     cache_hi=lo + rng.randrange(lo + 1))
            if op == "keep":
                c["drafts"] = _spread(rng, 1, 64)
            elif op == "fork":
                c["fan"] = rng.choice([1, 2, 4, 8, 16])
        w = work(c)
        if w["bytes"] <= most[op][0] and (op != "attend" or w["flops"] <= most[op][1]) and _pool_bytes(c) <= 2 << 30:
            return c


def _lengths(c):
    """(new, cached) tokens of every sequence."""
    rng = random.Random(c["shape"])
    new = [rng.randint(c.get("new_lo", 1), c.get("new_hi", 1)) for _ in range(c["B"])]
    cached = [rng.randint(c["cache_lo"], c["cache_hi"]) for _ in range(c["B"])]
    if c["op"] == "fork":                             # the beams that go on are the first of every fan
        cached = [n if b < _roots(c) else 0 for b, n in enumerate(cached)]
    return new, cached


def _roots(c):
    return -(-c["B"] // c["fan"])


def _parents(c):
    return [b // c["fan"] for b in range(c["B"])]


def _accepted(c, seed):
    """Ascending chunk positions of every sequence's accepted drafts."""
    rng = random.Random(seed)
    return [sorted(rng.sample(range(c["drafts"]), rng.randint(0, max(1, c["drafts"] * 3 // 4))))
            for _ in range(c["B"])]


def _pages(n, page):
    return -(-n // page)


def _pool(c):
    """(pages of the pool, pages of a table row)."""
    new, cached = _lengths(c)
    page, B = c["page"], c["B"]
    if c["op"] == "attend":
        held = [_pages(n + p, page) for n, p in zip(new, cached)]
        return sum(held), max(held)
    if c["op"] == "keep":
        held = [_pages(p + c["drafts"], page) for p in cached]
        return sum(held), max(held)
    if c["op"] == "fork":
        held = [_pages(p + 1, page) for p in cached]
        return 2 * B + sum(held), max(held) + 1
    held = [_pages(n + p, page) for n, p in zip(new, cached)]
    return sum(held) * 4 // 3 + 8, max(held)


def _pool_bytes(c):
    rows = _pool(c)[0] * c["page"]
    return rows * (2 * WIDE if c["op"] == "attend" else SIZE[c["kind"]] * c["layers"] if "layers" in c else 4)


def work(case):
    c = case
    new, cached = _lengths(c)
    page = c["page"]
    num_pages, max_pages = _pool(c)
    if c["op"] == "attend":
        H, T = c["H"], sum(new)
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, cached))
        return {"bytes": (T + sum(cached)) * 2 * WIDE + 2 * T * H * (DN + DR + DV) + 2 * H * R * (DN + DV),
                "flops": 2.0 * H * (pairs * (WIDE + R) + T * R * (DN + DV))}
    if c["op"] == "keep":
        moved = c["B"] * max(1, c["drafts"] * 3 // 4) / 2.0
        return {"bytes": 2 * moved * SIZE[c["kind"]] * c["layers"] + 4 * moved, "flops": 0}
    if c["op"] == "fork":
        copies = sum(1 for b, a in enumerate(_parents(c)) if cached[a] % page) - sum(1 for p in cached if p % page)
        table = sum(_pages(cached[a], page) for a in _parents(c))
        return {"bytes": 2 * copies * page * SIZE[c["kind"]] * c["layers"] + 16 * table, "flops": 0}
    if c["op"] == "step":
        fresh = sum(_pages(n + p, page) - _pages(p, page) for n, p in zip(new, cached))
        return {"bytes": 4 * num_pages + 16 * fresh + 16 * c["B"], "flops": 0}
    held = [_pages(p, page) for p in cached]
    moved = min(sum(held[0::2]), sum(held[1::2]))
    return {"bytes": 2 * moved * page * SIZE[c["kind"]] * c["layers"] + 4 * num_pages + 8 * sum(held), "flops": 0}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)


def _filled(g, kind, layers, rows):
    """A cache [layers][rows][elements] of random values."""
    wide, dtype = KINDS[kind]
    x = torch.empty(layers, rows, wide, device=DEV, dtype=dtype)
    if dtype == torch.uint8:
        x.random_(0, 120, generator=g)
    else:
        x.normal_(generator=g)
    return x


def _mask_rows(c, new, seed):
    """Every new token's visible new tokens as a whole number (bit j: token j)."""
    rng = random.Random(seed)
    rows = []
    for n in new:
        seen = []
        for i in range(n):
            if c["mask"] == "tree":                   # itself and its ancestors
                up = rng.randrange(-1, i) if i else -1
                seen.append(1 << i | (seen[up] if up >= 0 else 0))
            else:                                     # any set of them, none included
                seen.append(rng.getrandbits(n) if rng.random() < 0.9 else 0)
        rows += seen
    return rows


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = dict(case)
    new, cached = _lengths(c)
    B, page = c["B"], c["page"]
    num_pages, max_pages = _pool(c)
    g = torch.Generator(device=DEV).manual_seed(seed)
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    held = [_pages(p + (n if c["op"] == "attend" else c["drafts"] if c["op"] == "keep" else 0), page)
            for n, p in zip(new, cached)]
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
    refs[order[:sum(held)].long()] = 1
    if c["op"] == "step":                             # pages that sequences outside the call hold
        refs[order[(num_pages + sum(_pages(n + p, page) for n, p in zip(new, cached))) // 2:].long()] = 1
    at = 0
    for b, k in enumerate(held):
        table[b, :k] = order[at: at + k]
        at += k
    st = dict(c=c, B=B, page=page, num_pages=num_pages, max_pages=max_pages, table=table, refs=refs,
              cached=_ints(cached), status=torch.zeros(1, dtype=torch.int32, device=DEV))
    if c["op"] == "attend":
        T, H = sum(new), c["H"]
        st.update(T=T, max_new=max(new), max_seq=max(n + p for n, p in zip(new, cached)),
                  iro=torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32),
                  cache=_filled(g, "bf16", 1, num_pages * page)[0],
                  q=_normal(g, T, H, DN + DR).to(torch.bfloat16),
                  w_uk=_normal(g, H, R, DN, std=R ** -0.5).to(torch.bfloat16),
                  w_uv=_normal(g, H, DV, R, std=R ** -0.5).to(torch.bfloat16),
                  sink=_normal(g, B) if c["sink"] else None, mask=None, words=0,
                  out=torch.zeros(T, H, DV, dtype=torch.bfloat16, device=DEV))
        if c["mask"] != "causal":
            st["words"] = words = -(-max(new) // 32)
            bits = [[row >> 32 * w & 0xffffffff for w in range(words)] for row in _mask_rows(c, new, seed)]
            st["mask"] = torch.tensor(bits, dtype=torch.int64, device=DEV).to(torch.int32)
        return st
    if "layers" in c:
        st["cache"] = _filled(g, c["kind"], c["layers"], num_pages * page)
    if c["op"] == "keep":
        kept = _accepted(c, seed)
        st["width"] = max(1, max(map(len, kept)))
        st["keep"] = _ints([k + [-1] * (st["width"] - len(k)) for k in kept])
        st["counts"] = _ints([len(k) for k in kept])
        return st
    st["new"] = _ints(new)
    st["src"], st["dst"] = (torch.full((num_pages,), -1, dtype=torch.int32, device=DEV) for _ in range(2))
    st["count"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    st["touch"] = max(_pages(n + p, page) - p // page for n, p in zip(new, cached))
    if c["op"] == "fork":
        st["parents"] = _ints(_parents(c))
        st["tables"] = [table, torch.full_like(table, -1)]
        st["lengths"] = [st["cached"], torch.zeros_like(st["cached"])]
        st["turn"], st["touch"] = 0, 1
    elif c["op"] == "compact":
        odd = torch.arange(B, device=DEV) % 2 == 1
        full = st["cached"].clone()
        st["full"], st["turn"] = full, 0
        st["ends"] = [torch.where(odd, full, 0), torch.where(odd, 0, full)]         # what each turn keeps
        st["comes"] = [torch.where(odd, 0, full), torch.where(odd, full, 0)]        # and takes in again
        st["touch"] = max_pages
    return st


# ------------------------------------------------------------------ plain forms

def _plain_attend(s):
    c = s["c"]
    B, H, n, L, page = s["B"], c["H"], s["max_new"], s["max_seq"], s["page"]
    t = torch.arange(s["T"], device=DEV)
    tok = torch.searchsorted(s["iro"].long(), t, right=True) - 1
    i = t - s["iro"].long()[tok]
    cached = s["cached"].long()
    q = torch.zeros(B, n, H, DN + DR, device=DEV)
    q[tok, i] = s["q"].float()
    full = torch.cat([torch.einsum("bnhd,hkd->bnhk", q[..., :DN], s["w_uk"].float()), q[..., DN:]], -1)
    j = torch.arange(L, device=DEV)
    row = s["table"].long()[:, j // page] * page + j % page
    k = s["cache"][row.clamp(min=0)].float()
    # Bit j - cached of the token's mask row, or j <= its own position; all of the cached.
    at = j - cached[:, None]
    count = (s["iro"].long()[1:] - s["iro"].long()[:-1])[:, None]
    seen = torch.zeros(B, n, L, dtype=torch.bool, device=DEV)
    inside = (at >= 0) & (at < count)
    if s["mask"] is None:
        seen[tok, i] = at[tok] <= i[:, None]
    else:
        a = at.clamp(0, 32 * s["words"] - 1)[tok]
        seen[tok, i] = (s["mask"].long().gather(1, a // 32) >> a % 32 & 1).bool()
    seen = seen & inside[:, None] | (at < 0)[:, None]
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


def _plain_keep(s):
    page = s["page"]
    k = torch.arange(s["width"], device=DEV)
    b, k = torch.nonzero(k < s["counts"][:, None], as_tuple=True)
    to = s["cached"].long()[b] + k
    fro = s["cached"].long()[b] + s["keep"].long()[b, k]
    table = s["table"].long()
    s["cache"][:, table[b, to // page] * page + to % page] = \
        s["cache"][:, table[b, fro // page] * page + fro % page]
    return {"cache": s["cache"]}


def _plain_reserve(s, table, lengths, new):
    """Pages for new[b] tokens behind lengths[b], in the order of (sequence,
    page): missing ones, and copies of pages that others hold too."""
    page, refs = s["page"], s["refs"]
    s["src"].fill_(-1), s["dst"].fill_(-1)
    first, end = lengths.long() // page, (lengths.long() + new.long() + page - 1) // page
    slot = first[:, None] + torch.arange(s["touch"], device=DEV)
    b, i = torch.nonzero((slot < end[:, None]) & (new > 0)[:, None], as_tuple=True)
    slot = slot[b, i]
    old = table[b, slot].long()
    # A page's writers in order: all but the last of its holders take a copy.
    by, at = torch.sort(torch.where(old < 0, s["num_pages"], old), stable=True)
    rank = torch.empty_like(at)
    rank[at] = torch.arange(at.numel(), device=DEV) - torch.searchsorted(by, by)
    shared = (old >= 0) & (rank < refs[old.clamp(min=0)] - 1)
    take = shared | (old < 0)
    b, i, slot, old, shared = b[take], i[take], slot[take], old[take], shared[take]
    got = torch.nonzero(refs == 0)[:b.numel(), 0]
    refs.index_add_(0, old[shared], torch.full_like(old[shared], -1).int())
    refs[got] = 1
    table[b, slot] = got.int()
    copy = shared & (i == 0) & (lengths[b] % page != 0)
    n = int(copy.sum())
    s["src"][:n], s["dst"][:n] = old[copy].int(), got[copy].int()
    s["count"].fill_(n)


def _plain_free(s, table, lengths, keep):
    keep = torch.zeros_like(lengths) if keep is None else torch.minimum(lengths, keep)
    lost = (torch.arange(s["max_pages"], device=DEV) >= ((keep + s["page"] - 1) // s["page"])[:, None]) & (table >= 0)
    gone = table[lost].long()
    s["refs"].index_add_(0, gone, torch.full_like(gone, -1).int())
    table.masked_fill_(lost, -1)
    lengths.copy_(keep)


def _plain_copy(s):
    n = int(s["count"])
    pages = s["cache"].view(s["c"]["layers"], s["num_pages"], -1)
    pages[:, s["dst"][:n].long()] = pages[:, s["src"][:n].long()]


def _plain_fork(s):
    k = s["turn"]
    s["turn"] = 1 - k
    table, lengths = s["tables"][1 - k], s["lengths"][1 - k]
    was, p = s["tables"][k], s["parents"].long()
    more = torch.bincount(p, minlength=s["B"]) - 1
    b, j = torch.nonzero(was >= 0, as_tuple=True)
    s["refs"].index_add_(0, was[b, j].long(), more[b].int())
    table.copy_(was[p])
    lengths.copy_(s["lengths"][k][p])
    _plain_reserve(s, table, lengths, s["new"])
    _plain_copy(s)
    return _fork_outputs(s, table, lengths)


def _plain_step(s):
    _plain_reserve(s, s["table"], s["cached"], s["new"])
    mid = {"table": s["table"].clone(), "refs": s["refs"].clone()}
    _plain_free(s, s["table"], s["cached"], s["cached"].clone() if s["c"]["cache_hi"] else None)
    return {**mid, "table_after": s["table"], "refs_after": s["refs"], "lengths": s["cached"]}


def _plain_compact(s):
    k = s["turn"]
    s["turn"] = 1 - k
    table, refs = s["table"], s["refs"]
    _plain_free(s, table, s["cached"], s["ends"][k])
    live, holes = torch.nonzero(refs > 0)[:, 0].flip(0), torch.nonzero(refs == 0)[:, 0]
    n = min(live.numel(), holes.numel())
    fits = holes[:n] < live[:n]
    src, dst = live[:n][fits], holes[:n][fits]
    s["src"].fill_(-1), s["dst"].fill_(-1)
    s["src"][:src.numel()], s["dst"][:src.numel()] = src.int(), dst.int()
    s["count"].fill_(src.numel())
    refs[dst] = refs[src]
    refs[src] = 0
    to = torch.arange(s["num_pages"] + 1, device=DEV, dtype=torch.int32)
    to[src], to[-1] = dst.int(), -1
    table.copy_(to[table.long()])
    _plain_copy(s)
    moves = (s["src"].clone(), s["dst"].clone(), s["count"].clone())
    _plain_reserve(s, table, s["cached"], s["comes"][k])
    s["cached"].copy_(s["full"])
    return _compact_outputs(s, moves)


def _fork_outputs(s, table, lengths):
    n = s["B"]
    return {"table": table, "lengths": lengths, "refs": s["refs"], "copy_src": s["src"][:n], "copy_dst": s["dst"][:n],
            "count": s["count"], "cache": s["cache"]}


def _compact_outputs(s, moves):
    return {"table": s["table"], "refs": s["refs"], "src": moves[0], "dst": moves[1], "count": moves[2],
            "cache": s["cache"]}


# ------------------------------------------------------------------ the library's calls

def _own_attend(s, mla):
    c = s["c"]
    if "ws" not in s:
        s["bytes"] = mla.mla_chunk_attention_workspace_bytes(s["B"], c["H"], s["T"])
        s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    mla.check(mla.mla_chunk_attention(
        s["out"], None, s["q"], s["iro"], s["cached"], s["cache"], s["table"], s["num_pages"], s["page"],
        s["max_pages"], s["w_uk"], s["w_uv"], s["B"], c["H"], s["T"], (DN + DR) ** -0.5, chunk_mask=s["mask"],
        mask_words=s["words"], attn_sink=s["sink"], workspace=s["ws"], workspace_bytes=s["bytes"],
        d_status=s["status"]))
    return {"out": s["out"]}


def _own_keep(s, mla):
    c = s["c"]
    mla.check(mla.mla_cache_keep_rows(
        s["cache"], SIZE[c["kind"]], c["layers"], s["num_pages"] * s["page"] * SIZE[c["kind"]], s["cached"],
        s["keep"], s["width"], s["counts"], s["table"], s["num_pages"], s["page"], s["max_pages"], s["B"],
        d_status=s["status"]))
    return {"cache": s["cache"]}


def _own_reserve(s, mla, table, lengths, new):
    if "ws" not in s:
        s["bytes"] = mla.mla_pages_workspace_bytes(s["num_pages"], s["B"])
        s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    mla.check(mla.mla_pages_reserve(
        table, s["refs"], lengths, new, s["src"], s["dst"], s["count"], s["num_pages"], s["page"], s["max_pages"],
        s["B"], workspace=s["ws"], workspace_bytes=s["bytes"], d_status=s["status"]))


def _own_free(s, mla, table, lengths, keep):
    mla.check(mla.mla_pages_free(table, s["refs"], lengths, keep, s["num_pages"], s["page"], s["max_pages"], s["B"],
                                 d_status=s["status"]))


def _own_copy(s, mla, most):
    c = s["c"]
    size = s["page"] * SIZE[c["kind"]]
    mla.check(mla.mla_pages_copy(s["cache"], size, c["layers"], s["num_pages"] * size, s["src"], s["dst"], s["count"],
                                 most, s["num_pages"], d_status=s["status"]))


def _own_fork(s, mla):
    k = s["turn"]
    s["turn"] = 1 - k
    table, lengths = s["tables"][1 - k], s["lengths"][1 - k]
    mla.check(mla.mla_pages_fork(table, lengths, s["tables"][k], s["lengths"][k], s["refs"], s["parents"],
                                 s["num_pages"], s["max_pages"], s["B"], s["B"], d_status=s["status"]))
    _own_reserve(s, mla, table, lengths, s["new"])
    _own_copy(s, mla, s["B"])
    return _fork_outputs(s, table, lengths)


def _own_step(s, mla):
    _own_reserve(s, mla, s["table"], s["cached"], s["new"])
    mid = {"table": s["table"].clone(), "refs": s["refs"].clone()}
    _own_free(s, mla, s["table"], s["cached"], s["cached"] if s["c"]["cache_hi"] else None)
    return {**mid, "table_after": s["table"], "refs_after": s["refs"], "lengths": s["cached"]}


def _own_compact(s, mla):
    k = s["turn"]
    s["turn"] = 1 - k
    _own_free(s, mla, s["table"], s["cached"], s["ends"][k])
    if "ws" not in s:
        s["bytes"] = mla.mla_pages_workspace_bytes(s["num_pages"], s["B"])
        s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    mla.check(mla.mla_pages_compact(
        s["table"], s["refs"], s["src"], s["dst"], s["count"], s["num_pages"], s["num_pages"], s["max_pages"], s["B"],
        workspace=s["ws"], workspace_bytes=s["bytes"], d_status=s["status"]))
    _own_copy(s, mla, s["num_pages"])
    moves = (s["src"].clone(), s["dst"].clone(), s["count"].clone())
    _own_reserve(s, mla, s["table"], s["cached"], s["comes"][k])
    s["cached"].copy_(s["full"])
    return _compact_outputs(s, moves)


def run(state):
    op = state["c"]["op"]
    if own:
        import mla_prefill_attention_plan_gb300 as mla
        return globals()["_own_" + op](state, mla)
    return globals()["_plain_" + op](state)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The attention's definition in 64 bits, one sequence at a time; the others
    move and count whole numbers, which have to be equal."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    c, (new, cached) = s["c"], _lengths(case)
    w_uk, w_uv = s["w_uk"].double(), s["w_uv"].double()
    bits = _mask_rows(c, new, seed) if s["mask"] is not None else None
    outs, t = [], 0
    for b, (n, p) in enumerate(zip(new, cached)):
        j = torch.arange(n + p, device=DEV)
        pages = s["table"][b].long()[torch.div(j, s["page"], rounding_mode="floor")]
        k = s["cache"][pages * s["page"] + j.remainder(s["page"])].double()
        for a in range(0, n, 16):
            z = min(n, a + 16)
            q = s["q"][t + a: t + z].double()
            lat = torch.bmm(q[..., :DN].transpose(0, 1), w_uk.transpose(1, 2)).transpose(0, 1)
            x = torch.cat([lat, q[..., DN:]], -1) @ k.T / math.sqrt(DN + DR)
            hide = [[not (bits[t + i] >> m & 1 if bits else m <= i) for m in range(n)] for i in range(a, z)]
            hide = torch.cat([torch.zeros(z - a, p, dtype=torch.bool, device=DEV), torch.tensor(hide, device=DEV)], 1)
            x = x.masked_fill(hide[:, None], -math.inf)
            if s["sink"] is not None:
                x = torch.cat([x, s["sink"][b].double().expand(z - a, x.shape[1], 1)], -1)
            lse = torch.logsumexp(x, -1)
            pr = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[..., None])[..., : n + p]
            outs.append(torch.bmm((pr @ k[:, :R]).transpose(0, 1), w_uv.transpose(1, 2)).transpose(0, 1))
        t += n
    return {"out": torch.cat(outs)}
