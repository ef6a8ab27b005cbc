"""Cases of the operators for sequences that share pages of one KV cache.

Several continuations of one prompt (samples, beams, many questions about one
document, many requests behind one system prompt) hold the same pages for what
they have in common:

  fork     rows of the batch become copies of other rows (beams trade places, a
           prompt gets more samples) or end: page tables, holders of each page,
           the free list, and the rows of the last pages to copy
  compact  sequences keep a list of their positions and give the other pages back
  copy     cache rows to other slots, K and V of every head: what fork and
           compact ask for
  attn     attention of new tokens over caches with common prefixes, each prefix
           read once for all its sequences; with find, the prefixes are found in
           the page tables in the same pass, as the first layer of a step does

A case is a dict of plain values. Lengths and the families' shapes are drawn from
the case alone (so that its work is known); which pages they get, the order of the
families in the batch and the contents come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
WORDS = 4               # a tree mask has 128 bits
FULL_ROWS = 256         # query rows a KV head of one sequence that fill a tile by themselves


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def _case(name, op, **kw):
    c = dict(op=op, dtype="bf16", Hq=32, Hkv=32, d=128, page=16, families=1, fan=(1, 1), prefix=(0, 0), rest=(0, 0),
             n=(1, 1), tree=0, pad=0, find=0, min_keys=256, stay=0.5, end=0.0, keep=0.0, kind="", lens=1)
    c.update(kw)
    for k in ("fan", "prefix", "rest", "n"):
        c[k + "0"], c[k + "1"] = c.pop(k)
    if name:
        c["name"] = name
    return c


TABLES = dict(Hq=1, Hkv=1, d=64)      # the page operators read no keys


def listed():
    return [
        # one step of a beam search: eight requests of eight beams trade places; latency counts
        _case("fork_beams", "fork", **TABLES, families=8, fan=(8, 8), prefix=(2000, 8000), rest=(1, 300), stay=0.4, lens=11),
        # a full batch on 16-key pages: long prompts, most rows start again from another one, some end
        _case("fork_batch", "fork", **TABLES, families=16, fan=(32, 32), prefix=(4000, 32768), rest=(1, 2000), stay=0.2,
              end=0.1, lens=12),
        # one long cache keeps 1/8 of its positions
        _case("compact_one", "compact", **TABLES, fan=(1, 1), prefix=(0, 0), rest=(4096, 4096), keep=0.125, lens=21),
        # a serving batch keeps 1/16 of ragged caches, some of which share prefixes
        _case("compact_batch", "compact", **TABLES, families=48, fan=(1, 4), prefix=(0, 4000), rest=(2048, 16384),
              keep=0.0625, lens=22),
        # the partly filled last pages of 32 new samples, 32 heads
        _case("copy_tails", "copy", kind="tails", families=4, fan=(8, 8), rest=(1, 4000), lens=31),
        # the kept rows of a serving batch, grouped heads
        _case("copy_kept", "copy", kind="kept", Hkv=8, families=32, rest=(1000, 4000), keep=0.25, lens=32),
        # fp32 cache of one head (the smallest shape the framework decodes), four samples of one prompt
        _case("attn_tiny_f32", "attn", dtype="f32", Hq=1, Hkv=1, d=64, page=0, fan=(4, 4), prefix=(512, 512), rest=(0, 40),
              lens=41),
        # sixteen samples of one 4096-key prompt, 32 heads, single tokens: latency and bandwidth
        _case("attn_samples", "attn", fan=(16, 16), prefix=(4096, 4096), rest=(1, 256), lens=42),
        # decode of eight families of sixteen, grouped heads, prefixes found in the same pass
        _case("attn_serve", "attn", Hkv=8, families=8, fan=(16, 16), prefix=(2000, 8200), rest=(16, 512), find=1, lens=43),
        # drafted trees of a batch behind one system prompt; most keys are the sequences' own
        _case("attn_drafts", "attn", page=64, fan=(32, 32), prefix=(2048, 2048), rest=(100, 2000), n=(1, 8), tree=1, pad=5,
              lens=44),
        # 32 questions about one document of 131072 keys
        _case("attn_long", "attn", Hkv=8, fan=(32, 32), prefix=(131072, 131072), rest=(20, 600), lens=45),
        # 24 short prompts behind one system prompt, causal: bound by the tensor cores
        _case("attn_prompts", "attn", Hkv=8, page=64, fan=(24, 24), prefix=(8192, 8192), rest=(0, 0), n=(20, 63), pad=3,
              lens=46),
    ]


HEADS = [(1, 1), (8, 8), (32, 32), (8, 4), (32, 16), (16, 4), (32, 8), (32, 4), (8, 1), (64, 8)]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng, op):
    kw = dict(page=rng.choice([16, 16, 32, 48, 64, 128]), lens=rng.randrange(1 << 20))
    families = _logint(rng, 1, 40)
    fan = _logint(rng, 1, 64)
    prefix = _logint(rng, 1, 33000)
    rest = _logint(rng, 1, 8000)
    kw.update(families=families, fan=(rng.choice([1, fan]), fan), prefix=(rng.choice([0, prefix // 2, prefix]), prefix),
              rest=(rng.choice([0, rest // 2]), rest))
    if op == "fork":
        return _case(None, op, **TABLES, **kw, stay=rng.uniform(0, 0.9), end=rng.choice([0.0, 0.2]))
    if op == "compact":
        return _case(None, op, **TABLES, **kw, keep=rng.choice([1.0, 0.5, 0.1, 0.02]))
    Hq, Hkv = rng.choice(HEADS)
    kw.update(Hq=Hq, Hkv=Hkv, d=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if op == "copy":
        if rng.random() < 0.4:
            return _case(None, op, **kw, kind="tails")
        return _case(None, op, **{**kw, "fan": (1, 1), "prefix": (0, 0), "page": rng.choice([0, kw["page"]])}, kind="kept",
                     keep=rng.uniform(0.02, 0.5))
    tree = rng.choice([0, 0, 1])
    n = _logint(rng, 1, 128 if tree else 300)
    kw["prefix"] = (rng.choice([0, 1]) * kw["prefix"][0], _logint(rng, 1, 131072))
    if kw["prefix"][0] > kw["prefix"][1]:
        kw["prefix"] = (kw["prefix"][1],) * 2
    page = rng.choice([kw["page"], kw["page"], 0])
    return _case(None, op, **{**kw, "page": page}, n=rng.choice([(1, 1), (0, 1), (1, n), (n, n)]), tree=tree,
                 pad=rng.choice([0, 0, 1, 6, 40]), find=rng.randrange(2) if page else 0,
                 min_keys=rng.choice([1, 256, 256, 1000]))


def draw(rng):
    op = rng.choice(["fork", "compact", "copy", "attn", "attn", "attn"])
    most = {"bytes": 0, "flops": 0}
    for c in listed():
        if c["op"] == op:
            w = work(c)
            most = {k: max(most[k], w[k]) for k in most}
    while True:
        c = _draw_once(rng, op)
        rows = _rows(c)
        if len(rows) * c["Hq"] > 16384:
            continue
        if op == "attn":
            if sum(r["n"] for r in rows) == 0:
                continue
            # a contiguous cache holds every prefix once a sequence
            held = max(r["t"] for r in rows) * len(rows) * c["Hkv"] * c["d"] * _es(c) * 2
            pairs = sum(r["t"] * c["Hkv"] * c["d"] for r in rows)      # what the plain form casts
            # the plain form looks for prefixes row by row
            if not c["page"] and held > 6e9 or pairs > 6e9 or c["find"] and len(rows) > 400:
                continue
        if op == "copy" and sum(_move_n(c)) == 0:
            continue
        w = work(c)
        # fp32 products run on the CUDA cores, at a small part of the bf16 rate
        slow = 40 if c["dtype"] == "f32" and op == "attn" else 1
        if w["bytes"] <= most["bytes"] and w["flops"] * slow <= max(most["flops"], 1):
            return c


def _rows(case):
    """The rows of the batch, family by family: what they share with the family,
    their lengths, new tokens, surplus pages, and (fork) the row they come from."""
    r = random.Random(case["lens"])
    page, out = case["page"], []
    for f in range(case["families"]):
        fan, prefix = r.randint(case["fan0"], case["fan1"]), r.randint(case["prefix0"], case["prefix1"])
        first = len(out)
        for i in range(fan):
            t = prefix + r.randint(case["rest0"], case["rest1"])
            n = r.randint(case["n0"], case["n1"])
            x = r.random()
            parent = first + i if x < case["stay"] else -1 if x < case["stay"] + case["end"] else first + r.randrange(fan)
            shared = 0 if fan == 1 else prefix // page * page if page else prefix
            out.append(dict(family=f, first=first, fan=fan, shared=shared, t=t, n=n, extra=r.randrange(2), parent=parent))
    return out


def _kept(case):
    """Positions that each row keeps: the first ones, the last ones and some between; None: all, untouched."""
    out, r = [], np.random.default_rng(case["lens"] + 1)
    for row in _rows(case):
        t, m = row["t"], _keep_n(case, row)
        if t == 0 or r.random() < 0.1 and case["families"] > 1:
            out.append(None)
            continue
        sinks, last = min(m, int(r.integers(0, 70))), 0
        if m < t:
            last = min(m - sinks, int(r.integers(0, 200)))
        middle = np.sort(r.choice(np.arange(sinks, t - last), m - sinks - last, replace=False))
        out.append(np.concatenate([np.arange(sinks), middle, np.arange(t - last, t)]).astype(np.int64))
    return out


def _keep_n(case, row):
    return max(1, int(row["t"] * case["keep"])) if row["t"] else 0


def _cap(case):
    return max(1, max(_keep_n(case, r) for r in _rows(case)))


def _move_n(case):
    """(copy) Rows that each row of the batch has copied: those of the last page of
    the family's first row, or a part of its second half."""
    rows = _rows(case)
    if case["kind"] == "tails":
        return [rows[r["first"]]["t"] % case["page"] for r in rows]
    return [min(int(r["t"] * case["keep"]), r["t"] // 2) for r in rows]


def _es(case):
    return 2 if case["dtype"] == "bf16" else 4


def _ceil(a, b):
    return -(-a // b)


def _table_sizes(case, rows):
    """(columns of the table, pages held, pages of the pool)"""
    page = case["page"]
    wide = max(1, max(_ceil(r["t"], page) + r["extra"] for r in rows))
    held = sum(_ceil(r["t"], page) + r["extra"] - (r["shared"] // page if i != r["first"] else 0)
               for i, r in enumerate(rows))
    return wide, held, held + sum(_ceil(r["t"], page) if case["op"] == "compact" else 1 for r in rows) + 2


def work(case):
    rows, op, page = _rows(case), case["op"], case["page"]
    B, Hq, Hkv, d, es = len(rows), case["Hq"], case["Hkv"], case["d"], _es(case)
    if op in ("fork", "compact"):
        wide, _, pool = _table_sizes(case, rows)
        # tables, holders and free list in and out, lengths and page counts, the list of copies
        cap = page if op == "fork" else _cap(case)
        return {"bytes": 8 * (B * wide + 2 * pool) + 4 * 5 * B + 8 * B * cap + (4 * B * cap if op == "compact" else 0),
                "flops": 0}
    if op == "copy":
        n = _move_n(case)
        tails = case["kind"] == "tails"          # (a family's children read one page)
        read = sum(x for x, r in zip(n, rows) if not tails or r is rows[r["first"]])
        return {"bytes": 2 * (read + sum(n)) * Hkv * d * es + 8 * B * (page if tails else max(1, max(n))), "flops": 0}
    T = sum(r["n"] for r in rows)
    pairs = sum(r["n"] * r["t"] + (r["n"] if case["tree"] else r["n"] * (r["n"] + 1) // 2) for r in rows)
    keys = sum(r["t"] - r["shared"] + r["n"] for r in rows if r["n"])
    for f in {r["first"]: r for r in rows}.values():
        if any(r["n"] for r in rows[f["first"]:f["first"] + f["fan"]]):
            keys += f["shared"]
    return {"bytes": keys * Hkv * 2 * d * es + T * Hq * (2 * d * es + 4) + (16 * T if case["tree"] else 0),
            "flops": 4 * d * Hq * pairs}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
class State:
    pass


def _i32(a):
    return torch.tensor(np.asarray(a, np.int64), dtype=torch.int32, device=DEV)


def _order(case, rng):
    """Rows of the batch: the families in the seed's order, parents renumbered."""
    rows = _rows(case)
    first = sorted({r["first"] for r in rows})
    out = []
    for f in rng.permutation(len(first)):
        a = first[f]
        for r in rows[a:a + rows[a]["fan"]]:
            out.append(dict(r, old=a))
    start, seen = {}, 0
    for r in out:
        start.setdefault(r["old"], seen)
        seen += 1
    for i, r in enumerate(out):
        r["first"] = start[r["old"]]
        r["case_row"] = r["old"] + i - r["first"]
        if r["parent"] >= 0:
            r["parent"] += r["first"] - r["old"]
    return out


def prepare(case, seed):
    s = State()
    s.case, c = case, case
    rng = np.random.default_rng(1000003 * seed + 17)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * seed + 29)
    s.dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=s.dt)

    s.rows = rows = _order(c, rng)
    s.B, page, Hq, Hkv, d = len(rows), c["page"], c["Hq"], c["Hkv"], c["d"]
    s.t = [r["t"] for r in rows]
    s.lens = _i32(s.t)
    if page:
        s.wide, held, s.pool = _table_sizes(c, rows)
        ids = rng.permutation(s.pool)
        table, shares, at = np.full((s.B, s.wide), -1, np.int64), np.zeros(s.pool, np.int64), 0
        for b, r in enumerate(rows):
            same = r["shared"] // page if b != r["first"] else 0
            have = _ceil(r["t"], page) + r["extra"]
            table[b, :same] = table[r["first"], :same]
            shares[table[b, :same]] += 1
            table[b, same:have] = ids[at:at + have - same]
            at += have - same
        s.host_table = table
        s.table, s.shares, s.free, s.head = _i32(table), _i32(shares), _i32(ids), _i32([at])
        s.n_pages = _i32([_ceil(r["t"], page) + r["extra"] for r in rows])
        shape = (s.pool, Hkv, page, d)
    else:
        s.table, s.t_max = None, max(s.t) + 1
        shape = (s.B, Hkv, s.t_max, d)

    if c["op"] in ("fork", "compact"):
        z = dict(dtype=torch.int32, device=DEV)
        s.k = s.v = torch.zeros(*shape, dtype=s.dt, device=DEV) if own else None
        s.out = dict(table_out=torch.empty_like(s.table), lens_out=torch.empty(s.B, **z), n_pages_out=torch.empty(s.B, **z),
                     page_shares_out=torch.empty_like(s.shares), free_pages_out=torch.empty_like(s.free),
                     free_head_out=torch.empty(1, **z))
        if c["op"] == "fork":
            s.parent, s.cap = _i32([r["parent"] for r in rows]), page
        else:
            kept, s.cap = _kept(c), _cap(c)
            keep, m = np.zeros((s.B, s.cap), np.int64), np.full(s.B, -1, np.int64)
            for b, r in enumerate(rows):
                k = kept[r["case_row"]]
                if k is not None:
                    keep[b, :len(k)], m[b] = k, len(k)
            s.keep, s.keep_n = _i32(keep), _i32(m)
        s.src, s.dst = torch.empty(s.B, s.cap, **z), torch.empty(s.B, s.cap, **z)
    elif c["op"] == "copy":
        s.k, s.v = normal(*shape), normal(*shape)
        moves = _move_n(c)
        cap = page if c["kind"] == "tails" else max(1, max(moves))
        src, dst = np.full((s.B, cap), -1, np.int64), np.full((s.B, cap), -1, np.int64)
        free = ids[at:] if page else None
        for b, r in enumerate(rows):
            m, t = moves[r["case_row"]], r["t"]
            if c["kind"] == "tails":         # to a free page
                f = rows[r["first"]]
                if m:
                    src[b, :m] = table[r["first"], f["t"] // page] * page + np.arange(m)
                    dst[b, :m] = free[b] * page + np.arange(m)
                continue
            mv, to = np.sort(rng.choice(np.arange(t // 2, t), m, replace=False)), np.arange(m)
            src[b, :m] = table[b, mv // page] * page + mv % page if page else b * s.t_max + mv
            dst[b, :m] = table[b, to // page] * page + to % page if page else b * s.t_max + to
        s.src, s.dst = _i32(src), _i32(dst)
    else:
        _prepare_attn(s, rng, normal, shape)
    if own:
        import sparse_kv_selection_gb300 as S
        s.kv = S.KVCache(s.k, s.v, s.lens, Hq, block_table=s.table)
        if c["op"] in ("fork", "compact"):
            s.ws = S.make_pages_workspace(s.kv)
        if c["op"] == "attn":
            s.ws = S.make_shared_workspace(s.kv, s.T, s.max_new)
    return s


def _prepare_attn(s, rng, normal, shape):
    c, rows = s.case, s.rows
    B, Hq, Hkv, d, page = s.B, c["Hq"], c["Hkv"], c["d"], c["page"]
    s.n = [r["n"] for r in rows]
    s.T, s.max_new = sum(s.n) + c["pad"], max(s.n)
    cu = np.concatenate([[0], np.cumsum(s.n)])
    s.cu, s.cu_host = _i32(cu), cu
    s.k, s.v = normal(*shape), normal(*shape)
    # the first keys draw attention from every query, as sinks do
    for b, r in enumerate(rows):
        if r["t"] and (b == r["first"] or not r["shared"]):
            s.k[int(s.host_table[b, 0]) if page else b, :, :4, : d // 4] += 2.0
    if not page:
        for b, r in enumerate(rows):
            if b != r["first"] and r["shared"]:
                s.k[b, :, :r["shared"]] = s.k[r["first"], :, :r["shared"]]
                s.v[b, :, :r["shared"]] = s.v[r["first"], :, :r["shared"]]
    s.q = normal(s.T, Hq, d)
    s.q[..., : d // 4] += 0.25
    s.kn = normal(s.T, Hkv, d)
    s.vn = normal(s.T, Hkv * d + 64)[:, :Hkv * d].view(s.T, Hkv, d)      # a view of a wider buffer
    s.scale = d ** -0.5
    s.mask = None
    if c["tree"]:
        bits = np.zeros((s.T, 128), bool)
        for b in range(B):
            for j in range(s.n[b]):
                up = j - 1 - int(rng.integers(0, 4))
                if up >= 0:
                    bits[cu[b] + j] = bits[cu[b] + up]
                bits[cu[b] + j, j] = True
        s.mask = torch.from_numpy(np.ascontiguousarray(np.packbits(bits, axis=1, bitorder="little").view("<i4"))).to(DEV)
    # what a program knows of its batch: (first row, rows, shared keys, 0) of each row
    share = []
    for b, r in enumerate(rows):
        one = r["fan"] == 1 or r["shared"] == 0
        share.append([b, 1, 0, 0] if one else [r["first"], r["fan"], r["shared"], 0])
    s.share = _i32(share)
    s.out = torch.zeros(s.T, Hq, d, dtype=s.dt, device=DEV)
    s.lse = torch.zeros(s.T, Hq, dtype=torch.float32, device=DEV)


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def run(s):
    return {"fork": _fork, "compact": _compact, "copy": _copy, "attn": _attn}[s.case["op"]](s)


def _pages(s):
    return dict(n_pages=s.n_pages, page_shares=s.shares, free_pages=s.free, free_head=s.head, **s.out)


def _result(table, lens, n_pages, shares, free, head, src, dst):
    return dict(table=table.int(), lens=lens.int(), n_pages=n_pages.int(), shares=shares.int(), free=free.int(),
                head=head.int(), src=src.int(), dst=dst.int())


def _own_result(s):
    o = s.out
    return dict(table=o["table_out"], lens=o["lens_out"], n_pages=o["n_pages_out"], shares=o["page_shares_out"],
                free=o["free_pages_out"], head=o["free_head_out"], src=s.src, dst=s.dst)


def _give_back(s, table, gone, added, taken):
    """Holders, free list and its head after the entries of `table` flagged in
    `gone` are released and `added` (entries per page) joined: a page without
    holders goes back in the order of the first entry that released it."""
    P, size = s.pool, table.numel()
    page = torch.where(gone, table, P).flatten()
    left = torch.zeros(P + 1, dtype=torch.long, device=DEV)
    left[:P] = s.shares.long() + added
    left.index_add_(0, page, torch.full_like(page, -1))
    number = torch.arange(size, device=DEV)
    first = torch.full((P + 1,), size, dtype=torch.long, device=DEV).scatter_reduce(0, page, number, "amin")
    back = (page < P) & (left[page] == -1) & (first[page] == number)
    count = back.sum()
    head = s.head.long() + taken - count
    free = torch.cat([s.free.long(), s.free.new_zeros(1).long()])
    to = torch.where(back, head + torch.cumsum(back.long(), 0) - 1, free.numel() - 1)
    free = free.scatter(0, to, page)
    return torch.clamp(left[:P], min=0), free[:-1], head


def _fork(s):
    if own:
        import sparse_kv_selection_gb300 as S
        S.fork_seqs(s.kv, s.parent, s.src, s.dst, s.ws, **_pages(s))
        return _own_result(s)
    B, M, page = s.B, s.wide, s.case["page"]
    table, t, held, parent = s.table.long(), s.lens.long(), s.n_pages.long(), s.parent.long()
    row, col = torch.arange(B, device=DEV), torch.arange(M, device=DEV)[None]
    moved = parent != row
    fork = moved & (parent >= 0)
    p = torch.where(fork, parent, row)
    lens = torch.where(moved & ~fork, 0, t[p])
    blocks = (lens + page - 1) // page
    part = fork & (lens % page != 0)
    last = table[p, (blocks - 1).clamp(min=0)]
    # the first child of a row that leaves takes its last page over, the others copy it
    first = torch.full((B,), B, dtype=torch.long, device=DEV).scatter_reduce(
        0, torch.where(part, p, 0), torch.where(part, row, B), "amin")
    heir = part & moved[p] & (first[p] == row) & (s.shares.long()[last.clamp(min=0)] == 0)
    need = part & ~heir
    new = s.free.long()[(s.head.long() + torch.cumsum(need.long(), 0) - 1).clamp(0, s.pool - 1)]
    out = torch.where(col < blocks[:, None], table[p], -1)
    out = torch.where(need[:, None] & (col == blocks[:, None] - 1), new[:, None], out)
    out = torch.where(col >= torch.maximum(held, blocks)[:, None], table, out)
    out = torch.where(moved[:, None], out, table)
    joins = fork[:, None] & (col < (blocks - need.long())[:, None])
    added = torch.zeros(s.pool + 1, dtype=torch.long, device=DEV).index_add_(
        0, torch.where(joins, table[p], s.pool).flatten(), torch.ones(B * M, dtype=torch.long, device=DEV))
    gone = moved[:, None] & (col < held[:, None])
    shares, free, head = _give_back(s, table, gone, added[:-1], need.sum())
    r = torch.arange(page, device=DEV)[None]
    rows = need[:, None] & (r < (lens % page)[:, None])
    return _result(out, lens, torch.where(moved, blocks, held), shares, free, head,
                   torch.where(rows, last[:, None] * page + r, -1), torch.where(rows, new[:, None] * page + r, -1))


def _compact(s):
    if own:
        import sparse_kv_selection_gb300 as S
        S.compact_seqs(s.kv, s.keep, s.keep_n, s.src, s.dst, s.ws, **_pages(s))
        return _own_result(s)
    B, M, page, cap = s.B, s.wide, s.case["page"], s.cap
    table, t, held, keep, m = s.table.long(), s.lens.long(), s.n_pages.long(), s.keep.long(), s.keep_n.long()
    row, col, i = torch.arange(B, device=DEV)[:, None], torch.arange(M, device=DEV)[None], torch.arange(cap, device=DEV)[None]
    acts = m >= 0
    valid = i < m[:, None]
    same = torch.cumprod(((keep == i) & valid).long(), 1).sum(1)
    stay = same // page
    # a sequence that is only cut short keeps its new last page if it holds it alone
    tail = table.gather(1, stay.clamp(max=M - 1)[:, None])[:, 0]
    stay = stay + ((same == m) & (m % page != 0) & (s.shares.long()[tail.clamp(min=0)] == 0)).long()
    blocks = (m.clamp(min=0) + page - 1) // page
    need = torch.where(acts, blocks - stay, 0)
    at = s.head.long() + torch.cumsum(need, 0) - need
    fresh = s.free.long()[(at[:, None] + col - stay[:, None]).clamp(0, s.pool - 1)]
    out = torch.where(col < stay[:, None], table, torch.where(col < blocks[:, None], fresh, -1))
    out = torch.where(acts[:, None] & (col < held[:, None]), out, table)
    gone = acts[:, None] & (col >= stay[:, None]) & (col < held[:, None])
    shares, free, head = _give_back(s, table, gone, 0, need.sum())
    moves = valid & (i >= (stay * page)[:, None])
    src = table[row, (keep // page).clamp(0, M - 1)] * page + keep % page
    dst = out[row, (i // page).clamp(0, M - 1)] * page + i % page
    return _result(out, torch.where(acts, m, t), torch.where(acts, blocks, held), shares, free, head,
                   torch.where(moves, src, -1), torch.where(moves, dst, -1))


def _copy(s):
    if own:
        import sparse_kv_selection_gb300 as S
        S.copy_rows(s.kv, s.src, s.dst)
        return dict(k=s.k, v=s.v)
    src, dst = s.src.flatten().long(), s.dst.flatten().long()
    # entries without a copy repeat one that is made
    at = torch.argmax((src >= 0).long())
    src, dst = torch.where(src >= 0, src, src[at]), torch.where(src >= 0, dst, dst[at])
    per = s.case["page"] or s.t_max
    for x in (s.k, s.v):
        x[dst // per, :, dst % per] = x[src // per, :, src % per]
    return dict(k=s.k, v=s.v)


def _find(s):
    """Families of consecutive rows with new tokens: a row joins the one before it
    while that does not lower what the family saves, (rows - 1) * shared pages."""
    c, page = s.case, s.case["page"]
    table, t = s.table.long(), s.lens.long()
    n = s.cu.long()[1:] - s.cu.long()[:-1]
    M, zero = s.wide, torch.zeros((), dtype=torch.long, device=DEV)
    col = torch.arange(M, device=DEV)
    share = torch.zeros(s.B, 4, dtype=torch.long, device=DEV)
    share[:, 0], share[:, 1] = torch.arange(s.B, device=DEV), 1
    number = torch.arange(s.B, device=DEV)
    head, last, size, common = zero - 1, zero - 1, zero, zero
    for b in range(s.B):
        active = n[b] > 0
        alone = n[b] * (c["Hq"] // c["Hkv"]) >= FULL_ROWS
        prev = last.clamp(min=0)
        pages = torch.minimum(t.index_select(0, prev.view(1))[0], t[b]) // page
        above = table.index_select(0, prev.view(1))[0]
        equal = torch.where(last >= 0, torch.cumprod(((above == table[b]) & (col < pages)).long(), 0).sum(), 0)
        new = torch.where(size == 1, equal, torch.minimum(common, equal))
        worth = (size == 1) | (size * new >= (size - 1) * common)
        joins = active & ~alone & (size > 0) & (new * page >= c["min_keys"]) & (new > 0) & worth
        keys = torch.where(joins, new * page, 0)
        of = (number >= head) & (number <= b) & (n > 0) & joins
        entry = torch.stack([head, b - head + 1, keys, zero])
        share = torch.where(of[:, None], entry[None], share)
        starts = active & ~joins
        head = torch.where(starts, zero + b, head)
        size = torch.where(starts, torch.where(alone, 0, 1), torch.where(joins, size + 1, size))
        common = torch.where(starts, 0, torch.where(joins, new, common))
        last = torch.where(active, zero + b, last)
    return share.int()


def _cached(s, x, b):
    """Keys or values of sequence b's cache, [Hkv][t][d]."""
    c, t, page = s.case, s.t[b], s.case["page"]
    if not page:
        return x[b, :, :t]
    if t == 0:
        return x.new_zeros(c["Hkv"], 0, c["d"])
    return x[s.table[b, :_ceil(t, page)].long()].transpose(0, 1).reshape(c["Hkv"], -1, c["d"])[:, :t]


def _allowed(s, start, n):
    """[n][n] truth values: may new token j see new token p."""
    if s.mask is not None:
        w = s.mask[start:start + n].long() & 0xffffffff
        return ((w[..., None] >> torch.arange(32, device=DEV)) & 1).bool().flatten(1)[:, :n]
    j = torch.arange(n, device=DEV)
    return j[None] <= j[:, None]


def _attn(s):
    c = s.case
    if own:
        import sparse_kv_selection_gb300 as S
        if c["find"]:
            S.find_shared(s.kv, s.cu, s.share, min_keys=c["min_keys"])
        S.shared_attn(s.kv, s.q, s.kn, s.vn, s.scale, s.cu, s.max_new, s.share, s.out, s.lse, s.ws, tree_mask=s.mask)
        return dict(out=s.out, lse=s.lse, **(dict(share=s.share) if c["find"] else {}))
    G, d, Hkv = c["Hq"] // c["Hkv"], c["d"], c["Hkv"]
    for b in range(s.B):
        n, t, start = s.n[b], s.t[b], int(s.cu_host[b])
        if n == 0:
            continue
        at = slice(start, start + n)
        see = torch.cat([torch.ones(n, t, dtype=torch.bool, device=DEV), _allowed(s, start, n)], 1).repeat_interleave(G, 0)
        k = torch.cat([_cached(s, s.k, b), s.kn[at].transpose(0, 1)], 1).float()
        v = torch.cat([_cached(s, s.v, b), s.vn[at].transpose(0, 1)], 1).float()
        q = s.q[at].view(n, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, n * G, d).float()
        step = max(1, min(Hkv, (1 << 28) // max(1, n * G * (t + n))))
        for h in range(0, Hkv, step):
            x = (q[h:h + step] @ k[h:h + step].transpose(1, 2)) * s.scale
            x = torch.where(see[None], x, float("-inf"))
            top = x.amax(-1, keepdim=True)
            w = torch.exp(x - top)
            z = w.sum(-1, keepdim=True)
            o = (w @ v[h:h + step]) / z
            s.out[at].view(n, Hkv, G, d)[:, h:h + step] = o.view(-1, n, G, d).permute(1, 0, 2, 3).to(s.dt)
            s.lse[at].view(n, Hkv, G)[:, h:h + step] = (top + torch.log(z)).view(-1, n, G).permute(1, 0, 2)
    return dict(out=s.out, lse=s.lse, **(dict(share=_find(s)) if c["find"] else {}))


# --------------------------------------------------------------------------- #
# the definition in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    c = case
    if c["op"] != "attn":
        return None                                  # whole numbers, or rows that are copied
    s = prepare(case, seed)
    G, Hkv, d = c["Hq"] // c["Hkv"], c["Hkv"], c["d"]
    out = torch.zeros(s.T, c["Hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s.T, c["Hq"], dtype=torch.float64, device=DEV)
    for b in range(s.B):
        lo, hi, t = int(s.cu_host[b]), int(s.cu_host[b + 1]), s.t[b]
        if lo == hi:
            continue
        bias = torch.full((hi - lo, hi - lo), -math.inf, dtype=torch.float64, device=DEV)
        bias[_allowed(s, lo, hi - lo)] = 0.0
        kc, vc = _cached(s, s.k, b), _cached(s, s.v, b)
        for h in range(Hkv):
            keys, vals = kc[h].double(), vc[h].double()
            q = s.q[lo:hi, h * G:(h + 1) * G].double().transpose(0, 1) * s.scale          # [G][n][d]
            x = torch.cat([q @ keys.T, q @ s.kn[lo:hi, h].double().T + bias], 2)
            z = torch.logsumexp(x, 2)
            w = torch.exp(x - z[..., None])
            out[lo:hi, h * G:(h + 1) * G] = (w[..., :t] @ vals + w[..., t:] @ s.vn[lo:hi, h].double()).transpose(0, 1)
            lse[lo:hi, h * G:(h + 1) * G] = z.T
    return dict(out=out, lse=lse, **(dict(share=None) if c["find"] else {}))
