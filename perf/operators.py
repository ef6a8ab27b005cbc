"""Cases of the token-batch operators: a decode or verification step that feeds
several new tokens per sequence through the KV cache.

The operators, in the order in which a step calls them:

  plan    page tables, slot map, positions and tree masks of the new tokens,
          built on the GPU from the cache lengths and the tokens per sequence
  rope    rotary positions on q and k of every new token; k and v go to the
          cache (decode, prompt chunks) or stay packed (drafted tokens)
  tree    attention of the new tokens over their sequence's cache and over each
          other: a tree of drafted tokens by its mask, or a causal chunk
  commit  the accepted drafted tokens' rows go to the cache, lengths advance

A case is a dict of plain values. Lengths are drawn from the case alone (so
that its work is known) and given to the sequences in an order that the seed
decides; contents come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TREE_WORDS = 4          # a tree mask has 128 bits


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def _case(name, op, **kw):
    c = dict(op=op, dtype="bf16", B=1, Hq=32, Hkv=32, d=128, page=0, t=(0, 0), n=(1, 1), tree=0, pad=0,
             rot=0, interleaved=0, scaling="none", to_cache=1, accept=0, lens=1)
    c.update(kw)
    c["t0"], c["t1"] = c.pop("t")
    c["n0"], c["n1"] = c.pop("n")
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one verification step of a serving batch (32 sequences, 16-key pages): latency counts
        _case("plan_drafts", "plan", Hq=1, Hkv=1, d=64, B=32, page=16, t=(2048, 16384), n=(9, 64), tree=1, pad=7, lens=11),
        # prompts of a full batch are admitted at once: over a hundred thousand slots
        _case("plan_prompts", "plan", Hq=1, Hkv=1, d=64, B=256, page=64, t=(0, 4000), n=(1, 1024), pad=1, lens=12),
        # the smallest call: one decode token of one sequence, all heads, contiguous cache
        _case("rope_token", "rope", t=(4095, 4095), rot=128, lens=21),
        # a prompt chunk of 8 sequences written into a paged cache, grouped heads, long-context bands
        _case("rope_prompt", "rope", B=8, Hkv=8, page=16, t=(100, 4000), n=(1500, 2500), rot=128, scaling="bands",
              pad=3, lens=22),
        # fp32 cache of one head (the smallest shape the framework decodes), a tree of 13 tokens
        _case("tree_tiny_f32", "tree", dtype="f32", Hq=1, Hkv=1, d=64, t=(512, 512), n=(13, 13), tree=1, lens=31),
        # a tree of 16 drafted tokens over one 4096-key cache of 32 heads: latency and bandwidth
        _case("tree_llama", "tree", t=(4096, 4096), n=(16, 16), tree=1, lens=32),
        # grouped heads, four 32K-key caches, trees of 24 tokens (96 query rows a KV head)
        _case("tree_mistral", "tree", B=4, Hkv=8, t=(32768, 32768), n=(24, 24), tree=1, lens=33),
        # the serving batch: ragged paged caches, ragged trees, some sequences with one token
        _case("tree_paged", "tree", B=32, page=16, t=(2048, 16384), n=(1, 32), tree=1, pad=5, lens=34),
        # 131072 keys, a tree of 64 tokens: 256 query rows a KV head, bandwidth and tensor cores alike
        _case("tree_long", "tree", Hkv=8, t=(131072, 131072), n=(64, 64), tree=1, lens=35),
        # prompt chunks of two sequences on cached prefixes, causal: bound by the tensor cores
        _case("chunk_prompt", "tree", B=2, Hkv=8, page=64, t=(4000, 8200), n=(2000, 4200), lens=36),
        # the accepted path of one 26-token tree
        _case("commit_llama", "commit", t=(3000, 3000), n=(26, 26), tree=1, accept=6, lens=41),
        # accepted paths of a serving batch, up to 12 tokens each, 32 KV heads, paged
        _case("commit_paged", "commit", B=32, page=16, t=(20, 500), n=(12, 64), tree=1, accept=12, lens=42),
    ]


HEADS = [(1, 1), (8, 8), (32, 32), (8, 4), (32, 16), (16, 4), (32, 8), (32, 4), (8, 1), (64, 8)]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng, op):
    Hq, Hkv = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    page = rng.choice([0, 16, 16, 32, 64, 128, 48])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    pad = rng.choice([0, 0, 1, 6, 40])
    lens = rng.randrange(1 << 20)
    kw = dict(dtype=dtype, Hq=Hq, Hkv=Hkv, d=d, page=page, pad=pad, lens=lens)
    if op == "plan":
        tree = rng.randrange(2)
        n1 = _logint(rng, 1, 128 if tree else 2048)
        t1 = _logint(rng, 1, 40000)
        return _case(None, op, **{**kw, "B": _logint(rng, 1, 400), "t": (rng.choice([0, t1 // 3, t1]), t1),
                                  "n": (rng.choice([0, 1, n1]), n1), "tree": tree, "Hq": 1, "Hkv": 1, "d": 64})
    if op == "rope":
        rot = 16 * rng.randint(1, d // 16)
        n1 = _logint(rng, 1, 2500)
        t1 = _logint(rng, 1, 3000)
        return _case(None, op, **{**kw, "B": _logint(rng, 1, 16), "t": (t1 // 2, t1), "n": (rng.choice([1, n1]), n1),
                                  "rot": rot, "interleaved": rng.randrange(2), "to_cache": rng.randrange(2),
                                  "scaling": rng.choice(["none", "linear", "ntk", "bands", "ramp"])})
    if op == "tree":
        tree = rng.choice([1, 1, 0])
        n1 = _logint(rng, 1, 128 if tree else 4000)
        t1 = _logint(rng, 1, 131072)
        return _case(None, op, **{**kw, "B": _logint(rng, 1, 32), "t": (rng.choice([0, t1 // 4, t1]), t1),
                                  "n": (rng.choice([0, 1, n1]), n1), "tree": tree})
    n1 = _logint(rng, 1, 128)
    t1 = _logint(rng, 1, 500)
    return _case(None, op, **{**kw, "B": _logint(rng, 1, 32), "t": (t1 // 2, t1), "n": (rng.choice([1, n1]), n1),
                              "tree": 1, "accept": rng.randint(1, 16)})


def draw(rng):
    op = rng.choice(["plan", "rope", "tree", "tree", "tree", "commit"])
    most = {"bytes": 0, "flops": 0}
    for c in listed():
        if c["op"] == op:
            w = work(c)
            most = {k: max(most[k], w[k]) for k in most}
    while True:
        c = _draw_once(rng, op)
        if sum(_lengths(c)[1]) == 0:
            continue
        w = work(c)
        # fp32 products run on the CUDA cores, at a small part of the bf16 rate
        slow = 40 if c["dtype"] == "f32" and op == "tree" else 1
        if w["bytes"] <= most["bytes"] and w["flops"] * slow <= max(most["flops"], 1):
            return c


def _lengths(case):
    r = random.Random(case["lens"])
    t = [r.randint(case["t0"], case["t1"]) for _ in range(case["B"])]
    n = [r.randint(case["n0"], case["n1"]) for _ in range(case["B"])]
    return t, n


def _es(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    t, n = _lengths(case)
    T, B, Hq, Hkv, d, es = sum(n), case["B"], case["Hq"], case["Hkv"], case["d"], _es(case)
    if case["op"] == "plan":
        page = case["page"]
        new = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(t, n)) if page else 0
        cap = T + case["pad"]
        return {"bytes": B * 4 * 5 + cap * (8 + (20 if case["tree"] else 0)) + 8 * new, "flops": 0}
    if case["op"] == "rope":
        return {"bytes": 2 * T * (Hq + (2 if case["to_cache"] else 1) * Hkv) * d * es + 8 * T,
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    if case["op"] == "tree":
        pairs = sum(b * a + (b if case["tree"] else b * (b + 1) // 2) for a, b in zip(t, n))
        rows = sum(a + b for a, b in zip(t, n) if b)
        return {"bytes": rows * Hkv * 2 * d * es + T * Hq * (2 * d * es + 4) + (16 * T if case["tree"] else 0),
                "flops": 4 * d * Hq * pairs}
    m = sum(_accepted(case))
    return {"bytes": 4 * m * Hkv * d * es + 8 * m + 16 * B, "flops": 0}


def _accepted(case):
    r = random.Random(case["lens"] + 1)
    most = [min(case["accept"], b) for b in _lengths(case)[1]]
    return [r.randint(0 if b > 1 else b, b) for b in most]


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
class State:
    pass


def _i32(a):
    return torch.tensor(np.asarray(a, np.int64), dtype=torch.int32, device=DEV)


def prepare(case, seed):
    s = State()
    s.case, c = case, case
    rng = np.random.default_rng(1000003 * seed + 17)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * seed + 29)
    s.dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=s.dt)

    t, n = _lengths(c)
    m = _accepted(c)
    order = rng.permutation(c["B"])
    t, n, m = [t[i] for i in order], [n[i] for i in order], [m[i] for i in order]
    s.t, s.n, s.m = t, n, m
    B, Hq, Hkv, d, page, T = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], sum(n) + c["pad"]
    s.T, s.max_new = T, max(n)
    s.lens, s.n_new = _i32(t), _i32(n)
    cu = np.concatenate([[0], np.cumsum(n)])
    s.cu = _i32(cu)

    # parents of a drafted tree: an earlier token of the same sequence, or -1 (the last cached token)
    parents = np.full(T, -1, np.int64)
    for b in range(B):
        j = np.arange(n[b])
        par = j - 1 - rng.integers(0, 6, size=n[b])
        par[rng.random(n[b]) < 0.4] += 1
        parents[cu[b]:cu[b + 1]] = np.clip(np.minimum(par, j - 1), -1, None)
    s.parents = _i32(parents) if c["tree"] else None

    # the cache: contiguous, or pages in a random order
    most = max(a + b for a, b in zip(t, n))
    if page:
        s.mapped = [-(-a // page) for a in t]
        need = [-(-(a + b) // page) for a, b in zip(t, n)]
        s.max_blocks = max(1, max(need))
        pool = sum(need) + 3
        ids = rng.permutation(pool)
        table = np.full((B, s.max_blocks), -1, np.int64)
        full = np.full((B, s.max_blocks), -1, np.int64)
        at = 0
        for b in range(B):
            table[b, :s.mapped[b]] = ids[at:at + s.mapped[b]]
            full[b, :s.mapped[b]] = table[b, :s.mapped[b]]
            at += s.mapped[b]
        s.free = _i32(ids[at:])
        for b in range(B):
            full[b, s.mapped[b]:need[b]] = ids[at:at + need[b] - s.mapped[b]]
            at += need[b] - s.mapped[b]
        s.pool = pool
        s.table = _i32(table if c["op"] == "plan" else full)
        shape = (pool, Hkv, page, d)
        slot = [full[b][p // page] * page + p % page for b in range(B) for p in range(t[b], t[b] + n[b])]
    else:
        s.max_blocks, s.table = 0, None
        s.t_max = most + 5
        shape = (B, Hkv, s.t_max, d)
        slot = [b * s.t_max + p for b in range(B) for p in range(t[b], t[b] + n[b])]

    if c["op"] == "plan":
        s.k = s.v = torch.zeros(shape[0], Hkv, *shape[2:3], d, dtype=s.dt, device=DEV) if own else None
        s.n_pages = _i32(s.mapped) if page else None
        s.free_head = _i32([0]) if page else None
        z = dict(dtype=torch.int32, device=DEV)
        s.cu_out, s.positions, s.slots = torch.empty(B + 1, **z), torch.empty(T, **z), torch.empty(T, **z)
        s.mask = torch.empty(T, TREE_WORDS, **z) if c["tree"] else None
        s.free_head_out, s.n_pages_out = torch.empty(1, **z), torch.empty(B, **z)
    else:
        s.k, s.v = normal(*shape), normal(*shape)
        if c["op"] == "tree":
            # the first keys draw attention from every query, as sinks do
            for b in range(B):
                if page:
                    if t[b]:
                        s.k[int(full[b, 0]), :, :4, : d // 4] += 2.0
                else:
                    s.k[b, :, :4, : d // 4] += 2.0
        if c["op"] == "rope":
            pos = [p for b in range(B) for p in range(t[b], t[b] + n[b])]
            far = 100000 if c["scaling"] != "none" else 0          # chunks deep inside a long context
            s.positions = _i32([p + far for p in pos] + [0] * c["pad"])
            s.slots = _i32(list(slot) + [-1] * c["pad"])
            qkv = normal(T, (Hq + 2 * Hkv) * d)                    # the projection's output
            s.q = qkv[:, :Hq * d].view(T, Hq, d)
            s.kn = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
            s.vn = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
            s.q_out = torch.zeros(T, Hq, d, dtype=s.dt, device=DEV)
            s.k_out = torch.zeros(T, Hkv, d, dtype=s.dt, device=DEV)
            s.theta, s.mscale = _frequencies(c)
            s.theta = torch.tensor(s.theta, dtype=torch.float64, device=DEV)
        elif c["op"] == "tree":
            s.q = normal(T, Hq, d)
            s.q[..., : d // 4] += 0.25
            s.kn = normal(T, Hkv, d)
            s.vn = normal(T, Hkv * d + 64)[:, :Hkv * d].view(T, Hkv, d)   # a view of a wider buffer
            s.scale = d ** -0.5
            s.mask = _mask_words(parents, cu, T) if c["tree"] else None
            s.out = torch.zeros(T, Hq, d, dtype=s.dt, device=DEV)
            s.lse = torch.zeros(T, Hq, dtype=torch.float32, device=DEV)
        else:
            s.kn, s.vn = normal(T, Hkv, d), normal(T, Hkv, d)
            acc = np.zeros((B, max(1, c["accept"])), np.int64)
            for b in range(B):
                acc[b, :m[b]] = np.sort(rng.choice(n[b], size=m[b], replace=False)) if m[b] else 0
            s.acc, s.acc_n, s.new_lens = _i32(acc), _i32(m), torch.empty(B, dtype=torch.int32, device=DEV)
    if own:
        import sparse_kv_selection_gb300 as S
        s.kv = S.KVCache(s.k, s.v, s.lens, Hq, block_table=s.table)
        if c["op"] == "rope":
            s.rope = S.RopeTable(c["rot"], base=10000.0, interleaved=bool(c["interleaved"]), **SCALING[c["scaling"]])
        if c["op"] == "tree":
            s.ws = S.make_tree_workspace(s.kv, s.max_new)
    return s


SCALING = {
    "none": {},
    "linear": dict(scaling="linear", factor=4.0),
    "ntk": dict(scaling="ntk", factor=8.0),
    "bands": dict(scaling="bands", factor=8.0, original=8192, low=1.0, high=4.0),
    "ramp": dict(scaling="ramp", factor=16.0, original=4096, low=1.0, high=32.0),
}


def _frequencies(case):
    """Radians a position of each rotated pair, and the factor on cos and sin."""
    rot, kind = case["rot"], SCALING[case["scaling"]]
    f = kind.get("factor", 1.0)
    base = 10000.0
    if case["scaling"] == "ntk" and rot > 2:
        base *= f ** (rot / (rot - 2))
    theta = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    mscale = 1.0
    if case["scaling"] == "linear":
        theta = [x / f for x in theta]
    elif case["scaling"] == "bands":
        L, low, high = kind["original"], kind["low"], kind["high"]
        out = []
        for x in theta:
            turns = L * x / (2 * math.pi)            # turns over the original context
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            out.append(keep * x + (1 - keep) * x / f)
        theta = out
    elif case["scaling"] == "ramp":
        L, low, high = kind["original"], kind["low"], kind["high"]

        def dim(turns):
            return rot * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(base))

        a = max(0, math.floor(dim(high)))
        z = min(rot - 1, math.ceil(dim(low)))
        out = []
        for i, x in enumerate(theta):
            g = min(1.0, max(0.0, (i - a) / max(z - a, 0.001)))
            out.append(g * x / f + (1 - g) * x)
        theta = out
        mscale = 0.1 * math.log(f) + 1.0
    return theta, mscale


def _mask_words(parents, cu, T):
    """The mask bits of every token: itself and its ancestors, 128 bits a token."""
    bits = np.zeros((T, 128), bool)
    for b in range(len(cu) - 1):
        for j in range(cu[b + 1] - cu[b]):
            r = cu[b] + j
            if parents[r] >= 0:
                bits[r] = bits[cu[b] + parents[r]]
            bits[r, j] = True
    words = np.packbits(bits, axis=1, bitorder="little").view("<i4")
    return torch.from_numpy(np.ascontiguousarray(words)).to(DEV)


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def run(s):
    return {"plan": _plan, "rope": _rope, "tree": _tree, "commit": _commit}[s.case["op"]](s)


def _plan(s):
    c = s.case
    if own:
        import sparse_kv_selection_gb300 as S
        S.plan_tokens(s.kv, s.n_new, s.cu_out, s.positions, s.slots, parents=s.parents, tree_mask=s.mask,
                      **(dict(free_pages=s.free, free_head=s.free_head, n_pages=s.n_pages,
                              free_head_out=s.free_head_out, n_pages_out=s.n_pages_out) if c["page"] else {}))
        out = dict(cu=s.cu_out, positions=s.positions, slots=s.slots)
        if c["tree"]:
            out["mask"] = s.mask
        if c["page"]:
            out.update(table=s.kv.block_table, head=s.free_head_out, pages=s.n_pages_out)
        return out
    B, T, page = c["B"], s.T, c["page"]
    n, t = s.n_new.long(), s.lens.long()
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(n, 0)])
    tok = torch.arange(T, device=DEV)
    b = (tok[:, None] >= cu[None, 1:]).sum(1)
    real = b < B
    b = torch.clamp(b, max=B - 1)
    local = tok - cu[b]
    where = t[b] + local
    out = {}
    if page:
        have = s.n_pages.long()
        want = torch.maximum((t + n + page - 1) // page, have)
        take = want - have
        before = torch.cumsum(take, 0) - take
        col = torch.arange(s.max_blocks, device=DEV)[None]
        from_free = before[:, None] + col - have[:, None] + s.free_head.long()
        fresh = (col >= have[:, None]) & (col < want[:, None])
        picked = s.free.long()[from_free.clamp(0, s.free.numel() - 1)]
        table = torch.where(fresh, picked, s.table.long())
        slots = table[b, (where // page).clamp(max=s.max_blocks - 1)] * page + where % page
        out.update(table=table.int(), head=(s.free_head.long() + take.sum()).int(), pages=want.int())
    else:
        slots = b * s.t_max + where
    depth = local
    if c["tree"]:
        # ancestors by doubling: after round r a token knows those up to 2^r steps above it
        start = cu[b]
        par = torch.where(real & (s.parents >= 0), s.parents.long() + start, -1)
        anc = (torch.arange(128, device=DEV)[None] == local[:, None]) & real[:, None]
        up = par
        for _ in range(7):
            has = (up >= 0)[:, None]
            at = up.clamp(min=0)
            anc = anc | (anc[at] & has)
            up = torch.where(up >= 0, up[at], -1)
        depth = anc.sum(1) - 1
        w = (anc.view(T, TREE_WORDS, 32).long() << torch.arange(32, device=DEV)).sum(-1)
        out["mask"] = torch.where(w >= 1 << 31, w - (1 << 32), w).int()
    out.update(cu=cu.int(), positions=torch.where(real, t[b] + depth, 0).int(),
               slots=torch.where(real, slots, -1).int())
    return {k: out[k] for k in ("cu", "positions", "slots", "mask", "table", "head", "pages") if k in out}


def _rope(s):
    c = s.case
    rot, Hkv, page = c["rot"], c["Hkv"], c["page"]
    if own:
        import sparse_kv_selection_gb300 as S
        S.rope_append(s.kv, s.rope, s.positions, s.q, s.kn, s.vn, s.q_out, slots=s.slots if c["to_cache"] else None,
                      k_out=None if c["to_cache"] else s.k_out)
        return dict(q=s.q_out, k=s.k, v=s.v) if c["to_cache"] else dict(q=s.q_out, k=s.k_out)
    angle = s.positions.double()[:, None] * s.theta[None]
    cos, sin = (torch.cos(angle) * s.mscale).float()[:, None], (torch.sin(angle) * s.mscale).float()[:, None]

    def turn(x):
        x, co, si = x.float(), cos[:x.shape[0]], sin[:x.shape[0]]
        r, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            a, z = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * co - z * si, a * si + z * co], -1).flatten(-2)
        else:
            a, z = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * co - z * si, a * si + z * co], -1)
        return torch.cat([r, rest], -1).to(s.dt)

    T = sum(s.n)
    if not c["to_cache"]:
        return dict(q=turn(s.q), k=turn(s.kn))
    q = s.q_out.clone()
    q[:T] = turn(s.q[:T])
    slots = s.slots[:T].long()
    stride = page if page else s.t_max
    # [slot rows][heads] of the cache: page (or sequence), head, row in it
    s.k[slots // stride, :, slots % stride] = turn(s.kn[:T])
    s.v[slots // stride, :, slots % stride] = s.vn[:T]
    return dict(q=q, k=s.k, v=s.v)


def _rows(s, x, b):
    """Keys or values of sequence b's cache, [Hkv][t][d]."""
    c, t = s.case, s.t[b]
    page = c["page"]
    if not page:
        return x[b, :, :t]
    if t == 0:
        return x.new_zeros(c["Hkv"], 0, c["d"])
    ids = s.table[b, :-(-t // page)].long()
    return x[ids].transpose(0, 1).reshape(c["Hkv"], -1, c["d"])[:, :t]


def _allowed(s, b, start, n):
    """[n][n] truth values: may drafted token j of sequence b see token p."""
    if s.case["tree"]:
        w = s.mask[start:start + n].long() & 0xffffffff
        return ((w[..., None] >> torch.arange(32, device=DEV)) & 1).bool().flatten(1)[:, :n]
    j = torch.arange(n, device=DEV)
    return j[None] <= j[:, None]


def _tree(s):
    c = s.case
    if own:
        import sparse_kv_selection_gb300 as S
        S.tree_attn(s.kv, s.q, s.kn, s.vn, s.scale, s.cu, s.max_new, s.out, s.lse, s.ws, tree_mask=s.mask)
        return dict(out=s.out, lse=s.lse)
    G, d, Hkv = c["Hq"] // c["Hkv"], c["d"], c["Hkv"]
    start = 0
    for b in range(c["B"]):
        n, t = s.n[b], s.t[b]
        if n == 0:
            continue
        rows = slice(start, start + n)
        see = torch.cat([torch.ones(n, t, dtype=torch.bool, device=DEV), _allowed(s, b, start, n)], 1)
        see = see.repeat_interleave(G, 0)
        step = max(1, min(Hkv, (1 << 29) // max(1, n * G * (t + n))))
        for h in range(0, Hkv, step):
            hs = slice(h, min(Hkv, h + step))
            k = torch.cat([_rows(s, s.k, b)[hs], s.kn[rows, hs].transpose(0, 1)], 1).float()
            v = torch.cat([_rows(s, s.v, b)[hs], s.vn[rows, hs].transpose(0, 1)], 1).float()
            q = s.q[rows].view(n, Hkv, G, d)[:, hs].permute(1, 0, 2, 3).reshape(-1, n * G, d).float()
            x = (q @ k.transpose(1, 2)) * s.scale
            x = torch.where(see[None], x, float("-inf"))
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            z = p.sum(-1, keepdim=True)
            o = (p @ v) / z
            s.out[rows].view(n, Hkv, G, d)[:, hs] = o.view(-1, n, G, d).permute(1, 0, 2, 3).to(s.dt)
            s.lse[rows].view(n, Hkv, G)[:, hs] = (top + torch.log(z)).view(-1, n, G).permute(1, 0, 2)
        start += n
    return dict(out=s.out, lse=s.lse)


def _commit(s):
    c = s.case
    if own:
        import sparse_kv_selection_gb300 as S
        S.commit_tokens(s.kv, s.cu, s.acc_n, s.new_lens, accept_idx=s.acc, k_new=s.kn, v_new=s.vn)
        return dict(lens=s.new_lens, k=s.k, v=s.v)
    m, page = s.acc_n.long(), c["page"]
    b = torch.repeat_interleave(torch.arange(c["B"], device=DEV), m, output_size=sum(s.m))
    i = torch.arange(sum(s.m), device=DEV) - (torch.cumsum(m, 0) - m)[b]
    src = s.cu.long()[b] + s.acc.long()[b, i]
    pos = s.lens.long()[b] + i
    if page:
        block, row = s.table.long()[b, pos // page], pos % page
    else:
        block, row = b, pos
    s.k[block, :, row] = s.kn[src]
    s.v[block, :, row] = s.vn[src]
    return dict(lens=(s.lens.long() + m).int(), k=s.k, v=s.v)


# --------------------------------------------------------------------------- #
# the definition in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "plan":
        return None                                  # whole numbers only
    if c["op"] == "commit":
        return None                                  # rows are copied, nothing is computed
    if c["op"] == "rope":
        T = s.T if not c["to_cache"] else sum(s.n)
        turn = torch.polar(torch.full((s.T, c["rot"] // 2), float(s.mscale), dtype=torch.float64, device=DEV),
                           s.positions.to(torch.float64).view(-1, 1) * s.theta.view(1, -1))

        def rotated(x):
            y = x.to(torch.float64)
            r = y[..., :c["rot"]]
            if c["interleaved"]:
                z = torch.complex(r[..., ::2].contiguous(), r[..., 1::2].contiguous()) * turn[:, None]
                r = torch.view_as_real(z).reshape(*r.shape)
            else:
                h = c["rot"] // 2
                z = torch.complex(r[..., :h].contiguous(), r[..., h:].contiguous()) * turn[:, None]
                r = torch.cat([z.real, z.imag], -1)
            return torch.cat([r, y[..., c["rot"]:]], -1)

        if not c["to_cache"]:
            return dict(q=rotated(s.q), k=rotated(s.kn))
        q = torch.zeros(s.T, c["Hq"], c["d"], dtype=torch.float64, device=DEV)
        q[:T] = rotated(s.q)[:T]
        k = s.k.to(torch.float64)
        kr = rotated(s.kn)
        per = c["page"] or s.t_max
        at = torch.div(s.slots[:T].long(), per, rounding_mode="floor")
        heads = torch.arange(c["Hkv"], device=DEV)
        k.index_put_((at[:, None], heads[None], (s.slots[:T].long() - at * per)[:, None]), kr[:T])
        return dict(q=q, k=k, v=None)
    G, d = c["Hq"] // c["Hkv"], c["d"]
    out = torch.zeros(s.T, c["Hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s.T, c["Hq"], dtype=torch.float64, device=DEV)
    ends = np.cumsum(s.n)
    for b in range(c["B"]):
        n, t = s.n[b], s.t[b]
        lo = int(ends[b]) - n
        if n == 0:
            continue
        bias = torch.full((n, n), -math.inf, dtype=torch.float64, device=DEV)
        bias[_allowed(s, b, lo, n)] = 0.0
        for h in range(c["Hkv"]):
            keys, vals = _rows(s, s.k, b)[h].double(), _rows(s, s.v, b)[h].double()
            for g in range(G):
                q = s.q[lo:lo + n, h * G + g].double() * s.scale
                x = torch.cat([q @ keys.T, q @ s.kn[lo:lo + n, h].double().T + bias], 1)
                z = torch.logsumexp(x, 1)
                w = torch.exp(x - z[:, None])
                out[lo:lo + n, h * G + g] = w[:, :t] @ vals + w[:, t:] @ s.vn[lo:lo + n, h].double()
                lse[lo:lo + n, h * G + g] = z
    return dict(out=out, lse=lse)
