"""Plain 64-bit forms of the token-batch operators and inputs for their tests."""
import math

import numpy as np
import torch

TREE_MAX, WORDS = 128, 4


# --------------------------------------------------------------------------- #
# plan
# --------------------------------------------------------------------------- #
def ancestors(parents):
    """Ancestor sets (with itself) of one tree; parents outside [-1, j) read as -1."""
    out = []
    for j, p in enumerate(parents):
        out.append({j} | (out[p] if 0 <= p < j else set()))
    return out


def words_of(sets, T):
    w = np.zeros((T, WORDS), np.uint32)
    for i, s in enumerate(sets):
        for j in s:
            w[i, j // 32] |= np.uint32(1 << (j % 32))
    return w.view(np.int32)


def plan_ref(t, n, T, t_max, *, parents=None, page=0, table=None, free=None, head=0, n_pages=None):
    """(cu, positions, slots, masks, table, head, n_pages) of prhs_plan_tokens."""
    B = len(t)
    cu = [0]
    for x in n:
        cu.append(min(T, cu[-1] + max(0, x)))
    pos, slots, sets = np.zeros(T, int), np.full(T, -1), [set()] * T
    taken = 0
    table = None if table is None else np.array(table)
    pages = None if n_pages is None else list(n_pages)
    want_sum = 0
    for b in range(B):
        ok = n[b] >= 0 and not (parents is not None and n[b] > TREE_MAX)
        if n[b] > 0 and (t[b] + n[b] > t_max or cu[b] + n[b] > T):
            ok = False
        if page and ok and n[b] > 0:
            take = max(0, -(-(t[b] + n[b]) // page) - pages[b])
            if take and head + want_sum + take > len(free):
                ok = False
            if ok:
                for k in range(take):
                    table[b, pages[b] + k] = free[head + want_sum + k]
                if take:
                    taken = want_sum + take
                pages[b] += take
            want_sum += take
        anc = None
        if parents is not None and cu[b + 1] - cu[b] <= TREE_MAX:
            anc = ancestors(parents[cu[b]:cu[b + 1]])
        for j in range(cu[b + 1] - cu[b]):
            p = t[b] + j
            pos[cu[b] + j] = p
            if anc is not None:
                sets[cu[b] + j] = anc[j]
                pos[cu[b] + j] = t[b] + len(anc[j]) - 1
            if ok:
                slots[cu[b] + j] = table[b, p // page] * page + p % page if page else b * t_max + p
    return np.array(cu), pos, slots, words_of(sets, T), table, head + taken, pages


# --------------------------------------------------------------------------- #
# rope
# --------------------------------------------------------------------------- #
def rope_ref(x, positions, theta, mscale, rot, interleaved):
    """Rotation of [T][H][d] float64 rows."""
    ang = np.asarray(positions, np.float64)[:, None] * np.asarray(theta, np.float64)[None]
    c, s = (np.cos(ang) * mscale)[:, None], (np.sin(ang) * mscale)[:, None]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    return y


def theta_ref(rot, base=10000.0, kind=None, factor=1.0, original=0.0, low=0.0, high=0.0):
    i = np.arange(rot // 2)
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    th = base ** (-2.0 * i / rot)
    if kind == "linear":
        return th / factor, 1.0
    if kind == "bands":
        keep = np.clip((original / (2 * np.pi / th) - low) / (high - low), 0, 1)
        return keep * th + (1 - keep) * th / factor, 1.0
    if kind == "ramp":
        where = [rot * math.log(original / (x * 2 * math.pi)) / (2 * math.log(base)) for x in (high, low)]
        a, z = max(math.floor(where[0]), 0), min(math.ceil(where[1]), rot - 1)
        g = np.clip((i - a) / max(z - a, 0.001), 0, 1)
        return g * th / factor + (1 - g) * th, 0.1 * math.log(factor) + 1
    return th, 1.0


# --------------------------------------------------------------------------- #
# a cache with its logical rows
# --------------------------------------------------------------------------- #
class Cache:
    """A contiguous or paged cache of given lengths on the GPU; rows beyond each
    length hold NaN, so that using one shows."""

    def __init__(self, lens, Hq, Hkv, d, dtype, page=0, room=0, seed=0, t_max=None, spare=0):
        import sparse_kv_selection_gb300 as S
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.Hq, self.Hkv, self.d, self.dtype = list(lens), page, Hq, Hkv, d, dtype
        self.B = B = len(lens)
        most = max(lens) + room
        if page:
            have = [-(-t // page) for t in lens]
            need = [-(-(t + room) // page) for t in lens]
            pool = sum(need) + spare
            ids = rng.permutation(pool)
            self.table = np.full((B, max(1, max(need))), -1, np.int64)
            at = 0
            for b in range(B):
                self.table[b, :have[b]] = ids[at:at + have[b]]
                at += have[b]
            self.free, self.n_pages = ids[at:], have
            shape = (pool, Hkv, page, d)
        else:
            self.table = None
            shape = (B, Hkv, max(1, t_max or most), d)
        self.k = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        self.v = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        for b, t in enumerate(lens):
            if t:
                self.set_rows(b, 0, torch.randn(t, Hkv, d, generator=g, device="cuda", dtype=dtype),
                              torch.randn(t, Hkv, d, generator=g, device="cuda", dtype=dtype))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.kv = S.KVCache(self.k, self.v, torch.tensor(lens, **i32), Hq,
                            block_table=None if self.table is None else torch.tensor(self.table, **i32))

    @property
    def t_max(self):
        return self.kv.t_max

    def at(self, b, p):
        """Index of position p (an array) of sequence b in k and v: [block, :, row]."""
        p = np.asarray(p)
        if not self.page:
            return np.full(p.shape, b), p
        tab = self.kv.block_table[b].cpu().numpy() if hasattr(self, "kv") else self.table[b]
        return tab[p // self.page], p % self.page

    def set_rows(self, b, p0, k, v):
        blk, row = self.at(b, np.arange(p0, p0 + k.shape[0]))
        blk, row = torch.tensor(blk, device="cuda"), torch.tensor(row, device="cuda")
        self.k[blk, :, row] = k
        self.v[blk, :, row] = v

    def rows(self, b, t):
        """Logical K and V of positions [0, t) of sequence b, float64 [Hkv][t][d]."""
        blk, row = self.at(b, np.arange(t))
        blk, row = torch.tensor(blk, device="cuda", dtype=torch.long), torch.tensor(row, device="cuda", dtype=torch.long)
        return (self.k[blk, :, row].double().transpose(0, 1), self.v[blk, :, row].double().transpose(0, 1))


# --------------------------------------------------------------------------- #
# attention
# --------------------------------------------------------------------------- #
def attn_ref(q, kc, vc, kn, vn, see, scale, d, dtype):
    """One sequence in float64: q [n][Hq][d], cache rows [Hkv][t][d], new rows
    [n][Hkv][d], see [n][n]. Returns (out, lse, bound on |out|'s error, on lse's).

    The bounds count roundings. A logit of d products accumulated in fp32 is off
    by at most d 2^-23 L, L = scale sum |q_e k_e| (2^-23: adders may truncate),
    which is the relative error of its weight; sums of c weights add c / 16 + 64
    roundings of 2^-24 (running sums per 16 columns at least, and their joins).
    bf16 weights are rounded before the product with V: 2^-8; the result is
    rounded once to its type."""
    n, Hq, _ = q.shape
    Hkv, t = kc.shape[:2]
    G = Hq // Hkv
    k = torch.cat([kc, kn.transpose(0, 1)], 1).repeat_interleave(G, 0)   # [Hq][t + n][d]
    v = torch.cat([vc, vn.transpose(0, 1)], 1).repeat_interleave(G, 0)
    see = torch.cat([torch.ones(n, t, dtype=torch.bool, device=q.device), see], 1)[None]
    qh = q.transpose(0, 1)
    s = torch.where(see, (qh @ k.transpose(1, 2)) * scale, torch.tensor(-math.inf, dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(s, -1)
    w = torch.where(see, torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None]), 0.0)
    out = w @ v
    L = torch.where(see, qh.abs() @ k.abs().transpose(1, 2), 0.0).amax(-1) * abs(scale) if t + n else torch.zeros_like(lse)
    A = w @ v.abs()
    rel = d * 2.0 ** -23 * L + ((t + n) / 16 + 64) * 2.0 ** -24
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    weight = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    e_out = half * out.abs() + (1 + half) * (2 * rel + weight)[..., None] * A
    e_lse = rel + 2.0 ** -22 * (1 + lse.abs().nan_to_num(0, 0, 0))
    return out.transpose(0, 1), lse.T, e_out.transpose(0, 1), e_lse.T
