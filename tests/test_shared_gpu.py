"""Attention of new tokens over caches with common prefixes that are read once,
against the plain form in 64 bits (tokens_util.attn_ref, whose bounds count the
roundings; the join of a token's two states adds a handful to its 64 spare ones)."""
import numpy as np
import pytest

from tokens_util import WORDS, Cache, ancestors, attn_ref, words_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Batch:
    """Families [(rows, shared keys)] of a cache; each row has its own further keys
    and its new tokens."""

    def __init__(self, families, rest, n, Hq, Hkv, d, dtype, page=0, tree=False, pad=3, seed=0, wide=8):
        rng = np.random.default_rng(seed)
        self.first, self.keys = [], []
        for rows, keys in families:
            f = len(self.first)
            self.first += [f] * rows
            self.keys += [keys] * rows
        B = len(self.first)
        pick = lambda x: [int(v) for v in (rng.integers(x[0], x[1] + 1, B) if isinstance(x, tuple) else x)]  # noqa: E731
        self.lens = [k + r for k, r in zip(self.keys, pick(rest))]
        self.n = pick(n)
        self.c = c = Cache(self.lens, Hq, Hkv, d, dtype, page=page, room=1, seed=seed)
        self.share = []
        for b in range(B):
            f, rows, keys = self.first[b], self.first.count(self.first[b]), self.keys[b]
            if page:
                keys = keys // page * page
                c.kv.block_table[b, :keys // page] = c.kv.block_table[f, :keys // page].clone()
            elif b != f:                       # the first row's keys stand for all rows'
                c.k[b, :, :keys] = float("nan")
                c.v[b, :, :keys] = float("nan")
            self.keys[b] = keys
            self.share.append([f, rows, self.keys[b], 0] if rows > 1 and keys else [b, 1, 0, 0])
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        self.T = T = sum(self.n) + pad
        self.cu = np.concatenate([[0], np.cumsum(self.n)])
        mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
        self.q = mk(T, Hq, d)
        self.kn = mk(T, Hkv * d + wide * 8)[:, :Hkv * d].view(T, Hkv, d)
        self.vn = mk(T, Hkv * d + wide * 16)[:, wide * 8:wide * 8 + Hkv * d].view(T, Hkv, d)
        self.sets, self.mask = None, None
        if tree:
            par = [[int(max(-1, j - 1 - rng.integers(0, 5))) for j in range(x)] for x in self.n]
            self.sets = [ancestors(p) for p in par]
            self.mask = torch.tensor(words_of(sum(self.sets, []) + [set()] * pad, T), device="cuda")
        self.scale = d ** -0.5

    def ref(self, b):
        c, n = self.c, self.n[b]
        kc, vc = c.rows(b, self.lens[b])
        if not c.page and self.share[b][2]:
            k0, v0 = c.rows(self.share[b][0], self.share[b][2])
            kc, vc = torch.cat([k0, kc[:, k0.shape[1]:]], 1), torch.cat([v0, vc[:, v0.shape[1]:]], 1)
        at = slice(int(self.cu[b]), int(self.cu[b + 1]))
        see = torch.tril(torch.ones(n, n, dtype=torch.bool, device="cuda"))
        if self.sets is not None:
            see[:] = False
            for j, s in enumerate(self.sets[b]):
                see[j, list(s)] = True
        return attn_ref(self.q[at].double(), kc, vc, self.kn[at].double(), self.vn[at].double(), see, self.scale, c.d, c.dtype)

    def run(self, share=None, cu=None, max_new=None, ws=None, out=None):
        import sparse_kv_selection_gb300 as S
        c = self.c
        max_new = max(1, max(self.n)) if max_new is None else max_new
        if out is None:
            out = (torch.full((self.T, c.Hq, c.d), 7.0, dtype=c.dtype, device="cuda"),
                   torch.full((self.T, c.Hq), 7.0, dtype=F32, device="cuda"))
        if ws is None:
            ws = S.make_shared_workspace(c.kv, self.T, max_new)
            ws.fill_(0xff)                     # (needs no initialisation)
        S.shared_attn(c.kv, self.q, self.kn, self.vn, self.scale, i32(self.cu if cu is None else cu), max_new,
                      i32(self.share if share is None else share), out[0], out[1], ws, tree_mask=self.mask)
        return out

    def check(self, out, rows=None):
        o, l = out
        for b in range(len(self.n)) if rows is None else rows:
            if self.n[b] == 0:
                continue
            at = slice(int(self.cu[b]), int(self.cu[b + 1]))
            want, lse, e_out, e_lse = self.ref(b)
            assert ((o[at].double() - want).abs() <= e_out).all(), b
            assert ((l[at].double() - lse).abs() <= e_lse).all(), b
        assert (o[self.cu[-1]:] == 7.0).all() and (l[self.cu[-1]:] == 7.0).all()   # padding is left alone


def full(*args, **kw):
    import sparse_kv_selection_gb300 as S
    b = Batch(*args, **kw)
    out = b.run()
    assert S.last_error() == 0
    b.check(out)
    again = b.run()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
    return b, out


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (4, 4, 128), (8, 4, 64), (8, 2, 128), (8, 1, 64), (16, 2, 128)])
@pytest.mark.parametrize("page", [0, 16, 48, 128])
def test_single_tokens(dtype, Hq, Hkv, d, page):
    """Decode: families of every size, rows that are alone, rows without tokens."""
    full([(1, 0), (3, 300), (2, 128), (5, 640), (1, 70), (2, 1)], (0, 200), (0, 1), Hq, Hkv, d, dtype, page, seed=page + d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,page", [(2, 2, 64, 16), (8, 2, 128, 64), (8, 1, 128, 0), (4, 2, 64, 48)])
@pytest.mark.parametrize("n", [(1, 4), (0, 33), (60, 128)])
def test_several_tokens(dtype, tree, Hq, Hkv, d, page, n):
    full([(4, 260), (1, 0), (3, 96), (2, 1000)], (0, 150), n, Hq, Hkv, d, dtype, page, tree=tree, seed=n[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys,page", [(127, 0), (128, 0), (129, 0), (16, 16), (112, 16), (144, 16), (48, 48), (1920, 128)])
def test_prefixes_around_tiles(dtype, keys, page):
    """Shared keys around whole tiles, with and without keys of the rows' own."""
    full([(3, keys), (2, keys)], (0, 0), (1, 1), 4, 2, 64, dtype, page, seed=keys)
    full([(3, keys), (2, keys)], (1, 130), (1, 2), 4, 2, 64, dtype, page, seed=keys)


@pytest.mark.parametrize("dtype,keys", [(BF16, 60000), (F32, 20000)])
def test_long_prefix(dtype, keys):
    """One prefix over all CTAs, many records of a unit."""
    full([(9, keys)], (0, 500), (1, 3), 8, 2, 128, dtype, 16, seed=1)
    full([(70, keys // 10)], (0, 30), (1, 1), 8, 1, 64, dtype, 64, seed=2)      # more than two row tiles


def test_many_short_sequences():
    full([(2, 16)] * 100 + [(1, 0)] * 56, (0, 20), (0, 2), 2, 2, 64, BF16, 16, seed=3)
    full([(128, 32), (72, 16)], (0, 20), (0, 2), 2, 1, 64, F32, 16, seed=4)


def test_largest_batch():
    import sparse_kv_selection_gb300 as S
    b = Batch([(8, 16)] * 2048, (0, 3), (1, 1), 1, 1, 64, BF16, 16, seed=5)
    out = b.run()
    assert S.last_error() == 0
    b.check(out, rows=list(range(0, 16384, 41)) + list(range(16376, 16384)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [(0, 1), (0, 6)])
def test_small_groups_far_apart(dtype, n):
    """More sequences than are kept at hand; few of them have a group, and few of the
    batch's items have keys for the launch that looks for them."""
    rng = np.random.default_rng(n[1])
    families = [(int(rng.integers(1, 60)), int(rng.integers(0, 90)) if f % 3 == 0 else 0) for f in range(16)]
    full(families, (0, 500), n, 8, 4, 64, dtype, 16, seed=n[1])
    full([(1, 0)] * 150 + [(2, 64)] + [(1, 0)] * 150 + [(3, 256)] + [(1, 0)] * 150, (0, 300), n, 8, 4, 64, dtype, 0, seed=n[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_causal_chunks_share(dtype):
    """Chunks that fill tiles by themselves may share too."""
    full([(3, 500)], (0, 40), (200, 300), 4, 1, 64, dtype, 16, seed=6)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rest", [(0, 90), (5000, 6000)])
def test_alone_as_tree_attention(dtype, rest):
    """Without groups it is tree_attn."""
    import sparse_kv_selection_gb300 as S
    b = Batch([(5, 300), (2, 64)], rest, (0, 5), 4, 2, 64, dtype, 16, seed=7)
    b.check(b.run(share=[[i, 1, 0, 0] for i in range(7)]))
    o, l = torch.full((b.T, 4, 64), 7.0, dtype=dtype, device="cuda"), torch.full((b.T, 4), 7.0, device="cuda")
    S.tree_attn(b.c.kv, b.q, b.kn, b.vn, b.scale, i32(b.cu), max(b.n), o, l, S.make_tree_workspace(b.c.kv, max(b.n)))
    assert S.last_error() == 0
    b.check((o, l))


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 4, 64), (8, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("n,rest", [((1, 1), (400, 4200)), ((1, 9), (500, 2100)), ((1, 64), (0, 700)), ((1, 1), (4000, 9000)),
                                    ((30, 128), (900, 1100))])
def test_own_keys_of_every_length(Hq, Hkv, d, n, rest):
    """Own keys that several CTAs share, and those left to the tcgen05 kernel."""
    full([(3, 130), (2, 64), (1, 0)], rest, n, Hq, Hkv, d, BF16, 16, seed=rest[1])
    full([(3, 130), (1, 0)], rest, n, Hq, Hkv, d, BF16, 0, tree=n[1] > 1, seed=n[1])


def test_shared_keys_are_whole_pages():
    """Shared keys that end inside a page are rounded down to it."""
    b = Batch([(3, 64), (2, 32)], (20, 60), (1, 2), 4, 2, 64, BF16, 16, seed=8)
    for extra in (0, 1, 15):
        out = b.run(share=[[f, r, k + extra, 0] for f, r, k, _ in b.share])
        b.check(out)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_entries_that_do_not_fit(dtype):
    """Flagged, and the row attends its own keys."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_INDEX
    b = Batch([(4, 64), (3, 32)], (16, 60), (1, 2), 4, 2, 64, dtype, 16, seed=9)
    for row, entry in [(2, [5, 4, 64, 0]), (2, [-1, 4, 64, 0]), (2, [1 << 30, 4, 64, 0]), (3, [2, 4, 64, 0]), (5, [0, 4, 64, 0]),
                       (0, [0, 4, 1 << 20, 0]), (0, [0, 4, -16, 0]), (0, [0, 2, 64, 0]), (6, [6, 5, 1 << 20, 0])]:
        share = [list(x) for x in b.share]
        share[row] = entry
        out = b.run(share=share)
        assert S.last_error() == DEV_BAD_INDEX, (row, entry)
        b.check(out)
    # a length below the shared keys: that row alone is flagged
    b = Batch([(4, 64)], (16, 60), (1, 2), 4, 2, 64, dtype, 16, seed=10)
    b.c.kv.seq_lens[2] = b.lens[2] = 40
    out = b.run()
    assert S.last_error() == DEV_BAD_INDEX
    b.check(out)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lengths_and_groups_that_change_between_calls(dtype):
    """Calls back to back on one cache, lengths, offsets and groups written by copies in between."""
    import sparse_kv_selection_gb300 as S
    B = 96
    b = Batch([(24, 512)] * 4, (40, 400), (1, 1), 8, 4, 64, dtype, 16, pad=B, seed=40)
    rng = np.random.default_rng(41)
    full_lens = np.array(b.lens)
    states = []
    for i in range(8):
        cut = 0 if i % 3 == 0 else int(rng.integers(0, 512))
        n = rng.integers(0, 2 + i % 2, B)
        share = [[f, r, cut // 16 * 16 if i % 2 else k // 32 * 16, 0] for f, r, k, _ in b.share]
        share = [[j, 1, 0, 0] if not s[2] else s for j, s in enumerate(share)]
        states.append([i32(full_lens - rng.integers(0, 40, B)), i32(np.concatenate([[0], np.cumsum(n)])), i32(share)])
    lens, cu, share = (x.clone() for x in states[0])
    kv = S.KVCache(b.c.k, b.c.v, lens, b.c.Hq, block_table=b.c.kv.block_table)
    ws = S.make_shared_workspace(kv, b.T, 2)
    out = (torch.empty(b.T, b.c.Hq, b.c.d, dtype=dtype, device="cuda"), torch.empty(b.T, b.c.Hq, device="cuda"))

    def results(wait):
        got = []
        for s in states * 3:
            for x, y in zip((lens, cu, share), s):
                x.copy_(y)
            for x in out:
                x.fill_(7.0)
            if wait:
                torch.cuda.synchronize()
            S.shared_attn(kv, b.q, b.kn, b.vn, b.scale, cu, 2, share, *out, ws)
            if wait:
                torch.cuda.synchronize()
            got.append([x.clone() for x in out])
        return got

    for x, y in zip(results(True), results(False)):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert S.last_error() == 0


def test_batches_on_streams_of_their_own():
    """Four batches at once, each with its own workspace, eager and from graphs."""
    import sparse_kv_selection_gb300 as S
    sizes = [([(16, 4096)], (0, 200), (1, 1), 8, 8, 128, BF16, 16), ([(40, 700), (3, 64)], (0, 900), (0, 6), 16, 4, 64, BF16, 64),
             ([(60, 500)], (0, 900), (1, 1), 8, 2, 64, F32, 16), ([(4, 1000)] * 3, (0, 300), (30, 60), 8, 2, 128, F32, 48)]
    batches = [Batch(*x, seed=20 + i) for i, x in enumerate(sizes)]
    want = [b.run() for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    keep, graphs = [], []
    for b, w, st in zip(batches, want, streams):
        with torch.cuda.stream(st):
            ws = S.make_shared_workspace(b.c.kv, b.T, max(b.n))
            out = tuple(torch.full_like(x, 7.0) for x in w)
            cu, share = i32(b.cu), i32(b.share)
            call = lambda b=b, cu=cu, share=share, out=out, ws=ws: S.shared_attn(  # noqa: E731
                b.c.kv, b.q, b.kn, b.vn, b.scale, cu, max(b.n), share, out[0], out[1], ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                call()
        keep.append((out, call))
        graphs.append(g)
    torch.cuda.synchronize()
    for how in ("eager", "graph"):
        for out, _ in keep:
            out[0].fill_(7.0), out[1].fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(20):
            for st, (_, call), g in zip(streams, keep, graphs):
                with torch.cuda.stream(st):
                    call() if how == "eager" else g.replay()
        torch.cuda.synchronize()
        assert S.last_error() == 0
        for (out, _), w in zip(keep, want):
            assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_behind_32_bits(dtype):
    """The pages at the end of a pool of more than 2^31 elements; rows copied there and from there."""
    import sparse_kv_selection_gb300 as S
    b = Batch([(20, 300), (1, 0), (3, 64)], (0, 400), (1, 9), 4, 2, 64, dtype, 16, seed=30)
    want, c = b.run(), b.c
    pages, each = c.k.shape[0], c.k[0].numel()
    behind = (1 << 31) // each + 5
    k, v = (torch.empty(behind + pages, *c.k.shape[1:], dtype=dtype, device="cuda") for _ in range(2))
    k[behind:], v[behind:] = c.k, c.v
    table = torch.where(c.kv.block_table >= 0, c.kv.block_table + behind, -1)
    b.c.kv = S.KVCache(k, v, c.kv.seq_lens, c.Hq, block_table=table)
    got = b.run()
    assert S.last_error() == 0 and torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    slots = torch.arange(pages * 16, dtype=torch.int32, device="cuda")
    S.copy_rows(b.c.kv, slots + behind * 16, slots)
    bits = lambda x: x.contiguous().view(torch.int16 if dtype == BF16 else torch.int32)  # noqa: E731  (rows behind the ends are NaN)
    assert torch.equal(bits(k[:pages]), bits(c.k)) and torch.equal(bits(v[:pages]), bits(c.v))
    back = torch.flip(slots, (0,)) + behind * 16
    S.copy_rows(b.c.kv, slots, back)
    assert S.last_error() == 0
    flat = lambda x: bits(x.transpose(1, 2).reshape(pages * 16, -1))  # noqa: E731
    assert torch.equal(flat(k[behind:]), flat(c.k).flip(0)) and torch.equal(flat(v[behind:]), flat(c.v).flip(0))


@pytest.mark.parametrize("dtype,Hq", [(BF16, 2), (F32, 2), (F32, 16)])
def test_overlapping_groups_refused(dtype, Hq):
    """Every row the first of a group that reaches to the batch's end: more tokens than there are."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_INDEX
    b = Batch([(64, 64)], (0, 20), (1, 1), Hq, 2, 64, dtype, 16, seed=9)
    whole = b.run()
    b.run(share=[[r, 64 - r, 64, 0] for r in range(64)])
    assert S.last_error() == DEV_BAD_INDEX
    again = b.run()
    assert S.last_error() == 0 and torch.equal(whole[0], again[0]) and torch.equal(whole[1], again[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_and_lengths_refused(dtype):
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_LEN
    b = Batch([(4, 64), (2, 32)], (16, 60), [2, 1, 3, 2, 1, 1], 4, 2, 64, dtype, 16, seed=11)
    # offsets that step back: every row stays
    cu = b.cu.copy()
    cu[3] = 1
    out = b.run(cu=cu)
    assert S.last_error() == DEV_BAD_LEN
    assert (out[0] == 7.0).all() and (out[1] == 7.0).all()
    # more tokens than max_new: that sequence's rows stay, the group's others are right
    out = b.run(max_new=2)
    assert S.last_error() == DEV_BAD_LEN
    assert (out[0][3:6] == 7.0).all() and (out[1][3:6] == 7.0).all()
    b.check(out, rows=[0, 1, 3, 4, 5])
    # a sequence beyond T
    cu = b.cu.copy()
    cu[6] = b.T + 5
    out = b.run(cu=cu)
    assert S.last_error() == DEV_BAD_LEN
    b.check(out, rows=[0, 1, 2, 3, 4])
    assert (out[0][9:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_empty_masks_and_caches(dtype):
    """Tokens that see no token: with shared keys they attend those, without any keys
    the result is 0 and -inf."""
    import sparse_kv_selection_gb300 as S
    b = Batch([(2, 32), (1, 0)], [0, 3, 0], [2, 1, 2], 4, 2, 64, dtype, 16, tree=True, seed=12)
    b.sets = [[set() for _ in range(x)] for x in b.n]
    b.mask = torch.zeros(b.T, WORDS, dtype=torch.int32, device="cuda")
    out = b.run()
    assert S.last_error() == 0
    b.check(out, rows=[0, 1])
    assert (out[0][3:5] == 0).all() and torch.isneginf(out[1][3:5]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_and_infinity(dtype):
    import sparse_kv_selection_gb300 as S
    b = Batch([(3, 160), (2, 32)], (5, 60), (1, 1), 4, 2, 64, dtype, 16, seed=13)
    clean = b.run()
    b.q[1, 2, 5] = float("nan")                # one row of one query
    out = b.run()
    assert torch.isnan(out[0][1, 2]).all() and torch.isnan(out[1][1, 2])
    keep = torch.ones_like(clean[1], dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(out[0][keep], clean[0][keep]) and torch.equal(out[1][keep], clean[1][keep])
    b.q[1, 2, 5] = 0.5
    clean = b.run()
    page = int(b.c.kv.block_table[3, 1])       # a shared key of the second family, KV head 1
    b.c.k[page, 1, 3, 0] = float("nan")
    out = b.run()
    assert torch.isnan(out[0][3:5, 2:]).all() and torch.isnan(out[1][3:5, 2:]).all()
    assert torch.equal(out[0][:3], clean[0][:3]) and torch.equal(out[0][3:5, :2], clean[0][3:5, :2])
    assert S.last_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pages_outside_the_pool(dtype):
    """A shared page outside the pool is flagged and not attended."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_BLOCK
    b = Batch([(3, 160)], (5, 60), (1, 1), 4, 2, 64, dtype, 16, seed=14)
    bad = b.c.kv.block_table.clone()
    b.c.kv.block_table[:, 4] = 1 << 20
    out = b.run()
    assert S.last_error() == DEV_BAD_BLOCK
    b.c.kv.block_table.copy_(bad)
    for r in range(3):                         # the definition without keys 64 .. 79
        kc, vc = b.c.rows(r, b.lens[r])
        kc, vc = (torch.cat([x[:, :64], x[:, 80:]], 1) for x in (kc, vc))
        at = slice(r, r + 1)
        want, lse, e_out, e_lse = attn_ref(b.q[at].double(), kc, vc, b.kn[at].double(), b.vn[at].double(),
                                           torch.ones(1, 1, dtype=torch.bool, device="cuda"), b.scale, 64, dtype)
        assert ((out[0][at].double() - want).abs() <= e_out).all()
        assert ((out[1][at].double() - lse).abs() <= e_lse).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_growing_maxima(dtype):
    """States whose maxima lie far apart: the shared keys' weights vanish, or the rest's."""
    for boost in (0, 1):
        b = Batch([(4, 320)], (30, 60), (1, 2), 4, 2, 64, dtype, 16, seed=15)
        tab = b.c.kv.block_table.cpu().numpy()
        for r in range(4):
            for j in range(20):
                if boost == 0 and r == 0:
                    b.c.k[int(tab[0, j])] *= 1 + j           # rises along the prefix
        if boost:
            b.kn.mul_(30)
        out = b.run()
        b.check(out)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_other_scales(scale):
    b = Batch([(4, 200), (1, 0)], (0, 60), (1, 3), 4, 2, 64, BF16, 16, seed=16)
    b.scale = scale
    b.check(b.run())


def test_binding_refusals():
    import sparse_kv_selection_gb300 as S
    b = Batch([(3, 64)], (5, 9), (1, 1), 4, 2, 64, BF16, 16, seed=17)
    ws = S.make_shared_workspace(b.c.kv, b.T, 1)
    with pytest.raises(ValueError):
        b.run(share=np.zeros((3, 3)))
    with pytest.raises(S.PrhsError):
        b.run(ws=ws[:-512])
    with pytest.raises(S.PrhsError):
        b.run(ws=ws[1:])
    with pytest.raises(S.PrhsError):
        S.shared_workspace_size(b.c.kv, 0, 1)
    with pytest.raises(S.PrhsError):
        S.shared_workspace_size(b.c.kv, 4, 0)
