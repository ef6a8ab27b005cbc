"""Forking, compacting and freeing sequences of a paged cache, copying their rows
and finding shared prefixes, against step-by-step forms on the host."""
import numpy as np
import pytest

from pages_util import Pages, compact_ref, find_ref, fork_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("table", "lens", "n_pages", "shares", "free", "head")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def make_state(rng, families, fan, prefix, rest, page, extra=2, spare=None):
    """Families of rows that share whole pages of a common prefix."""
    lens, shared = [], []
    for _ in range(families):
        f, p = rng.integers(fan[0], fan[1] + 1), rng.integers(prefix[0], prefix[1] + 1)
        for i in range(f):
            lens.append(int(p + rng.integers(rest[0], rest[1] + 1)))
            shared.append(int(p // page) if i else -1)
    B = len(lens)
    held = [-(-t // page) + int(rng.integers(0, extra + 1)) for t in lens]
    wide = max(1, max(held)) + 3
    total = sum(h - max(0, s) for h, s in zip(held, shared))
    pool = total + (sum(held) + B if spare is None else spare)
    ids = rng.permutation(pool)
    table, shares, at, first = np.full((B, wide), -1), np.zeros(pool, int), 0, 0
    for b in range(B):
        same = max(0, shared[b])
        first = b if shared[b] < 0 else first
        table[b, :same] = table[first, :same]
        shares[table[b, :same]] += 1
        table[b, same:held[b]] = ids[at:at + held[b] - same]
        at += held[b] - same
    s = Pages(table, lens, held, shares, ids, at, page)
    s.check()
    return s


class Device:
    """A state on the GPU, with a cache of one head."""

    def __init__(self, s, kv_rows=False):
        import sparse_kv_selection_gb300 as S
        shape = (len(s.shares), 1, s.page, 64)
        self.k = torch.randn(shape, device="cuda").to(BF16) if kv_rows else torch.zeros(shape, dtype=BF16, device="cuda")
        self.v = torch.randn(shape, device="cuda").to(BF16) if kv_rows else self.k
        self.kv = S.KVCache(self.k, self.v, i32(s.lens), 1, block_table=i32(s.table))
        self.pages = dict(n_pages=i32(s.n_pages), page_shares=i32(s.shares), free_pages=i32(s.free), free_head=i32([s.head]))
        self.ws = S.make_pages_workspace(self.kv)

    def outs(self):
        p = self.pages
        return dict(table_out=torch.full_like(self.kv.block_table, -9), lens_out=torch.full_like(self.kv.seq_lens, -9),
                    **{k + "_out": torch.full_like(v, -9) for k, v in p.items()})

    def state(self, out=None):
        if out is None:
            x = (self.kv.block_table, self.kv.seq_lens, *self.pages.values())
        else:
            x = (out["table_out"], out["lens_out"], *[out[k + "_out"] for k in self.pages])
        return [t.cpu().numpy() for t in x]


def call(d, what, args, cap, in_place):
    import sparse_kv_selection_gb300 as S
    src, dst = (torch.full((d.kv.B, cap), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    out = {} if in_place else d.outs()
    getattr(S, what)(d.kv, *[i32(a) for a in args], src, dst, d.ws, **d.pages, **out)
    bits = S.last_error()
    return d.state(None if in_place else out), src.cpu().numpy(), dst.cpu().numpy(), bits


def same_state(got, want):
    for name, g in zip(NAMES, got):
        w = [want.head] if name == "head" else getattr(want, name)
        assert np.array_equal(g, w), name


def check(s, what, args, want_bits=0):
    """In place and into other arrays, twice each (one possible result)."""
    cap = s.page if what == "fork_seqs" else np.asarray(args[0]).shape[1]
    ref = fork_ref(s, *args) if what == "fork_seqs" else compact_ref(s, *[np.asarray(a) for a in args])
    assert (ref is None) == (want_bits != 0)
    after, src, dst = ref if ref is not None else (s, -1, -1)
    for in_place in (False, True, True):
        d = Device(s)
        got, gs, gd, bits = call(d, what, args, cap, in_place)
        assert bits == want_bits
        same_state(got, after)
        assert (gs == src).all() and (gd == dst).all()
        if not in_place:
            same_state(d.state(), s)           # what was there stays
    if ref is not None:
        after.check()
    return after


def random_parents(rng, B, stay, end, within=None):
    out = []
    for b in range(B):
        x = rng.random()
        lo, hi = (0, B) if within is None else (b // within * within, min(B, b // within * within + within))
        out.append(b if x < stay else -1 if x < stay + end else int(rng.integers(lo, hi)))
    return out


SHAPES = [(1, (1, 1), (0, 0), (0, 0)), (1, (2, 2), (0, 0), (1, 1)), (1, (5, 5), (33, 33), (0, 40)), (3, (1, 9), (0, 200), (0, 70)),
          (8, (8, 8), (300, 900), (1, 90)), (40, (1, 40), (0, 60), (0, 9)), (2, (3, 3), (20000, 40000), (0, 5000))]


@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("stay,end", [(0.3, 0.1), (0.0, 0.0), (0.5, 0.5), (0.0, 1.0), (1.0, 0.0)])
def test_fork(page, shape, stay, end):
    rng = np.random.default_rng(page + shape[0])
    s = make_state(rng, *shape, page)
    check(s, "fork_seqs", [random_parents(rng, len(s.lens), stay, end)])


def test_fork_many_steps():
    """A beam search: twenty steps of the operator on its own results."""
    rng = np.random.default_rng(3)
    s = make_state(rng, 4, (6, 6), (100, 300), (1, 30), 16)
    d = Device(s)
    for i in range(20):
        parent = random_parents(rng, 24, 0.3, 0.05 if i > 10 else 0.0, within=6)
        want, src, dst = fork_ref(s, parent)
        got, gs, gd, bits = call(d, "fork_seqs", [parent], 16, True)
        assert bits == 0
        same_state(got, want)
        assert np.array_equal(gs, src) and np.array_equal(gd, dst)
        want.check()
        s = want


def test_fork_swap_and_cycle():
    """Rows that trade places: every last page is taken over, nothing is copied."""
    rng = np.random.default_rng(4)
    s = make_state(rng, 6, (1, 1), (0, 0), (5, 90), 16, extra=0)
    after = check(s, "fork_seqs", [[1, 0, 3, 4, 2, 5]])
    assert after.head == s.head and np.array_equal(after.lens, s.lens[[1, 0, 3, 4, 2, 5]])
    # a row that leaves without a child gives everything back
    after = check(s, "fork_seqs", [[1, 1, 1, 3, 4, -1]])
    assert after.lens[5] == 0 and after.n_pages[5] == 0


def test_fork_of_a_shared_last_page_copies_it():
    rng = np.random.default_rng(5)
    s = make_state(rng, 1, (3, 3), (40, 40), (0, 0), 16, extra=0)
    s.shares[s.table[1, 2]] = 1                       # another row of some other batch holds it too
    s2, src, dst = fork_ref(s, [0, 2, 1])
    assert (src[2] >= 0).any() and not (src[1] >= 0).any()
    check_free = Device(s)
    got, gs, gd, bits = call(check_free, "fork_seqs", [[0, 2, 1]], 16, True)
    assert bits == 0 and np.array_equal(gs, src) and np.array_equal(gd, dst)
    same_state(got, s2)


def test_fork_refusals():
    from sparse_kv_selection_gb300.binding import DEV_BAD_BLOCK, DEV_BAD_INDEX, DEV_BAD_LEN, DEV_CAPACITY
    rng = np.random.default_rng(6)

    def state(**kw):
        return make_state(rng, 4, (2, 2), (40, 60), (3, 9), 16, **kw)

    def refused(s, parent, bits):
        for in_place in (False, True):
            d = Device(s)
            got, gs, gd, b = call(d, "fork_seqs", [parent], 16, in_place)
            assert b == bits
            same_state(got, s)
            assert (gs == -1).all() and (gd == -1).all()

    ident = list(range(8))
    check(state(), "fork_seqs", [[8] + ident[1:]], DEV_BAD_INDEX)
    check(state(), "fork_seqs", [[-2] + ident[1:]], DEV_BAD_INDEX)
    check(state(spare=1), "fork_seqs", [[1, 1, 3, 3] + ident[4:]], DEV_CAPACITY)     # two copies, one page
    check(state(spare=2), "fork_seqs", [[1, 1, 3, 3] + ident[4:]])
    s = state()
    s.lens[1] = 1 << 20
    refused(s, [1] + ident[1:], DEV_BAD_LEN)
    s = state()
    s.n_pages[1] = 0
    refused(s, [1] + ident[1:], DEV_BAD_LEN)
    s = state()
    s.n_pages[0] = s.table.shape[1] + 1
    refused(s, [-1] + ident[1:], DEV_BAD_LEN)
    s = state()
    s.head = len(s.free) + 1
    refused(s, [-1] + ident[1:], DEV_BAD_LEN)
    s = state()
    s.table[1, 0] = len(s.shares)                    # named by the new row and given up by the old one
    refused(s, [1] + ident[1:], DEV_BAD_BLOCK)
    refused(s, [0, -1] + ident[2:], DEV_BAD_BLOCK)
    s = state()
    s.table[1, s.lens[1] // 16] = -7                 # the page to copy
    refused(s, [1] + ident[1:], DEV_BAD_BLOCK)
    s = state()
    s.free[s.head] = len(s.shares) + 5               # the page to copy it to
    refused(s, [1] + ident[1:], DEV_BAD_BLOCK)
    # more pages come back than were ever taken from the list
    s = state()
    s.free = s.free[s.head:].copy()
    s.head = 0
    refused(s, [-1] * 8, DEV_CAPACITY)
    refused(s, [1, 1, 0, 0] + [-1] * 4, DEV_CAPACITY)


@pytest.mark.parametrize("what", ["fork_seqs", "compact_seqs"])
def test_large_tables_from_a_graph(what):
    """A table that all SMs take: captured once, replayed with other arguments on what it left."""
    import sparse_kv_selection_gb300 as S
    rng = np.random.default_rng(12)
    s = make_state(rng, 8, (8, 8), (17000, 18000), (1, 90), 16)
    assert len(s.lens) * s.table.shape[1] > 1 << 16
    d, cap = Device(s), 16 if what == "fork_seqs" else 12000
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        src, dst = (torch.full((64, cap), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        args = [i32(list(range(64)))] if what == "fork_seqs" else [torch.zeros(64, cap, dtype=torch.int32, device="cuda"), i32([-1] * 64)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            getattr(S, what)(d.kv, *args, src, dst, d.ws, **d.pages)
        for i in range(3):
            if what == "fork_seqs":
                new = [np.array(random_parents(rng, 64, 0.3, 0.1, within=8))]
            else:
                m = np.minimum(s.lens, rng.integers(0, cap, 64))
                keep = np.zeros((64, cap), int)
                for b in range(64):
                    keep[b, :m[b]] = np.sort(rng.choice(s.lens[b], m[b], replace=False)) if s.lens[b] else []
                new = [keep, m]
            for x, y in zip(args, new):
                x.copy_(i32(y))
            g.replay()
            stream.synchronize()
            assert S.last_error() == 0
            s, want_src, want_dst = fork_ref(s, *new) if what == "fork_seqs" else compact_ref(s, *new)
            same_state(d.state(), s)
            assert np.array_equal(src.cpu().numpy(), want_src) and np.array_equal(dst.cpu().numpy(), want_dst)


def random_keep(rng, s, share, leave=0.1):
    """Kept positions: leading ones, some of the middle, the last ones."""
    m, rows = [], []
    for t in s.lens:
        if rng.random() < leave:
            m.append(-1)
            rows.append(np.zeros(0, int))
            continue
        n = int(t * share)
        lead = min(n, int(rng.integers(0, 100)))
        tail = min(n - lead, int(rng.integers(0, 50))) if n < t else 0
        mid = np.sort(rng.choice(np.arange(lead, t - tail), n - lead - tail, replace=False))
        rows.append(np.concatenate([np.arange(lead), mid, np.arange(t - tail, t)]))
        m.append(n)
    cap = max(1, max(len(r) for r in rows)) + 2
    keep = np.full((len(m), cap), -5)
    for b, r in enumerate(rows):
        keep[b, :len(r)] = r
    return keep, np.array(m)


@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("share", [0.0, 0.05, 0.5, 1.0])
def test_compact(page, shape, share):
    rng = np.random.default_rng(page + shape[0])
    s = make_state(rng, *shape, page)
    check(s, "compact_seqs", random_keep(rng, s, share))


@pytest.mark.parametrize("m", [0, 1, 15, 16, 17, 39, 40, 47, 48, 50])
def test_compact_cuts_short(m):
    """The first m positions: a last page that others hold too is copied."""
    rng = np.random.default_rng(7)
    s = make_state(rng, 1, (3, 3), (48, 48), (2, 2), 16)
    keep = np.tile(np.arange(50), (3, 1))
    after = check(s, "compact_seqs", (keep, np.array([m, -1, m])))
    assert after.lens.tolist() == [m, 50, m]
    check(s, "compact_seqs", (keep, np.array([m, m, m])))


def test_compact_refusals():
    from sparse_kv_selection_gb300.binding import DEV_BAD_BLOCK, DEV_BAD_INDEX, DEV_BAD_LEN, DEV_CAPACITY
    rng = np.random.default_rng(8)
    s = make_state(rng, 3, (1, 1), (0, 0), (60, 70), 16, spare=1)
    n = np.array([-1, 3, -1])

    def keep(*row):
        return np.array([[0] * 5, list(row) + [0] * (5 - len(row)), [0] * 5])

    check(s, "compact_seqs", (keep(2, 5, 9), n))
    for bad in ((2, 2, 9), (5, 2, 9), (-1, 2, 9), (2, 9, int(s.lens[1])), (0, 1, -3)):
        check(s, "compact_seqs", (keep(*bad), n), DEV_BAD_INDEX)
    d = Device(s)
    got, gs, gd, bits = call(d, "compact_seqs", (keep(1, 2, 3, 4, 5), np.array([-1, 6, -1])), 5, True)
    assert bits == DEV_BAD_LEN and (gs == -1).all()
    same_state(got, s)
    long = np.tile(np.arange(200), (3, 1))
    d = Device(s)
    got, gs, gd, bits = call(d, "compact_seqs", (long, np.array([-1, int(s.lens[1]) + 1, -1])), 200, True)
    assert bits == DEV_BAD_LEN
    same_state(got, s)
    # one free page for two rows
    check(s, "compact_seqs", (np.tile([1, 4], (3, 1)), np.array([2, 2, -1])), DEV_CAPACITY)
    s.table[1, 2] = -1                               # a kept position on no page
    d = Device(s)
    got, gs, gd, bits = call(d, "compact_seqs", (keep(2, 40), np.array([-1, 2, -1])), 5, False)
    assert bits == DEV_BAD_BLOCK
    same_state(got, s)


def test_largest_batch():
    """16384 rows, several of a thread's in each pass."""
    rng = np.random.default_rng(9)
    s = make_state(rng, 2048, (8, 8), (16, 40), (0, 20), 16, extra=1)
    check(s, "fork_seqs", [random_parents(rng, 16384, 0.4, 0.1, within=8)])
    check(s, "compact_seqs", random_keep(rng, s, 0.6))


@pytest.mark.parametrize("B", [3800, 4090, 4096, 6130, 6144, 6200])
def test_batches_around_48_kb_of_shared_memory(B):
    """Arrays of a number or three a row that just fit, or just do not, what a launch has unasked."""
    import sparse_kv_selection_gb300 as S
    rng = np.random.default_rng(B)
    s = make_state(rng, B // 2, (2, 2), (16, 40), (0, 9), 16, extra=0)
    d = Device(s)
    parent = random_parents(rng, B, 0.5, 0.1, within=2)
    want, src, dst = fork_ref(s, parent)
    got, gs, gd, bits = call(d, "fork_seqs", [parent], 16, True)
    assert bits == 0
    same_state(got, want)
    assert np.array_equal(gs, src) and np.array_equal(gd, dst)
    shared = torch.full((B, 4), -9, dtype=torch.int32, device="cuda")
    n = np.ones(B, int)
    S.find_shared(d.kv, i32(np.arange(B + 1)), shared, min_keys=1)
    assert S.last_error() == 0
    assert np.array_equal(shared.cpu().numpy(), find_ref(want.table, want.lens, n, 16, 1, 1))


# --------------------------------------------------------------------------- #
# row copies
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hkv,d,page", [(1, 64, 16), (1, 64, 0), (3, 128, 48), (8, 64, 128), (32, 128, 16)])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_copy_rows(dtype, Hkv, d, page, n):
    import sparse_kv_selection_gb300 as S
    rng = np.random.default_rng(n + d)
    slots = 40 * (page or 51)
    k, v = (torch.randn(40, Hkv, page or 51, d, device="cuda").to(dtype) for _ in range(2))
    table = i32(np.zeros((2, 4))) if page else None
    kv = S.KVCache(k.clone(), v.clone(), i32([0, 0] if page else [0] * 40), Hkv, block_table=table)
    pick = rng.permutation(slots)
    src, dst = pick[:n].copy(), pick[n:2 * n].copy()
    if n > 3:
        src[1], dst[2], src[3] = -1, -1, src[0]        # no copies; a row copied twice
    S.copy_rows(kv, i32(src), i32(dst))
    assert S.last_error() == 0
    per = page or 51
    for x, y in ((k, kv.k), (v, kv.v)):
        want = x.clone()
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                want[b // per, :, b % per] = x[a // per, :, a % per]
        assert torch.equal(want, y)


def test_copy_rows_between_caches_and_refusals():
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_INDEX
    a = S.KVCache(torch.randn(2, 4, 30, 64, device="cuda"), torch.randn(2, 4, 30, 64, device="cuda"), i32([30, 30]), 4)
    pool = [torch.zeros(5, 4, 16, 64, device="cuda") for _ in range(2)]
    b = S.KVCache(*pool, i32([30]), 8, block_table=i32([[3, 1]]))
    src = i32(np.arange(30) + 30)                      # the contiguous cache's second sequence
    dst = i32([(3, 1)[p // 16] * 16 + p % 16 for p in range(30)])
    S.copy_rows(b, src, dst, source=a)
    assert S.last_error() == 0
    got = b.k[[3, 1]].transpose(0, 1).reshape(4, 32, 64)
    assert torch.equal(got[:, :30], a.k[1]) and not got[:, 30:].any() and not b.k[[0, 2, 4]].any()
    assert torch.equal(b.v[[3, 1]].transpose(0, 1).reshape(4, 32, 64)[:, :30], a.v[1])
    before = b.k.clone()
    for s, t in ((60, 0), (-2, 0), (0, 80), (0, -5)):
        S.copy_rows(b, i32([s]), i32([t]), source=a)
        assert S.last_error() == DEV_BAD_INDEX
        assert torch.equal(b.k, before)
    S.copy_rows(b, i32([]), i32([]))
    with pytest.raises(ValueError):
        S.copy_rows(b, i32([1, 2]), i32([3]))
    with pytest.raises(S.PrhsError):
        S.copy_rows(b, i32([1]), i32([3]), source=S.KVCache(torch.zeros(1, 2, 4, 64, device="cuda"),
                                                            torch.zeros(1, 2, 4, 64, device="cuda"), i32([1]), 2))


def test_fork_and_compact_move_rows():
    """Metadata and rows together: every sequence reads what its parent read."""
    import sparse_kv_selection_gb300 as S
    rng = np.random.default_rng(10)
    s = make_state(rng, 3, (4, 4), (70, 200), (1, 40), 16)
    d = Device(s, kv_rows=True)

    def logical(st):
        out = []
        for b, t in enumerate(st.lens):
            p = np.arange(t)
            out.append(d.kv.k[torch.tensor(st.table[b, p // 16], device="cuda"), 0, torch.tensor(p % 16, device="cuda")].clone())
        return out

    for step in range(6):
        rows = logical(s)
        if step % 2 == 0:
            parent = random_parents(rng, 12, 0.3, 0.05)
            s, src, dst = fork_ref(s, parent)
            got, gs, gd, bits = call(d, "fork_seqs", [parent], 16, True)
            want = [rows[p] if p >= 0 else rows[0][:0] for p in parent]
        else:
            keep, m = random_keep(rng, s, 0.8)
            s, src, dst = compact_ref(s, keep, m)
            got, gs, gd, bits = call(d, "compact_seqs", (keep, m), keep.shape[1], True)
            want = [r if n < 0 else r[torch.tensor(k[:n], device="cuda")] for r, k, n in zip(rows, keep, m)]
        assert bits == 0
        same_state(got, s)
        S.copy_rows(d.kv, i32(gs), i32(gd))
        assert S.last_error() == 0
        for w, g in zip(want, logical(s)):
            assert torch.equal(w, g)


# --------------------------------------------------------------------------- #
# shared prefixes
# --------------------------------------------------------------------------- #
def run_find(table, lens, n, page, group, min_keys):
    import sparse_kv_selection_gb300 as S
    pool = int(np.max(table)) + 1
    k = torch.zeros(max(1, pool), 1, page, 64, dtype=BF16, device="cuda")
    kv = S.KVCache(k, k, i32(lens), group, block_table=i32(table))
    out = torch.full((len(lens), 4), -9, dtype=torch.int32, device="cuda")
    S.find_shared(kv, i32(np.concatenate([[0], np.cumsum(n)])), out, min_keys=min_keys)
    assert S.last_error() == 0
    return out.cpu().numpy()


@pytest.mark.parametrize("page,min_keys", [(16, 1), (16, 256), (48, 100), (64, 0)])
@pytest.mark.parametrize("B,wide", [(1, 1), (2, 40), (17, 300), (200, 700), (1500, 30)])
def test_find_shared(page, min_keys, B, wide):
    """Tables whose neighbours share random numbers of pages, nested in chains."""
    rng = np.random.default_rng(B + page)
    table = np.zeros((B, wide), int)
    fresh = 0
    for b in range(B):
        table[b] = np.arange(fresh, fresh + wide)
        fresh += wide
        if b and rng.random() < 0.85:
            same = int(rng.choice([wide, wide // 2, wide // 3, rng.integers(0, wide + 1)]))
            table[b, :same] = table[b - 1, :same]
    table %= 60000                                    # (numbers far apart stay distinct in a chain)
    lens = rng.integers(0, wide * page + 1, B)
    lens[rng.random(B) < 0.5] = wide * page
    n = rng.integers(0, 3, B)
    n[rng.random(B) < 0.05] = 300
    for group in (1, 4):
        got = run_find(table, lens, n, page, group, min_keys)
        assert np.array_equal(got, find_ref(table, lens, n, page, group, min_keys))


def test_find_shared_chain_of_the_largest_batch():
    B = 16384
    rng = np.random.default_rng(1)
    table = np.tile(np.arange(6), (B, 1))
    table[:, 5] = np.arange(B) + 6
    lens, n = rng.integers(80, 97, B), rng.integers(0, 2, B)
    got = run_find(table, lens, n, 16, 1, 16)
    assert np.array_equal(got, find_ref(table, lens, n, 16, 1, 16))


def test_find_shared_contiguous_cache_has_none():
    import sparse_kv_selection_gb300 as S
    k = torch.zeros(3, 1, 8, 64, dtype=BF16, device="cuda")
    kv = S.KVCache(k, k, i32([8, 8, 8]), 1)
    out = torch.full((3, 4), -9, dtype=torch.int32, device="cuda")
    S.find_shared(kv, i32([0, 1, 2, 3]), out, min_keys=0)
    assert S.last_error() == 0
    assert out.cpu().tolist() == [[0, 1, 0, 0], [1, 1, 0, 0], [2, 1, 0, 0]]
