"""Sequences that share pages, used together: prompts, forks, decoding with shared
prefixes, beams that trade places, compaction, ends; also from a graph and on a
stream of their own."""
import numpy as np
import pytest

from pages_util import Pages
from tokens_util import attn_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Twin:
    """A cache of two layers with its pool, and every sequence's keys and values as
    lists of rows: what a program without pages would hold."""

    def __init__(self, B, Hq, Hkv, d, dtype, page=16, pool=400, wide=40, stream=None):
        import sparse_kv_selection_gb300 as S
        self.B, self.Hq, self.Hkv, self.d, self.dtype, self.page = B, Hq, Hkv, d, dtype, page
        nan = lambda: torch.full((pool, Hkv, page, d), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        table, lens = i32(np.full((B, wide), -1)), i32([0] * B)
        self.kv = [S.KVCache(nan(), nan(), lens, Hq, block_table=table) for _ in range(2)]
        assert self.kv[0].block_table.data_ptr() == self.kv[1].block_table.data_ptr()
        ids = np.random.default_rng(0).permutation(pool)
        self.pool = S.PagePool(self.kv[0], free_pages=i32(ids), n_pages=i32([0] * B), layers=self.kv[1:], stream=stream)
        rope = S.RopeTable(16, device="cuda")
        self.steps = [S.TokenBatch(kv, rope, max_tokens=64, max_new=40, share_prefixes=True, min_shared=16, stream=stream,
                                   **self.pool.pages) for kv in self.kv]
        self.rows = [[[torch.zeros(0, Hkv, d, dtype=dtype, device="cuda") for _ in range(2)] for _ in range(2)] for _ in range(B)]
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(1)

    def feed(self, n, check=True):
        """A step of n[b] tokens: planned once, the other layer takes the plan's word."""
        import sparse_kv_selection_gb300 as S
        T = 64
        cu = np.concatenate([[0], np.cumsum(n)])
        first, second = self.steps
        first.plan(i32(n))
        for x in ("cu_new", "positions", "slots", "shared"):
            getattr(second, x).copy_(getattr(first, x))
        second.v, second.tree_mask = None, None
        for layer, step in enumerate(self.steps):
            mk = lambda h: torch.randn(T, h, self.d, generator=self.g, device="cuda").to(self.dtype)  # noqa: E731
            q, k, v = mk(self.Hq), mk(self.Hkv), mk(self.Hkv)
            step.rotate(q, k, v)
            step.attend()
            assert S.last_error() == 0
            for b in range(self.B):
                if n[b] == 0:
                    continue
                at = slice(int(cu[b]), int(cu[b + 1]))
                kc, vc = self.rows[b][layer]
                if check:
                    see = torch.tril(torch.ones(n[b], n[b], dtype=torch.bool, device="cuda"))
                    want, lse, e_out, e_lse = attn_ref(step.q[at].double(), kc.double().transpose(0, 1), vc.double().transpose(0, 1),
                                                       step.k[at].double(), v[at].double(), see, self.d ** -0.5, self.d, self.dtype)
                    assert ((step.out[at].double() - want).abs() <= e_out).all(), (b, layer)
                    assert ((step.lse[at].double() - lse).abs() <= e_lse).all(), (b, layer)
                self.rows[b][layer] = [torch.cat([kc, step.k[at]]), torch.cat([vc, v[at]])]
        lens = self.kv[0].seq_lens.clone()
        second.commit(i32(n))                       # rows of the second layer, lengths too
        self.kv[0].seq_lens.copy_(lens)
        first.commit(i32(n))
        assert S.last_error() == 0

    def check(self):
        """Every sequence's cached rows, and the bookkeeping."""
        p = self.pool.pages
        s = Pages(self.kv[0].block_table.cpu().numpy(), self.kv[0].seq_lens.cpu().numpy(), p["n_pages"].cpu().numpy(),
                  self.pool.page_shares.cpu().numpy(), p["free_pages"].cpu().numpy(), p["free_head"][0], self.page)
        s.check()
        for b in range(self.B):
            t = len(self.rows[b][0][0])
            assert s.lens[b] == t
            at = np.arange(t)
            blk, row = torch.tensor(s.table[b, at // self.page], device="cuda"), torch.tensor(at % self.page, device="cuda")
            for layer in range(2):
                assert torch.equal(self.kv[layer].k[blk, :, row], self.rows[b][layer][0])
                assert torch.equal(self.kv[layer].v[blk, :, row], self.rows[b][layer][1])
        return s

    def fork(self, parent):
        import sparse_kv_selection_gb300 as S
        self.pool.fork(i32(parent))
        assert S.last_error() == 0
        empty = [[x[:0] for x in layer] for layer in self.rows[0]]
        self.rows = [list(self.rows[p]) if p >= 0 else list(empty) for p in parent]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 64, 16), (2, 2, 128, 48)])
def test_samples_beams_and_compaction(dtype, Hq, Hkv, d, page):
    import sparse_kv_selection_gb300 as S
    rng = np.random.default_rng(1)
    m = Twin(8, Hq, Hkv, d, dtype, page)
    for _ in range(4):                              # two prompts of 150 and 120 tokens
        m.feed([37, 0, 0, 0, 21, 0, 0, 0])
    m.feed([2, 0, 0, 0, 36, 0, 0, 0])
    m.check()
    m.fork([0, 0, 0, 0, 4, 4, 4, 4])                # four samples of each
    s = m.check()
    whole = 150 // page
    assert (s.shares[s.table[0, :whole]] == 3).all()
    for _ in range(20):                             # decoding runs over a page's end
        m.feed([1] * 8)
    assert m.steps[0].shared[:, 2].cpu().tolist() == [whole * page] * 4 + [120 // page * page] * 4
    m.check()
    for _ in range(6):                              # beams
        parent = [int(x) for x in np.concatenate([rng.integers(0, 4, 4), rng.integers(4, 8, 4)])]
        m.fork(parent)
        m.check()
        m.feed([int(x) for x in rng.integers(0, 5, 8)])
    m.check()
    m.pool.free(torch.tensor([False, True, False, False, False, False, True, False], device="cuda"))
    assert S.last_error() == 0
    for b in (1, 6):
        m.rows[b] = [[x[:0] for x in layer] for layer in m.rows[b]]
    m.check()
    m.feed([1, 0, 1, 1, 1, 1, 0, 1])
    keep, n = np.zeros((8, 200), int), [-1] * 8
    for b in (0, 3, 7):
        t = len(m.rows[b][0][0])
        pick = np.concatenate([np.arange(40), np.sort(rng.choice(np.arange(40, t - 20), 17, replace=False)), np.arange(t - 20, t)])
        keep[b, :len(pick)], n[b] = pick, len(pick)
        m.rows[b] = [[x[torch.tensor(pick, device="cuda")] for x in layer] for layer in m.rows[b]]
    m.pool.compact(i32(keep), i32(n))
    assert S.last_error() == 0
    m.check()
    m.feed([1, 3, 1, 1, 1, 1, 2, 1])
    s = m.check()
    m.fork([-1] * 8)                                # everything comes back
    s = m.check()
    assert s.head == 0 and not s.shares.any()


def test_steps_from_a_graph():
    """Fork, plan, find, attend and commit captured once and replayed; another graph
    shares the workspaces."""
    import sparse_kv_selection_gb300 as S
    B, Hq, Hkv, d, T = 6, 4, 2, 64, 16
    stream = torch.cuda.Stream()
    rng = np.random.default_rng(2)
    with torch.cuda.stream(stream):
        m = Twin(B, Hq, Hkv, d, BF16, stream=stream)
        kv, step = m.kv[0], m.steps[0]
        m.feed([40, 0, 0, 0, 0, 0], check=False)
        parent, n = i32([0] * B), i32([1] * B)
        q, k, v = (torch.randn(64, h, d, device="cuda").to(BF16) for h in (Hq, Hkv, Hkv))

        def one():
            m.pool.fork(parent)
            step.plan(n)
            step.rotate(q, k, v)
            step.attend()
            step.commit(n)

        one()                                       # (function attributes are set outside captures)
        stream.synchronize()
        state = [x.clone() for x in (kv.block_table, kv.seq_lens, m.pool.page_shares, kv.k, kv.v, *m.pool.pages.values())]
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                one()
            graphs.append(g)
        parents = [rng.integers(0, B, B) for _ in range(12)]
        results = []
        for how in ("eager", "graph"):
            for x, y in zip((kv.block_table, kv.seq_lens, m.pool.page_shares, kv.k, kv.v, *m.pool.pages.values()), state):
                x.copy_(y)
            out = []
            for i, p in enumerate(parents):
                parent.copy_(i32(p))
                q.copy_(torch.randn(64, Hq, d, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").to(BF16))
                if how == "eager":
                    one()
                else:
                    graphs[i % 2].replay()
                out.append([x.clone() for x in (step.out[:B], step.lse[:B], kv.block_table, kv.seq_lens, m.pool.page_shares,
                                                m.pool.pages["free_head"], m.pool.pages["free_pages"])])
            results.append(out)
        stream.synchronize()
    assert S.last_error() == 0
    for a, b in zip(*results):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_pool_refusals():
    import sparse_kv_selection_gb300 as S
    k = torch.zeros(4, 1, 16, 64, device="cuda")
    flat = S.KVCache(k, k, i32([0] * 4), 1)
    paged = S.KVCache(k, k, i32([0, 0]), 1, block_table=i32([[0, 1], [2, 3]]))
    other = S.KVCache(k, k, i32([0, 0]), 1, block_table=i32([[0, 1], [2, 3]]))
    kw = dict(free_pages=i32([0]), n_pages=i32([0, 0]))
    with pytest.raises(ValueError):
        S.PagePool(flat, **kw)
    with pytest.raises(ValueError):
        S.PagePool(paged, layers=[other], **kw)
    with pytest.raises(ValueError):
        S.PagePool(paged, layers=[flat], **kw)
    pool = S.PagePool(paged, **kw)
    with pytest.raises(ValueError):
        pool.fork(i32([0]))
    with pytest.raises(ValueError):
        pool.fork(torch.tensor([0, 1], device="cuda"))
    with pytest.raises(ValueError):
        pool.compact(i32([[0]]), i32([1, 1]))
    with pytest.raises(ValueError):
        S.fork_seqs(flat, i32([0] * 4), i32([0]), i32([0]), pool.ws, page_shares=i32([0] * 4), free_head=i32([0]), **kw)


def test_prefixes_on_a_contiguous_cache_are_the_callers():
    """share_prefixes on a contiguous cache finds nothing and changes nothing."""
    import sparse_kv_selection_gb300 as S
    kv = S.KVCache(torch.randn(3, 2, 90, 64, device="cuda").to(BF16), torch.randn(3, 2, 90, 64, device="cuda").to(BF16),
                   i32([40, 60, 0]), 4)
    rope = S.RopeTable(16)
    q, k, v = (torch.randn(8, h, 64, device="cuda").to(BF16) for h in (4, 2, 2))
    outs = []
    for share in (False, True):
        step = S.TokenBatch(kv, rope, max_tokens=8, max_new=4, share_prefixes=share)
        step.plan(i32([1, 3, 2]))
        step.rotate(q, k, v)
        step.attend()
        outs.append((step.out.clone(), step.lse.clone()))
    assert S.last_error() == 0
    assert (outs[0][0][:6].float() - outs[1][0][:6].float()).abs().max() <= 2 ** -6      # (checked against 64 bits elsewhere)
    assert (outs[0][1][:6] - outs[1][1][:6]).abs().max() <= 1e-5
