"""Sparse decoding (SparseDecoder) of sequences that are forked, ended and compacted: a row that
becomes another, or whose positions change, has no anchors of what it was."""
import gc

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

B, HQ, HKV, D, PAGE, T = 4, 4, 2, 64, 16, 320


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Case:
    """Four sequences of 320 keys, decoded once; with tau = -1 a head reuses whatever anchor it has."""

    def __init__(self, dtype, layers=1, stream=None):
        import sparse_kv_selection_gb300 as S
        g = torch.Generator(device="cuda").manual_seed(3)
        wide, pool = T // PAGE + 4, 200
        table = np.full((B, wide), -1)
        table[:, :T // PAGE] = np.random.default_rng(1).permutation(pool)[:B * (T // PAGE)].reshape(B, -1)
        used = table[:, :T // PAGE].reshape(-1)
        free = np.concatenate([used, np.setdiff1d(np.arange(pool), used)])
        lens, table = i32([T] * B), i32(table)
        mk = lambda: torch.randn(pool, HKV, PAGE, D, generator=g, device="cuda").to(dtype)  # noqa: E731
        self.kv = [S.KVCache(mk(), mk(), lens, HQ, block_table=table) for _ in range(layers)]
        self.pool = S.PagePool(self.kv[0], free_pages=i32(free), free_head=i32([len(used)]),
                               n_pages=i32([T // PAGE] * B), layers=self.kv[1:], stream=stream)
        self.dec = [self.decoder(kv) for kv in self.kv]
        self.q = torch.randn(B, HQ, D, generator=g, device="cuda").to(dtype)
        for dec in self.dec:
            dec.step(self.q)
            assert not dec.reuse.any()
            dec.step(self.q)
            assert dec.reuse.all()
        assert S.last_error() == 0

    def decoder(self, kv):
        import sparse_kv_selection_gb300 as S
        return S.SparseDecoder(kv, N=24, w=2, tau=-1.0)

    def check(self, fresh):
        """The rows in `fresh` retrieve, the others reuse; those that retrieve do as a new decoder."""
        import sparse_kv_selection_gb300 as S
        for kv, dec in zip(self.kv, self.dec):
            before = dec.out.clone()
            dec.step(self.q)
            new = self.decoder(kv)
            new.step(self.q)
            assert S.last_error() == 0
            for b in range(B):
                assert dec.reuse[b].bool().logical_not().all() == (b in fresh) and dec.reuse[b].bool().any() == (b not in fresh)
                if b in fresh:
                    n = int(new.n_sel[b, 0])
                    assert torch.equal(dec.n_sel[b], new.n_sel[b]) and torch.equal(dec.idx[b, :, :n], new.idx[b, :, :n])
                    assert torch.equal(dec.out[b], new.out[b]) and torch.equal(dec.lse[b], new.lse[b])
                else:
                    assert torch.equal(dec.out[b], before[b])
            dec.step(self.q)                    # and again all of them reuse
            assert dec.reuse.all() and S.last_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layers", [1, 2])
def test_rows_that_fork_retrieve_again(dtype, layers):
    c = Case(dtype, layers)
    c.pool.fork(i32([1, 0, 2, 2]))
    c.check({0, 1, 3})


def test_a_row_that_ends_and_is_filled_again_retrieves():
    c = Case(torch.bfloat16)
    c.pool.free(torch.tensor([False, True, False, False], device="cuda"))
    c.pool.fork(i32([0, 0, 2, 3]))
    c.check({1})


def test_compacted_rows_retrieve_again():
    c = Case(torch.float32)
    keep = np.zeros((B, T), int)
    keep[1, :T // 2] = np.arange(0, T, 2)
    keep[3, :40] = np.arange(100, 140)
    c.pool.compact(i32(keep), i32([-1, T // 2, -1, 40]))
    c.check({1, 3})


def test_refused_calls_lose_anchors_only():
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_INDEX
    c = Case(torch.bfloat16)
    c.pool.fork(i32([0, 9, 3, 3]))              # refused as a whole
    assert S.last_error() == DEV_BAD_INDEX
    c.check({1, 2})


def test_forks_from_a_graph():
    """A captured fork takes the anchors at every replay, and keeps the decoders that it resets."""
    import sparse_kv_selection_gb300 as S
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c = Case(torch.bfloat16, stream=stream)
        parent = i32([0, 1, 2, 3])
        c.pool.fork(parent)
        other = c.decoder(c.kv[0])
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            c.pool.fork(parent)
        there = other.anchor_n.data_ptr()
        del other
        gc.collect()
        for p, fresh in (([0, 1, 2, 3], set()), ([0, 0, 2, 3], {1}), ([3, 1, 2, 0], {0, 3})):
            parent.copy_(i32(p))
            g.replay()
            c.check(fresh)
        taken = [torch.zeros(B, HQ, dtype=torch.int32, device="cuda") for _ in range(64)]
        assert there not in [x.data_ptr() for x in taken]
        stream.synchronize()
    assert S.last_error() == 0


def test_decoders_that_are_gone_are_not_kept():
    import weakref
    c = Case(torch.bfloat16)
    dec = weakref.ref(c.dec[0])
    c.pool.fork(i32([1, 0, 2, 2]))
    c.dec = []
    gc.collect()
    assert dec() is None
    c.pool.fork(i32([1, 0, 2, 2]))


def test_reset_of_some_rows():
    """For sequences that a program moves itself."""
    c = Case(torch.bfloat16)
    c.dec[0].reset(torch.tensor([True, False, False, True], device="cuda"))
    c.check({0, 3})
    for bad in (torch.tensor([True], device="cuda"), i32([1, 0, 0, 1]), torch.tensor([True, False, False, True])):
        with pytest.raises(ValueError):
            c.dec[0].reset(bad)
    c.dec[0].reset()
    c.check({0, 1, 2, 3})
