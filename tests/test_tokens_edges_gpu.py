"""Token batches at the edges of their contract: sequences that planning refused,
page state that batches share, NaN, angles near quarter turns, long runs of key
tiles."""
import os
import subprocess
import sys

import numpy as np
import pytest

from tokens_util import Cache, attn_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def rows_of(T, c, seed):
    """q, k, v rows of T tokens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kw = dict(device="cuda", dtype=c.dtype, generator=g)
    return torch.randn(T, c.Hq, c.d, **kw), torch.randn(T, c.Hkv, c.d, **kw), torch.randn(T, c.Hkv, c.d, **kw)


def same(x, y):
    return torch.equal(x.nan_to_num(99.0), y.nan_to_num(99.0))


# --------------------------------------------------------------------------- #
# committing
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_lengths_only_commit_looks_at_the_pages(entry):
    """A sequence whose new positions are not mapped keeps its length, rows or none."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_BLOCK
    c = Cache([10, 700, 16], 2, 1, 64, BF16, page=16, room=64, seed=2)
    c.kv.block_table[1, 44:48] = i32(c.free[:4])
    c.kv.block_table[2, 1] = entry
    new = i32([-9, -9, -9])
    # sequence 0 stays inside its page, 1 on mapped ones, 2 goes one position too far
    S.commit_tokens(c.kv, i32([0, 6, 70, 75]), i32([6, 64, 1]), new)
    assert S.last_error() == DEV_BAD_BLOCK
    assert new.tolist() == [16, 764, 16] and c.kv.seq_lens.tolist() == [10, 700, 16]


@pytest.mark.parametrize("stale", [False, True])
def test_a_chunk_that_found_no_pages_is_not_committed(stale):
    """Pages run out at sequence 1: it keeps its length although its positions were
    offered, whatever its table row holds beyond its own pages; once there are pages
    again its chunk goes through."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_CAPACITY
    c = Cache([20, 30, 5], 4, 2, 64, BF16, page=16, room=80, seed=3)
    if stale:                                      # an earlier occupant's pages, now sequence 0's
        c.kv.block_table[1, 2:5] = int(c.table[0, 0])
    free = i32(c.free[:3])
    batch = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=120, max_new=60, free_pages=free, n_pages=i32(c.n_pages))
    n = [40, 40, 8]
    q, k, v = rows_of(120, c, 1)
    batch.plan(i32(n))
    assert S.last_error() == DEV_CAPACITY
    wk, wv = c.k.clone(), c.v.clone()
    batch.rotate(q, k, v, append=True)
    batch.attend()
    batch.commit(i32(n))
    assert S.last_error() == DEV_CAPACITY
    assert c.kv.seq_lens.tolist() == [60, 30, 13]
    for have, want in ((c.k, wk), (c.v, wv)):      # sequence 1's rows are as they were
        for p in c.table[1, :2]:
            assert same(have[int(p)], want[int(p)])
    # three more pages
    again = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=120, max_new=60, free_pages=i32(c.free[3:8]),
                         n_pages=batch.pages["n_pages"])
    again.plan(i32([0, 40, 0]))
    again.rotate(q, k, v, append=True)
    again.commit(i32([0, 40, 0]))
    assert S.last_error() == 0 and c.kv.seq_lens.tolist() == [60, 70, 13]
    assert torch.equal(c.rows(1, 70)[1][:, 30:].transpose(0, 1), v[:40].double())


def test_accepted_tokens_without_a_slot_stay_out_of_other_pages():
    """Accepted tokens of a refused tree do not land in the pages that its table row
    still names."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_CAPACITY
    c = Cache([16, 40], 2, 1, 64, BF16, page=16, room=32, seed=4)
    c.kv.block_table[0, 1:3] = i32(c.table[1, :2])  # sequence 1's pages
    batch = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=12, max_new=8, free_pages=i32([]), n_pages=i32(c.n_pages))
    batch.plan(i32([6, 5]), i32([-1, 0, 1, 1, 0, 4, -1, 0, 1, 2, 3, -1]))
    assert S.last_error() == DEV_CAPACITY
    assert batch.slots[:6].tolist() == [-1] * 6 and (batch.slots[6:11] >= 0).all()
    q, k, v = rows_of(12, c, 2)
    batch.rotate(q, k, v)
    batch.attend()
    wk, wv = c.k.clone(), c.v.clone()
    batch.commit(i32([3, 2]), i32([[0, 1, 3], [0, 1, 0]]))
    assert S.last_error() == DEV_CAPACITY
    assert c.kv.seq_lens.tolist() == [16, 42]
    at = int(c.table[1, 2])
    wk[at, 0, 8:10], wv[at, 0, 8:10] = batch.k[6:8, 0], v[6:8, 0]
    assert same(c.k, wk) and same(c.v, wv)


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("append", [False, True])
def test_part_of_a_refused_chunk_is_not_committed(page, append):
    """A chunk beyond t_max, and one cut by the batch's token count, have no slots;
    accepting only as many tokens as would fit changes nothing."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_CAPACITY
    c = Cache([60, 10, 20], 2, 1, 64, BF16, page=page, room=4, t_max=64, seed=5)
    kw = {}
    if page:                                       # every position is mapped, four pages a sequence
        assert c.t_max == 64
        c.kv.block_table[1, 1:], c.kv.block_table[2, 2:] = i32([12, 13, 14]), i32([15, 16])
        c.k, c.v = [torch.randn(17, 1, 16, 64, device="cuda", dtype=BF16) for _ in range(2)]
        c.kv = S.KVCache(c.k, c.v, c.kv.seq_lens, 2, block_table=c.kv.block_table)
        kw = dict(free_pages=i32([]), n_pages=i32([4, 4, 4]))
    batch = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=14, max_new=8, **kw)
    q, k, v = rows_of(14, c, 2)
    batch.plan(i32([6, 5, 7]))                     # 66 positions; placed; cut
    assert S.last_error() == DEV_CAPACITY
    batch.rotate(q, k, v, append=append)
    wk = c.k.clone()
    batch.commit(i32([2, 5, 3]))
    assert S.last_error() == DEV_CAPACITY
    assert c.kv.seq_lens.tolist() == [60, 15, 20]
    if append:
        assert same(c.k, wk)
    else:
        assert (c.k.nan_to_num(99.0) != wk.nan_to_num(99.0)).any(-1).sum() == 5


def test_a_plan_is_committed_once():
    """The second commit of one plan finds slots that are not the next positions'."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_INDEX
    c = Cache([20, 7], 2, 1, 64, BF16, page=16, room=40, seed=6)
    batch = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=13, max_new=8, free_pages=i32(c.free), n_pages=i32(c.n_pages))
    batch.plan(i32([8, 4]))
    batch.rotate(*rows_of(13, c, 2), append=True)
    batch.commit(i32([4, 0]))
    assert S.last_error() == 0 and c.kv.seq_lens.tolist() == [24, 7]
    batch.commit(i32([4, 4]))
    assert S.last_error() == DEV_BAD_INDEX and c.kv.seq_lens.tolist() == [24, 11]


def test_a_batch_of_no_tokens_is_committed():
    import sparse_kv_selection_gb300 as S
    c = Cache([20, 7], 2, 1, 64, BF16, page=16, room=40, seed=6)
    batch = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=0, max_new=1, free_pages=i32(c.free), n_pages=i32(c.n_pages))
    batch.plan(i32([0, 0]))
    batch.rotate(*rows_of(0, c, 2), append=True)
    batch.commit(i32([0, 0]))
    assert S.last_error() == 0 and c.kv.seq_lens.tolist() == [20, 7]


# --------------------------------------------------------------------------- #
# batches that share a cache
# --------------------------------------------------------------------------- #
def test_two_batches_hand_out_different_pages():
    """A batch for prompts and one for drafts on one cache take pages from one list."""
    import sparse_kv_selection_gb300 as S
    c = Cache([20, 30], 2, 1, 64, BF16, page=16, room=200, seed=7)
    state = dict(free_pages=i32(c.free), n_pages=i32(c.n_pages), free_head=i32([0]))
    prompts = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=100, max_new=90, **state)
    drafts = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=20, max_new=10, **prompts.pages)
    for step in range(3):
        for batch, n in ((prompts, [30, 0]), (drafts, [4, 9]), (prompts, [0, 17])):
            batch.plan(i32(n))
            batch.rotate(*rows_of(batch.positions.numel(), c, step), append=True)
            batch.commit(i32(n))
    assert S.last_error() == 0
    assert c.kv.seq_lens.tolist() == [20 + 3 * 34, 30 + 3 * 26]
    held = c.kv.block_table.cpu().numpy()
    pages = [int(held[b, i]) for b, t in enumerate(c.kv.seq_lens.tolist()) for i in range(-(-t // 16))]
    assert len(set(pages)) == len(pages)
    assert int(state["free_head"][0]) == len(pages) - sum(c.n_pages)


def test_pages_of_a_sequence_that_ends_are_handed_out_again():
    """Given back in front of the free ones, between two steps, without the host
    reading a counter; what the sequence's table row still names is not used."""
    import sparse_kv_selection_gb300 as S
    c = Cache([0, 0], 2, 1, 64, BF16, page=16, room=48, seed=7)
    free = i32(c.free[:5])
    batch = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=48, max_new=48, free_pages=free, n_pages=i32(c.n_pages))

    def feed(n):
        batch.plan(i32(n))
        batch.rotate(*rows_of(48, c, sum(n)), append=True)
        batch.commit(i32(n))

    feed([40, 0])
    feed([0, 20])
    assert S.last_error() == 0 and c.kv.seq_lens.tolist() == [40, 20]
    head, n_pages = batch.pages["free_head"], batch.pages["n_pages"]
    head -= n_pages[0]
    free[head.long() + torch.arange(3, device="cuda")] = c.kv.block_table[0, :3]
    n_pages[0] = 0
    c.kv.seq_lens[0] = 0
    feed([0, 28])                                  # one page more
    feed([30, 0])                                  # two
    assert S.last_error() == 0 and c.kv.seq_lens.tolist() == [30, 48]
    table = c.kv.block_table.tolist()
    assert sorted(table[1][:3] + table[0][:2]) == sorted(c.free[:5].tolist())


def test_a_tree_through_a_batch_for_prompts():
    """max_new above the largest tree: one batch serves prompts and trees."""
    import sparse_kv_selection_gb300 as S
    c = Cache([0, 40], 4, 2, 64, BF16, t_max=900, seed=8)
    batch = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=710, max_new=700)
    small = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=710, max_new=128)
    q, k, v = rows_of(710, c, 1)
    batch.plan(i32([700, 9]))
    batch.rotate(q, k, v, append=True)
    batch.attend()
    batch.commit(i32([700, 9]))
    assert S.last_error() == 0
    parents = i32(list(range(-1, 127)) + [-1, 0, 0, 1] + [-1] * 578)
    for x in (batch, small):
        x.plan(i32([128, 4]), parents)
        x.rotate(q, k, v)
        x.attend()
    assert S.last_error() == 0
    assert torch.equal(batch.out[:132], small.out[:132]) and torch.equal(batch.lse[:132], small.lse[:132])


def test_a_new_plan_forgets_the_rotated_rows():
    """Nothing is committed of a plan whose tokens were not rotated."""
    import sparse_kv_selection_gb300 as S
    c = Cache([20], 2, 1, 64, BF16, t_max=64, seed=9)
    batch = S.TokenBatch(c.kv, S.RopeTable(64), max_tokens=8, max_new=8)
    batch.plan(i32([8]))
    batch.rotate(*rows_of(8, c, 1), append=True)
    batch.commit(i32([8]))
    batch.plan(i32([8]))
    with pytest.raises(ValueError):
        batch.commit(i32([8]))
    assert S.last_error() == 0 and c.kv.seq_lens.tolist() == [28]


def test_a_batch_made_for_another_stream():
    """The batch's buffers are set on its own stream: a busy current stream does not
    set them after they have been used."""
    import sparse_kv_selection_gb300 as S
    c = Cache([20, 30], 2, 1, 64, BF16, page=16, room=40, seed=7)
    s = torch.cuda.Stream()
    rope, n, free, n_pages = S.RopeTable(64), i32([17, 3]), i32(c.free), i32(c.n_pages)
    for handle in (s, s.cuda_stream):
        want_lens = c.kv.seq_lens.tolist()
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)             # the current stream is busy for about 0.1 s
        batch = S.TokenBatch(c.kv, rope, max_tokens=20, max_new=17, free_pages=free, n_pages=n_pages, stream=handle)
        batch.plan(n)
        torch.cuda.synchronize()
        assert S.last_error() == 0
        assert batch.positions.tolist() == list(range(20, 37)) + list(range(30, 33))
        assert batch.cu_new.tolist() == [0, 17, 20] and (batch.slots >= 0).all()
        assert c.kv.seq_lens.tolist() == want_lens


# --------------------------------------------------------------------------- #
# attention
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("Hq,Hkv,n,t", [(2, 2, 3, 60), (8, 1, 30, 300), (4, 4, 20, 9000), (2, 1, 1, 20000), (8, 2, 3, 0)])
def test_nan_reaches_the_rows_that_attend_it(dtype, d, Hq, Hkv, n, t):
    """A query with NaN in it has NaN for its output and its log-sum-exp, whether its
    keys are split over CTAs or not, and no other row has; a NaN key of an
    unattended token changes nothing."""
    import sparse_kv_selection_gb300 as S
    c = Cache([t, 40], Hq, Hkv, d, dtype, page=16, room=1, seed=3)
    T = n + 2
    q, k, v = rows_of(T, c, 1)
    mask = torch.zeros(T, 4, dtype=torch.int32, device="cuda")
    for j in range(n):                             # each sees itself and the first
        mask[j, 0] = 1 | (1 << j)
    mask[n, 0] = 1                                 # sequence 1: the second token sees only itself
    mask[n + 1, 0] = 2
    cu, ws = i32([0, n, T]), S.make_tree_workspace(c.kv, n + 2)

    def attend(q, k):
        out, lse = torch.full_like(q, 3.0), torch.full((T, Hq), 3.0, device="cuda")
        S.tree_attn(c.kv, q, k, v, d ** -0.5, cu, n + 2, out, lse, ws, tree_mask=mask)
        assert S.last_error() == 0
        return out, lse

    want, wl = attend(q, k)
    bad = torch.zeros(T, Hq, dtype=torch.bool, device="cuda")
    bad[n - 1, Hq - 1] = True
    q2 = q.clone()
    q2[n - 1, Hq - 1, d // 2] = float("nan")
    out, lse = attend(q2, k)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])
    k2 = k.clone()
    k2[n + 1, :, 1] = float("nan")                 # only its own rows attend it
    bad[:] = False
    bad[n + 1] = True
    out, lse = attend(q, k2)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_that_step_back(dtype):
    """Offsets that go back and forth give every second sequence all tokens, more key
    tiles than 32 bits count although the call's own sizes are small: the call is
    flagged and writes nothing."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_LEN
    B, T, Hq, Hkv, d, page, blocks = 256, 8192, 64, 8, 64, 4096, 256
    tiles, units = page * blocks // 128, T * (Hq // Hkv) // 256
    assert (units + B) * Hkv * (tiles + T // 128 + 2) < 1 << 31 <= B // 2 * Hkv * units * tiles
    pool = torch.zeros(1, Hkv, page, d, device="cuda", dtype=dtype)
    kv = S.KVCache(pool, pool.clone(), i32([page * blocks] * B), Hq,
                   block_table=torch.zeros(B, blocks, dtype=torch.int32, device="cuda"))
    q, k = torch.zeros(T, Hq, d, device="cuda", dtype=dtype), torch.zeros(T, Hkv, d, device="cuda", dtype=dtype)
    out, lse = torch.full_like(q, 3.0), torch.full((T, Hq), 3.0, device="cuda")
    S.tree_attn(kv, q, k, k, 0.125, i32([0, T] * (B // 2) + [0]), T, out, lse, S.make_tree_workspace(kv, T))
    assert S.last_error() == DEV_BAD_LEN
    assert (out == 3.0).all() and (lse == 3.0).all()


def tiles_a_run(c, n):
    """Key tiles of 128 that a CTA takes, of how many a unit has (units of 256 rows, one a KV head here)."""
    import sparse_kv_selection_gb300 as S
    assert max(n) * (c.Hq // c.Hkv) <= 256
    unit = [-(-t // 128) + -(-x // 128) for t, x in zip(c.lens, n)]
    return -(-c.Hkv * sum(unit) // S.num_sms()), max(unit)


def check_rows(c, q, k, v, n, out, lse):
    """Causal results of every sequence against float64."""
    scale = c.d ** -0.5
    lo = 0
    for b, x in enumerate(n):
        r = slice(lo, lo + x)
        kc, vc = c.rows(b, c.lens[b])
        see = torch.ones(x, x, dtype=torch.bool, device="cuda").tril()
        wo, wl, eo, el = attn_ref(q[r].double(), kc, vc, k[r].double(), v[r].double(), see, scale, c.d, c.dtype)
        assert ((out[r].double() - wo).abs() <= eo).all(), (b, ((out[r].double() - wo).abs() / eo).max().item())
        assert ((lse[r].double() - wl).abs() <= el).all(), b
        lo += x


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("B,Hkv,G,n", [(4, 16, 1, 3), (4, 16, 8, 1), (2, 32, 2, 60), (4, 16, 8, 20), (4, 16, 1, 200)])
@pytest.mark.parametrize("top", [400, 90, 40, -300])
def test_maximum_that_grows_along_a_run(d, B, Hkv, G, n, top):
    """Runs of more than four tiles of one unit, so that a stream's output is
    rescaled while it is summed: the maximum moves by 37, 8, 4 and -28 (base 2) a
    tile, with one row tile (streams on every second tile) and with two."""
    import sparse_kv_selection_gb300 as S
    t = 2000
    c = Cache([t] * B, G * Hkv, Hkv, d, BF16, seed=3)
    run, unit = tiles_a_run(c, [n] * B)
    assert 4 < run and 12 < unit                   # (units of up to 12 tiles are not cut)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    # queries of ones on key rows of a constant: logits rise by `top` over the cache
    ramp = torch.linspace(0, top, t, device="cuda")[None, None, :, None] / d ** 0.5
    c.k[:, :, :t] = (ramp + torch.randn(B, Hkv, t, d, generator=g, device="cuda") * 0.1).to(BF16)
    q = torch.ones(B * n, G * Hkv, d, device="cuda", dtype=BF16)
    k, v = torch.randn(2, B * n, Hkv, d, generator=g, device="cuda").to(BF16)
    out, lse = torch.empty_like(q), torch.empty(B * n, G * Hkv, device="cuda")
    S.tree_attn(c.kv, q, k, v, d ** -0.5, i32(np.arange(B + 1) * n), n, out, lse, S.make_tree_workspace(c.kv, n))
    assert S.last_error() == 0
    check_rows(c, q, k, v, [n] * B, out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [0, 16, 32, 64, 128, 48])
@pytest.mark.parametrize("G,n", [(1, 2), (8, 20)])
def test_every_value_row_counts_on_long_runs(dtype, page, G, n):
    """Runs of more than 32 tiles of one unit, past every window of page numbers. A
    value row is one in the column of its 16-key group (modulo 61) and zero
    elsewhere, so that each column is the weight of few groups, and a group that is
    lost or taken from another place shows in full."""
    import sparse_kv_selection_gb300 as S
    B, Hkv, d, t = 20, 8, 64, 5100
    c = Cache([t] * B, G * Hkv, Hkv, d, dtype, page=page, room=1, seed=4)
    run, unit = tiles_a_run(c, [n] * B)
    assert run > 32 and unit > 32
    col = (torch.arange(t, device="cuda") // 16) % 61
    rows = torch.nn.functional.one_hot(col, d).to(dtype)[:, None].expand(t, Hkv, d)
    for b in range(B):
        c.set_rows(b, 0, c.rows(b, t)[0].transpose(0, 1).to(dtype), rows)
    q, k, v = rows_of(B * n, c, 1)
    q *= 0.5
    v.zero_()
    out, lse = torch.empty_like(q), torch.empty(B * n, G * Hkv, device="cuda")
    S.tree_attn(c.kv, q, k, v, d ** -0.5, i32(np.arange(B + 1) * n), n, out, lse, S.make_tree_workspace(c.kv, n))
    assert S.last_error() == 0
    check_rows(c, q, k, v, [n] * B, out, lse)
    # the bound sees a tile or a 16-key group of V that comes from elsewhere
    kc, vc = c.rows(0, t)
    see = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    wo, _, eo, _ = attn_ref(q[:n].double(), kc, vc, k[:n].double(), v[:n].double(), see, d ** -0.5, d, dtype)
    for to, frm, size in ((4096, 0, 128), (512, 0, 16), (4224, 4096, 128), (4992, 4480, 16)):
        wrong = vc.clone()
        wrong[:, to:to + size] = vc[:, frm:frm + size]
        bad = attn_ref(q[:n].double(), kc, wrong, k[:n].double(), v[:n].double(), see, d ** -0.5, d, dtype)[0]
        assert ((bad - wo).abs() > 4 * eo).any(-1).all(), (to, frm)


# --------------------------------------------------------------------------- #
# rotary angles
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("interleaved", [False, True])
def test_sine_and_cosine_near_their_zeros(interleaved):
    """Pairs (1, 0) become (cos, sin) exactly, so fp32 results show the angle's own
    error. The angle is folded to the nearest quarter turn as integers and keeps 34
    bits behind the point: 2 pi 2^-34; its conversion to fp32 is off by 2^-24 of it
    and sine or cosine by two units of the last place, 5 * 2^-24 of the value."""
    import sparse_kv_selection_gb300 as S
    d, T = 128, 4096
    c = Cache([3], 1, 1, d, F32, t_max=8, seed=1)
    rope = S.RopeTable(d, interleaved=interleaved)
    positions = np.random.default_rng(5).integers(0, 1 << 20, T)
    q = torch.zeros(T, 1, d, device="cuda")
    q[..., 0::2] = 1.0 if interleaved else 0.0
    if not interleaved:
        q[..., :d // 2] = 1.0
    got, k = torch.empty_like(q), torch.zeros(T, 1, d, device="cuda")
    S.rope_append(c.kv, rope, i32(positions), q, k, None, got)
    assert S.last_error() == 0
    got = got[:, 0].double().cpu().numpy()
    cos, sin = (got[:, 0::2], got[:, 1::2]) if interleaved else (got[:, :d // 2], got[:, d // 2:])
    turn = positions.astype(np.uint64)[:, None] * rope.turns.cpu().numpy().astype(np.uint64)[None]   # modulo 2^64
    quarter = (turn + np.uint64(1 << 61)) >> np.uint64(62)
    rest = (turn - (quarter << np.uint64(62))).astype(np.int64).astype(np.float64) * (2 * np.pi * 2.0 ** -64)
    s, z = np.sin(rest), np.cos(rest)
    quarter = (quarter & np.uint64(3)).astype(int)
    want_cos, want_sin = np.choose(quarter, [z, -s, -z, s]), np.choose(quarter, [s, z, -s, -z])
    assert (np.abs(want_sin) < 2.0 ** -9).sum() > 100 and (np.abs(want_cos) < 2.0 ** -9).sum() > 100
    for x, w in ((cos, want_cos), (sin, want_sin)):
        assert (np.abs(x - w) <= 5 * 2.0 ** -24 * np.abs(w) + 2 * np.pi * 2.0 ** -34).all()


# --------------------------------------------------------------------------- #
# the ends of the ranges
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tree", [False, True])
def test_the_most_sequences_a_call_takes(dtype, tree):
    """16384 sequences, a step from planning to committing: every sequence's pages,
    rows and length, and the attention of some."""
    import sparse_kv_selection_gb300 as S
    rng = np.random.default_rng(5)
    B, d, page, blocks = 16384, 64, 16, 3
    lens, n = rng.integers(0, 33, B), rng.integers(0, 3, B)
    have = -(-lens // page)
    table = np.full((B, blocks), -1)
    ids = rng.permutation(B * blocks)
    for i in range(blocks):
        table[have > i, i] = ids[i * B:(i + 1) * B][have > i]
    free = np.setdiff1d(ids, table)
    pool = torch.randn(B * blocks, 1, page, d, device="cuda", dtype=dtype)
    kv = S.KVCache(pool, torch.randn_like(pool), i32(lens), 1, block_table=i32(table))
    T = int(n.sum()) + 3
    batch = S.TokenBatch(kv, S.RopeTable(d), max_tokens=T, max_new=2, free_pages=i32(free), n_pages=i32(have))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q, k, v = torch.randn(3, T, 1, d, generator=g, device="cuda").to(dtype)
    parents = np.full(T, -1)
    cu = np.concatenate([[0], np.cumsum(n)])
    parents[cu[:-1][n == 2] + 1] = rng.integers(-1, 1, (n == 2).sum())
    batch.plan(i32(n), i32(parents) if tree else None)
    batch.rotate(q, k, v, append=not tree)
    batch.attend()
    before = kv.k.clone(), kv.v.clone()
    batch.commit(i32(n))
    assert S.last_error() == 0
    assert kv.seq_lens.cpu().numpy().tolist() == (lens + n).tolist()
    got = kv.block_table.cpu().numpy()
    need = -(-(lens + n) // page)
    held = [got[:, i][need > i] for i in range(blocks)]
    assert len(np.unique(np.concatenate(held))) == need.sum()
    b = np.repeat(np.arange(B), n)
    pos = lens[b] + np.arange(cu[-1]) - cu[b]
    at, row = torch.tensor(got[b, pos // page], device="cuda"), torch.tensor(pos % page, device="cuda")
    assert torch.equal(kv.k[at, 0, row], batch.k[:cu[-1], 0]) and torch.equal(kv.v[at, 0, row], v[:cu[-1], 0])
    for b in rng.integers(0, B, 60).tolist() + [B - 1]:
        r = slice(int(cu[b]), int(cu[b + 1]))
        if n[b] == 0:
            continue
        p = np.arange(lens[b])
        kc, vc = [x[torch.tensor(got[b, p // page], device="cuda").long(), :, torch.tensor(p % page, device="cuda")]
                  .double().transpose(0, 1) for x in before]
        see = torch.ones(n[b], n[b], dtype=torch.bool, device="cuda").tril()
        if tree and n[b] == 2:
            see[1, 0] = bool(parents[cu[b] + 1] == 0)
        wo, wl, eo, el = attn_ref(batch.q[r].double(), kc, vc, batch.k[r].double(), v[r].double(), see, batch.scale, d, dtype)
        assert ((batch.out[r].double() - wo).abs() <= eo).all() and ((batch.lse[r].double() - wl).abs() <= el).all()


def test_the_first_step_of_a_process_is_captured(tmp_path):
    """No call has been made before the capture, in a process of its own."""
    script = tmp_path / "first.py"
    script.write_text(FIRST)
    r = subprocess.run([sys.executable, str(script)], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0, r.stdout + r.stderr


FIRST = """
import torch
import sparse_kv_selection_gb300 as S
for dtype in (torch.bfloat16, torch.float32):
    k, v = torch.randn(2, 8, 2, 16, 64, device="cuda").to(dtype)
    z = dict(dtype=torch.int32, device="cuda")
    kv = S.KVCache(k, v, torch.tensor([20, 0], **z), 4, block_table=torch.tensor([[0, 1, -1], [-1, -1, -1]], **z))
    batch = S.TokenBatch(kv, S.RopeTable(64), max_tokens=9, max_new=6, free_pages=torch.arange(2, 8, **z),
                         n_pages=torch.tensor([2, 0], **z))
    q, kn, vn = torch.randn(9, 4, 64, device="cuda").to(dtype), *torch.randn(2, 9, 2, 64, device="cuda").to(dtype)
    n, parents = torch.tensor([3, 6], **z), torch.tensor([-1, 0, 0, -1, 0, 1, 2, 3, 4], **z)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        batch.plan(n, parents)
        batch.rotate(q, kn, vn)
        batch.attend()
        batch.commit(n)
    g.replay()
    assert S.last_error() == 0
    assert kv.seq_lens.tolist() == [23, 6], kv.seq_lens
    assert batch.out.float().isfinite().all() and (batch.lse != 0).all()
"""
