"""Token-batch operators on the GPU against plain 64-bit forms: planning,
rotary positions with the cache append, tree attention, committing."""
import math

import numpy as np
import pytest

from tokens_util import (TREE_MAX, WORDS, Cache, ancestors, attn_ref, plan_ref, rope_ref, theta_ref,
                         words_of)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def random_parents(rng, n, back=6):
    return [int(max(-1, j - 1 - rng.integers(0, back))) if rng.random() < 0.9 else -1 for j in range(n)]


# --------------------------------------------------------------------------- #
# plan
# --------------------------------------------------------------------------- #
def run_plan(c, n, T, parents=None, free=None, head=0, in_place=False):
    import sparse_kv_selection_gb300 as S
    B = c.B
    cu, pos, slots = i32(np.full(B + 1, -9)), i32(np.full(T, -9)), i32(np.full(T, -9))
    mask = None if parents is None else i32(np.full((T, WORDS), -9))
    kw = {}
    if c.page:
        fh, npg = i32([head]), i32(c.n_pages)
        kw = dict(free_pages=i32(c.free if free is None else free), free_head=fh, n_pages=npg)
        if not in_place:
            kw.update(free_head_out=i32([-9]), n_pages_out=i32(np.full(B, -9)))
    S.plan_tokens(c.kv, i32(n), cu, pos, slots, parents=None if parents is None else i32(parents),
                  tree_mask=mask, **kw)
    bits = S.last_error()
    res = [x.cpu().numpy() for x in (cu, pos, slots)] + [None if mask is None else mask.cpu().numpy()]
    if c.page:
        res += [c.kv.block_table.cpu().numpy(), int(kw["free_head" if in_place else "free_head_out"][0]),
                kw["n_pages" if in_place else "n_pages_out"].cpu().numpy().tolist()]
    return res, bits


def check_plan(c, n, T, want_bits=0, parents=None, free=None, head=0, in_place=False):
    want = plan_ref(c.lens, n, T, c.t_max, parents=parents, page=c.page, table=c.table,
                    free=c.free if c.page and free is None else free, head=head,
                    n_pages=c.n_pages if c.page else None)
    got, bits = run_plan(c, n, T, parents, free, head, in_place)
    assert bits == want_bits
    for name, g, w in zip(("cu", "positions", "slots", "mask", "table", "head", "n_pages"), got, want):
        if w is None or (name == "mask" and parents is None):
            continue
        assert np.array_equal(np.asarray(g), np.asarray(w)), name


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,t,n,pad", [(1, (0, 0), (1, 1), 0), (1, (17, 17), (128, 128), 3),
                                       (5, (0, 70), (0, 40), 9), (33, (1, 500), (0, 64), 1),
                                       (700, (0, 60), (0, 12), 0)])
def test_plan(page, tree, B, t, n, pad):
    rng = np.random.default_rng(B + page)
    lens = rng.integers(t[0], t[1] + 1, B).tolist()
    new = rng.integers(n[0], n[1] + 1, B).tolist()
    c = Cache(lens, 1, 1, 64, BF16, page=page, room=n[1], seed=1, spare=5)
    T = sum(new) + pad
    parents = sum([random_parents(rng, x) for x in new], []) + [-1] * pad if tree else None
    check_plan(c, new, T, parents=parents, in_place=bool(B % 2))


@pytest.mark.parametrize("page", [0, 64])
def test_plan_long_chunks(page):
    """Prompts of thousands of tokens: the cluster's CTAs share the tokens."""
    c = Cache([0, 5, 63, 64, 4000], 1, 1, 64, BF16, page=page, room=9000, seed=2)
    check_plan(c, [9000, 1, 0, 4097, 777], 9000 + 1 + 4097 + 777 + 11)


def test_plan_chain_tree_is_deep():
    """A tree that is one path of 128 tokens: masks are full prefixes."""
    c = Cache([7], 1, 1, 64, BF16, page=16, room=128, seed=3)
    check_plan(c, [128], 128, parents=list(range(-1, 127)))


def test_plan_surplus_pages_are_used_before_new_ones():
    c = Cache([20, 20], 1, 1, 64, BF16, page=16, room=200, seed=4)
    c.n_pages[0] = 6                                   # four pages left by rejected tokens
    c.table[0, 2:6] = c.free[:4]
    c.kv.block_table[0, 2:6] = i32(c.free[:4])
    check_plan(c, [70, 13], 83, head=4)                # 90 positions fit 6 pages; one page for b = 1
    check_plan(c, [120, 13], 133, head=4)


def test_plan_refusals():
    from sparse_kv_selection_gb300.binding import DEV_BAD_BLOCK, DEV_BAD_INDEX, DEV_BAD_LEN, DEV_CAPACITY
    # pages run out at sequence 1; sequence 2 needs one too and gets none, sequence 3 needs none
    c = Cache([16, 16, 16, 10], 1, 1, 64, BF16, page=16, room=64, seed=5)
    check_plan(c, [16, 33, 1, 3], 53, DEV_CAPACITY, free=c.free[:3])
    # beyond t_max
    c = Cache([10, 30], 1, 1, 64, BF16, seed=6, t_max=32)
    check_plan(c, [22, 3], 25, DEV_CAPACITY)
    # tokens beyond T: the sequence that is cut and those behind it are not placed
    c = Cache([10, 30, 4], 1, 1, 64, BF16, seed=6, t_max=64)
    check_plan(c, [5, 8, 2], 9, DEV_CAPACITY)
    # a negative count is read as none
    check_plan(c, [5, -3, 2], 9, DEV_BAD_LEN)
    # a tree above 128 tokens gets no masks and no slots
    c = Cache([10, 3], 1, 1, 64, BF16, seed=7, t_max=300)
    check_plan(c, [129, 2], 131, DEV_BAD_LEN, parents=[-1] * 131)
    # a parent that is not an earlier token
    c = Cache([10, 3], 1, 1, 64, BF16, seed=7, t_max=300)
    check_plan(c, [3, 4], 7, DEV_BAD_INDEX, parents=[-1, 1, -2, -1, 0, 1, 3])
    # a page outside the pool: flagged, its tokens have no slot
    c = Cache([16], 1, 1, 64, BF16, page=16, room=64, seed=8)
    got, bits = run_plan(c, [20], 20, free=[10 ** 6, 0])
    assert bits == DEV_BAD_BLOCK
    assert (got[2][:16] == -1).all() and (got[2][16:] == np.arange(4)).all()


# --------------------------------------------------------------------------- #
# rope
# --------------------------------------------------------------------------- #
SCALINGS = {
    "plain": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=8.0),
    "bands": dict(scaling="bands", factor=8.0, original=8192, low=1.0, high=4.0),
    "ramp": dict(scaling="ramp", factor=16.0, original=4096, low=1.0, high=32.0),
}


def rope_tol(x, rot, dtype):
    """|x| and |y| of a pair bound the result's terms; cos and sin are off by
    2^-22 (angle in half turns to 2^-25, pi times that in radians, and the
    functions' and mscale's roundings), two products and a sum by 3 2^-24, and
    the result is rounded once."""
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    return lambda y, m: half * np.abs(y) + 1.5 * m * (2.0 ** -22 + 3 * 2.0 ** -24)


def check_rotated(got, x, positions, kind, rot, interleaved, dtype):
    kw = dict(kind)
    theta, ms = theta_ref(rot, 10000.0, kw.pop("scaling", None), **kw)
    want = rope_ref(x, positions, theta, ms, rot, interleaved)
    mag = np.abs(x).max(-1, keepdims=True) * 2
    assert (np.abs(got - want) <= rope_tol(x, rot, dtype)(want, mag)).all()
    assert np.array_equal(got[..., rot:], x[..., rot:])      # the rest of the head is kept


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,d,rot", [(1, 1, 64, 64), (8, 2, 128, 128), (4, 4, 128, 48), (8, 1, 64, 16),
                                          (32, 8, 128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [1, 37])
def test_rope_packed(dtype, Hq, Hkv, d, rot, interleaved, T):
    import sparse_kv_selection_gb300 as S
    c = Cache([3], Hq, Hkv, d, dtype, t_max=8, seed=1)
    before = c.k.clone()
    rng = np.random.default_rng(T + rot)
    positions = rng.integers(0, 200000, T)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * d, device="cuda", dtype=dtype)      # a fused projection's output
    q = qkv[:, :Hq * d].view(T, Hq, d)
    k = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
    rope = S.RopeTable(rot, interleaved=interleaved)
    q_out, k_out = torch.full((T, Hq, d), 7.0, device="cuda", dtype=dtype), torch.full((T, Hkv, d), 7.0, device="cuda", dtype=dtype)
    S.rope_append(c.kv, rope, i32(positions), q, k, None, q_out, k_out=k_out)
    assert S.last_error() == 0
    check_rotated(f64(q_out), f64(q), positions, {}, rot, interleaved, dtype)
    check_rotated(f64(k_out), f64(k), positions, {}, rot, interleaved, dtype)
    assert torch.equal(c.k.nan_to_num(), before.nan_to_num())
    # in place, from packed rows
    q2, k2 = q.contiguous(), k.contiguous()
    S.rope_append(c.kv, rope, i32(positions), q2, k2, None, q2, k_out=k2)
    assert torch.equal(q2, q_out) and torch.equal(k2, k_out)


@pytest.mark.parametrize("kind", list(SCALINGS))
@pytest.mark.parametrize("rot,dtype", [(128, F32), (64, BF16)])
def test_rope_scalings_and_far_positions(kind, rot, dtype):
    """Every scaling, at positions up to the ends of int32 (the fixed-point
    angle is as exact there as near 0)."""
    import sparse_kv_selection_gb300 as S
    c = Cache([3], 2, 1, 128, dtype, t_max=8, seed=1)
    positions = np.array([0, 1, 131071, 1 << 20, (1 << 31) - 1, -1, -(1 << 31)])
    T = len(positions)
    q, k = torch.randn(T, 2, 128, device="cuda", dtype=dtype), torch.randn(T, 1, 128, device="cuda", dtype=dtype)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    S.rope_append(c.kv, S.RopeTable(rot, **SCALINGS[kind]), i32(positions), q, k, None, q_out, k_out=k_out)
    assert S.last_error() == 0
    # float64 angles of the reference are off by position * theta * 2^-52 radians: 2^-21 at 2^31
    kw = dict(SCALINGS[kind])
    theta, ms = theta_ref(rot, 10000.0, kw.pop("scaling", None), **kw)
    for got, x in ((q_out, q), (k_out, k)):
        want = rope_ref(f64(x), positions, theta, ms, rot, False)
        m = np.abs(f64(x)).max(-1, keepdims=True) * 2
        slack = np.abs(positions)[:, None, None] * 2.0 ** -51 * m
        assert (np.abs(f64(got) - want) <= rope_tol(x, rot, dtype)(want, m) + slack).all()


@pytest.mark.parametrize("page", [0, 16, 32])
@pytest.mark.parametrize("dtype,Hq,Hkv,d", [(BF16, 8, 2, 128), (F32, 2, 2, 64), (BF16, 1, 1, 64)])
@pytest.mark.parametrize("big", [False, True])
def test_rope_append(page, dtype, Hq, Hkv, d, big):
    """k and v land in the rows of their slots, everything else is left alone,
    padding tokens and bad slots write nothing; one and two tasks a thread."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_INDEX
    n = [700, 3, 0, 2100] if big else [5, 3, 0, 11]
    if big and Hkv == 1:
        n = [n[0], 3, 0, 60000]
    elif big and dtype == F32:
        n = [n[0], 3, 0, 4200]
    lens = [20, 0, 9, 33]
    c = Cache(lens, Hq, Hkv, d, dtype, page=page, room=max(n), seed=2)
    T = sum(n) + 4
    got, bits = run_plan(c, n, T)
    assert bits == 0
    slots, positions = got[2].copy(), got[1]
    slots[-1] = 1 << 30                                   # outside the cache: flagged, not written
    slots[-2] = -7
    q, k = torch.randn(T, Hq, d, device="cuda", dtype=dtype), torch.randn(T, Hkv, d, device="cuda", dtype=dtype)
    v = torch.randn(T, Hkv, d, device="cuda", dtype=dtype)
    q_out = torch.full_like(q, 5.0)
    k_out = torch.full_like(k, 5.0)
    wk, wv = c.k.clone(), c.v.clone()
    S.rope_append(c.kv, S.RopeTable(d), i32(positions), q, k, v, q_out, slots=i32(slots), k_out=k_out)
    assert S.last_error() == DEV_BAD_INDEX
    real = sum(n)
    assert (q_out[real:] == 5.0).all() and (k_out[real:] == 5.0).all()
    check_rotated(f64(q_out[:real]), f64(q[:real]), positions[:real], {}, d, False, dtype)
    check_rotated(f64(k_out[:real]), f64(k[:real]), positions[:real], {}, d, False, dtype)
    cu = got[0]
    for b in range(4):
        if n[b] == 0:
            continue
        blk, row = c.at(b, np.arange(lens[b], lens[b] + n[b]))
        blk, row = torch.tensor(blk, device="cuda"), torch.tensor(row, device="cuda")
        wk[blk, :, row] = k_out[cu[b]:cu[b + 1]]
        wv[blk, :, row] = v[cu[b]:cu[b + 1]]
    for have, want in ((c.k, wk), (c.v, wv)):
        assert torch.equal(have.nan_to_num(99.0), want.nan_to_num(99.0))


# --------------------------------------------------------------------------- #
# tree attention
# --------------------------------------------------------------------------- #
def tree_inputs(c, n, pad, seed, masks=None, stride_extra=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = sum(n) + pad
    kw = dict(device="cuda", dtype=c.dtype, generator=g)
    q = torch.randn(T, c.Hq, c.d, **kw)
    k = torch.randn(T, c.Hkv * c.d + stride_extra, **kw)[:, :c.Hkv * c.d].view(T, c.Hkv, c.d)
    v = torch.randn(T, c.Hkv * c.d + stride_extra, **kw)[:, :c.Hkv * c.d].view(T, c.Hkv, c.d)
    if pad:
        q[-pad:] = k[-pad:] = v[-pad:] = float("nan")
    return q, k, v


def check_tree(c, n, pad=0, seed=0, sets=None, scale=None, max_new=None, stride_extra=0, bits=0, skip=(), calls=1,
               q_gain=1.0):
    """sets: per token, the new tokens it may attend (None: causal)."""
    import sparse_kv_selection_gb300 as S
    T = sum(n) + pad
    q, k, v = tree_inputs(c, n, pad, seed, stride_extra=stride_extra)
    q *= q_gain
    scale = c.d ** -0.5 if scale is None else scale
    cu = np.concatenate([[0], np.cumsum(n)])
    mask = None if sets is None else torch.tensor(words_of(list(sets) + [set()] * pad, T), device="cuda")
    max_new = max(n) if max_new is None else max_new
    ws = S.make_tree_workspace(c.kv, max_new)
    for _ in range(calls):
        out = torch.full((T, c.Hq, c.d), 3.0, device="cuda", dtype=c.dtype)
        lse = torch.full((T, c.Hq), 3.0, device="cuda")
        S.tree_attn(c.kv, q, k, v, scale, i32(cu), max_new, out, lse, ws, tree_mask=mask)
    assert S.last_error() == bits
    assert (out[cu[-1]:] == 3.0).all() and (lse[cu[-1]:] == 3.0).all()
    for b in range(c.B):
        if n[b] == 0 or b in skip:
            continue
        r = slice(int(cu[b]), int(cu[b + 1]))
        if sets is None:
            see = torch.ones(n[b], n[b], dtype=torch.bool, device="cuda").tril()
        else:
            see = torch.zeros(n[b], n[b], dtype=torch.bool)
            for j in range(n[b]):
                for p in sets[cu[b] + j]:
                    if p < n[b]:
                        see[j, p] = True
            see = see.cuda()
        kc, vc = c.rows(b, c.lens[b])
        wo, wl, eo, el = attn_ref(q[r].double(), kc, vc, k[r].double(), v[r].double(), see, scale, c.d, c.dtype)
        go, gl = out[r].double(), lse[r].double()
        dead = torch.isinf(wl)
        assert torch.equal(torch.isinf(gl) & (gl < 0), dead), b
        assert (go[dead] == 0).all(), b
        assert ((go - wo).abs() <= eo).all(), (b, ((go - wo).abs() / eo.clamp(min=1e-30)).max().item())
        ok = ((gl - wl).abs() <= el) | dead
        assert ok.all(), (b, (gl - wl)[~dead].abs().max().item())
    return out, lse


def random_sets(rng, n):
    return sum([ancestors(random_parents(rng, x)) for x in n], [])


HEADS = [(1, 1), (4, 4), (4, 2), (8, 2), (8, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("page", [0, 16])
def test_tree_shapes(dtype, d, Hq, Hkv, page):
    rng = np.random.default_rng(Hq * 10 + Hkv)
    n = [7, 1, 0, 33, 64]
    c = Cache([300, 1, 50, 0, 129], Hq, Hkv, d, dtype, page=page, room=1, seed=Hq + d)
    check_tree(c, n, pad=3, seed=d, sets=random_sets(rng, n), calls=2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [0, 16, 48, 128])
@pytest.mark.parametrize("t", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 1000])
def test_tree_cache_lengths(dtype, page, t):
    rng = np.random.default_rng(t)
    c = Cache([t, max(0, t - 1)], 4, 2, 128, dtype, page=page, room=1, seed=t)
    check_tree(c, [5, 12], seed=t, sets=random_sets(rng, [5, 12]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1), (8, 4)])
@pytest.mark.parametrize("n", [1, 2, 16, 31, 32, 33, 64, 65, 127, 128])
def test_tree_sizes(dtype, Hq, Hkv, n):
    """Every row count around a row tile's edges, through the largest tree."""
    rng = np.random.default_rng(n)
    c = Cache([200, 77], Hq, Hkv, 128, dtype, seed=n)
    check_tree(c, [n, 3], seed=n, sets=random_sets(rng, [n, 3]))


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF16, 128), (BF16, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("n", [[1, 1, 1], [129, 0, 5], [400, 1000, 255]])
def test_causal_chunks(dtype, d, Hq, Hkv, n):
    c = Cache([0, 130, 700], Hq, Hkv, d, dtype, page=32, room=1, seed=sum(n))
    check_tree(c, n, pad=2, seed=1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masks_that_leave_rows_empty(dtype):
    """No cached key and no bit: out = 0, lse = -inf; a token may be kept from
    seeing itself, see later ones, and bits beyond its sequence are ignored."""
    c = Cache([0, 0, 5], 4, 2, 128, dtype, t_max=16, seed=3)
    sets = [set(), {0}, {2, 0}, {100, 3, 127}] + [set(), set()] + [set(), {1, 0, 90}]
    check_tree(c, [4, 2, 2], seed=5, sets=sets)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales_and_large_logits(dtype, scale):
    rng = np.random.default_rng(1)
    c = Cache([300, 40], 4, 1, 64, dtype, seed=3)
    check_tree(c, [9, 30], seed=5, sets=random_sets(rng, [9, 30]), scale=scale, q_gain=4.0)


def test_growing_maximum():
    """Each later key outweighs all before it: the running maximum moves at
    every tile, by a lot."""
    c = Cache([1500], 2, 1, 128, BF16, seed=3)
    ramp = torch.linspace(0, 60, 1500, device="cuda")[None, None, :, None]
    c.k[:, :, :1500] = (torch.ones_like(c.k[:, :, :1500], dtype=F32) * ramp / 128 ** 0.5).to(BF16)
    import sparse_kv_selection_gb300 as S
    q = torch.ones(3, 2, 128, device="cuda", dtype=BF16)
    k, v = torch.randn(2, 3, 1, 128, device="cuda", dtype=BF16)
    out, lse = torch.empty(3, 2, 128, device="cuda", dtype=BF16), torch.empty(3, 2, device="cuda")
    S.tree_attn(c.kv, q, k, v, 128 ** -0.5, i32([0, 3]), 3, out, lse, S.make_tree_workspace(c.kv, 3))
    assert S.last_error() == 0
    kc, vc = c.rows(0, 1500)
    see = torch.ones(3, 3, dtype=torch.bool, device="cuda").tril()
    wo, wl, eo, el = attn_ref(q.double(), kc, vc, k.double(), v.double(), see, 128 ** -0.5, 128, BF16)
    assert ((out.double() - wo).abs() <= eo).all() and ((lse.double() - wl).abs() <= el).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_views_of_wider_buffers(dtype):
    rng = np.random.default_rng(1)
    c = Cache([90, 17], 8, 2, 64, dtype, page=16, seed=3)
    check_tree(c, [9, 20], pad=1, seed=5, sets=random_sets(rng, [9, 20]), stride_extra=64)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_max_new_bounds_a_sequence(dtype):
    """A sequence above max_new is flagged and its rows are left; a larger bound changes nothing."""
    from sparse_kv_selection_gb300.binding import DEV_BAD_LEN
    c = Cache([90, 17, 40], 4, 2, 64, dtype, seed=3)
    out, lse = check_tree(c, [9, 20, 9], seed=5, max_new=9, bits=DEV_BAD_LEN, skip=(1,))
    assert (out[9:29] == 3.0).all() and (lse[9:29] == 3.0).all()
    check_tree(c, [9, 20, 9], seed=5, max_new=500)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page,bad", [(16, [0]), (16, [3, 4, 9]), (64, [1]), (16, list(range(13)))])
def test_pages_outside_the_pool_are_not_attended(dtype, page, bad):
    from sparse_kv_selection_gb300.binding import DEV_BAD_BLOCK
    import sparse_kv_selection_gb300 as S
    c = Cache([200, 100], 4, 2, 128, dtype, page=page, seed=3)
    q, k, v = tree_inputs(c, [6, 4], 0, 1)
    good = [p for p in range(200) if p // page not in bad]
    kc, vc = [x[:, good] for x in c.rows(0, 200)]
    for i, x in enumerate(bad):
        c.kv.block_table[0, x] = 10 ** 6 if i % 2 else -3
    out, lse = torch.empty_like(q), torch.empty(10, 4, device="cuda")
    S.tree_attn(c.kv, q, k, v, 128 ** -0.5, i32([0, 6, 10]), 6, out, lse, S.make_tree_workspace(c.kv, 6))
    assert S.last_error() == DEV_BAD_BLOCK
    see = torch.ones(6, 6, dtype=torch.bool, device="cuda").tril()
    wo, wl, eo, el = attn_ref(q[:6].double(), kc, vc, k[:6].double(), v[:6].double(), see, 128 ** -0.5, 128, dtype)
    assert ((out[:6].double() - wo).abs() <= eo).all()
    assert ((lse[:6].double() - wl).abs() <= el).all()


def test_bad_lengths_are_flagged():
    from sparse_kv_selection_gb300.binding import DEV_BAD_LEN
    import sparse_kv_selection_gb300 as S
    c = Cache([20, 30], 2, 1, 64, BF16, seed=3)
    q, k, v = tree_inputs(c, [3, 4], 0, 1)
    ws = S.make_tree_workspace(c.kv, 4)
    for cu in ([0, 3, 99], [0, 5, 3], [-1, 3, 7]):
        out, lse = torch.full_like(q, 3.0), torch.full((7, 2), 3.0, device="cuda")
        S.tree_attn(c.kv, q, k, v, 0.125, i32(cu), 4, out, lse, ws)
        assert S.last_error() == DEV_BAD_LEN, cu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hq,Hkv,t,n", [(1, 8, 2, 20000, 13), (2, 8, 8, 9000, 3), (3, 8, 1, 5000, 70)])
def test_keys_split_over_ctas(dtype, B, Hq, Hkv, t, n):
    rng = np.random.default_rng(t)
    lens = [t, t // 2, 1][:B]
    c = Cache(lens, Hq, Hkv, 128, dtype, page=16, seed=4)
    ns = [n, 1, n][:B]
    check_tree(c, ns, seed=2, sets=random_sets(rng, ns), calls=2)


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements, the last sequence at its end."""
    t_max = 1 << 18
    c = Cache([5, 3, 200], 8, 8, 128, BF16, t_max=int(t_max * 4.2), seed=1)
    assert c.k.numel() > 1 << 31
    check_tree(c, [3, 1, 4], seed=2)


# --------------------------------------------------------------------------- #
# commit
# --------------------------------------------------------------------------- #
def run_commit(c, n, acc, m, stride_extra=0, in_place=False, copy=True, seed=0):
    import sparse_kv_selection_gb300 as S
    _, k, v = tree_inputs(c, n, 0, seed, stride_extra=stride_extra)
    cu = i32(np.concatenate([[0], np.cumsum(n)]))
    old = c.kv.seq_lens.clone()
    new = c.kv.seq_lens if in_place else torch.full_like(old, -9)
    rows = dict(k_new=k, v_new=v) if copy else dict(T=sum(n))
    S.commit_tokens(c.kv, cu, i32(m), None if in_place else new, accept_idx=None if acc is None else i32(acc), **rows)
    bits = S.last_error()
    if not in_place:
        assert torch.equal(c.kv.seq_lens, old)
    return k, v, new.cpu().numpy().tolist(), bits


def check_commit(c, n, acc, m, want_bits=0, refused=(), **kw):
    wk, wv = c.k.clone(), c.v.clone()
    k, v, new, bits = run_commit(c, n, acc, m, **kw)
    assert bits == want_bits
    cu = np.concatenate([[0], np.cumsum(n)])
    for b in range(c.B):
        if b in refused:
            assert new[b] == c.lens[b]
            continue
        assert new[b] == c.lens[b] + m[b]
        for i in range(m[b] if kw.get("copy", True) else 0):
            blk, row = c.at(b, c.lens[b] + i)
            src = cu[b] + (acc[b][i] if acc is not None else i)
            wk[int(blk), :, int(row)] = k[src]
            wv[int(blk), :, int(row)] = v[src]
    for have, want in ((c.k, wk), (c.v, wv)):
        assert torch.equal(have.nan_to_num(99.0), want.nan_to_num(99.0))


def paged_room(c, room):
    """Map pages for `room` more positions of every sequence."""
    at = 0
    for b, t in enumerate(c.lens):
        for blk in range(-(-t // c.page), -(-(t + room) // c.page)):
            c.kv.block_table[b, blk] = int(c.free[at])
            at += 1


@pytest.mark.parametrize("dtype,Hkv,d", [(BF16, 1, 64), (BF16, 8, 128), (F32, 2, 64)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_paths(dtype, Hkv, d, page, in_place):
    c = Cache([0, 15, 100, 31], Hkv, Hkv, d, dtype, page=page, room=40, seed=2)
    if page:
        paged_room(c, 40)
    n, m = [5, 40, 0, 12], [2, 7, 0, 12]
    acc = np.zeros((4, 12), int)
    acc[0, :2], acc[1, :7], acc[3] = [4, 0], [0, 3, 3, 9, 20, 38, 39], np.arange(12)[::-1]
    check_commit(c, n, acc, m, in_place=in_place, stride_extra=64)


@pytest.mark.parametrize("page", [0, 32])
def test_commit_first_tokens_and_lengths_only(page):
    c = Cache([10, 700], 4, 2, 128, BF16, page=page, room=900, seed=2)
    if page:
        paged_room(c, 900)
    check_commit(c, [900, 4], None, [777, 4])               # without numbers: the first tokens
    check_commit(c, [900, 4], None, [900, 0], copy=False)   # rows already in the cache


def test_commit_refusals_leave_the_sequence():
    from sparse_kv_selection_gb300.binding import DEV_BAD_BLOCK, DEV_BAD_INDEX, DEV_BAD_LEN, DEV_CAPACITY
    c = Cache([10, 30, 5], 2, 1, 64, BF16, t_max=32, seed=2)
    n = [6, 6, 6]
    ok = [[0, 1, 2]] * 3
    check_commit(c, n, ok, [3, 3, 3], DEV_CAPACITY, refused=(1,))                      # no room
    check_commit(c, n, ok, [7, 2, -1], DEV_BAD_LEN, refused=(0, 2))                    # more than offered, negative
    check_commit(c, n, ok, [4, 2, 3], DEV_BAD_LEN, refused=(0,))                       # above accept_cap
    check_commit(c, n, [[0, 1, 6], [0, 0, 0], [-1, 0, 0]], [3, 1, 1], DEV_BAD_INDEX, refused=(0, 2))
    c = Cache([10, 30], 2, 1, 64, BF16, page=16, room=32, seed=2)
    check_commit(c, [8, 8], [list(range(8))] * 2, [6, 3], DEV_BAD_BLOCK, refused=(1,))  # page not mapped


# --------------------------------------------------------------------------- #
# steps as they are used
# --------------------------------------------------------------------------- #
class Model:
    """Random q, k, v rows of a token stream, shared by both sides."""

    def __init__(self, B, Hq, Hkv, d, dtype, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.shape, self.dtype = (B, Hq, Hkv, d), dtype

    def qkv(self, T):
        _, Hq, Hkv, d = self.shape
        x = torch.randn(T, (Hq + 2 * Hkv) * d, generator=self.g, device="cuda", dtype=self.dtype)
        return (x[:, :Hq * d].view(T, Hq, d), x[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d),
                x[:, (Hq + Hkv) * d:].view(T, Hkv, d))


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("graph", [False, True])
def test_prompt_verify_decode_run(page, graph):
    """A prompt chunk, two verified trees and sparse decode steps on one cache,
    against float64 over the same rows; the verification step also replayed
    from a graph."""
    import sparse_kv_selection_gb300 as S
    B, Hq, Hkv, d, dtype, rot = 3, 8, 2, 128, BF16, 128
    c = Cache([0, 0, 0], Hq, Hkv, d, dtype, page=page, room=900, seed=2)
    kv, m = c.kv, Model(B, Hq, Hkv, d, dtype, 3)
    rope = S.RopeTable(rot)
    pages = dict(free_pages=i32(c.free), n_pages=i32(c.n_pages)) if page else {}
    # prompt
    T = 900
    batch = S.TokenBatch(kv, rope, max_tokens=T, max_new=700, **pages)
    n = [500, 0, 133]
    batch.plan(i32(n))
    q, k, v = m.qkv(T)
    batch.rotate(q, k, v, append=True)
    batch.attend()
    batch.commit(i32(n))
    assert S.last_error() == 0
    assert kv.seq_lens.cpu().tolist() == n
    cu = np.concatenate([[0], np.cumsum(n)])
    for b in (0, 2):
        kc, vc = c.rows(b, n[b])
        r = slice(int(cu[b]), int(cu[b + 1]))
        check_rotated(f64(kc.transpose(0, 1)), f64(k[r]), np.arange(n[b]), {}, rot, False, dtype)
        assert torch.equal(vc.transpose(0, 1), v[r].double())
        see = torch.ones(n[b], n[b], dtype=torch.bool, device="cuda").tril()
        wo, wl, eo, el = attn_ref(batch.q[r].double(), kc[:, :0], vc[:, :0], kc.transpose(0, 1), vc.transpose(0, 1),
                                  see, batch.scale, d, dtype)
        assert ((batch.out[r].double() - wo).abs() <= eo).all()
        assert ((batch.lse[r].double() - wl).abs() <= el).all()
    # two trees verified
    rng = np.random.default_rng(5)
    T = 40
    if page:
        pages.update(n_pages=batch.pages["n_pages"])
        used = int(batch.pages["free_head"][0])
        pages["free_pages"] = i32(c.free[used:])
    tree = S.TokenBatch(kv, rope, max_tokens=T, max_new=24, **pages)
    n_dev, par_dev, acc_dev, m_dev = i32([0] * B), i32([-1] * T), i32(np.zeros((B, 4))), i32([0] * B)
    qkv = torch.zeros(T, (Hq + 2 * Hkv) * d, device="cuda", dtype=dtype)
    parts = (qkv[:, :Hq * d].view(T, Hq, d), qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d),
             qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d))

    def step():
        tree.plan(n_dev, par_dev)
        tree.rotate(*parts)
        tree.attend()
        tree.commit(m_dev, acc_dev)

    g = None
    if graph:
        # with no tokens and nothing accepted a step changes nothing
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    for round_ in range(2):
        n = [[9, 24, 5], [1, 7, 20]][round_]
        parents = sum([random_parents(rng, x) for x in n], [])
        sets = sum([ancestors(parents[sum(n[:b]):sum(n[:b + 1])]) for b in range(B)], [])
        cu = np.concatenate([[0], np.cumsum(n)])
        # accept the path to each sequence's last token, at most four
        path = [sorted(sets[cu[b + 1] - 1])[:4] for b in range(B)]
        acc = np.zeros((B, 4), int)
        for b in range(B):
            acc[b, :len(path[b])] = path[b]
        q, k, v = m.qkv(T)
        for dst, src in zip(parts, (q, k, v)):
            dst.copy_(src)
        n_dev.copy_(i32(n)), par_dev.copy_(i32(parents + [-1] * (T - len(parents))))
        acc_dev.copy_(i32(acc)), m_dev.copy_(i32([len(p) for p in path]))
        lens = kv.seq_lens.cpu().tolist()
        before = [c.rows(b, lens[b]) for b in range(B)]
        g.replay() if graph else step()
        assert S.last_error() == 0
        assert kv.seq_lens.cpu().tolist() == [lens[b] + len(path[b]) for b in range(B)]
        for b in range(B):
            r = slice(int(cu[b]), int(cu[b + 1]))
            depth = np.array([len(sets[i]) - 1 for i in range(cu[b], cu[b + 1])])
            check_rotated(f64(tree.k[r]), f64(k[r]), lens[b] + depth, {}, rot, False, dtype)
            see = torch.zeros(n[b], n[b], dtype=torch.bool)
            for j in range(n[b]):
                see[j, sorted(sets[cu[b] + j])] = True
            kc, vc = before[b]
            wo, wl, eo, el = attn_ref(tree.q[r].double(), kc, vc, tree.k[r].double(), v[r].double(), see.cuda(),
                                      tree.scale, d, dtype)
            assert ((tree.out[r].double() - wo).abs() <= eo).all(), (round_, b)
            assert ((tree.lse[r].double() - wl).abs() <= el).all(), (round_, b)
            kc, vc = c.rows(b, lens[b] + len(path[b]))
            src = torch.tensor([cu[b] + p for p in path[b]], device="cuda")
            assert torch.equal(kc[:, lens[b]:].transpose(0, 1), tree.k[src].double())
            assert torch.equal(vc[:, lens[b]:].transpose(0, 1), v[src].double())
            assert torch.equal(kc[:, :lens[b]], before[b][0])
    # the framework's decode steps go on from there
    lens = kv.seq_lens.cpu().tolist()
    c.k.nan_to_num_(0.0), c.v.nan_to_num_(0.0)
    dec = S.SparseDecoder(kv, N=4096, w=0)
    q = torch.randn(B, Hq, d, device="cuda", dtype=dtype)
    dec.step(q)
    one = S.TokenBatch(kv, rope, max_tokens=B, max_new=1, **pages)
    assert S.last_error() == 0
    for b in range(B):
        kc, vc = [x.repeat_interleave(Hq // Hkv, 0) for x in c.rows(b, lens[b])]
        s = (q[b].double()[:, None] @ kc.transpose(1, 2))[:, 0] * d ** -0.5
        w = torch.softmax(s, -1)
        assert (dec.out[b].double() - (w[:, None] @ vc)[:, 0]).abs().max().item() <= 2e-3
    assert one.out.shape == (B, Hq, d)


def test_two_streams_with_their_own_workspaces():
    import sparse_kv_selection_gb300 as S
    rng = np.random.default_rng(5)
    jobs = []
    for seed in (1, 2):
        c = Cache([3000, 1700], 8, 2, 128, BF16, page=16, seed=seed)
        n = [12, 30]
        q, k, v = tree_inputs(c, n, 0, seed)
        mask = torch.tensor(words_of(random_sets(rng, n), 42), device="cuda")
        out, lse = torch.empty_like(q), torch.empty(42, 8, device="cuda")
        ws = S.make_tree_workspace(c.kv, 30)
        args = (c.kv, q, k, v, 128 ** -0.5, i32([0, 12, 42]), 30)
        S.tree_attn(*args, out, lse, ws, tree_mask=mask)
        jobs.append((args, mask, out, lse, ws, torch.empty_like(out), torch.empty_like(lse), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, mask, out, lse, ws, o2, l2, st in jobs:
            S.tree_attn(*args, o2, l2, ws, tree_mask=mask, stream=st)
    torch.cuda.synchronize()
    assert S.last_error() == 0
    for args, mask, out, lse, ws, o2, l2, st in jobs:
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("Hq,Hkv,n,page", [(32, 32, [16], 0), (32, 8, [64, 3], 0), (8, 8, [30, 1, 9, 17], 16),
                                           (32, 4, [300, 70], 64)])
def test_results_repeat_from_a_cold_cache(Hq, Hkv, n, page):
    """Loads that arrive late and out of step change nothing: every call from a
    flushed L2 gives the same bits."""
    import sparse_kv_selection_gb300 as S
    lens = [4096, 2500, 7000, 130][:len(n)]
    c = Cache(lens, Hq, Hkv, 128, BF16, page=page, room=1, seed=7)
    q, k, v = tree_inputs(c, n, 0, 3)
    cu = i32(np.concatenate([[0], np.cumsum(n)]))
    ws = S.make_tree_workspace(c.kv, max(n))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for call in range(12):
        out, lse = torch.empty_like(q), torch.empty(sum(n), Hq, device="cuda")
        flush.fill_(call)
        S.tree_attn(c.kv, q, k, v, 128 ** -0.5, cu, max(n), out, lse, ws)
        if first is None:
            first = (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), call
    assert S.last_error() == 0


def test_two_graphs_share_a_workspace():
    import sparse_kv_selection_gb300 as S
    jobs = []
    ws = None
    s = torch.cuda.Stream()
    for seed, n in ((1, [12, 40]), (2, [3, 5])):
        c = Cache([2100, 900], 8, 2, 128, BF16, seed=seed)
        q, k, v = tree_inputs(c, n, 0, seed)
        args = (c.kv, q, k, v, 128 ** -0.5, i32(np.concatenate([[0], np.cumsum(n)])), 40)
        ws = S.make_tree_workspace(c.kv, 40) if ws is None else ws
        out, lse = torch.empty_like(q), torch.empty(sum(n), 8, device="cuda")
        S.tree_attn(*args, out, lse, ws)
        torch.cuda.synchronize()
        want = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.tree_attn(*args, out, lse, ws)
        jobs.append((g, args, out, lse, want))
    for _ in range(5):
        for g, args, out, lse, want in jobs:
            out.zero_()
            g.replay()
            assert torch.equal(out, want)
    assert S.last_error() == 0
    del s


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F32, 64), (BF16, 128)])
def test_many_short_sequences(dtype, d):
    """More sequences than a CTA has threads, some without tokens or cache."""
    rng = np.random.default_rng(3)
    B = 1100
    lens, n = rng.integers(0, 40, B).tolist(), rng.integers(0, 4, B).tolist()
    lens[5], n[5], lens[700], n[700] = 900, 120, 300, 0
    c = Cache(lens, 4, 2, d, dtype, page=16, room=1, seed=1)
    import sparse_kv_selection_gb300 as S
    q, k, v = tree_inputs(c, n, 0, 2)
    cu = np.concatenate([[0], np.cumsum(n)])
    out, lse = torch.empty_like(q), torch.empty(sum(n), 4, device="cuda")
    S.tree_attn(c.kv, q, k, v, d ** -0.5, i32(cu), 120, out, lse, S.make_tree_workspace(c.kv, 120))
    assert S.last_error() == 0
    for b in [0, 1, 5, 6, 383, 384, 385, 699, 701, 767, 768, B - 1] + rng.integers(0, B, 40).tolist():
        if n[b] == 0:
            continue
        r = slice(int(cu[b]), int(cu[b + 1]))
        kc, vc = c.rows(b, lens[b])
        see = torch.ones(n[b], n[b], dtype=torch.bool, device="cuda").tril()
        wo, wl, eo, el = attn_ref(q[r].double(), kc, vc, k[r].double(), v[r].double(), see, d ** -0.5, d, dtype)
        assert ((out[r].double() - wo).abs() <= eo).all() and ((lse[r].double() - wl).abs() <= el).all(), b


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2)])
def test_one_token_is_dense_attention_after_append(dtype, Hq, Hkv):
    """The form of plain decode, against the library's own append and dense attention."""
    import sparse_kv_selection_gb300 as S
    c = Cache([40, 0, 333], Hq, Hkv, 128, dtype, t_max=400, seed=5)
    q, k, v = tree_inputs(c, [1, 1, 1], 0, 2)
    out, lse = torch.empty_like(q), torch.empty(3, Hq, device="cuda")
    S.tree_attn(c.kv, q, k, v, 128 ** -0.5, i32([0, 1, 2, 3]), 1, out, lse, S.make_tree_workspace(c.kv, 1))
    S.binding.append_kv(c.kv, k.contiguous(), v.contiguous())
    o2, l2 = torch.empty(3, Hq, 128, device="cuda"), torch.empty(3, Hq, device="cuda")
    S.dense_attn(c.kv, q, 128 ** -0.5, o2, l2, S.make_workspace(c.kv))
    assert S.last_error() == 0
    tol = 2.0 ** -7 if dtype == BF16 else 2.0 ** -16     # weights and result in bf16: 2 * 2^-8 of |v|'s mean
    assert ((out.float() - o2).abs() <= tol * (1 + o2.abs())).all() and ((lse - l2).abs() <= 2.0 ** -15).all()


def test_batches_without_tokens():
    import sparse_kv_selection_gb300 as S
    c = Cache([5, 0], 4, 2, 64, BF16, page=16, room=4, seed=1)
    got, bits = run_plan(c, [0, 0], 0, parents=[])
    assert bits == 0 and got[0].tolist() == [0, 0, 0]
    got, bits = run_plan(c, [0, 0], 3)
    assert bits == 0 and got[2].tolist() == [-1, -1, -1] and got[5] == 0 and got[6] == c.n_pages
    for T in (0, 3):
        q, k = torch.full((T, 4, 64), 2.0, device="cuda", dtype=BF16), torch.zeros(T, 2, 64, device="cuda", dtype=BF16)
        out, lse = torch.full_like(q, 3.0), torch.full((T, 4), 3.0, device="cuda")
        S.tree_attn(c.kv, q, k, k, 0.125, i32([0, 0, 0]), 7, out, lse, S.make_tree_workspace(c.kv, 7))
        S.rope_append(c.kv, S.RopeTable(64), i32([0] * T), q, k, k, out, slots=i32([-1] * T))
        assert (out == 3.0).all() and (lse == 3.0).all()
    new = i32([9, 9])
    S.commit_tokens(c.kv, i32([0, 0, 0]), i32([0, 0]), new)
    assert S.last_error() == 0 and new.tolist() == [5, 0]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [0, 128])
def test_long_cache_of_few_heads(dtype, page):
    """Many tiles a CTA, whole boxes of 128 rows, windows of 32 boxes crossed."""
    c = Cache([70000], 2, 1, 128, dtype, page=page, room=1, seed=4)
    check_tree(c, [5], seed=2)
    c = Cache([33000, 9000], 8, 1, 128, dtype, page=page, room=1, seed=4)
    check_tree(c, [40, 2], seed=2)


def test_tensors_of_another_kind_are_refused():
    import sparse_kv_selection_gb300 as S
    c = Cache([50], 4, 2, 64, BF16, seed=1)
    q, k, v = tree_inputs(c, [3], 0, 1)
    out, lse, ws = torch.empty_like(q), torch.empty(3, 4, device="cuda"), S.make_tree_workspace(c.kv, 3)
    cu = i32([0, 3])
    bad = [(q.float(), k, v, cu, out, lse, ws), (q, k.cpu(), v, cu, out, lse, ws), (q, k, v[:2], cu, out, lse, ws),
           (q, k, v, cu.long(), out, lse, ws), (q, k, v, cu[:1], out, lse, ws), (q, k, v, cu, out.float(), lse, ws),
           (q, k, v, cu, out, lse[:, :2], ws), (q, k, v, cu, out, lse, ws.cpu())]
    for q_, k_, v_, cu_, out_, lse_, ws_ in bad:
        with pytest.raises(ValueError):
            S.tree_attn(c.kv, q_, k_, v_, 0.1, cu_, 3, out_, lse_, ws_)
    with pytest.raises(S.PrhsError) as e:
        S.tree_attn(c.kv, q, k, v, 0.1, cu, 3, out, lse, ws[:1024])
    assert e.value.status == 3
    with pytest.raises(ValueError):
        S.tree_attn(c.kv, q, k, v, 0.1, cu, 3, out, lse, ws, tree_mask=torch.zeros(3, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        S.rope_append(c.kv, S.RopeTable(64, device="cpu"), i32([0] * 3), q, k, v, out)
    with pytest.raises(S.PrhsError):
        S.rope_append(c.kv, S.RopeTable(128), i32([0] * 3), q, k, v, out)     # rot_dim above d


@pytest.mark.parametrize("Hq,Hkv,n", [(2, 1, 3), (8, 1, 20), (4, 1, 64)])
def test_growing_maximum_in_every_row_tile(Hq, Hkv, n):
    """The maximum rises by about 13 (base 2) a tile of keys, above and below the
    rescaling threshold, with one and with two row tiles, masked new tokens last."""
    import sparse_kv_selection_gb300 as S
    t = 2000
    c = Cache([t], Hq, Hkv, 128, BF16, seed=3)
    ramp = torch.linspace(0, 140, t, device="cuda")[None, None, :, None]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    noise = torch.randn(1, Hkv, t, 128, generator=g, device="cuda") * 0.1
    c.k[:, :, :t] = (ramp / 128 ** 0.5 + noise).to(BF16)
    q = torch.ones(n, Hq, 128, device="cuda", dtype=BF16)
    k, v = torch.randn(2, n, Hkv, 128, generator=g, device="cuda").to(BF16)
    out, lse = torch.empty_like(q), torch.empty(n, Hq, device="cuda")
    S.tree_attn(c.kv, q, k, v, 128 ** -0.5, i32([0, n]), n, out, lse, S.make_tree_workspace(c.kv, n))
    assert S.last_error() == 0
    kc, vc = c.rows(0, t)
    see = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    wo, wl, eo, el = attn_ref(q.double(), kc, vc, k.double(), v.double(), see, 128 ** -0.5, 128, BF16)
    assert ((out.double() - wo).abs() <= eo).all() and ((lse.double() - wl).abs() <= el).all()


@pytest.mark.parametrize("seed", range(40))
def test_tree_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    Hq, Hkv = HEADS[rng.integers(len(HEADS))]
    Hq, Hkv = (Hq * 4, Hkv * 4) if rng.random() < 0.3 else (Hq, Hkv)
    dtype = BF16 if rng.random() < 0.75 else F32
    B = int(rng.integers(1, 9))
    tree = rng.random() < 0.6
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(6000), B))]
    n = [int(x) for x in np.exp(rng.uniform(0, np.log(129 if tree else 700), B))]
    for b in range(B):
        if rng.random() < 0.1:
            lens[b] = 0
        if rng.random() < 0.1 and B > 1:
            n[b] = 0
    n[0] = max(n[0], 1)
    c = Cache(lens, Hq, Hkv, int(rng.choice([64, 128])), dtype, page=int(rng.choice([0, 16, 32, 48, 64, 128, 256])),
              room=1, seed=seed)
    check_tree(c, n, pad=int(rng.integers(0, 20)), seed=seed, sets=random_sets(rng, n) if tree else None,
               stride_extra=int(rng.choice([0, 64])), scale=float(rng.uniform(0.02, 0.3)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n,tree", [(1, 1, [1], True), (8, 1, [1], True), (4, 1, [2, 2], True), (8, 1, [4], False),
                                           (2, 1, [9], True), (8, 1, [5, 9, 13], True), (8, 2, [17, 33], False),
                                           (8, 1, [128], True), (8, 1, [41, 25], False), (1, 1, [257], False)])
def test_fp32_forms_and_unit_shares(d, Hq, Hkv, n, tree):
    """Row counts on both sides of 8, 32 and 64 and of equal shares, over caches
    whose tiles are cut into more records than a join takes at once, and next to
    caches that hold less than a tile."""
    c = Cache([12000] + [40] * (len(n) - 1), Hq, Hkv, d, F32, page=16, room=1, seed=2)
    check_tree(c, n, seed=3, sets=random_sets(np.random.default_rng(7), n) if tree else None)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("max_new", [1, 2, 5, 40, 10 ** 6])
def test_workspace_of_more_tokens_than_the_batch_has(dtype, max_new):
    """max_new names the workspace; a batch of one token fits any of them exactly."""
    import sparse_kv_selection_gb300 as S
    c = Cache([3000], 8, 1, 128, dtype, seed=1)
    q, k, v = tree_inputs(c, [1], 0, 1)
    need = S.tree_workspace_size(c.kv, max_new)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:]
    out, lse = torch.empty_like(q), torch.empty(1, 8, device="cuda")
    S.tree_attn(c.kv, q, k, v, 0.1, i32([0, 1]), max_new, out, lse, ws[:need])
    assert S.last_error() == 0 and (ws[need:] == 0xA5).all()
    want, wl = torch.empty_like(q), torch.empty(1, 8, device="cuda")
    S.tree_attn(c.kv, q, k, v, 0.1, i32([0, 1]), 1, want, wl, S.make_tree_workspace(c.kv, 1))
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("seed", range(40))
def test_tree_random_short_caches(seed):
    """Units of a few tiles, which are shared out whole, on batches from one unit
    to many a CTA, with sequences without tokens between them."""
    rng = np.random.default_rng(2000 + seed)
    Hq, Hkv = HEADS[rng.integers(len(HEADS))]
    m = int(rng.choice([1, 2, 4]))
    B = int(np.exp(rng.uniform(0, np.log(40))))
    tree = rng.random() < 0.5
    top = int(rng.choice([1, 100, 400, 1200]))
    lens = [int(rng.integers(0, top + 1)) for _ in range(B)]
    n = [0 if rng.random() < 0.2 else int(np.exp(rng.uniform(0, np.log(129 if tree else 260)))) for _ in range(B)]
    n[int(rng.integers(B))] = 1
    c = Cache(lens, Hq * m, Hkv * m, int(rng.choice([64, 128])), BF16 if rng.random() < 0.8 else F32,
              page=int(rng.choice([0, 16, 64])), room=1, seed=seed)
    check_tree(c, n, pad=int(rng.integers(0, 5)), seed=seed, sets=random_sets(rng, n) if tree else None)


@pytest.mark.parametrize("B,Hq,Hkv,d,t,n,page", [(40, 32, 32, 64, 1600, 1, 16), (2, 64, 16, 128, 21000, 16, 0),
                                                 (24, 32, 32, 64, 2100, 6, 64)])
def test_fp32_sums_in_blocks(B, Hq, Hkv, d, t, n, page):
    """Runs of many tiles in one CTA, whose sums are folded on the way: in units
    that end there, begin there and pass through."""
    c = Cache([t] * B, Hq, Hkv, d, F32, page=page, room=1, seed=6)
    check_tree(c, [n] * B, seed=5, sets=random_sets(np.random.default_rng(3), [n] * B))
