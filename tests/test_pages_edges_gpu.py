"""Forks and compactions of which some arrays are updated in place and others are not, on long
pages and wide tables; refused ones too."""
import numpy as np
import pytest

from pages_util import compact_ref, fork_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_pages_gpu import Device, i32, make_state, random_keep, random_parents  # noqa: E402

ARRAYS = ("table", "lens", "n_pages", "page_shares", "free_pages", "free_head")


@pytest.mark.parametrize("what", ["fork_seqs", "compact_seqs"])
@pytest.mark.parametrize("page,wide", [(16, 0), (512, 0), (16, 3000)])
@pytest.mark.parametrize("refused", [False, True])
def test_some_arrays_in_place(what, page, wide, refused):
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_CAPACITY
    rng = np.random.default_rng(page + wide)
    s = make_state(rng, 6, (1, 6), (0, 40 * page), (1, 3 * page), page, spare=0 if refused else None)
    s.table = np.concatenate([s.table, np.full((len(s.lens), wide), -1)], 1)
    B = len(s.lens)
    if what == "fork_seqs":
        args = [random_parents(rng, B, 0.3, 0.1)]
        if refused:
            args = [[int(np.argmax(s.lens % page > 0))] * B]
        ref, cap = fork_ref(s, *args), page
    else:
        args = list(random_keep(rng, s, 0.5))
        ref, cap = compact_ref(s, *args), args[0].shape[1]
    assert (ref is None) == refused
    after, src, dst = ref if ref is not None else (s, -1, -1)
    new = dict(zip(ARRAYS, (after.table, after.lens, after.n_pages, after.shares, after.free, [after.head])))
    old = dict(zip(ARRAYS, (s.table, s.lens, s.n_pages, s.shares, s.free, [s.head])))
    for apart in [{x} for x in ARRAYS] + [set(ARRAYS) - {x} for x in ARRAYS]:
        d = Device(s)
        here = dict(table=d.kv.block_table, lens=d.kv.seq_lens, **d.pages)
        out = {x + "_out": torch.full_like(here[x], -9) for x in apart}
        lists = [torch.full((B, cap), -9, dtype=torch.int32, device="cuda") for _ in range(2)]
        getattr(S, what)(d.kv, *[i32(a) for a in args], *lists, d.ws, **d.pages, **out)
        assert S.last_error() == (DEV_CAPACITY if refused else 0)
        for x in ARRAYS:
            got = out[x + "_out"] if x in apart else here[x]
            assert np.array_equal(got.cpu().numpy(), new[x]), (x, apart)
            if x in apart:
                assert np.array_equal(here[x].cpu().numpy(), old[x]), (x, apart)
        assert (lists[0].cpu().numpy() == src).all() and (lists[1].cpu().numpy() == dst).all()
