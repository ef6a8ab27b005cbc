"""PagePool: layers that do not fit, buffers of calls of many widths, arguments that are refused;
row copies of many KV heads."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def caches(num_blocks=(64, 64)):
    import sparse_kv_selection_gb300 as S
    table, lens = i32(np.arange(32).reshape(4, 8)), i32([100, 40, 0, 128])
    mk = lambda n: torch.randn(n, 1, 16, 64, device="cuda")  # noqa: E731
    return [S.KVCache(mk(n), mk(n), lens, 1, block_table=table) for n in num_blocks], table, lens


def pool_args():
    return dict(free_pages=i32(np.arange(64)), free_head=i32([32]), n_pages=i32([8, 8, 8, 8]))


def test_layers_that_do_not_fit_are_refused():
    """A layer on other lengths, rows or a pool of another size would be left behind by a fork."""
    import sparse_kv_selection_gb300 as S
    (kv, same), table, lens = caches()
    larger = torch.zeros(80, 1, 16, 64, device="cuda")
    S.PagePool(kv, layers=[same, S.KVCache(larger, larger, lens, 1, block_table=table)], **pool_args())
    k = torch.zeros(64, 1, 16, 64, device="cuda")
    for bad in (S.KVCache(k, k, lens.clone(), 1, block_table=table),                    # lengths of its own
                S.KVCache(k[:40], k[:40], lens, 1, block_table=table),                  # fewer pages
                S.KVCache(k, k, lens[:2], 1, block_table=table[:2])):                   # fewer rows
        with pytest.raises(ValueError):
            S.PagePool(kv, layers=[bad], **pool_args())


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_row_lists_of_many_widths(order):
    """Calls of many widths keep less than four times what the widest needs: buffers double, so the
    last is below twice that, and those before it are no more together."""
    import sparse_kv_selection_gb300 as S
    (kv, _), _, lens = caches()
    pool = S.PagePool(kv, **pool_args())
    nothing = i32([-1] * 4)
    widest = 20000
    widths = [w for w in range(1, widest, 37)] + [widest]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for w in widths if order == "rising" else widths[::-1]:
        pool.compact(torch.zeros(4, w, dtype=torch.int32, device="cuda"), nothing)
    torch.cuda.synchronize()
    assert S.last_error() == 0
    assert torch.cuda.memory_allocated() - before <= 4 * (2 * 4 * widest * 4) + (1 << 16)


def test_row_lists_of_a_graph_outlive_wider_calls():
    import sparse_kv_selection_gb300 as S
    (kv, _), table, lens = caches()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        pool = S.PagePool(kv, stream=stream, **pool_args())
        keep, n = torch.zeros(4, 24, dtype=torch.int32, device="cuda"), i32([-1] * 4)
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            pool.compact(keep, n)
        wide = torch.zeros(4, 5000, dtype=torch.int32, device="cuda")
        pool.compact(wide, n)
        junk = [torch.full((4, 24), 7, dtype=torch.int32, device="cuda") for _ in range(64)]
        want = kv.k[table[0, torch.arange(90, 100, device="cuda") // 16].long(), 0, torch.arange(90, 100, device="cuda") % 16].clone()
        keep[0, :10] = torch.arange(90, 100, device="cuda")
        n.copy_(i32([10, -1, -1, -1]))
        g.replay()
        pool.compact(wide, i32([-1] * 4))
        stream.synchronize()
        assert S.last_error() == 0
        assert lens.tolist() == [10, 40, 0, 128]
        assert torch.equal(kv.k[int(table[0, 0]), 0, :10], want)
        assert all((x == 7).all() for x in junk)


def test_free_takes_one_flag_a_row():
    import sparse_kv_selection_gb300 as S
    (kv, _), _, lens = caches()
    pool = S.PagePool(kv, **pool_args())
    for bad in (torch.tensor([True], device="cuda"), torch.tensor(True, device="cuda"), i32([1, 0, 0, 0]),
                torch.tensor([[True, False, False, False]], device="cuda"), torch.tensor([True, False, False, False])):
        with pytest.raises(ValueError):
            pool.free(bad)
    assert lens.tolist() == [100, 40, 0, 128]
    pool.free(torch.tensor([True, False, False, False], device="cuda"))
    assert S.last_error() == 0 and lens.tolist() == [0, 40, 0, 128]
    pool.free(torch.tensor([[False, True], [True, False]] * 2, device="cuda")[:, 0])    # (any stride)
    assert S.last_error() == 0 and lens.tolist() == [0, 0, 0, 0]
