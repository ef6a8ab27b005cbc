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
