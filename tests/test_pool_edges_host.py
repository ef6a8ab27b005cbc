"""Sizes that the operators for sequences that share pages count in 32 bits: larger ones are
refused before anything is done, not cut to 32 bits on the way."""
import ctypes
import types

import pytest

torch = pytest.importorskip("torch")

from test_abi import lib  # noqa: E402,F401
from test_pages_host import compact, pages, paged  # noqa: E402

META = torch.device("meta")


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device=META)


def fake(b, B=4, **over):
    """A cache of which only what the binding looks at is there."""
    d = paged(b, B=B, **over)
    return types.SimpleNamespace(desc=d, ref=lambda: ctypes.byref(d), device=META, dtype=torch.bfloat16, index=0, B=B, Hq=d.Hq,
                                 k=torch.zeros(1, dtype=torch.bfloat16, device=META), block_table=i32(B, d.max_blocks),
                                 seq_lens=i32(B))


@pytest.mark.parametrize("cap", [(1 << 30) + 1, (1 << 31) - 1])
def test_compaction_of_wider_rows_than_a_cache_has(lib, cap):  # noqa: F811
    from sparse_kv_selection_gb300 import binding as b
    assert compact(lib, b, paged(b), pages(b), pages(b), cap=cap) == b.PRHS_EUNSUPPORTED


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 5])
def test_copies_of_more_rows_than_32_bits_count(lib, n):  # noqa: F811
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300 import binding as b
    with pytest.raises(ValueError, match="rows"):
        S.copy_rows(fake(b), i32(n), i32(n))


def test_a_pools_calls_of_more_rows_than_a_copy_takes(lib):  # noqa: F811
    """Refused before the table changes, not when the rows are to be copied."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300 import binding as b
    pool = S.PagePool(fake(b, B=4096), free_pages=i32(64), n_pages=i32(4096))
    with pytest.raises(ValueError, match="rows"):
        pool.compact(i32(4096, 1 << 19), i32(4096))


@pytest.mark.parametrize("least", [1 << 32, (1 << 32) + 16, 1 << 31, -1])
def test_shortest_prefixes_outside_32_bits(lib, least):  # noqa: F811
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300 import binding as b
    kv = fake(b)
    if least >= 0:
        with pytest.raises(ValueError, match="min_keys"):
            S.find_shared(kv, i32(5), i32(4, 4), min_keys=least)
    with pytest.raises(ValueError, match="min_shared"):
        S.TokenBatch(kv, None, max_tokens=4, max_new=1, share_prefixes=True, min_shared=least, free_pages=i32(4), n_pages=i32(4))


@pytest.mark.parametrize("most", [1 << 32, (1 << 32) + 1, 1 << 31])
def test_token_counts_outside_32_bits(lib, most):  # noqa: F811
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300 import binding as b
    kv = fake(b)
    rows = torch.zeros(4, kv.Hq, 128, dtype=torch.bfloat16, device=META)
    out, lse = torch.zeros_like(rows), torch.zeros(4, kv.Hq, device=META)
    with pytest.raises(ValueError, match="max_new"):
        S.shared_attn(kv, rows, rows, rows, 0.1, i32(5), most, i32(4, 4), out, lse, torch.zeros(8, dtype=torch.uint8, device=META))
    with pytest.raises(ValueError, match="max_new"):
        S.tree_attn(kv, rows, rows, rows, 0.1, i32(5), most, out, lse, torch.zeros(8, dtype=torch.uint8, device=META))
