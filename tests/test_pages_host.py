"""Refusals of the operators for sequences that share pages, on the host."""
import ctypes

import pytest

from test_abi import _kv, lib  # noqa: F401


def paged(b, **over):
    return _kv(b, **{**dict(block_table=512, block_size=16, max_blocks=8, num_blocks=64), **over})


def pages(b, **over):
    a = dict(block_table=None, seq_lens=None, n_pages=64, page_shares=64, free_pages=64, n_free=4, free_head=64)
    return b.prhs_pages(*{**a, **over}.values())


WS, BYTES = 1 << 20, 1 << 40


def fork(lib, b, kv, now, nxt, parent=64, src=64, dst=64, ws=WS, size=BYTES):  # noqa: F811
    by = [None if x is None else ctypes.byref(x) for x in (kv, now, nxt)]
    return lib.prhs_fork_seqs(by[0], by[1], parent, by[2], src, dst, ws, size, None)


def compact(lib, b, kv, now, nxt, keep=64, cap=8, keep_n=64, src=64, dst=64, ws=WS, size=BYTES):  # noqa: F811
    by = [None if x is None else ctypes.byref(x) for x in (kv, now, nxt)]
    return lib.prhs_compact_seqs(by[0], by[1], keep, cap, keep_n, by[2], src, dst, ws, size, None)


@pytest.mark.parametrize("call", [fork, compact])
def test_pages_refusals(lib, call):  # noqa: F811
    from sparse_kv_selection_gb300 import binding as b
    kv = paged(b)
    for over in (dict(n_pages=None), dict(page_shares=None), dict(free_head=None), dict(free_pages=None), dict(n_free=-1),
                 dict(n_free=5), dict(block_table=1024), dict(seq_lens=1024)):
        assert call(lib, b, kv, pages(b, **over), pages(b)) == b.PRHS_EINVAL, over
        assert lib.prhs_last_message().decode() != ""
    for over in (dict(n_pages=None), dict(page_shares=None), dict(free_head=None), dict(free_pages=None), dict(n_free=3)):
        assert call(lib, b, kv, pages(b), pages(b, **over)) == b.PRHS_EINVAL, over
    for over in (dict(src=None), dict(dst=None), dict(src=66), dict(dst=66)):
        assert call(lib, b, kv, pages(b), pages(b), **over) == b.PRHS_EINVAL, over
    assert call(lib, b, None, pages(b), pages(b)) == b.PRHS_EINVAL
    assert call(lib, b, kv, None, pages(b)) == b.PRHS_EINVAL
    assert call(lib, b, kv, pages(b), None) == b.PRHS_EINVAL
    assert call(lib, b, _kv(b), pages(b), pages(b)) == b.PRHS_EINVAL            # contiguous cache
    assert call(lib, b, paged(b, max_blocks=1 << 24, B=64, Hq=1, Hkv=1, block_size=32), pages(b), pages(b)) == b.PRHS_EUNSUPPORTED
    if call is fork:
        assert call(lib, b, kv, pages(b), pages(b), parent=None) == b.PRHS_EINVAL
    else:
        for over in (dict(keep=None), dict(keep_n=None), dict(cap=0), dict(cap=-4)):
            assert call(lib, b, kv, pages(b), pages(b), **over) == b.PRHS_EINVAL, over


def test_pages_workspace(lib):  # noqa: F811
    from sparse_kv_selection_gb300 import binding as b
    need = lib.prhs_pages_workspace_size(ctypes.byref(paged(b)))
    assert need > 0 and need % 256 == 0
    assert lib.prhs_pages_workspace_size(ctypes.byref(_kv(b))) == 0
    assert lib.prhs_pages_workspace_size(ctypes.byref(paged(b, d=96))) == 0


@pytest.mark.parametrize("over", [dict(n=-1), dict(src=None), dict(dst=None)])
def test_copy_rows_refusals(lib, over):  # noqa: F811
    from sparse_kv_selection_gb300 import binding as b
    a = {**dict(n=4, src=64, dst=64), **over}
    assert lib.prhs_copy_rows(ctypes.byref(_kv(b)), None, *a.values(), None) == b.PRHS_EINVAL
    for bad in (dict(dtype=b.PRHS_F32), dict(d=64), dict(Hkv=2), dict(k=None)):
        assert lib.prhs_copy_rows(ctypes.byref(_kv(b)), ctypes.byref(_kv(b, **bad)), 4, 64, 64, None) == b.PRHS_EINVAL
    assert lib.prhs_copy_rows(None, None, 4, 64, 64, None) == b.PRHS_EINVAL


@pytest.mark.parametrize("over", [dict(cu=None), dict(min_keys=-1), dict(shared=None), dict(shared=72)])
def test_find_shared_refusals(lib, over):  # noqa: F811
    from sparse_kv_selection_gb300 import binding as b
    a = {**dict(cu=64, min_keys=16, shared=64), **over}
    assert lib.prhs_find_shared(ctypes.byref(paged(b)), *a.values(), None) == b.PRHS_EINVAL
    assert lib.prhs_last_message().decode() != ""


SHARED = dict(q=64, k=64, ks=512, v=64, vs=512, scale=0.1, T=4, cu=64, max_new=4, mask=None, shared=64, out=64, lse=64,
              ws=256, bytes=1 << 40)


@pytest.mark.parametrize("over", [dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(shared=None), dict(out=None),
                                  dict(lse=None), dict(q=72), dict(k=72), dict(v=72), dict(out=72), dict(mask=72),
                                  dict(shared=72), dict(ks=510), dict(vs=100), dict(T=-1), dict(max_new=0),
                                  dict(max_new=129, mask=64)])
def test_shared_attn_refusals(lib, over):  # noqa: F811
    from sparse_kv_selection_gb300 import binding as b
    a = {**SHARED, **over}
    assert lib.prhs_shared_attn(ctypes.byref(_kv(b)), *a.values(), None) == b.PRHS_EINVAL
    assert lib.prhs_last_message().decode() != ""
    assert lib.prhs_shared_workspace_size(ctypes.byref(_kv(b)), 0, 4) == 0
    assert lib.prhs_shared_workspace_size(ctypes.byref(_kv(b)), 4, 0) == 0
    assert lib.prhs_shared_workspace_size(ctypes.byref(_kv(b, d=96)), 4, 4) == 0
