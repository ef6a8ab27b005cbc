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


@pytest.mark.parametrize("dtype,Hkv,d", [(torch.float32, 16384, 128), (torch.bfloat16, 5000, 64), (torch.bfloat16, 16383, 128)])
def test_copies_of_rows_of_many_heads(dtype, Hkv, d):
    """An entry of up to 2^20 pieces, begun in the middle of a thread block's share."""
    import sparse_kv_selection_gb300 as S
    k, v = (torch.randn(3, Hkv, 16, d, device="cuda").to(dtype) for _ in range(2))
    kv = S.KVCache(k.clone(), v.clone(), i32([0]), Hkv, block_table=i32([[0, 1]]))
    src, dst = [0, 17, -1, 31, 40], [33, 2, 5, 47, 16]
    S.copy_rows(kv, i32(src), i32(dst))
    assert S.last_error() == 0
    for x, y in ((k, kv.k), (v, kv.v)):
        want = x.clone()
        for a, b in zip(src, dst):
            if a >= 0:
                want[b // 16, :, b % 16] = x[a // 16, :, a % 16]
        assert torch.equal(want, y)


FIRST = """
import torch
import sparse_kv_selection_gb300 as S
z = dict(dtype=torch.int32, device="cuda")
for dtype in (torch.bfloat16, torch.float32):
    for B, wide in ((4, 8), (64, 2000)):            # a cluster's table, and one for all SMs
        k, v = torch.randn(2, 300, 2, 16, 64, device="cuda").to(dtype)
        table = torch.full((B, wide), -1, **z)
        table[:2, :2] = torch.tensor([[0, 1], [2, 3]], **z)
        lens, held = torch.zeros(B, **z), torch.zeros(B, **z)
        lens[:2], held[:2] = torch.tensor([20, 32], **z), 2
        kv = S.KVCache(k, v, lens, 4, block_table=table)
        pool = S.PagePool(kv, free_pages=torch.arange(300, **z), free_head=torch.full((1,), 4, **z), n_pages=held)
        batch = S.TokenBatch(kv, S.RopeTable(64), max_tokens=9, max_new=6, share_prefixes=True, min_shared=16, **pool.pages)
        q, kn, vn = torch.randn(9, 4, 64, device="cuda").to(dtype), *torch.randn(2, 9, 2, 64, device="cuda").to(dtype)
        n, parent = torch.zeros(B, **z), torch.arange(B, **z)
        n[:4], parent[2:4] = torch.tensor([1, 2, 3, 1], **z), torch.tensor([0, 0], **z)
        keep, m = torch.arange(24, **z).repeat(B, 1), torch.full((B,), -1, **z)
        m[1] = 24
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pool.fork(parent)
            pool.compact(keep, m)
            batch.plan(n)
            batch.rotate(q, kn, vn)
            batch.attend()
            batch.commit(n)
        g.replay()
        assert S.last_error() == 0
        assert lens[:4].tolist() == [21, 26, 23, 21] and not lens[4:].any(), lens
        assert pool.page_shares[0] == 2 and torch.isfinite(batch.out[:7]).all()
"""


def test_a_process_whose_first_call_is_captured(tmp_path):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    script = tmp_path / "first.py"
    script.write_text(FIRST)
    r = subprocess.run([sys.executable, str(script)], cwd=root, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": root})
    assert r.returncode == 0, r.stdout + r.stderr
