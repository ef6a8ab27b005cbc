"""The gate with few heads and long anchor sets (a cluster of CTAs a head) under a bound on
consecutive reuses, many steps: one decision for all CTAs of a head at each."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,max_run", [(4096, 1), (4096, 2), (4096, 3), (8192, 4), (512, 3)])
def test_bounded_runs_by_clusters(dtype, N, max_run):
    import sparse_kv_selection_gb300 as S
    B, H, t, d = 2, 2, 20000, 64
    g = torch.Generator(device="cuda").manual_seed(N + max_run)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    kv = S.KVCache(mk(B, H, t, d), mk(B, H, t, d), torch.tensor([t, t - 7], dtype=torch.int32, device="cuda"), H)
    dec = S.SparseDecoder(kv, N=N, w=1, tau=-1.0, max_run=max_run)
    q = mk(B, H, d)
    first = dilated = None
    for step in range(60):
        dec.step(q)
        reuse = dec.reuse.bool()
        sets = [dec.idx[b, h, :int(dec.n_sel[b, h])].clone() for b in range(B) for h in range(H)]
        if step % max_run == 0:                       # a new anchor, then max_run - 1 reuses of it
            assert not reuse.any(), step
            first = first or sets
            assert all(torch.equal(x, y) for x, y in zip(first, sets))
            assert all(len(x) == N for x in sets)
        else:
            assert reuse.all(), step
            if dilated is None:
                dilated = sets
                for x, y, n in zip(first, sets, [t] * H + [t - 7] * H):
                    near = torch.zeros(n + 2, dtype=torch.bool, device="cuda")
                    for s in (0, 1, 2):
                        near[x.long() + s] = True
                    assert torch.equal(torch.nonzero(near[1:-1]).flatten().int(), y)
            assert all(torch.equal(x, y) for x, y in zip(dilated, sets))
        assert (dec.anchor_age == step % max_run).all()
    assert S.last_error() == 0
