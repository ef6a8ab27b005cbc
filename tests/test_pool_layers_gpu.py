"""A model of several layers on one pool: every layer's batch plans for itself (pages that the
first one took are there for the others) and one commit moves the lengths."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_pool_gpu import BF16, F32, Twin, i32  # noqa: E402
from tokens_util import ancestors, attn_ref  # noqa: E402


class Model(Twin):
    def feed(self, n, check=True, trees=None, accept=None):
        """Chunks, or trees of which accept[b] (numbers) join the cache."""
        import sparse_kv_selection_gb300 as S
        T = 64
        cu = np.concatenate([[0], np.cumsum(n)])
        parents = None
        if trees is not None:
            parents = np.full(T, -1)
            parents[:cu[-1]] = sum(trees, [])
            parents = i32(parents)
        heads, slots = [], []
        for layer, step in enumerate(self.steps):
            mk = lambda h: torch.randn(T, h, self.d, generator=self.g, device="cuda").to(self.dtype)  # noqa: E731
            q, k, v = mk(self.Hq), mk(self.Hkv), mk(self.Hkv)
            step.plan(i32(n), parents)
            heads.append(int(self.pool.pages["free_head"]))
            slots.append(step.slots.clone())
            step.rotate(q, k, v, append=trees is None)
            step.attend()
            assert S.last_error() == 0
            for b in range(self.B):
                if n[b] == 0:
                    continue
                at = slice(int(cu[b]), int(cu[b + 1]))
                kc, vc = self.rows[b][layer]
                see = torch.tril(torch.ones(n[b], n[b], dtype=torch.bool, device="cuda"))
                if trees is not None:
                    see[:] = False
                    for j, s in enumerate(ancestors(trees[b])):
                        see[j, list(s)] = True
                want, lse, e_out, e_lse = attn_ref(step.q[at].double(), kc.double().transpose(0, 1), vc.double().transpose(0, 1),
                                                   step.k[at].double(), v[at].double(), see, self.d ** -0.5, self.d, self.dtype)
                assert ((step.out[at].double() - want).abs() <= e_out).all(), (b, layer)
                assert ((step.lse[at].double() - lse).abs() <= e_lse).all(), (b, layer)
                pick = torch.tensor(accept[b] if accept is not None else range(n[b]), dtype=torch.long, device="cuda")
                self.rows[b][layer] = [torch.cat([kc, step.k[at][pick]]), torch.cat([vc, v[at][pick]])]
        assert heads[0] == heads[1] and torch.equal(*slots)
        last = self.steps[-1]
        if trees is None:                           # the rows are in the caches: the lengths alone
            last.commit(i32(n))
        else:
            m, idx = [len(x) for x in accept], np.zeros((self.B, max(n)), int)
            for b, x in enumerate(accept):
                idx[b, :len(x)] = x
            first, scratch = self.steps[0], torch.empty_like(self.kv[0].seq_lens)
            S.commit_tokens(first.kv, first.cu_new, i32(m), scratch, slots=first.slots, accept_idx=i32(idx), k_new=first.k,
                            v_new=first.v)
            last.commit(i32(m), i32(idx))
        assert S.last_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layers_of_a_model(dtype):
    rng = np.random.default_rng(7)
    m = Model(6, 4, 2, 64, dtype)
    for _ in range(3):
        m.feed([37, 0, 0, 0, 21, 0])
    m.check()
    m.fork([0, 0, 0, 0, 4, 4])
    for _ in range(18):
        m.feed([1] * 6)
    m.check()
    for _ in range(4):
        n = [int(x) for x in rng.integers(1, 8, 6)]
        trees = [[int(max(-1, j - 1 - rng.integers(0, 3))) for j in range(x)] for x in n]
        accept = []
        for t in trees:                             # a path from a root
            j, path = int(rng.integers(0, len(t))), []
            while j >= 0:
                path.append(j)
                j = t[j]
            accept.append(path[::-1])
        m.feed(n, trees=trees, accept=accept)
        m.check()
        m.fork([int(x) for x in np.concatenate([rng.integers(0, 4, 4), rng.integers(4, 6, 2)])])
    m.check()
    m.fork([-1] * 6)
    assert m.check().head == 0
