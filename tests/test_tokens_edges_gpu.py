"""Token batches at the edges of their contract: sequences that planning refused,
page state that batches share, NaN, angles near quarter turns, long runs of key
tiles."""
import numpy as np
import pytest

from tokens_util import Cache, attn_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


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


