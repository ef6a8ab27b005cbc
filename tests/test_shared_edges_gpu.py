"""Entries of shared_attn that differ within a group."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_shared_gpu import BF16, F32, Batch  # noqa: E402


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("entry", [[0, 4, 32, 0], [0, 4, 48, 0], [0, 4, 80, 0], [0, 3, 64, 0], [0, 5, 64, 0]])
def test_an_entry_that_differs_from_its_groups_is_flagged(dtype, entry):
    """Row 2 shares two pages with its group, not the four that the first row's entry names; its
    own entry differs from the first row's, so it is flagged and attends all its own keys."""
    import sparse_kv_selection_gb300 as S
    from sparse_kv_selection_gb300.binding import DEV_BAD_INDEX
    b = Batch([(4, 64), (2, 32)], (16, 60), (1, 2), 4, 2, 64, dtype, 16, seed=50)
    b.c.kv.block_table[2, 2:4] = torch.tensor(b.c.table[2, 2:4], dtype=torch.int32, device="cuda")
    share = [list(x) for x in b.share]
    share[2] = entry
    out = b.run(share=share)
    assert S.last_error() == DEV_BAD_INDEX
    b.check(out)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_single_tokens_on_longer_own_keys_than_the_few_rows_part_takes(Hq, Hkv, d):
    """Own keys around and above 32768: tiles and runs of steps in one launch."""
    import sparse_kv_selection_gb300 as S
    b = Batch([(3, 64), (2, 160), (1, 0)], [32760, 32767, 32768, 40000, 10, 33000], (1, 1), Hq, Hkv, d, BF16, 16, seed=51)
    out = b.run()
    assert S.last_error() == 0
    b.check(out)
