"""Token-batch operators on the host: rotary frequencies and refusals."""
import ctypes
import math

import numpy as np
import pytest

from test_abi import _kv, lib  # noqa: F401
from tokens_util import theta_ref

KINDS = [("plain", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
         ("bands", dict(factor=8.0, original=8192.0, low=1.0, high=4.0)),
         ("ramp", dict(factor=16.0, original=4096.0, low=1.0, high=32.0)),
         ("ramp", dict(factor=4.0, original=32.0, low=1.0, high=32.0))]


@pytest.mark.parametrize("kind,kw", KINDS)
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 10000.0), (128, 500000.0)])
def test_rope_turns(lib, kind, kw, rot, base):  # noqa: F811
    from sparse_kv_selection_gb300 import binding
    turns, mscale = binding.rope_turns(rot, base, kind, **kw)
    theta, ms = theta_ref(rot, base, None if kind == "plain" else kind, **kw)
    assert len(turns) == rot // 2
    got = np.array([t / 2.0 ** 64 for t in turns]) * 2 * math.pi
    # float64 powers and quotients are off by a few units of 2^-53 of theta; cutting the
    # fraction after 64 bits takes up to 2^-64 turns off, whatever theta is
    assert (np.abs(got - theta) <= 2.0 ** -49 * theta + 2 * math.pi * 2.0 ** -64).all()
    assert abs(mscale - ms) <= 2.0 ** -23 * ms


@pytest.mark.parametrize("args", [
    (0, 8, 10000.0, 1.0, 0.0, 0.0, 0.0),          # rot_dim below 16
    (0, 24, 10000.0, 1.0, 0.0, 0.0, 0.0),         # not a multiple of 16
    (0, 64, 1.0, 1.0, 0.0, 0.0, 0.0),             # base
    (0, 64, float("nan"), 1.0, 0.0, 0.0, 0.0),
    (1, 64, 10000.0, 0.5, 0.0, 0.0, 0.0),         # factor below 1
    (1, 64, 10000.0, float("inf"), 0.0, 0.0, 0.0),
    (3, 64, 10000.0, 2.0, 0.0, 1.0, 4.0),         # no original context
    (3, 64, 10000.0, 2.0, 8192.0, 4.0, 4.0),      # high must exceed low
    (4, 64, 10000.0, 2.0, 8192.0, 0.0, 4.0),
    (5, 64, 10000.0, 2.0, 8192.0, 1.0, 4.0),      # unknown kind
    (-1, 64, 10000.0, 2.0, 8192.0, 1.0, 4.0),
])
def test_rope_turns_refusals(lib, args):  # noqa: F811
    out = (ctypes.c_uint64 * 64)()
    ms = ctypes.c_float()
    assert lib.prhs_rope_turns(*args, out, ctypes.byref(ms)) == 1
    assert lib.prhs_last_message().decode() != ""
    assert lib.prhs_rope_turns(0, 64, 10000.0, 1.0, 0.0, 0.0, 0.0, None, ctypes.byref(ms)) == 1


def paged(binding):
    return _kv(binding, block_table=512, block_size=16, max_blocks=8, num_blocks=64)


PLAN = dict(n_new=64, T=8, parents=None, free=64, n_free=4, head=64, pages=64, cu=64, pos=64, slots=64, mask=None,
            head_out=64, pages_out=64)


@pytest.mark.parametrize("over", [dict(n_new=None), dict(cu=None), dict(T=-1), dict(pos=None), dict(slots=None),
                                  dict(parents=64), dict(mask=64), dict(parents=64, mask=72), dict(head=None),
                                  dict(pages=None), dict(head_out=None), dict(pages_out=None), dict(n_free=-1),
                                  dict(free=None)])
def test_plan_refusals(lib, over):  # noqa: F811
    from sparse_kv_selection_gb300 import binding
    a = {**PLAN, **over}
    assert lib.prhs_plan_tokens(ctypes.byref(paged(binding)), *a.values(), None) == binding.PRHS_EINVAL
    assert lib.prhs_plan_tokens(None, *PLAN.values(), None) == binding.PRHS_EINVAL


ROPE = dict(T=4, pos=64, slots=64, q=64, qs=512, k=64, ks=512, v=64, vs=512, q_out=128, k_out=None)


@pytest.mark.parametrize("over", [dict(T=-1), dict(pos=None), dict(q=None), dict(k=None), dict(v=None), dict(q_out=None),
                                  dict(q=72), dict(k=72), dict(v=72), dict(q_out=72), dict(k_out=72), dict(qs=511),
                                  dict(qs=516), dict(ks=504), dict(vs=513), dict(qs=-512), dict(q=128, qs=1024),
                                  dict(k_out=64, ks=1024)])
def test_rope_append_refusals(lib, over):  # noqa: F811
    from sparse_kv_selection_gb300 import binding
    rope = binding.prhs_rope(128, 0, 64, 1.0)
    kv = _kv(binding)
    a = {**ROPE, **over}
    assert lib.prhs_rope_append(ctypes.byref(kv), ctypes.byref(rope), *a.values(), None) == binding.PRHS_EINVAL
    for bad in (binding.prhs_rope(120, 0, 64, 1.0), binding.prhs_rope(144, 0, 64, 1.0), binding.prhs_rope(0, 0, 64, 1.0),
                binding.prhs_rope(128, 0, None, 1.0), binding.prhs_rope(128, 0, 68, 1.0)):
        assert lib.prhs_rope_append(ctypes.byref(kv), ctypes.byref(bad), *ROPE.values(), None) == binding.PRHS_EINVAL
    assert lib.prhs_rope_append(ctypes.byref(kv), None, *ROPE.values(), None) == binding.PRHS_EINVAL
    huge = {**ROPE, "T": (1 << 31) - 1}
    assert lib.prhs_rope_append(ctypes.byref(kv), ctypes.byref(rope), *huge.values(), None) == binding.PRHS_EUNSUPPORTED


TREE = dict(q=64, k=64, ks=512, v=64, vs=512, scale=0.1, T=4, cu=64, max_new=4, mask=None, out=64, lse=64, ws=256,
            bytes=1 << 40)


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(cu=None), 1), (dict(out=None), 1), (dict(lse=None), 1),
    (dict(q=72), 1), (dict(k=72), 1), (dict(v=72), 1), (dict(out=72), 1), (dict(mask=72), 1), (dict(ks=510), 1),
    (dict(vs=100), 1), (dict(T=-1), 1), (dict(max_new=0), 1), (dict(max_new=129, mask=64), 1)])
def test_tree_attn_refusals(lib, over, status):  # noqa: F811
    from sparse_kv_selection_gb300 import binding
    a = {**TREE, **over}
    assert lib.prhs_tree_attn(ctypes.byref(_kv(binding)), *a.values(), None) == status
    assert lib.prhs_last_message().decode() != ""
    assert lib.prhs_tree_workspace_size(ctypes.byref(_kv(binding)), 0) == 0
    assert lib.prhs_tree_workspace_size(ctypes.byref(_kv(binding, d=96)), 4) == 0


COMMIT = dict(T=4, cu=64, idx=64, cap=4, n=64, k=64, ks=512, v=64, vs=512, lens=64)


@pytest.mark.parametrize("over", [dict(T=-1), dict(cu=None), dict(n=None), dict(lens=None), dict(cap=0), dict(k=None),
                                  dict(v=None), dict(k=72), dict(v=72), dict(ks=100), dict(vs=514)])
def test_commit_refusals(lib, over):  # noqa: F811
    from sparse_kv_selection_gb300 import binding
    a = {**COMMIT, **over}
    assert lib.prhs_commit_tokens(ctypes.byref(_kv(binding)), *a.values(), None) == binding.PRHS_EINVAL


def test_binding_checks_shapes_and_types(lib):  # noqa: F811
    """The binding's checks need no GPU: wrong arrays never reach the library."""
    import torch

    from sparse_kv_selection_gb300 import binding as b
    dev = torch.device("cpu")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    assert b._rows(x, "x", 4, 2, 64, torch.bfloat16, dev) == (x.data_ptr(), 128)
    wide = torch.zeros(4, 512, dtype=torch.bfloat16)[:, :128].view(4, 2, 64)
    assert b._rows(wide, "x", 4, 2, 64, torch.bfloat16, dev)[1] == 512
    for bad in (x.float(), x[:3], x.transpose(0, 1), x.transpose(1, 2), x[..., :32]):
        with pytest.raises(ValueError):
            b._rows(bad, "x", 4, 2, 64, torch.bfloat16, dev)
    with pytest.raises(ValueError):
        b._rows(x.transpose(0, 1).contiguous().transpose(0, 1), "x", 4, 2, 64, torch.bfloat16, dev)
    with pytest.raises(ValueError):
        b._array(torch.zeros(3, dtype=torch.int64), "n", (3,), torch.int32, dev)
    with pytest.raises(ValueError):
        b._array(None, "n", (3,), torch.int32, dev)
    with pytest.raises(ValueError):
        b._array(torch.zeros(6, dtype=torch.int32)[::2], "n", (3,), torch.int32, dev)
    with pytest.raises(ValueError):
        b.rope_turns(64, kind="other")
