"""Refusals of the token-batch forms on the host."""
import ctypes

import pytest

from test_abi import _kv, lib  # noqa: F401

PLANNED = dict(T=4, cu=64, slots=64, idx=64, cap=4, n=64, k=64, ks=512, v=64, vs=512, lens=64)


@pytest.mark.parametrize("over", [dict(T=-1), dict(cu=None), dict(slots=None), dict(n=None), dict(lens=None), dict(cap=0),
                                  dict(k=None), dict(v=None), dict(k=72), dict(v=72), dict(ks=100), dict(vs=514)])
def test_commit_planned_refusals(lib, over):  # noqa: F811
    from sparse_kv_selection_gb300 import binding
    a = {**PLANNED, **over}
    assert lib.prhs_commit_planned(ctypes.byref(_kv(binding)), *a.values(), None) == binding.PRHS_EINVAL
    assert lib.prhs_last_message().decode() != ""
    assert lib.prhs_commit_planned(None, *PLANNED.values(), None) == binding.PRHS_EINVAL
