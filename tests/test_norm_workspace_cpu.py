"""The norm's backward leaves a partial of the weights' gradients per
workgroup, and tokens of few narrow heads share a workgroup: what the library
asks for shows how many workgroups there are (no GPU)."""
import ctypes

import pytest

from tests.test_state_abi_cpu import lib, norm_desc  # noqa: F401  (lib is a fixture)


def partials(lib, **kw):  # noqa: F811
    d = norm_desc(rot=8, **kw)
    n = lib.gscan_qk_norm_rope_workspace_bytes(ctypes.byref(d))
    assert n % (2 * d.D * 4) == 0
    return n // (2 * d.D * 4)


@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 32), (1, 0, 64), (3, 2, 8), (1, 0, 8), (1, 0, 72), (2, 1, 32)])
def test_few_narrow_heads_share_a_workgroup(lib, Hq, Hk, D):  # noqa: F811
    # at most 8 tokens have their angles in LDS; 7 or 8 of these heads' rows fill less than one pass
    assert partials(lib, tokens=560, Hq=Hq, Hk=Hk, D=D) <= 560 // 7
    assert partials(lib, tokens=1, Hq=Hq, Hk=Hk, D=D) == 1
    assert partials(lib, tokens=0, Hq=Hq, Hk=Hk, D=D) == 1
    assert partials(lib, tokens=2 ** 31 - 200, Hq=Hq, Hk=Hk, D=D) == 1024


def test_many_heads_have_a_workgroup_of_their_own(lib):  # noqa: F811
    assert partials(lib, tokens=300, Hq=2 ** 20, Hk=2 ** 20, D=256) == 300
    for kw in (dict(Hq=0), dict(Hk=-1), dict(Hq=2 ** 20 + 1), dict(Hk=2 ** 20 + 1)):
        assert lib.gscan_qk_norm_rope_workspace_bytes(ctypes.byref(norm_desc(**kw))) == 0
