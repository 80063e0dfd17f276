"""mx_rms_norm without rows still makes the column copy's zeros, and its kernels read the
weight for that: a missing or unaligned one is refused, as with rows.  CPU only, on fake
addresses."""

import pytest

from tests.test_ffn_limits import NORM, P, _call
from tests.test_library import host_only_lib, lib  # noqa: F401  (fixtures)


@pytest.mark.parametrize("K", [64, 1056])                # both copies in one kernel, and in two
@pytest.mark.parametrize("change,status", [({"w": None}, 1), ({"w": P + 2}, 3)])
def test_weight_without_rows(host_only_lib, K, change, status):  # noqa: F811
    args = dict(M=0, K=K, x=None, r=None, total=None, rstd=None, y=None, q=None, scale=None, M_cap=32)
    assert _call(host_only_lib, "mx_rms_norm", NORM, **args, **change) == status
    assert _call(host_only_lib, "mx_rms_norm", NORM, **{**args, "M_cap": 0}, **change) == 0
