"""Refusals and sizes of the calls around the operators' edges, before any HIP call."""
import pytest

import gated_delta_rule_65_amd as kda
from tests.test_layer_abi import FAKE, call, expect, last_error

BEHIND = dict(cu=FAKE, N=2, total=9, a=FAKE, a_row=6, b=None, b_row=0, stream=None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(cu=None), 1, "cu_seqlens"), (dict(cu=FAKE + 2), 4, "cu_seqlens"), (dict(N=-1), 2, "N"),
    (dict(total=-1), 2, "total"), (dict(total=1 << 31), 2, "int32"), (dict(a=None), 1, "a"), (dict(a=FAKE + 8), 4, "a"),
    (dict(a_row=3), 2, "even"), (dict(a_row=-2), 2, "even"), (dict(a_row=1 << 27), 2, "even"),
    (dict(b=FAKE + 2, b_row=4), 4, "b"), (dict(b=FAKE, b_row=5), 2, "even"),
])
def test_zero_behind_validation(kw, status, msg):
    expect("kda_scan_zero_behind", BEHIND, kw, status, msg)


def test_zero_behind_nothing_to_do():
    assert call("kda_scan_zero_behind", BEHIND, total=0, a=None, cu=None) == 0
    assert call("kda_scan_zero_behind", BEHIND, a_row=0, a=None, cu=None) == 0
    assert last_error() == ""
