"""Refusals of linear attention and of the group norm (include/kda_layer.h): every case is rejected, or found to be nothing to
do, before any HIP call; and what the front ends refuse before they call."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_65_amd as kda
from gated_delta_rule_65_amd.groupnorm import GroupNormForm

FAKE = 1 << 20  # 16-byte aligned stand-in addresses; never dereferenced
FAR = 1 << 40


def last_error():
    return kda.load_library().kda_last_error().decode()


def call(name, defaults, **kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    args = {**defaults, **kw}
    if args.get("form") is not None:
        args["form"] = ctypes.byref(args["form"])
    return getattr(kda.load_library(), name)(*args.values())


def expect(name, defaults, kw, status, msg):
    assert call(name, defaults, **kw) == status, last_error()
    assert msg in last_error()


DIMS = dict(H=2, Dk=64, Dv=128, scale=1.0, dtype=1)
WS = dict(workspace=FAKE, workspace_bytes=1 << 40, stream=None)
QKVG = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE)
GRADS = dict(d_o=FAKE, d_sfinal=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ds0=FAR)
FWD = dict(**QKVG, s0=FAKE, o=FAKE, s_final=FAR, B=2, T=3, **DIMS, **WS)
VARLEN = dict(**QKVG, cu_seqlens=FAKE, N=2, total=9, s0=FAKE, o=FAKE, s_final=FAR, **DIMS, **WS)
BWD = dict(**QKVG, s0=FAKE, **GRADS, B=2, T=3, **DIMS, **WS)
VARLEN_BWD = dict(**QKVG, cu_seqlens=FAKE, N=2, total=9, s0=FAKE, **GRADS, **DIMS, **WS)
STEP = dict(**QKVG, s_in=FAKE, s_out=FAR, o=FAKE, B=2, **DIMS, stream=None)
CALLS = [("kda_linattn_fwd", FWD), ("kda_linattn_varlen_fwd", VARLEN), ("kda_linattn_bwd", BWD),
         ("kda_linattn_varlen_bwd", VARLEN_BWD), ("kda_linattn_step", STEP)]


@pytest.mark.parametrize("name,defaults", CALLS, ids=lambda x: x if isinstance(x, str) else "")
@pytest.mark.parametrize("kw,status,msg", [
    (dict(q=None), 1, "q"), (dict(k=None), 1, "k"), (dict(v=None), 1, "v"), (dict(g=None), 1, "g"), (dict(g=FAKE + 2), 4, "g"),
    (dict(q=FAKE + 2), 4, "q"), (dict(v=FAKE + 8), 4, "v"), (dict(H=0), 2, "H"), (dict(H=65537), 2, "H"),
    (dict(Dk=32), 2, "Dk"), (dict(Dv=256), 2, "Dv"), (dict(dtype=2), 3, "dtype"),
])
def test_common_validation(name, defaults, kw, status, msg):
    expect(name, defaults, kw, status, msg)


@pytest.mark.parametrize("name,defaults,kw,status,msg", [
    ("kda_linattn_fwd", FWD, dict(B=-1), 2, "B"), ("kda_linattn_fwd", FWD, dict(T=-1), 2, "T"),
    ("kda_linattn_fwd", FWD, dict(B=1 << 30, T=1 << 30), 2, "2^40"), ("kda_linattn_fwd", FWD, dict(B=1 << 30, T=1), 2, "out of range"),
    ("kda_linattn_fwd", FWD, dict(T=1 << 34), 2, "out of range"), ("kda_linattn_fwd", FWD, dict(o=None), 1, "o"),
    ("kda_linattn_fwd", FWD, dict(s0=FAKE + 4), 4, "s0"), ("kda_linattn_fwd", FWD, dict(s_final=FAKE), 2, "overlap"),
    ("kda_linattn_fwd", FWD, dict(T=100000, workspace=None), 1, "workspace"),
    ("kda_linattn_fwd", FWD, dict(T=100000, workspace_bytes=64), 2, "workspace"),
    ("kda_linattn_varlen_fwd", VARLEN, dict(N=-1), 2, "N"), ("kda_linattn_varlen_fwd", VARLEN, dict(total=-1), 2, "total"),
    ("kda_linattn_varlen_fwd", VARLEN, dict(total=1 << 31), 2, "int32"),
    ("kda_linattn_varlen_fwd", VARLEN, dict(cu_seqlens=None), 1, "cu_seqlens"),
    ("kda_linattn_varlen_fwd", VARLEN, dict(cu_seqlens=FAKE + 2), 4, "cu_seqlens"),
    ("kda_linattn_bwd", BWD, dict(d_o=None), 1, "d_o"), ("kda_linattn_bwd", BWD, dict(dq=None), 1, "dq"),
    ("kda_linattn_bwd", BWD, dict(dk=None), 1, "dk"), ("kda_linattn_bwd", BWD, dict(dv=FAKE + 2), 4, "dv"),
    ("kda_linattn_bwd", BWD, dict(ds0=FAKE), 2, "overlap"),
    ("kda_linattn_bwd", BWD, dict(T=100000, workspace=None), 1, "workspace"),
    ("kda_linattn_varlen_bwd", VARLEN_BWD, dict(total=100000, workspace_bytes=64), 2, "workspace"),
    ("kda_linattn_step", STEP, dict(B=-1), 2, "B"), ("kda_linattn_step", STEP, dict(s_in=None), 1, "s_in"),
    ("kda_linattn_step", STEP, dict(s_out=None), 1, "s_out"), ("kda_linattn_step", STEP, dict(s_out=FAKE + 16), 2, "overlap"),
])
def test_linattn_validation(name, defaults, kw, status, msg):
    expect(name, defaults, kw, status, msg)


def test_linattn_nothing_to_do():
    none = dict(q=None, k=None, v=None, g=None)
    assert call("kda_linattn_fwd", FWD, B=0, **none, o=None, s0=None, s_final=None) == 0
    assert call("kda_linattn_fwd", FWD, T=0, **none, o=None, s_final=None) == 0
    assert call("kda_linattn_varlen_fwd", VARLEN, N=0, total=0, cu_seqlens=None, **none, o=None) == 0
    grads = dict(d_o=None, dq=None, dk=None, dv=None, ds0=None)
    assert call("kda_linattn_bwd", BWD, T=0, **none, **grads) == 0
    assert call("kda_linattn_varlen_bwd", VARLEN_BWD, N=0, total=0, cu_seqlens=None, **none, **grads) == 0
    assert call("kda_linattn_step", STEP, B=0, **none, s_in=None, s_out=None, o=None) == 0


def test_linattn_workspace_sizes():
    for size in (kda.linattn_workspace_bytes, kda.linattn_bwd_workspace_bytes):
        for dtype in (torch.bfloat16, torch.float32):
            assert size(0, 5, 2, 64, 64, dtype) == size(1, 0, 2, 64, 64, dtype) == size(1, 5, 0, 64, 64, dtype) == 0
            assert size(1, 5, 2, 32, 64, dtype) == size(1 << 30, 1 << 30, 65536, 64, 64, dtype) == 0
            assert size(1, 1 << 20, 8, 128, 128, dtype) > 0


@pytest.mark.parametrize("N,total,H", [(1, 1 << 20, 8), (4096, 4096 * 64, 16), (65536, 65536, 64), (3, 40011, 16), (1, 999, 1),
                                       (100000, 3000000, 4)])
def test_linattn_workspace_is_for_what_lies_between_segments(N, total, H):
    """768 segments of all heads at most have a state to hand on, however many sequences there are."""
    for size, ways in ((kda.linattn_workspace_bytes, 1), (kda.linattn_bwd_workspace_bytes, 2)):
        assert size(N, total, H, 64, 128, torch.bfloat16) <= ways * 768 * 64 * 128 * 4


def test_linattn_more_workgroups_than_a_grid_has():
    grid = dict(T=1, H=1, Dk=128, Dv=128, s0=None)  # one workgroup a sequence: of 256 threads in bf16, of 512 in fp32
    expect("kda_linattn_fwd", FWD, dict(B=1 << 24, **grid), 2, "grid limit")
    expect("kda_linattn_fwd", FWD, dict(B=9 << 20, dtype=0, **grid), 2, "grid limit")
    expect("kda_linattn_bwd", BWD, dict(B=3 << 20, dtype=0, d_sfinal=None, **grid), 2, "grid limit")


GN = dict(x=FAKE, x_stride=128, weight=FAKE, bias=FAKE, gate=FAKE, gate_stride=128, y=FAKE, tokens=3, groups=2, width=64,
          form=GroupNormForm(1, 1, 1, 1e-5), stream=None)
GN_BWD = dict(x=FAKE, x_stride=128, weight=FAKE, bias=FAKE, gate=FAKE, gate_stride=128, dy=FAKE, dx=FAKE, dgate=FAKE,
              dweight=FAKE, dbias=FAKE, tokens=3, groups=2, width=64, form=GroupNormForm(1, 1, 1, 1e-5), workspace=FAKE,
              workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("name,defaults", [("kda_groupnorm_fwd", GN), ("kda_groupnorm_bwd", GN_BWD)])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(x=None), 1, "x"), (dict(x=FAKE + 1), 4, "x"), (dict(gate=FAKE + 1), 4, "gate"), (dict(weight=FAKE + 2), 4, "weight"),
    (dict(bias=FAKE + 2), 4, "bias"), (dict(form=None), 1, "form"), (dict(form=GroupNormForm(2, 1, 1, 0.0)), 3, "x_dtype"),
    (dict(form=GroupNormForm(1, 7, 1, 0.0)), 3, "y_dtype"), (dict(form=GroupNormForm(1, 1, 3, 0.0)), 2, "act"),
    (dict(form=GroupNormForm(1, 1, 1, -1.0)), 2, "eps"), (dict(form=GroupNormForm(1, 1, 1, math.nan)), 2, "eps"),
    (dict(tokens=-1), 2, "tokens"), (dict(groups=0), 2, "groups"), (dict(width=0), 2, "width"),
    (dict(width=(1 << 16) + 1), 2, "width"), (dict(groups=1 << 20, width=64), 2, "2^24"), (dict(x_stride=127), 2, "x_stride"),
    (dict(gate_stride=100), 2, "gate_stride"), (dict(tokens=1 << 40), 2, "2^40"), (dict(x_stride=1 << 41), 2, "2^40"),
])
def test_groupnorm_validation(name, defaults, kw, status, msg):
    expect(name, defaults, kw, status, msg)


@pytest.mark.parametrize("name,defaults,kw,status,msg", [
    ("kda_groupnorm_fwd", GN, dict(y=None), 1, "y"), ("kda_groupnorm_fwd", GN, dict(y=FAKE + 1), 4, "y"),
    ("kda_groupnorm_bwd", GN_BWD, dict(dy=None), 1, "dy"), ("kda_groupnorm_bwd", GN_BWD, dict(dx=None), 1, "dx"),
    ("kda_groupnorm_bwd", GN_BWD, dict(dgate=None), 1, "dgate"), ("kda_groupnorm_bwd", GN_BWD, dict(gate=None), 2, "dgate"),
    ("kda_groupnorm_bwd", GN_BWD, dict(dbias=None), 1, "dbias"), ("kda_groupnorm_bwd", GN_BWD, dict(dweight=None), 1, "dweight"),
])
def test_groupnorm_call_validation(name, defaults, kw, status, msg):
    expect(name, defaults, kw, status, msg)


def test_groupnorm_nothing_to_do():
    assert call("kda_groupnorm_fwd", GN, tokens=0, x=None, y=None, gate=None) == 0
    assert call("kda_groupnorm_bwd", GN_BWD, tokens=0, x=None, dy=None, dx=None, gate=None, dgate=None, dweight=None, dbias=None) == 0
    assert kda.group_norm_act_workspace_bytes(0, 2, 64) == kda.group_norm_act_workspace_bytes(5, 0, 64) == 0
    assert kda.group_norm_act_workspace_bytes(5, 2, 1 << 17) == 0


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("f,error,msg", [
    (lambda: kda.linattn_fwd(t(2, 3, 64), t(2, 3, 64), t(2, 3, 64), t(2)), ValueError, "B, T, H, Dk"),
    (lambda: kda.linattn_fwd([1], t(2, 3, 2, 64), t(2, 3, 2, 64), t(2)), TypeError, "torch.Tensor"),
    (lambda: kda.linattn_fwd(*(t(2, 3, 2, 64, dtype=torch.float16),) * 3, t(2)), TypeError, "float32 or bfloat16"),
    (lambda: kda.linattn_fwd(*(t(2, 3, 2, 64),) * 3, t(2)), ValueError, "GPU"),
    (lambda: kda.linattn_varlen_fwd(*(t(3, 2, 64),) * 3, t(2), None), ValueError, "cu_seqlens"),
    (lambda: kda.linattn_varlen_bwd(*(t(3, 2, 64),) * 3, t(2), None, t(3, 2, 64)), ValueError, "cu_seqlens"),
    (lambda: kda.linattn_step(*(t(3, 1, 2, 64),) * 3, t(2), t(3, 2, 64, 64)), ValueError, "H, Dk"),
    (lambda: kda.group_norm_act_fwd(t(3, 64), 5), ValueError, "groups must divide"),
    (lambda: kda.group_norm_act_fwd(t(3, 64), 0), ValueError, "groups must divide"),
    (lambda: kda.group_norm_act_fwd(t(3, 64), 2, act="gelu"), ValueError, "act must be one of"),
    (lambda: kda.group_norm_act_fwd(t(3, 64, dtype=torch.float16), 2), TypeError, "float32 or bfloat16"),
    (lambda: kda.group_norm_act_fwd(t(3, 64), 2), ValueError, "GPU"),
    (lambda: kda.group_norm_act_fwd("x", 2), TypeError, "torch.Tensor"),
])
def test_front_end_refusals(f, error, msg):
    with pytest.raises(error, match=msg):
        f()
