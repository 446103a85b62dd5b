"""Refusals and sizes of the calls around the operators' edges, before any HIP call."""
import subprocess

import pytest

import gated_delta_rule_65_amd as kda
from gated_delta_rule_65_amd import _build
from tests.test_layer_abi import BWD, FAKE, FWD, PACK, QKF, STEP, VBWD, VFWD, call, expect, last_error, qk_form

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


def segments(N, T=None, total=None):
    """Chains and the segments of each: of equally long sequences of T tokens, or of packed rows."""
    if T is not None and T >= 32:
        return N, -(-T // 64)
    return 1, -(-(total if T is None else N * T) // 64)


def sizes(N, total, D):
    return kda.scan_workspace_bytes(N, total, D), kda.scan_carry_bytes(N, total, D)


def used(chains, per, D):
    """Bytes of the words that segments, groups of 8 and blocks of 64 of them publish (none where no chain is longer than a
    segment), and of the states at the segments."""
    words = chains * D * (per + -(-per // 8) + -(-per // 64))
    return 256 + 8 * words if per > 1 else 0, chains * per * D * 4


@pytest.mark.parametrize("N", [1, 2, 3, 7, 31, 64, 65, 255, 1000, 16384])
def test_scan_sizes_hold_what_is_used(N):
    for T in [*range(1, 70), 95, 96, 127, 128, 129, 511, 512, 513, 4095, 4096, 4097, 4160, 8192]:
        for layout in (dict(T=T), dict(total=N * T)):
            got, want = sizes(N, N * T, 5), used(*segments(N, **layout), 5)
            assert got[0] >= want[0] and got[1] >= want[1], (N, layout)
    for total in (1, 2, 63, 64, 65, 100, 640, 4097, 100003):  # packed: any number of sequences, most of them empty
        got, want = sizes(N, total, 3), used(*segments(N, total=total), 3)
        assert got[0] >= want[0] and got[1] >= want[1], (N, total)


@pytest.mark.parametrize("N,total", [(16384, 32768), (1 << 20, 1 << 20), (100000, 7), (4096, 4096 * 16), (1 << 16, 65)])
def test_scan_sizes_do_not_grow_with_empty_and_short_sequences(N, total):
    """Only sequences of 32 tokens and more have segments of their own."""
    D, segs = 8, -(-total // 64)
    ws, carry = sizes(N, total, D)
    assert ws <= 256 + 8 * D * (8 * segs + 8) and carry <= 4 * D * (3 * segs + 1)


def test_scan_lds_buffers_are_aligned_for_wide_access(tmp_path):
    """Their rows are read and written 16 bytes at a time, in every kernel that declares one."""
    probe = tmp_path / "probe.hip"
    probe.write_text("""#include "kda_scan.h"
static_assert(alignof(kda::Exchange<1>) >= 16 && alignof(kda::Exchange<4>) >= 16, "exchange");
static_assert(alignof(kda::Kept<1, true>) >= 16 && alignof(kda::Kept<4, true>) >= 16, "kept");
static_assert(sizeof(kda::Exchange<4>::A[0]) % 16 == 0 && sizeof(kda::Kept<4, true>::rows[0][0]) % 16 == 0, "rows");
static_assert(offsetof(kda::Exchange<4>, b) % 16 == 0 && offsetof(kda::Exchange<4>, before) % 16 == 0, "parts");
""")
    r = subprocess.run([_build.hipcc(), *_build.HIPCC_FLAGS, "--offload-device-only", "-fsyntax-only", str(probe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


ODD = {"kda_scan_fwd": dict(FWD, D=37), "kda_scan_varlen_fwd": dict(VFWD, D=37), "kda_scan_bwd": dict(BWD, D=37),
       "kda_scan_varlen_bwd": dict(VBWD, D=37), "kda_scan_step": dict(STEP, B=1, D=37)}


@pytest.mark.parametrize("name", ODD)
@pytest.mark.parametrize("kw,size", [(dict(x=FAKE + 1), 2), (dict(g=FAKE + 2), 4)])
def test_rows_read_an_element_at_a_time_begin_at_an_element(name, kw, size):
    expect(name, ODD[name], kw, 4, f"is not {size}-byte aligned")


@pytest.mark.parametrize("name,kw,what", [
    ("kda_scan_fwd", dict(y=FAKE + 1), "y is not 2"), ("kda_scan_fwd", dict(h0=FAKE + 2), "h0 is not 4"),
    ("kda_scan_fwd", dict(h_final=FAKE + 2), "h_final is not 4"), ("kda_scan_fwd", dict(carry=FAKE + 2), "carry is not 4"),
    ("kda_scan_fwd", dict(ws=FAKE + 8), "workspace is not 16"), ("kda_scan_bwd", dict(dy=FAKE + 1), "dy is not 2"),
    ("kda_scan_bwd", dict(dg=FAKE + 2), "dg is not 4"), ("kda_scan_bwd", dict(dh0=FAKE + 2), "dh0 is not 4"),
    ("kda_scan_step", dict(h_in=FAKE + 2), "h_in is not 4"), ("kda_scan_step", dict(B=4, x=FAKE + 8), "x is not 16"),
])
def test_alignment_is_named(name, kw, what):
    expect(name, ODD[name], kw, 4, what)


@pytest.mark.parametrize("kw,what", [(dict(x=FAKE + 1), "x is not 2"), (dict(x=FAKE + 2, dtype=0), "x is not 4"),
                                     (dict(x=FAKE + 8, cols=64), "x is not 16"), (dict(codes=FAKE + 8, cols=64), "codes is not 16")])
def test_ckpt8_alignment_is_named(kw, what):
    expect("kda_ckpt8_pack", dict(PACK, cols=37), kw, 4, what)


@pytest.mark.parametrize("kw,what", [(dict(pos=FAKE + 4), "pos is not 8"), (dict(freqs=FAKE + 4), "freqs is not 8"),
                                     (dict(pos=FAKE + 2, form=qk_form(pos_bytes=4)), "pos is not 4")])
def test_qknorm_alignment_is_named(kw, what):
    expect("kda_qknorm_fwd", QKF, kw, 4, what)
