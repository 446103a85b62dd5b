"""Refusals of the operators around the recurrence (include/kda_layer.h): every case is rejected, or found to be nothing to
do, before any HIP call."""
import ctypes

import pytest
import torch

import gated_delta_rule_65_amd as kda
from gated_delta_rule_65_amd.layer import QkNormForm, ScanForm

FAKE = 1 << 20  # 16-byte aligned stand-in addresses; never dereferenced
FAR = 1 << 40


def last_error():
    return kda.load_library().kda_last_error().decode()


def call(name, defaults, **kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    args = {**defaults, **kw}
    form = args.get("form")
    if form is not None:
        args["form"] = ctypes.byref(form)
    return getattr(kda.load_library(), name)(*args.values())


def expect(name, defaults, kw, status, msg):
    assert call(name, defaults, **kw) == status, last_error()
    assert msg in last_error()


PACK = dict(x=FAKE, codes=FAKE, scales=FAKE, rows=3, cols=40, dtype=1, stream=None)


@pytest.mark.parametrize("name", ["kda_ckpt8_pack", "kda_ckpt8_unpack"])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(x=None), 1, "x"), (dict(codes=None), 1, "codes"), (dict(scales=None), 1, "scales"),
    (dict(rows=-1), 2, "rows"), (dict(cols=-1), 2, "cols"), (dict(rows=1 << 40, cols=2), 2, "2^40"), (dict(rows=1, cols=1 << 31), 2, "2^31"),
    (dict(rows=1 << 32, cols=8), 2, "grid limit"), (dict(rows=1 << 28, cols=512), 2, "grid limit"),
    (dict(dtype=2), 3, "dtype"), (dict(codes=FAKE + 1), 4, "codes"), (dict(x=FAKE + 8), 4, "x"),
])
def test_ckpt8_validation(name, kw, status, msg):
    if name == "kda_ckpt8_unpack":
        order = ["codes", "scales", "x", "rows", "cols", "dtype", "stream"]
        defaults = {k: PACK[k] for k in order}
    else:
        defaults = PACK
    expect(name, defaults, kw, status, msg)


def test_ckpt8_nothing_to_do():
    assert call("kda_ckpt8_pack", PACK, rows=0, x=None, codes=None, scales=None) == 0
    assert call("kda_ckpt8_pack", PACK, cols=0, x=None, codes=None, scales=None) == 0


def scan_form(x=1, g=0, logit=0, mix=0):
    return ScanForm(x, g, logit, mix)


FWD = dict(x=FAKE, g=FAKE, h0=None, y=FAKE, h_final=None, carry=None, u=None, us=None, B=2, T=100, D=64,
           form=scan_form(), ws=FAKE, ws_bytes=1 << 40, stream=None)
VFWD = dict(x=FAKE, g=FAKE, cu=FAKE, N=2, total=100, h0=None, y=FAKE, h_final=None, carry=None, u=None, us=None, D=64,
            form=scan_form(), ws=FAKE, ws_bytes=1 << 40, stream=None)
BWD = dict(x=FAKE, g=FAKE, h0=None, carry=FAKE, u=None, us=None, dy=FAKE, dh_final=None, dx=FAKE, dg=FAKE, dh0=None,
           B=2, T=100, D=64, form=scan_form(), ws=FAKE, ws_bytes=1 << 40, stream=None)
VBWD = dict(x=FAKE, g=FAKE, cu=FAKE, N=2, total=100, h0=None, carry=FAKE, u=None, us=None, dy=FAKE, dh_final=None,
            dx=FAKE, dg=FAKE, dh0=None, D=64, form=scan_form(), ws=FAKE, ws_bytes=1 << 40, stream=None)
STEP = dict(x=FAKE, g=FAKE, h_in=FAKE, h_out=FAKE, y=FAKE, B=4, D=64, form=scan_form(), stream=None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(form=None), 1, "form"), (dict(form=scan_form(x=5)), 3, "x_dtype"), (dict(form=scan_form(g=-1)), 3, "g_dtype"),
    (dict(D=0), 2, "D"), (dict(D=1 << 31), 2, "range"), (dict(x=None), 1, "x"), (dict(g=None), 1, "g"),
    (dict(x=FAKE + 2), 4, "x"), (dict(g=FAKE + 4), 4, "g"), (dict(h0=FAKE + 8), 4, "h0"),
])
@pytest.mark.parametrize("name,defaults", [("kda_scan_fwd", FWD), ("kda_scan_varlen_fwd", VFWD), ("kda_scan_bwd", BWD),
                                           ("kda_scan_varlen_bwd", VBWD)])
def test_scan_validation(name, defaults, kw, status, msg):
    expect(name, defaults, kw, status, msg)


@pytest.mark.parametrize("name,defaults,kw,status,msg", [
    ("kda_scan_fwd", FWD, dict(y=None), 1, "y"), ("kda_scan_fwd", FWD, dict(B=-1), 2, "B"),
    ("kda_scan_fwd", FWD, dict(T=-1), 2, "T"), ("kda_scan_fwd", FWD, dict(B=1 << 30, T=1 << 30), 2, "2^40"),
    ("kda_scan_fwd", FWD, dict(B=1 << 22, T=1, D=(1 << 17) + 1), 2, "grid limit"),
    ("kda_scan_fwd", FWD, dict(u=FAKE), 1, "u_scales"), ("kda_scan_fwd", FWD, dict(us=FAKE), 1, "u_codes"),
    ("kda_scan_fwd", FWD, dict(carry=FAKE + 4), 4, "carry"),
    ("kda_scan_fwd", FWD, dict(h0=FAKE, h_final=FAKE), 2, "overlap"),
    ("kda_scan_fwd", FWD, dict(h0=FAKE, h_final=FAKE + 256), 2, "overlap"),
    ("kda_scan_varlen_fwd", VFWD, dict(cu=None), 1, "cu_seqlens"),
    ("kda_scan_varlen_fwd", VFWD, dict(cu=FAKE + 2), 4, "cu_seqlens"),
    ("kda_scan_varlen_fwd", VFWD, dict(N=-1), 2, "N"), ("kda_scan_varlen_fwd", VFWD, dict(total=1 << 31), 2, "int32"),
    ("kda_scan_bwd", BWD, dict(x=None), 1, "x and carry"), ("kda_scan_bwd", BWD, dict(carry=None), 1, "x and carry"),
    ("kda_scan_bwd", BWD, dict(x=None, carry=None, u=FAKE), 1, "u_scales"),
    ("kda_scan_bwd", BWD, dict(x=None, carry=None, us=FAKE), 1, "u_codes"),
    ("kda_scan_bwd", BWD, dict(dy=None), 1, "dy"), ("kda_scan_bwd", BWD, dict(dx=None), 1, "dx"),
    ("kda_scan_bwd", BWD, dict(dg=None), 1, "dg"), ("kda_scan_bwd", BWD, dict(dh0=FAKE, dh_final=FAKE), 2, "overlap"),
    ("kda_scan_bwd", BWD, dict(dh0=FAKE, h0=FAKE), 2, "overlap"),
    ("kda_scan_varlen_bwd", VBWD, dict(cu=None), 1, "cu_seqlens"),
    ("kda_scan_step", STEP, dict(form=None), 1, "form"), ("kda_scan_step", STEP, dict(y=None), 1, "y"),
    ("kda_scan_step", STEP, dict(h_in=None), 1, "h_in"), ("kda_scan_step", STEP, dict(h_out=FAKE + 16), 2, "overlap"),
    ("kda_scan_step", STEP, dict(B=-1), 2, "B"), ("kda_scan_step", STEP, dict(D=0), 2, "D"),
    # launches of 2^32 threads and more: 512 to 64 tokens of 64 channels, or of 256 where D % 4 == 0; a thread to a
    # value of a step, or to 4
    ("kda_scan_fwd", FWD, dict(B=1, T=1 << 29, D=1), 2, "grid limit"),
    ("kda_scan_varlen_bwd", VBWD, dict(total=1 << 29, D=257 * 4), 2, "grid limit"),
    ("kda_scan_step", STEP, dict(B=(1 << 16) + 1, D=(1 << 16) + 1), 2, "grid limit"),
    ("kda_scan_step", STEP, dict(B=1 << 18, D=1 << 16), 2, "grid limit"),
])
def test_scan_entry_validation(name, defaults, kw, status, msg):
    expect(name, defaults, kw, status, msg)


@pytest.mark.parametrize("name,defaults", [("kda_scan_fwd", dict(FWD, B=4, T=4096)),
                                           ("kda_scan_varlen_fwd", dict(VFWD, total=4096)),
                                           ("kda_scan_bwd", dict(BWD, B=4, T=4096)),
                                           ("kda_scan_varlen_bwd", dict(VBWD, total=4096))])
def test_scan_workspace_validation(name, defaults):
    N, total = (defaults["B"], defaults["B"] * defaults["T"]) if "B" in defaults else (2, 4096)
    need = kda.scan_workspace_bytes(N, total, 64)
    assert need > 0
    expect(name, defaults, dict(ws=None), 1, "workspace")
    expect(name, defaults, dict(ws_bytes=need - 1), 2, "workspace")
    expect(name, defaults, dict(ws=FAKE + 8), 4, "workspace")


def test_scan_nothing_to_do():
    none = dict(x=None, g=None, y=None, ws=None, ws_bytes=0)
    assert call("kda_scan_fwd", FWD, T=0, **none) == 0 and call("kda_scan_fwd", FWD, B=0, **none) == 0
    assert call("kda_scan_varlen_fwd", VFWD, N=0, cu=None, **none) == 0
    assert call("kda_scan_varlen_fwd", VFWD, total=0, **none) == 0
    none = dict(x=None, g=None, dy=None, dx=None, dg=None, carry=None, ws=None, ws_bytes=0)
    assert call("kda_scan_bwd", BWD, T=0, **none) == 0 and call("kda_scan_bwd", BWD, B=0, **none) == 0
    assert call("kda_scan_step", STEP, B=0, x=None, g=None, h_in=None, h_out=None, y=None) == 0
    assert last_error() == ""


def test_scan_sizes_of_unsupported_or_empty_are_zero():
    for f in (kda.scan_workspace_bytes, kda.scan_carry_bytes):
        assert f(0, 10, 8) == 0 and f(2, 0, 8) == 0 and f(2, 10, 0) == 0 and f(2, -1, 8) == 0
        assert f(2, 1 << 40, 8) == 0
    assert kda.scan_carry_bytes(3, 200, 5) == (200 // 64 + 3) * 5 * 4


def qk_form(norm=1, eps=1e-6, rot=64, interleaved=0, pos_bytes=8):
    return QkNormForm(norm, eps, rot, interleaved, pos_bytes)


QKF = dict(q=FAKE, k=FAKE, qs=None, ks=None, q_stride=256, k_stride=128, wq=None, wk=None, pos=FAKE, freqs=FAKE,
           q_out=FAKE, k_out=FAKE, q8=None, q8s=None, k8=None, k8s=None, tokens=5, Hq=2, Hk=1, D=128, dtype=1,
           form=qk_form(), stream=None)
QKB = dict(q=FAKE, k=FAKE, qs=None, ks=None, q_stride=256, k_stride=128, wq=FAKE, wk=FAKE, pos=FAKE, freqs=FAKE,
           d_q=FAKE, d_k=FAKE, dq=FAKE, dk=FAKE, dwq=FAKE, dwk=FAKE, tokens=5, Hq=2, Hk=1, D=128, dtype=1,
           grad_dtype=0, form=qk_form(), ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(form=None), 1, "form"), (dict(dtype=9), 3, "dtype"), (dict(Hq=0), 2, "Hq"), (dict(Hk=70000), 2, "Hk"),
    (dict(D=96), 2, "D"), (dict(tokens=-1), 2, "tokens"), (dict(form=qk_form(norm=2)), 2, "norm"),
    (dict(form=qk_form(eps=-1.0)), 2, "eps"), (dict(form=qk_form(eps=float("nan"))), 2, "eps"),
    (dict(form=qk_form(rot=8)), 2, "rot"), (dict(form=qk_form(rot=144)), 2, "rot"), (dict(form=qk_form(rot=-16)), 2, "rot"),
    (dict(form=qk_form(pos_bytes=2)), 3, "pos_bytes"), (dict(q_stride=255), 2, "stride"),
    (dict(q_stride=260), 2, "stride"), (dict(k_stride=120), 2, "stride"), (dict(tokens=1 << 33, q_stride=1024), 2, "2^40"),
    (dict(q=None), 1, "q"), (dict(k=None), 1, "k"), (dict(k=FAKE + 2), 4, "k"), (dict(qs=FAKE), 1, "k_scales"),
    (dict(ks=FAKE), 1, "q_scales"), (dict(qs=FAKE, ks=FAKE, q_stride=512), 2, "contiguous"),
    (dict(pos=None), 1, "pos"), (dict(freqs=None), 1, "freqs"), (dict(wq=FAKE + 4), 4, "wq"),
])
@pytest.mark.parametrize("name,defaults", [("kda_qknorm_fwd", QKF), ("kda_qknorm_bwd", QKB)])
def test_qknorm_validation(name, defaults, kw, status, msg):
    expect(name, defaults, kw, status, msg)


@pytest.mark.parametrize("name,defaults,kw,status,msg", [
    ("kda_qknorm_fwd", QKF, dict(q_out=None), 1, "q_out"), ("kda_qknorm_fwd", QKF, dict(q8=FAKE), 1, "k8"),
    ("kda_qknorm_fwd", QKF, dict(q8=FAKE, k8=FAKE, q8s=FAKE), 1, "k8_scales"),
    ("kda_qknorm_fwd", QKF, dict(qs=FAKE, ks=FAKE, q8=FAKE, k8=FAKE, q8s=FAKE, k8s=FAKE), 2, "packed already"),
    ("kda_qknorm_bwd", QKB, dict(grad_dtype=3), 3, "grad_dtype"), ("kda_qknorm_bwd", QKB, dict(d_q=None), 1, "d_q"),
    ("kda_qknorm_bwd", QKB, dict(dk=None), 1, "dk"), ("kda_qknorm_bwd", QKB, dict(dwk=None), 1, "dwk"),
    ("kda_qknorm_bwd", QKB, dict(ws=None), 1, "workspace"), ("kda_qknorm_bwd", QKB, dict(ws_bytes=8), 2, "workspace"),
])
def test_qknorm_entry_validation(name, defaults, kw, status, msg):
    expect(name, defaults, kw, status, msg)


def test_qknorm_nothing_to_do():
    assert call("kda_qknorm_fwd", QKF, tokens=0, q=None, k=None, pos=None, q_out=None, k_out=None) == 0
    assert call("kda_qknorm_bwd", QKB, tokens=0, dwq=None, dwk=None, ws=None, ws_bytes=0) == 0
    assert kda.qk_norm_rope_workspace_bytes(0, 2, 1, 128) == 0 and kda.qk_norm_rope_workspace_bytes(5, 2, 1, 96) == 0


def test_torch_front_ends_reject_what_the_kernels_do_not_take():
    x, g = torch.zeros(2, 5, 8), torch.zeros(2, 5, 8)
    with pytest.raises(ValueError, match="GPU"):
        kda.scan_fwd(x, g)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        kda.scan_fwd(x.half(), g)
    with pytest.raises(ValueError, match="channels"):
        kda.scan_fwd(x[0], g[0])
    with pytest.raises(ValueError, match="GPU"):
        kda.ckpt8_pack(x)
    with pytest.raises(TypeError, match="Packed8"):
        kda.ckpt8_unpack(x)
    with pytest.raises(ValueError, match="GPU"):
        kda.qk_norm_rope_fwd(torch.zeros(5, 2, 64), torch.zeros(5, 2, 64))
    with pytest.raises(TypeError, match="both be packed"):
        kda.qk_norm_rope_fwd(kda.Packed8(x, x, torch.float32), torch.zeros(5, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        kda.scan_step(x[0], g[0], x[0])
    with pytest.raises(ValueError, match="GPU"):
        kda.scan_bwd(g, x, x, x=x)


@pytest.mark.parametrize("shape,view,stride", [
    ((6, 4, 128), lambda t: t, 512), ((6, 8, 128), lambda t: t[:, 2:4], 1024), ((2, 3, 8, 128), lambda t: t[:, :, :4], 1024),
    ((1, 4, 128), lambda t: t, 512), ((6, 1, 64), lambda t: t, 64),
])
def test_token_strides(shape, view, stride):
    from gated_delta_rule_65_amd.layer import _token_stride
    assert _token_stride(view(torch.zeros(shape)), "q") == stride


@pytest.mark.parametrize("view", [lambda t: t[:, :, ::2], lambda t: t.transpose(1, 2), lambda t: t[:, ::2, :2],
                                  lambda t: t.transpose(0, 1), lambda t: t[..., ::2]])
def test_token_strides_refused(view):
    from gated_delta_rule_65_amd.layer import _token_stride
    with pytest.raises(ValueError):
        _token_stride(view(torch.zeros(3, 5, 4, 128)), "q")
