"""The operators around the recurrence on the GPU against their 64-bit forms (tests/layer_ref.py, which also gives the
bounds: 32-bit arithmetic, and half a step of the output's type)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_65_amd as kda
import oracle
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, kind="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[kind]).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def near(got, want, kind, what):
    """|got - value| <= bound + half a step of the type, everywhere."""
    value, bound = want
    got = host(got).reshape(value.shape)
    room = bound * (1 + ref.ROUND[kind]) + ref.ROUND[kind] * np.abs(value) + 2.0 ** -130
    over = np.abs(got - value) - room
    bad = ~(over <= 0)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} against {value[bad][0]} +- {room[bad][0]}"


# ----------------------------------------------------------------- checkpoints in 8 bits

def same_pack(x, kind):
    t = dev(x, kind)
    p = kda.ckpt8_pack(t)
    rows = host(t).reshape(-1, x.shape[-1])
    codes, scales, values = ref.pack8(rows)
    assert (p.scales.cpu().numpy().reshape(scales.shape) == scales).all()
    got = p.codes.cpu().numpy().reshape(codes.shape)
    assert ((got == codes) | ((values == 0) & (got & 127 == 0))).all()
    for out in TYPES:
        u = kda.ckpt8_unpack(p, TYPES[out])
        assert u.dtype == TYPES[out] and u.shape == t.shape
        assert (host(u).reshape(values.shape) == values).all()
    assert kda.ckpt8_unpack(p).dtype == t.dtype


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (5, 32), (7, 33), (2, 3, 100), (4, 128), (33, 1000), (3, 4096), (70000, 8),
                                   (300, 64), (9, 24), (5, 1), (2, 16), (64,)])
def test_ckpt8_is_the_nearest_code(shape, kind):
    rng = np.random.default_rng(sum(shape))
    x = rng.normal(size=shape) * np.exp(rng.normal(size=shape) * 3)
    same_pack(np.atleast_2d(x) if x.ndim == 1 else x, kind)


def test_ckpt8_every_bf16_value():
    bits = np.arange(65536, dtype=np.uint32)
    bits = bits[(bits & 0x7f80) != 0x7f80]  # finite
    x = (bits << 16).astype(np.uint32).view(np.float32)
    same_pack(np.sort(x).reshape(-1, 32), "bf16")  # blocks of like size, among them the largest and the denormal ones
    same_pack(x.reshape(32, -1).T.copy(), "bf16")  # blocks that span everything


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_ckpt8_infinities_and_nan_leave_their_block_alone(kind):
    x = np.random.default_rng(1).normal(size=(40, 70)).astype(np.float32)
    bad = x.copy()
    bad[3, 5], bad[3, 40], bad[10, 69], bad[20] = np.inf, -np.inf, np.nan, np.nan
    clean = np.where(np.isfinite(bad), bad, 0)
    p, q = kda.ckpt8_pack(dev(bad, kind)), kda.ckpt8_pack(dev(clean, kind))
    assert torch.equal(p.scales, q.scales)
    u, v = host(kda.ckpt8_unpack(p)), host(kda.ckpt8_unpack(q))
    assert (np.isnan(u) == ~np.isfinite(bad)).all() and (u[np.isfinite(bad)] == v[np.isfinite(bad)]).all()


def test_ckpt8_empty_and_out_of_alignment():
    for shape in ((0, 5), (3, 0)):
        p = kda.ckpt8_pack(torch.empty(shape, device="cuda"))
        assert kda.ckpt8_unpack(p).shape == shape
    with pytest.raises(kda.KDAError, match="aligned"):
        kda.ckpt8_pack(torch.zeros(65, device="cuda")[1:])


# ----------------------------------------------------------------- gated scan

def scan_data(rows, D, N, logit, seed, xk, gk, far=0.05):
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(rows, D)) * 1.5 - 2
    g = z if logit else -np.logaddexp(z, 0)
    pick = rng.random((rows, D))
    edge = (8.0, -30.0) if logit else (-6.0, 0.5)
    g = np.where(pick < far, edge[0], np.where(pick < 2 * far, edge[1], g))
    if not logit:
        g = np.where((pick > 0.95) & (pick < 0.96), -np.inf, np.where(pick > 0.99, 0.0, g))
    d = {"x": dev(rng.normal(size=(rows, D)), xk), "g": dev(g, gk), "dy": dev(rng.normal(size=(rows, D)), xk),
         "h0": dev(rng.normal(size=(N, D))), "dh": dev(rng.normal(size=(N, D)))}
    return d, {k: host(v) for k, v in d.items()}


def check_scan(where, D, xk, gk, logit, mix, batch=None, cu=None, total=None, h0=True, seed=1):
    """Both directions and both forms of what the backward pass keeps."""
    N, rows = len(where), total if total is not None else where[-1][1]
    d, h = scan_data(rows, D, N, logit, seed, xk, gk)
    if not h0:
        d["h0"], h["h0"] = None, np.zeros_like(h["h0"])
    form = {"g_logit": logit, "complement": mix}
    (y, hf, u) = ref.scan(h["x"], h["g"], h["h0"], where, logit, mix)
    grads = ref.scan_grad(h["x"], h["g"], h["h0"], h["dy"], h["dh"], where, logit, mix)
    shape = (*batch, D) if batch else (rows, D)
    x, g, dy = (d[k].reshape(shape) for k in ("x", "g", "dy"))
    inside = np.zeros(rows, bool)
    for i, j in where:
        inside[i:j] = True

    def fwd(save):
        if cu is None:
            return kda.scan_fwd(x, g, d["h0"], save=save, **form)
        return kda.scan_varlen_fwd(x, g, cu, d["h0"], save=save, **form)

    def bwd(saved, x, h0):
        if cu is None:
            return kda.scan_bwd(g, dy, saved, x=x, h0=h0, dh_final=d["dh"], **form)
        return kda.scan_varlen_bwd(g, cu, dy, saved, x=x, h0=h0, dh_final=d["dh"], **form)

    def rows_near(got, want, kind, what):
        near(got.reshape(rows, D)[torch.from_numpy(inside).cuda()], (want[0][inside], want[1][inside]), kind, what)

    y0, hf0, none = fwd(None)
    assert none is None and y0.dtype == TYPES[xk] and y0.shape == shape
    rows_near(y0, y, xk, "y")
    near(hf0, hf, "f32", "h_final")
    for save in ("carry", "ckpt8"):
        y1, hf1, saved = fwd(save)
        assert torch.equal(y1.reshape(rows, D)[inside], y0.reshape(rows, D)[inside]) and torch.equal(hf1, hf0), \
            "what is kept changed the result"
        if save == "carry":
            dx, dg, dh0 = bwd(saved, x, d["h0"])
            want = grads
        else:
            codes, scales = saved.codes.cpu().numpy(), saved.scales.cpu().numpy()
            got = ref.unpack8(codes[inside], scales[inside])
            value, bound = u[0][inside], u[1][inside]
            step = 2.0 ** (np.repeat(scales[inside].astype(float), 32, 1)[:, :D] - 127)
            room = bound + np.maximum(2.0 ** -4 * (np.abs(value) + bound), 2.0 ** -10 * step)
            assert (np.abs(got - value) <= room).all(), "u in 8 bits"
            _, _, packed = ref.pack8(value)
            apart = (got != packed).mean()
            assert apart <= 0.002, f"{apart} of the codes are not the nearest"  # those within 32-bit rounding of a tie
            dx, dg, dh0 = bwd(saved, None, None)
            given = np.zeros((rows, D))
            given[inside] = got
            want = ref.scan_grad(h["x"], h["g"], h["h0"], h["dy"], h["dh"], where, logit, mix, u=given)
        assert dx.dtype == TYPES[xk] and dg.dtype == TYPES[gk] and dx.shape == shape
        rows_near(dx, want[0], xk, f"dx ({save})")
        rows_near(dg, want[1], gk, f"dg ({save})")
        near(dh0, want[2], "f32", f"dh0 ({save})")


@pytest.mark.parametrize("D", [1, 36, 200])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (2, 7), (5, 63), (1, 64), (2, 65), (3, 130), (1, 515), (2, 700), (70, 1),
                                 (40, 20), (23, 31), (4, 32), (300, 3)])
def test_scan_batches(B, T, D):
    check_scan([(i * T, (i + 1) * T) for i in range(B)], D, "bf16", "bf16", D == 36, B % 2 == 1, batch=(B, T), h0=T != 7)


@pytest.mark.parametrize("xk,gk", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("logit,mix", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("D", [130, 264])
def test_scan_types_and_forms(xk, gk, logit, mix, D):
    check_scan([(0, 200), (200, 400)], D, xk, gk, logit, mix, batch=(2, 200))


@pytest.mark.parametrize("D", [8, 515, 520, 1024])
@pytest.mark.parametrize("xk,gk", [("bf16", "bf16"), ("f32", "f32")])
def test_scan_channels(D, xk, gk):
    check_scan([(0, 150)], D, xk, gk, True, True, batch=(1, 150))


@pytest.mark.parametrize("T", [4097, 9000])
def test_scan_long(T):
    """Long memory: gates near one carry over many segments."""
    check_scan([(0, T)], 12, "f32", "f32", False, False, batch=(1, T))


@pytest.mark.parametrize("lengths", [[5, 0, 1, 64, 63, 0, 129, 200], [1] * 70, [0, 0, 3], [300], [64, 64, 128], [0],
                                     [1, 700, 2, 0, 0], [2, 5000]])
@pytest.mark.parametrize("xk,gk,D", [("bf16", "bf16", 136), ("f32", "f32", 37)])
def test_scan_packed(lengths, xk, gk, D):
    where = ref.spans(lengths)
    if sum(lengths) == 0:
        where, total = [(0, 0)], 0
        x = torch.zeros(0, D, device="cuda")
        h0 = torch.randn(1, D, device="cuda")
        y, h, saved = kda.scan_varlen_fwd(x, x, torch.zeros(2, dtype=torch.int32, device="cuda"), h0, save="carry")
        assert torch.equal(h, h0) and y.shape == (0, D)
        dh0 = kda.scan_varlen_bwd(x, torch.zeros(2, dtype=torch.int32, device="cuda"), x, saved, x=x, dh_final=h0)[2]
        assert torch.equal(dh0, h0)
        return
    cu = torch.tensor([0] + [b for _, b in where], dtype=torch.int32, device="cuda")
    check_scan(where, D, xk, gk, len(lengths) % 2 == 0, D == 136, cu=cu)


def test_scan_rows_behind_the_last_sequence_stay():
    """A buffer longer than its sequences: the rows behind are neither read into a state nor written."""
    lengths, D, total = [70, 0, 33], 72, 200
    where = ref.spans(lengths)
    cu = torch.tensor([0, 70, 70, 103], dtype=torch.int32, device="cuda")
    check_scan(where, D, "bf16", "f32", False, True, cu=cu, total=total)
    d, _ = scan_data(total, D, 3, False, 5, "bf16", "f32")
    L = kda.load_library()
    y = torch.full((total, D), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, dg = torch.full_like(y, 7.0), torch.full((total, D), 7.0, device="cuda")
    u, us = (torch.full((total, n), 7, dtype=torch.uint8, device="cuda") for n in (D, 3))
    d["x"][103:] = float("nan")
    d["g"][103:] = float("nan")
    d["dy"][103:] = float("nan")
    import ctypes
    form = ctypes.byref(kda.layer.ScanForm(1, 0, 0, 0))
    ws = torch.empty(max(16, kda.scan_workspace_bytes(3, total, D)), dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    hf, dh0 = torch.empty(3, D, device="cuda"), torch.empty(3, D, device="cuda")
    assert L.kda_scan_varlen_fwd(d["x"].data_ptr(), d["g"].data_ptr(), cu.data_ptr(), 3, total, d["h0"].data_ptr(),
                                 y.data_ptr(), hf.data_ptr(), None, u.data_ptr(), us.data_ptr(), D, form,
                                 ws.data_ptr(), ws.numel(), st) == 0
    assert L.kda_scan_varlen_bwd(None, d["g"].data_ptr(), cu.data_ptr(), 3, total, None, None, u.data_ptr(),
                                 us.data_ptr(), d["dy"].data_ptr(), d["dh"].data_ptr(), dx.data_ptr(), dg.data_ptr(),
                                 dh0.data_ptr(), D, form, ws.data_ptr(), ws.numel(), st) == 0
    for t in (y, dx, dg, u, us):
        assert (t[103:] == 7).all()
        assert torch.isfinite(t[:103].float()).all()
    assert torch.isfinite(hf).all() and torch.isfinite(dh0).all() and torch.equal(hf[1], d["h0"][1])


@pytest.mark.parametrize("packed", [False, True])
def test_scan_nan_and_infinity_stay_in_their_sequence_and_channel(packed):
    D, T = 40, 150
    d, _ = scan_data(3 * T, D, 3, False, 8, "f32", "f32")
    x, g, dy = (d[k].reshape(3, T, D).clone() for k in ("x", "g", "dy"))
    x[1, 20, 5], x[1, 149, 6], g[1, 149, 7], dy[1, 0, 8], dy[1, 100, 9] = (float(s) for s in
                                                                        ("inf", "nan", "nan", "inf", "nan"))
    clean = [torch.nan_to_num(t, 0.0, 0.0, 0.0) for t in (x, dy)] + [torch.nan_to_num(g, 0.0, 0.0, float("-inf"))]
    cu = torch.arange(4, dtype=torch.int32, device="cuda") * T

    def both(x, g, dy):
        if packed:
            f = [t.reshape(3 * T, D) for t in (x, g, dy)]
            y, h, s = kda.scan_varlen_fwd(f[0], f[1], cu, d["h0"], save="carry")
            dx, dg, dh0 = kda.scan_varlen_bwd(f[1], cu, f[2], s, x=f[0], h0=d["h0"], dh_final=d["dh"])
            return y.view(3, T, D), h, dx.view(3, T, D), dg.view(3, T, D), dh0
        y, h, s = kda.scan_fwd(x, g, d["h0"], save="carry")
        return (y, h, *kda.scan_bwd(g, dy, s, x=x, h0=d["h0"], dh_final=d["dh"]))

    got, want = both(x, g, dy), both(clean[0], clean[2], clean[1])
    rest = [c for c in range(D) if c not in (5, 6, 7, 8, 9)]
    for a, b in zip(got, want):
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1][..., rest], b[1][..., rest])
    y, h, dx, dg, dh0 = got
    assert not torch.isfinite(y[1, 20:, 5]).any() and torch.equal(y[1, :20, 5], want[0][1, :20, 5])
    assert not torch.isfinite(h[1, [5, 6, 7]]).any()
    assert not torch.isfinite(dx[1, :101, 9]).any() and torch.equal(dx[1, 101:, 9], want[2][1, 101:, 9])
    assert not torch.isfinite(dh0[1, [8, 9]]).any()


def test_scan_offsets_beyond_32_bits():
    """2^31 and more elements; what a tail row holds depends on the rows close before it only."""
    D, T = 65536, 33000
    x = torch.empty((1, T, D), dtype=torch.bfloat16, device="cuda").normal_()
    g = torch.full((1, T, D), -1.0, dtype=torch.bfloat16, device="cuda")
    y, h, saved = kda.scan_fwd(x, g, save="carry")
    t = 192  # e^-128 is behind it
    y2, h2, _ = kda.scan_fwd(x[:, -t:].contiguous(), g[:, -t:].contiguous())
    # both round a value known to 2^-20 of itself or better: at most one step apart
    torch.testing.assert_close(y[:, -64:].float(), y2[:, -64:].float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(h, h2, rtol=1e-5, atol=1e-5)
    dx, dg, dh0 = kda.scan_bwd(g, x, saved, x=x)
    dx2, dg2, _ = kda.scan_bwd(g[:, -t:].contiguous(), x[:, -t:].contiguous(),
                               kda.scan_fwd(x[:, -t:].contiguous(), g[:, -t:].contiguous(), save="carry")[2],
                               x=x[:, -t:].contiguous())
    torch.testing.assert_close(dx[:, -64:].float(), dx2[:, -64:].float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(dg[:, -64:].float(), dg2[:, -64:].float(), rtol=2.0 ** -7, atol=1e-4)


@pytest.mark.parametrize("xk,gk,D", [("bf16", "bf16", 2048), ("f32", "bf16", 37), ("bf16", "f32", 260)])
def test_scan_steps_are_the_scan(xk, gk, D):
    B, T = 3, 70
    d, _ = scan_data(B * T, D, B, True, 9, xk, gk)
    x, g = d["x"].reshape(B, T, D), d["g"].reshape(B, T, D)
    _, h = ref.scan(host(d["x"]), host(d["g"]), host(d["h0"]), [(i * T, (i + 1) * T) for i in range(B)], True, True)[:2]
    y, hf, _ = kda.scan_fwd(x, g, d["h0"], g_logit=True, complement=True)
    s = d["h0"].clone()
    for t in range(T):
        out, s2 = kda.scan_step(x[:, t].contiguous(), g[:, t].contiguous(), s, g_logit=True, complement=True)
        o2, same = kda.scan_step(x[:, t].contiguous(), g[:, t].contiguous(), s, inplace=True, g_logit=True,
                                 complement=True)
        assert same is s and torch.equal(s, s2) and torch.equal(out, o2)
    near(s, h, "f32", "state after the steps")
    near(hf, h, "f32", "state after the scan")


def test_scan_bits_streams_and_graphs():
    """The same bits on every call, on another stream, with a dirty workspace of another call, and replayed from a graph
    among eager work."""
    B, T, D = 2, 1500, 264
    d, _ = scan_data(B * T, D, B, False, 11, "bf16", "bf16")
    x, g, dy = (d[k].reshape(B, T, D) for k in ("x", "g", "dy"))

    def step(ws=None):
        y, h, s = kda.scan_fwd(x, g, d["h0"], save="carry", workspace=ws)
        y8, _, s8 = kda.scan_fwd(x, g, d["h0"], save="ckpt8", workspace=ws)
        return (y, h, *kda.scan_bwd(g, dy, s, x=x, h0=d["h0"], dh_final=d["dh"], workspace=ws), y8,
                *kda.scan_bwd(g, dy, s8, dh_final=d["dh"], workspace=ws))

    want = [t.clone() for t in step()]
    ws = torch.full((max(16, kda.scan_workspace_bytes(B, B * T, D)),), 255, dtype=torch.uint8, device="cuda")
    for got in (step(), step(ws), step(ws)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    keep = x.clone()
    for i in range(4):
        x.copy_(keep if i % 2 == 0 else torch.zeros_like(keep))
        graph.replay()
        fresh = step()  # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, fresh))
        assert torch.equal(out[0], want[0]) == (i % 2 == 0)


def test_scans_on_two_streams_at_once():
    """Workgroups of one call wait only for others of that call: two that share the card end with the bits of each alone."""
    B, T, D = 2, 8192, 1024
    data = [scan_data(B * T, D, B, False, seed, "bf16", "bf16")[0] for seed in (31, 32)]

    def step(d):
        x, g, dy = (d[k].reshape(B, T, D) for k in ("x", "g", "dy"))
        y, h, s = kda.scan_fwd(x, g, d["h0"], save="carry")
        return (y, h, *kda.scan_bwd(g, dy, s, x=x, h0=d["h0"], dh_final=d["dh"]))

    want = [step(d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[], []]
    for _ in range(4):
        for i, d in enumerate(data):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(d))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.parametrize("ckpt8", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_scan_autograd(ckpt8, packed):
    B, T, D = 2, 90, 48
    d, h = scan_data(B * T, D, B, True, 12, "f32", "f32")
    where = [(i * T, (i + 1) * T) for i in range(B)]
    leaves = [d["x"], d["g"], d["h0"]]
    if not packed:
        leaves = [leaves[0].reshape(B, T, 6, 8), leaves[1].reshape(B, T, 6, 8), leaves[2].reshape(B, 6, 8)]
    x, g, h0 = (t.clone().requires_grad_() for t in leaves)
    if packed:
        cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
        y, hf = kda.VarlenGatedScan.apply(x, g, cu, h0, True, True, ckpt8)
    else:
        y, hf = kda.GatedScan.apply(x, g, h0, True, True, ckpt8)
    ((y.reshape(-1, D) * d["dy"]).sum() + (hf.reshape(B, D) * d["dh"]).sum()).backward()
    dx, dg, dh0 = ref.scan_grad(h["x"], h["g"], h["h0"], h["dy"], h["dh"], where, True, True)
    near(x.grad, dx, "f32", "dx")
    near(h0.grad, dh0, "f32", "dh0")
    if ckpt8:
        u = ref.scan(h["x"], h["g"], h["h0"], where, True, True)[2]
        _, e, _ = ref.scan_grad(h["x"], h["g"], h["h0"], h["dy"], h["dh"], where, True, True, u=np.ones_like(u[0]))
        # u is kept to 2^-4 of itself, or to 2^-10 of a scale of at most amax / 224
        top = np.abs(u[0]).reshape(B * T, -1)
        amax = np.stack([np.abs(top[:, 32 * i:32 * i + 32]).max(1) for i in range(2)], 1).repeat(32, 1)[:, :D]
        near(g.grad, (dg[0], dg[1] + (2.0 ** -4 * top + amax / 224 * 2.0 ** -10) * np.abs(e[0]) * 1.01), "f32", "dg")
    else:
        near(g.grad, dg, "f32", "dg")


# ----------------------------------------------------------------- head norm with rotation

def qk_data(tokens, Hq, Hk, D, rot, kind, weight, seed, pos=None, gk=None):
    rng = np.random.default_rng(seed)
    d = {"q": dev(rng.normal(size=(tokens, Hq, D)), kind), "k": dev(rng.normal(size=(tokens, Hk, D)) * 3, kind),
         "dq": dev(rng.normal(size=(tokens, Hq, D)), gk or kind), "dk": dev(rng.normal(size=(tokens, Hk, D)), gk or kind),
         "wq": dev(1 + 0.2 * rng.normal(size=D)) if weight else None,
         "wk": dev(1 + 0.2 * rng.normal(size=D)) if weight else None, "pos": None, "freqs": None}
    angle = np.zeros((tokens, 0))
    if rot:
        at = np.arange(tokens) * 37 if pos is None else pos
        d["pos"] = torch.from_numpy(np.asarray(at)).cuda()
        f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
        d["freqs"] = torch.from_numpy(f).cuda()
        angle = np.asarray(at, np.float64)[:, None] * f
    return d, angle


def check_qk(tokens, Hq, Hk, D, rot, kind="bf16", norm="rms", eps=1e-5, weight=True, interleaved=False, seed=1, pos=None,
             gk=None, view=None, packed=False):
    d, angle = qk_data(tokens, Hq, Hk, D, rot, kind, weight, seed, pos, gk)
    q, k = view(d["q"], d["k"]) if view else (d["q"], d["k"])
    form = {"weight_q": d["wq"], "weight_k": d["wk"], "pos": d["pos"], "freqs": d["freqs"], "norm": norm, "eps": eps,
            "interleaved": interleaved}
    qo, ko, none = kda.qk_norm_rope_fwd(q, k, **form)
    assert none is None and qo.is_contiguous() and qo.dtype == TYPES[kind]
    raw, at = (q, k), (host(q), host(k))
    if packed:
        q2, k2, raw = kda.qk_norm_rope_fwd(q, k, ckpt8=True, **form)
        assert torch.equal(q2, qo) and torch.equal(k2, ko), "what is kept changed the result"
        for p, t in zip(raw, (q, k)):
            want = kda.ckpt8_pack(t.contiguous())
            assert torch.equal(p.codes, want.codes) and torch.equal(p.scales, want.scales)
        at = tuple(host(kda.ckpt8_unpack(p)) for p in raw)
        qo, ko, _ = kda.qk_norm_rope_fwd(*raw, **form)
    grads = kda.qk_norm_rope_bwd(*raw, d["dq"], d["dk"], **form)
    for i, (x, o, w, dy, n) in enumerate(((at[0], qo, d["wq"], d["dq"], "q"), (at[1], ko, d["wk"], d["dk"], "k"))):
        y, dx, dw = ref.qk_norm(x, None if w is None else host(w), angle, norm == "rms", np.float32(eps), interleaved,
                                host(dy))
        near(o, y, kind, n)
        near(grads[i], dx, kind, "d" + n)
        assert grads[i].dtype == TYPES[kind] and (grads[2 + i] is None) == (w is None)
        if w is not None:
            near(grads[2 + i], dw, "f32", "dw" + n)


@pytest.mark.parametrize("tokens,Hq,Hk", [(1, 1, 1), (3, 2, 1), (33, 4, 4), (130, 16, 16), (7, 31, 5)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_qk_heads_and_tokens(tokens, Hq, Hk, D, kind):
    check_qk(tokens, Hq, Hk, D, D, kind, interleaved=Hq % 2 == 0)


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 112, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,eps,weight", [("l2", 0.0, False), ("rms", 1e-6, True)])
def test_qk_rotations(rot, interleaved, norm, eps, weight):
    check_qk(19, 3, 2, 128, rot, norm=norm, eps=eps, weight=weight, interleaved=interleaved)


@pytest.mark.parametrize("kind,gk", [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("packed", [False, True])
def test_qk_types(kind, gk, packed):
    check_qk(41, 5, 3, 128, 64, kind, gk=gk, packed=packed)
    check_qk(41, 5, 3, 64, 32, kind, gk=gk, packed=packed, interleaved=True, norm="l2", weight=False)


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 32), (64, 48), (128, 16), (128, 48), (128, 64), (128, 96)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_qk_halves_of_part_of_the_head(D, rot, kind):
    check_qk(21, 3, 2, D, rot, kind, packed=True)


@pytest.mark.parametrize("D,rot", [(64, 32), (128, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("ckpt8", [False, True])
def test_qk_large_calls_have_the_bits_of_small_ones(D, rot, ckpt8):
    """Rows of calls of more than 128 MiB go past the caches; a row's result does not depend on that."""
    tokens, Hq, Hk, n = 36000 * 128 // D, 5, 3, 50
    d, _ = qk_data(tokens, Hq, Hk, D, rot, "bf16", False, 9)
    form = {"freqs": d["freqs"], "eps": 1e-6}
    q8 = kda.qk_norm_rope_fwd(d["q"], d["k"], pos=d["pos"], ckpt8=ckpt8, **form)
    dq = kda.qk_norm_rope_bwd(*(q8[2] if ckpt8 else (d["q"], d["k"])), d["dq"], d["dk"], pos=d["pos"], **form)
    for at in (0, tokens // 2, tokens - n):
        part = {k: d[k][at:at + n] for k in ("q", "k", "dq", "dk", "pos")}
        s8 = kda.qk_norm_rope_fwd(part["q"], part["k"], pos=part["pos"], ckpt8=ckpt8, **form)
        raw = s8[2] if ckpt8 else (part["q"], part["k"])
        ds = kda.qk_norm_rope_bwd(*raw, part["dq"], part["dk"], pos=part["pos"], **form)
        for big, small in (*zip(q8[:2], s8[:2]), *zip(dq[:2], ds[:2])):
            assert torch.equal(big[at:at + n], small)
        if ckpt8:
            for big, small in zip(q8[2], s8[2]):
                assert torch.equal(big.codes[at:at + n], small.codes)
                assert torch.equal(big.scales[at:at + n], small.scales)


@pytest.mark.parametrize("pos", [np.arange(11, dtype=np.int64) * 10 ** 8, np.arange(11, dtype=np.int32) - 5,
                                 np.full(11, 2 ** 31 - 1, np.int32), np.full(11, 1048575, np.int64)])
def test_qk_far_and_negative_positions(pos):
    check_qk(11, 2, 2, 64, 64, "f32", pos=pos)


def test_qk_columns_of_a_projection():
    def view(q, k):
        rows = torch.randn(q.shape[0], 1024, device="cuda").to(q.dtype)
        rows[:, 256:512], rows[:, 512:640] = q.flatten(1), k.flatten(1)
        return rows[:, 256:512].view(-1, 2, 128), rows[:, 512:640].view(-1, 1, 128)
    check_qk(29, 2, 1, 128, 128, view=view)
    check_qk(29, 2, 1, 128, 32, view=view, packed=True)


def test_qk_leading_dimensions_and_one_weight():
    d, angle = qk_data(12, 2, 2, 64, 64, "f32", True, 4)
    q, k, dq, dk = (d[n].view(3, 4, 2, 64) for n in ("q", "k", "dq", "dk"))
    form = dict(pos=d["pos"].view(3, 4), freqs=d["freqs"], weight_k=d["wk"], norm="l2")
    qo, ko, _ = kda.qk_norm_rope_fwd(q, k, **form)
    gq, gk, none, dwk = kda.qk_norm_rope_bwd(q, k, dq, dk, **form)
    assert none is None and qo.shape == q.shape
    y, dx, _ = ref.qk_norm(host(d["q"]), None, angle, False, 0.0, False, host(d["dq"]))
    near(qo, y, "f32", "q")
    near(gq, dx, "f32", "dq")
    y, dx, dw = ref.qk_norm(host(d["k"]), host(d["wk"]), angle, False, 0.0, False, host(d["dk"]))
    near(ko, y, "f32", "k")
    near(gk, dx, "f32", "dk")
    near(dwk, dw, "f32", "dwk")


def test_qk_gradient_of_absent_weights_is_that_of_ones():
    import ctypes
    d, angle = qk_data(70, 2, 1, 64, 32, "f32", False, 9)
    out = [torch.empty_like(d["q"]), torch.empty_like(d["k"]), *(torch.full((64,), 7.0, device="cuda") for _ in range(2))]
    ws = torch.empty(kda.qk_norm_rope_workspace_bytes(70, 2, 1, 64), dtype=torch.uint8, device="cuda")
    form = kda.layer.QkNormForm(0, 0.0, 32, 0, 8)
    rc = kda.load_library().kda_qknorm_bwd(
        d["q"].data_ptr(), d["k"].data_ptr(), None, None, 128, 64, None, None, d["pos"].data_ptr(), d["freqs"].data_ptr(),
        d["dq"].data_ptr(), d["dk"].data_ptr(), *(t.data_ptr() for t in out), 70, 2, 1, 64, 0, 0, ctypes.byref(form),
        ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for i, n in enumerate("qk"):
        _, dx, dw = ref.qk_norm(host(d[n]), None, angle, False, 0.0, False, host(d["d" + n]))
        near(out[i], dx, "f32", "d" + n)
        near(out[2 + i], dw, "f32", "dw" + n)


def test_qk_rows_of_any_size():
    """Zero rows stay zero; rows whose squares overflow or vanish in float32 are normed all the same; infinity and
    NaN stay in their row."""
    rng = np.random.default_rng(6)
    base = rng.normal(size=(8, 2, 64))
    size = np.array([0.0, 1e-30, 1e30, 1e38 / 8, 2.0 ** -100, 1.0, 1.0, 1.0])[:, None, None]
    q = dev(base * size, "f32")
    q[5, 0, 3], q[6, 1, 9] = float("inf"), float("nan")
    k = dev(base, "f32")
    qo, ko, _ = kda.qk_norm_rope_fwd(q, k)
    assert (qo[0] == 0).all() and torch.isnan(qo[5, 0]).all() and torch.isnan(qo[6, 1]).all()
    assert torch.isfinite(qo[5, 1]).all() and torch.isfinite(qo[6, 0]).all()
    keep = [1, 2, 3, 4, 7]
    x = host(q)[keep]
    y = x / np.abs(x).max(-1, keepdims=True)
    y = y / np.sqrt((y * y).sum(-1, keepdims=True))
    np.testing.assert_allclose(host(qo)[keep], y, rtol=32 * ref.U, atol=0)
    dq, _, _, _ = kda.qk_norm_rope_bwd(q, k, torch.ones_like(q), torch.ones_like(k))
    assert (dq[0] == 0).all() and torch.isfinite(dq[[2, 3, 4, 7]]).all()


def test_qk_many_tokens_sum_in_order():
    """More rows than one pass of the grid; the weights' sums give the same bits on every call and in a graph."""
    d, angle = qk_data(9001, 4, 2, 64, 32, "bf16", True, 7)
    form = {"weight_q": d["wq"], "weight_k": d["wk"], "pos": d["pos"], "freqs": d["freqs"], "norm": "rms", "eps": 1e-6}

    def step():
        q, k, raw = kda.qk_norm_rope_fwd(d["q"], d["k"], ckpt8=True, **form)
        return (q, k, *kda.qk_norm_rope_bwd(*raw, d["dq"], d["dk"], **form))

    want = [t.clone() for t in step()]
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        fresh = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(a, b) for a, b in zip(fresh, want))
    x = [host(kda.ckpt8_unpack(p)) for p in kda.qk_norm_rope_fwd(d["q"], d["k"], ckpt8=True, **form)[2]]
    for i, (w, dy) in enumerate(((d["wq"], d["dq"]), (d["wk"], d["dk"]))):
        _, dx, dw = ref.qk_norm(x[i], host(w), angle, True, np.float32(1e-6), False, host(dy))
        near(want[2 + i], dx, "bf16", "dx")
        near(want[4 + i], dw, "f32", "dw")


# ----------------------------------------------------------------- together, as a layer uses them

@pytest.mark.parametrize("ckpt8", [False, True])
def test_layer_forward_and_backward(ckpt8):
    """Columns of a projection -> norm and rotation -> recurrence, the values smoothed by a gated scan; gradients against the
    64-bit forms of all of it, at the values that the checkpoints stand for."""
    B, T, H, D = 2, 130, 2, 64
    rng = np.random.default_rng(21)
    rows = dev(rng.normal(size=(B, T, 3 * H * D)), "bf16")
    q0, k0, v0 = (rows[..., i * H * D:(i + 1) * H * D].view(B, T, H, D) for i in range(3))
    gv = dev(rng.normal(size=(B, T, H, D)) - 2, "bf16")
    g = dev(-np.logaddexp(rng.normal(size=(B, T, H, D)), 0))
    beta = dev(1 / (1 + np.exp(-rng.normal(size=(B, T, H)))))
    wq, wk = dev(1 + 0.1 * rng.normal(size=D)), dev(1 + 0.1 * rng.normal(size=D))
    pos = torch.arange(T, device="cuda").repeat(B, 1)
    freqs = torch.from_numpy(10000.0 ** (-np.arange(0, D, 2) / D)).cuda()
    s0, d_o = dev(0.1 * rng.normal(size=(B, H, D, D))), dev(rng.normal(size=(B, T, H, D)))
    leaves = [t.clone().requires_grad_() for t in (q0, k0, v0.contiguous(), gv, g, beta, s0, wq, wk)]
    q, k, v, gate, gg, bb, ss, a, b = leaves
    vs, _ = kda.GatedScan.apply(v, gate, None, True, True, ckpt8)
    o, sf = kda.NormChunkKDA.apply(q, k, vs, gg, bb, ss, a, b, pos, freqs, "l2", 1e-6, False, ckpt8)
    o.backward(d_o)
    assert all(t.grad is not None and torch.isfinite(t.grad).all() and t.grad.dtype == t.dtype for t in leaves)

    # forward: norm and rotation against their 64-bit form; then the oracle on the rows as they are handed over, in bf16
    # (the recurrence's bar is for the inputs it gets: half a step of q, 2^-8 |q|, moves o by up to 2^-8 sum_i |q_i S_ij|,
    # which is not small beside o)
    flat = (B * T, H, D)
    angle = host(pos).reshape(-1)[:, None] * host(freqs)
    cu = np.array([0, T, 2 * T])
    form = {"weight_q": wq, "weight_k": wk, "pos": pos, "freqs": freqs, "norm": "l2", "eps": 1e-6}
    normed = kda.qk_norm_rope_fwd(q0, k0, **form)[:2]
    for got, x, w in zip(normed, (q, k), (wq, wk)):
        near(got, ref.qk_norm(host(x).reshape(flat), host(w), angle, False, 1e-6, False), "bf16", "normed")
    qn, kn = (host(t).reshape(flat) for t in normed)
    want, _ = oracle.forward(qn, kn, host(vs).reshape(flat), host(g).reshape(flat), host(beta).reshape(B * T, H), cu,
                             s0=host(s0))
    off = oracle.rel_err(host(o).reshape(want.shape), want)
    assert off <= 2e-2
    # backward: at the kept values
    kept = [kda.ckpt8_unpack(kda.ckpt8_pack(t.detach().contiguous())) if ckpt8 else t.detach() for t in (q, k, vs)]
    qr, kr, _ = kda.qk_norm_rope_fwd(kept[0], kept[1], **form)
    r = oracle.backward(host(qr).reshape(flat), host(kr).reshape(flat), host(kept[2]).reshape(flat), host(g).reshape(flat),
                        host(beta).reshape(B * T, H), cu, host(d_o).reshape(flat), s0=host(s0))
    for got, key in ((gg.grad, "dg"), (bb.grad, "dbeta"), (ss.grad, "ds0")):
        assert oracle.rel_err(host(got).reshape(r[key].shape), r[key]) <= 1e-3, key
    for x, w, got, dw, key in ((kept[0], wq, q.grad, a.grad, "dq"), (kept[1], wk, k.grad, b.grad, "dk")):
        off = 1e-3 * np.sqrt(np.mean(r[key] ** 2))  # the recurrence's gradient is within this of the oracle's
        xh = host(x).reshape(flat)
        _, dx, dwv = ref.qk_norm(xh, host(w), angle, False, 1e-6, False, r[key])
        size = 1 / np.sqrt((xh * xh).sum(-1, keepdims=True) + 1e-6)
        # dx is linear in it: turned back (sqrt 2), times w and r, less a projection (at most its length, sqrt(D) entries)
        room = size * np.abs(host(w)).max() * off * np.sqrt(2) * (1 + np.sqrt(D)) + np.zeros_like(dx[0])
        near(got, (dx[0], dx[1] + room), "bf16", key)
        near(dw, (dwv[0], dwv[1] + off * np.sqrt(2) * np.abs(xh * size).sum((0, 1))), "f32", "w of " + key)


def test_layer_prefill_then_steps():
    """Prefill of packed prompts, then single tokens from its states: norm, rotation and gated scan agree with one pass over the
    whole sequences."""
    H, D, more = 2, 64, 3
    lengths = [5, 70, 1]
    total = sum(lengths) + more * len(lengths)
    rng = np.random.default_rng(31)
    full = [n + more for n in lengths]
    q, k, v, g = (dev(rng.normal(size=(total, H, D)), "bf16") for _ in range(4))
    freqs = torch.from_numpy(10000.0 ** (-np.arange(0, D, 2) / D)).cuda()
    pos = torch.cat([torch.arange(n) for n in full]).cuda()
    cu_full = torch.tensor(np.concatenate([[0], np.cumsum(full)]), dtype=torch.int32, device="cuda")
    qo, ko, _ = kda.qk_norm_rope_fwd(q, k, pos=pos, freqs=freqs)
    y, h, _ = kda.scan_varlen_fwd(v, g, cu_full, g_logit=True)
    at = cu_full.tolist()
    first = torch.cat([torch.arange(at[i], at[i] + n) for i, n in enumerate(lengths)]).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    y1, state, _ = kda.scan_varlen_fwd(v[first], g[first], cu, g_logit=True)
    q1, k1, _ = kda.qk_norm_rope_fwd(q[first], k[first], pos=pos[first], freqs=freqs)
    assert torch.equal(q1, qo[first]) and torch.equal(k1, ko[first])
    # two orders of the same sums of at most 73 terms, each rounded once to bf16: a step apart at most
    torch.testing.assert_close(y1.float(), y[first].float(), rtol=2.0 ** -7, atol=2.0 ** -20)
    for s in range(more):
        rows = torch.tensor([at[i] + n + s for i, n in enumerate(lengths)], device="cuda")
        out, state = kda.scan_step(v[rows], g[rows], state, g_logit=True)
        qs, ks, _ = kda.qk_norm_rope_fwd(q[rows], k[rows], pos=pos[rows], freqs=freqs)
        assert torch.equal(qs, qo[rows]) and torch.equal(ks, ko[rows])
        torch.testing.assert_close(out.float(), y[rows].float(), rtol=2.0 ** -7, atol=2.0 ** -20)
    torch.testing.assert_close(state, h, rtol=1e-5, atol=1e-5)
