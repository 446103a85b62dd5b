"""The operators around the recurrence at the edges of what their calls allow: buffers longer than their sequences, views at
any offset, 16-bit gates in training, positions and rows of any size."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import gated_delta_rule_65_amd as kda
from tests import layer_ref as ref
from tests.test_gpu_layer import TYPES, dev, host, near, scan_data

pytestmark = pytest.mark.gpu


def dirty(*shapes):
    """Leaves NaN behind in the memory that buffers of these shapes and types get next."""
    held = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(4)]
    torch.cuda.synchronize()
    del held


# ----------------------------------------------------------------- rows behind the last sequence

@pytest.mark.parametrize("ckpt8", [False, True])
@pytest.mark.parametrize("xk,gk,D", [("bf16", "f32", 72), ("f32", "bf16", 37), ("bf16", "bf16", 1)])
@pytest.mark.parametrize("lengths,total", [([70, 0, 33], 200), ([5], 6), ([0, 0], 9), ([], 3), ([64], 64), ([130, 3], 133)])
def test_scan_autograd_gives_zeros_behind_the_last_sequence(lengths, total, xk, gk, D, ckpt8):
    where, N, used = ref.spans(lengths) if lengths else [], len(lengths), sum(lengths)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    d, h = scan_data(total, D, N, True, 3, xk, gk)
    x, g, h0 = (d[k].clone().requires_grad_() for k in ("x", "g", "h0"))
    with torch.no_grad():
        for t in (x, g):
            t[used:] = float("nan")
    dirty(((total, D), TYPES[xk]), ((total, D), TYPES[gk]), ((total, D), torch.float32))
    y, hf = kda.VarlenGatedScan.apply(x, g, cu, h0, True, True, ckpt8)
    assert (y[used:] == 0).all()
    dy = d["dy"].clone()
    dy[used:] = float("nan")
    dirty(((total, D), TYPES[xk]), ((total, D), TYPES[gk]), ((total, D), torch.float32))
    torch.autograd.backward((y, hf), (dy, d["dh"]))
    assert (x.grad[used:] == 0).all() and (g.grad[used:] == 0).all()
    (want, _), (dx, _) = ref.scan(h["x"], h["g"], h["h0"], where, True, True)[0], ref.scan_grad(
        h["x"], h["g"], h["h0"], h["dy"], h["dh"], where, True, True)[0]
    for got, full in ((y, want), (x.grad, dx)):
        torch.testing.assert_close(got[:used].double().cpu(), torch.from_numpy(full[:used]), rtol=2.0 ** -7, atol=1e-4)
    assert torch.isfinite(g.grad).all() and torch.isfinite(h0.grad).all() and torch.isfinite(hf).all()


# ----------------------------------------------------------------- views at any offset

@pytest.mark.parametrize("C", [37, 36])
def test_gradients_that_come_as_views_at_any_offset(C):
    """A concatenation hands its backward pass contiguous views that begin anywhere."""
    torch.manual_seed(3)
    x, g = torch.randn(2, 3, C, device="cuda").bfloat16(), (-torch.rand(2, 3, C, device="cuda")).bfloat16()
    grads = []
    for joined in (False, True):
        a, b = x.clone().requires_grad_(), g.clone().requires_grad_()
        y = [kda.GatedScan.apply(a[i:i + 1].clone(), b[i:i + 1].clone())[0] for i in range(2)]
        cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
        z = [kda.VarlenGatedScan.apply(a[i].clone(), b[i].clone(), cu)[0] for i in range(2)]
        w = torch.arange(12 * C, device="cuda").view(4, 3, C).bfloat16()
        if joined:
            torch.cat([*y, *(t[None] for t in z)]).backward(w)
        else:
            torch.autograd.backward([*y, *z], [w[0:1].clone(), w[1:2].clone(), w[2].clone(), w[3].clone()])
        grads.append((a.grad, b.grad))
    assert all(torch.equal(*pair) for pair in zip(*grads))


@pytest.mark.parametrize("norm", [False, True])
def test_layer_gradients_that_come_as_views_at_any_offset(norm):
    torch.manual_seed(4)
    B, T, H, D = 1, 5, 1, 64
    q, k, v = (torch.randn(B, T, H, D, device="cuda") * 0.2 for _ in range(3))
    g, beta = -torch.rand(B, T, H, D, device="cuda"), torch.rand(B, T, H, device="cuda")
    f = kda.NormChunkKDA if norm else kda.ChunkKDA
    grads = []
    for joined in (False, True):
        leaves = [t.clone().requires_grad_() for t in (q, k, v, g, beta)]
        o, s = f.apply(*leaves)
        w, ws = torch.randn(1 + o.numel(), generator=torch.Generator().manual_seed(1)).cuda(), torch.ones_like(s)
        if joined:
            torch.autograd.backward([torch.cat([torch.ones(1, device="cuda"), o.flatten()]),
                                     torch.cat([torch.ones(1, device="cuda"), s.flatten()])],
                                    [w, torch.ones(1 + s.numel(), device="cuda")])
        else:
            torch.autograd.backward([o, s], [w[1:].clone().view(o.shape), ws])
        grads.append([t.grad for t in leaves])
    assert all(torch.equal(*pair) for pair in zip(*grads))


# ----------------------------------------------------------------- 16-bit gates in training

@pytest.mark.parametrize("norm", [False, True])
def test_layer_trains_with_16_bit_gates(norm):
    """What the forward pass takes the backward pass takes: gradients at the gates' values, in their type."""
    B, T, H, D = 1, 70, 2, 64
    rng = np.random.default_rng(5)
    q, k, v = (dev(0.2 * rng.normal(size=(B, T, H, D)), "bf16") for _ in range(3))
    g, beta = dev(-rng.random(size=(B, T, H, D)), "bf16"), dev(rng.random(size=(B, T, H)), "bf16")
    f = kda.NormChunkKDA if norm else kda.ChunkKDA
    grads = []
    for wide in (False, True):
        leaves = [t.clone().requires_grad_() for t in (q, k, v, g.float() if wide else g, beta.float() if wide else beta)]
        o, _ = f.apply(*leaves)
        o.backward(torch.ones_like(o))
        grads.append([t.grad for t in leaves])
        assert all(t.grad.dtype == t.dtype for t in leaves)
    assert all(torch.equal(a, b.to(a.dtype)) for a, b in zip(*grads))


# ----------------------------------------------------------------- positions and rows of any size

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651")


def angles(pos, freqs):
    """pos * freq mod a turn, in rational arithmetic up to the last rounding."""
    out = np.zeros((len(pos), len(freqs)))
    for i, p in enumerate(pos):
        for j, f in enumerate(freqs):
            turns = int(p) * Fraction(float(f)) / (2 * PI)
            out[i, j] = float((turns - round(turns)) * 2 * PI)
    return out


FAR = [0, 1, -1, 2 ** 28, 2 ** 30 + 1, 2 ** 31 - 1, 2 ** 36 - 5, 2 ** 40, -2 ** 40 - 1, 2 ** 50 + 3, 2 ** 53 + 1, -2 ** 53 - 1,
       2 ** 62 + 12345, 2 ** 63 - 1, -2 ** 63]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 12])
@pytest.mark.parametrize("kind", [np.int64, np.int32])
def test_qk_any_position_keeps_its_angle(kind, scale, interleaved):
    pos = np.array([p for p in FAR if np.iinfo(kind).min <= p <= np.iinfo(kind).max], kind)
    n, H, D = len(pos), 2, 64
    rng = np.random.default_rng(8)
    q, k, dq, dk = (dev(rng.normal(size=(n, H, D))) for _ in range(4))
    f = scale * 10000.0 ** (-np.arange(0, D, 2) / D)
    angle = angles(pos, f)
    form = {"pos": torch.from_numpy(pos).cuda(), "freqs": torch.from_numpy(f).cuda(), "eps": 1e-6, "interleaved": interleaved}
    out = kda.qk_norm_rope_fwd(q, k, **form)
    grads = kda.qk_norm_rope_bwd(q, k, dq, dk, **form)
    for i, (x, d) in enumerate(((q, dq), (k, dk))):
        y, dx, _ = ref.qk_norm(host(x), None, angle, False, np.float32(1e-6), interleaved, host(d))
        near(out[i], y, "f32", "y")
        near(grads[i], dx, "f32", "dx")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_qk_rows_of_the_largest_size(D, norm):
    """Rows whose length is beyond float32 altogether are normed as closely as others, both ways."""
    rng = np.random.default_rng(9)
    size = np.linspace(0.9, 1.0, 4001).astype(np.float32) * np.float32(3.4e38)
    r = 1 / (size.astype(float) * np.sqrt(D if norm == "l2" else 1))
    size = size[np.argsort(-np.abs(r.astype(np.float32) / r - 1))[:40]]  # whose reciprocal length rounds worst as one float
    q = dev(size[:, None, None] * rng.choice([-1.0, 1.0], size=(40, 1, D)))
    k = dev(1e30 * rng.normal(size=(40, 1, D)))
    dq, dk = (dev(2.0 ** 60 * rng.normal(size=(40, 1, D))) for _ in range(2))
    w = dev(1 + 0.2 * rng.normal(size=D))
    out = kda.qk_norm_rope_fwd(q, k, weight_q=w, weight_k=w, norm=norm)
    grads = kda.qk_norm_rope_bwd(q, k, dq, dk, weight_q=w, weight_k=w, norm=norm)
    for i, (x, d) in enumerate(((q, dq), (k, dk))):
        y, dx, dw = ref.qk_norm(host(x), host(w), np.zeros((40, 0)), norm == "rms", 0.0, False, host(d))
        near(out[i], y, "f32", "y")
        near(grads[i], dx, "f32", "dx")
        near(grads[2 + i], dw, "f32", "dw")


# ----------------------------------------------------------------- rows read an element at a time begin anywhere

@pytest.mark.parametrize("xk,gk", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_scan_of_odd_channels_takes_views_at_any_offset(xk, gk):
    """Channel counts that are no multiple of 4 are read an element at a time: a row of a larger tensor is taken as it is."""
    B, T, D = 1, 130, 37
    d, _ = scan_data(3 * T, D, 3, False, 6, xk, gk)
    d["x"], d["g"], d["dy"] = (d[n].view(3, T, D) for n in ("x", "g", "dy"))
    part = {n: t[1:2] for n, t in d.items()}
    assert any(t.data_ptr() % 16 for t in part.values())
    whole = {n: t.clone() for n, t in part.items()}
    results = []
    for p in (part, whole):
        for save in ("carry", "ckpt8"):
            y, h, saved = kda.scan_fwd(p["x"], p["g"], p["h0"], save=save)
            grads = kda.scan_bwd(p["g"], p["dy"], saved, x=p["x"], h0=p["h0"], dh_final=p["dh"])
            results.append((y, h, *grads))
        out, state = kda.scan_step(p["x"][:, 5], p["g"][:, 5], p["h0"])
        results.append((out, state))
    for a, b in zip(results[:3], results[3:]):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_ckpt8_of_odd_rows_takes_views_at_any_offset(kind):
    x = torch.randn(5, 37, device="cuda").to(TYPES[kind])
    p = kda.ckpt8_pack(x)
    part = kda.ckpt8_pack(x[1:4])
    assert torch.equal(part.codes, p.codes[1:4]) and torch.equal(part.scales, p.scales[1:4])
    view = kda.Packed8(p.codes[1:4], p.scales[1:4], p.dtype)
    assert torch.equal(kda.ckpt8_unpack(view), kda.ckpt8_unpack(p)[1:4])


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_qk_positions_and_frequencies_begin_anywhere(kind):
    q = torch.randn(9, 2, 64, device="cuda")
    pos = torch.arange(20, device="cuda", dtype=kind)
    f = 10000.0 ** (-torch.arange(0, 66, 2, dtype=torch.float64, device="cuda") / 64)
    for at in (1, 2, 3):
        a = kda.qk_norm_rope_fwd(q, q, pos=pos[at:at + 9], freqs=f[1:])
        b = kda.qk_norm_rope_fwd(q, q, pos=pos[at:at + 9].clone(), freqs=f[1:].clone())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ----------------------------------------------------------------- large calls

def scan_both(x, g, dy, cu, h0, dh, save):
    if cu is None:
        y, h, saved = kda.scan_fwd(x, g, h0, save=save, g_logit=True, complement=True)
        grads = kda.scan_bwd(g, dy, saved, x=x, h0=h0, dh_final=dh, g_logit=True, complement=True)
    else:
        y, h, saved = kda.scan_varlen_fwd(x, g, cu, h0, save=save, g_logit=True, complement=True)
        grads = kda.scan_varlen_bwd(g, cu, dy, saved, x=x, h0=h0, dh_final=dh, g_logit=True, complement=True)
    return (y, *grads[:2]), (h, grads[2]), saved


@pytest.mark.parametrize("save", ["carry", "ckpt8"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("xk,gk,blocks", [("bf16", "bf16", 22), ("bf16", "f32", 17), ("f32", "bf16", 13), ("f32", "f32", 11)])
def test_scan_large_calls_have_the_bits_of_small_ones(xk, gk, blocks, packed, save):
    """Rows of calls of more than 128 MiB go past the caches; a sequence's results do not depend on that.  Packed rows are cut
    where sequences begin at whole blocks of 64 segments, so that sums are taken in the same order."""
    D, rows = 256, 4096 * blocks + (0 if packed else 4)  # batches end inside a segment
    assert rows * D * ((4 if xk == "bf16" else 8) + (2 if gk == "bf16" else 4)) > 1 << 27
    torch.manual_seed(blocks)
    x, dy = (torch.randn(rows, D, device="cuda").to(TYPES[xk]) for _ in range(2))
    g = (torch.randn(rows, D, device="cuda") * 1.5 - 2).to(TYPES[gk])
    if packed:
        lengths = [1000, 3096, 5, 0, 4091, *[4096] * (blocks - 6), 9000, 3000, 1, 287, 0, 4096]
        cuts = np.cumsum([0, *lengths])
        assert cuts[-1] == rows and cuts[-2] == rows - 4096
        cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        N = len(lengths)
        parts = [(0, 2, 0, 4096), (2, 5, 4096, 8192), (N - 6, N - 1, rows - 4 * 4096, rows - 4096),
                 (N - 1, N, rows - 4096, rows)]  # sequences and rows of each
    else:
        N, T = 4, rows // 4
        cu, parts = None, [(0, 1, 0, T), (3, 4, 3 * T, 4 * T)]
    h0, dh = torch.randn(N, D, device="cuda"), torch.randn(N, D, device="cuda")
    shape = (rows, D) if packed else (N, T, D)
    large = scan_both(x.view(shape), g.view(shape), dy.view(shape), cu, h0, dh, save)
    for i, j, a, b in parts:
        part = [t[a:b] if packed else t[a:b][None] for t in (x, g, dy)]
        small = scan_both(*part, (cu[i:j + 1] - cu[i]).contiguous() if packed else None, h0[i:j], dh[i:j], save)
        for s, t in zip(large[0], small[0]):
            assert torch.equal(s.view(rows, D)[a:b], t.view(b - a, D))
        for s, t in zip(large[1], small[1]):
            assert torch.equal(s[i:j], t)
        if save == "ckpt8":
            assert torch.equal(large[2].codes[a:b], small[2].codes) and torch.equal(large[2].scales[a:b], small[2].scales)


@pytest.mark.parametrize("D,rot", [(64, 32), (128, 64), (128, 32), (128, 0)])
@pytest.mark.parametrize("ckpt8", [False, True])
def test_qk_large_fp32_calls_have_the_bits_of_small_ones(D, rot, ckpt8):
    tokens, Hq, Hk, n = 20000 * 128 // D, 5, 3, 50
    torch.manual_seed(D + rot)
    q, dq = (torch.randn(tokens, Hq, D, device="cuda") for _ in range(2))
    k, dk = (torch.randn(tokens, Hk, D, device="cuda") for _ in range(2))
    assert tokens * (Hq + Hk) * D * 8 > 1 << 27
    pos = torch.arange(tokens, device="cuda") * 37 if rot else None
    form = {"freqs": 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot) if rot else None}

    def both(at, end):
        p = {**form, "pos": pos[at:end] if rot else None, "norm": "rms", "eps": 1e-6}
        qo, ko, raw = kda.qk_norm_rope_fwd(q[at:end], k[at:end], ckpt8=ckpt8, **p)
        grads = kda.qk_norm_rope_bwd(*(raw if ckpt8 else (q[at:end], k[at:end])), dq[at:end], dk[at:end], **p)
        return [qo, ko, *grads[:2], *([t for r in raw for t in r[:2]] if ckpt8 else [])]

    large = both(0, tokens)
    for at in (0, tokens // 2, tokens - n):
        assert all(torch.equal(s[at:at + n], t) for s, t in zip(large, both(at, at + n)))


@pytest.mark.parametrize("cols", [32, 33, 40])
def test_ckpt8_offsets_beyond_32_bits(cols):
    rows = (1 << 31) // cols + 1001
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    p = kda.ckpt8_pack(x)
    u = kda.ckpt8_unpack(p)
    for at in (0, rows // 2, rows - 1000):
        small = kda.ckpt8_pack(x[at:at + 1000].clone())
        assert torch.equal(p.codes[at:at + 1000], small.codes) and torch.equal(p.scales[at:at + 1000], small.scales)
        assert torch.equal(u[at:at + 1000], kda.ckpt8_unpack(small))


def test_qk_offsets_beyond_32_bits():
    tokens, Hq, Hk, D, n = (1 << 20) + 77, 16, 1, 128, 100
    q, dq = (torch.empty(tokens, Hq, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    k, dk = (torch.empty(tokens, Hk, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    pos, f = torch.arange(tokens, device="cuda"), 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)

    def both(at, end):
        p = {"freqs": f, "pos": pos[at:end], "eps": 1e-6}
        qo, ko, raw = kda.qk_norm_rope_fwd(q[at:end], k[at:end], ckpt8=True, **p)
        return [qo, ko, *kda.qk_norm_rope_bwd(*raw, dq[at:end], dk[at:end], **p)[:2], *(t for r in raw for t in r[:2])]

    large = both(0, tokens)
    for at in (0, tokens // 2, tokens - n):
        assert all(torch.equal(s[at:at + n], t) for s, t in zip(large, both(at, at + n)))


@pytest.mark.parametrize("B", [1, 300])
@pytest.mark.parametrize("save", ["carry", "ckpt8"])
def test_scan_of_a_batch_without_tokens(B, save):
    D = 37
    x, h0, dh = torch.zeros(B, 0, D, device="cuda"), torch.randn(B, D, device="cuda"), torch.randn(B, D, device="cuda")
    (y, dx, dg), (h, dh0), _ = scan_both(x, x, x, None, h0, dh, save)
    assert torch.equal(h, h0) and torch.equal(dh0, dh) and y.shape == dx.shape == dg.shape == x.shape
    assert (scan_both(x, x, x, None, None, dh, save)[1][0] == 0).all()


def test_scan_passes_empty_sequences_in_a_few_steps():
    """A million empty sequences between two tokens: the results without them, and not a step for each."""
    D, E = 4, 10 ** 6
    x, g, dy = torch.randn(300, D, device="cuda"), -torch.rand(300, D, device="cuda"), torch.randn(300, D, device="cuda")
    few = torch.tensor([0, 70, 100, 130, 300], dtype=torch.int32, device="cuda")
    many = torch.cat([few[:3], torch.full((E,), 100, dtype=torch.int32, device="cuda"), few[3:]])
    real = torch.tensor([0, 1, E + 2, E + 3], device="cuda")  # the sequences that have tokens
    h0, dh = torch.randn(E + 4, D, device="cuda"), torch.randn(E + 4, D, device="cuda")
    want = scan_both(x, g, dy, few, h0[real], dh[real], "carry")
    for _ in range(2):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        got = scan_both(x, g, dy, many, h0, dh, "carry")
        end.record()
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[0], want[0]))
    empty = torch.ones(E + 4, dtype=torch.bool, device="cuda")
    empty[real] = False
    for a, b, through in zip(got[1], want[1], (h0, dh)):
        assert torch.equal(a[real], b) and torch.equal(a[empty], through[empty])
    print(f"{start.elapsed_time(end):.2f} ms")
    assert start.elapsed_time(end) < 30  # a step for each takes 170 ms, a search well under 10


# ----------------------------------------------------------------- together, captured, and on other streams

@pytest.mark.parametrize("name", ["GatedScan", "VarlenGatedScan", "ChunkKDA", "NormChunkKDA"])
def test_second_order_gradients_are_refused(name):
    torch.manual_seed(5)
    x = (0.3 * torch.randn(1, 70, 2, 64, device="cuda")).requires_grad_()
    g, beta = -torch.rand(1, 70, 2, 64, device="cuda"), torch.rand(1, 70, 2, device="cuda")
    cu = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    y = {"GatedScan": lambda: kda.GatedScan.apply(x, g)[0],
         "VarlenGatedScan": lambda: kda.VarlenGatedScan.apply(x.flatten(0, 1), g.flatten(0, 1), cu)[0],
         "ChunkKDA": lambda: kda.ChunkKDA.apply(x, x, x, g, beta)[0],
         "NormChunkKDA": lambda: kda.NormChunkKDA.apply(x, x, x, g, beta)[0]}[name]
    first, = torch.autograd.grad(y().sum(), x)
    dx, = torch.autograd.grad(y().sum() + (x ** 3).sum(), x, create_graph=True)
    torch.testing.assert_close(dx.detach(), first + 3 * x.detach() ** 2)
    with pytest.raises(RuntimeError, match="first-order"):
        (dx ** 2).sum().backward()


def test_zero_behind_in_a_graph_and_on_another_stream():
    """The end of the last sequence is the device's: a replay follows the offsets as they then are."""
    total, D = 333, 37
    cu = torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda")
    a, b = torch.empty(total, D, device="cuda"), torch.empty(total, D, dtype=torch.bfloat16, device="cuda")

    def step():
        a.fill_(1)
        b.fill_(2)
        kda.layer._zero_behind(cu, a, b)

    def check(used):
        torch.cuda.synchronize()
        assert (a[:used] == 1).all() and (a[used:] == 0).all() and (b[:used] == 2).all() and (b[used:] == 0).all()

    step()
    check(200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    check(200)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for used in (200, 1, 333, 0, 332, 200):
        cu.copy_(torch.tensor([0, used // 2, used], dtype=torch.int32))
        graph.replay()
        check(used)
        step()
        check(used)


@pytest.mark.parametrize("used", [5, 69990])
def test_zero_behind_beyond_32_bits(used):
    total, D = 70000, 65536
    a = torch.ones(total, D, dtype=torch.bfloat16, device="cuda")
    kda.layer._zero_behind(torch.tensor([0, used], dtype=torch.int32, device="cuda"), a)
    assert not a[used:].any() and a[:used].all()


def test_packed_layer_with_padding():
    """A padded buffer of packed prompts through norm, rotation and scan in training: what stands behind the sequences has no
    part in any gradient."""
    D, H, total, lengths = 64, 2, 260, [70, 1, 0, 129]
    used = sum(lengths)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    torch.manual_seed(6)
    base, gate = torch.randn(total, H * D, device="cuda"), torch.randn(total, H, D, device="cuda")
    weight = torch.randn(H * D, H * D, device="cuda") / 12
    grads = []
    for n, fill in ((used, 0.0), (total, 3.0), (total, 1e30)):
        x, z, w = base[:n].clone(), gate[:n].clone(), weight.clone().requires_grad_()
        x[used:], z[used:] = fill, fill
        z.requires_grad_()
        v = (x @ w).view(n, H, D)
        y, h = kda.VarlenGatedScan.apply(v, z, cu, None, True, True)
        (y ** 2).sum().backward()
        grads.append((w.grad, z.grad[:used]))
    for w, z in grads[1:]:
        # rows of zeros add nothing; another number of rows may be summed in another order
        torch.testing.assert_close(w, grads[0][0], rtol=1e-4, atol=1e-3)
        torch.testing.assert_close(z, grads[0][1], rtol=1e-5, atol=1e-5)
