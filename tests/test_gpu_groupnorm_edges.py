"""The group norm's activation on the GPU far from zero, where e^-u leaves the range of 32 bits, and how exact it is."""
import pytest
import torch

import gated_delta_rule_65_amd as kda
from tests.test_gpu_groupnorm import E, TYPES, check_bwd, check_fwd, make, near

pytestmark = pytest.mark.gpu
FLOOR = 128 * 2.0 ** -126  # a sigmoid below the smallest normal number may be zero; |u| is below 128


def parts(u, act):
    s = torch.sigmoid(u.double())
    return (s, s * (1 - s), s) if act == "sigmoid" else (u.double() * s, s + u.double() * s * (1 - s), s)


def rows(tokens, groups, width):
    """Rows of +1 and -1, as many of either: their own norm exactly."""
    return torch.tensor([1.0, -1.0]).repeat(tokens, groups * width // 2)


def sweep(values, C, dtype=torch.float32):
    """[rows, C], the last row filled up with what lies in the middle."""
    n = -(-values.numel() // C) * C
    return torch.cat([values, values[:1].expand(n - values.numel())]).view(-1, C).to(dtype)


FAR = torch.cat([torch.linspace(-104, -80, 20001), torch.linspace(80, 104, 2001),
                 torch.tensor([-3e38, -1e4, -200.0, -100.0, -88.75, -88.5, 3e38 ** 0.5, 1e4])])
WIDTHS = [(2, 64), (3, 50), (2, 3000), (1, 4098)]  # in registers, 16 bytes and an element or two at a time; too wide for them


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("groups,width", WIDTHS)
def test_far_gates(groups, width, act):
    """Every step as in 64 bits: sigmoids to 12 half steps of 32 bits (the exponential's and the reciprocal's whole steps, four
    roundings) or to the smallest normal number."""
    C = groups * width
    gate = sweep(FAR[FAR.abs() < 1e4], C)
    x, dy = rows(gate.shape[0], groups, width), torch.ones_like(gate)
    w = torch.ones(C)
    kw = {"weight": w.cuda(), "bias": torch.zeros(C).cuda(), "gate": gate.cuda(), "act": act, "eps": 0.0}
    f, slope, s = parts(gate, act)
    y = kda.group_norm_act_fwd(x.cuda(), groups, **kw)
    near(y, x * f, 12 * E * f.abs() + FLOOR, "y")
    dx, dw, db, dgate = kda.group_norm_act_bwd(x.cuda(), groups, dy.cuda(), **kw)
    near(dgate, x * slope, 16 * E * (f.abs() + s) + FLOOR, "dgate")
    many = lambda t: t.unflatten(-1, (groups, width))  # noqa: E731
    mean = many(f).mean(-1, keepdim=True)
    along = (many(f) * many(x.double())).mean(-1, keepdim=True)
    most = many(f).abs().amax(-1, keepdim=True)
    near(many(dx), many(f) - mean - many(x.double()) * along, (3 * (width / 8 + 16) + 12) * E * most + 4 * FLOOR, "dx")
    size = f.abs().sum(0)
    near(dw, (f * x).sum(0), (gate.shape[0] + 12) * E * size + gate.shape[0] * FLOOR, "dweight")
    near(db, f.sum(0), (gate.shape[0] + 12) * E * size + gate.shape[0] * FLOOR, "dbias")


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("groups,width", WIDTHS)
def test_far_values(groups, width, act):
    """The same of the normed values themselves: a weight of zero leaves the bias."""
    C = groups * width
    for bias in sweep(FAR[FAR.abs() < 1e4], C)[:40]:
        x = rows(1, groups, width)
        kw = {"weight": torch.zeros(C).cuda(), "bias": bias.cuda(), "act": act, "eps": 0.0}
        f, slope, s = parts(bias, act)
        near(kda.group_norm_act_fwd(x.cuda(), groups, **kw)[0], f, 12 * E * f.abs() + FLOOR, "y")
        dx, dw, db, _ = kda.group_norm_act_bwd(x.cuda(), groups, torch.ones(1, C).cuda(), **kw)
        assert not bool(dx.any())
        near(dw, slope * x[0], 16 * E * (f.abs() + s) + FLOOR, "dweight")
        near(db, slope, 16 * E * (f.abs() + s) + FLOOR, "dbias")


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("groups,width", WIDTHS)
def test_largest_gates_leave_gradients_finite(groups, width, act):
    """Gates to the end of float32's range: y, dx, dgate and the weights' gradients are numbers wherever the formula's are."""
    C = groups * width
    gate = sweep(FAR, C)
    gate[-1, -2:] = torch.tensor([-3.4e38, 1e18])
    x, dy = rows(gate.shape[0], groups, width), torch.ones_like(gate)
    kw = {"weight": torch.ones(C).cuda(), "bias": torch.zeros(C).cuda(), "gate": gate.cuda(), "act": act, "eps": 0.0}
    assert bool(torch.isfinite(kda.group_norm_act_fwd(x.cuda(), groups, **kw)).all())
    for name, t in zip(("dx", "dw", "db", "dgate"), kda.group_norm_act_bwd(x.cuda(), groups, dy.cuda(), **kw)):
        assert bool(torch.isfinite(t).all()), name


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("xt", list(TYPES))
@pytest.mark.parametrize("groups,width", WIDTHS)
def test_gates_of_16_bits_have_gradients_of_32(groups, width, xt, act):
    """With gates and outputs in bf16 the weights' gradients are as exact as with float32 ones: one token, so that each sum is one
    term."""
    C = groups * width
    gate = torch.linspace(-86.0, -20.0, C).bfloat16()[None]
    x, dy = rows(1, groups, width).to(TYPES[xt]), torch.ones(1, C, dtype=torch.bfloat16)
    kw = {"weight": torch.ones(C).cuda(), "bias": torch.zeros(C).cuda(), "gate": gate.cuda(), "act": act, "eps": 0.0}
    f, slope, s = parts(gate, act)
    dx, dw, db, dgate = kda.group_norm_act_bwd(x.cuda(), groups, dy.cuda(), **kw)
    near(dw, (f * x)[0], 12 * E * f[0].abs() + FLOOR, "dweight")
    near(db, f[0], 12 * E * f[0].abs() + FLOOR, "dbias")
    near(dgate, x * slope, 2.0 ** -8 * slope.abs() * (1 + 16 * E) + 16 * E * (f.abs() + s) + FLOOR, "dgate")


@pytest.mark.parametrize("width", [64, 50, 3000])
def test_gradients_without_the_weights(width):
    """dx and dgate are the same bits with the weights' sums and without."""
    x, w, b, gate, dy = (t.cuda() for t in make(3, 70, 2, width, "bf16", "bf16"))
    kw = {"weight": w, "bias": b, "gate": gate}
    dx, dw, db, dgate = kda.group_norm_act_bwd(x, 2, dy, **kw)
    some = kda.group_norm_act_bwd(x, 2, dy, output_dweights=False, **kw)
    assert some[1] is None and some[2] is None and dw is not None and db is not None
    assert torch.equal(some[0], dx) and torch.equal(some[3], dgate)


@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("width", [64, 256, 1536, 2048])
@pytest.mark.parametrize("skip", [1, 2, 4])
def test_starts_that_are_not_aligned(skip, width, xt, yt):
    """Widths and strides that wide loads divide, and each tensor in turn at another place: to the same bounds."""
    x, w, b, gate, dy = make(skip + width, 19, 2, width, xt, yt)

    def off(t):
        return torch.cat([t.new_zeros(skip), t.flatten()]).cuda()[skip:].view(t.shape)

    def columns(t):
        wide = t.new_zeros(19, 2 * width + 16)
        wide[:, skip:skip + 2 * width] = t
        return wide.cuda()[:, skip:skip + 2 * width]

    for i, moved in [(i, off) for i in range(5)] + [(0, columns), (3, columns)]:
        X, W, B, G, D = (moved(t) if i == j else t.cuda() for j, t in enumerate((x, w, b, gate, dy)))
        check_fwd(kda.group_norm_act_fwd(X, 2, weight=W, bias=B, gate=G), x, 2, w, b, gate, "silu", 1e-5)
        check_bwd(kda.group_norm_act_bwd(X, 2, D, weight=W, bias=B, gate=G), x, 2, dy, w, b, gate, "silu", 1e-5)


@pytest.mark.parametrize("width", [17, 33, 48, 49, 65, 97, 129, 192, 193, 257, 384, 386, 513])
@pytest.mark.parametrize("gated", [False, True])
def test_widths_around_every_shape(width, gated):
    """The first and last widths of each number of lanes and pieces, groups that fill a workgroup and one more."""
    for groups, tokens, xt, yt in ((1, 40, "f32", "f32"), (17, 9, "bf16", "bf16"), (5, 23, "f32", "bf16")):
        x, w, b, gate, dy = make(width + groups, tokens, groups, width, xt, yt)
        gate = gate if gated else None
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        kw = {"weight": w.cuda(), "bias": b.cuda(), "gate": c(gate)}
        check_fwd(kda.group_norm_act_fwd(x.cuda(), groups, dtype=dy.dtype, **kw), x, groups, w, b, gate, "silu", 1e-5)
        check_bwd(kda.group_norm_act_bwd(x.cuda(), groups, dy.cuda(), **kw), x, groups, dy, w, b, gate, "silu", 1e-5)
