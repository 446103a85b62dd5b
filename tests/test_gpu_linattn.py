"""Linear attention with a decay for each head on the GPU, against the 64-bit recurrence."""
import math

import pytest
import torch

import gated_delta_rule_65_amd as kda
from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gpu(*tensors):
    return tuple(None if t is None else t.cuda() for t in tensors)


def near(got, want, allowed, what):
    got = got.detach().cpu().double()
    off = (got - want).abs()
    bad = ~(off <= allowed)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst {float((off / allowed).max()):.2f}x"


def check_fwd(o, sf, q, k, v, g, s0, cu, scale, steps):
    want, end = ref.attend(q, k, v, g, s0, cu, scale)
    size, end_size = ref.magnitude(ref.attend, q, k, v, g, s0=s0, cu=cu, scale=abs(scale))
    used = q.shape[0] if cu is None else int(cu[-1])
    near(o[:used], want[:used], ref.bound(q.dtype, want, size, steps)[:used], "o")
    if sf is not None:
        near(sf, end, ref.state_bound(end, end_size, steps), "s_final")


def check_bwd(got, q, k, v, g, d_o, s0, d_sf, cu, scale, steps):
    want = ref.attend_grads(q, k, v, g, d_o, s0, d_sf, cu, scale)
    size = ref.magnitude(ref.attend_grads, q, k, v, g, d_o=d_o, s0=s0, d_sf=d_sf, cu=cu, scale=abs(scale))
    used = q.shape[0] if cu is None else int(cu[-1])
    for name, x, w, m in zip(("dq", "dk", "dv"), got, want, size):
        near(x[:used], w[:used], ref.bound(q.dtype, w, m, steps)[:used], name)
    near(got[3], want[3], ref.state_bound(want[3], size[3], steps), "ds0")


SIZES = [(1, 1, 1), (3, 2, 3), (2, 63, 2), (1, 64, 3), (2, 65, 8), (1, 127, 2), (1, 130, 9), (2, 333, 3), (1, 1100, 2)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,T,H", SIZES)
def test_batch(B, T, H, dk, dv, dtype):
    q, k, v, d_o, g, s0, d_sf = ref.inputs(B * 1000 + T, (B, T), H, dk, dv, TYPES[dtype], B)
    if T % 2:
        s0 = d_sf = None
    scale, steps = (1.0 if T % 3 else dk ** -0.5), T + dk + dv + 64
    Q, K, V, G, S0, DO, DS = gpu(q, k, v, g, s0, d_o, d_sf)
    o, sf = kda.linattn_fwd(Q, K, V, G, S0, scale=scale)
    check_fwd(o, sf, q, k, v, g, s0, None, scale, steps)
    check_bwd(kda.linattn_bwd(Q, K, V, G, DO, S0, DS, scale=scale), q, k, v, g, d_o, s0, d_sf, None, scale, steps)


PACKED = [[0], [0, 0], [0, 1], [0, 5, 5, 6, 70], [0, 64, 128, 256], [0, 0, 0, 200, 201, 201, 777, 777],
          [0, 700, 1500], list(range(0, 67)), [0, 3, 2100]]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("behind", [0, 37])
@pytest.mark.parametrize("cu", PACKED, ids=lambda c: f"n{len(c) - 1}_t{c[-1]}")
def test_packed(cu, behind, dtype):
    total, n, H, dk, dv = cu[-1] + behind, len(cu) - 1, 3, 64, 128
    if len(cu) % 2:
        dk, dv = 128, 64
    q, k, v, d_o, g, s0, d_sf = ref.inputs(total + n, (total,), H, dk, dv, TYPES[dtype], n)
    for t in (q, k, v, d_o):
        t[cu[-1]:] = math.nan  # rows behind the last sequence are not read into any
    cu = torch.tensor(cu, dtype=torch.int32)
    Q, K, V, G, S0, DO, DS, CU = gpu(q, k, v, g, s0, d_o, d_sf, cu)
    steps = int(cu[-1]) + 256
    o, sf = kda.linattn_varlen_fwd(Q, K, V, G, CU, S0, scale=0.3)
    check_fwd(o, sf, q, k, v, g, s0, cu, 0.3, steps)
    got = kda.linattn_varlen_bwd(Q, K, V, G, CU, DO, S0, DS, scale=0.3)
    check_bwd(got, q, k, v, g, d_o, s0, d_sf, cu, 0.3, steps)


def test_rows_behind_are_left():
    cu = torch.tensor([0, 70, 100], dtype=torch.int32, device="cuda")
    L, H, D = kda.load_library(), 2, 64
    q, k, v, d_o, g, s0, d_sf = gpu(*ref.inputs(5, (150,), H, D, D, torch.bfloat16, 2))
    outs = [torch.full_like(q, 7.0) for _ in range(4)]
    ws = torch.empty(max(kda.linattn_workspace_bytes(2, 150, H, D, D, q.dtype),
                         kda.linattn_bwd_workspace_bytes(2, 150, H, D, D, q.dtype), 1), dtype=torch.uint8, device="cuda")
    p = [t.data_ptr() for t in (q, k, v, g, cu)]
    tail = (H, D, D, 1.0, 1, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert L.kda_linattn_varlen_fwd(*p, 2, 150, s0.data_ptr(), outs[0].data_ptr(), None, *tail) == 0
    assert L.kda_linattn_varlen_bwd(*p, 2, 150, s0.data_ptr(), d_o.data_ptr(), None, *(o.data_ptr() for o in outs[1:]), None,
                                    *tail) == 0
    torch.cuda.synchronize()
    for o in outs:
        assert bool((o[100:] == 7.0).all()) and not bool((o[:100] == 7.0).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,H", [(1, 1), (5, 3), (33, 8)])
def test_step(B, H, dk, dv, dtype):
    q, k, v, _, g, s0, _ = ref.inputs(B + H, (B,), H, dk, dv, TYPES[dtype], B)
    Q, K, V, G, S0 = gpu(q, k, v, g, s0)
    o, s = kda.linattn_step(Q, K, V, G, S0, scale=0.5)
    one = lambda t: t[:, None]  # noqa: E731
    check_fwd(o[:, None], s, one(q), one(k), one(v), g, s0, None, 0.5, dk + dv + 8)
    assert torch.equal(S0.cpu(), s0)
    o2, s2 = kda.linattn_step(Q, K, V, G, S0, scale=0.5, inplace=True)
    assert s2 is S0 and torch.equal(s2, s) and torch.equal(o2, o)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_prompt_then_tokens(dtype):
    """A prompt's state, continued a token at a time, gives what the whole sequence gives."""
    q, k, v, _, g, _, _ = ref.inputs(9, (2, 90), 4, 64, 64, TYPES[dtype], 2)
    Q, K, V, G = gpu(q, k, v, g)
    cut = lambda t, *at: t[:, slice(*at)].contiguous()  # noqa: E731
    o, s = kda.linattn_fwd(cut(Q, 70), cut(K, 70), cut(V, 70), G, scale=0.125)
    rest = []
    for t in range(70, 90):
        x, s = kda.linattn_step(Q[:, t].contiguous(), K[:, t].contiguous(), V[:, t].contiguous(), G, s, scale=0.125)
        rest.append(x)
    check_fwd(torch.cat([o, torch.stack(rest, 1)], 1), s, q, k, v, g, None, None, 0.125, 90 + 192)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("at", [0, 37, 64, 1090])
def test_not_finite(what, bad, at, dtype):
    """q's reaches its own row, k's and v's that row and those behind, v's its own channel."""
    q, k, v, _, g, s0, _ = ref.inputs(3, (2, 1200), 2, 64, 64, TYPES[dtype], 2, kinds=[-0.01, -0.3])
    clean, _ = kda.linattn_fwd(*gpu(q, k, v, g, s0))
    {"q": q, "k": k, "v": v}[what][1, at, 1, 5] = bad
    o, s = kda.linattn_fwd(*gpu(q, k, v, g, s0))
    hit = torch.zeros(o.shape, dtype=torch.bool)
    if what == "q":
        hit[1, at, 1] = True
    elif what == "k":
        hit[1, at:, 1] = True
    else:
        hit[1, at:, 1, 5] = True
    assert torch.equal(~torch.isfinite(o.cpu()), hit)
    assert torch.equal(o.cpu()[~hit], clean.cpu()[~hit])
    state = torch.zeros(s.shape, dtype=torch.bool)
    if what == "k":
        state[1, 1, 5] = True
    elif what == "v":
        state[1, 1, :, 5] = True
    assert torch.equal(~torch.isfinite(s.cpu()), state)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("at", [5, 64, 999])
def test_not_finite_gradients(at, dtype):
    """What is not finite in d_o reaches dq of its row, and dk, dv of that row and those before."""
    q, k, v, d_o, g, s0, d_sf = ref.inputs(4, (1, 1100), 2, 64, 128, TYPES[dtype], 1, kinds=[-0.01, -0.3])
    clean = kda.linattn_bwd(*gpu(q, k, v, g, d_o, s0, d_sf))
    d_o[0, at, 1, 70] = math.nan
    dq, dk, dv, _ = kda.linattn_bwd(*gpu(q, k, v, g, d_o, s0, d_sf))
    hits = [torch.zeros(t.shape, dtype=torch.bool) for t in (dq, dk, dv)]
    hits[0][0, at, 1] = True
    hits[1][0, :at + 1, 1] = True
    hits[2][0, :at + 1, 1, 70] = True
    for got, was, hit in zip((dq, dk, dv), clean, hits):
        assert torch.equal(~torch.isfinite(got.cpu()), hit)
        assert torch.equal(got.cpu()[~hit], was.cpu()[~hit])


def test_one_mistake_a_head():
    """A decay that is not a number makes its own head so, and no other."""
    q, k, v, _, g, s0, _ = ref.inputs(3, (1, 100), 3, 64, 64, torch.bfloat16, 1, kinds=[-0.1, math.nan, -0.2])
    o, s = kda.linattn_fwd(*gpu(q, k, v, g, s0))
    assert bool(torch.isfinite(o[:, :, [0, 2]]).all()) and bool(torch.isfinite(s[:, [0, 2]]).all())
    assert bool(torch.isnan(s[:, 1]).all()) and bool(torch.isnan(o[:, 1:, 1]).all())


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 40])
def test_sizes_of_values(size):
    """Values far from one keep their relative accuracy."""
    q, k, v, d_o, g, s0, d_sf = ref.inputs(11, (1, 200), 3, 64, 64, torch.bfloat16, 1)
    v, s0 = v * size, s0 * size
    check_fwd(*kda.linattn_fwd(*gpu(q, k, v, g, s0)), q, k, v, g, s0, None, 1.0, 400)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_long(dtype):
    """A sequence of many segments, decays that reach across all of it and none at all."""
    q, k, v, d_o, g, s0, d_sf = ref.inputs(12, (1, 20011), 3, 64, 64, TYPES[dtype], 1, kinds=[-1e-5, 0.0, -0.002])
    Q = gpu(q, k, v, g, s0)
    steps = 600  # chunks of 64 tokens, and within one: what a term passes on its way
    check_fwd(*kda.linattn_fwd(*Q, scale=0.125), q, k, v, g, s0, None, 0.125, steps)
    check_bwd(kda.linattn_bwd(*Q[:4], *gpu(d_o, s0, d_sf), scale=0.125), q, k, v, g, d_o, s0, d_sf, None, 0.125, steps)


def test_many_sequences_in_one_call():
    """More sequence-heads than the chip has places, in a batch and packed: the same bits."""
    B, T, H, D = 70, 129, 9, 64
    q, k, v, d_o, g, s0, d_sf = gpu(*ref.inputs(13, (B, T), H, D, D, torch.bfloat16, B))
    flat = [t.flatten(0, 1) for t in (q, k, v)]
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    o, s = kda.linattn_fwd(q, k, v, g, s0)
    o2, s2 = kda.linattn_varlen_fwd(*flat, g, cu, s0)
    one, s1 = kda.linattn_fwd(q[37:38].contiguous(), k[37:38].contiguous(), v[37:38].contiguous(), g, s0[37:38].contiguous())
    for a, b in ((o, one), (s, s1)):
        assert float((a[37].double() - b[0].double()).norm()) <= 4 * 2 ** -8 * float(b.double().norm())
    for a, b in ((o.flatten(0, 1), o2), (s, s2)):
        assert float((a.double() - b.double()).norm()) <= 4 * 2 ** -8 * float(b.double().norm())


SEGMENTS = [[0, 5000], [0, 40, 3000, 3100, 3101], [0, 2500, 2500, 5100], [0, 63, 1500, 1564, 4000], [0, 640, 1280, 1921, 4000]]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128)])
@pytest.mark.parametrize("cu", SEGMENTS, ids=lambda c: "_".join(map(str, c)))
def test_packed_segments(cu, dk, dv, dtype):
    """Sequences of one, of up to eight and of more segments in one call, ends inside and at segments; decays that reach far."""
    q, k, v, d_o, g, s0, d_sf = ref.inputs(cu[-1], (cu[-1],), 2, dk, dv, TYPES[dtype], len(cu) - 1, kinds=[-1e-4, -0.004])
    cu = torch.tensor(cu, dtype=torch.int32)
    Q, K, V, G, S0, DO, DS, CU = gpu(q, k, v, g, s0, d_o, d_sf, cu)
    o, sf = kda.linattn_varlen_fwd(Q, K, V, G, CU, S0, scale=0.125)
    check_fwd(o, sf, q, k, v, g, s0, cu, 0.125, 600)
    got = kda.linattn_varlen_bwd(Q, K, V, G, CU, DO, S0, DS, scale=0.125)
    check_bwd(got, q, k, v, g, d_o, s0, d_sf, cu, 0.125, 600)


def test_more_sequences_than_a_fold_would_have_workgroups_for():
    """Over a million sequences of one token: o = scale (q . k) v, and nothing in the way of the grid."""
    B, H, D = 70000, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((B, 1, H, D), generator=gen, device="cuda").bfloat16() for _ in range(3))
    g = torch.full((H,), -0.1, device="cuda")
    o, _ = kda.linattn_fwd(q, k, v, g, scale=0.25, output_final_state=False)
    for at in (slice(0, 500), slice(35000, 35500), slice(B - 500, B)):
        dots = (q[at].double() * k[at].double()).sum(-1, keepdim=True)
        want = 0.25 * dots * v[at].double()
        # half a step of bf16, and 128 products, the scale and the score's planes in 24 and 16 bits
        allowed = want.abs() * 2 ** -8 + 0.25 * (q[at].double() * k[at].double()).abs().sum(-1, keepdim=True) * v[at].double().abs() * 2 ** -15
        assert bool(((o[at].double() - want).abs() <= allowed + 1e-30).all())


@pytest.mark.parametrize("dtype", list(TYPES))
def test_differences(dtype):
    """o is linear in q, in k, in v and in s0: central differences of the forward call are the gradients, up to rounding."""
    q, k, v, d_o, g, s0, d_sf = ref.inputs(21, (2, 150), 3, 64, 128, torch.float32, 2)
    ins = [t.cuda() for t in (q, k, v, s0)]
    G, DO, DS = gpu(g, d_o, d_sf)
    if dtype == "bf16":
        ins = [t.bfloat16() for t in ins[:3]] + ins[3:]
        DO = DO.bfloat16()
    grads = kda.linattn_bwd(*ins[:3], G, DO, ins[3], DS, scale=0.2)

    def loss(q, k, v, s0):
        o, s = kda.linattn_fwd(q, k, v, G, s0, scale=0.2)
        return float((o.double() * DO.double()).sum() + (s.double() * DS.double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, grad in enumerate(grads):
        d = torch.randint(-1, 2, ins[i].shape, generator=gen, device="cuda").to(ins[i].dtype) * 4  # sums stay in the type's reach
        up, down = list(ins), list(ins)
        up[i], down[i] = (ins[i] + d), (ins[i] - d)
        step = (up[i].double() - down[i].double())
        diff, slope = loss(*up) - loss(*down), float((grad.double() * step).sum())
        # every value of o and of the gradient is off by half a step: the sums of as many random ones
        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -18
        scale = float((grad.double() * step).norm()) + float((kda.linattn_fwd(*up[:3], G, up[3], scale=0.2)[0].double() *
                                                              DO.double()).norm()) * 2
        assert abs(diff - slope) <= 8 * half * scale, (i, diff, slope, scale)


@pytest.mark.parametrize("packed", [False, True])
def test_autograd(packed):
    q, k, v, d_o, g, s0, d_sf = gpu(*ref.inputs(31, (2, 140), 3, 64, 64, torch.bfloat16, 2))
    leaves = [t.clone().requires_grad_() for t in (q, k, v, s0)]
    want = kda.linattn_bwd(q, k, v, g, d_o, s0, d_sf, scale=0.25)
    if packed:
        rows = [t.flatten(0, 1) for t in leaves[:3]]
        rows = [torch.cat([t, torch.ones_like(t[:9])]) for t in rows]  # a padded batch
        cu = torch.tensor([0, 140, 280], dtype=torch.int32, device="cuda")
        o, s = kda.VarlenLinearAttention.apply(*rows, g, cu, leaves[3], 0.25)
        assert bool((o[280:] == 0).all())
        torch.autograd.backward((o[:280], s), (d_o.flatten(0, 1), d_sf))
    else:
        o, s = kda.LinearAttention.apply(*leaves[:3], g, leaves[3], 0.25)
        torch.autograd.backward((o, s), (d_o, d_sf))
    for t, w in zip(leaves, want):
        assert torch.equal(t.grad, w)


def test_autograd_refusals():
    q, k, v, d_o, g, s0, d_sf = gpu(*ref.inputs(32, (1, 20), 2, 64, 64, torch.float32, 1))
    o, _ = kda.LinearAttention.apply(q.requires_grad_(), k, v, g.clone().requires_grad_())
    with pytest.raises(ValueError, match="constants"):
        o.sum().backward()
    o, _ = kda.LinearAttention.apply(q, k, v, g)
    grad, = torch.autograd.grad(o.sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="first-order"):
        grad.sum().backward()


def test_graph():
    """Captured and replayed, with eager calls between, on inputs that change."""
    first, other = ([*gpu(*ref.inputs(seed, (1, 2500), 2, 128, 64, torch.bfloat16, 1))] for seed in (41, 42))
    q, k, v, d_o, g, s0, d_sf = [t.clone() for t in first]

    def calls(q, k, v, d_o, g, s0, d_sf):
        o, s = kda.linattn_fwd(q, k, v, g, s0)
        x, s = kda.linattn_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), g, s)
        return (o, s, x, *kda.linattn_bwd(q, k, v, g, d_o, s0, d_sf))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(q, k, v, d_o, g, s0, d_sf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(q, k, v, d_o, g, s0, d_sf)
    for values in (first, other, first):
        for to, x in zip((q, k, v, d_o, g, s0, d_sf), values):
            to.copy_(x)
        graph.replay()
        want = calls(*values)
        torch.cuda.synchronize()
        for x, w in zip(outs, want):
            assert torch.equal(x, w)


def test_two_streams():
    """Two calls at once, each with its own workspace."""
    sets = [gpu(*ref.inputs(s, (1, 3000), 2, 64, 64, torch.bfloat16, 1)) for s in (51, 52)]
    want = [kda.linattn_fwd(q, k, v, g, s0) + kda.linattn_bwd(q, k, v, g, d_o, s0, d_sf) for q, k, v, d_o, g, s0, d_sf in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for st, (q, k, v, d_o, g, s0, d_sf) in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(kda.linattn_fwd(q, k, v, g, s0) + kda.linattn_bwd(q, k, v, g, d_o, s0, d_sf))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(x, want[i % 2]))


def test_nothing_to_do():
    g = torch.zeros(2, device="cuda")
    for B, T in ((0, 5), (2, 0)):
        q = torch.empty((B, T, 2, 64), device="cuda")
        s0 = torch.randn((B, 2, 64, 64), device="cuda")
        o, s = kda.linattn_fwd(q, q, q, g, s0)
        assert o.shape == q.shape and torch.equal(s, s0)
        dq, dk, dv, ds0 = kda.linattn_bwd(q, q, q, g, q, s0, s0)
        assert dq.shape == q.shape and torch.equal(ds0, s0)
        _, s = kda.linattn_fwd(q, q, q, g)
        assert not bool(s.any())


def test_without_final_state():
    q, k, v, _, g, s0, _ = gpu(*ref.inputs(3, (2, 700), 2, 64, 64, torch.bfloat16, 2))
    o, s = kda.linattn_fwd(q, k, v, g, s0, output_final_state=False)
    assert s is None and torch.equal(o, kda.linattn_fwd(q, k, v, g, s0)[0])
