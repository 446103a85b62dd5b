"""Linear attention and the group norm on the GPU where sizes end: offsets past 2^31 elements, segments of hundreds of chunks,
workspaces of the caller, token counts around the blocks of the weights' sums, tensors of views, one input in several places."""
import math

import pytest
import torch

import gated_delta_rule_65_amd as kda
from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def near(got, want, allowed, what):
    off = (got.detach().cpu().double() - want).abs()
    assert bool((off <= allowed).all()), f"{what}: worst {float((off / allowed).max()):.2f}x"


def test_offsets_past_32_bits():
    """2^31 elements and more a tensor, segments of 513 chunks.  The decays forget what is 700 tokens back (e^-35), so that the
    ends can be checked alone; the packed call has its last sequence there."""
    T, H, D, K = 1050000, 16, 128, 700
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, d_o = (torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(4))
    assert q.numel() > 1 << 31
    g = torch.linspace(-0.05, -1.0, H, device="cuda")
    scale, steps = D ** -0.5, 2 * K + 64 + 600  # tokens, chunks of a segment
    heads = [0, 7, 15]

    def part(t, at):
        return t[at][:, heads].cpu()

    def check_end(o, sf, first, what):
        """The last 100 rows and the state, from rows `first` on."""
        at = slice(first, T)
        args = [part(t, at)[None] for t in (q, k, v)] + [g.cpu()[heads]]
        want, end = ref.attend(*args, None, None, scale)
        size, end_size = ref.magnitude(ref.attend, *args, scale=scale)
        near(part(o, slice(T - 100, T)), want[0, -100:], ref.bound(torch.bfloat16, want, size, steps)[0, -100:], what)
        # what is left out: e^-35 of a state of sums of sqrt(20) products at most
        near(sf[-1, heads], end[0], ref.state_bound(end, end_size, steps)[0] + 1e-13, what)

    o, sf = kda.linattn_fwd(q[None], k[None], v[None], g, scale=scale)
    check_end(o[0], sf, T - 100 - K, "batch")
    dq, dk, dv, _ = kda.linattn_bwd(q[None], k[None], v[None], g, d_o[None], scale=scale)
    args = [part(t, slice(T - 100 - K, T))[None] for t in (q, k, v)] + [g.cpu()[heads]]
    D_o = part(d_o, slice(T - 100 - K, T))[None]
    want = ref.attend_grads(*args, D_o, None, None, None, scale)
    size = ref.magnitude(ref.attend_grads, *args, d_o=D_o, scale=scale)
    for got, w, m, name in zip((dq, dk, dv), want, size, ("dq", "dk", "dv")):
        near(part(got[0], slice(T - 100, T)), w[0, -100:], ref.bound(torch.bfloat16, w, m, steps)[0, -100:], name)
    args = [part(t, slice(0, 100 + K))[None] for t in (q, k, v)] + [g.cpu()[heads]]
    D_o = part(d_o, slice(0, 100 + K))[None]
    want = ref.attend_grads(*args, D_o, None, None, None, scale)
    size = ref.magnitude(ref.attend_grads, *args, d_o=D_o, scale=scale)
    for got, w, m, name in zip((dq, dk, dv), want, size, ("dq", "dk", "dv")):
        near(part(got[0], slice(0, 100)), w[0, :100], ref.bound(torch.bfloat16, w, m, steps)[0, :100], name)
    del dq, dk, dv, o
    cu = torch.tensor([0, 5, T - 300, T], dtype=torch.int32, device="cuda")
    o, sf = kda.linattn_varlen_fwd(q, k, v, g, cu, scale=scale)
    check_end(o, sf, T - 300, "packed")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,T,H", [(3, 1100, 40), (1, 1300, 171), (2, 1100, 129), (1, 600, 511), (2, 600, 256), (3, 400, 200)])
def test_parts_of_equal_lengths(B, T, H, dtype):
    """Lengths cut in four, two, one part for the places there are; some heads are checked, each is its own."""
    q, k, v, d_o, g, s0, d_sf = ref.inputs(T + H, (B, T), H, 64, 64, TYPES[dtype], B, kinds=[-0.003, -0.2, 0.0, -1e-4, -30.0])
    Q, K, V, DO, G, S0, DS = (t.cuda() for t in (q, k, v, d_o, g, s0, d_sf))
    heads = [0, 1, H // 2, H - 1]
    of = lambda t: t[:, :, heads].contiguous()  # noqa: E731
    args, s, ds = [of(t) for t in (q, k, v)] + [g[heads]], s0[:, heads], d_sf[:, heads]
    o, end = kda.linattn_fwd(Q, K, V, G, S0, scale=0.125)
    want, last = ref.attend(*args, s, None, 0.125)
    size, last_size = ref.magnitude(ref.attend, *args, s0=s, scale=0.125)
    steps = 400  # chunks of 64 tokens, within one, and segments
    near(of(o), want, ref.bound(q.dtype, want, size, steps), "o")
    near(end[:, heads], last, ref.state_bound(last, last_size, steps), "s_final")
    got = kda.linattn_bwd(Q, K, V, G, DO, S0, DS, scale=0.125)
    want = ref.attend_grads(*args, of(d_o), s, ds, None, 0.125)
    size = ref.magnitude(ref.attend_grads, *args, d_o=of(d_o), s0=s, d_sf=ds, scale=0.125)
    for name, x, w, m in zip(("dq", "dk", "dv"), got, want, size):
        near(of(x), w, ref.bound(q.dtype, w, m, steps), name)
    near(got[3][:, heads], want[3], ref.state_bound(want[3], size[3], steps), "ds0")


@pytest.mark.parametrize("backward", [False, True])
def test_workspaces_of_the_caller(backward):
    q, k, v, d_o, g, s0, d_sf = (t.cuda() for t in ref.inputs(1, (1, 3000), 4, 64, 128, torch.bfloat16, 1))
    size = (kda.linattn_bwd_workspace_bytes if backward else kda.linattn_workspace_bytes)(1, 3000, 4, 64, 128, q.dtype)

    def run(ws):
        return kda.linattn_bwd(q, k, v, g, d_o, s0, d_sf, workspace=ws) if backward else kda.linattn_fwd(q, k, v, g, s0, workspace=ws)

    want = run(None)
    big = torch.full((size + 512,), 255, dtype=torch.uint8, device="cuda")  # no initial contents are needed: NaN in every word
    assert all(torch.equal(a, b) for a, b in zip(run(big[256:256 + size]), want))
    assert bool((big[:256] == 255).all()) and bool((big[256 + size:] == 255).all())  # nothing behind it
    with pytest.raises((RuntimeError, ValueError), match="workspace"):
        run(big[256:256 + size - 16])


def test_one_tensor_in_several_places():
    """q, k and v (and d_o) may be one tensor."""
    x, _, _, _, g, s0, _ = ref.inputs(2, (2, 150), 3, 64, 64, torch.bfloat16, 2)
    X, G, S0 = x.cuda(), g.cuda(), s0.cuda()
    o, _ = kda.linattn_fwd(X, X, X, G, S0, scale=0.125)
    want, _ = ref.attend(x, x, x, g, s0, None, 0.125)
    size, _ = ref.magnitude(ref.attend, x, x, x, g, s0=s0, scale=0.125)
    near(o, want, ref.bound(x.dtype, want, size, 150 + 192), "o")
    got = kda.linattn_bwd(X, X, X, G, X, S0, scale=0.125)
    other = [t.clone() for t in (X, X, X, X)]
    assert all(torch.equal(a, b) for a, b in zip(got, kda.linattn_bwd(*other[:3], G, other[3], S0, scale=0.125)))


def test_no_heads_in_common():
    """A head's results are its own: the same bits with other values in the other heads."""
    q, k, v, d_o, g, s0, d_sf = (t.cuda() for t in ref.inputs(3, (1, 700), 4, 128, 64, torch.bfloat16, 1))
    first = kda.linattn_fwd(q, k, v, g, s0) + kda.linattn_bwd(q, k, v, g, d_o, s0, d_sf)
    for t in (q, k, v, d_o):
        t[:, :, [0, 1, 3]] = math.nan
    for t in (s0, d_sf):
        t[:, [0, 1, 3]] = math.inf
    second = kda.linattn_fwd(q, k, v, g, s0) + kda.linattn_bwd(q, k, v, g, d_o, s0, d_sf)
    for i, (a, b) in enumerate(zip(first, second)):
        axis = 1 if i in (1, 5) else 2
        assert torch.equal(a.select(axis, 2), b.select(axis, 2)), i


@pytest.mark.parametrize("tokens", [15, 16, 17, 8191, 8192, 8193, 8209])
def test_norm_weights_sums_around_the_blocks(tokens):
    gen = torch.Generator().manual_seed(tokens)
    x, dy, w = torch.randn((tokens, 64), generator=gen), torch.randn((tokens, 64), generator=gen), torch.randn(64, generator=gen)
    dx, dw, db, _ = kda.group_norm_act_bwd(x.cuda(), 2, dy.cuda(), weight=w.cuda(), bias=w.cuda(), act="none")
    want = ref.group_norm_grads(x, 2, dy, w, w, None, "none", 1e-5)
    p, _, dz, _ = want["parts"]
    # a block's rows and the blocks one after another, and a few roundings of a row's mean and length
    adds = 2 * (16 + tokens / 512 + 512 / 32 + 32) + 64 + 64
    near(dw, want["dw"], adds * 2.0 ** -24 * ((dz * p["n"]).abs() + dz.abs()).sum(0).flatten() + 1e-12, "dw")
    near(db, want["db"], adds * 2.0 ** -24 * dz.abs().sum(0).flatten() + 1e-12, "db")


def test_norm_offsets_past_32_bits():
    """Rows beyond 2^31 elements, of a tensor and of a view whose tokens lie far apart."""
    tokens, C = 1050000, 2048
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty((tokens, C), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = torch.randn(C, generator=gen, device="cuda")
    y = kda.group_norm_act_fwd(x, 16, weight=w, gate=x)
    dx, dw, _, dgate = kda.group_norm_act_bwd(x, 16, y, weight=w, gate=x)
    at = slice(tokens - 50, tokens)
    xs, ys, W = x[at].cpu(), y[at].cpu(), w.cpu()
    p = ref.group_norm(xs, 16, W, None, xs, "silu", 1e-5)
    # half a step, and of the values before it some roundings of 32 bits (sums of 128, a root, an exponential)
    near(y[at], p["y"], 2.0 ** -8 * p["y"].abs() + 256 * 2.0 ** -24 * ((p["n"].abs() + 1) * p["W"] * p["f"]).abs().flatten(-2), "y")
    want = ref.group_norm_grads(xs, 16, ys, W, None, xs, "silu", 1e-5)
    p, D, dz, dn = want["parts"]
    size = (p["r"] * (dn.abs() + dn.abs().mean(-1, keepdim=True) + p["n"].abs() * (dn * p["n"]).abs().mean(-1, keepdim=True))).flatten(-2)
    near(dx[at], want["dx"], 2.0 ** -8 * want["dx"].abs() + 512 * 2.0 ** -24 * size, "dx")
    near(dgate[at], want["dgate"], 2.0 ** -8 * want["dgate"].abs() +
         256 * 2.0 ** -24 * (D.abs() * (p["n"].abs() + 1) * p["W"].abs() * (p["slope"].abs() + p["f"].abs() + 1)).flatten(-2), "dgate")
    total, size = torch.zeros(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    for i in range(0, tokens, 50000):
        X, Y = x[i:i + 50000].double().unflatten(-1, (16, -1)), y[i:i + 50000].double()
        n = (X - X.mean(-1, keepdim=True)) / torch.sqrt(X.var(-1, correction=0, keepdim=True) + 1e-5)
        u = x[i:i + 50000].double()
        term = Y * u * torch.sigmoid(u) * n.flatten(-2)
        total += term.sum(0)
        size += term.abs().sum(0)
    # a thread's 2051 rows and the 512 blocks, one after another
    near(dw, total.cpu(), ((2051 + 512) * 2.0 ** -24 + 2.0 ** -16) * size.cpu(), "dw")
    del dx, dgate, y
    far = x.view(-1)[:(tokens - 1) // 1024 * 1024 * C].view(-1, 1024, C)[:, 5]  # a token in 1024, 2^21 elements apart
    near(kda.group_norm_act_fwd(far, 16, weight=w)[-3:], ref.group_norm(far[-3:].cpu(), 16, W, None, None, "silu", 1e-5)["y"],
         2.0 ** -8 * ref.group_norm(far[-3:].cpu(), 16, W, None, None, "silu", 1e-5)["y"].abs() + 256 * 2.0 ** -24 *
         (ref.group_norm(far[-3:].cpu(), 16, W, None, None, "silu", 1e-5)["z"].abs().flatten(-2) + w.cpu().abs()), "far")
