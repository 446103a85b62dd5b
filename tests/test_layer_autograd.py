"""The autograd functions' own work (what they keep, refuse and hand on), with plain stand-ins on the CPU for the calls that
run kernels."""
import pytest
import torch

import gated_delta_rule_65_amd as kda
from gated_delta_rule_65_amd import layer


def plain_scan(x, g, where, h0):
    """y and the last states of the scan of log gates, rows x [total, D]."""
    a, y, last = torch.exp(g.clamp(-5, 0)), [None] * len(x), []
    for n, (i, j) in enumerate(where):
        h = torch.zeros_like(x[0]) if h0 is None else h0[n]
        for t in range(i, j):
            h = a[t] * h + x[t]
            y[t] = h
        last.append(h)
    return torch.stack([torch.zeros_like(x[0]) if v is None else v for v in y]), torch.stack(last)


def spans_of(cu):
    return list(zip(cu.tolist()[:-1], cu.tolist()[1:]))


@pytest.fixture
def stand_ins(monkeypatch):
    def varlen_fwd(x, g, cu, h0=None, **kw):
        with torch.no_grad():
            return (*plain_scan(x, g, spans_of(cu), h0), torch.zeros(1))

    def varlen_bwd(g, cu, dy, saved, *, x, h0, dh_final, **kw):
        with torch.enable_grad():
            leaves = [t.detach().requires_grad_() for t in (x, g, torch.zeros_like(dh_final) if h0 is None else h0)]
            out = plain_scan(leaves[0], leaves[1], spans_of(cu), leaves[2])
            return torch.autograd.grad(out, leaves, (dy.detach(), dh_final.detach()), allow_unused=True)

    def offsets(x):
        return torch.arange(x.shape[0] + 1, dtype=torch.int32) * x.shape[1]

    def fwd(x, g, h0=None, **kw):
        y, h, saved = varlen_fwd(x.flatten(0, 1), g.flatten(0, 1), offsets(x), h0)
        return y.view(x.shape), h, saved

    def bwd(g, dy, saved, *, x, h0, dh_final, **kw):
        dx, dg, dh0 = varlen_bwd(g.flatten(0, 1), offsets(x), dy.flatten(0, 1), saved, x=x.flatten(0, 1), h0=h0,
                                 dh_final=dh_final)
        return dx.view(x.shape), dg.view(x.shape), dh0

    def norm_fwd(q, k, **kw):
        return q.detach() * 2, k.detach() * 2, None

    def norm_bwd(q, k, dq, dk, **kw):
        return dq.detach().to(q.dtype) * 2, dk.detach().to(k.dtype) * 2, None, None

    def chunk_fwd(q, k, v, g, beta, s0=None):
        return (q * k * v).detach().float(), torch.zeros(q.shape[0], q.shape[2], q.shape[3], v.shape[3])

    def chunk_bwd(q, k, v, g, beta, d_o, s0=None, d_sfinal=None):
        if g.dtype != torch.float32 or beta.dtype != torch.float32:
            raise TypeError("g must be torch.float32")
        d = d_o.detach()
        return d * (k * v), d * (q * v), d * (q * k), torch.ones_like(g), torch.ones_like(beta), torch.zeros(1)

    def zero_behind(cu, *tensors):
        for t in tensors:
            t[cu[-1]:] = 0

    for name, f in (("_zero_behind", zero_behind), ("scan_fwd", fwd), ("scan_bwd", bwd), ("scan_varlen_fwd", varlen_fwd), ("scan_varlen_bwd", varlen_bwd),
                    ("qk_norm_rope_fwd", norm_fwd), ("qk_norm_rope_bwd", norm_bwd), ("chunk_fwd", chunk_fwd),
                    ("chunk_bwd", chunk_bwd)):
        monkeypatch.setattr(layer, name, f)
    monkeypatch.setattr(kda, "chunk_fwd", chunk_fwd)
    monkeypatch.setattr(kda, "chunk_bwd", chunk_bwd)


def applied(name, x, g):
    """y of an autograd function at x and g, both [1, T, H, D]."""
    if name == "GatedScan":
        return kda.GatedScan.apply(x, g, None)[0]
    if name == "VarlenGatedScan":
        cu = torch.tensor([0, 2, x.shape[1]], dtype=torch.int32)
        return kda.VarlenGatedScan.apply(x.flatten(0, 1), g.flatten(0, 1), cu, None)[0]
    beta = torch.ones(x.shape[:3])
    return getattr(kda, name).apply(x, x, x, g, beta)[0]


@pytest.mark.parametrize("name", ["GatedScan", "VarlenGatedScan", "ChunkKDA", "NormChunkKDA"])
@pytest.mark.parametrize("weighted", [False, True])
def test_second_order_gradients_are_refused(stand_ins, name, weighted):
    """A penalty on a gradient needs the gradient's gradient, which the backward kernels do not give: an error, also where
    other terms have theirs and where the gradient that comes in has no graph of its own."""
    torch.manual_seed(1)
    x, g = torch.randn(1, 5, 2, 4).requires_grad_(), (-torch.rand(1, 5, 2, 4)).requires_grad_()
    y = applied(name, x, g)
    loss = ((y * y).sum() if weighted else y.sum()) + (x ** 3).sum()
    dx, = torch.autograd.grad(loss, x, create_graph=True)
    assert torch.isfinite(dx).all()  # the gradient itself is there
    with pytest.raises(RuntimeError, match="first-order"):
        (dx ** 2).sum().backward()


@pytest.mark.parametrize("name", ["GatedScan", "VarlenGatedScan", "ChunkKDA", "NormChunkKDA"])
def test_first_order_gradients_are_the_same_with_a_graph(stand_ins, name):
    torch.manual_seed(2)
    x, g = torch.randn(1, 5, 2, 4).requires_grad_(), (-torch.rand(1, 5, 2, 4)).requires_grad_()
    grads = [torch.autograd.grad((applied(name, x, g) ** 2).sum(), (x, g), create_graph=graph) for graph in (False, True)]
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    assert not any(t.requires_grad for t in grads[0])


def test_offsets_changed_before_the_backward_pass_are_an_error(stand_ins):
    """Offsets are kept like the other tensors: rewritten in place in between, they would give another batch's gradients."""
    x, g = torch.randn(6, 3).requires_grad_(), (-torch.rand(6, 3)).requires_grad_()
    cu = torch.tensor([0, 2, 6], dtype=torch.int32)
    y, _ = kda.VarlenGatedScan.apply(x, g, cu, None)
    cu.copy_(torch.tensor([0, 5, 6]))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("name", ["GatedScan", "VarlenGatedScan", "ChunkKDA", "NormChunkKDA"])
def test_what_is_kept_passes_the_hooks_of_saved_tensors(stand_ins, name):
    """Hooks that move saved tensors away see all of them."""
    x, g = torch.randn(1, 5, 2, 4).requires_grad_(), (-torch.rand(1, 5, 2, 4)).requires_grad_()
    kinds = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kinds.append(t.dtype) or t.clone(), lambda t: t):
        y = applied(name, x, g)
    assert (torch.int32 in kinds) == (name == "VarlenGatedScan")
    y.sum().backward()
    assert torch.isfinite(x.grad).all() and torch.isfinite(g.grad).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_come_to_the_kernels_whole_and_aligned(dtype):
    """torch hands a backward pass views that begin anywhere; the kernels read 16 bytes at a time."""
    whole = torch.arange(33, dtype=torch.float32).to(dtype)
    for t in (whole[1:], whole[4:], whole[:32].view(4, 8).t(), whole[:1].expand(5), whole[16:]):
        for to in (torch.float32, torch.bfloat16):
            got = kda._aligned_grad(t, to)
            assert got.is_contiguous() and got.data_ptr() % 16 == 0 and got.dtype == to
            assert torch.equal(got, t.to(to))
    assert kda._aligned_grad(whole, dtype) is whole  # no copy where none is needed


@pytest.mark.parametrize("name", ["ChunkKDA", "NormChunkKDA"])
def test_gates_that_the_forward_pass_takes_in_16_bits_have_gradients(stand_ins, name):
    q, g, beta = torch.randn(1, 5, 2, 4), -torch.rand(1, 5, 2, 4).bfloat16(), torch.rand(1, 5, 2).bfloat16()
    leaves = [t.requires_grad_() for t in (q, g, beta)]
    getattr(kda, name).apply(leaves[0], leaves[0], leaves[0], leaves[1], leaves[2])[0].sum().backward()
    assert all(t.grad is not None and t.grad.dtype == t.dtype for t in leaves)


def test_frequencies_that_want_a_gradient_are_refused(stand_ins):
    """The rotation gives its frequencies none; learned ones would stay as they were, silently."""
    x, g, beta = torch.randn(1, 5, 2, 4).requires_grad_(), -torch.rand(1, 5, 2, 4), torch.rand(1, 5, 2)
    pos, freqs = torch.arange(5)[None], torch.ones(2, dtype=torch.float64)
    args = lambda f: (x, x, x, g, beta, None, None, None, pos, f)
    learned = freqs.clone().requires_grad_()
    with pytest.raises(ValueError, match="freqs"):
        kda.NormChunkKDA.apply(*args(learned))[0].sum().backward()
    with torch.no_grad():
        kda.NormChunkKDA.apply(*args(learned))  # without gradients they are as good as any
    kda.NormChunkKDA.apply(*args(freqs))[0].sum().backward()
    assert x.grad is not None
