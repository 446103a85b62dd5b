"""The 64-bit forms that the linear attention and the group norm are held to, against closed forms, torch's own and differences;
and the autograd functions' own work, with plain stand-ins for the calls that run kernels.  All on the CPU."""
import math

import pytest
import torch

import gated_delta_rule_65_amd as kda
from gated_delta_rule_65_amd import groupnorm, layer, linattn
from tests import linattn_ref as ref


def test_closed_form_of_a_constant_sequence():
    """k_t v_t^T = k v^T for all t: S_t is (1 - a^t) / (1 - a) of it, and a^t S_0."""
    T, a = 37, 0.9
    g = torch.tensor([math.log(a)], dtype=torch.float64)
    q, k, v = (torch.randn(1, 1, 1, n, dtype=torch.float64).expand(1, T, 1, n) for n in (3, 3, 5))
    s0 = torch.randn(1, 1, 3, 5, dtype=torch.float64)
    o, end = ref.attend(q, k, v, g, s0, None, 0.5)
    outer = k[0, 0, 0][:, None] * v[0, 0, 0][None]
    for t in range(1, T + 1):
        S = (1 - a ** t) / (1 - a) * outer + a ** t * s0[0, 0]
        assert torch.allclose(o[0, t - 1, 0], 0.5 * q[0, 0, 0] @ S, rtol=1e-12)
    assert torch.allclose(end[0, 0], S, rtol=1e-12)


def test_decays_of_none_and_all():
    """g = 0 (or above) forgets nothing: cumulative sums.  Minus infinity keeps nothing: the token alone."""
    q, k, v, _, _, s0, _ = ref.inputs(1, (1, 9), 2, 4, 6, torch.float32, 1)
    o, end = ref.attend(q, k, v, torch.tensor([2.0, -math.inf]), s0)
    sums = torch.cumsum(k.double().unsqueeze(-1) * v.double().unsqueeze(-2), 1)[0, :, 0] + s0[0, 0].double()
    assert torch.allclose(o[0, :, 0], (q[0, :, 0].double().unsqueeze(1) @ sums)[:, 0], rtol=1e-12)
    dots = (q[0, :, 1].double() * k[0, :, 1].double()).sum(-1, keepdim=True)
    assert torch.allclose(o[0, :, 1], dots * v[0, :, 1].double(), rtol=1e-12)
    assert torch.allclose(end[0, 1], k[0, -1, 1].double()[:, None] * v[0, -1, 1].double()[None], rtol=1e-12)


@pytest.mark.parametrize("packed", [False, True])
def test_gradients_of_the_form(packed):
    """The reverse recurrence against torch's gradients through the forward one."""
    q, k, v, d_o, g, s0, d_sf = (t.double() for t in ref.inputs(2, (2, 11) if not packed else (25,), 3, 4, 6, torch.float32, 2))
    cu = torch.tensor([0, 9, 22]) if packed else None
    leaves = [t.clone().requires_grad_() for t in (q, k, v, s0)]
    a = torch.exp(g.clamp(max=0))[:, None, None]
    rows = [t.reshape(-1, *t.shape[-2:]) for t in leaves[:3]]
    loss = 0.0
    for n, (i, j) in enumerate(ref.spans(q, cu)):
        S = leaves[3][n]
        for t in range(i, j):
            S = a * S + rows[1][t].unsqueeze(-1) * rows[2][t].unsqueeze(-2)
            loss = loss + (0.3 * (rows[0][t].unsqueeze(-1) * S).sum(-2) * d_o.reshape(-1, 3, 6)[t]).sum()
        loss = loss + (S * d_sf[n]).sum()
    loss.backward()
    for leaf, want in zip(leaves, ref.attend_grads(q, k, v, g, d_o, s0, d_sf, cu, 0.3)):
        assert torch.allclose(leaf.grad, want, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
def test_group_norm_form(act, gated):
    x, w, b, gate, dy = (torch.randn(n, dtype=torch.float64) for n in ((7, 12), (12,), (12,), (7, 12), (7, 12)))
    gate = gate if gated else None
    leaves = [t.clone().requires_grad_() for t in (x, w, b)] + ([gate.clone().requires_grad_()] if gated else [])
    z = torch.nn.functional.group_norm(leaves[0], 3, leaves[1], leaves[2], 1e-3)
    f = {"none": lambda u: u, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[act]
    y = z * f(leaves[3]) if gated else f(z)
    assert torch.allclose(y, ref.group_norm(x, 3, w, b, gate, act, 1e-3)["y"], rtol=1e-12, atol=1e-14)
    y.backward(dy)
    got = ref.group_norm_grads(x, 3, dy, w, b, gate, act, 1e-3)
    for leaf, name in zip(leaves, ("dx", "dw", "db", "dgate")):
        assert torch.allclose(leaf.grad, got[name], rtol=1e-9, atol=1e-12)


@pytest.fixture
def stand_ins(monkeypatch):
    def fwd(q, k, v, g, s0=None, *, scale=1.0, **kw):
        o, s = ref.attend(q.detach(), k.detach(), v.detach(), g.detach(), s0, None, scale)
        return o.to(q.dtype), s.float()

    def bwd(q, k, v, g, d_o, s0=None, d_sfinal=None, *, scale=1.0, **kw):
        assert d_o.dtype == q.dtype and d_o.is_contiguous() and d_sfinal.dtype == torch.float32
        return tuple(t.to(q.dtype) for t in ref.attend_grads(q, k, v, g, d_o, s0, d_sfinal, None, scale))

    def varlen_fwd(q, k, v, g, cu, s0=None, *, scale=1.0, **kw):
        o, s = ref.attend(q.detach(), k.detach(), v.detach(), g.detach(), s0, cu, scale)
        o[cu[-1]:] = math.nan  # unwritten
        return o.to(q.dtype), s.float()

    def varlen_bwd(q, k, v, g, cu, d_o, s0=None, d_sfinal=None, *, scale=1.0, **kw):
        out = ref.attend_grads(q, k, v, g, d_o, s0, d_sfinal, cu, scale)
        for t in out[:3]:
            t[cu[-1]:] = math.nan
        return tuple(t.to(q.dtype) for t in out)

    def zero_behind(cu, *tensors):
        for t in tensors:
            t[cu[-1]:] = 0

    def norm_fwd(x, groups, *, weight=None, bias=None, gate=None, act="silu", eps=1e-5, dtype=None):
        return ref.group_norm(x.detach(), groups, weight, bias, gate, act, eps)["y"].detach().to(dtype or x.dtype)

    def norm_bwd(x, groups, dy, *, weight=None, bias=None, gate=None, act="silu", eps=1e-5, **kw):
        p = ref.group_norm_grads(x, groups, dy, weight, bias, gate, act, eps)
        return (p["dx"].to(x.dtype), None if weight is None else p["dw"].float(), None if bias is None else p["db"].float(),
                None if gate is None else p["dgate"].to(gate.dtype))

    for name, f in (("linattn_fwd", fwd), ("linattn_bwd", bwd), ("linattn_varlen_fwd", varlen_fwd), ("linattn_varlen_bwd", varlen_bwd)):
        monkeypatch.setattr(linattn, name, f)
    monkeypatch.setattr(layer, "_zero_behind", zero_behind)
    monkeypatch.setattr(groupnorm, "group_norm_act_fwd", norm_fwd)
    monkeypatch.setattr(groupnorm, "group_norm_act_bwd", norm_bwd)


def applied(name, x, g):
    """An autograd function's outputs at x, [1, T, H, D]."""
    if name == "LinearAttention":
        return kda.LinearAttention.apply(x, x, x, g)[0]
    if name == "VarlenLinearAttention":
        rows = x.flatten(0, 1)
        return kda.VarlenLinearAttention.apply(rows, rows, rows, g, torch.tensor([0, 2, x.shape[1] - 1], dtype=torch.int32))[0]
    return kda.GroupNormAct.apply(x.flatten(2), 2, g.repeat_interleave(4).detach(), None, x.flatten(2), "silu")


NAMES = ["LinearAttention", "VarlenLinearAttention", "GroupNormAct"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_of_gradients_are_refused(stand_ins, name, weighted):
    x = torch.randn(1, 5, 2, 4).requires_grad_()
    y = applied(name, x, torch.tensor([-0.1, -0.5]))
    loss = ((y * y).sum() if weighted else y.sum()) + (x ** 3).sum()
    dx, = torch.autograd.grad(loss, x, create_graph=True)
    assert torch.isfinite(dx).all()  # rows behind the last sequence have zeros
    with pytest.raises(RuntimeError, match="first-order"):
        (dx ** 2).sum().backward()


@pytest.mark.parametrize("name", NAMES)
def test_what_is_kept_passes_the_hooks_of_saved_tensors(stand_ins, name):
    x, kinds = torch.randn(1, 5, 2, 4).requires_grad_(), []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kinds.append(t.dtype) or t.clone(), lambda t: t):
        y = applied(name, x, torch.tensor([-0.1, -0.5]))
    assert (torch.int32 in kinds) == (name == "VarlenLinearAttention")
    y.sum().backward()
    assert torch.isfinite(x.grad).all() and bool(x.grad.any())


@pytest.mark.parametrize("name", ["LinearAttention", "VarlenLinearAttention"])
def test_decays_that_want_a_gradient_are_refused(stand_ins, name):
    x, g = torch.randn(1, 5, 2, 4).requires_grad_(), torch.tensor([-0.1, -0.5]).requires_grad_()
    with pytest.raises(ValueError, match="constants"):
        applied(name, x, g).sum().backward()
    with torch.no_grad():
        applied(name, x, g)  # without gradients they are as good as any


def test_offsets_changed_before_the_backward_pass_are_an_error(stand_ins):
    x, cu = torch.randn(6, 2, 4).requires_grad_(), torch.tensor([0, 2, 6], dtype=torch.int32)
    o, _ = kda.VarlenLinearAttention.apply(x, x, x, torch.tensor([-0.1, -0.5]), cu)
    cu.copy_(torch.tensor([0, 5, 6]))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


def test_a_shared_weight_and_state_have_the_sum_of_their_gradients(stand_ins):
    """One initial state for all sequences, one norm weight for two norms."""
    x, s0 = torch.randn(2, 5, 2, 4), torch.randn(1, 2, 4, 4).requires_grad_()
    g = torch.tensor([-0.1, -0.5])
    o, s = kda.LinearAttention.apply(x, x, x, g, s0.expand(2, -1, -1, -1))
    (o.sum() + s.sum()).backward()
    want = ref.attend_grads(x, x, x, g, torch.ones_like(x), s0.detach().expand(2, -1, -1, -1), torch.ones(2, 2, 4, 4))[3].sum(0)
    assert torch.allclose(s0.grad[0].double(), want, rtol=1e-5, atol=1e-5)
    w = torch.randn(8).requires_grad_()
    y = kda.GroupNormAct.apply(x.flatten(2), 2, w, None, None, "silu") * 2 + kda.GroupNormAct.apply(x.flatten(2), 2, w, None, None, "none")
    y.sum().backward()
    one = torch.ones(2, 5, 8)
    want = (ref.group_norm_grads(x.flatten(2), 2, 2 * one, w.detach(), None, None, "silu", 1e-5)["dw"] +
            ref.group_norm_grads(x.flatten(2), 2, one, w.detach(), None, None, "none", 1e-5)["dw"])
    assert torch.allclose(w.grad.double(), want, rtol=1e-4, atol=1e-4)
