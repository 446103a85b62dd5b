"""What the autograd functions of linear attention and of the group norm ask the calls that run kernels for, with plain stand-ins on
the CPU."""
import pytest
import torch

import gated_delta_rule_65_amd as kda
from tests import linattn_ref as ref
from tests.test_linattn_ref import stand_ins  # noqa: F401

G = torch.tensor([-0.1, -0.5])


@pytest.fixture
def asked(stand_ins, monkeypatch):  # noqa: F811
    """What each call got, by name; a state or a gradient that is not asked for is not there."""
    seen = {}

    def fwd(name, f):
        def run(*args, output_final_state=True, **kw):
            seen[name] = {"final": output_final_state}
            o, s = f(*args, **kw)
            return o, (s if output_final_state else None)
        return run

    def bwd(name, f, at):
        def run(*args, output_ds0=True, **kw):
            seen[name] = {"d_sfinal": args[at], "ds0": output_ds0}
            args = list(args)
            if args[at] is None:
                args[at] = torch.zeros(1, 2, 4, 4)
            *grads, ds0 = f(*args, **kw)
            return (*grads, ds0 if output_ds0 else None)
        return run

    from gated_delta_rule_65_amd import linattn
    for name in ("linattn_fwd", "linattn_varlen_fwd"):
        monkeypatch.setattr(linattn, name, fwd(name, getattr(linattn, name)))
    monkeypatch.setattr(linattn, "linattn_bwd", bwd("linattn_bwd", linattn.linattn_bwd, 6))
    monkeypatch.setattr(linattn, "linattn_varlen_bwd", bwd("linattn_varlen_bwd", linattn.linattn_varlen_bwd, 7))
    return seen


def leaves(packed):
    x = torch.randn((5, 2, 4) if packed else (1, 5, 2, 4)).requires_grad_()
    return x, torch.randn(1, 2, 4, 4).requires_grad_(), (torch.tensor([0, 5], dtype=torch.int32),) if packed else ()


@pytest.mark.parametrize("packed", [False, True])
def test_states_that_nobody_asks_for(asked, packed):
    """Without a final state none is written and no gradient of it is read; a state before that wants no gradient has none."""
    f, tag = (kda.VarlenLinearAttention, "linattn_varlen") if packed else (kda.LinearAttention, "linattn")
    x, s0, cu = leaves(packed)
    for before, wanted in ((None, False), (s0.detach(), False), (s0, True)):
        x.grad = s0.grad = None
        o, s = f.apply(x, x, x, G, *cu, before, 0.5, False)
        assert s is None and asked[tag + "_fwd"] == {"final": False}
        o.sum().backward()
        assert asked[tag + "_bwd"] == {"d_sfinal": None, "ds0": wanted}
        assert (s0.grad is not None) == wanted
        rows = x.detach().view(1, 5, 2, 4)
        want = ref.attend_grads(rows, rows, rows, G, torch.ones(1, 5, 2, 4), None if before is None else before.detach(), None, None, 0.5)
        assert torch.allclose(x.grad.double().view(1, 5, 2, 4), sum(want[:3]), rtol=1e-5, atol=1e-5)
        if wanted:
            assert torch.allclose(s0.grad.double(), want[3], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("packed", [False, True])
def test_a_final_state_is_there_unless_it_is_left_out(asked, packed):
    f, tag = (kda.VarlenLinearAttention, "linattn_varlen") if packed else (kda.LinearAttention, "linattn")
    x, s0, cu = leaves(packed)
    o, s = f.apply(x, x, x, G, *cu, s0)
    (o.sum() + 2 * s.sum()).backward()
    assert asked[tag + "_fwd"] == {"final": True} and asked[tag + "_bwd"]["ds0"]
    assert torch.equal(asked[tag + "_bwd"]["d_sfinal"], torch.full((1, 2, 4, 4), 2.0)) and s0.grad is not None


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_weights_that_want_no_gradient(stand_ins, monkeypatch, weight, bias):  # noqa: F811
    """The sums over tokens are made only where the weight or the bias wants one."""
    from gated_delta_rule_65_amd import groupnorm
    whole, seen = groupnorm.group_norm_act_bwd, {}

    def bwd(*args, output_dweights=True, **kw):
        seen["sums"] = output_dweights
        dx, dw, db, dgate = whole(*args, **kw)
        return (dx, dw, db, dgate) if output_dweights else (dx, None, None, dgate)

    monkeypatch.setattr(groupnorm, "group_norm_act_bwd", bwd)
    x, w, b = torch.randn(3, 8).requires_grad_(), torch.randn(8), torch.randn(8)
    kda.GroupNormAct.apply(x, 2, w.requires_grad_(weight), b.requires_grad_(bias), None, "silu").sum().backward()
    assert seen["sums"] == (weight or bias) and (w.grad is not None) == weight and (b.grad is not None) == bias
    want = ref.group_norm_grads(x.detach(), 2, torch.ones(3, 8), w.detach(), b.detach(), None, "silu", 1e-5)
    assert torch.allclose(x.grad.double(), want["dx"], rtol=1e-5, atol=1e-5)
    for leaf, name in ((w, "dw"), (b, "db")):
        assert leaf.grad is None or torch.allclose(leaf.grad.double(), want[name], rtol=1e-5, atol=1e-5)
