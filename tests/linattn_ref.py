"""Plain 64-bit forms of linear attention with a decay for each head and of the group norm with an activation, a token and a
channel's formula at a time, on the CPU."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value


def decays(g):
    return torch.exp(torch.where(g > 0, 0.0, g.double()))


def spans(q, cu):
    """(rows view of [total, H, D] tensors, the spans of the sequences)."""
    if cu is None:
        B, T = q.shape[:2]
        return [(b * T, (b + 1) * T) for b in range(B)]
    return [(int(i), int(j)) for i, j in zip(cu[:-1], cu[1:])]


def rows(t):
    return t.reshape(-1, *t.shape[-2:]).double()


def attend(q, k, v, g, s0=None, cu=None, scale=1.0):
    """o (v's shape, zeros behind the last packed sequence) and the final states."""
    where, a = spans(q, cu), decays(g)[:, None, None]
    Q, K, V = rows(q), rows(k), rows(v)
    o = torch.zeros_like(V)
    end = torch.zeros((len(where), *K.shape[1:], V.shape[-1]), dtype=torch.float64)
    for n, (i, j) in enumerate(where):
        S = torch.zeros_like(end[n]) if s0 is None else s0[n].double()
        for t in range(i, j):
            S = a * S + K[t].unsqueeze(-1) * V[t].unsqueeze(-2)
            o[t] = scale * (Q[t].unsqueeze(-1) * S).sum(-2)
        end[n] = S
    return o.view(v.shape), end


def attend_grads(q, k, v, g, d_o, s0=None, d_sf=None, cu=None, scale=1.0):
    """dq, dk, dv, ds0 from the recurrence's reverse."""
    where, a = spans(q, cu), decays(g)[:, None, None]
    Q, K, V, D = rows(q), rows(k), rows(v), rows(d_o)
    dq, dk, dv = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    ds0 = torch.zeros((len(where), *K.shape[1:], V.shape[-1]), dtype=torch.float64)
    for n, (i, j) in enumerate(where):
        S = torch.zeros_like(ds0[n]) if s0 is None else s0[n].double()
        for t in range(i, j):
            S = a * S + K[t].unsqueeze(-1) * V[t].unsqueeze(-2)
            dq[t] = scale * (S * D[t].unsqueeze(-2)).sum(-1)
        G = torch.zeros_like(ds0[n]) if d_sf is None else d_sf[n].double()
        for t in range(j - 1, i - 1, -1):
            G = G + scale * Q[t].unsqueeze(-1) * D[t].unsqueeze(-2)
            dk[t] = (G * V[t].unsqueeze(-2)).sum(-1)
            dv[t] = (K[t].unsqueeze(-1) * G).sum(-2)
            G = a * G
        ds0[n] = G
    return dq.view(q.shape), dk.view(k.shape), dv.view(v.shape), ds0


def magnitude(f, *tensors, **kw):
    """f of the absolute values: what the roundings of its terms are relative to."""
    return f(*(t.abs() if i != 3 else t for i, t in enumerate(tensors)),
             **{n: t.abs() if isinstance(t, torch.Tensor) and n in ("s0", "d_sf", "d_o") else t for n, t in kw.items()})


def bound(dtype, ref, size, steps):
    """How far a result of `dtype` may be off: half a step of its own rounding, and of the sums before it one rounding of 32
    bits for each of at most `steps` additions on the way of a term, which has at most the magnitude `size`.  Products of
    16-bit operands take both as pairs of 16-bit numbers, off by at most half a step of half a step (2^-16) each: a term goes
    through its score, or through its weighted value and the state, two at most."""
    own = HALF[dtype] * ref.abs()
    return own + (steps * 2.0 ** -24 + (2 * 2.0 ** -16 if dtype == torch.bfloat16 else 0.0)) * size * (1 + HALF[dtype]) + 1e-37


def state_bound(ref, size, steps):
    """Of a state: 32 bits, its terms' products taken to 24 bits."""
    return (steps + 4) * 2.0 ** -24 * size + 1e-37


def group_norm(x, groups, w, b, gate, act, eps):
    """z, act's argument and the outputs, all [..., groups, width] but y, in 64 bits."""
    X = x.double().unflatten(-1, (groups, -1))
    mean = X.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(((X - mean) ** 2).mean(-1, keepdim=True) + eps)
    n = (X - mean) * r
    W = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    z = n * W.view(groups, -1) + (0.0 if b is None else b.double().view(groups, -1))
    u = z if gate is None else gate.double().unflatten(-1, (groups, -1))
    s = torch.sigmoid(u)
    f, slope = {"none": (u, torch.ones_like(u)), "silu": (u * s, s + u * s * (1 - s)), "sigmoid": (s, s * (1 - s))}[act]
    y = f if gate is None else z * f
    return {"n": n, "r": r, "z": z, "f": f, "slope": slope, "W": W.view(groups, -1), "y": y.flatten(-2)}


def group_norm_grads(x, groups, dy, w, b, gate, act, eps):
    p = group_norm(x, groups, w, b, gate, act, eps)
    D = dy.double().unflatten(-1, (groups, -1))
    dz = D * (p["slope"] if gate is None else p["f"])
    dn = dz * p["W"]
    dx = p["r"] * (dn - dn.mean(-1, keepdim=True) - p["n"] * (dn * p["n"]).mean(-1, keepdim=True))
    lead = tuple(range(x.dim() - 1))
    return {"dx": dx.flatten(-2), "dw": (dz * p["n"]).sum(lead).flatten(), "db": dz.sum(lead).flatten(),
            "dgate": None if gate is None else (D * p["z"] * p["slope"]).flatten(-2), "parts": (p, D, dz, dn)}


def inputs(seed, lead, H, Dk, Dv, dtype, n, kinds=None):
    """q, k, v, d_o, g, s0, d_sf on the CPU; kinds: the log decays, cyclic over the heads."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen).to(dtype)

    kinds = kinds or [-0.01, 0.0, -0.7, -math.inf, -40.0, 1.5, -1e-5, -6.0]
    g = torch.tensor([kinds[h % len(kinds)] for h in range(H)])
    q, k = normal(*lead, H, Dk, dtype=dtype), normal(*lead, H, Dk, dtype=dtype)
    v, d_o = normal(*lead, H, Dv, dtype=dtype), normal(*lead, H, Dv, dtype=dtype)
    return q, k, v, d_o, g, normal(n, H, Dk, Dv), normal(n, H, Dk, Dv)
