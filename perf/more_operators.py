"""What is measured of linear attention with a decay for each head, and of the group norm with an activation that its
outputs pass.

``own = False`` computes the plain forms (elementary torch operations in 32 bits); ``own = True`` makes the calls that a
user of the package makes.  Sizes: 16 heads of 128 channels with 8192 tokens and four sequences are this repository's own
prefill batch, 256 sequences of 32 heads its decode batch, 32 packed sequences its packed one; the others are generic.
"""
import math
import random

import torch

own = False

STEP, LIN, TRAIN, NORM, NORMTRAIN = "step", "lin", "lin_train", "norm", "norm_train"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases

def _lin(kind, seqs, tokens, heads, dk, dv, x="bf16", packed=False, state=True):
    """`tokens` per sequence, or in all sequences together where they are packed; state: whether there is one before."""
    return {"kind": kind, "seqs": seqs, "tokens": tokens, "heads": heads, "dk": dk, "dv": dv, "x": x, "packed": packed,
            "state": state}


def _norm(kind, tokens, groups, width, x="bf16", y="bf16", act="silu", gate=True, affine=True, fused=False):
    """gate: the activation is of a second tensor that multiplies the normed one; fused: that tensor is columns of a
    wider projection."""
    return {"kind": kind, "tokens": tokens, "groups": groups, "width": width, "x": x, "y": y, "act": act, "gate": gate,
            "affine": affine, "fused": fused}


def listed():
    cases = {
        # serving: a token of each of few running sequences; latency counts
        "lin_step_b4_h8_d64": _lin(STEP, 4, 1, 8, 64, 64),
        # serving: the repository's decode batch
        "lin_step_b256_h32_d128": _lin(STEP, 256, 1, 32, 128, 128),
        # prefill of the repository's batch
        "lin_b4_t8192_h16_d128": _lin(LIN, 4, 8192, 16, 128, 128, state=False),
        # one long document with few heads: the time axis has to be split
        "lin_b1_t131072_h8_d128": _lin(LIN, 1, 131072, 8, 128, 128),
        # packed ragged prompts of a serving batch, keys narrower than values
        "lin_packed_n32_h16_d64_128": _lin(LIN, 32, 40011, 16, 64, 128, packed=True),
        # a short odd prompt in fp32
        "lin_b2_t333_h4_d128_f32": _lin(LIN, 2, 333, 4, 128, 128, x="f32"),
        # a training step
        "lin_train_b4_t4096_h16_d128": _lin(TRAIN, 4, 4096, 16, 128, 128, state=False),
        # a training step over packed documents, values narrower than keys
        "lin_train_packed_n16_h8_d128_64": _lin(TRAIN, 16, 24001, 8, 128, 64, packed=True),
        # serving: the outputs of one token of each of 64 running sequences, gated
        "norm_t64_g16_w128": _norm(NORM, 64, 16, 128),
        # prefill: fp32 outputs of the repository's recurrence on that batch, gated by columns of a projection, to bf16
        "norm_t32768_g16_w128_f32": _norm(NORM, 32768, 16, 128, x="f32", act="sigmoid", fused=True),
        # a training step of the gated norm
        "norm_train_t32768_g16_w128": _norm(NORMTRAIN, 32768, 16, 128),
        # training in fp32 without a gate, rows that wide loads do not divide
        "norm_train_t4099_g12_w90_f32": _norm(NORMTRAIN, 4099, 12, 90, x="f32", y="f32", gate=False),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice([STEP, LIN, LIN, TRAIN, TRAIN, NORM, NORMTRAIN])
    if kind in (NORM, NORMTRAIN):
        width = rng.choice([64, 128, 256, _spread(rng, 16, 1024)])
        groups = _spread(rng, 1, max(1, min(64, 8192 // width)))
        x, y = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        gate = rng.random() < 0.6
        tokens = _spread(rng, 1, min(1 << 16, (1 << 26) // SIZE[x] * 2 // (groups * width)))
        return _norm(kind, tokens, groups, width, x, y, rng.choice(["silu", "sigmoid", "none"] if not gate else
                                                                   ["silu", "sigmoid"]),
                     gate, rng.random() < 0.7, gate and rng.random() < 0.4)
    dk, dv, x = rng.choice([64, 128]), rng.choice([64, 128]), rng.choice(["bf16", "bf16", "f32"])
    heads = _spread(rng, 1, 32)
    if kind == STEP:
        return _lin(STEP, _spread(rng, 1, 256), 1, heads, dk, dv, x)
    packed, seqs = rng.random() < 0.5, _spread(rng, 1, 32)
    most = (1 << (25 if kind == TRAIN else 26)) // (heads * max(dk, dv) * SIZE[x] // 2)
    tokens = _spread(rng, 1, min(131072, most))
    if not packed:
        tokens = max(1, tokens // seqs)
    return _lin(kind, seqs, tokens, heads, dk, dv, x, packed, rng.random() < 0.5)


def _offsets(case):
    """Where the sequences begin, and the end: lengths that differ widely, an empty one and one of a token among them."""
    n, tokens = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [i * tokens for i in range(n + 1)]
    rng = random.Random(n * 1000003 + tokens)
    cuts = sorted(rng.randint(0, tokens) for _ in range(n - 1))
    if n >= 4:
        cuts[1], cuts[2] = cuts[0], min(tokens, cuts[0] + 1)
        cuts.sort()
    return [0] + cuts + [tokens]


def work(case):
    kind = case["kind"]
    if kind in (NORM, NORMTRAIN):
        n = case["tokens"] * case["groups"] * case["width"]
        xb, yb, gates = SIZE[case["x"]], SIZE[case["y"]], int(case["gate"])
        if kind == NORM:
            return {"bytes": n * (xb + yb * (1 + gates)), "flops": 12 * n}
        return {"bytes": n * (2 * xb + yb * (2 + 2 * gates)), "flops": 35 * n}
    xb, dk, dv = SIZE[case["x"]], case["dk"], case["dv"]
    rows = (case["seqs"] if kind == STEP else _offsets(case)[-1]) * case["heads"]
    states = case["seqs"] * case["heads"] * dk * dv * 4
    given = int(case["state"] or kind == STEP)
    # token by token, an element of the state is decayed (1), gains a product (2) and is read (2); the backward pass makes
    # the state again and does as much with its gradient, which is read twice
    # an element of the state is decayed, gains a product and is read, for each token: six operations; the gradients
    # take twice as many products again
    if kind in (STEP, LIN):
        return {"bytes": rows * (2 * dk + 2 * dv) * xb + states * (1 + given), "flops": 5 * rows * dk * dv}
    return {"bytes": rows * (4 * dk + 4 * dv) * xb + states * (2 + 2 * given), "flops": 17 * rows * dk * dv}


# ------------------------------------------------------------------------------------------------ inputs

CHUNK = 128  # tokens that the plain form takes together


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["kind"] in (NORM, NORMTRAIN):
        t, c = case["tokens"], case["groups"] * case["width"]
        x_type, y_type = TYPES[case["x"]], TYPES[case["y"]]
        # the recurrence's outputs: heads of different size, a mean that is not zero
        size = torch.exp(normal(1, case["groups"], 1))
        x = (normal(t, case["groups"], case["width"]) + 0.3 * normal(t, case["groups"], 1)) * size
        s["x"] = x.to(x_type).view(t, c)
        s["w"] = 1 + 0.1 * normal(c) if case["affine"] else None
        s["b"] = 0.1 * normal(c) if case["affine"] else None
        s["gate"] = None
        if case["gate"]:
            s["gate"] = normal(t, 2 * c, dtype=y_type)[:, c:] if case["fused"] else normal(t, c, dtype=y_type)
        s["eps"] = 1e-5
        if case["kind"] == NORMTRAIN:
            s["dy"] = normal(t, c, dtype=y_type)
        return s
    x_type, n, h, dk, dv = TYPES[case["x"]], case["seqs"], case["heads"], case["dk"], case["dv"]
    shape = (n,) if case["kind"] == STEP else (case["tokens"],) if case["packed"] else (n, case["tokens"])
    s["q"], s["k"] = (normal(*shape, h, dk, dtype=x_type, scale=dk ** -0.25) for _ in range(2))
    s["v"] = normal(*shape, h, dv, dtype=x_type)
    # a memory of 2 to 1024 tokens, spread over the heads, and one head that forgets nothing
    reach = 1 + 9 * (torch.arange(h, device="cuda", dtype=torch.float64) + torch.rand(
        h, generator=gen, device="cuda", dtype=torch.float64)) / h
    s["g"] = torch.log1p(-torch.exp2(-reach)).float()
    if h > 4:
        s["g"][h - 1] = 0.0
    s["s0"] = normal(n, h, dk, dv, scale=0.5) if case["state"] or case["kind"] == STEP else None
    s["scale"] = dk ** -0.5
    if case["kind"] == STEP:
        return s
    at = _offsets(case)
    s["cu"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    if case["kind"] == TRAIN:
        s["do"], s["ds"] = normal(*shape, h, dv, dtype=x_type), normal(n, h, dk, dv, scale=0.5)
    # for the plain form: pieces of up to CHUNK tokens of a sequence each
    pieces = [(i, p, min(CHUNK, at[i + 1] - p)) for i in range(n) for p in range(at[i], at[i + 1], CHUNK)]
    whose, first, size = (torch.tensor(x, device="cuda") for x in zip(*pieces))
    row = torch.arange(CHUNK, device="cuda")
    s["whose"], s["first"], s["size"] = whose, first, size
    s["begin"] = torch.tensor(at[:-1], device="cuda")[whose]
    s["end"] = torch.tensor(at[1:], device="cuda")
    s["inside"] = row < size[:, None]
    s["rows"] = torch.where(s["inside"], first[:, None] + row, 0)
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_step(s):
    a = torch.exp(s["g"])[:, None, None]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    state = a * s["s0"] + k[..., :, None] * v[..., None, :]
    o = s["scale"] * torch.matmul(q[..., None, :], state)[..., 0, :]
    return {"o": o.to(s["q"].dtype), "s": state}


def _pieces(s, x):
    """x [..., H, D] as fp32 pieces [H, pieces, CHUNK, D], zeros behind the last token of each."""
    flat = x.reshape(-1, *x.shape[-2:]).float()
    return torch.where(s["inside"][..., None, None], flat[s["rows"]], 0.0).permute(2, 0, 1, 3).contiguous()


def _powers(g, steps, where):
    """exp(g steps) for each head where `where`, else zero; the product of a small rate and a long way in 64 bits."""
    shown = (slice(None), *(None,) * steps.dim())
    return torch.where(where, torch.exp(g.double()[shown] * torch.where(where, steps, 0).double()), 0.0).float()


def _attend(s, g, q, k, v, begin, back):
    """o_t = sum over i up to t (from t on with `back`) of a^|t - i| (q_t . k_i) v_i, and the states at the ends: `begin`
    is what there is before the first token (behind the last one).  Pieces [H, P, CHUNK, D]."""
    h, p, c, dk = q.shape
    dv = v.shape[-1]
    row, size, first = torch.arange(c, device=g.device), s["size"], s["first"]
    apart = row[:, None] - row
    if back:
        apart = -apart
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2).contiguous()) * _powers(g, apart, apart >= 0)[:, None], v)
    # what a piece leaves at its end (with `back` before its first token)
    left = row + 1 + 0 * size[:, None] if back else size[:, None] - 1 - row
    weight = _powers(g, left, s["inside"])
    own_part = torch.matmul((k * weight[..., None]).transpose(-1, -2).contiguous(), v).view(h, p, dk * dv)
    same = s["whose"][:, None] == s["whose"]
    if back:
        gap = first - (first + size)[:, None]  # from the end of piece i to the begin of piece j
        before = same & (first > first[:, None])
        reach, since = row - size[:, None], s["end"][s["whose"]] - first - size
        start = begin
    else:
        gap = first[:, None] - (first + size)
        before = same & (first < first[:, None])
        reach, since = row + 1 + 0 * size[:, None], first - s["begin"]
        start = begin
    at = torch.matmul(_powers(g, gap, before), own_part)
    if start is not None:
        start = start.transpose(0, 1).reshape(h, -1, dk * dv)
        at = at + _powers(g, since, since >= 0)[..., None] * start[:, s["whose"]]
    at = at.view(h, p, dk, dv)
    if back:
        reach = -reach - 1  # a row's way to the end of its piece, without its own decay
    o = o + _powers(g, reach, s["inside"])[..., None] * torch.matmul(q, at)
    # the whole sequence's state: every piece's part, brought to the end
    n = s["end"].numel()
    own_seq = torch.arange(n, device=g.device)[:, None] == s["whose"]
    begins = s["cu"][:-1].long()
    far = (first - begins[s["whose"]] if back else s["end"][s["whose"]] - first - size).expand(n, p)
    whole = torch.matmul(_powers(g, far, own_seq), own_part)
    if start is not None:
        length = s["end"] - begins
        whole = whole + _powers(g, length, length >= 0)[..., None] * start
    return o, whole.view(h, n, dk, dv).transpose(0, 1).contiguous()


def _rows(s, o, like):
    """Pieces back to the rows of `like`."""
    out = torch.empty((like.numel() // (o.shape[0] * o.shape[-1]), o.shape[0], o.shape[-1]), dtype=like.dtype,
                      device=like.device)
    out[s["rows"][s["inside"]]] = o.permute(1, 2, 0, 3)[s["inside"]].to(like.dtype)
    return out.view(*like.shape[:-1], o.shape[-1])


def _plain_lin(s):
    g, scale = s["g"], s["scale"]
    q, k, v = (_pieces(s, s[n]) for n in ("q", "k", "v"))
    o, end = _attend(s, g, q * scale, k, v, s["s0"], False)
    out = {"o": _rows(s, o, s["v"]), "s": end}
    if s["case"]["kind"] == LIN:
        return out
    do = _pieces(s, s["do"])
    turned = None if s["s0"] is None else s["s0"].transpose(-1, -2)
    dq, _ = _attend(s, g, do, v, k, turned, False)
    dk, _ = _attend(s, g, v, do, q * scale, s["ds"].transpose(-1, -2), True)
    dv, ds0 = _attend(s, g, k, q * scale, do, s["ds"], True)
    out |= {"dq": _rows(s, dq * scale, s["q"]), "dk": _rows(s, dk, s["k"]), "dv": _rows(s, dv, s["v"])}
    if s["s0"] is not None:
        out["ds0"] = ds0
    return out


def _plain_norm(s):
    c = s["case"]
    shape = (c["tokens"], c["groups"], c["width"])

    def split(t):
        return None if t is None else t.float().reshape(-1, *shape[1:])

    x, w, b, gate = split(s["x"]), split(s["w"]), split(s["b"]), split(s["gate"])
    centred = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((centred * centred).mean(-1, keepdim=True) + s["eps"])
    n = centred * r
    z = n if w is None else n * w + b
    u = z if gate is None else gate
    sig = 1 / (1 + torch.exp(-u))
    f, slope = {"silu": (u * sig, sig * (1 + u * (1 - sig))), "sigmoid": (sig, sig * (1 - sig)),
                "none": (u, torch.ones_like(u))}[c["act"]]
    y = f if gate is None else z * f
    out = {"y": y.to(TYPES[c["y"]]).view(s["x"].shape)}
    if c["kind"] == NORM:
        return out
    dy = split(s["dy"])
    dz = dy * slope if gate is None else dy * f
    dn = dz if w is None else dz * w
    dx = r * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    out["dx"] = dx.to(TYPES[c["x"]]).view(s["x"].shape)
    if gate is not None:
        out["dgate"] = (dy * z * slope).to(TYPES[c["y"]]).view(s["x"].shape)
    if w is not None:
        out["dw"], out["db"] = (dz * n).sum(0).view(-1), dz.sum(0).view(-1)
    return out


# ------------------------------------------------------------------------------------------------ the framework's calls

def _own_lin(kda, s):
    c, scale = s["case"], s["scale"]
    if c["kind"] == STEP:
        o, end = kda.linattn_step(s["q"], s["k"], s["v"], s["g"], s["s0"], scale=scale)
        return {"o": o, "s": end}
    args = (s["q"], s["k"], s["v"], s["g"])
    if c["packed"]:
        o, end = kda.linattn_varlen_fwd(*args, s["cu"], s["s0"], scale=scale)
    else:
        o, end = kda.linattn_fwd(*args, s["s0"], scale=scale)
    out = {"o": o, "s": end}
    if c["kind"] == LIN:
        return out
    if c["packed"]:
        dq, dk, dv, ds0 = kda.linattn_varlen_bwd(*args, s["cu"], s["do"], s["s0"], s["ds"], scale=scale)
    else:
        dq, dk, dv, ds0 = kda.linattn_bwd(*args, s["do"], s["s0"], s["ds"], scale=scale)
    out |= {"dq": dq, "dk": dk, "dv": dv}
    if s["s0"] is not None:
        out["ds0"] = ds0
    return out


def _own_norm(kda, s):
    c = s["case"]
    form = {"weight": s["w"], "bias": s["b"], "gate": s["gate"], "act": c["act"], "eps": s["eps"]}
    out = {"y": kda.group_norm_act_fwd(s["x"], c["groups"], dtype=TYPES[c["y"]], **form)}
    if c["kind"] == NORM:
        return out
    dx, dw, db, dgate = kda.group_norm_act_bwd(s["x"], c["groups"], s["dy"], **form)
    out["dx"] = dx
    if c["gate"]:
        out["dgate"] = dgate
    if c["affine"]:
        out["dw"], out["db"] = dw, db
    return out


def run(state):
    kind = state["case"]["kind"]
    if own:
        import gated_delta_rule_65_amd as kda
        return _own_norm(kda, state) if kind in (NORM, NORMTRAIN) else _own_lin(kda, state)
    if kind in (NORM, NORMTRAIN):
        return _plain_norm(state)
    return _plain_step(state) if kind == STEP else _plain_lin(state)


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_lin(s):
    """The recurrence, a token of each sequence at a time: the longest sequences first, so that those that still run are
    the first ones of the batch."""
    c = s["case"]
    n, h = c["seqs"], c["heads"]
    at = list(range(n + 1)) if c["kind"] == STEP else _offsets(c)
    lengths = [at[i + 1] - at[i] for i in range(n)]
    order = sorted(range(n), key=lambda i: -lengths[i])
    begins = torch.tensor([at[i] for i in order], device="cuda")
    a = torch.exp(s["g"].double())[:, None, None]
    flat = {x: s[x].reshape(-1, *s[x].shape[-2:]).double() for x in ("q", "k", "v", "do") if x in s}
    q, k, v, scale = flat["q"], flat["k"], flat["v"], s["scale"]
    running = [sum(x > t for x in lengths) for t in range(max(lengths))]
    state = torch.zeros((n, h, c["dk"], c["dv"]), dtype=torch.float64, device="cuda")
    if s["s0"] is not None:
        state = s["s0"].double()[order]
    back = torch.empty_like(state)
    o = torch.empty_like(v)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    train = c["kind"] == TRAIN
    for t, m in enumerate(running):
        rows = begins[:m] + t
        now = state[:m]
        now.mul_(a).addcmul_(k[rows].unsqueeze(-1), v[rows].unsqueeze(-2))
        o[rows] = scale * (q[rows].unsqueeze(-1) * now).sum(-2)
        if train:
            dq[rows] = scale * (now * flat["do"][rows].unsqueeze(-2)).sum(-1)
    back[order] = state
    out = {"o": o.view(s["v"].shape), "s": back.clone()}
    if not train:
        return out
    grad = s["ds"].double()[order]
    for t in range(len(running) - 1, -1, -1):
        m = running[t]
        rows = begins[:m] + t
        now = grad[:m]
        now.addcmul_(q[rows].unsqueeze(-1), scale * flat["do"][rows].unsqueeze(-2))
        dk[rows] = (now * v[rows].unsqueeze(-2)).sum(-1)
        dv[rows] = (k[rows].unsqueeze(-1) * now).sum(-2)
        now.mul_(a)
    back[order] = grad
    out |= {"dq": dq.view(s["q"].shape), "dk": dk.view(s["k"].shape), "dv": dv.view(s["v"].shape)}
    if s["s0"] is not None:
        out["ds0"] = back
    return out


def _exact_norm(s):
    c = s["case"]
    g, width = c["groups"], c["width"]
    x = s["x"].double().view(-1, g, width)
    spread, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    size = torch.sqrt(spread + s["eps"])
    n = (x - mean) / size
    w = torch.ones(g * width, dtype=torch.float64, device="cuda") if s["w"] is None else s["w"].double()
    b = torch.zeros_like(w) if s["b"] is None else s["b"].double()
    w, b = w.view(g, width), b.view(g, width)
    z = n * w + b
    u = z if s["gate"] is None else s["gate"].double().reshape(-1, g, width)
    half = 0.5 * (1 + torch.tanh(u / 2))
    if c["act"] == "silu":
        f, slope = u * half, half + u * half * (1 - half)
    elif c["act"] == "sigmoid":
        f, slope = half, half * (1 - half)
    else:
        f, slope = u, torch.ones_like(u)
    flat = s["x"].shape
    out = {"y": (f if s["gate"] is None else f * z).view(flat)}
    if c["kind"] == NORM:
        return out
    dy = s["dy"].double().view(-1, g, width)
    dz = dy * (slope if s["gate"] is None else f)
    dn = dz * w
    along = torch.einsum("tgc,tgc->tg", dn, n)[..., None] / width
    out["dx"] = ((dn - dn.sum(-1, keepdim=True) / width - along * n) / size).view(flat)
    if s["gate"] is not None:
        out["dgate"] = (dy * z * slope).view(flat)
    if s["w"] is not None:
        out["dw"], out["db"] = torch.einsum("tgc,tgc->gc", dz, n).view(-1), dz.sum(0).view(-1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["kind"] in (NORM, NORMTRAIN) else _exact_lin(s)
