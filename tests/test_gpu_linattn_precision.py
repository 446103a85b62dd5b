"""Linear attention where terms cancel: the state, the scores and the weighted values hold 32-bit floats' 24 bits in every type, so
that an output is off by its own rounding and by a few roundings of 32 bits of its terms, however small it is beside them."""
import pytest
import torch

import gated_delta_rule_65_amd as kda
from tests import linattn_ref as ref
from tests.test_gpu_linattn import TYPES, gpu, near

pytestmark = pytest.mark.gpu
G = -2.0 ** -12  # two tokens next to each other, opposite in sign, leave 2^-12 of either


def steps(T):
    """Roundings of 32 bits that a term meets: its power, its scales, its split and its products (12 together), and in each chunk
    of at least 32 tokens a decay of the state that is rounded, its product and a sum."""
    return 12 + 3 * (T // 32 + 1)


def allowed(dtype, want, size, T, more=0):
    """A result's own rounding, and a half step of 32 bits of its terms for each rounding; `more`: of the sums of many terms."""
    half = ref.HALF[dtype]
    return half * want.abs() + (steps(T) + more) * 2.0 ** -24 * size * (1 + half) + 1e-37


def inputs(seed, T, H, dk, dv, dtype):
    gen = torch.Generator().manual_seed(seed)
    q, k = (torch.randn((1, T, H, dk), generator=gen) for _ in range(2))
    v, d_o = (torch.randn((1, T, H, dv), generator=gen) for _ in range(2))
    return [t.to(dtype) for t in (q, k, v, d_o)] + [torch.full((H,), G)]


def one_channel(t, c):
    """t with its channel c alone."""
    out = torch.zeros_like(t)
    out[..., c] = t[..., c]
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [20, 60, 130])
def test_two_keys(T, dk, dv, dtype):
    """Two keys alone, with opposite values: o and dq are what their decay leaves of them, within a chunk and through the state."""
    q, k, v, d_o, g = inputs(T, T, 6, dk, dv, TYPES[dtype])
    q, d_o = one_channel(q, 17), one_channel(d_o, 33)
    keys = torch.zeros_like(k)
    keys[:, 3:5, :, 17] = k[:, 3:4, :, 17]
    v[:, 4] = -v[:, 3]
    Q, K, V, D, A = gpu(q, keys, v, d_o, g)
    o, s = kda.linattn_fwd(Q, K, V, A, scale=0.3)
    want, end = ref.attend(q, keys, v, g, None, None, 0.3)
    size, end_size = ref.magnitude(ref.attend, q, keys, v, g, scale=0.3)
    near(o, want, allowed(q.dtype, want, size, T), "o")
    near(s, end, steps(T) * 2.0 ** -24 * end_size + 1e-37, "s_final")
    dq = kda.linattn_bwd(Q, K, V, A, D, scale=0.3)[0]
    want = ref.attend_grads(q, keys, v, g, d_o, scale=0.3)[0]
    size = ref.magnitude(ref.attend_grads, q, keys, v, g, d_o=d_o, scale=0.3)[0]
    near(dq, want, allowed(q.dtype, want, size, T), "dq")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [20, 60, 130])
def test_two_queries(T, dk, dv, dtype):
    """Two queries alone, with opposite gradients: dk, dv and ds0 are what their decay leaves of them."""
    q, k, v, d_o, g = inputs(T + 1, T, 6, dk, dv, TYPES[dtype])
    k, v = one_channel(k, 17), one_channel(v, 33)
    queries = torch.zeros_like(q)
    queries[:, T - 5:T - 3, :, 17] = q[:, T - 5:T - 4, :, 17]
    d_o[:, T - 4] = -d_o[:, T - 5]
    got = kda.linattn_bwd(*gpu(queries, k, v, g, d_o), scale=0.3)
    want = ref.attend_grads(queries, k, v, g, d_o, scale=0.3)
    size = ref.magnitude(ref.attend_grads, queries, k, v, g, d_o=d_o, scale=0.3)
    for i, name in ((1, "dk"), (2, "dv")):
        near(got[i], want[i], allowed(q.dtype, want[i], size[i], T), name)
    near(got[3], want[3], steps(T) * 2.0 ** -24 * size[3] + 1e-37, "ds0")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_state_before(dk, dv, dtype):
    """Two rows of the state before the sequence, nearly opposite; and behind it, of its gradient."""
    T = 100
    q, k, v, d_o, g = inputs(5, T, 6, dk, dv, TYPES[dtype])
    gen = torch.Generator().manual_seed(6)
    s0, d_sf = torch.zeros((1, 6, dk, dv)), torch.zeros((1, 6, dk, dv))
    row, col = torch.randn((1, 6, dv), generator=gen), torch.randn((1, 6, dk), generator=gen)
    s0[:, :, 9], s0[:, :, 10] = row, -row * (1 - 2.0 ** -12)
    d_sf[..., 9], d_sf[..., 10] = col, -col * (1 - 2.0 ** -12)
    q[..., 10] = q[..., 9]
    pair = torch.zeros_like(q)
    pair[..., 9:11] = q[..., 9:11]
    o, _ = kda.linattn_fwd(*gpu(pair, torch.zeros_like(k), v, g, s0), scale=0.3)
    want, _ = ref.attend(pair, torch.zeros_like(k), v, g, s0, None, 0.3)
    size, _ = ref.magnitude(ref.attend, pair, torch.zeros_like(k), v, g, s0=s0, scale=0.3)
    near(o, want, allowed(q.dtype, want, size, T), "o")
    v[..., 10] = v[..., 9]
    values = torch.zeros_like(v)
    values[..., 9:11] = v[..., 9:11]
    args = (torch.zeros_like(q), k, values, g)
    dk_got = kda.linattn_bwd(*gpu(*args, d_o, None, d_sf), scale=0.3)[1]
    want = ref.attend_grads(*args, d_o, None, d_sf, None, 0.3)[1]
    size = ref.magnitude(ref.attend_grads, *args, d_o=d_o, d_sf=d_sf, scale=0.3)[1]
    near(dk_got, want, allowed(q.dtype, want, size, T), "dk")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_every_segment_alike(dtype):
    """A row is as exact in the middle of a sequence of several segments as at its end: each head has two keys alone at a place of its
    own, and the 60 rows behind them read."""
    T, H = 700, 40
    q, k, v, d_o, g = inputs(8, T, H, 64, 64, TYPES[dtype])
    keys, queries = torch.zeros_like(k), torch.zeros_like(q)
    for h in range(H):
        p = 1 + 16 * h
        keys[:, p:p + 2, h, 17] = k[:, p:p + 1, h, 17]
        v[:, p + 1, h] = -v[:, p, h]
        queries[:, p:p + 60, h, 17] = q[:, p:p + 60, h, 17]
    want, _ = ref.attend(queries, keys, v, g, None, None, 0.3)
    size, _ = ref.magnitude(ref.attend, queries, keys, v, g, scale=0.3)
    o, _ = kda.linattn_fwd(*gpu(queries, keys, v, g), scale=0.3)
    near(o, want, allowed(q.dtype, want, size, 128), "o")  # four chunks at most, with a segment's state handed on between
