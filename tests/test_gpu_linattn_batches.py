"""Linear attention of more sequence-heads than the chip has places, where a batch and packed sequences are cut differently: every value
of either against the 64-bit recurrence."""
import pytest
import torch

import gated_delta_rule_65_amd as kda
from tests import linattn_ref as ref
from tests.test_gpu_linattn import TYPES, gpu, near
from tests.test_gpu_linattn_precision import allowed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,T,H", [(70, 129, 9), (33, 100, 16), (130, 65, 4)])
def test_every_value_of_many_sequences(B, T, H, dtype):
    """No row, head or state of any sequence is another's, in a batch, packed and packed with a tail; a sequence alone gives the same
    within the same bounds."""
    D, scale = 64, 0.25
    q, k, v, d_o, g, s0, d_sf = ref.inputs(B + T, (B, T), H, D, D, TYPES[dtype], B)
    want, end = ref.attend(q, k, v, g, s0, None, scale)
    size, end_size = ref.magnitude(ref.attend, q, k, v, g, s0=s0, scale=scale)
    grads = ref.attend_grads(q, k, v, g, d_o, s0, d_sf, None, scale)
    sizes = ref.magnitude(ref.attend_grads, q, k, v, g, d_o=d_o, s0=s0, d_sf=d_sf, scale=scale)
    steps = T + 2 * D  # additions that a term meets at most, on top of the roundings that `allowed` counts

    def check(got, at=slice(None)):
        o, s, dq, dk, dv, ds0 = (t.view(w[at].shape) for t, w in zip(got, (want, end, *grads)))
        near(o, want[at], allowed(q.dtype, want, size, T, steps)[at], "o")
        near(s, end[at], ((T + 64) * 2.0 ** -24 * end_size + 1e-37)[at], "s_final")
        for name, x, w, m in zip(("dq", "dk", "dv"), (dq, dk, dv), grads, sizes):
            near(x, w[at], allowed(q.dtype, w, m, T, steps)[at], name)
        near(ds0, grads[3][at], ((T + 64) * 2.0 ** -24 * sizes[3] + 1e-37)[at], "ds0")

    Q, K, V, DO, G, S0, DS = gpu(q, k, v, d_o, g, s0, d_sf)
    check((*kda.linattn_fwd(Q, K, V, G, S0, scale=scale), *kda.linattn_bwd(Q, K, V, G, DO, S0, DS, scale=scale)))
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    for tail in (0, 70):
        rows = [torch.cat([t.flatten(0, 1), t.new_full((tail, H, D), float("nan"))]) for t in (Q, K, V, DO)]
        o, s = kda.linattn_varlen_fwd(*rows[:3], G, cu, S0, scale=scale)
        dq, dk, dv, ds0 = kda.linattn_varlen_bwd(*rows[:3], G, cu, rows[3], S0, DS, scale=scale)
        check((o[:B * T], s, dq[:B * T], dk[:B * T], dv[:B * T], ds0))
    for n in (0, B // 2, B - 1):
        one = [t[n:n + 1].contiguous() for t in (Q, K, V)]
        states = [t[n:n + 1].contiguous() for t in (S0, DS)]
        check((*kda.linattn_fwd(*one, G, states[0], scale=scale),
               *kda.linattn_bwd(*one, G, DO[n:n + 1].contiguous(), *states, scale=scale)), slice(n, n + 1))
