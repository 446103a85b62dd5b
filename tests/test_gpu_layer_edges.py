"""The operators around the recurrence at the edges of what their calls allow: buffers longer than their sequences, views at
any offset, 16-bit gates in training, positions and rows of any size."""
import numpy as np
import pytest
import torch

import gated_delta_rule_65_amd as kda
from tests import layer_ref as ref
from tests.test_gpu_layer import TYPES, dev, host, near, scan_data

pytestmark = pytest.mark.gpu


def dirty(*shapes):
    """Leaves NaN behind in the memory that buffers of these shapes and types get next."""
    held = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(4)]
    torch.cuda.synchronize()
    del held


# ----------------------------------------------------------------- rows behind the last sequence

@pytest.mark.parametrize("ckpt8", [False, True])
@pytest.mark.parametrize("xk,gk,D", [("bf16", "f32", 72), ("f32", "bf16", 37), ("bf16", "bf16", 1)])
@pytest.mark.parametrize("lengths,total", [([70, 0, 33], 200), ([5], 6), ([0, 0], 9), ([], 3), ([64], 64), ([130, 3], 133)])
def test_scan_autograd_gives_zeros_behind_the_last_sequence(lengths, total, xk, gk, D, ckpt8):
    where, N, used = ref.spans(lengths) if lengths else [], len(lengths), sum(lengths)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    d, h = scan_data(total, D, N, True, 3, xk, gk)
    x, g, h0 = (d[k].clone().requires_grad_() for k in ("x", "g", "h0"))
    with torch.no_grad():
        for t in (x, g):
            t[used:] = float("nan")
    dirty(((total, D), TYPES[xk]), ((total, D), TYPES[gk]), ((total, D), torch.float32))
    y, hf = kda.VarlenGatedScan.apply(x, g, cu, h0, True, True, ckpt8)
    assert (y[used:] == 0).all()
    dy = d["dy"].clone()
    dy[used:] = float("nan")
    dirty(((total, D), TYPES[xk]), ((total, D), TYPES[gk]), ((total, D), torch.float32))
    torch.autograd.backward((y, hf), (dy, d["dh"]))
    assert (x.grad[used:] == 0).all() and (g.grad[used:] == 0).all()
    (want, _), (dx, _) = ref.scan(h["x"], h["g"], h["h0"], where, True, True)[0], ref.scan_grad(
        h["x"], h["g"], h["h0"], h["dy"], h["dh"], where, True, True)[0]
    for got, full in ((y, want), (x.grad, dx)):
        torch.testing.assert_close(got[:used].double().cpu(), torch.from_numpy(full[:used]), rtol=2.0 ** -7, atol=1e-4)
    assert torch.isfinite(g.grad).all() and torch.isfinite(h0.grad).all() and torch.isfinite(hf).all()
