"""The 64-bit references of the operators around the recurrence: their gradients against differences, and the 8-bit
format against hand-worked values."""
import numpy as np
import pytest

from tests import layer_ref as ref


def differences(f, x, step=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        out[i] = (up - f()) / (2 * step)
        x[i] = keep
    return out


@pytest.mark.parametrize("logit", [False, True])
@pytest.mark.parametrize("mix", [False, True])
def test_scan_gradients_are_the_differences(logit, mix):
    rng = np.random.default_rng(3)
    where = ref.spans([3, 0, 1, 4])
    x, dy = rng.normal(size=(8, 3)), rng.normal(size=(8, 3))
    g = rng.normal(size=(8, 3)) if logit else -rng.uniform(0.01, 4.9, size=(8, 3))
    g[1, 0], g[5, 1] = (6.0, 7.0) if logit else (-5.5, 0.3)  # beyond the clamp: no gradient
    h0, dh = rng.normal(size=(4, 3)), rng.normal(size=(4, 3))

    def loss():
        (y, _), (h, _), _ = ref.scan(x, g, h0, where, logit, mix)
        return (y * dy).sum() + (h * dh).sum()

    (dx, _), (dg, _), (dh0, _) = ref.scan_grad(x, g, h0, dy, dh, where, logit, mix)
    for got, at in ((dx, x), (dg, g), (dh0, h0)):
        # central differences of step 1e-6: truncation ~1e-12, cancellation ~1e-16 * |loss| / 1e-6
        np.testing.assert_allclose(got, differences(loss, at), rtol=1e-6, atol=1e-7)
    assert dg[1, 0] == 0 and dg[5, 1] == 0


@pytest.mark.parametrize("rms,interleaved,rot", [(False, False, 4), (True, True, 8), (True, False, 0)])
def test_head_norm_gradients_are_the_differences(rms, interleaved, rot):
    rng = np.random.default_rng(4)
    x, dy, w = rng.normal(size=(2, 2, 8)), rng.normal(size=(2, 2, 8)), rng.normal(size=8)
    angle = rng.normal(size=(2, rot // 2)) * 100

    def loss():
        return (ref.qk_norm(x, w, angle, rms, 1e-3, interleaved)[0] * dy).sum()

    _, (dx, _), (dw, _) = ref.qk_norm(x, w, angle, rms, 1e-3, interleaved, dy)
    np.testing.assert_allclose(dx, differences(loss, x), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(dw, differences(loss, w), rtol=1e-6, atol=1e-7)


def test_rotation_keeps_lengths_and_turns_back():
    rng = np.random.default_rng(5)
    z, angle = rng.normal(size=(3, 2, 8)), rng.normal(size=(3, 3)) * 1e6
    for interleaved in (False, True):
        t = ref.turned(z, angle, interleaved)
        np.testing.assert_allclose((t ** 2).sum(-1), (z ** 2).sum(-1), rtol=1e-12)
        np.testing.assert_allclose(ref.turned(t, angle, interleaved, -1.0), z, rtol=1e-9, atol=1e-9)
        assert (t[..., 6:] == z[..., 6:]).all()


def test_packed_values_by_hand():
    # amax 448: scale 1.  1.0625 lies between 1 and 1.125: the even code (1); 1.1875 rounds to 1.25, even too
    codes, scales, values = ref.pack8(np.array([[448.0, 1.0625, 1.1875, -1.0625, 2.0 ** -9, 2.0 ** -10, 0.0]]))
    assert scales[0, 0] == 127
    assert values[0].tolist() == [448.0, 1.0, 1.25, -1.0, 2.0 ** -9, 0.0, 0.0]
    assert codes[0].tolist() == [0x7e, 0x38, 0x3a, 0xb8, 0x01, 0x00, 0x00]
    # one step above 448 doubles the scale, half of it does not change it
    assert ref.pack8(np.array([[448.0001]]))[1][0, 0] == 128 and ref.pack8(np.array([[224.0001]]))[1][0, 0] == 127
    assert ref.pack8(np.array([[224.0]]))[1][0, 0] == 126
    # the smallest scale, and the top that does not unpack to infinity
    assert ref.pack8(np.array([[1e-44, 0.0]]))[1][0, 0] == 7
    _, scales, values = ref.pack8(np.array([[3.4e38]]))
    assert scales[0, 0] == 247 and values[0, 0] == 1.875 * 2.0 ** 127
    codes, scales, values = ref.pack8(np.random.default_rng(0).normal(size=(3, 70)))
    assert scales.shape == (3, 3) and (ref.unpack8(codes, scales) == values).all()
