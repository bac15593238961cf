"""Pins of oracle/adapters.py: brute force over scalars, differences of the
forward for every gradient, closed forms of the activations."""
import math

import numpy as np
import pytest

from oracle import adapters as oa, hadamard as oh, linear as ol
import workloads as wl

OFF, IDS = [1, 4, 4, 6, 9], [1, 0, -1, 0]      # rows 0 and 9 outside, an empty segment, one without adapter


def _case(seed, M=10, N=5, K=7, R=3, A=2):
    g = np.random.default_rng(seed)
    return (g.standard_normal((M, K)), g.standard_normal((A, R, K)), g.standard_normal((A, N, R)),
            g.standard_normal(A), g.standard_normal((M, N)))


def test_row_adapters():
    assert oa.row_adapters(OFF, IDS, 10, 2).tolist() == [-1, 1, 1, 1, -1, -1, 0, 0, 0, -1]
    assert oa.row_adapters([0, 2], [2], 3, 2).tolist() == [-1, -1, -1]


def test_forward_brute_force():
    x, down, up, c, base = _case(1)
    out, la = oa.lora_forward(x, down, up, OFF, IDS, c, base)
    rows = [-1, 1, 1, 1, -1, -1, 0, 0, 0, -1]
    for m, a in enumerate(rows):
        for n in range(5):
            want = base[m, n]
            for r in range(3):
                l = sum(x[m, k] * down[a, r, k] for k in range(7)) if a >= 0 else 0.0
                assert la[m, r] == pytest.approx(l, abs=1e-12)
                want += c[a] * l * up[a, n, r] if a >= 0 else 0.0
            assert out[m, n] == pytest.approx(want, abs=1e-12)


def test_gradients_against_differences():
    x, down, up, c, _ = _case(2)
    dy = np.random.default_rng(3).standard_normal((10, 5))
    _, la = oa.lora_forward(x, down, up, OFF, IDS, c)
    dx, d_down, d_up, _ = oa.lora_backward(dy, la, x, down, up, OFF, IDS, c)

    def loss():
        return float((oa.lora_forward(x, down, up, OFF, IDS, c)[0] * dy).sum())
    for arr, grad in ((x, dx), (down, d_down), (up, d_up)):
        for at in np.ndindex(arr.shape):
            keep = arr[at]
            arr[at] = keep + 1e-6
            up_ = loss()
            arr[at] = keep - 1e-6
            dn = loss()
            arr[at] = keep
            assert grad[at] == pytest.approx((up_ - dn) / 2e-6, abs=2e-8 * 1e2)


@pytest.mark.parametrize("rot", [16, 64, 256, 1024])
def test_restore_input_inverts_the_quantizer(rot):
    xb = wl.activation(61, rot, 6, 1024)
    q = ol.rotate_quantize(xb, rot, "int8", "row", None)
    back = oa.restore_input(q["codes"].reshape(6, 1024).view(np.int8), q["scales"], rot)
    x = wl.f32_from_bf16_bits(xb).astype(np.float64)
    # the rotation keeps lengths: the error is that of the codes, at most half a step each
    step = np.asarray(q["scales"], np.float64)
    err = np.linalg.norm(back - x, axis=1)
    assert np.all(err <= 0.5 * step * math.sqrt(1024) * 1.001)
    H = oh.regular_hadamard(rot)
    one = np.zeros((1, 1024))
    one[0, 3] = 1.0
    assert np.allclose(oa.restore_input(one, [2.0], rot)[0, :rot], 2.0 * H[3] / math.sqrt(rot))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "swiglu"])
def test_activation_slopes_against_differences(act):
    z = np.random.default_rng(5).uniform(-6, 6, (4, 12))
    C = 6 if act == "swiglu" else 12
    dy = np.random.default_rng(6).standard_normal((4, C))
    dz = oa.act_backward(dy, z, act)
    for at in np.ndindex(z.shape):
        p, n = z.copy(), z.copy()
        p[at] += 1e-5
        n[at] -= 1e-5
        d = ((oa.act_value(p, act) - oa.act_value(n, act)) * dy).sum() / 2e-5
        assert dz[at] == pytest.approx(d, abs=1e-8)


def test_activation_values():
    z = np.array([[0.0, 1.0, -1.0, 30.0]])
    phi1 = 0.8413447460685429                    # Phi(1)
    assert np.allclose(oa.act_value(z, "gelu"), [[0.0, phi1, -(1 - phi1), 30.0]], atol=1e-15)
    t = math.tanh(math.sqrt(2 / math.pi) * 1.044715)
    assert np.allclose(oa.act_value(z, "gelu_tanh"), [[0.0, (1 + t) / 2, -(1 - t) / 2, 30.0]], atol=1e-15)
    s1 = 1 / (1 + math.exp(-1))
    assert np.allclose(oa.act_value(np.array([[1.0, -1.0, 2.0, 3.0]]), "swiglu"), [[2 * s1, -3 * (1 - s1)]])


def test_checkpoint_round_trip():
    z = wl.f32_from_bf16_bits(wl.activation(62, 1, 5, 192))
    z[2, 64:128] = 0
    codes, scales = oa.checkpoint(z)
    assert codes.dtype == np.int8 and scales.shape == (5, 3) and scales[2, 1] == 0
    back = oa.restore_checkpoint(codes, scales)
    assert np.all(np.abs(back - z) <= np.repeat(scales, 64, axis=1) * 0.5 * (1 + 1e-6))
