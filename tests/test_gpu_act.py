"""GPU parity of convrot_act_checkpoint / convrot_act_backward against the
float64 oracle, and a training step that runs them with the quantized linear
and its adapters.

Codes and scales are the library's symmetric quantizer: bit for bit. y and dz
are float32 evaluations rounded once to bf16. Bound: half a step (2^-8 of the
value) plus 64 float32 roundings (2^-24 each) of the value and of the parts
that cancel in it (dy (1 + |z|) bounds those of a slope; for GELU_TANH the
exponent 2 t of the sigmoid carries |2 t| roundings into it)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import workloads as wl  # noqa: E402
from oracle import adapters as oa  # noqa: E402
from tests.gpu_helpers import DEV, bf16_dev, bf16_to_f32, dev, host, rel_l2, say  # noqa: E402

ACTS = ["gelu", "gelu_tanh", "swiglu"]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a8_rotated_quantized_amd as m
    assert m.device_check() == 0, "device is not gfx950"
    return m


def _act(cr, name):
    return {"gelu": cr.ACT.GELU, "gelu_tanh": cr.ACT.GELU_TANH, "swiglu": cr.ACT.SWIGLU}[name]


def _f32(t):
    return t.float().cpu().numpy().astype(np.float64)


def _value_bound(z, want, act):
    if act == "swiglu":
        g = z[:, :z.shape[1] // 2]
        soft = np.abs(want) * (1 + np.abs(g))
    elif act == "gelu_tanh":
        soft = np.abs(want) * (1 + np.abs(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    else:                                           # erfc of an argument that is off by a rounding: z^2 of them
        soft = np.abs(want) * (1 + z * z)
    return 2.0 ** -8 * np.abs(want) + 64 * U * soft + 2.0 ** -126


def _slope_bound(dy, z, want, act):
    if act == "swiglu":
        C = z.shape[1] // 2
        g, u = z[:, :C], z[:, C:]
        s = 1 / (1 + np.exp(-np.clip(g, -700, 700)))
        parts = np.concatenate([np.abs(dy * u) * s * (1 + np.abs(g)) ** 2, np.abs(dy * g) * s * (1 + np.abs(g))], 1)
    else:
        small = np.exp(-np.clip(z * z / 2, 0, 700)) if act == "gelu" else 1.0
        parts = np.abs(dy) * np.minimum(1.0, (1 + np.abs(z)) * small + (z > 0)) * (1 + np.minimum(z * z, 40.0))
    return 2.0 ** -8 * np.abs(want) + 64 * U * parts + 2.0 ** -126


SHAPES = [(1, 64), (3, 128), (7, 192), (22, 2560), (65, 1024), (257, 320), (130, 4160)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_checkpoint_and_backward(cr, act, shape):
    rows, C = shape
    say(f"act {act} {shape}")
    W = 2 * C if act == "swiglu" else C
    zb = wl.activation(71, rows + W, rows, W, n_outliers=max(1, W // 200), outlier_scale=6.0)
    z = bf16_to_f32(zb)
    if rows > 2:
        z[1, :64] = 0
        z[2, W - 64:] = np.float32(-0.0)
        zb = wl.bf16_bits_from_f32(z)
    y, codes, scales = cr.convrot_act_checkpoint(bf16_dev(zb), _act(cr, act))
    q_want, s_want = oa.checkpoint(z)
    assert np.array_equal(host(codes), q_want), "codes differ"
    assert np.array_equal(host(scales).view(np.uint32), s_want.view(np.uint32)), "scales differ"
    z64 = z.astype(np.float64)
    want = oa.act_value(z64, act)
    assert np.all(np.abs(_f32(y) - want) <= _value_bound(z64, want, act))
    dyb = wl.activation(72, rows + C, rows, C)
    dy = bf16_to_f32(dyb).astype(np.float64)
    dz = cr.convrot_act_backward(bf16_dev(dyb), codes, scales, _act(cr, act))
    kept = oa.restore_checkpoint(q_want, s_want)
    dz_want = oa.act_backward(dy, kept, act)
    assert dz.shape == (rows, W)
    assert np.all(np.abs(_f32(dz) - dz_want) <= _slope_bound(dy, kept, dz_want, act))


@pytest.mark.parametrize("act", ACTS)
def test_every_bf16_value(cr, act):
    """All finite bf16 values, each in a group of its own size class."""
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    v = bf16_to_f32(bits)
    # a 127 / A without a float32 value is the documented exception: tested below
    v = v[np.isfinite(v) & ((np.abs(v) > 3.9e-37) | (v == 0))]
    v = np.sort(v)
    v = np.concatenate([v, np.zeros(-len(v) % 256, np.float32)]).reshape(-1, 128)
    z = np.concatenate([v, np.ones_like(v)], 1) if act == "swiglu" else v
    y, codes, scales = cr.convrot_act_checkpoint(bf16_dev(wl.bf16_bits_from_f32(z)), _act(cr, act))
    q_want, s_want = oa.checkpoint(z)
    assert np.array_equal(host(codes), q_want) and np.array_equal(host(scales), s_want)
    z64 = z.astype(np.float64)
    with np.errstate(over="ignore"):
        want = oa.act_value(z64, act)
    got = _f32(y)
    # bounded tails: beyond |z| = 10 the value is z or within 2^-70 of 0
    mid = np.abs(v) <= 10
    assert np.all((np.abs(got - want) <= _value_bound(z64, want, act))[mid])
    assert np.all(got[v > 10] == v[v > 10]) and np.all(np.abs(got[v < -10]) <= 2e-3) and np.all(np.isfinite(got))
    dy = torch.ones(v.shape, dtype=torch.bfloat16, device=DEV)
    dz = _f32(cr.convrot_act_backward(dy, codes, scales, _act(cr, act)))
    kept = oa.restore_checkpoint(q_want, s_want)
    with np.errstate(over="ignore", invalid="ignore"):
        dz_want = oa.act_backward(np.ones(v.shape), np.clip(kept, -60, 60), act)
    one = dz[:, :v.shape[1]]
    k = kept[:, :v.shape[1]]
    mid = np.abs(k) <= 10
    assert np.all((np.abs(one - dz_want[:, :v.shape[1]]) <= _slope_bound(np.ones(v.shape), np.clip(kept, -60, 60),
                                                                         dz_want, act)[:, :v.shape[1]])[mid])
    assert np.all(np.abs(one[k > 10] - 1) <= 1e-2) and np.all(np.abs(one[k < -10]) <= 1e-2)
    assert np.all(np.isfinite(one))


def test_groups_without_a_float32_scale(cr):
    z = np.zeros((4, 128), np.float32)
    z[0, 3] = 1e-38
    z[1, 70] = np.inf
    z[2, 5] = np.nan
    z[3, :] = 2.0
    t = torch.from_numpy(z).to(torch.bfloat16).to(DEV)
    y, codes, scales = cr.convrot_act_checkpoint(t, cr.ACT.GELU)
    s, q = host(scales), host(codes)
    assert s[0, 0] == 0 and not q[0].any()
    assert np.isnan(s[1, 1]) and s[1, 0] == 0 and not q[1].any()
    assert np.isnan(s[2, 0]) and s[2, 1] == 0 and not q[2].any()
    dz = _f32(cr.convrot_act_backward(torch.ones((4, 128), dtype=torch.bfloat16, device=DEV), codes, scales, cr.ACT.GELU))
    assert np.isnan(dz[1, 64:]).all() and np.isnan(dz[2, :64]).all() and np.isfinite(dz[[0, 3]]).all()
    assert (dz[0] == 0.5).all() and np.isfinite(dz[1, :64]).all()
    for name in ("gelu_tanh", "swiglu"):
        _, c, sc = cr.convrot_act_checkpoint(t, _act(cr, name))
        d = _f32(cr.convrot_act_backward(torch.ones((4, 64 if name == "swiglu" else 128), dtype=torch.bfloat16, device=DEV),
                                         c, sc, _act(cr, name)))
        assert np.isnan(d[2, :64]).all() and np.isfinite(d[3]).all()


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(cr, act):
    """The slope that the backward applies, at the values the codes stand for,
    against central differences of the oracle's forward in float64."""
    z = np.linspace(-5, 5, 256).astype(np.float32).reshape(2, 128)
    zb = wl.bf16_bits_from_f32(z)
    _, codes, scales = cr.convrot_act_checkpoint(bf16_dev(zb), _act(cr, act))
    C = 64 if act == "swiglu" else 128
    dz = _f32(cr.convrot_act_backward(torch.ones((2, C), dtype=torch.bfloat16, device=DEV), codes, scales, _act(cr, act)))
    kept = oa.restore_checkpoint(host(codes), host(scales))
    h = 1e-5
    diff = np.empty_like(kept)
    for half in range(2 if act == "swiglu" else 1):
        step = np.zeros_like(kept)
        step[:, half * C:(half + 1) * C] = h
        diff[:, half * C:(half + 1) * C] = (oa.act_value(kept + step, act) - oa.act_value(kept - step, act)) / (2 * h)
    # truncation and cancellation of the difference: below 1e-8 here
    assert np.all(np.abs(dz - diff) <= 2.0 ** -8 * np.abs(diff) + 1e-5)


def test_strided_rows_other_stream_and_replay(cr):
    rows, C = 50, 192
    for act in ACTS:
        W = 2 * C if act == "swiglu" else C
        zb = wl.activation(73, W, rows, W)
        dyb = wl.activation(74, C, rows, C)
        y, codes, scales = cr.convrot_act_checkpoint(bf16_dev(zb), _act(cr, act))
        dz = cr.convrot_act_backward(bf16_dev(dyb), codes, scales, _act(cr, act))
        zw = torch.zeros((rows, W + 40), dtype=torch.bfloat16, device=DEV)
        zw[:, :W] = bf16_dev(zb)
        yw = torch.full((rows + 1, C + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        dw = torch.full((rows + 1, W + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        y2, c2, s2 = cr.convrot_act_checkpoint(zw[:, :W], _act(cr, act), y=yw[:rows, :C], stream=s)
        d2 = cr.convrot_act_backward(bf16_dev(dyb), c2, s2, _act(cr, act), dz=dw[:rows, :W], stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y2, y) and torch.equal(c2, codes) and torch.equal(s2, scales) and torch.equal(d2, dz)
        assert (yw[rows:] == 7).all() and (yw[:, C:] == 7).all() and (dw[rows:] == 7).all() and (dw[:, W:] == 7).all()
        z_d, dy_d = bf16_dev(zb), bf16_dev(dyb)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = cr.convrot_act_checkpoint(z_d, _act(cr, act))
            back = cr.convrot_act_backward(dy_d, held[1], held[2], _act(cr, act))
        for _ in range(3):
            for v in (*held, back):
                v.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(held[0], y) and torch.equal(held[1], codes) and torch.equal(back, dz)


def test_refusals(cr):
    z = torch.zeros((4, 128), dtype=torch.bfloat16, device=DEV)
    y, codes, scales = cr.convrot_act_checkpoint(z, cr.ACT.GELU)
    for a in ((z.float(), 0), (z.cpu(), 0), (z, 3), (z, -1), (z[:, :96], 0), (z[:, :64], 2), (z[:0], 0), (z[:, 4:68], 0)):
        with pytest.raises((ValueError, cr.ConvRotError)):
            cr.convrot_act_checkpoint(*a)
    for a in ((z, codes[:, :64], scales, 0), (z, codes, scales[:, :1], 0), (z, codes.float(), scales, 0),
              (z, codes, scales, 2), (z.float(), codes, scales, 0), (z, codes.cpu(), scales, 0)):
        with pytest.raises((ValueError, cr.ConvRotError)):
            cr.convrot_act_backward(*a)


def test_training_step_of_a_gated_mlp(cr):
    """The operators as they run together: two quantized projections with two
    adapters each around a gated activation; the inputs are kept as the INT8
    codes the projections read, the activation's input as 8-bit codes. Every
    stage is compared with the oracle fed with the stage's own inputs, and the
    adapters' gradients with those of a float64 step without checkpoints."""
    M, H, F, R, A = 150, 512, 512, 16, 2
    g = np.random.default_rng(81)
    off_h, ids_h = np.array([0, 70, 140]), np.array([1, 0])      # ten padded rows
    off, ids = dev(np.int32(off_h)), dev(np.int32(ids_h))

    def bf(a):
        b = wl.bf16_bits_from_f32(np.asarray(a, np.float32))
        return bf16_dev(b), bf16_to_f32(b).astype(np.float64)
    x_d, x = bf(g.standard_normal((M, H)))
    dy_d, dy = bf(g.standard_normal((M, H)) * 0.1)
    layers = []
    for N, K in ((2 * F, H), (H, F)):
        w_d, w = bf(g.standard_normal((N, K)) / math.sqrt(K))
        wc, ws, _, _ = cr.convrot_rotate_quantize(w_d, 256, cr.Q.SYM_INT8, cr.GRAN.TENSOR)
        back = cr.convrot_dequantize_weights(wc, ws, N, K, cr.Q.SYM_INT8, cr.GRAN.TENSOR, rot_group=256)
        layers.append((N, K, wc, ws, _f32(back), bf(g.standard_normal((A, R, K)) / math.sqrt(K)),
                       bf(g.standard_normal((A, N, R)) * 0.3)))

    def project(inp, layer):
        N, K, wc, ws, _, down, up = layer
        codes, s, _, _ = cr.convrot_rotate_quantize(inp, 256, cr.Q.SYM_INT8, cr.GRAN.TENSOR)
        base = cr.int8_tensorwise_gemm(codes, s, wc, ws, M, N, K)
        out, la = cr.convrot_lora_forward(inp, down[0], up[0], off, ids, base=base)
        return out, la, codes, s
    z, la1, c1, s1 = project(x_d, layers[0])
    h, zc, zs = cr.convrot_act_checkpoint(z, cr.ACT.SWIGLU)
    out, la2, c2, s2 = project(h, layers[1])

    def back(grad, la, codes, s, layer):
        N, K, _, _, w, down, up = layer
        base = (grad.float() @ torch.from_numpy(w).float().to(DEV)).to(torch.bfloat16)
        return cr.convrot_lora_backward(grad, la, codes, down[0], up[0], off, ids, x_scales=s, dx_base=base)
    dh, dd2, du2 = back(dy_d, la2, c2, s2, layers[1])
    dz = cr.convrot_act_backward(dh, zc, zs, cr.ACT.SWIGLU)
    dx, dd1, du1 = back(dz, la1, c1, s1, layers[0])

    # the same step in float64 from x and dy alone, nothing quantized but the weights
    (N1, K1, _, _, w1, (_, a1), (_, b1)), (N2, K2, _, _, w2, (_, a2), (_, b2)) = layers
    z_r, l1 = oa.lora_forward(x, a1, b1, off_h, ids_h, None, x @ w1.T)
    h_r = oa.act_value(z_r, "swiglu")
    out_r, l2 = oa.lora_forward(h_r, a2, b2, off_h, ids_h, None, h_r @ w2.T)
    dh_r, dd2_r, du2_r, _ = oa.lora_backward(dy, l2, h_r, a2, b2, off_h, ids_h, None, dy @ w2)
    dz_r = oa.act_backward(dh_r, z_r, "swiglu")
    dx_r, dd1_r, du1_r, _ = oa.lora_backward(dz_r, l1, x, a1, b1, off_h, ids_h, None, dz_r @ w1)
    # 8-bit codes with one scale for a near-normal tensor of 4 to 5 sigma: a step is A / 127, the error
    # step / sqrt 12, about 1.1 % of sigma; each quantity passes at most four such roundings (input codes
    # twice, z codes, weights are shared) and a handful of bf16 ones (0.2 %): below 5 %
    for got, want, name in ((out, out_r, "out"), (dx, dx_r, "dx"), (dd1, dd1_r, "d_down1"), (du1, du1_r, "d_up1"),
                            (dd2, dd2_r, "d_down2"), (du2, du2_r, "d_up2")):
        e = rel_l2(_f32(got), want)
        say(f"{name}: rel-L2 {e:.2e}")
        assert e <= 0.05, name
    # the gradients of this step's own checkpoints, to float32
    xh = oa.restore_input(host(c2), np.broadcast_to(host(s2), (M,)), 256)
    _, dd_w, du_w, _ = oa.lora_backward(dy, _f32(la2), xh, a2, b2, off_h, ids_h)
    assert rel_l2(_f32(dd2), dd_w) <= 1e-5 and rel_l2(_f32(du2), du_w) <= 1e-5
