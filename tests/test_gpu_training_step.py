"""One training step of adapters over a frozen 4-bit base, by the entry points
alone and as they would be used together: modulated layer norm, rotation and
quantization, the 4-bit product, the adapters beside it, the loss's gradient
back through adapters, base and norm, and the optimizer's step on the adapters.
Each stage is held to the oracle on what the stage before it gave, so the bounds are
those of the single operators; the whole step runs on a side stream, twice
with the same result, and once more from a captured graph."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import workloads as wl  # noqa: E402
from oracle import mx, training as tr  # noqa: E402
from tests.gpu_helpers import DEV, bf16_dev, dev, say  # noqa: E402

M, K, N, R, ROT = 203, 512, 768, 16, 256
OFF = [0, 60, 60, 190, 203]


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a8_rotated_quantized_amd as m
    assert m.device_check() == 0, "device is not gfx950"
    return m


def _f64(t):
    return t.double().cpu().numpy()


def _setup(cr):
    g = np.random.default_rng(31)
    S = len(OFF) - 1
    s = {"x": bf16_dev(wl.activation(95, 0, M, K, n_outliers=3, outlier_scale=15.0)),
         "shift": dev((g.standard_normal((S, K)) * 0.3).astype(np.float32)), "scale": dev((g.standard_normal((S, K)) * 0.3).astype(np.float32)),
         "off": torch.tensor(OFF, dtype=torch.int32, device=DEV), "bias": bf16_dev(wl.activation(95, 1, 1, N)[0]),
         "target": dev(g.standard_normal((M, N)).astype(np.float32)),
         "seg": torch.tensor([0, M], dtype=torch.int32, device=DEV), "ids": torch.zeros(1, dtype=torch.int32, device=DEV)}
    w = wl.weight(95, 2, N, K)
    s["w"] = cr.mxfp4_quantize(bf16_dev(w), ROT)
    # the gradient's side: W in the layer's own basis, quantized along N
    s["wt"] = cr.mxfp4_quantize(bf16_dev(np.ascontiguousarray(w.reshape(N, K).T)), ROT)
    s["down"] = dev((g.standard_normal((1, R, K)) / math.sqrt(K)).astype(np.float32))
    s["up"] = dev((g.standard_normal((1, N, R)) * 0.02).astype(np.float32))
    for k in ("down", "up"):
        s[k + "_bf"] = s[k].to(torch.bfloat16)
        n = s[k].numel()
        s[k + "_m"], s[k + "_v"] = torch.zeros(n, dtype=torch.int8, device=DEV), torch.zeros(n, dtype=torch.uint8, device=DEV)
        s[k + "_ms"], s[k + "_vs"] = torch.zeros(-(-n // 256), device=DEV), torch.zeros(-(-n // 256), device=DEV)
    return s


def _step(cr, s, step, seed, stream=None):
    on = {"stream": stream}
    o = {}
    o["h"], o["mean"], o["rstd"] = cr.convrot_layer_norm_forward(s["x"], s["scale"], s["shift"], seg_offsets=s["off"], one_plus=True, **on)
    o["codes"], o["scales"] = cr.mxfp4_quantize(o["h"], ROT, **on)
    o["base"] = cr.mxfp4_gemm(o["codes"], o["scales"], *s["w"], bias=s["bias"], out_type=cr.OUT.F32, **on)
    o["y"], o["la"] = cr.convrot_lora_forward(o["h"], s["down_bf"], s["up_bf"], s["seg"], s["ids"], base=o["base"], out_type=cr.OUT.F32,
                                              **on)
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        o["dy"] = ((o["y"] - s["target"]) * (2 / N)).to(torch.bfloat16)
    dyq = cr.mxfp4_quantize(o["dy"], ROT, **on)
    o["dyq"] = dyq
    o["dh_base"] = cr.mxfp4_gemm(*dyq, *s["wt"], out_type=cr.OUT.F32, **on)
    o["dh"], d_down, d_up = cr.convrot_lora_backward(o["dy"], o["la"], o["h"], s["down_bf"], s["up_bf"], s["seg"], s["ids"],
                                                     dx_base=o["dh_base"], dx_type=cr.OUT.F32, **on)
    o["dx"], o["dscale"], o["dshift"] = cr.convrot_layer_norm_backward(o["dh"], s["x"], o["mean"], o["rstd"], s["scale"],
                                                                       seg_offsets=s["off"], one_plus=True, **on)
    o["d_down"], o["d_up"] = d_down, d_up
    cr.convrot_adamw_step([s["down"], s["up"]], [d_down, d_up], [s["down_m"], s["up_m"]], [s["down_v"], s["up_v"]], step=step, lr=1e-3,
                          copies=[s["down_bf"], s["up_bf"]], exp_avg_scales=[s["down_ms"], s["up_ms"]],
                          exp_avg_sq_scales=[s["down_vs"], s["up_vs"]], seed=seed, **on)
    return o


def _bf16_values(t):
    return t.float().cpu().numpy()


def test_stages_against_the_oracle(cr):
    s = _setup(cr)
    before = {k: v.clone() for k, v in s.items() if isinstance(v, torch.Tensor)}
    o = _step(cr, s, 1, 9)
    rows = tr.sequences(OFF, M)
    scale, shift, x = _f64(s["scale"]), _f64(s["shift"]), _f64(s["x"])
    # float32 evaluations rounded to bf16: half a step, and 2^-15 of the terms that meet in a sum for 200 float32 roundings
    h, mean, rstd = tr.norm_forward(x, scale, shift, rows, 1.0)
    terms = np.abs((x - mean[:, None]) * rstd[:, None] * (1 + scale[rows])) + np.abs(shift[rows])
    assert np.all(np.abs(_f64(o["h"]) - h) <= 2.0 ** -8 * np.abs(h) + 2.0 ** -15 * terms)
    # codes of the bf16 rows the norm gave, bit for bit; the product of what they stand for
    hv = _bf16_values(o["h"])
    c, b = mx.quantize(hv, ROT)
    packed = mx.pack(c, b)
    assert np.array_equal(o["scales"].cpu().numpy(), packed[1])
    av, wv = mx.values(c, b), mx.values(*mx.unpack(*(t.cpu().numpy() for t in s["w"]), K))
    want, mag = mx.gemm(av, wv, _f64(s["bias"]))
    assert np.all(np.abs(_f64(o["base"]) - want) <= 2.0 ** -23 * (K + 2) * mag)
    # y: the base and the adapters' product, K and R sums of exact products
    down, up = _f64(before["down_bf"])[0], _f64(before["up_bf"])[0]
    la = hv.astype(np.float64) @ down.T
    y = _f64(o["base"]) + la @ up.T
    near = np.abs(hv) @ np.abs(down).T @ np.abs(up).T
    assert np.all(np.abs(_f64(o["y"]) - y) <= 2.0 ** -23 * (K + R + 4) * (near + np.abs(y)))
    # the gradient through the base: dy and W^T quantized along N
    dyv = _bf16_values(o["dy"])
    dc, db = mx.quantize(dyv, ROT)
    want, mag = mx.gemm(mx.values(dc, db), mx.values(*mx.unpack(*(t.cpu().numpy() for t in s["wt"]), N)))
    assert np.all(np.abs(_f64(o["dh_base"]) - want) <= 2.0 ** -23 * (N + 2) * mag)
    exact = dyv.astype(np.float64) @ wl.f32_from_bf16_bits(wl.weight(95, 2, N, K)).reshape(N, K).astype(np.float64)
    assert np.linalg.norm(_f64(o["dh_base"]) - exact) < 0.25 * np.linalg.norm(exact)
    # adapters' gradients, norm's gradients
    dla = dyv.astype(np.float64) @ up
    assert np.allclose(_f64(o["d_up"])[0], dyv.astype(np.float64).T @ la, rtol=1e-4, atol=1e-4 * np.abs(dyv).max() * np.abs(la).max())
    assert np.allclose(_f64(o["d_down"])[0], dla.T @ hv, rtol=1e-4, atol=1e-4 * np.abs(dla).max() * np.abs(hv).max())
    dx, dw, dbias = tr.norm_backward(_f64(o["dh"]), x, _f64(o["mean"]), _f64(o["rstd"]), scale, rows, 1.0, len(OFF) - 1)
    size = rstd[:, None] * (np.abs(_f64(o["dh"])).max(1, keepdims=True) * 4 * (1 + np.abs(x - mean[:, None]) * rstd[:, None]))
    assert np.all(np.abs(_f64(o["dx"]) - dx) <= 2.0 ** -8 * np.abs(dx) + 2.0 ** -15 * size)
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    for q in range(len(OFF) - 1):
        at = rows == q
        assert np.all(np.abs(_f64(o["dscale"])[q] - dw[q]) <= 2.0 ** -15 * (np.abs(_f64(o["dh"])) * xh)[at].sum(0))
        assert np.all(np.abs(_f64(o["dshift"])[q] - dbias[q]) <= 2.0 ** -15 * np.abs(_f64(o["dh"]))[at].sum(0))
    # the step itself: codes bit for bit from the gradients that came
    for i, k in enumerate(("down", "up")):
        grad = o["d_" + k].reshape(-1).cpu().numpy()
        w = tr.adamw8(before[k].reshape(-1).cpu().numpy(), grad, before[k + "_m"].cpu().numpy(), before[k + "_ms"].cpu().numpy(),
                      before[k + "_v"].cpu().numpy(), before[k + "_vs"].cpu().numpy(), 1, 1e-3, 0.9, 0.999, 1e-8, 0.01, 9, i)
        assert np.array_equal(s[k + "_m"].cpu().numpy(), w[1]) and np.array_equal(s[k + "_v"].cpu().numpy(), w[3])
        assert np.abs(_f64(s[k]).reshape(-1) - w[0]).max() <= 2.0 ** -22 * max(1e-3, np.abs(w[0]).max())
        assert torch.equal(s[k + "_bf"], s[k].to(torch.bfloat16))


def _state(s):
    return {k: v.clone() for k, v in s.items() if isinstance(v, torch.Tensor)}


def test_side_stream_and_graph_give_the_same_steps(cr):
    """Three steps eagerly, three on a side stream with other work beside them, three replays of a captured step."""
    say("training step on a side stream and from a graph")
    s = _setup(cr)
    start = _state(s)
    eager = []
    for _ in range(3):
        o = _step(cr, s, 5, 3)
        eager.append((o["dx"].clone(), _state(s)))
    for k, v in start.items():
        s[k].copy_(v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for dx, state in eager:
        noise = torch.randn(512, 512, device=DEV)
        o = _step(cr, s, 5, 3, stream=side)
        noise = noise @ noise
        side.synchronize()
        assert torch.equal(o["dx"], dx)
        assert all(torch.equal(s[k], v) for k, v in state.items())
    for k, v in start.items():
        s[k].copy_(v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = _step(cr, s, 5, 3)
    for dx, state in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o["dx"], dx)
        assert all(torch.equal(s[k], v) for k, v in state.items())
        torch.randn(300, 300, device=DEV).sum().item()
