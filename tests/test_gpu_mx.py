"""GPU parity of the microscaled 4-bit linear against the float64 oracle.

Codes and scale bytes: bit for bit. Values read back without rotation are
exact in float32 (a bf16 value is one of them rounded: exact too, 3 bits).
With a rotation, log2(n) float32 sums of magnitudes up to sum |v| over the
group: log2(n) + 1 roundings of 2^-24 times that sum / sqrt(n), and half a step
of the output type. Products: exact terms, K sums, each off by at most 2^-23
of what it has summed (matrix cores may cut instead of rounding): 2^-23 (K + 2)
sum |a w|, and half a step."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import workloads as wl  # noqa: E402
from oracle import mx  # noqa: E402
from tests.gpu_helpers import DEV, bf16_dev, bf16_to_f32, dev, host, say  # noqa: E402

HALF = {"bf16": 2.0 ** -9, "f32": 2.0 ** -25}     # of a value's power of two, that is at most 2^-8 / 2 of the value


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a8_rotated_quantized_amd as m
    assert m.device_check() == 0, "device is not gfx950"
    return m


def _out(cr, name):
    return cr.OUT.BF16 if name == "bf16" else cr.OUT.F32


def _f64(t):
    return t.double().cpu().numpy()


def _step(want, out):
    return 2 * HALF[out] * np.abs(want) * (1 + 2.0 ** -8)


def _check_codes(codes, scales, x, rot):
    want = mx.pack(*mx.quantize(x, rot))
    got_c, got_s = host(codes), host(scales)
    assert np.array_equal(got_s, want[1]), "scale bytes differ"
    # a zero's sign stands for nothing
    def plain(c):
        lo, hi = c & 15, c >> 4
        return np.where(lo == 8, 0, lo), np.where(hi == 8, 0, hi)
    for a, b in zip(plain(got_c), plain(want[0])):
        assert np.array_equal(a, b), "codes differ"


SHAPES = [(1, 32), (1, 1024), (2, 96), (3, 160), (5, 1024), (15, 2080), (16, 256), (17, 4096), (33, 1056), (70, 3072),
          (257, 2048)]


@pytest.mark.parametrize("rot", [0, 16, 64, 256, 1024])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_and_back(cr, shape, rot):
    rows, K = shape
    if rot and K % max(rot, 32):
        pytest.skip("columns are no multiple of the rotation")
    say(f"mx quantize {shape} rot {rot}")
    xb = wl.activation(91, rows + K + rot, rows, K, n_outliers=K // 100, outlier_scale=25.0)
    x = bf16_to_f32(xb).copy()
    if K >= 64:
        x[0, :32] = 0
    xb = wl.bf16_bits_from_f32(x)
    # rows further apart than they are long, on both ends
    wide = torch.full((rows, K + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    wide[:, :K] = bf16_dev(xb)
    codes, scales = cr.mxfp4_quantize(wide[:, :K], rot)
    _check_codes(codes, scales, x, rot)
    c, b = mx.quantize(x, rot)
    for out in ("bf16", "f32"):
        v = mx.values(c, b)
        plain = cr.mxfp4_dequantize(codes, scales, K, 0, out_type=_out(cr, out))
        assert np.array_equal(_f64(plain), v)
        if rot:
            hold = torch.full((rows, K + 8), -3.0, dtype=plain.dtype, device=DEV)
            cr.mxfp4_dequantize(codes, scales, K, rot, out_type=_out(cr, out), out=hold[:, :K])
            assert bool((hold[:, K:] == -3).all())
            want = mx.dequantize(c, b, rot)
            mag = np.repeat(np.abs(v).reshape(rows, K // rot, rot).sum(-1), rot, axis=1) / math.sqrt(rot)
            assert np.all(np.abs(_f64(hold[:, :K]) - want) <= (math.log2(rot) + 1) * 2.0 ** -24 * mag + _step(want, out))


def test_every_bf16_value_at_every_power(cr):
    """Each finite bf16 value as a block of its own size class, and as the small one of larger blocks."""
    bits = np.arange(1 << 15, dtype=np.uint32).astype(np.uint16)
    v = bf16_to_f32(bits)
    v = v[np.isfinite(v)]
    x = np.zeros((len(v), 32), np.float32)
    x[:, 0], x[:, 1] = v, -v
    with np.errstate(over="ignore"):
        for i, f in enumerate((1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 5, 7, 9, 17, 40)):
            w = np.minimum(v.astype(np.float64) / f, 3e38).astype(np.float32)
            x[:, 2 + i] = bf16_to_f32(wl.bf16_bits_from_f32(w))
    codes, scales = cr.mxfp4_quantize(bf16_dev(wl.bf16_bits_from_f32(x)), 0)
    _check_codes(codes, scales, x, 0)


@pytest.mark.parametrize("rot", [16, 64, 256, 1024])
def test_tiny_and_huge_rotated(cr, rot):
    g = np.random.default_rng(rot)
    x = g.standard_normal((40, 1024)).astype(np.float32) * np.exp2(np.linspace(-132, 116, 40))[:, None].astype(np.float32)
    x = bf16_to_f32(wl.bf16_bits_from_f32(x))
    codes, scales = cr.mxfp4_quantize(bf16_dev(wl.bf16_bits_from_f32(x)), rot)
    _check_codes(codes, scales, x, rot)


@pytest.mark.parametrize("rot", [0, 64, 256])
def test_not_finite_stays_in_its_block(cr, rot):
    x = bf16_to_f32(wl.activation(92, 0, 6, 768)).copy()
    clean = x.copy()
    x[1, 40], x[3, 700], x[4, 0] = np.inf, np.nan, -np.inf
    t = torch.from_numpy(x).to(DEV).to(torch.bfloat16)
    codes, scales = cr.mxfp4_quantize(t, rot)
    group = rot or 32
    back = _f64(cr.mxfp4_dequantize(codes, scales, 768, 0, out_type=cr.OUT.F32))
    c, b = mx.quantize(clean, rot)
    want = mx.values(c, b)
    for r, k in ((1, 40), (3, 700), (4, 0)):
        want[r, k // group * group:(k // group + 1) * group] = np.nan
    assert np.array_equal(back, want, equal_nan=True)
    # ... and in its row of a product
    w, ws = cr.mxfp4_quantize(bf16_dev(wl.weight(92, 1, 128, 768)), rot)
    for M in (6, 70):
        rep = torch.cat([t] * (-(-M // 6)))[:M].contiguous()
        y = _f64(cr.mxfp4_gemm(*cr.mxfp4_quantize(rep, rot), w, ws))
        bad = np.isin(np.arange(M) % 6, [1, 3, 4])
        assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()


def _operand(cr, cfg, rows, K, spread=True):
    """Random codes and scale bytes in the oracle's and the library's layout: all codes, wide powers."""
    g = np.random.default_rng([cfg, rows, K])
    codes = g.integers(0, 16, (rows, K)).astype(np.uint8)
    byte = (127 + g.integers(-6, 7, (rows, K // 32))).astype(np.uint8) if spread else np.full((rows, K // 32), 127, np.uint8)
    c, b = mx.pack(codes, byte)
    return mx.values(codes, byte), dev(c), dev(b)


GEMM = [(1, 8, 32), (1, 4096, 2560), (2, 24, 160), (7, 72, 4096), (16, 128, 128), (17, 2560, 1056), (33, 136, 2048), (49, 264, 384),
        (64, 1000, 2560), (65, 64, 128), (66, 200, 96), (100, 72, 12288), (128, 128, 2048), (300, 328, 1024), (513, 4096, 256),
        (1531, 2568, 608), (2049, 2056, 512)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("shape", GEMM)
def test_gemm(cr, shape, out):
    M, N, K = shape
    say(f"mx gemm {shape} {out}")
    a, ac, ab = _operand(cr, 1, M, K)
    w, wc, wb = _operand(cr, 2, N, K)
    biasb = wl.activation(93, N, 1, N)[0]
    bias = bf16_to_f32(biasb).astype(np.float64)
    for b in (None, bias):
        want, mag = mx.gemm(a, w, b)
        hold = torch.full((M, N + 16), -5.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device=DEV)
        y = cr.mxfp4_gemm(ac, ab, wc, wb, bias=None if b is None else bf16_dev(biasb), out_type=_out(cr, out), out=hold[:, :N])
        got = _f64(y)
        assert np.all(np.abs(got - want) <= 2.0 ** -23 * (K + 2) * mag + _step(want, out)), np.abs(got - want).max()
        assert bool((hold[:, N:] == -5).all())


@pytest.mark.parametrize("M", [1, 40, 65, 200, 4100])
def test_gemm_integers_exact(cr, M):
    """Unit powers: products are quarters, their float32 sums exact."""
    N, K = 2056 if M == 4100 else 520, 1536
    a, ac, ab = _operand(cr, 3, M, K, spread=False)
    w, wc, wb = _operand(cr, 4, N, K, spread=False)
    want, _ = mx.gemm(a, w)
    assert np.array_equal(_f64(cr.mxfp4_gemm(ac, ab, wc, wb, out_type=cr.OUT.F32)), want)


@pytest.mark.parametrize("M,N", [(3, 64), (130, 192)])
def test_every_byte_of_scale(cr, M, N):
    """Each power of two that the format has, against one that brings the product back to ordinary numbers."""
    K = 32 * 256
    codes_a, codes_w = np.full((M, K), 2, np.uint8), np.full((N, K), 4, np.uint8)      # 1 and 2
    byte_a = np.tile(np.arange(256, dtype=np.uint8), (M, 1))
    byte_a[:, 255] = 254
    byte_w = np.tile((254 - np.arange(256)).clip(0).astype(np.uint8), (N, 1))
    (ca, ba), (cw, bw) = mx.pack(codes_a, byte_a), mx.pack(codes_w, byte_w)
    want, mag = mx.gemm(mx.values(codes_a, byte_a), mx.values(codes_w, byte_w))
    got = _f64(cr.mxfp4_gemm(dev(ca), dev(ba), dev(cw), dev(bw), out_type=cr.OUT.F32))
    assert np.all(np.abs(got - want) <= 2.0 ** -23 * (K + 2) * mag)


@pytest.mark.parametrize("rot", [0, 256])
def test_linear_and_its_gradient(cr, rot):
    """Forward and dx = dy W of one linear by the entry points alone."""
    M, N, K = 77, 512, 1024
    x, w = wl.activation(94, 0, M, K, n_outliers=5, outlier_scale=20.0), wl.weight(94, 1, N, K)
    dy = wl.activation(94, 2, M, N)
    wt = np.ascontiguousarray(bf16_to_f32(w).T)
    y = _f64(cr.mxfp4_gemm(*cr.mxfp4_quantize(bf16_dev(x), rot), *cr.mxfp4_quantize(bf16_dev(w), rot), out_type=cr.OUT.F32))
    av, wv = (mx.values(*mx.quantize(bf16_to_f32(t), rot)) for t in (x, w))
    want, mag = mx.gemm(av, wv)
    assert np.all(np.abs(y - want) <= 2.0 ** -23 * (K + 2) * mag)
    dx = _f64(cr.mxfp4_gemm(*cr.mxfp4_quantize(bf16_dev(dy), rot), *cr.mxfp4_quantize(bf16_dev(wl.bf16_bits_from_f32(wt)), rot),
                            out_type=cr.OUT.F32))
    want, mag = mx.gemm(mx.values(*mx.quantize(bf16_to_f32(dy), rot)), mx.values(*mx.quantize(wt, rot)))
    assert np.all(np.abs(dx - want) <= 2.0 ** -23 * (N + 2) * mag)
    exact = bf16_to_f32(dy).astype(np.float64) @ bf16_to_f32(w).astype(np.float64)
    assert np.linalg.norm(dx - exact) < 0.25 * np.linalg.norm(exact)


@pytest.mark.parametrize("rot", [16, 64, 256, 1024])
def test_rotated_at_the_largest_values(cr, rot):
    """Finite values whose sums leave float32: the blocks in which that happens stand for NaN, others keep their codes."""
    g = np.random.default_rng(rot + 1)
    x = g.uniform(-1, 1, (24, 1024)).astype(np.float32) * np.exp2(np.linspace(118, 127.9, 24))[:, None].astype(np.float32)
    x[20:, 1::2] = 0
    x[22:, 5:] = 0                                       # few large ones: their sums stay finite
    x = bf16_to_f32(wl.bf16_bits_from_f32(x))
    assert np.isfinite(x).all()
    want = mx.quantize(x, rot)[1]
    assert (want == 255).any() and (want[:, :] != 255).any()
    codes, scales = cr.mxfp4_quantize(bf16_dev(wl.bf16_bits_from_f32(x)), rot)
    _check_codes(codes, scales, x, rot)
    small = np.abs(x).max(1) < 2.0 ** 128 / rot
    assert not (want[small] == 255).any()
