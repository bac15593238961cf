"""GPU parity of convrot_lora_forward and convrot_lora_backward against the
float64 oracle.

Bounds, derived before the first run (u = 2^-24, a float32 rounding; sums on
the matrix cores are allowed 2u per added term, whatever their order):
  lora_act   (K + 16) 2u sum|x down|
  out        |c| err(la) |up| + (3R + 4) 2u sum|c la up| + 2u (|base| + |delta|),
             for bf16 outputs plus half a step, 2^-8 of the value
  dx, d_up, d_down alike; d_down from codes has (2 log2 n) u more for the
  rotation of sums bounded by sum|dla s q| / sqrt(n) over each group.
Integer inputs whose sums stay below 2^24 must come out exactly.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import workloads as wl  # noqa: E402
from oracle import adapters as oa  # noqa: E402
from tests.gpu_helpers import DEV, bf16_dev, bf16_to_f32, dev, host, say  # noqa: E402

U2 = 2.0 ** -23


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a8_rotated_quantized_amd as m
    assert m.device_check() == 0, "device is not gfx950"
    return m


def _bf16(a):
    """(device bf16 tensor, its values in float64)"""
    bits = wl.bf16_bits_from_f32(np.asarray(a, np.float32))
    return bf16_dev(bits), bf16_to_f32(bits).astype(np.float64)


def _segments(mix, M, S, A, g, none=0.1):
    if mix == "tokens":
        off = np.arange(M + 1)
    elif mix == "prompt":
        off = np.concatenate([[0], np.arange(M - S + 1, M + 1)])
    elif mix == "gaps":        # rows before the first and behind the last segment
        lo, hi = M // 5, M - M // 7
        off = np.concatenate([[lo], np.sort(g.integers(lo, hi + 1, S - 1)), [hi]])
    else:
        off = np.concatenate([[0], np.sort(g.integers(0, M + 1, S - 1)), [M]])
    ids = g.integers(0, A, len(off) - 1)
    ids[g.random(ids.size) < none] = g.choice([-1, A, -2 ** 31, 2 ** 31 - 1])
    return off, ids


class Case:
    def __init__(self, M, N, K, R, A, S, mix="ragged", seed=0, scale=True):
        g = self.g = np.random.default_rng([M, N, K, R, A, S, seed])
        self.M, self.N, self.K, self.R, self.A = M, N, K, R, A
        self.off, self.ids = _segments(mix, M, S, A, g)
        self.off_d, self.ids_d = dev(self.off.astype(np.int32)), dev(self.ids.astype(np.int64).astype(np.int32))
        self.x_d, self.x = _bf16(g.standard_normal((M, K)))
        self.down_d, self.down = _bf16(g.standard_normal((A, R, K)) / math.sqrt(K))
        self.up_d, self.up = _bf16(g.standard_normal((A, N, R)))
        self.dy_d, self.dy = _bf16(g.standard_normal((M, N)))
        self.c = (g.random(A) + 0.5).astype(np.float32) if scale else None
        self.c_d = None if self.c is None else dev(self.c)
        self.c64 = np.ones(A) if self.c is None else self.c.astype(np.float64)
        self.rows = oa.row_adapters(self.off, self.ids, M, A)

    def base(self, cols, f32, seed=1):
        v = np.random.default_rng([seed, cols]).standard_normal((self.M, cols)).astype(np.float32)
        return (dev(v), v.astype(np.float64)) if f32 else _bf16(v)

    def fwd(self, cr, **k):
        return cr.convrot_lora_forward(self.x_d, self.down_d, self.up_d, self.off_d, self.ids_d, scale=self.c_d, **k)

    def bwd(self, cr, la_d, **k):
        return cr.convrot_lora_backward(self.dy_d, la_d, k.pop("x", self.x_d), self.down_d, self.up_d, self.off_d,
                                        self.ids_d, scale=self.c_d, **k)

    def two_products(self, a, first, second, base, exact, f32):
        """Bounds of (a first^T) and of base + c (a first^T) second^T, row by row:
        first [A, R, *], second [A, *, R]."""
        e1, e2 = np.zeros((self.M, self.R)), np.zeros(exact.shape)
        for i in range(self.A):
            at = self.rows == i
            mid = np.abs(a[at] @ first[i].T)
            e1[at] = (a.shape[1] + 16) * U2 * (np.abs(a[at]) @ np.abs(first[i]).T)
            c = abs(self.c64[i])
            d = c * (mid @ np.abs(second[i]).T)
            e2[at] = c * (e1[at] @ np.abs(second[i]).T) + (3 * self.R + 4) * U2 * d + U2 * d
        e2 += U2 * np.abs(base)
        e2 += 1e-37
        if not f32:
            e2 += 2.0 ** -8 * (np.abs(exact) + e2)
        return e1 + 1e-37, e2


def _near(got, want, tol, what):
    got = got.float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} for {want[bad][0]} (bound {np.broadcast_to(tol, got.shape)[bad][0]:.3g})"


# M, N, K, R, A, S, mix
SHAPES = [
    (1, 8, 8, 8, 1, 1, "ragged"), (1, 4096, 2560, 16, 8, 1, "tokens"), (2, 136, 72, 24, 3, 2, "tokens"),
    (16, 128, 64, 8, 2, 3, "ragged"), (17, 520, 200, 40, 2, 4, "ragged"), (64, 256, 512, 32, 9, 64, "tokens"),
    (63, 1000, 264, 64, 4, 5, "gaps"), (65, 264, 1000, 128, 2, 3, "ragged"), (256, 136, 136, 120, 3, 9, "gaps"),
    (257, 512, 256, 16, 5, 70, "ragged"), (300, 200, 520, 48, 4, 300, "tokens"), (519, 640, 384, 32, 6, 41, "prompt"),
    (700, 72, 2056, 72, 2, 130, "gaps"), (1033, 384, 640, 64, 3, 7, "ragged"),
    (64, 4104, 4096, 32, 4, 64, "tokens"), (33, 2056, 136, 24, 2, 3, "gaps"), (200, 2048, 72, 8, 3, 9, "gaps"),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(cr, shape, f32):
    say(f"lora forward {shape} f32={f32}")
    t = Case(*shape[:6], mix=shape[6])
    kind = cr.OUT.F32 if f32 else cr.OUT.BF16
    base_d, base = t.base(t.N, f32)
    want, la_want = oa.lora_forward(t.x, t.down, t.up, t.off, t.ids, t.c, base)
    out, la = t.fwd(cr, base=base_d, out_type=kind)
    e1, e2 = t.two_products(t.x, t.down, t.up, base, want, f32)
    _near(la, la_want, e1, "lora_act")
    _near(out, want, e2, "out")
    none = t.rows < 0
    assert torch.equal(out[dev(none)], base_d[dev(none)]) and not la[dev(none)].any()
    # in place: the same bits, rows without adapter not written
    own = base_d.clone()
    out2, la2 = t.fwd(cr, base=own, out=own, out_type=kind)
    assert out2 is own and torch.equal(own, out) and torch.equal(la2, la)
    # no base
    want0, _ = oa.lora_forward(t.x, t.down, t.up, t.off, t.ids, t.c)
    out0, _ = t.fwd(cr, out_type=kind)
    _near(out0, want0, t.two_products(t.x, t.down, t.up, np.zeros_like(want0), want0, f32)[1], "out without base")
    assert not out0[dev(none)].any()


# Enough rows for the tall tiles and the wide shrink blocks of each rank
TALL = [(8200, 8200, 72, 64, 2, 5, "ragged"), (8200, 2056, 200, 24, 2, 5, "gaps"), (8209, 2056, 136, 128, 3, 9, "ragged"),
        (8300, 520, 264, 16, 2, 70, "ragged")]


@pytest.mark.parametrize("shape", TALL)
def test_forward_many_rows(cr, shape):
    say(f"lora forward {shape}")
    t = Case(*shape[:6], mix=shape[6])
    base_d, base = t.base(t.N, False)
    want, la_want = oa.lora_forward(t.x, t.down, t.up, t.off, t.ids, t.c, base)
    out, la = t.fwd(cr, base=base_d)
    e1, e2 = t.two_products(t.x, t.down, t.up, base, want, False)
    _near(la, la_want, e1, "lora_act")
    _near(out, want, e2, "out")


# expand in tiles of 32, 32 and 64 rows
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("shape", [(1000, 4104, 72, 64, 3, 7, "ragged"), (700, 4104, 72, 128, 2, 3, "gaps"),
                                   (2000, 4104, 72, 40, 2, 90, "ragged")])
def test_forward_middle_tiles(cr, shape, f32):
    test_forward(cr, shape, f32)


def test_no_row_has_an_adapter(cr):
    t = Case(70, 136, 264, 16, 3, 4, seed=23)
    base_d, _ = t.base(t.N, False)
    la = dev(t.g.standard_normal((t.M, t.R)).astype(np.float32))
    for off, ids in (([0, 20, 20, 50, 70], [-1, 0, 3, -7]), ([0, 0, 0, 0, 0], [0, 1, 2, 0]), ([70, 70, 70, 70, 70], [0, 1, 2, 0])):
        t.off_d, t.ids_d = dev(np.int32(off)), dev(np.int32(ids))
        out, la1 = t.fwd(cr, base=base_d)
        assert torch.equal(out, base_d) and not la1.any()
        dx, dd, du = t.bwd(cr, la)
        assert not dx.any() and not dd.any() and not du.any()


def test_forward_without_scale_and_with_strided_rows(cr):
    t = Case(77, 264, 136, 24, 3, 6, seed=3, scale=False)
    want, la_want = oa.lora_forward(t.x, t.down, t.up, t.off, t.ids)
    wide = torch.full((t.M + 1, t.K + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:t.M, :t.K] = t.x_d
    ybuf = torch.full((t.M + 2, t.N + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    labuf = torch.full((t.M + 1, t.R), 7.0, device=DEV)
    out, la = cr.convrot_lora_forward(wide[:t.M, :t.K], t.down_d, t.up_d, t.off_d, t.ids_d,
                                      out=ybuf[1:t.M + 1, :t.N], lora_act=labuf[:t.M])
    e1, e2 = t.two_products(t.x, t.down, t.up, np.zeros_like(want), want, False)
    _near(la, la_want, e1, "lora_act")
    _near(out, want, e2, "out")
    assert (ybuf[0] == 7).all() and (ybuf[-1] == 7).all() and (ybuf[:, t.N:] == 7).all() and (labuf[t.M:] == 7).all()


def _whole(g, shape, top):
    return g.integers(-top, top + 1, shape).astype(np.float32)


@pytest.mark.parametrize("M,N,K,R", [(5, 40, 128, 8), (70, 264, 512, 64), (300, 136, 264, 128)])
def test_integers_come_out_exactly(cr, M, N, K, R):
    """lora_act beyond 16 bits needs all three bf16 terms of its float32 value."""
    g = np.random.default_rng(M)
    A, off, ids = 2, [0, M // 3, M], [1, 0]
    x = _whole(g, (M, K), 100)
    down = _whole(g, (A, R, K), 60)
    down[:, :, 4:] *= (g.random((A, R, K - 4)) < 8.0 / K)
    x[:, :4] = 255                                 # lora_act up to about 2^18
    down[:, :, :4] = _whole(g, (A, R, 4), 240)
    up = _whole(g, (A, N, R), 1) * (g.random((A, N, R)) < 8.0 / R)
    want, la_want = oa.lora_forward(x, down, up, off, ids)
    assert np.abs(la_want).max() > 2 ** 16 and np.abs(want).max() < 2 ** 24
    args = [_bf16(v)[0] for v in (x, down, up)]
    out, la = cr.convrot_lora_forward(*args, dev(np.int32(off)), dev(np.int32(ids)), out_type=cr.OUT.F32)
    assert np.array_equal(host(la), la_want) and np.array_equal(host(out), want)
    # backward: dla beyond 16 bits, and gradients of whole numbers below 2^24
    dy = _whole(g, (M, N), 1) * (g.random((M, N)) < 8.0 / N)
    dy[:, 0] = 128
    up[:, 0, :] = _whole(g, (A, R), 250)
    la_in = _whole(g, (M, R), 2 ** 17 // M)
    xs = _whole(g, (M, K), 1) * (g.random((M, K)) < 0.05)
    dn = _whole(g, (A, R, K), 1) * (g.random((A, R, K)) < 8.0 / R)
    dx, d_down, d_up, dla = oa.lora_backward(dy, la_in, xs, dn, up, off, ids)
    for v in (dx, d_down, d_up):
        assert np.abs(v).max() < 2 ** 24
    got = cr.convrot_lora_backward(_bf16(dy)[0], dev(la_in), _bf16(xs)[0], _bf16(dn)[0], _bf16(up)[0],
                                   dev(np.int32(off)), dev(np.int32(ids)), dx_type=cr.OUT.F32)
    for a, b, w in zip(got, (dx, d_down, d_up), ("dx", "d_down", "d_up")):
        assert np.array_equal(host(a), b), w


def _codes(t, rot, tensor, cr):
    """Checkpoint of t.x as codes, by the quantizer, and the input they stand for."""
    gran = cr.GRAN.TENSOR if tensor else cr.GRAN.ROW
    codes, scales, _, _ = cr.convrot_rotate_quantize(t.x_d, rot, cr.Q.SYM_INT8, gran)
    q, s = host(codes), host(scales)
    s_rows = np.broadcast_to(s, (t.M,))
    return codes, scales, q.astype(np.float64) * s_rows[:, None], oa.restore_input(q, s_rows, rot)


def _weight_bounds(t, dla_err, la, dla, x_abs, dy_abs):
    """Bounds of (d_down, d_up) for float32 la, dla with |dla error| <= dla_err."""
    bd, bu = np.zeros((t.A, t.R, x_abs.shape[1])), np.zeros((t.A, t.N, t.R))
    for a in range(t.A):
        at = t.rows == a
        n = 3 * at.sum() + 32
        bd[a] = (dla_err[at] + (n + 2) * U2 * np.abs(dla[at])).T @ x_abs[at]
        bu[a] = abs(t.c64[a]) * (n + 2) * U2 * (dy_abs[at].T @ np.abs(la[at]))
    return bd + 1e-37, bu + 1e-37


@pytest.mark.parametrize("shape", [(8200, 264, 2056, 64, 2, 5, "ragged"), (8201, 136, 520, 16, 3, 7, "gaps"),
                                   (8200, 72, 8200, 32, 2, 70, "ragged")])
def test_backward_many_rows(cr, shape):
    test_backward(cr, shape, False)


@pytest.mark.parametrize("shape", [(1500, 72, 136, 24, 1, 95, "prompt"), (2600, 40, 264, 16, 2, 150, "prompt"),
                                   (4200, 8, 8, 8, 1, 700, "ragged"), (70, 136, 264, 32, 90, 2, "ragged"),
                                   (3, 520, 72, 128, 70, 2, "tokens"), (70, 136, 264, 16, 110, 2, "ragged")])
def test_backward_many_segments_or_adapters(cr, shape):
    test_backward(cr, shape, True)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(cr, shape, f32):
    say(f"lora backward {shape} f32={f32}")
    t = Case(*shape[:6], mix=shape[6], seed=5)
    base_d, base = t.base(t.K, f32, seed=2)
    la32 = t.g.standard_normal((t.M, t.R)).astype(np.float32)
    dx_w, dd_w, du_w, dla = oa.lora_backward(t.dy, la32, t.x, t.down, t.up, t.off, t.ids, t.c, base)
    dx, dd, du = t.bwd(cr, dev(la32), dx_base=base_d, dx_type=cr.OUT.F32 if f32 else cr.OUT.BF16)
    up_t, down_t = t.up.transpose(0, 2, 1), t.down.transpose(0, 2, 1)
    c_up = t.c64[:, None, None] * up_t             # dla carries the factor c already
    keep, t.c64 = t.c64, np.ones(t.A)
    e1, e2 = t.two_products(t.dy, c_up, down_t, base, dx_w, f32)
    t.c64 = keep
    _near(dx, dx_w, e2, "dx")
    bd, bu = _weight_bounds(t, e1, la32, dla, np.abs(t.x), np.abs(t.dy))
    _near(dd, dd_w, bd, "d_down")
    _near(du, du_w, bu, "d_up")
    for a in range(t.A):
        if not (t.rows == a).any():
            assert not dd[a].any() and not du[a].any()
    # parts alone and in other company: the same bits
    dx1, n1, n2 = t.bwd(cr, None, x=None, dx_base=base_d, dx_type=cr.OUT.F32 if f32 else cr.OUT.BF16, want_weights=False)
    assert n1 is None and n2 is None and torch.equal(dx1, dx)
    n0, dd1, du1 = t.bwd(cr, dev(la32), want_dx=False)
    assert n0 is None and torch.equal(dd1, dd) and torch.equal(du1, du)


CODE_SHAPES = [(1, 8, 256, 8, 1, 1, "ragged"), (33, 136, 512, 24, 2, 4, "gaps"), (300, 72, 1024, 16, 3, 9, "ragged"),
               (513, 264, 2048, 64, 2, 5, "ragged"), (700, 128, 1024, 128, 1, 3, "gaps")]


@pytest.mark.parametrize("tensor", [False, True])
@pytest.mark.parametrize("rot", [16, 64, 256, 1024])
@pytest.mark.parametrize("shape", CODE_SHAPES)
def test_backward_from_codes(cr, shape, rot, tensor):
    if shape[2] % rot:
        pytest.skip("K is not a multiple of the rotation group")
    say(f"lora backward from codes {shape} rot {rot} tensor={tensor}")
    t = Case(*shape[:6], mix=shape[6], seed=7)
    la32 = t.g.standard_normal((t.M, t.R)).astype(np.float32)
    codes, scales, rotated, x_hat = _codes(t, rot, tensor, cr)
    _, dd_w, du_w, dla = oa.lora_backward(t.dy, la32, x_hat, t.down, t.up, t.off, t.ids, t.c)
    _, dd, du = t.bwd(cr, dev(la32), x=codes, x_scales=scales, rot_group=rot, want_dx=False)
    c_up = t.c64[:, None, None] * t.up.transpose(0, 2, 1)
    e1 = np.zeros((t.M, t.R))
    for a in range(t.A):
        at = t.rows == a
        e1[at] = (t.N + 16) * U2 * (np.abs(t.dy[at]) @ np.abs(c_up[a]).T)
    # in the rotated basis, then through the rotation
    bd, bu = _weight_bounds(t, e1, la32, dla, np.abs(rotated), np.abs(t.dy))
    for a in range(t.A):
        at = t.rows == a
        bd[a] += 2 * math.log2(rot) * U2 * (np.abs(dla[at]).T @ np.abs(rotated[at]))
    g = bd.reshape(t.A, t.R, -1, rot).sum(-1, keepdims=True) / math.sqrt(rot)
    bd = np.broadcast_to(g, (t.A, t.R, g.shape[2], rot)).reshape(bd.shape)
    _near(dd, dd_w, bd, "d_down")
    _near(du, du_w, bu, "d_up")


@pytest.mark.parametrize("rot", [64, 1024])
@pytest.mark.parametrize("shape", [(3000, 40, 1024, 16, 1, 2, "ragged"), (40, 72, 1024, 40, 9, 3, "ragged")])
def test_backward_from_codes_many_parts_or_adapters(cr, shape, rot):
    test_backward_from_codes(cr, shape, rot, False)


def test_adapters_without_rows(cr):
    """Their gradients are zeros whatever their weights and factors hold, or stay what they were."""
    t = Case(37, 136, 256, 24, 8, 2, seed=10)
    t.ids_d.fill_(5)
    la = dev(t.g.standard_normal((t.M, t.R)).astype(np.float32))
    codes, scales, _, _ = cr.convrot_rotate_quantize(t.x_d, 256, cr.Q.SYM_INT8, cr.GRAN.ROW)
    others = [a for a in range(t.A) if a != 5]
    want = [t.bwd(cr, la, **k) for k in ({}, {"x": codes, "x_scales": scales})]
    for v in (t.down_d, t.up_d, t.c_d):
        v[others] = math.inf
    for k, w in zip(({}, {"x": codes, "x_scales": scales}), want):
        got = t.bwd(cr, la, **k)
        assert all(torch.equal(a, b) for a, b in zip(got, w))
        for d in got[1:]:
            assert not d[others].any() and d[5].any()
        a, b = torch.randn_like(got[1]), torch.randn_like(got[2])
        _, dd, du = t.bwd(cr, la, d_down=a.clone(), d_up=b.clone(), accumulate=True, **k)
        assert torch.equal(dd, a + got[1]) and torch.equal(du, b + got[2])


def test_descending_offsets_end_and_stay_inside(cr):
    """What they name more than once is unspecified; rows and adapters they do not name are not."""
    t = Case(64, 72, 64, 8, 3, 300, seed=12)
    off = np.zeros(301, np.int32)
    off[1::2] = 48
    off_d, ids_d = dev(off), dev(np.zeros(300, np.int32))
    la = torch.zeros((t.M, t.R), dtype=torch.float32, device=DEV)
    dx, dd, du = cr.convrot_lora_backward(t.dy_d, la, t.x_d, t.down_d, t.up_d, off_d, ids_d)
    torch.cuda.synchronize()
    assert dx.shape == (t.M, t.K) and not dd[1:].any() and not du.any()


def test_accumulate(cr):
    t = Case(200, 136, 256, 16, 3, 5, seed=9)
    la = dev(t.g.standard_normal((t.M, t.R)).astype(np.float32))
    codes, scales, _, _ = cr.convrot_rotate_quantize(t.x_d, 256, cr.Q.SYM_INT8, cr.GRAN.ROW)
    for k in ({}, {"x": codes, "x_scales": scales}):
        _, dd, du = t.bwd(cr, la, want_dx=False, **k)
        a, b = torch.randn_like(dd), torch.randn_like(du)
        _, dd2, du2 = t.bwd(cr, la, want_dx=False, d_down=a.clone(), d_up=b.clone(), accumulate=True, **k)
        # one more float32 addition
        assert torch.equal(dd2, a + dd) and torch.equal(du2, b + du)
    with pytest.raises(ValueError):
        t.bwd(cr, la, accumulate=True)


def test_gradients_against_differences(cr):
    """out is linear in x, in down and in up: with whole numbers the difference
    of two forward passes is the directional derivative exactly."""
    g = np.random.default_rng(11)
    M, N, K, R, A = 40, 72, 64, 16, 2
    off, ids = dev(np.int32([2, 20, 33])), dev(np.int32([1, 0]))
    def few(shape, top=3):
        return _whole(g, shape, top) * (g.random(shape) < 0.3)
    x, down, up, dy = few((M, K)), few((A, R, K)), few((A, N, R)), few((M, N))
    dev3 = [_bf16(v)[0] for v in (x, down, up)]
    f = lambda a: cr.convrot_lora_forward(*a, off, ids, out_type=cr.OUT.F32)
    out, la = f(dev3)
    grads = cr.convrot_lora_backward(_bf16(dy)[0], la, *dev3, off, ids, dx_type=cr.OUT.F32)
    for i, v in enumerate((x, down, up)):
        step = few(v.shape)
        moved = list(dev3)
        moved[i] = _bf16(v + step)[0]
        change = (f(moved)[0].double() - out.double()).cpu().numpy()
        assert (change * dy).sum() == (host(grads[i]).astype(np.float64) * step).sum() != 0


def test_not_a_number_stays_in_its_row(cr):
    """Infinities and NaN of one row reach that row alone, and in the weight
    gradients its adapter alone; rows without adapter reach nothing."""
    t = Case(90, 136, 264, 16, 3, 5, seed=13)
    t.off, t.ids = np.array([0, 20, 40, 60, 80]), np.array([0, 1, -1, 2])
    t.off_d, t.ids_d = dev(np.int32(t.off)), dev(np.int32(t.ids))
    la = dev(t.g.standard_normal((t.M, t.R)).astype(np.float32))
    out, la1 = t.fwd(cr)
    dx, dd, du = t.bwd(cr, la)
    x, dy, lad = t.x_d, t.dy_d, la
    t.x_d, t.dy_d, la = x.clone(), dy.clone(), lad.clone()
    for m, v in ((5, float("nan")), (7, float("inf")), (45, float("nan")), (46, float("-inf")), (85, float("nan"))):
        t.x_d[m] = v
        t.dy_d[m] = v
        la[m] = v
    out2, la2 = t.fwd(cr)
    dx2, dd2, du2 = t.bwd(cr, la)
    fine = torch.ones(90, dtype=torch.bool, device=DEV)
    fine[[5, 7]] = False
    assert torch.equal(out2[fine], out[fine]) and torch.equal(la2[fine], la1[fine]) and torch.equal(dx2[fine], dx[fine])
    assert not torch.isfinite(la2[5]).any() and not torch.isfinite(la2[7]).any()
    assert torch.isnan(out2[5]).all() and torch.isnan(dx2[5]).all()
    for a in (1, 2):
        assert torch.equal(dd2[a], dd[a]) and torch.equal(du2[a], du[a])
    assert torch.isnan(dd2[0]).all() and torch.isnan(du2[0]).all()


def test_infinite_low_rank_value(cr):
    """An infinite lora_act times a positive weight is infinite, not NaN."""
    x = torch.full((3, 64), 3.0e38, dtype=torch.bfloat16, device=DEV)
    down = torch.ones((1, 8, 64), dtype=torch.bfloat16, device=DEV)
    up = torch.ones((1, 40, 8), dtype=torch.bfloat16, device=DEV)
    out, la = cr.convrot_lora_forward(x, down, up, dev(np.int32([0, 3])), dev(np.int32([0])))
    assert torch.isposinf(la).all() and torch.isposinf(out).all()


def test_offsets_outside_the_batch_are_clamped(cr):
    t = Case(50, 72, 64, 8, 2, 3, seed=15)
    buf = torch.full((t.M + 2, t.N), 7.0, dtype=torch.bfloat16, device=DEV)
    off = dev(np.int32([-5, 10, 60, 100]))
    ids = dev(np.int32([0, 1, 0]))
    out, _ = cr.convrot_lora_forward(t.x_d, t.down_d, t.up_d, off, ids, out=buf[1:-1])
    want, _ = cr.convrot_lora_forward(t.x_d, t.down_d, t.up_d, dev(np.int32([0, 10, 50, 50])), ids)
    assert torch.equal(out, want) and (buf[0] == 7).all() and (buf[-1] == 7).all()


def test_same_bits_twice_and_any_workspace(cr):
    t = Case(600, 256, 512, 64, 2, 7, seed=17)
    la = dev(t.g.standard_normal((t.M, t.R)).astype(np.float32))
    need = cr.convrot_lora_backward_workspace_size(t.M, t.N, t.K, t.R, t.A)
    first = t.bwd(cr, la, workspace=torch.zeros(need, dtype=torch.uint8, device=DEV))
    second = t.bwd(cr, la, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV))
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    a, b = t.fwd(cr), t.fwd(cr)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(cr.ConvRotError):
        t.bwd(cr, la, workspace=torch.zeros(need - 16, dtype=torch.uint8, device=DEV))


def test_other_stream_and_two_at_once(cr):
    t, o = Case(500, 256, 512, 32, 2, 7, seed=19), Case(333, 512, 256, 16, 3, 5, seed=20)
    want = [c.fwd(cr) + c.bwd(cr, c.fwd(cr)[1]) for c in (t, o)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for c, s in zip((t, o), streams):
            out, la = c.fwd(cr, stream=s)
            got.append((out, la) + c.bwd(cr, la, stream=s))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        for a, b in zip(g, want[k % 2]):
            assert torch.equal(a, b)


def test_captured_and_replayed(cr):
    t = Case(300, 256, 512, 32, 2, 5, seed=21)
    codes, scales, _, _ = cr.convrot_rotate_quantize(t.x_d, 256, cr.Q.SYM_INT8, cr.GRAN.ROW)
    def both():
        out, la = t.fwd(cr)
        return (out, la) + t.bwd(cr, la) + t.bwd(cr, la, x=codes, x_scales=scales)
    want = [v.clone() for v in both()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    x0 = t.x_d.clone()
    for k in range(4):
        for v in held:
            v.fill_(3)
        # other inputs in between: a replay reads what the tensors hold then
        t.x_d.copy_(x0 * (2 if k % 2 else 1))
        eager = both()
        for v in held:
            v.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)
        if k % 2 == 0:
            for a, b in zip(held, want):
                assert torch.equal(a, b)


def test_counters(cr):
    for M, launches in ((20, 1), (300, 2)):          # few rows: one launch
        t = Case(M, 72, 64, 8, 2, 3)
        cr.reset_counters()
        t.fwd(cr)
        c = cr.get_counters()
        assert c["lora"] == launches and c["fallbacks"] == 0


def test_counters_of_the_backward(cr):
    # dla with what is laid out anew, gradients; or layout, dla, gradients, and the parts' sum
    for M, R, launches in ((20, 32, 2), (300, 32, 3), (300, 40, 4)):
        t = Case(M, 72, 64, R, 2, 3)
        la = torch.zeros((M, R), dtype=torch.float32, device=DEV)
        cr.reset_counters()
        t.bwd(cr, la)
        c = cr.get_counters()
        assert c["lora"] == launches and c["fallbacks"] == 0


def test_refusals(cr):
    t = Case(20, 72, 64, 8, 2, 3)
    ok = (t.x_d, t.down_d, t.up_d, t.off_d, t.ids_d)
    def bad(i, v, **k):
        a = list(ok)
        a[i] = v
        with pytest.raises((ValueError, cr.ConvRotError)):
            cr.convrot_lora_forward(*a, **k)
    bad(0, t.x_d.float())
    bad(0, t.x_d.cpu())
    bad(0, t.x_d.t().contiguous().t())
    bad(0, t.x_d[:1].expand(20, 64))              # rows at one address
    bad(0, t.x_d[:0])
    bad(1, t.down_d[:, :, :56].contiguous())
    bad(1, t.down_d[:, :4].contiguous())
    bad(2, t.up_d.transpose(1, 2))
    bad(2, t.up_d[:1])
    bad(3, t.off_d.long())
    bad(3, t.off_d[:-1])
    bad(4, t.ids_d.cpu())
    bad(0, t.x_d, scale=t.c_d.double())
    bad(0, t.x_d, out_type=cr.OUT.I32_RAW)
    bad(0, t.x_d, base=torch.zeros((20, 72), device=DEV))
    bad(0, t.x_d, out=torch.zeros((20, 64), dtype=torch.bfloat16, device=DEV))
    bad(0, t.x_d, lora_act=torch.zeros((20, 8), dtype=torch.bfloat16, device=DEV))
    buf = torch.zeros((20, 80), dtype=torch.bfloat16, device=DEV)
    bad(0, t.x_d[:, 4:])                           # rows not 16-byte aligned
    la = torch.zeros((20, 8), device=DEV)
    codes = torch.zeros((20, 64), dtype=torch.int8, device=DEV)
    for k in ({"x": codes}, {"x": codes, "x_scales": torch.zeros(20, device=DEV)}, {"x": None}, {"dx": buf},
              {"want_dx": False, "want_weights": False}, {"d_down": torch.zeros((2, 8, 64), device=DEV).bfloat16()},
              {"workspace": torch.zeros(16, dtype=torch.uint8, device=DEV)}):
        with pytest.raises((ValueError, AttributeError, cr.ConvRotError)):
            t.bwd(cr, la, **k)
