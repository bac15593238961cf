"""GPU parity of layer norm and its gradients against the float64 oracle.

With u = 2^-24: a sum over a row takes at most 64 values a lane, 6 steps over the
wave and 8 over waves, so it is off by at most D = 80 u of the sum of magnitudes;
a sum over the rows of a sequence by at most (rows + 30) u. What follows
from these and from one rounding an operation stands in _forward_bound and
_backward_bound; an output of a type adds half a step."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import training as tr  # noqa: E402
from tests.gpu_helpers import DEV, dev, say  # noqa: E402

U = 2.0 ** -24
D = 80 * U
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a8_rotated_quantized_amd as m
    assert m.device_check() == 0, "device is not gfx950"
    return m


def _out(cr, dtype):
    return cr.OUT.BF16 if dtype is torch.bfloat16 else cr.OUT.F32


def _f64(t):
    return t.double().cpu().numpy()


def _input(g, shape, dtype, std=1.0, shift=0.0, pad=0):
    """Random rows on the GPU, further apart by pad columns that hold something else."""
    wide = np.full((shape[0], shape[1] + pad), 1e4, np.float32)
    wide[:, :shape[1]] = g.standard_normal(shape) * std + shift
    return dev(wide).to(dtype)[:, :shape[1]]


def _forward_bound(x, w, y, mean, rstd, dtype, eps):
    d = np.abs(x - mean[:, None])
    dm = D * np.abs(x).mean(1) + U * np.abs(mean)
    var = 1 / rstd ** 2
    rel = D + 8 * U + (2 * dm * d.mean(1) + dm * dm) / var
    xh = d * rstd[:, None]
    return (np.abs(w) * (rstd[:, None] * dm[:, None] + xh * (rel[:, None] + 4 * U)) + (2 * U + HALF[dtype] * (1 + 2 ** -8)) * np.abs(y)
            + 2 * U * np.abs(w) * xh + 1e-37), dm, rel * rstd


def _backward_bound(dy, x, mean, rstd, w, dx, dtype):
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    g = np.abs(dy * w)
    a, b = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    part = 4 * U * g + (D + 4 * U) * a + (D + 12 * U) * xh * b + 4 * U * (g + a + xh * b)
    return rstd[:, None] * part + (2 * U + HALF[dtype] * (1 + 2 ** -8)) * np.abs(dx) + 1e-37


def _sequences(g, M, S):
    """Ragged offsets with empty sequences, and rows in none at both ends where there is room."""
    lo, hi = (M // 9, M - M // 7) if M > 20 else (0, M)
    return np.concatenate([[lo], np.sort(g.integers(lo, hi + 1, S - 1)), [hi]]).astype(np.int32)


# columns at the borders between the variants: waves a row and values a lane
COLS = [8, 72, 512, 520, 1024, 1032, 2048, 2056, 2560, 4096, 4104, 8192, 8200, 12288, 16384]
CASES = [(M, C, S, x, y) for i, C in enumerate(COLS) for M, S in ((1, 0), (5, 3), (70, 0), (203, 9))
         for x, y in [(("bf16", "f32")[(i + M) % 2], ("f32", "bf16")[(i // 2 + S) % 2])]]


def _case(cr, M, C, S, xt, dyt, affine, plus):
    g = np.random.default_rng([M, C, S])
    x = _input(g, (M, C), TYPES[xt], 1.5, 0.7, 8)
    dy = _input(g, (M, C), TYPES[dyt], 0.1, 0.01, 16)
    shape = (S, C) if S else (C,)
    w = dev((g.standard_normal(shape) * 0.3 + (0 if plus else 1)).astype(np.float32)).to(TYPES[affine])
    b = dev((g.standard_normal(shape) * 0.3).astype(np.float32)).to(TYPES[affine])
    off = _sequences(g, M, S) if S else None
    rows = tr.sequences(off, M) if S else np.zeros(M, np.int64)
    return x, dy, w, b, off, rows


@pytest.mark.parametrize("M,C,S,xt,yt", CASES)
def test_forward_and_backward(cr, M, C, S, xt, yt):
    say(f"norm {M}x{C} sequences {S} {xt} -> {yt}")
    plus = bool(S)
    affine = "bf16" if (M + C // 8) % 2 else "f32"
    x, dy, w, b, off, rows = _case(cr, M, C, S, xt, yt, affine, plus)
    toff = None if off is None else dev(off)
    ytype = TYPES[yt]
    hold = torch.full((M, C + 8), -9.0, dtype=ytype, device=DEV)
    mean, rstd = torch.full((M,), -7.0, device=DEV), torch.full((M,), -7.0, device=DEV)
    cr.convrot_layer_norm_forward(x, w, b, seg_offsets=toff, one_plus=plus, eps=1e-5, out_type=_out(cr, ytype), out=hold[:, :C],
                                  mean=mean, rstd=rstd)
    assert bool((hold[:, C:] == -9).all())
    at = rows >= 0
    x64, w64, b64 = _f64(x), _f64(w), _f64(b)
    want, m64, r64 = tr.norm_forward(x64, w64, b64, rows, float(plus), 1e-5)
    wr = w64.reshape(-1, C)[rows] + plus
    bound, dm, dr = _forward_bound(x64, wr, want, m64, r64, ytype, 1e-5)
    y = _f64(hold[:, :C])
    assert np.all((np.abs(y - want) <= bound)[at]), (np.abs(y - want) / bound)[at].max()
    assert np.all((np.abs(_f64(mean) - m64) <= dm)[at]) and np.all((np.abs(_f64(rstd) - r64) <= dr)[at])
    assert np.all(y[~at] == -9) and np.all(_f64(mean)[~at] == -7) and np.all(_f64(rstd)[~at] == -7)

    # backward, from the float32 moments the forward pass kept
    n = max(S, 1)
    base = _input(np.random.default_rng(5), (M, C), ytype, 0.1, 0.0, 8) if M % 2 else None
    dx = torch.full((M, C), -9.0, dtype=ytype, device=DEV)
    _, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=toff, one_plus=plus, dx_base=base,
                                               dx_type=_out(cr, ytype), dx=dx)
    mk, rk, dy64 = _f64(mean), _f64(rstd), _f64(dy)
    dxw, dww, dbw = tr.norm_backward(dy64, x64, mk, rk, w64, rows, float(plus), n, None if base is None else _f64(base))
    bound = _backward_bound(dy64, x64, mk, rk, wr, dxw, ytype)
    got = _f64(dx)
    assert np.all((np.abs(got - dxw) <= bound)[at]), (np.abs(got - dxw) / bound)[at].max()
    assert np.all(got[~at] == -9)
    xh = np.abs((x64 - mk[:, None]) * rk[:, None])
    for s in range(n):
        r = rows == s
        most = (int(r.sum()) + 34) * U
        assert np.all(np.abs(_f64(dw).reshape(n, C)[s] - dww[s]) <= most * (np.abs(dy64) * xh)[r].sum(0))
        assert np.all(np.abs(_f64(db).reshape(n, C)[s] - dbw[s]) <= most * np.abs(dy64)[r].sum(0))


@pytest.mark.parametrize("M,C,S", [(3000, 640, 0), (2500, 2560, 40), (8200, 72, 5), (1100, 4096, 130), (600, 8192, 2)])
def test_many_rows(cr, M, C, S):
    say(f"norm rows {M}x{C} sequences {S}")
    x, dy, w, b, off, rows = _case(cr, M, C, S, "bf16", "bf16", "bf16", bool(S))
    toff = None if off is None else dev(off)
    _, mean, rstd = cr.convrot_layer_norm_forward(x, w, b, seg_offsets=toff, one_plus=bool(S),
                                                  mean=torch.zeros(M, device=DEV), rstd=torch.zeros(M, device=DEV))
    n = max(S, 1)
    first = None
    for _ in range(3):
        _, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=toff, one_plus=bool(S), want_dx=False)
        if first is not None:
            assert torch.equal(dw, first[0]) and torch.equal(db, first[1]), "sums depend on timing"
        first = dw, db
    x64, dy64, mk, rk = _f64(x), _f64(dy), _f64(mean), _f64(rstd)
    _, dww, dbw = tr.norm_backward(dy64, x64, mk, rk, _f64(w), rows, float(bool(S)), n)
    xh = np.abs((x64 - mk[:, None]) * rk[:, None])
    for s in range(n):
        r = rows == s
        most = (int(r.sum()) + 34) * U
        assert np.all(np.abs(_f64(dw).reshape(n, C)[s] - dww[s]) <= most * (np.abs(dy64) * xh)[r].sum(0))
        assert np.all(np.abs(_f64(db).reshape(n, C)[s] - dbw[s]) <= most * np.abs(dy64)[r].sum(0))
    # added to what is there
    dw2, db2 = first[0].clone(), first[1].clone()
    cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=toff, one_plus=bool(S), want_dx=False, d_weight=dw2,
                                   d_bias=db2, accumulate=True)
    assert torch.equal(dw2, first[0] + first[0]) and torch.equal(db2, first[1] + first[1])


def test_gradient_by_differences(cr):
    """dx and dw against differences of the forward call itself, in float32."""
    g = np.random.default_rng(8)
    M, C = 4, 64
    x, dy = dev(g.standard_normal((M, C)).astype(np.float32)), dev(g.standard_normal((M, C)).astype(np.float32))
    w, b = dev(g.standard_normal(C).astype(np.float32)), dev(g.standard_normal(C).astype(np.float32))
    def loss(x, w, b):
        y, _, _ = cr.convrot_layer_norm_forward(x, w, b, out_type=cr.OUT.F32)
        return float((y.double() * dy.double()).sum())
    _, mean, rstd = cr.convrot_layer_norm_forward(x, w, b, out_type=cr.OUT.F32)
    dx, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, dx_type=cr.OUT.F32)
    # h = 2^-6: the third derivative gives about h^2 / 6 of order-one terms, rounding C 2^-24 / h
    h = 2.0 ** -6
    for i, j in ((0, 0), (1, 17), (3, 63)):
        e = torch.zeros_like(x)
        e[i, j] = h
        assert abs((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * h) - float(dx[i, j])) < 2e-3 * float(dx.abs().max())
    for j in (0, 40):
        e = torch.zeros_like(w)
        e[j] = h
        assert abs((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h) - float(dw[j])) < 2e-3 * float(dw.abs().max())
        assert abs((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h) - float(db[j])) < 2e-3 * float(db.abs().max())


def test_without_weight_or_bias_and_partial_gradients(cr):
    g = np.random.default_rng(9)
    M, C = 37, 328
    x, dy = _input(g, (M, C), torch.bfloat16), _input(g, (M, C), torch.float32)
    y, mean, rstd = cr.convrot_layer_norm_forward(x, out_type=cr.OUT.F32)
    want, m64, r64 = tr.norm_forward(_f64(x))
    bound, _, _ = _forward_bound(_f64(x), np.ones((M, C)), want, m64, r64, torch.float32, 1e-6)
    assert np.all(np.abs(_f64(y) - want) <= bound)
    b = dev(g.standard_normal(C).astype(np.float32))
    y2, _, _ = cr.convrot_layer_norm_forward(x, bias=b, one_plus=True, out_type=cr.OUT.F32)
    assert torch.equal(y2, y + b)
    dx, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, dx_type=cr.OUT.F32)
    only, none, _ = cr.convrot_layer_norm_backward(dy, x, mean, rstd, dx_type=cr.OUT.F32, want_weights=False)
    assert none is None and torch.equal(only, dx)
    # the residual's gradient in place
    same = dx.clone()
    base = dev(g.standard_normal((M, C)).astype(np.float32))
    apart, _, _ = cr.convrot_layer_norm_backward(dy, x, mean, rstd, dx_base=base, dx_type=cr.OUT.F32, want_weights=False)
    inplace = base.clone()
    cr.convrot_layer_norm_backward(dy, x, mean, rstd, dx_base=inplace, dx=inplace, dx_type=cr.OUT.F32, want_weights=False)
    assert torch.equal(apart, inplace) and torch.equal(same, dx)


def test_constant_rows_and_not_finite(cr):
    """A row without variance has xh = 0; an infinity or NaN stays in its row, and in its sequence's sums."""
    M, C = 9, 264
    g = np.random.default_rng(10)
    x = _input(g, (M, C), torch.float32)
    x[0], x[1], x[2] = 3.0, 0.0, -1e30
    w, b = torch.ones((3, C), device=DEV), torch.full((3, C), 0.25, device=DEV)
    off = torch.tensor([0, 3, 6, 9], dtype=torch.int32, device=DEV)
    x[4, 100], x[5, 3] = float("inf"), float("nan")
    y, mean, rstd = cr.convrot_layer_norm_forward(x, w, b, seg_offsets=off, out_type=cr.OUT.F32, eps=1e-5)
    assert bool((y[:3] == 0.25).all())
    # a float32 sum of 264 equal values and its product with a rounded 1 / 264: off by at most D like any mean
    assert abs(float(mean[0]) - 3) <= D * 3 and float(mean[1]) == 0 and abs(float(mean[2]) + 1e30) <= (D + U) * 1e30
    assert bool(torch.isfinite(y[[0, 1, 2, 3, 6, 7, 8]]).all()) and bool(torch.isnan(y[4]).any()) and bool(torch.isnan(y[5]).all())
    dy = torch.ones((M, C), device=DEV)
    dx, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=off, dx_type=cr.OUT.F32)
    assert bool(torch.isfinite(dx[[0, 1, 2, 3, 6, 7, 8]]).all()) and bool(torch.isfinite(dw[[0, 2]]).all())
    assert bool(torch.isnan(dw[1]).any()) and bool((db == 3).all())


def test_offsets_that_descend(cr):
    """One below an earlier one counts as that one; what lies outside the batch is cut off."""
    g = np.random.default_rng(11)
    M, C = 50, 80
    x, dy = _input(g, (M, C), torch.float32), _input(g, (M, C), torch.float32)
    for off in ([0, 30, 10, 45], [-7, 20, 20, 90], [5, 4, 3, 2], [60, 70, 80, 90], [50, 50, 50, 50]):
        S = len(off) - 1
        w = dev(g.standard_normal((S, C)).astype(np.float32))
        to = torch.tensor(off, dtype=torch.int32, device=DEV)
        rows = tr.sequences(off, M)
        y = torch.full((M, C), -9.0, device=DEV)
        mean, rstd = torch.zeros(M, device=DEV), torch.zeros(M, device=DEV)
        cr.convrot_layer_norm_forward(x, w, seg_offsets=to, out_type=cr.OUT.F32, out=y, mean=mean, rstd=rstd)
        assert np.array_equal((_f64(y) == -9).all(1), rows < 0), off
        _, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=to, want_dx=False)
        _, dww, dbw = tr.norm_backward(_f64(dy), _f64(x), _f64(mean), _f64(rstd), _f64(w), rows, 0.0, S)
        assert np.allclose(_f64(dw), dww, atol=1e-4, rtol=1e-4) and np.allclose(_f64(db), dbw, atol=1e-4, rtol=1e-4), off


def test_modulation_columns(cr):
    """Weight and bias as column blocks of one modulation tensor, as the adaLN layer gives it."""
    g = np.random.default_rng(13)
    M, C, S = 90, 328, 3
    x, dy = _input(g, (M, C), torch.bfloat16), _input(g, (M, C), torch.bfloat16)
    off = torch.tensor([0, 30, 31, 90], dtype=torch.int32, device=DEV)
    for dtype in (torch.bfloat16, torch.float32):
        mod = dev(g.standard_normal((S, 6 * C)).astype(np.float32)).to(dtype)
        shift, scale = mod.chunk(6, 1)[3], mod.chunk(6, 1)[1]
        y, mean, rstd = cr.convrot_layer_norm_forward(x, scale, shift, seg_offsets=off, one_plus=True)
        y2, _, _ = cr.convrot_layer_norm_forward(x, scale.contiguous(), shift.contiguous(), seg_offsets=off, one_plus=True)
        assert torch.equal(y, y2)
        a = cr.convrot_layer_norm_backward(dy, x, mean, rstd, scale, seg_offsets=off, one_plus=True)
        b = cr.convrot_layer_norm_backward(dy, x, mean, rstd, scale.contiguous(), seg_offsets=off, one_plus=True)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    # one sequence takes its only row wherever the next would lie
    y, _, _ = cr.convrot_layer_norm_forward(x, scale[:1], shift[:1], seg_offsets=off[[0, 3]].contiguous())
    want, _, _ = cr.convrot_layer_norm_forward(x, scale[0].contiguous(), shift[0].contiguous())
    assert torch.equal(y, want)


@pytest.mark.parametrize("C", [72, 640, 1200, 4104])
@pytest.mark.parametrize("S,kind", [(300, "ragged"), (1500, "even"), (4096, "ragged"), (700, "descending")])
def test_many_sequences(cr, C, S, kind):
    """Hundreds and thousands of sequences: whole in a part, across parts, empty; offsets that descend here and there."""
    M = 2100
    say(f"norm {S} {kind} sequences of {C}")
    g = np.random.default_rng([S, C])
    off = np.arange(S + 1) * M // S if kind == "even" else np.sort(np.concatenate([[3, M - 5], g.integers(0, M + 1, S - 1)]))
    if kind == "descending":
        at = g.integers(1, S, 60)
        off[at] = g.integers(-50, M, 60)
    off = off.astype(np.int32)
    rows = tr.sequences(off, M)
    x, dy = _input(g, (M, C), torch.bfloat16, 1.5, 0.7), _input(g, (M, C), torch.bfloat16, 0.1)
    w, b = (dev((g.standard_normal((S, C)) * 0.3).astype(np.float32)) for _ in range(2))
    to = dev(off)
    y = torch.full((M, C), -9.0, device=DEV)
    mean, rstd = torch.zeros(M, device=DEV), torch.zeros(M, device=DEV)
    cr.convrot_layer_norm_forward(x, w, b, seg_offsets=to, one_plus=True, out_type=cr.OUT.F32, out=y, mean=mean, rstd=rstd)
    want, m64, r64 = tr.norm_forward(_f64(x), _f64(w), _f64(b), rows, 1.0)
    wr = _f64(w)[rows] + 1
    bound, _, _ = _forward_bound(_f64(x), wr, want, m64, r64, torch.float32, 1e-6)
    at = rows >= 0
    assert np.all((np.abs(_f64(y) - want) <= bound)[at]) and np.all(_f64(y)[~at] == -9)
    start = torch.ones((S, C), device=DEV), torch.full((S, C), 2.0, device=DEV)
    dx, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=to, one_plus=True, dx_type=cr.OUT.F32)
    dxw, dww, dbw = tr.norm_backward(_f64(dy), _f64(x), _f64(mean), _f64(rstd), _f64(w), rows, 1.0, S)
    assert np.all((np.abs(_f64(dx) - dxw) <= _backward_bound(_f64(dy), _f64(x), _f64(mean), _f64(rstd), wr, dxw, torch.float32))[at])
    xh = np.abs((_f64(x) - _f64(mean)[:, None]) * _f64(rstd)[:, None])
    mag_w, mag_b, most = np.zeros((S, C)), np.zeros((S, C)), np.zeros((S, 1))
    np.add.at(mag_w, rows[at], (np.abs(_f64(dy)) * xh)[at])
    np.add.at(mag_b, rows[at], np.abs(_f64(dy))[at])
    np.add.at(most, rows[at], 1.0)
    assert np.all(np.abs(_f64(dw) - dww) <= (most + 34) * U * mag_w) and np.all(np.abs(_f64(db) - dbw) <= (most + 34) * U * mag_b)
    cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=to, one_plus=True, want_dx=False, d_weight=start[0], d_bias=start[1],
                                   accumulate=True)
    assert torch.equal(start[0], dw + 1) and torch.equal(start[1], db + 2)


def test_one_row(cr):
    """One part: the backward pass in one launch gives the sums itself."""
    g = np.random.default_rng(14)
    x, dy = _input(g, (1, 520), torch.float32), _input(g, (1, 520), torch.float32)
    _, mean, rstd = cr.convrot_layer_norm_forward(x)
    cr.reset_counters()
    _, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, dx_type=cr.OUT.F32)
    assert cr.get_counters()["act"] == 1 and cr.get_counters()["fallbacks"] == 0
    assert torch.equal(db, dy[0]) and torch.equal(dw, dy[0] * ((x[0] - mean) * rstd))


def test_side_stream_and_graph(cr):
    """On a given stream, and captured: replays equal the eager results, other work between them."""
    g = np.random.default_rng(12)
    M, C, S = 300, 2560, 4
    x, dy = _input(g, (M, C), torch.bfloat16), _input(g, (M, C), torch.bfloat16)
    w, b = dev(g.standard_normal((S, C)).astype(np.float32)), dev(g.standard_normal((S, C)).astype(np.float32))
    off = torch.tensor([0, 100, 100, 250, 300], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = cr.convrot_layer_norm_forward(x, w, b, seg_offsets=off, one_plus=True, stream=side)
    grads = cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=off, one_plus=True, stream=side)
    side.synchronize()
    want = (y.clone(), *[t.clone() for t in grads])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cy, cm, crs = cr.convrot_layer_norm_forward(x, w, b, seg_offsets=off, one_plus=True)
        cg = cr.convrot_layer_norm_backward(dy, x, cm, crs, w, seg_offsets=off, one_plus=True)
    for _ in range(4):
        for t in (cy, *cg):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, e in zip((cy, *cg), want):
            assert torch.equal(t, e)
        (x.float() @ x.float().t()).sum().item()


@pytest.mark.parametrize("M,C,S,xt,yt", [(4100, 2056, 3, "bf16", "f32"), (4203, 2560, 0, "f32", "bf16"), (4200, 1200, 6, "bf16", "bf16"),
                                         (2101, 2048, 4, "f32", "f32"), (1531, 1536, 2, "bf16", "bf16"), (900, 3000, 5, "bf16", "f32"),
                                         (2050, 2568, 0, "bf16", "bf16"), (701, 6000, 3, "f32", "f32"), (517, 10008, 4, "bf16", "bf16"),
                                         (5000, 400, 30, "bf16", "bf16")])
def test_shapes_of_many_rows(cr, M, C, S, xt, yt):
    """Variants that only many rows take, and parts of several rounds of every group."""
    test_forward_and_backward(cr, M, C, S, xt, yt)


def test_what_stands_in_no_sequence_does_not_matter(cr):
    g = np.random.default_rng(21)
    M, C = 700, 2560
    off = torch.tensor([90, 300, 300, 610], dtype=torch.int32, device=DEV)
    x, dy = _input(g, (M, C), torch.bfloat16, 1.5, 0.7), _input(g, (M, C), torch.bfloat16)
    w, b = dev(g.standard_normal((3, C)).astype(np.float32)), dev(g.standard_normal((3, C)).astype(np.float32))

    def run():
        y, dx = torch.full((M, C), -9.0, device=DEV), torch.full((M, C), -9.0, device=DEV)
        mean, rstd = torch.zeros(M, device=DEV), torch.zeros(M, device=DEV)
        cr.convrot_layer_norm_forward(x, w, b, seg_offsets=off, out_type=cr.OUT.F32, out=y, mean=mean, rstd=rstd)
        return (y, mean, rstd, *cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=off, dx_type=cr.OUT.F32, dx=dx))

    want = run()
    for v in (float("nan"), float("inf"), -3e38):
        for t in (x, dy):
            t[:90] = v
            t[610:] = v
        for a, e in zip(run(), want):
            assert torch.equal(a, e)


def test_the_smallest_eps(cr):
    """Rows without variance are all bias, whatever the eps above 0."""
    x = torch.cat([torch.zeros((3, 520), device=DEV), torch.full((2, 520), 4.0, device=DEV)])
    b = torch.randn(520, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    for eps in (2.0 ** -149, 2.0 ** -126, 1e-6):
        y, mean, rstd = cr.convrot_layer_norm_forward(x, bias=b, eps=eps, out_type=cr.OUT.F32)
        assert torch.equal(y[:3], b.expand(3, -1)) and bool(torch.isfinite(rstd).all()) and bool((mean[:3] == 0).all())
        # the mean of 520 fours is within 80 roundings of 4, or no row without variance: y stays finite
        assert bool(torch.isfinite(y).all())
    with pytest.raises(cr.ConvRotError):
        cr.convrot_layer_norm_forward(x, eps=1e-50)
