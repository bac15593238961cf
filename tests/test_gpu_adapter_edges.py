"""Calls of the adapter and checkpoint entry points at the edges of what their
documentation allows: offsets in any order, tensors that are freed right after
a call on another stream, infinite weights, codes of a smoothed input, loops
with several stages per wave, the far tails of the activations, addresses
beyond 32 bits, gradients in place.

Bounds are those of test_gpu_lora.py and test_gpu_act.py unless a test derives
its own."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import tests.test_gpu_act as act_tests  # noqa: E402
import tests.test_gpu_lora as lora_tests  # noqa: E402
import workloads as wl  # noqa: E402
from oracle import adapters as oa  # noqa: E402
from tests.gpu_helpers import DEV, bf16_dev, bf16_to_f32, dev, host, rel_l2, say  # noqa: E402
from tests.test_gpu_lora import U2, Case, _near, _weight_bounds, cr  # noqa: E402, F401


def _descending(kind, M, S, g):
    if kind == "up and down":                      # 48 of 64 rows named again and again
        off = np.zeros(S + 1, np.int64)
        off[1::2] = 3 * M // 4
    elif kind == "falling":
        off = np.linspace(3 * M // 4, 0, S + 1).astype(np.int64)
    else:
        off = g.integers(-M // 4, 3 * M // 4, S + 1)
    return off


@pytest.mark.parametrize("kind", ["up and down", "falling", "any"])
@pytest.mark.parametrize("M,N,K,R,A,S", [(64, 72, 64, 8, 3, 300), (40, 136, 72, 40, 2, 9), (700, 264, 136, 24, 3, 130),
                                         (300, 72, 256, 64, 1, 66)])
def test_offsets_in_any_order(cr, M, N, K, R, A, S, kind):
    """An offset below an earlier one counts as that earlier one. Every row is
    written, rows that no segment names are base and reach no gradient."""
    say(f"offsets {kind} {M} {N} {K} {R} {A} {S}")
    t = Case(M, N, K, R, A, S, seed=31)
    t.off, t.ids = _descending(kind, M, S, t.g), t.g.integers(0, A, S)
    t.off_d, t.ids_d = dev(t.off.astype(np.int32)), dev(t.ids.astype(np.int32))
    off = np.maximum.accumulate(np.clip(t.off, 0, M))
    t.rows = oa.row_adapters(off, t.ids, M, A)
    none = t.rows < 0
    assert none[3 * M // 4 + 1:].all()
    la32 = t.g.standard_normal((M, R)).astype(np.float32)
    la_d, none_d = dev(la32), dev(none)
    for v in (t.x_d, t.dy_d, la_d):
        v[none_d] = float("nan")
    for v in (t.x, t.dy, la32):
        v[none] = 0
    base_d, base = t.base(N, True)
    out, la = t.fwd(cr, base=base_d, out_type=cr.OUT.F32, out=torch.full((M, N), float("nan"), device=DEV),
                    lora_act=torch.full((M, R), float("nan"), device=DEV))
    want, la_want = oa.lora_forward(t.x, t.down, t.up, off, t.ids, t.c, base)
    e1, e2 = t.two_products(t.x, t.down, t.up, base, want, True)
    _near(la, la_want, e1, "lora_act")
    _near(out, want, e2, "out")
    assert torch.equal(out[none_d], base_d[none_d]) and not la[none_d].any()
    base_d, base = t.base(K, True, seed=2)
    dx, dd, du = t.bwd(cr, la_d, dx_base=base_d, dx_type=cr.OUT.F32, dx=torch.full((M, K), float("nan"), device=DEV))
    dx_w, dd_w, du_w, dla = oa.lora_backward(t.dy, la32, t.x, t.down, t.up, off, t.ids, t.c, base)
    c_up = t.c64[:, None, None] * t.up.transpose(0, 2, 1)
    keep, t.c64 = t.c64, np.ones(A)
    e1, e2 = t.two_products(t.dy, c_up, t.down.transpose(0, 2, 1), base, dx_w, True)
    t.c64 = keep
    _near(dx, dx_w, e2, "dx")
    assert torch.equal(dx[none_d], base_d[none_d])
    bd, bu = _weight_bounds(t, e1, la32, dla, np.abs(t.x), np.abs(t.dy))
    _near(dd, dd_w, bd, "d_down")
    _near(du, du_w, bu, "d_up")
    # the same call with the offsets written out: the same bits
    t.off_d = dev(off.astype(np.int32))
    fwd = t.fwd(cr, base=t.base(N, True)[0], out_type=cr.OUT.F32)
    bwd = t.bwd(cr, la_d, dx_base=base_d, dx_type=cr.OUT.F32)
    for a, b in zip((out, la, dx, dd, du), fwd + bwd):
        assert torch.equal(a, b)


def test_inputs_freed_while_another_stream_reads_them(cr):
    """A call on a given stream keeps the memory of its tensors: what the
    caller frees right after it is not given out again before the call ends."""
    t = Case(300, 136, 256, 16, 2, 5, seed=33)
    la_d = dev(t.g.standard_normal((t.M, t.R)).astype(np.float32))
    codes, scales, _, _ = cr.convrot_rotate_quantize(t.x_d, 256, cr.Q.SYM_INT8, cr.GRAN.ROW)
    base, dx_base = t.base(t.N, False)[0], t.base(t.K, False, seed=2)[0]
    z = t.dy_d[:, :128].contiguous()
    _, zc, zs = cr.convrot_act_checkpoint(z, cr.ACT.GELU)
    adapters = (t.down_d, t.up_d, t.off_d, t.ids_d, t.c_d)
    calls = (
        ("forward", lambda s, x, b, *a: cr.convrot_lora_forward(x, *a, base=b, stream=s), (t.x_d, base, *adapters)),
        ("backward", lambda s, dy, la, x, xs, b, ws, *a: cr.convrot_lora_backward(
            dy, la, x, *a, x_scales=xs, dx_base=b, workspace=ws, stream=s),
         (t.dy_d, la_d, codes, scales, dx_base,
          torch.zeros(cr.convrot_lora_backward_workspace_size(t.M, t.N, t.K, t.R, t.A), dtype=torch.uint8, device=DEV),
          *adapters)),
        ("checkpoint", lambda s, v: cr.convrot_act_checkpoint(v, cr.ACT.GELU, stream=s), (z,)),
        ("slope", lambda s, *v: (cr.convrot_act_backward(*v, cr.ACT.GELU, stream=s),), (z, zc, zs)))
    for name, call, args in calls:
        say(f"freed inputs: {name}")
        want = call(None, *args)
        held = [v.clone() for v in args]
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            torch.cuda._sleep(50_000_000)          # the call waits behind it
        got = call(other, *held)
        freed = {v.data_ptr() for v in held}
        del held
        fresh = [torch.full_like(v, 3) for v in args]
        waiting = not other.query()
        assert not waiting or not freed & {v.data_ptr() for v in fresh}, name
        torch.cuda.synchronize()
        assert waiting, "the other stream ended before the memory was asked for"
        for a, b in zip(got, want):
            assert torch.equal(a, b), name


def test_captured_on_a_given_stream(cr):
    t = Case(300, 136, 256, 16, 2, 5, seed=34)
    z = t.dy_d[:, :128].contiguous()
    def all_of_them(s):
        out, la = t.fwd(cr, stream=s)
        y, codes, scales = cr.convrot_act_checkpoint(z, cr.ACT.GELU_TANH, stream=s)
        return (out, la, *t.bwd(cr, la, stream=s), y, cr.convrot_act_backward(y, codes, scales, cr.ACT.GELU_TANH, stream=s))
    want = all_of_them(None)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = all_of_them(side)
    for _ in range(3):
        for v in held:
            v.fill_(5)
        again = all_of_them(None)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(held, again, want):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_codes_of_a_smoothed_input(cr):
    """Codes made with `smooth` stand for x * smooth: the call gives that
    input's d_down, and dividing its columns by smooth gives the gradient."""
    t = Case(200, 136, 512, 16, 2, 4, seed=35)
    la32 = t.g.standard_normal((t.M, t.R)).astype(np.float32)
    smooth = np.exp2(t.g.integers(-3, 4, t.K)).astype(np.float32)      # powers of two: x * smooth and the division are exact
    codes, scales, _, _ = cr.convrot_rotate_quantize(t.x_d, 256, cr.Q.SYM_INT8, cr.GRAN.ROW, smooth=dev(smooth))
    _, dd, _ = t.bwd(cr, dev(la32), x=codes, x_scales=scales, want_dx=False)
    x_hat = oa.restore_input(host(codes), host(scales), 256)
    _, want, _, dla = oa.lora_backward(t.dy, la32, x_hat / smooth, t.down, t.up, t.off, t.ids, t.c)
    # what the sums and the rotation (8 steps, two roundings each) of rotated codes may be off by
    rotated = np.abs(host(codes).astype(np.float64) * host(scales).astype(np.float64)[:, None])
    c_up = t.c64[:, None, None] * t.up.transpose(0, 2, 1)
    e1 = np.zeros((t.M, t.R))
    for a in range(t.A):
        at = t.rows == a
        e1[at] = (t.N + 16) * U2 * (np.abs(t.dy[at]) @ np.abs(c_up[a]).T)
    bd, _ = _weight_bounds(t, e1, la32, dla, rotated, np.abs(t.dy))
    for a in range(t.A):
        at = t.rows == a
        bd[a] += 16 * U2 * (np.abs(dla[at]).T @ rotated[at])
    g = bd.reshape(t.A, t.R, -1, 256).sum(-1, keepdims=True) / 16
    bd = np.broadcast_to(g, (t.A, t.R, g.shape[2], 256)).reshape(bd.shape)
    _near(dd / dev(smooth), want, bd / smooth, "d_down / smooth")
    # and that is the gradient of x itself up to the codes' 8 bits: a row of four to six sigma has a step
    # of 1/21 sigma at most, an error of step / sqrt 12, 1.4 percent of sigma (x * smooth: of its largest columns)
    _, true, _, _ = oa.lora_backward(t.dy, la32, t.x, t.down, t.up, t.off, t.ids, t.c)
    assert rel_l2(host(dd), true * smooth) <= 0.05


def test_infinite_weights_and_gradients(cr):
    """An infinite bf16 value makes exactly the sums it enters infinite or NaN:
    which of the two is open where it meets a float32 factor, and an infinity
    where a bf16 one meets bf16. All other values keep their bits."""
    t = Case(90, 136, 264, 16, 2, 3, seed=36, scale=False)
    t.off_d, t.ids_d = dev(np.int32([0, 30, 60, 90])), dev(np.int32([0, 1, -1]))
    la_d = dev(np.where(t.g.random((t.M, t.R)) < 0.5, 1.0, t.g.standard_normal((t.M, t.R))).astype(np.float32))
    out, la = t.fwd(cr)
    dx, dd, du = t.bwd(cr, la_d)
    def only(got, was, at, what):
        """got is not finite exactly where `at` says, and was's bits elsewhere"""
        m = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
        m[at] = True
        assert not torch.isfinite(got[m]).any() and torch.equal(got[~m], was[~m]), what
    rows0, every = slice(0, 30), slice(None)
    keep = t.up_d[0, 70, 3].clone()
    t.up_d[0, 70, 3] = float("inf")                # enters column 70 of out and rank 3 of dla
    out2, la2 = t.fwd(cr)
    dx2, dd2, du2 = t.bwd(cr, la_d)
    only(out2, out, (rows0, 70), "out, up")
    only(dx2, dx, (rows0, every), "dx, up")
    only(dd2, dd, (0, 3), "d_down, up")
    assert torch.equal(la2, la) and torch.equal(du2, du)
    t.up_d[0, 70, 3] = keep
    keep = t.down_d[0, 5, 200].clone()
    t.down_d[0, 5, 200] = float("inf")             # enters rank 5 of lora_act and column 200 of dx
    out2, la2 = t.fwd(cr)
    dx2, dd2, du2 = t.bwd(cr, la_d)
    only(la2, la, (rows0, 5), "lora_act, down")
    assert torch.isinf(la2[:30, 5]).all()
    only(out2, out, (rows0, every), "out, down")
    only(dx2, dx, (rows0, 200), "dx, down")
    assert torch.equal(dd2, dd) and torch.equal(du2, du)
    t.down_d[0, 5, 200] = keep
    keep = t.dy_d[40, 9].clone()
    t.dy_d[40, 9] = float("-inf")                  # enters row 40 of dx and column 9 of adapter 1's d_up
    dx2, dd2, du2 = t.bwd(cr, la_d)
    only(dx2, dx, (40, every), "dx, dy")
    only(dd2, dd, (1, every), "d_down, dy")
    only(du2, du, (1, 9), "d_up, dy")
    t.dy_d[40, 9] = keep
    t.x_d[40, 11] = float("inf")                   # enters row 40 of lora_act and column 11 of adapter 1's d_down
    out2, la2 = t.fwd(cr)
    dx2, dd2, du2 = t.bwd(cr, la_d)
    only(la2, la, (40, every), "lora_act, x")
    assert torch.isinf(la2[40]).all()
    only(out2, out, (40, every), "out, x")
    only(dd2, dd, (1, every, 11), "d_down, x")
    assert torch.equal(dx2, dx) and torch.equal(du2, du)


def test_gated_slope_of_the_largest_values(cr):
    """silu' reaches 1.1: u silu'(g) beyond float32's largest value must not
    make dg infinite while dy u silu'(g) has a value."""
    g = np.repeat(np.float32([1.5, 2.375, 3.0, -1.25, 20.0, 0.5]), 64).reshape(6, 64)
    top = np.float32(3.3895313892515355e38)        # the largest bf16 value
    u = np.full((6, 64), top, np.float32)
    u[3:, ::2] = -top
    for dy in (2.0 ** -7, 0.5, -2.0 ** -60):
        z = torch.from_numpy(np.concatenate([g, u], 1)).to(torch.bfloat16).to(DEV)
        y, codes, scales = cr.convrot_act_checkpoint(z, cr.ACT.SWIGLU)
        dy_d = torch.full((6, 64), dy, dtype=torch.bfloat16, device=DEV)
        dz = host(cr.convrot_act_backward(dy_d, codes, scales, cr.ACT.SWIGLU).float()).astype(np.float64)
        kept = oa.restore_checkpoint(host(codes), host(scales))
        want = oa.act_backward(np.full((6, 64), dy), kept, "swiglu")
        assert np.isfinite(dz).all()
        # half a bf16 step, and the float32 roundings that test_gpu_act.py allows a slope
        k = np.concatenate([kept[:, :64], kept[:, :64]], 1)
        assert np.all(np.abs(dz - want) <= np.abs(want) * (2.0 ** -8 + 64 * 2.0 ** -24 * (1 + np.abs(k)) ** 2))


# Sizes that give every wave of the first product several stages of 64 columns, so that the slots of its
# rings are used again and the start column wraps, for each of its variants: waves a block, rows and ranks
# of a block, stages in flight. M, the sum's length, R, A, S
RINGS = [(300, 5000, 16, 2, 5), (800, 5000, 64, 2, 5),                     # 16 waves, 16 rows, 16 ranks, 2 stages
         (2000, 2056, 32, 2, 5), (5000, 2056, 32, 3, 70),                  # 8 waves, 32 ranks, 2 stages
         (4300, 2056, 16, 2, 5), (4500, 1544, 8, 2, 9),                    # 8 waves, 16 ranks, 3 stages of x and 2 of the weights
         (8300, 1608, 32, 2, 7), (8192, 2560, 24, 3, 5),                   # 5 waves, 32 rows, 32 ranks, 2 stages
         (2100, 2056, 64, 2, 5), (1300, 2056, 120, 3, 5),                  # 8 waves, 64 ranks, 1 stage
         (8300, 2056, 64, 2, 5), (4200, 1608, 120, 2, 9),                  # 6 waves, 32 rows, 64 ranks, 1 stage
         (48, 5000, 16, 2, 3), (130, 4104, 24, 2, 9)]                      # both products in one launch


@pytest.mark.parametrize("M,C,R,A,S", RINGS)
def test_long_rows_forward(cr, M, C, R, A, S):
    _forward(cr, (M, 72, C, R, A, S), False)


@pytest.mark.parametrize("M,C,R,A,S", RINGS)
def test_long_rows_backward(cr, M, C, R, A, S):
    """dla is the same product over dy; up to rank 16, and up to 32 with few rows, it reads up as it lies."""
    lora_tests.test_backward(cr, (M, C, 72, R, A, S, "ragged"), False)


def _forward(cr, shape, f32):
    say(f"lora forward {shape} f32={f32}")
    t = Case(*shape, seed=37)
    base_d, base = t.base(t.N, f32)
    want, la_want = oa.lora_forward(t.x, t.down, t.up, t.off, t.ids, t.c, base)
    out, la = t.fwd(cr, base=base_d, out_type=cr.OUT.F32 if f32 else cr.OUT.BF16)
    e1, e2 = t.two_products(t.x, t.down, t.up, base, want, f32)
    _near(la, la_want, e1, "lora_act")
    _near(out, want, e2, "out")


# the second product in tiles of 256 rows: ranks of one, two and four register steps
TALL = [(8200, 8200, 16, 2, 5), (8256, 7696, 64, 3, 9), (8300, 4104, 128, 2, 7)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,C,R,A,S", TALL)
def test_tall_tiles_forward(cr, M, C, R, A, S, f32):
    _forward(cr, (M, C, 72, R, A, S), f32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,C,R,A,S", TALL)
def test_tall_tiles_backward(cr, M, C, R, A, S, f32):
    lora_tests.test_backward(cr, (M, 72, C, R, A, S, "ragged"), f32)


def _bf16_values():
    v = bf16_to_f32(np.arange(1 << 16, dtype=np.uint32).astype(np.uint16))
    return np.sort(v[np.isfinite(v) & ((np.abs(v) > 3.9e-37) | (v == 0))])


@pytest.mark.parametrize("act", act_tests.ACTS)
def test_value_of_every_bf16_number(cr, act):
    """The bound of ordinary values holds for all: in the negative tail, down to
    float32's smallest normal value, the relative precision is kept, and beyond
    it the result is that close to the tiny one, never positive."""
    v = _bf16_values()
    v = np.concatenate([v, np.zeros(-len(v) % 128, np.float32)]).reshape(-1, 128)
    z = np.concatenate([v, np.ones_like(v)], 1) if act == "swiglu" else v
    y, _, _ = cr.convrot_act_checkpoint(bf16_dev(wl.bf16_bits_from_f32(z)), act_tests._act(cr, act))
    got, z64 = act_tests._f32(y), z.astype(np.float64)
    want = oa.act_value(z64, act)
    assert np.all(np.abs(got - want) <= act_tests._value_bound(z64, want, act))
    assert np.all(got[v < 0] <= 0) and np.all(got[v > 0] >= 0)


@pytest.mark.parametrize("act", act_tests.ACTS)
def test_slope_of_the_tails(cr, act):
    """Groups of one value each, so that the codes stand for it to a float32
    rounding, from 1/8 to 256 either way.

    GELU_TANH: p + z p q a (1 + 3 b z^2) with p = sigma(2 t): 2 t is off by four
    roundings, p by |2 t| times that and by four of its own, the second part by six
    more: 64 (1 + |2 t|) roundings of either part cover it. Below float32's normal
    values p keeps 2^-149, which the second part multiplies by less than 2^10
    before p is 0."""
    v = _bf16_values()
    v = v[(np.abs(v) >= 0.125) & (np.abs(v) <= 256)]
    z = np.repeat(v, 64).reshape(-1, 64)
    if act == "swiglu":
        z = np.concatenate([z, np.ones_like(z)], 1)
    _, codes, scales = cr.convrot_act_checkpoint(bf16_dev(wl.bf16_bits_from_f32(z)), act_tests._act(cr, act))
    kept = oa.restore_checkpoint(host(codes), host(scales))
    assert np.all(np.abs(kept - z) <= 2.0 ** -22 * np.abs(z))
    ones = np.ones((len(v), 64))
    got = act_tests._f32(cr.convrot_act_backward(dev(ones.astype(np.float32)).bfloat16(), codes, scales,
                                                 act_tests._act(cr, act)))
    want = oa.act_backward(ones, kept, act)
    if act == "gelu_tanh":
        a, b = 2 * np.sqrt(2 / np.pi), 0.044715
        t2 = a * (kept + b * kept ** 3)
        with np.errstate(over="ignore"):
            p, q = 1 / (1 + np.exp(-t2)), 1 / (1 + np.exp(t2))
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -126 + 64 * 2.0 ** -24 * (1 + np.abs(t2)) * (
            p + np.abs(kept) * p * q * a * (1 + 3 * b * kept * kept))
    else:
        bound = act_tests._slope_bound(ones, kept, want, act)
    assert np.all(np.abs(got - want) <= bound)


def test_misaligned_operands_are_named(cr):
    """Views that start between multiples of 16 bytes are refused, by name."""
    t = Case(20, 72, 64, 8, 2, 3, seed=38)
    la = torch.zeros((20, 8), device=DEV)
    shifted = lambda v: torch.cat([v.flatten()[:1], v.flatten()])[1:].view(v.shape)
    def refused(name, call):
        with pytest.raises(cr.ConvRotError, match=rf"\({name}: not at a multiple of 16 bytes\): invalid argument") as e:
            call()
        assert e.value.status == 1
    fwd = dict(x=t.x_d, down=t.down_d, up=t.up_d, seg_offsets=t.off_d, seg_adapter=t.ids_d, scale=t.c_d)
    for k in fwd:
        refused(k, lambda: cr.convrot_lora_forward(**{**fwd, k: shifted(fwd[k])}))
    bwd = dict(fwd, dy=t.dy_d, lora_act=la)
    for k in bwd:
        refused(k, lambda: cr.convrot_lora_backward(**{**bwd, k: shifted(bwd[k])}))
    z = t.dy_d[:, :64].contiguous()
    y, codes, scales = cr.convrot_act_checkpoint(z, cr.ACT.GELU)
    refused("z", lambda: cr.convrot_act_checkpoint(shifted(z), cr.ACT.GELU))
    back = dict(dy=y, codes=codes, scales=scales)
    for k in back:
        refused(k, lambda: cr.convrot_act_backward(**{**back, k: shifted(back[k])}, act=cr.ACT.GELU))
    refused("x, scale", lambda: cr.convrot_lora_forward(**{**fwd, "x": shifted(t.x_d), "scale": shifted(t.c_d)}))
    # what is not read is not named
    cr.convrot_lora_backward(**{**bwd, "x": shifted(t.x_d), "lora_act": shifted(la)}, want_weights=False)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,R,A,S", [(37, 72, 264, 16, 2, 5), (700, 136, 520, 40, 3, 9), (2100, 72, 4104, 24, 2, 7)])
def test_backward_in_place(cr, M, N, K, R, A, S, f32):
    """dx may be dx_base itself: the same bits, rows without adapter as they were."""
    t = Case(M, N, K, R, A, S, mix="gaps", seed=39)
    kind = cr.OUT.F32 if f32 else cr.OUT.BF16
    la = dev(t.g.standard_normal((M, R)).astype(np.float32))
    base = t.base(K, f32)[0]
    want = t.bwd(cr, la, dx_base=base, dx_type=kind)
    own = base.clone()
    got = t.bwd(cr, la, dx_base=own, dx=own, dx_type=kind)
    assert got[0] is own
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    none = dev(t.rows < 0)
    assert none.any() and torch.equal(own[none], base[none])


def _far(v, ld):
    """v in rows ld elements apart"""
    wide = torch.empty((v.shape[0], ld), dtype=v.dtype, device=DEV)
    wide[:, :v.shape[1]] = v
    return wide[:, :v.shape[1]]


def test_rows_beyond_32_bits(cr):
    """Rows up to 2^31 elements and more behind the first one: the bits of dense rows."""
    t = Case(1100, 264, 136, 24, 2, 5, seed=40)
    ld = 1 << 21                                   # the last row starts at 1.07 * 2^31 elements
    la = dev(t.g.standard_normal((t.M, t.R)).astype(np.float32))
    base, dx_base = t.base(t.N, False)[0], t.base(t.K, False, seed=2)[0]
    want, want_b = t.fwd(cr, base=base), t.bwd(cr, la, dx_base=dx_base)
    x, dy, y = t.x_d, t.dy_d, torch.empty((t.M, ld), dtype=torch.bfloat16, device=DEV)
    t.x_d, t.dy_d = _far(x, ld), _far(dy, ld)
    got = t.fwd(cr, base=_far(base, ld), out=y[:, :t.N])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    got = t.bwd(cr, la, dx_base=_far(dx_base, ld), dx=y[:, :t.K])
    for a, b in zip(got, want_b):
        assert torch.equal(a, b)
    for act in (cr.ACT.GELU, cr.ACT.SWIGLU):
        z, d = x[:, :128].contiguous(), dy[:, :64 if act == cr.ACT.SWIGLU else 128].contiguous()
        want = cr.convrot_act_checkpoint(z, act)
        got = cr.convrot_act_checkpoint(_far(z, ld), act, y=y[:, :d.shape[1]])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        dz = cr.convrot_act_backward(d, want[1], want[2], act)
        assert torch.equal(cr.convrot_act_backward(_far(d, ld), want[1], want[2], act, dz=y[:, :128]), dz)


def test_adapters_beyond_32_bits(cr):
    """down of 2^31 values and more: the last adapter's rows get its weights."""
    A, R, K, N, M = 4096, 128, 4104, 8, 70
    g = np.random.default_rng(41)
    put = lambda *shape: torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(DEV).bfloat16()
    x, d, u = put(M, K), put(2, R, K), put(2, N, R)
    off, one = dev(np.int32([0, 40, 70])), torch.zeros((A, N, R), dtype=torch.bfloat16, device=DEV)
    want = cr.convrot_lora_forward(x, d, u, off, dev(np.int32([1, 0])))
    down = torch.empty((A, R, K), dtype=torch.bfloat16, device=DEV)
    assert down.numel() > 2 ** 31
    down[A - 1], one[A - 1] = d[1], u[1]
    down[7], one[7] = d[0], u[0]
    got = cr.convrot_lora_forward(x, down, one, off, dev(np.int32([A - 1, 7])))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", ["gelu_tanh", "swiglu"])
def test_codes_beyond_32_bits(cr, act):
    """2^31 codes and more: the last rows are those of a call of their own."""
    rows, C = (530_000, 4096) if act == "gelu_tanh" else (270_000, 4096)
    kind = act_tests._act(cr, act)
    W = 2 * C if act == "swiglu" else C
    z = torch.empty((rows, W), dtype=torch.bfloat16, device=DEV).normal_()
    assert z.numel() > 2 ** 31
    y, codes, scales = cr.convrot_act_checkpoint(z, kind)
    last = slice(rows - 3, rows)
    for a, b in zip((y, codes, scales), cr.convrot_act_checkpoint(z[last], kind)):
        assert torch.equal(a[last], b)
    dz = cr.convrot_act_backward(y, codes, scales, kind)
    assert torch.equal(dz[last], cr.convrot_act_backward(y[last], codes[last], scales[last], kind))
