"""Ends of the ranges of the microscaled 4-bit linear, of layer norm and of the
optimizer step: every block shape of the product at ragged sizes, addresses
beyond 32 bits, calls side by side on several streams, memory freed while a call on
another stream still runs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import mx, training as tr  # noqa: E402
from tests.gpu_helpers import DEV, dev, say  # noqa: E402


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a8_rotated_quantized_amd as m
    assert m.device_check() == 0, "device is not gfx950"
    return m


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _operand(seed, rows, K):
    g = np.random.default_rng([seed, rows, K])
    codes, byte = g.integers(0, 16, (rows, K)).astype(np.uint8), (127 + g.integers(-3, 4, (rows, K // 32))).astype(np.uint8)
    c, b = mx.pack(codes, byte)
    return mx.values(codes, byte), dev(c), dev(b)


# one size for each block shape: few tokens by 16 and 8 waves, 64 x 64 alone, in four groups and many, 128 x 64,
# 128 x 128, 256 x 256; stages fewer than a ring, groups with unequal stages
SHAPES = [(3, 1000, 2080), (50, 4360, 416), (70, 200, 352), (70, 200, 2336), (90, 152, 2080), (65, 8, 4256), (513, 4096, 160), (1531, 2568, 96),
          (2049, 2056, 32), (3850, 4088, 416)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_block_shapes(cr, shape, out):
    M, N, K = shape
    say(f"mx block shapes {shape} {out}")
    a, ac, ab = _operand(1, M, K)
    w, wc, wb = _operand(2, N, K)
    bias = torch.randn(N, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(torch.bfloat16)
    want, mag = mx.gemm(a, w, bias.double().cpu().numpy())
    hold = torch.full((M, N + 8), -5.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device=DEV)
    y = cr.mxfp4_gemm(ac, ab, wc, wb, bias=bias, out_type=cr.OUT.BF16 if out == "bf16" else cr.OUT.F32, out=hold[:, :N])
    half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    # exact products, K + 1 float32 sums that may cut (2^-23 each), one rounding
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -23 * (K + 2) * mag + half * (1 + 2.0 ** -8) * np.abs(want))
    assert bool((hold[:, N:] == -5).all())


def test_rows_of_a_product_do_not_depend_on_others(cr):
    """The same block shape: a row's result is the same whatever lies in the others."""
    _, ac, ab = _operand(3, 300, 512)
    _, wc, wb = _operand(4, 520, 512)
    y = cr.mxfp4_gemm(ac, ab, wc, wb)
    ac2, ab2 = ac.clone(), ab.clone()
    ac2[:, 100:] = 0x77
    ab2[:, 200:] = 255
    z = cr.mxfp4_gemm(ac2, ab2, wc, wb)
    assert torch.equal(y[:100], z[:100]) and bool(torch.isnan(z[200:]).all())


def test_codes_beyond_32_bits(cr):
    """33.5 million rows: 4.3 GB of codes, the second tile from 2^31 on, 17 GB of values."""
    rows, K, period = (1 << 25) + 5, 256, 4099
    say("mx codes beyond 32 bits")
    base = torch.randn((period, K), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    x = base.repeat(-(-rows // period), 1)[:rows]
    codes, scales = cr.mxfp4_quantize(x, 256)
    want = cr.mxfp4_quantize(base, 256)
    at = torch.cat([torch.arange(0, 50), torch.arange((1 << 24) - 30, (1 << 24) + 30), torch.arange(rows - 70, rows)]).to(DEV)
    assert torch.equal(codes[:, at], want[0][:, at % period]) and torch.equal(scales[:, at], want[1][:, at % period])
    del x
    back = cr.mxfp4_dequantize(codes, scales, K, 256)
    assert torch.equal(back[at], cr.mxfp4_dequantize(*want, K, 256)[at % period])
    del back
    w = cr.mxfp4_quantize(torch.randn((72, K), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(torch.bfloat16), 256)
    y = cr.mxfp4_gemm(codes, scales, *w, out_type=cr.OUT.F32)          # 9.7 GB
    near = cr.mxfp4_gemm(*want, *w, out_type=cr.OUT.F32)
    # two block shapes may sum in two orders: 256 exact products, each sum off by at most 2^-23
    mag = torch.linalg.vector_norm(cr.mxfp4_dequantize(*want, K, out_type=cr.OUT.F32), dim=1)[at % period, None] * torch.linalg.vector_norm(
        cr.mxfp4_dequantize(*w, K, out_type=cr.OUT.F32), dim=1)
    assert bool(((y[at] - near[at % period]).abs() <= 2 * 2.0 ** -23 * 258 * mag).all())


def test_norm_beyond_32_bits(cr):
    """1.1 million rows of 4096: 9 GB a tensor."""
    rows, C, period = 1100003, 4096, 2003
    say("norm beyond 32 bits")
    g = torch.Generator(device=DEV).manual_seed(3)
    bx, bdy = torch.randn((period, C), generator=g, device=DEV).to(torch.bfloat16), torch.randn((period, C), generator=g, device=DEV).to(torch.bfloat16)
    w, b = torch.randn((2, C), generator=g, device=DEV), torch.randn((2, C), generator=g, device=DEV)
    cut = 600000
    off = torch.tensor([0, cut, rows], dtype=torch.int32, device=DEV)
    n = -(-rows // period)
    x, dy = bx.repeat(n, 1)[:rows], bdy.repeat(n, 1)[:rows]
    y, mean, rstd = cr.convrot_layer_norm_forward(x, w, b, seg_offsets=off)
    dx, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, w, seg_offsets=off)
    at = torch.cat([torch.arange(0, 40), torch.arange((1 << 19) - 20, (1 << 19) + 20), torch.arange(rows - 60, rows)]).to(DEV)
    for s, rows_of in ((0, at[at < cut]), (1, at[at >= cut])):
        y2, m2, r2 = cr.convrot_layer_norm_forward(bx, w[s].contiguous(), b[s].contiguous())
        dx2, _, _ = cr.convrot_layer_norm_backward(bdy, bx, m2, r2, w[s].contiguous(), want_weights=False)
        # float32 sums in the order of another variant: within a step of bf16
        for p, q in ((y, y2), (dx, dx2)):
            p, q = p[rows_of].double(), q[rows_of % period].double()
            assert bool(((p - q).abs() <= 2.0 ** -7 * q.abs() + 2.0 ** -16 * q.abs().amax(1, keepdim=True)).all())
    xh = (bx.double() - bx.double().mean(1, keepdim=True)) * (bx.double().var(1, unbiased=False, keepdim=True) + 1e-6).rsqrt()
    count = torch.zeros((2, period), dtype=torch.float64, device=DEV)
    for s, (lo, hi) in enumerate(((0, cut), (cut, rows))):
        count[s] = torch.bincount(torch.arange(lo, hi, device=DEV) % period, minlength=period).double()
        for got, terms in ((dw, bdy.double() * xh), (db, bdy.double())):
            want, mag = (count[s][:, None] * terms).sum(0), (count[s][:, None] * terms.abs()).sum(0)
            # at most (rows of a part + parts) float32 sums on the way, each 2^-24 of the magnitudes
            assert bool(((got[s].double() - want).abs() <= 2.0 ** -24 * (rows / 768 + 768) * 2 * mag).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_the_largest_tensor(cr, bits):
    """2^31 - 1 elements beside a small tensor: the ends of both against small calls."""
    n, tail = (1 << 31) - 1, 2303
    say(f"adamw {n} elements, {bits} bits")
    g = torch.Generator(device=DEV).manual_seed(4)
    grad = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    ends = torch.randn((2, tail), generator=g, device=DEV).to(torch.bfloat16)
    start = n - tail
    assert start % 256 == 0
    grad[:tail], grad[start:] = ends[0], ends[1]
    p = torch.zeros(n, device=DEV)
    small = [torch.ones(70, device=DEV), torch.ones(70, dtype=torch.bfloat16, device=DEV)]
    kind = (lambda k: torch.zeros(k, device=DEV)) if bits == 32 else None
    if bits == 8:
        state = [[torch.zeros(k, dtype=d, device=DEV) for k in (70, n)] for d in (torch.int8, torch.uint8)]
        extra = dict(exp_avg_scales=[torch.zeros(-(-k // 256), device=DEV) for k in (70, n)],
                     exp_avg_sq_scales=[torch.zeros(-(-k // 256), device=DEV) for k in (70, n)], seed=11)
    else:
        state, extra = [[kind(k) for k in (70, n)] for _ in range(2)], {}
    cr.convrot_adamw_step([small[0], p], [small[1], grad], *state, step=1, lr=0.125, weight_decay=0.0, **extra)
    assert not bool(p[tail:start:65537].any())
    for at, e in ((0, 0), (start, 1)):
        q, m, v = torch.zeros(tail, device=DEV), torch.zeros(tail, device=DEV), torch.zeros(tail, device=DEV)
        cr.convrot_adamw_step([q], [ends[e].clone()], [m], [v], step=1, lr=0.125, weight_decay=0.0)
        assert torch.equal(p[at:at + tail], q)
        if bits == 32:
            assert torch.equal(state[0][1][at:at + tail], m) and torch.equal(state[1][1][at:at + tail], v)
        else:
            key = tr._mix(np.array((11 + 0x9E3779B9 * 2) & 0xFFFFFFFF, np.uint32))
            h = tr._mix(tr._mix(np.arange(at, at + tail, dtype=np.uint64).astype(np.uint32)) ^ key)
            um, uv = (h & np.uint32(0xFFFF)).astype(np.float32) / np.float32(65536), (h >> np.uint32(16)).astype(np.float32) / np.float32(65536)
            f = np.float32
            ge = ends[e].float().cpu().numpy()
            mc, ms = tr.encode(ge * f(1 - 0.9), um, 127)
            vc, vs = tr.encode(np.sqrt((ge * ge) * f(1 - 0.999)), uv, 255)
            for got, want in ((state[0][1][at:at + tail], mc), (state[1][1][at:at + tail], vc),
                              (extra["exp_avg_scales"][1][at // 256:at // 256 + len(ms)], ms),
                              (extra["exp_avg_sq_scales"][1][at // 256:at // 256 + len(vs)], vs)):
                assert np.array_equal(got.cpu().numpy(), want)


def test_refused_addresses_are_named(cr):
    flat = torch.zeros(64, device=DEV)
    ok, off = flat[:16], flat[17:33]
    with pytest.raises(cr.ConvRotError, match="grads: not at a multiple of 16 bytes"):
        cr.convrot_adamw_step([ok], [off], [flat[32:48]], [flat[48:]], step=1, lr=1e-3)
    x = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device=DEV)[1:257].view(4, 64)
    with pytest.raises(cr.ConvRotError, match="x: not at a multiple of 16 bytes"):
        cr.mxfp4_quantize(x)
    with pytest.raises(cr.ConvRotError, match="x: not at a multiple of 16 bytes"):
        cr.convrot_layer_norm_forward(x)
    wide = torch.zeros((4, 68), dtype=torch.bfloat16, device=DEV)
    for call in (lambda: cr.mxfp4_quantize(wide[:, :64]), lambda: cr.convrot_layer_norm_forward(wide[:, :64])):
        with pytest.raises(cr.ConvRotError):                 # rows 68 apart
            call()


def test_calls_side_by_side(cr):
    """Four streams at once, each with its own chain of calls: the results of one after the other."""
    g = torch.Generator(device=DEV).manual_seed(6)
    M, C, N = 700, 2560, 1536
    xs = [torch.randn((M, C), generator=g, device=DEV).to(torch.bfloat16) for _ in range(4)]
    w = cr.mxfp4_quantize((torch.randn((N, C), generator=g, device=DEV) * 0.02).to(torch.bfloat16), 256)
    weight, bias = torch.randn(C, generator=g, device=DEV), torch.randn(C, generator=g, device=DEV)

    def chain(x, stream):
        h, mean, rstd = cr.convrot_layer_norm_forward(x, weight, bias, stream=stream)
        y = cr.mxfp4_gemm(*cr.mxfp4_quantize(h, 256, stream=stream), *w, out_type=cr.OUT.F32, stream=stream)
        dx, dw, db = cr.convrot_layer_norm_backward(h, x, mean, rstd, weight, stream=stream)
        p, m, v = dw.clone() if stream is None else dw, torch.zeros(C, device=DEV), torch.zeros(C, device=DEV)
        return h, y, dx, dw, db, p, m, v

    want = [[t.clone() for t in chain(x, None)] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [chain(x, s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a[:5], b[:5]))


def test_memory_freed_under_a_call(cr):
    """Inputs, workspaces and outputs of a call on a given stream, dropped at once: their memory is not given out before it has ended."""
    g = torch.Generator(device=DEV).manual_seed(7)
    x = torch.randn((6000, 4096), generator=g, device=DEV).to(torch.bfloat16)
    w = cr.mxfp4_quantize(torch.randn((2048, 4096), generator=g, device=DEV).to(torch.bfloat16), 256)
    want = cr.mxfp4_gemm(*cr.mxfp4_quantize(x, 256), *w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        y = x.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        codes = cr.mxfp4_quantize(y, 256, stream=side)
        out = cr.mxfp4_gemm(*codes, *w, stream=side)
        del y, codes
        junk = [torch.full((6000, 4096), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        junk += [torch.full((32, 6000, 64), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
        side.synchronize()
        assert torch.equal(out, want)
        del junk


def _spread(rows):
    return torch.cat([torch.arange(0, 70), torch.arange(rows // 2 - 35, rows // 2 + 35), torch.arange(rows - 70, rows)]).to(DEV)


def test_more_blocks_than_a_grid_row(cr):
    """Beyond 2^20 blocks the grid goes on along its second axis: rows at its ends and in
    the middle are those of a call on them alone, and nothing behind the last is written."""
    rows = (1 << 26) - 1
    g = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn(rows, 8, generator=g, device=DEV, dtype=torch.bfloat16)
    at = _spread(rows)
    out = torch.full((rows + 3, 8), 7.0, device=DEV, dtype=torch.bfloat16)
    mean, rstd = torch.full((rows + 3,), 7.0, device=DEV), torch.full((rows + 3,), 7.0, device=DEV)
    cr.convrot_layer_norm_forward(x, out=out[:rows], mean=mean[:rows], rstd=rstd[:rows])
    y, m, r = cr.convrot_layer_norm_forward(x[at])
    assert torch.equal(out[at], y) and torch.equal(mean[at], m) and torch.equal(rstd[at], r)
    assert bool((out[rows:] == 7).all()) and bool((mean[rows:] == 7).all()) and bool((rstd[rows:] == 7).all())
    del x, out, mean, rstd
    rows = (1 << 21) + 3                                # a row a block
    x = torch.randn(rows, 1032, generator=g, device=DEV, dtype=torch.bfloat16)
    at = _spread(rows)
    y, m, r = cr.convrot_layer_norm_forward(x)
    small = cr.convrot_layer_norm_forward(x[torch.cat([at] * 6)])   # more than 1024 rows: the same shape of block
    assert torch.equal(y[at], small[0][:at.numel()]) and torch.equal(r[at], small[2][:at.numel()])
    del x, y
    rows = (1 << 24) + 5
    x = torch.randn(rows, 64, generator=g, device=DEV, dtype=torch.bfloat16)
    at = _spread(rows)
    for rot in (0, 64):
        codes, scales = cr.mxfp4_quantize(x, rot)
        some = cr.mxfp4_quantize(x[at], rot)
        assert torch.equal(codes[:, at], some[0]) and torch.equal(scales[:, at], some[1])
        back = cr.mxfp4_dequantize(codes, scales, 64, rot)
        assert torch.equal(back[at], cr.mxfp4_dequantize(*some, 64, rot))


def test_adamw_longest_tensor(cr):
    """A tensor of nearly 2^31 elements fills a launch: the next one takes another."""
    sizes = [(1 << 31) - 8, 5001, 1 << 20]
    some = [torch.cat([torch.arange(0, 9), torch.arange(n // 2 - 4, n // 2 + 5), torch.arange(n - 9, n)]).to(DEV) for n in sizes]
    g = torch.Generator(device=DEV).manual_seed(12)
    lists = []
    for kind in range(4):                               # parameters, gradients, both moments: zeros but for some
        lists.append([])
        for n, at in zip(sizes, some):
            t = torch.zeros(n, device=DEV, dtype=torch.bfloat16 if kind == 1 else torch.float32)
            t[at] = torch.rand(at.numel(), generator=g, device=DEV).to(t.dtype)
            lists[-1].append(t)
    few = [[t[at].clone() for t, at in zip(l, some)] for l in lists]
    kw = dict(step=3, lr=0.01, weight_decay=0.1)
    cr.convrot_adamw_step(*lists, **kw)
    cr.convrot_adamw_step(*few, **kw)
    for l, f in zip(lists, few):
        for t, at, want in zip(l, some, f):
            assert torch.equal(t[at], want)
            t[at] = 0
            assert t.count_nonzero() == 0


# 256 x 256 blocks with more stages than their ring of four has places: 10, 12 and 21 of them, ragged at every end
LARGE = [(3850, 4088, 1184), (3850, 4088, 1536), (1531, 9208, 2592)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("shape", LARGE)
def test_large_blocks_past_their_ring(cr, shape, out):
    M, N, K = shape
    say(f"mx large blocks {shape} {out}")
    a, ac, ab = _operand(1, M, K)
    w, wc, wb = _operand(2, N, K)
    bias = torch.randn(N, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(torch.bfloat16)
    want, mag = mx.gemm(a, w, bias.double().cpu().numpy())
    hold = torch.full((M + 1, N + 8), -5.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device=DEV)
    y = cr.mxfp4_gemm(ac, ab, wc, wb, bias=bias, out_type=cr.OUT.BF16 if out == "bf16" else cr.OUT.F32, out=hold[:M, :N])
    half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    # exact products, K + 1 float32 sums that may cut (2^-23 each), one rounding
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -23 * (K + 2) * mag + half * (1 + 2.0 ** -8) * np.abs(want))
    assert bool((hold[:, N:] == -5).all()) and bool((hold[M] == -5).all())


@pytest.mark.parametrize("shape", LARGE)
def test_large_blocks_exact(cr, shape):
    """Unit powers: products are quarters of whole numbers up to 144, so their sums stay below 2^24 quarters and are exact."""
    M, N, K = shape
    g = np.random.default_rng([9, M, N, K])
    one = np.full((1, K // 32), 127, np.uint8)
    ca, cw = (g.integers(0, 16, (rows, K)).astype(np.uint8) for rows in (M, N))
    (pa, ba), (pw, bw) = (mx.pack(c, np.repeat(one, len(c), 0)) for c in (ca, cw))
    # whole numbers: the float32 product of values times two is exact too
    two = [torch.from_numpy(2 * mx.values(c, np.repeat(one, len(c), 0))).float().to(DEV) for c in (ca, cw)]
    want = (two[0].double() @ two[1].double().T) / 4
    for _ in range(3):
        assert torch.equal(cr.mxfp4_gemm(dev(pa), dev(ba), dev(pw), dev(bw), out_type=cr.OUT.F32).double(), want)


def test_sizes_take_the_blocks_that_they_test(cr):
    """The kernel that each size of this file runs: a change of the rule that drops one from the tests shows here."""
    few = {(3, 1000, 2080): "mx_few_kernel<1, 16,", (50, 4360, 416): "mx_few_kernel<4, 8,"}
    small = {(70, 200, 352): "64, 64, 1, 1, 4, 4, 1,", (70, 200, 2336): "64, 64, 1, 1, 4, 1, 4,", (90, 152, 2080): "64, 64, 1, 1, 4, 1, 4,",
             (65, 8, 4256): "64, 64, 1, 1, 4, 1, 4,", (513, 4096, 160): "64, 64, 1, 1, 4, 4, 1,", (1531, 2568, 96): "128, 64, 2, 1,",
             (2049, 2056, 32): "128, 128, 2, 2,", (3850, 4088, 416): "256, 256, 4, 2,"}
    want = {**few, **{s: f"mx_gemm_kernel<{t}" for s, t in small.items()}, **{s: "mx_gemm_kernel<256, 256, 4, 2," for s in LARGE}}
    assert set(SHAPES) | set(LARGE) == set(want)
    torch.cuda.synchronize()
    from torch.profiler import ProfilerActivity, profile
    for (M, N, K), name in want.items():
        a, w = ((torch.zeros((-(-K // 128), r, 64), dtype=torch.uint8, device=DEV), torch.zeros((-(-K // 128), r, 4), dtype=torch.uint8, device=DEV))
                for r in (M, N))
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA], acc_events=True) as trace:
            cr.mxfp4_gemm(*a, *w)
            torch.cuda.synchronize()
        ran = [e.name for e in trace.events() if "mx_" in e.name]
        if not ran:
            pytest.skip("no kernel trace on this host")
        assert len(ran) == 1 and name in ran[0], ((M, N, K), ran)


@pytest.mark.parametrize("C", [2568, 4104, 8200])
def test_more_rows_of_a_block_each_than_a_grid_row(cr, C):
    """Three, four and eight waves a row, a row a block: beyond 2^20 rows the grid goes on along its second axis, whose surplus
    blocks write nothing. The block's shape depends on the columns alone here, so rows equal those of a call on them alone."""
    rows = (1 << 20) + 3
    say(f"norm {rows} rows of {C}")
    g = torch.Generator(device=DEV).manual_seed(C)
    x = torch.randn(rows, C, generator=g, device=DEV, dtype=torch.bfloat16)
    w, b = torch.randn((2, C), generator=g, device=DEV), torch.randn((2, C), generator=g, device=DEV)
    cut = rows // 2
    off = torch.tensor([0, cut, rows], dtype=torch.int32, device=DEV)
    out = torch.full((rows + 3, C), 7.0, device=DEV, dtype=torch.bfloat16)
    mean, rstd = torch.full((rows + 3,), 7.0, device=DEV), torch.full((rows + 3,), 7.0, device=DEV)
    cr.convrot_layer_norm_forward(x, w, b, seg_offsets=off, out=out[:rows], mean=mean[:rows], rstd=rstd[:rows])
    at = torch.cat([_spread(rows), torch.arange((1 << 20) - 40, rows, device=DEV)]).unique()
    some = torch.tensor([0, int((at < cut).sum()), at.numel()], dtype=torch.int32, device=DEV)
    y, m, r = cr.convrot_layer_norm_forward(x[at], w, b, seg_offsets=some)
    assert torch.equal(out[at], y) and torch.equal(mean[at], m) and torch.equal(rstd[at], r)
    assert bool((out[rows:] == 7).all()) and bool((mean[rows:] == 7).all()) and bool((rstd[rows:] == 7).all())
    for lo in range(0, rows, 1 << 17):                   # every row is normalised: mean 0, variance 1 before weight and bias
        hi = min(rows, lo + (1 << 17))
        t = x[lo:hi].float()
        assert bool(((mean[lo:hi] - t.mean(1)).abs() < 1e-5).all()) and bool(((rstd[lo:hi] * t.std(1, unbiased=False) - 1).abs() < 1e-4).all())


@pytest.mark.parametrize("C", [512, 520, 2048, 4096, 8192])
def test_sums_of_many_rows(cr, C):
    """d_weight and d_bias of terms of one sign, the hardest for a sum: off by at most 2^-24 of the magnitudes for each sum on
    a term's way. Those are the rows of a part that one group of the block takes, the groups, and the parts."""
    rows = 60001
    groups = 8 if C <= 512 else 4 if C <= 1536 else 3 if C <= 2048 else 2 if C <= 4096 else 1
    parts = 512 if C <= 512 else 256
    part = -(-(-(-rows // parts)) // groups) * groups
    g = torch.Generator(device=DEV).manual_seed(C)
    x = torch.rand((rows, C), generator=g, device=DEV).to(torch.bfloat16)
    dy = (torch.rand((rows, C), generator=g, device=DEV) + 0.5).to(torch.bfloat16)
    mean, rstd = torch.full((rows,), -1.0, device=DEV), torch.full((rows,), 1.0, device=DEV)      # xh = x + 1: above 0
    _, dw, db = cr.convrot_layer_norm_backward(dy, x, mean, rstd, want_dx=False)
    xh = x.double() + 1
    sums = part // groups + groups + min(-(-rows // part), parts)
    for got, want, own in ((db, dy.double().sum(0), 0), (dw, (dy.double() * xh).sum(0), 2)):     # x - mean and its product: rounded
        assert bool(((got.double() - want).abs() <= (sums + own) * 2.0 ** -24 * want).all())


def test_steps_side_by_side(cr):
    """Four streams at once, each reading codes back and stepping two optimizers with them: the results of one after the other."""
    g = torch.Generator(device=DEV).manual_seed(8)
    rows, K = 520, 1056
    codes = [cr.mxfp4_quantize(torch.randn((rows, K), generator=g, device=DEV).to(torch.bfloat16)) for _ in range(4)]
    n = rows * K

    def state():
        return ([torch.ones(n, device=DEV)], [torch.zeros(n, device=DEV)], [torch.zeros(n, device=DEV)],
                [torch.ones(n, device=DEV)], [torch.zeros(n, dtype=torch.int8, device=DEV)], [torch.zeros(n, dtype=torch.uint8, device=DEV)],
                [torch.zeros(-(-n // 256), device=DEV)], [torch.zeros(-(-n // 256), device=DEV)])

    def chain(c, s, stream):
        for step in range(1, 6):
            grad = cr.mxfp4_dequantize(*c, K, out_type=cr.OUT.F32, stream=stream)
            cr.convrot_adamw_step(s[0], [grad], s[1], s[2], step=step, lr=1e-2, stream=stream)
            cr.convrot_adamw_step(s[3], [grad], s[4], s[5], step=step, lr=1e-2, exp_avg_scales=s[6], exp_avg_sq_scales=s[7], seed=step,
                                  stream=stream)

    want = [state() for _ in codes]
    for c, s in zip(codes, want):
        chain(c, s, None)
    assert not torch.equal(want[0][0][0], want[1][0][0]) and bool(want[0][4][0].any())
    streams = [torch.cuda.Stream() for _ in codes]
    for _ in range(3):
        got = [state() for _ in codes]
        torch.cuda.synchronize()
        for c, s, q in zip(codes, got, streams):
            chain(c, s, q)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p[0], q[0]) for p, q in zip(a, b))
