"""GPU parity of the AdamW step against the oracle.

float32 moments, u = 2^-24: a constant rounded, two products and a sum, so m is off by at
most 4 u (|b1 m| + |c1 g|) (and v by 5 u of itself, its terms being positive); p by 3 u |p|,
what m's error makes of the update, and 20 u of the update (root, two products,
sum, quotient, product, and half of v's 5 u).
8-bit moments: codes and scales are float32 operations rounded once, so they are equal
bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import training as tr  # noqa: E402
from tests.gpu_helpers import DEV, dev, say  # noqa: E402

U = 2.0 ** -24
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.995, eps=1e-8, weight_decay=0.02)


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a8_rotated_quantized_amd as m
    assert m.device_check() == 0, "device is not gfx950"
    return m


def _np(t):
    return t.float().cpu().numpy()


def _grad(g, n, grad):
    t = dev((g.standard_normal(n) * np.exp2(g.uniform(-12, 0, n))).astype(np.float32))
    return t.to(torch.bfloat16) if grad == "bf16" else t


def _check_p(got, p, g, m, v, step, want):
    m64, v64 = (np.asarray(t, np.float64) for t in (m, v))
    h = HYPER
    root = np.sqrt((h["beta2"] * v64 + (1 - h["beta2"]) * g ** 2) / (1 - h["beta2"] ** step)) + h["eps"]
    rate = h["lr"] / (1 - h["beta1"] ** step)
    dm = 4 * U * (h["beta1"] * np.abs(m64) + (1 - h["beta1"]) * np.abs(g))
    update = np.abs(want - np.asarray(p, np.float64) * (1 - h["lr"] * h["weight_decay"]))
    bound = 3 * U * np.abs(p) + 20 * U * update + rate * dm / root + U * np.abs(want)
    assert np.all(np.abs(got - want) <= bound), (np.abs(got - want) / bound).max()


SIZES = [1, 3, 0, 255, 256, 257, 1023, 1024, 1025, 2047, 2048, 2049, 5000, 40961]


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("repeat", [1, 9])
def test_float_moments(cr, grad, repeat):
    """Sizes around every border; with 9 repeats more tensors than one launch takes."""
    sizes = SIZES * repeat
    say(f"adamw 32 {grad} {len(sizes)} tensors")
    g = np.random.default_rng([repeat, len(grad)])
    p0 = [(g.standard_normal(n)).astype(np.float32) for n in sizes]
    P = [dev(p) for p in p0]
    G = [_grad(g, n, grad) for n in sizes]
    M, V = [torch.zeros(n, device=DEV) for n in sizes], [torch.zeros(n, device=DEV) for n in sizes]
    copies = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for n in sizes]
    clip = torch.tensor([0.37], device=DEV)
    for step in (1, 2, 3):
        before = [(_np(p), _np(m), _np(v)) for p, m, v in zip(P, M, V)]
        cr.convrot_adamw_step(P, G, M, V, step=step, copies=copies, grad_scale=clip, **HYPER)
        for i, n in enumerate(sizes):
            p, m, v = before[i]
            g64 = (_np(G[i]) * np.float32(0.37)).astype(np.float64)
            wp, wm, wv = tr.adamw(p, g64, m, v, step, HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], HYPER["weight_decay"])
            gm, gv = _np(M[i]).astype(np.float64), _np(V[i]).astype(np.float64)
            assert np.all(np.abs(gm - wm) <= 4 * U * (0.9 * np.abs(m) + 0.1 * np.abs(g64)) + 1e-44)
            assert np.all(np.abs(gv - wv) <= 6 * U * wv + 1e-44)
            _check_p(_np(P[i]).astype(np.float64), p, g64, m, v, step, wp)
            assert torch.equal(copies[i], P[i].to(torch.bfloat16))


def _codes(n):
    b = -(-n // 256)
    return (torch.zeros(n, dtype=torch.int8, device=DEV), torch.zeros(n, dtype=torch.uint8, device=DEV),
            torch.zeros(b, device=DEV), torch.zeros(b, device=DEV))


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("repeat", [1, 5, 7])
def test_moments_in_8_bits(cr, grad, repeat):
    sizes = SIZES * repeat
    say(f"adamw 8 {grad} {len(sizes)} tensors")
    g = np.random.default_rng([7, repeat, len(grad)])
    P = [dev(g.standard_normal(n).astype(np.float32)) for n in sizes]
    M, V, MS, VS = (list(t) for t in zip(*[_codes(n) for n in sizes]))
    h = HYPER
    for step, seed in ((1, 5), (2, 0xFFFFFFFF), (3, 77), (4, 1 << 31)):
        G = [_grad(g, n, grad) for n in sizes]
        if step == 3:
            for t in G:
                t[::7] = 0
        before = [tuple(t.cpu().numpy() for t in e) for e in zip(P, M, MS, V, VS)]
        cr.convrot_adamw_step(P, G, M, V, step=step, exp_avg_scales=MS, exp_avg_sq_scales=VS, seed=seed, **h)
        read = cr.convrot_adamw_moments(M, V, MS, VS)
        at = 0
        for i, n in enumerate(sizes):
            p, mc, ms, vc, vs = before[i]
            want = tr.adamw8(p, _np(G[i]), mc, ms, vc, vs, step, h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"], seed, i)
            for got, exact, what in zip((M[i], MS[i], V[i], VS[i]), want[1:], ("m", "m scales", "v", "v scales")):
                assert np.array_equal(got.cpu().numpy(), exact), (what, n, step)
            m, r = tr.decode(mc, ms, 127), tr.decode(vc, vs, 255)
            _check_p(_np(P[i]).astype(np.float64), p, _np(G[i]).astype(np.float64), m, r * r, step, want[0])
            r = tr.decode(want[3], want[4], 255)
            assert np.array_equal(read[0][at:at + n].cpu().numpy(), tr.decode(want[1], want[2], 127))
            assert np.array_equal(read[1][at:at + n].cpu().numpy(), r * r)
            at += n


def test_a_root_keeps_a_code(cr):
    """After one large gradient, small ones do not meet a second moment of zero."""
    n = 1024
    P, (m, v, ms, vs) = [torch.zeros(n, device=DEV)], _codes(n)
    for step in range(1, 30):
        grad = torch.full((n,), 1e-4, device=DEV)
        grad[::256] = 1e3 if step == 1 else 0.0
        before = P[0].clone()
        cr.convrot_adamw_step(P, [grad], [m], [v], step=step, exp_avg_scales=[ms], exp_avg_sq_scales=[vs], seed=step, lr=1e-3,
                              weight_decay=0.0)
        # |m| / sqrt(v) of any history of gradients is at most (1 - b1) / sqrt(1 - b2) over sqrt-corrected rates;
        # a code one step up on m and sqrt(v) held at s / 65025 multiply it by less than 16
        assert float((P[0] - before).abs().max()) < 1e-3 * 60


def test_not_finite(cr):
    n = 1000
    for bits in (8, 32):
        P = [torch.ones(n, device=DEV)]
        G = [torch.ones(n, device=DEV)]
        G[0][300], G[0][700] = float("inf"), float("nan")
        if bits == 8:
            m, v, ms, vs = _codes(n)
            cr.convrot_adamw_step(P, G, [m], [v], step=1, lr=0.1, exp_avg_scales=[ms], exp_avg_sq_scales=[vs])
            assert torch.isnan(ms).tolist() == [False, True, True, False] and torch.isnan(vs).tolist() == [False, True, True, False]
        else:
            cr.convrot_adamw_step(P, G, [torch.zeros(n, device=DEV)], [torch.zeros(n, device=DEV)], step=1, lr=0.1)
        bad = torch.isnan(P[0])
        assert bad.nonzero().flatten().tolist() == [300, 700]


def test_stream_graph_and_untouched_neighbours(cr):
    """Slices of one buffer: neighbours stay; a captured step replayed equals eager steps with its constants."""
    n = 777
    for bits in (8, 32):
        flat = torch.full((3, 800), 5.0, device=DEV)
        P = [flat[i, :n] for i in range(3)]
        G = [torch.randn(n, device=DEV, generator=torch.Generator(device=DEV).manual_seed(i)) for i in range(3)]
        if bits == 8:
            M, V, MS, VS = (list(t) for t in zip(*[_codes(n) for _ in range(3)]))
            extra = dict(exp_avg_scales=MS, exp_avg_sq_scales=VS, seed=3)
            state = [*P, *M, *V, *MS, *VS]
        else:
            M, V = [torch.zeros(n, device=DEV) for _ in range(3)], [torch.zeros(n, device=DEV) for _ in range(3)]
            extra = {}
            state = [*P, *M, *V]
        start = [t.clone() for t in state]
        eager = []
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            cr.convrot_adamw_step(P, G, M, V, step=4, lr=0.01, stream=side, **extra)
            side.synchronize()
            eager.append([t.clone() for t in state])
        assert bool((flat[:, n:] == 5.0).all())
        for t, s in zip(state, start):
            t.copy_(s)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            cr.convrot_adamw_step(P, G, M, V, step=4, lr=0.01, **extra)
        for want in eager:
            graph.replay()
            torch.cuda.synchronize()
            for t, e in zip(state, want):
                assert torch.equal(t, e)
            torch.randn(100, device=DEV).sum().item()


def test_trains_without_sticking(cr):
    """A quadratic's gradient: 8-bit moments follow float32 ones within the size of their codes' steps."""
    n = 4096
    g = torch.Generator(device=DEV).manual_seed(4)
    target = torch.randn(n, device=DEV, generator=g)
    a, b = [torch.zeros(n, device=DEV)], [torch.zeros(n, device=DEV)]
    M, V = [torch.zeros(n, device=DEV)], [torch.zeros(n, device=DEV)]
    m, v, ms, vs = _codes(n)
    for step in range(1, 101):
        noise = torch.randn(n, device=DEV, generator=g)
        cr.convrot_adamw_step(a, [a[0] - target + noise], M, V, step=step, lr=1e-2)
        cr.convrot_adamw_step(b, [b[0] - target + noise], [m], [v], step=step, lr=1e-2, exp_avg_scales=[ms], exp_avg_sq_scales=[vs], seed=step)
    assert torch.isfinite(b[0]).all()
    m8, v8 = cr.convrot_adamw_moments([m], [v], [ms], [vs])
    # rounding up and down by turns: the moments are those of the float32 run on average
    assert abs(float(v8.mean() / V[0].mean()) - 1) < 0.05


@pytest.mark.parametrize("given", [False, True])
def test_a_backward_pass_behind_the_step_is_refused(cr, given):
    """What a graph of before the step needs of the parameters and their copies is gone: autograd says so."""
    stream = torch.cuda.Stream() if given else None
    p = torch.ones(64, device=DEV, requires_grad=True)
    copy = torch.ones(64, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    late, late_copy = (p * p).sum(), (copy * copy).sum()
    early, = torch.autograd.grad((p * 3.0).sum(), p)
    torch.cuda.synchronize()
    cr.convrot_adamw_step([p], [early], [torch.zeros(64, device=DEV)], [torch.zeros(64, device=DEV)], step=1, lr=0.5, weight_decay=0.0,
                          copies=[copy], stream=stream)
    torch.cuda.synchronize()
    for loss in (late, late_copy):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    again, = torch.autograd.grad((p * p).sum(), p)
    assert torch.equal(again, 2 * p.detach()) and torch.equal(copy.detach(), p.detach().to(torch.bfloat16))
    # 1 - 0.5 * 3 / (3 + 1e-8), a few roundings off
    assert float((p.detach() - 0.5).abs().max()) < 1e-6


@pytest.mark.parametrize("bits", [32, 8])
def test_the_smallest_eps(cr, bits):
    """Elements without a gradient stay where they are; the others move by the rate (m / sqrt(v) is 1 in a first step)."""
    n = 600
    p, grad = torch.ones(n, device=DEV), torch.zeros(n, device=DEV)
    grad[::3] = 1e-4
    if bits == 8:
        m, v, ms, vs = _codes(n)
        extra = dict(exp_avg_scales=[ms], exp_avg_sq_scales=[vs], seed=9)
    else:
        m, v, extra = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), {}
    cr.convrot_adamw_step([p], [grad], [m], [v], step=1, lr=0.25, eps=2.0 ** -126, weight_decay=0.0, **extra)
    want = torch.ones(n, device=DEV)
    want[::3] = 0.75
    # 24 roundings on the way to the update of a quarter
    assert float((p - want).abs().max()) <= 24 * U and torch.equal(p[1::3], want[1::3])


def _kernel_steps(cr, n):
    state = _codes(n)

    def step(grad, t):
        m, v, ms, vs = state
        cr.convrot_adamw_step([torch.zeros(n, device=DEV)], [dev(grad)], [m], [v], step=t, lr=1e-3, weight_decay=0.0,
                              exp_avg_scales=[ms], exp_avg_sq_scales=[vs], seed=t)
        return v.cpu().numpy()

    step.state = state
    return step


def test_codes_are_right_on_average(cr):
    """Roots that decay by less than a code's step, and first moments on their way to another gradient, arrive."""
    from tests import test_oracle_training as oracle
    check = oracle.check_decaying_roots
    check(*oracle.decaying_roots(_kernel_steps(cr, oracle.WIDE))[:2])
    first, then, at = oracle.turning_gradients()
    step = _kernel_steps(cr, oracle.WIDE)
    for t in range(1, 121):
        step(first if t <= 60 else then, t)
    m, v, ms, vs = step.state
    values, _ = cr.convrot_adamw_moments([m], [v], [ms], [vs])
    oracle.check_first_moment(values.double().cpu().numpy(), first, then, at, 60)
