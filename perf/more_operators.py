"""What is measured of the operators around the quantized linear that a training step of adapters over a 4-bit base,
and its serving, run besides those of operators.py.

Five kinds of case:
  mx_round    a matrix quantized to microscaled 4-bit floating point (E2M1 codes, one power of two per 32 columns) and read back
  mx_linear   y = Q(x H) Q(W H)^T + bias: activations quantized in the call, weights quantized beforehand
  norm        layer norm with one weight and bias, or one pair per sequence (adaLN modulation)
  norm_back   its gradients: input, and weight and bias summed over the rows of each sequence
  adamw       one optimizer step over a list of tensors, moments in float32 or in 8 bits
"""
import math

import numpy as np
import torch

own = False

TILE = 128         # columns of one tile of the 4-bit layout
BLOCK = 32         # columns that share a power of two
STATE = 256        # elements that share a scale of an 8-bit moment
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = 8192 * 4096 * 12288


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _round(name, **k):
    return {"name": name, "kind": "mx_round", "M": 1, "K": 2560, "rot": 0, "out": "bf16", "pad": 0, **k}


def _linear(name, **k):
    return {"name": name, "kind": "mx_linear", "M": 1, "K": 2560, "N": 4096, "rot": 256, "out": "bf16", "bias": True,
            "pad": 0, **k}


def _norm(name, **k):
    return {"name": name, "kind": "norm", "M": 1, "C": 2560, "S": 0, "x": "bf16", "out": "bf16", "pad": 0, **k}


def _back(name, **k):
    return {"name": name, "kind": "norm_back", "M": 1, "C": 2560, "S": 0, "x": "bf16", "out": "bf16", "base": True,
            "pad": 0, **k}


def _adamw(name, **k):
    return {"name": name, "kind": "adamw", "T": 1, "R": 16, "K": 2560, "N": 2560, "bits": 32, "grad": "f32", **k}


def listed():
    return [
        # a short prompt's ragged rows, columns that are no multiple of a tile, kept unrotated
        _round("mx_round_257", M=257, K=1056, rot=0, pad=8),
        # an MLP weight, rotated and quantized, and read back for what trains against it
        _round("mx_round_9216", M=9216, K=2560, rot=256, out="f32"),
        # one token through a projection: the weights are the traffic
        _linear("mx_linear_1", M=1, K=4096, N=4096),
        # a short prompt into a gated MLP's wide side
        _linear("mx_linear_22", M=22, K=2560, N=9728, rot=0, bias=False),
        # a ragged text batch
        _linear("mx_linear_1531", M=1531, K=2560, N=9216, out="f32"),
        # the image tokens of an MMDiT block
        _linear("mx_linear_8192", M=8192, K=4096, N=12288),
        # a prompt's rows before a projection: latency
        _norm("norm_77", M=77, C=2560, out="f32"),
        # image tokens of six edits, modulated each by its own scale and shift
        _norm("norm_8192", M=8192, C=4096, S=6),
        # a ragged text batch's gradients, the residual's gradient added in
        _back("norm_back_1531", M=1531, C=2560),
        # image tokens of five edits
        _back("norm_back_8192", M=8192, C=4096, S=5),
        # eight adapters of rank 16
        _adamw("adamw_8", T=8, R=16, K=2560, N=4096),
        # the adapters of 36 layers, seven projections each, rank 32, moments in 8 bits
        _adamw("adamw_252", T=252, R=32, K=2560, N=4096, bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["mx_round", "mx_linear", "mx_linear", "norm", "norm_back", "adamw"])
    pad = rng.choice([0, 0, 8, 64])
    M = _log(rng, 1, 8192)
    if kind in ("mx_round", "mx_linear"):
        rot = rng.choice([0, 256, 64])
        K = 256 * _log(rng, 1, 32) if rot else BLOCK * _log(rng, 1, 256)
        c = {"kind": kind, "M": M, "K": K, "rot": rot, "out": rng.choice(["bf16", "f32"]), "pad": pad}
        if kind == "mx_linear":
            c.update(N=8 * _log(rng, 1, max(1, min(1536, LARGEST // (8 * M * K)))), bias=rng.random() < 0.5)
        return c
    if kind == "adamw":
        return {"kind": kind, "T": 2 * _log(rng, 1, 64), "R": rng.choice([8, 16, 24, 32, 64, 128]), "K": 8 * _log(rng, 8, 512),
                "N": 8 * _log(rng, 8, 512), "bits": rng.choice([8, 32]), "grad": rng.choice(["f32", "bf16"])}
    c = {"kind": kind, "M": M, "C": 8 * _log(rng, 8, 1024), "S": rng.choice([0, 0, min(M, _log(rng, 1, 48))]),
         "x": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]), "pad": pad}
    if kind == "norm_back":
        c["base"] = rng.random() < 0.5
    return c


def spans(case):
    """Offsets [S + 1] of a case's sequences, fixed by the case alone: ragged, empty ones among them."""
    M, S = case["M"], case["S"]
    g = np.random.default_rng([M, S, case["C"]])
    return np.concatenate([[0], np.sort(g.integers(0, M + 1, S - 1)), [M]]).astype(np.int64)


def sizes(case):
    """Elements of each tensor of an optimizer step: down [R, K] and up [N, R] in turn."""
    return [case["R"] * (case["K"] if i % 2 == 0 else case["N"]) for i in range(case["T"])]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _rows(g, M, C, pad, std, dtype):
    """[M, C] in rows of C + pad elements, as a slice of a wider buffer."""
    return _normal(g, (M, C + pad), std, dtype)[:, :C]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf, s = torch.bfloat16, {"case": case}
    if case["kind"] in ("mx_round", "mx_linear"):
        M, K = case["M"], case["K"]
        s["x"] = _rows(g, M, K, case["pad"], 1.0, bf)
        s["x"][:, torch.randint(0, K, (max(1, K // 200),), generator=g, device="cuda")] *= 20      # outlier channels
        if case["kind"] == "mx_linear":
            w = _normal(g, (case["N"], K), 1 / math.sqrt(K), bf)
            s["w_codes"], s["w_scales"] = _encode(w, case["rot"])       # the quantized weights a program keeps
            s["bias"] = _normal(g, (case["N"],), 0.1, bf) if case["bias"] else None
        return s
    if case["kind"] == "adamw":
        n = sum(sizes(case))
        cut = lambda t: list(torch.split(t, sizes(case)))  # noqa: E731
        s["flat"] = {"p": _normal(g, (n,), 0.02, torch.float32), "copy": torch.zeros(n, dtype=bf, device="cuda")}
        s["g"] = cut(_normal(g, (n,), 1e-3, DTYPES[case["grad"]]))
        m, v = _normal(g, (n,), 3e-4, torch.float32), _normal(g, (n,), 1e-3, torch.float32) ** 2
        if case["bits"] == 8:
            # every tensor's blocks are its own: scales and codes tensor by tensor
            blocks = [-(-k // STATE) for k in sizes(case)]
            per = lambda t: list(torch.split(t, blocks))  # noqa: E731
            s["flat"]["m"], s["flat"]["v"] = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
            s["flat"]["ms"], s["flat"]["vs"] = torch.zeros(sum(blocks), device="cuda"), torch.zeros(sum(blocks), device="cuda")
            s["ms"], s["vs"] = per(s["flat"]["ms"]), per(s["flat"]["vs"])
            for i, (a, b) in enumerate(zip(cut(m), cut(v))):
                half = torch.full_like(a, 0.5)
                a, sa = _encode_moment(a, half, 127)
                b, sb = _encode_moment(_sqrt(b), half, 255)
                cut(s["flat"]["m"])[i].copy_(a)
                cut(s["flat"]["v"])[i].copy_(b)
                s["ms"][i].copy_(sa)
                s["vs"][i].copy_(sb)
        else:
            s["flat"]["m"], s["flat"]["v"] = m, v
        for k in ("p", "copy", "m", "v"):
            s[k] = cut(s["flat"][k])
        s["hyper"] = {"lr": 2e-4, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
        s["step"], s["seed"] = 100, seed % 65521
        s["clip"] = torch.rand(1, generator=g, device="cuda") * 0.5 + 0.5        # the gradient-norm clip's factor
        return s
    M, C, S = case["M"], case["C"], case["S"]
    s["x"] = _rows(g, M, C, case["pad"], 1.5, DTYPES[case["x"]])
    s["x"] += 0.5
    shape = (S, C) if S else (C,)
    s["w"], s["b"] = _normal(g, shape, 0.2, bf), _normal(g, shape, 0.2, bf)
    if S:                                     # modulation: 1 + scale
        s["off"] = torch.from_numpy(spans(case).astype(np.int32)).cuda()
    else:
        s["w"] += 1
        s["off"] = None
    if case["kind"] == "norm_back":
        s["dy"] = _rows(g, M, C, case["pad"], 0.01, bf)
        s["base"] = _rows(g, M, C, case["pad"], 0.01, DTYPES[case["out"]]) if case["base"] else None
        s["mean"], s["rstd"] = _moments(s["x"].float())                  # kept from the forward pass
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _hadamard_rows(v, n):
    """Groups of n columns times the regular Hadamard matrix (unnormalised), in float32 butterflies h = 1, 2, .., n/2."""
    rows, K = v.shape
    j = torch.arange(n, device="cuda")
    zeros = sum((((j >> (2 * d)) & 3) == 0).int() for d in range(int(math.log(n, 4) + 0.5)))
    sign = (1 - 2 * (zeros & 1)).float()
    v = (v.view(-1, n) * sign)
    h = 1
    while h < n:
        w = v.view(-1, n // (2 * h), 2, h)
        v = torch.stack([w[:, :, 0] + w[:, :, 1], w[:, :, 0] - w[:, :, 1]], 2).view(-1, n)
        h *= 2
    d = int(math.log(n, 4) + 0.5)
    return (v * sign * (-1.0) ** d).view(rows, K)


def _encode(x, rot):
    """E2M1 codes [tiles, rows, 64] (two a byte, even column low) and power-of-two bytes [tiles, rows, 4]."""
    v = x.float()
    rows, K = v.shape
    if rot:
        v = _hadamard_rows(v, rot)
    tiles = -(-K // TILE)
    if K < tiles * TILE:
        v = torch.cat([v, v.new_zeros(rows, tiles * TILE - K)], 1)
    v = v.view(rows, tiles * 4, BLOCK)
    top = v.abs().amax(-1)
    power = torch.frexp(top)[1] - 3                               # floor(log2 top) - 2
    half = int(math.log(rot, 4) + 0.5) if rot else 0              # 1 / sqrt(rot) = 2^-half
    byte = (power + 127 - half).clamp(0, 254)
    r = v * torch.ldexp(torch.ones_like(top), 127 - byte - half)[:, :, None]
    a = r.abs()
    # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; halves to the even code
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5).int())
    code = code + 8 * (r < 0).int()
    byte = torch.where(top > 0, byte, torch.zeros_like(byte))
    code = code.view(rows, tiles, TILE)
    packed = (code[:, :, 0::2] + 16 * code[:, :, 1::2]).to(torch.uint8)
    return packed.permute(1, 0, 2).contiguous(), byte.to(torch.uint8).view(rows, tiles, 4).permute(1, 0, 2).contiguous()


def _decode(codes, scales, K):
    """float32 [rows, K] of codes and power-of-two bytes."""
    tiles, rows, _ = codes.shape
    c = codes.permute(1, 0, 2).reshape(rows, tiles * 64).int()
    c = torch.stack([c & 15, c >> 4], -1).view(rows, tiles * 4, BLOCK)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    byte = scales.permute(1, 0, 2).reshape(rows, tiles * 4).int()
    v = table[c] * torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte - 127)[:, :, None]
    return v.view(rows, tiles * TILE)[:, :K]


def _plain_round(s, case):
    v = _decode(*_encode(s["x"], case["rot"]), case["K"])
    if case["rot"]:
        v = _hadamard_rows(v.contiguous(), case["rot"]) / math.sqrt(case["rot"])
    return {"x": v.to(DTYPES[case["out"]])}


def _plain_linear(s, case):
    x = _decode(*_encode(s["x"], case["rot"]), case["K"])
    y = x @ _decode(s["w_codes"], s["w_scales"], case["K"]).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.to(DTYPES[case["out"]])}


def _moments(x):
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    return mean, 1 / torch.sqrt(var + 1e-6)


def _of_rows(s, case):
    """Sequence of each row."""
    row = torch.arange(case["M"], device="cuda", dtype=torch.int32)
    return torch.searchsorted(s["off"][1:].contiguous(), row, right=True)


def _plain_norm(s, case):
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    mean, rstd = _moments(x)
    if case["S"]:
        at = _of_rows(s, case)
        w, b = 1 + w[at], b[at]
    y = (x - mean[:, None]) * rstd[:, None] * w + b
    return {"y": y.to(DTYPES[case["out"]]), "mean": mean, "rstd": rstd}


def _plain_back(s, case):
    x, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    if case["S"]:
        at = _of_rows(s, case)
        g = dy * (1 + w[at])
        member = (at[None, :] == torch.arange(case["S"], device="cuda")[:, None]).float()
        dw, db = member @ (dy * xh), member @ dy
    else:
        g = dy * w
        dw, db = (dy * xh).sum(0), dy.sum(0)
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["base"] is not None:
        dx = dx + s["base"].float()
    return {"dx": dx.to(DTYPES[case["out"]]), "dw": dw, "db": db}


def _sqrt(x):
    """Rounded once to float32."""
    return torch.sqrt(x.double()).float()


def _random16(seed, tensor, n):
    """Two 16-bit numbers for each element, as float32 in [0, 1): a hash of (seed, tensor, element)."""
    def mix(x):
        x = x ^ (x >> 16)
        x = (x * 0x6A09E667) & 0xFFFFFFFF
        x = x ^ (x >> 15)
        x = (x * 0xBB67AE85) & 0xFFFFFFFF
        return x ^ (x >> 16)

    i = torch.arange(n, device="cuda", dtype=torch.int64)
    key = mix(torch.tensor((seed + 0x9E3779B9 * (tensor + 1)) & 0xFFFFFFFF, device="cuda"))
    h = mix(mix(i & 0xFFFFFFFF) ^ key)
    return (h & 0xFFFF).float() / 65536, (h >> 16).float() / 65536


def _blocks(x):
    """[blocks, 256] of a flat tensor, zeros behind its end."""
    pad = -x.numel() % STATE
    return torch.cat([x, x.new_zeros(pad)]).view(-1, STATE) if pad else x.view(-1, STATE)


def _encode_moment(x, u, most):
    """Codes of x = s (c / most) |c / most| with s the largest magnitude of each 256, rounded up with chance u, and the scales."""
    v = _blocks(x)
    top = v.abs().amax(1)
    q = (v.abs().double() / top.double()[:, None]).float()
    t = _sqrt(q) * most
    c = torch.floor(t + _blocks(u)).clamp(max=most)
    if most == 255:
        c = torch.where(v > 0, c.clamp(min=1), c)               # a root that is not zero stays above zero
    c = torch.where(top[:, None] > 0, c, torch.zeros_like(c))
    return (c * torch.sign(v)).view(-1)[:x.numel()].to(torch.int8 if most == 127 else torch.uint8), top


def _decode_moment(c, top, most):
    """s (c / most) |c / most|, the integer c |c| times s / most^2."""
    v = _blocks(c.float())
    step = (top.double() / (most * most)).float()
    return (v * v.abs() * step[:, None]).view(-1)[:c.numel()]


def _plain_adamw(s, case):
    h, t = s["hyper"], s["step"]
    c1, c2 = 1 - h["beta1"] ** t, 1 - h["beta2"] ** t
    read = {"m": [], "v": []}
    for i in range(case["T"]):
        g = s["g"][i].float() * s["clip"]
        if case["bits"] == 8:
            m, r = _decode_moment(s["m"][i], s["ms"][i], 127), _decode_moment(s["v"][i], s["vs"][i], 255)
            v = r * r
        else:
            m, v = s["m"][i], s["v"][i]
        m = m * h["beta1"] + g * (1 - h["beta1"])
        v = v * h["beta2"] + g * g * (1 - h["beta2"])
        root = _sqrt(v)
        p = s["p"][i] * (1 - h["lr"] * h["weight_decay"])
        p = p - (m / (root * (1 / math.sqrt(c2)) + h["eps"])) * (h["lr"] / c1)
        s["p"][i].copy_(p)
        s["copy"][i].copy_(p)
        if case["bits"] == 8:
            um, uv = _random16(s["seed"], i, m.numel())
            c, top = _encode_moment(m, um, 127)
            s["m"][i].copy_(c)
            s["ms"][i].copy_(top)
            read["m"].append(_decode_moment(c, top, 127))
            c, top = _encode_moment(root, uv, 255)
            s["v"][i].copy_(c)
            s["vs"][i].copy_(top)
            read["v"].append(_decode_moment(c, top, 255) ** 2)
        else:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
    out = {"p": s["flat"]["p"], "copy": s["flat"]["copy"], "m": s["flat"]["m"], "v": s["flat"]["v"]}
    if case["bits"] == 8:
        out.update(m=torch.cat(read["m"]), v=torch.cat(read["v"]))
    return out


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    plain = {"mx_round": _plain_round, "mx_linear": _plain_linear, "norm": _plain_norm, "norm_back": _plain_back,
             "adamw": _plain_adamw}
    return plain[case["kind"]](state, case)


def _own(s, case):
    import w4a8_rotated_quantized_amd as cr
    kind = case["kind"]
    if kind == "adamw":
        moments = {}
        if case["bits"] == 8:
            moments = {"exp_avg_scales": s["ms"], "exp_avg_sq_scales": s["vs"], "seed": s["seed"]}
        cr.convrot_adamw_step(s["p"], s["g"], s["m"], s["v"], step=s["step"], copies=s["copy"], grad_scale=s["clip"],
                              **s["hyper"], **moments)
        out = {"p": s["flat"]["p"], "copy": s["flat"]["copy"], "m": s["flat"]["m"], "v": s["flat"]["v"]}
        if case["bits"] == 8:
            out["m"], out["v"] = cr.convrot_adamw_moments(s["m"], s["v"], s["ms"], s["vs"])
        return out
    kind_out = {"bf16": cr.OUT.BF16, "f32": cr.OUT.F32}[case["out"]]
    if kind == "mx_round":
        codes, scales = cr.mxfp4_quantize(s["x"], case["rot"])
        return {"x": cr.mxfp4_dequantize(codes, scales, case["K"], case["rot"], out_type=kind_out)}
    if kind == "mx_linear":
        codes, scales = cr.mxfp4_quantize(s["x"], case["rot"])
        return {"y": cr.mxfp4_gemm(codes, scales, s["w_codes"], s["w_scales"], bias=s["bias"], out_type=kind_out)}
    if kind == "norm":
        y, mean, rstd = cr.convrot_layer_norm_forward(s["x"], s["w"], s["b"], seg_offsets=s["off"], one_plus=bool(case["S"]),
                                                      eps=1e-6, out_type=kind_out)
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dw, db = cr.convrot_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], seg_offsets=s["off"],
                                                one_plus=bool(case["S"]), dx_base=s["base"], dx_type=kind_out)
    return {"dx": dx, "dw": dw, "db": db}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    wide = {"bf16": 2, "f32": 4}
    if case["kind"] == "adamw":
        n = sum(sizes(case))
        g = wide[case["grad"]]
        if case["bits"] == 32:
            return {"bytes": n * (8 + g + 8 + 8 + 2), "flops": 15 * n}
        # the moments' codes in and out, their scales, and what is read out of them
        return {"bytes": n * (8 + g + 4 + 2 + 8) + n // STATE * 16, "flops": 50 * n}
    M = case["M"]
    if case["kind"] in ("mx_round", "mx_linear"):
        K, e, mx = case["K"], wide[case["out"]], lambda n: n // 2 + n // BLOCK  # noqa: E731
        if case["kind"] == "mx_round":
            return {"bytes": M * K * (2 + e) + 2 * mx(M * K), "flops": 20 * M * K}
        N = case["N"]
        return {"bytes": M * K * 2 + 2 * mx(M * K) + mx(N * K) + M * N * e + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    C, S = case["C"], max(1, case["S"])
    x, o = wide[case["x"]], wide[case["out"]]
    if case["kind"] == "norm":
        return {"bytes": M * C * (x + o) + 8 * M + 4 * S * C, "flops": 8 * M * C}
    return {"bytes": M * C * (x + 2 + o + (o if case["base"] else 0)) + 8 * M + (2 + 8) * S * C, "flops": 16 * M * C}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _rotation(n):
    """The regular Hadamard matrix of order n as products of the order-4 one."""
    h4 = torch.tensor([[-1, 1, 1, 1], [1, 1, -1, 1], [1, -1, 1, 1], [1, 1, 1, -1]], dtype=torch.float64, device="cuda")
    h = h4
    while h.shape[0] < n:
        h = torch.kron(h, h4)
    return h


def _exact_values(x, rot):
    """What the 4-bit codes of a matrix stand for. The rotation's sums round to float32 one by one: that is the quantizer's definition."""
    v = x.double()
    rows, K = v.shape
    if rot:
        h4 = _rotation(4)
        bits = rot.bit_length() - 1
        v = v.reshape(rows * K // rot, *([2] * bits))
        # the signs of H are those of D S D: D[j] = (-1)^(zero base-4 digits of j)
        first = torch.tensor([-1.0, 1, 1, 1], dtype=torch.float64, device="cuda")
        d = first
        while d.numel() < rot:
            d = torch.kron(d, first)
        v = v * d.view(*([2] * bits))
        for axis in range(bits, 0, -1):
            lo, hi = v.select(axis, 0), v.select(axis, 1)
            v = torch.stack([(lo + hi).float().double(), (lo - hi).float().double()], axis)
        v = (v * d.view(*([2] * bits)) * (h4[0, 0] ** (bits // 2))).reshape(rows, K) / math.sqrt(rot)
    out = torch.zeros_like(v)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    middle = (grid[1:] + grid[:-1]) / 2
    for c in range(0, K, BLOCK):
        b = v[:, c:c + BLOCK]
        top = b.abs().max(1, keepdim=True).values
        unit = 2.0 ** (torch.floor(torch.log2(top.clamp(min=1e-300))) - 2).clamp(min=-127)
        a = b.abs() / unit
        low = torch.bucketize(a, middle, right=False)           # a half goes to the lower code here ...
        high = torch.bucketize(a, middle, right=True)           # ... and to the upper one here
        code = torch.where(low % 2 == 0, low, high)
        out[:, c:c + BLOCK] = torch.where(top > 0, torch.sign(b) * grid[code] * unit, 0.0)
    return out


def _exact_codes(codes, scales, K):
    c = codes.permute(1, 0, 2).reshape(codes.shape[1], -1).to(torch.int64)
    c = torch.stack([c % 16, c // 16], 2).flatten(1)[:, :K]
    size = c % 8
    a = torch.where(size < 4, size * 0.5, (2 + size % 2).double() * 2.0 ** (size // 2 - 2).double())
    unit = 2.0 ** (scales.permute(1, 0, 2).reshape(codes.shape[1], -1).double() - 127)
    return torch.where(c < 8, a, -a) * unit.repeat_interleave(BLOCK, 1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "mx_round":
        v = _exact_values(s["x"], case["rot"])
        if case["rot"]:
            v = (v.view(-1, case["rot"]) @ _rotation(case["rot"])).view(v.shape) / math.sqrt(case["rot"])
        return {"x": v}
    if kind == "mx_linear":
        y = _exact_values(s["x"], case["rot"]) @ _exact_codes(s["w_codes"], s["w_scales"], case["K"]).T
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    if kind == "adamw":
        return _exact_adamw(s, case)
    x, w = s["x"].double(), s["w"].double()
    M, C = x.shape
    off = spans(case) if case["S"] else np.array([0, M])
    w, b = (1 + w, s["b"].double()) if case["S"] else (w[None], s["b"].double()[None])
    if kind == "norm":
        y, mean, rstd = torch.empty_like(x), x.sum(1) / C, torch.empty(M, dtype=torch.float64, device="cuda")
        for i, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
            d = x[lo:hi] - mean[lo:hi, None]
            rstd[lo:hi] = (d.square().sum(1) / C + 1e-6) ** -0.5
            y[lo:hi] = d * rstd[lo:hi, None] * w[i] + b[i]
        return {"y": y, "mean": mean, "rstd": rstd}
    dy = s["dy"].double()
    dx, dw, db = torch.empty_like(x), torch.zeros_like(w), torch.zeros_like(w)
    for i, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        xh = (x[lo:hi] - s["mean"][lo:hi, None].double()) * s["rstd"][lo:hi, None].double()
        g = dy[lo:hi] * w[i]
        dx[lo:hi] = s["rstd"][lo:hi, None].double() * (g - g.sum(1, keepdim=True) / C - xh * (g * xh).sum(1, keepdim=True) / C)
        dw[i], db[i] = (dy[lo:hi] * xh).sum(0), dy[lo:hi].sum(0)
    if s["base"] is not None:
        dx += s["base"].double()
    return {"dx": dx, "dw": dw if case["S"] else dw[0], "db": db if case["S"] else db[0]}


def _exact_adamw(s, case):
    """One step in 64 bits. The codes' rounding has no value in 64 bits: the moments of 8-bit cases are left out."""
    h, t = s["hyper"], s["step"]
    p, ms, vs = [], [], []
    for i in range(case["T"]):
        g = s["g"][i].double() * s["clip"].double()
        m, v = s["m"][i].double(), s["v"][i].double()
        if case["bits"] == 8:
            wide = lambda top: top.double().repeat_interleave(STATE)[:m.numel()]  # noqa: B023,E731
            m = wide(s["ms"][i]) * torch.sign(m) * (m / 127) ** 2
            v = (wide(s["vs"][i]) * (v / 255) ** 2) ** 2
        m = h["beta1"] * m + (1 - h["beta1"]) * g
        v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
        ms.append(m)
        vs.append(v)
        bias1, bias2 = 1 - h["beta1"] ** t, 1 - h["beta2"] ** t
        p.append(s["p"][i].double() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * (m / bias1) / ((v / bias2) ** 0.5 + h["eps"]))
    p = torch.cat(p)
    coded = case["bits"] == 8
    return {"p": p, "copy": p, "m": None if coded else torch.cat(ms), "v": None if coded else torch.cat(vs)}
