"""What is measured of the operators around a quantized linear that serve and train low-rank adapters.

Three kinds of case:
  lora_forward   many requests' low-rank adapters beside one shared projection: out = base + c_a (x down_a^T) up_a^T
  lora_backward  the adapters' gradients and the input gradient, with the saved input in bf16 or as rotated INT8 codes
  act_step       an MLP activation that keeps its input as 8-bit codes, and its backward pass from those codes
"""
import math

import numpy as np
import torch

own = False

ROT = 256          # columns of one rotation group
GROUP = 64         # columns of one checkpoint scale
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _fwd(name, **k):
    return {"name": name, "kind": "lora_forward", "M": 1, "S": 1, "tail": 0, "mix": "ragged", "A": 1, "K": 2560,
            "N": 4096, "R": 16, "out": "bf16", "pad": 0, **k}


def _bwd(name, **k):
    return {"name": name, "kind": "lora_backward", "M": 1, "S": 1, "tail": 0, "mix": "ragged", "A": 1, "K": 2560,
            "N": 4096, "R": 16, "out": "bf16", "saved": "bf16", "pad": 0, **k}


def _act(name, **k):
    return {"name": name, "kind": "act_step", "M": 1, "C": 2560, "act": "gelu", "pad": 0, **k}


def listed():
    return [
        # one request decodes one token with its adapter out of a pool of eight: latency alone
        _fwd("decode_one", M=1, S=1, A=8, K=2560, N=4096, R=16),
        # a decode step of 64 requests over 32 adapters, one token each: the adapters' weights are the traffic
        _fwd("decode_64", M=64, S=64, A=32, mix="tokens", K=4096, N=4096, R=32),
        # a prompt of about 1500 tokens joins 47 decoding requests; padded rows at the end, some requests without adapter
        _fwd("chunk_mixed", M=1555, S=48, tail=12, A=16, mix="prompt", K=2560, N=9216, R=16),
        # the image tokens of six edits with four adapters of rank 64, float32 projection outputs
        _fwd("prefill_8192", M=8192, S=6, A=4, K=4096, N=12288, R=64, out="f32"),
        # one training step of one adapter on a text batch of ragged length
        _bwd("train_text", M=1531, S=3, A=1, K=2560, N=2560, R=32),
        # three adapters trained at once on 16 sequences, float32 input gradient
        _bwd("train_8192", M=8192, S=16, A=3, K=4096, N=4096, R=16, out="f32"),
        # a short batch whose inputs were saved as the INT8 codes of the forward pass
        _bwd("train_codes_300", M=300, S=4, tail=9, A=2, K=2560, N=4096, R=8, saved="codes"),
        # the MLP down projection of an image batch, inputs saved as INT8 codes
        _bwd("train_codes_8192", M=8192, S=5, A=1, K=12288, N=4096, R=64, saved="codes"),
        # a short prompt through a gated MLP: latency
        _act("swiglu_22", M=22, C=2560, act="swiglu"),
        # text tokens of an MMDiT block, exact GELU
        _act("gelu_512", M=512, C=12288, act="gelu"),
        # a ragged text batch through a gated MLP
        _act("swiglu_1531", M=1531, C=9216, act="swiglu"),
        # image tokens of an MMDiT block, tanh GELU
        _act("gelu_tanh_8192", M=8192, C=12288, act="gelu_tanh"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["lora_forward", "lora_forward", "lora_backward", "lora_backward", "act_step"])
    pad = rng.choice([0, 0, 8, 64])
    M = _log(rng, 1, 8192)
    if kind == "act_step":
        act = rng.choice(["gelu", "gelu_tanh", "swiglu"])
        return {"kind": kind, "M": M, "C": 64 * _log(rng, 1, 96 if act == "swiglu" else 192), "act": act, "pad": pad}
    tail = rng.choice([0, 0, rng.randrange(0, 1 + M // 4)])
    S = min(_log(rng, 1, 96), max(1, M - tail))
    A = _log(rng, 1, 32 if M <= 512 else 4)
    c = {"kind": kind, "M": M, "S": S, "tail": tail, "mix": rng.choice(["ragged", "prompt", "even"]), "A": A,
         "K": 8 * _log(rng, 8, 1024), "N": 8 * _log(rng, 8, 1024), "R": rng.choice([8, 16, 24, 32, 64, 128]),
         "out": rng.choice(["bf16", "f32"]), "pad": pad}
    if M <= 96 and rng.random() < 0.5:
        c.update(S=M, tail=0, mix="tokens")
    if kind == "lora_backward":
        c["saved"] = rng.choice(["bf16", "codes"])
        if c["saved"] == "codes":
            c["K"] = ROT * _log(rng, 1, 32)
    return c


def spans(case):
    """Offsets [S + 1] and adapter numbers [S] of a case's segments: fixed by the case alone, so that the work is."""
    S, rows = case["S"], case["M"] - case["tail"]
    g = np.random.default_rng([case["M"], S, case["A"], case["K"], case["N"]])
    if case["mix"] == "tokens":          # every row a request of its own
        off = np.arange(S + 1)
    elif case["mix"] == "prompt":        # one long prompt, then single tokens
        off = np.concatenate([[0], np.arange(rows - S + 1, rows + 1)])
    elif case["mix"] == "even":
        off = np.arange(S + 1) * rows // S
    else:                                # ragged lengths, empty ones among them
        off = np.concatenate([[0], np.sort(g.integers(0, rows + 1, S - 1)), [rows]])
    ids = g.integers(0, case["A"], S)
    ids[g.random(S) < (0.1 if S > 8 else 0.0)] = -1      # requests that use the base alone
    return off.astype(np.int64), ids.astype(np.int64)


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
    bf = torch.bfloat16
    s = {"case": case}
    if case["kind"] == "act_step":
        width = case["C"] * (2 if case["act"] == "swiglu" else 1)
        s["z"] = _rows(g, case["M"], width, case["pad"], 1.5, bf)
        s["dy"] = _rows(g, case["M"], case["C"], case["pad"], 0.01, bf)
        return s
    M, N, K, R, A, pad = (case[k] for k in ("M", "N", "K", "R", "A", "pad"))
    off, ids = spans(case)
    s["off"] = torch.from_numpy(off.astype(np.int32)).cuda()
    s["ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
    s["scale"] = torch.rand(A, generator=g, device="cuda") + 0.5
    s["down"] = _normal(g, (A, R, K), 1 / math.sqrt(K), bf)
    s["up"] = _normal(g, (A, N, R), 1 / math.sqrt(R), bf)
    if case["kind"] == "lora_forward":
        s["x"] = _rows(g, M, K, pad, 1.0, bf)
        s["base"] = _rows(g, M, N, pad, 1.0, DTYPES[case["out"]])
        return s
    s["dy"] = _rows(g, M, N, pad, 0.01, bf)
    s["la"] = torch.randn((M, R), generator=g, device="cuda")
    s["base"] = _rows(g, M, K, pad, 0.01, DTYPES[case["out"]])
    if case["saved"] == "bf16":
        s["x"] = _rows(g, M, K, pad, 1.0, bf)
    else:   # the codes of rotated rows: near normal, the largest at 127
        v = torch.randn((M, K), generator=g, device="cuda")
        top = v.abs().amax(1)
        s["x"] = torch.round(v * (127.0 / top)[:, None]).to(torch.int8)
        s["x_scales"] = top / 127.0
        s["rotation"] = _hadamard(ROT)      # kept by a program without the framework, which has it built in
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _members(s, M, A):
    """[M, A] float: 1 where row m belongs to a segment of adapter a."""
    row = torch.arange(M, device="cuda", dtype=torch.int32)
    seg = torch.searchsorted(s["off"][1:].contiguous(), row, right=True)
    ids = torch.cat([s["ids"], s["ids"].new_full((1,), -1)])[seg]
    return (ids[:, None] == torch.arange(A, device="cuda", dtype=torch.int32)).float()


def _plain_forward(s, case):
    M, N, K, R, A = (case[k] for k in ("M", "N", "K", "R", "A"))
    member = _members(s, M, A)[:, :, None]
    every = (s["x"].float() @ s["down"].float().view(A * R, K).T).view(M, A, R) * member
    up = s["up"].float().permute(0, 2, 1).reshape(A * R, N)
    delta = (every * s["scale"][:, None]).view(M, A * R) @ up
    return {"out": (s["base"].float() + delta).to(DTYPES[case["out"]]), "lora_act": every.sum(1)}


def _hadamard(n):
    """The regular Hadamard matrix of order n = 4^d over sqrt(n), from its sign formula."""
    j = torch.arange(n, device="cuda")
    both = j[:, None] & j[None, :]
    bits = torch.arange(n.bit_length() - 1, device="cuda")
    ones = ((both[:, :, None] >> bits) & 1).sum(-1)
    zero = (((j[:, None] >> (2 * torch.arange(bits.numel() // 2, device="cuda"))) & 3) == 0).sum(-1)
    sign = 1 - 2 * ((ones + zero[:, None] + zero[None, :] + bits.numel() // 2) & 1)
    return sign.float() / math.sqrt(n)


def _plain_backward(s, case):
    M, N, K, R, A = (case[k] for k in ("M", "N", "K", "R", "A"))
    member = _members(s, M, A)[:, :, None]
    weighted = member * s["scale"][:, None]
    dy = s["dy"].float()
    up = s["up"].float().permute(1, 0, 2).reshape(N, A * R)
    dla = ((dy @ up).view(M, A, R) * weighted).view(M, A * R)
    dx = s["base"].float() + dla @ s["down"].float().view(A * R, K)
    la = (s["la"][:, None, :] * weighted).view(M, A * R)
    if case["saved"] == "bf16":
        x = s["x"].float()
    else:
        x = ((s["x"].float() * s["x_scales"][:, None]).view(M * K // ROT, ROT) @ s["rotation"]).view(M, K)
    return {"dx": dx.to(DTYPES[case["out"]]), "d_down": (dla.T @ x).view(A, R, K),
            "d_up": (la.T @ dy).view(A, R, N).permute(0, 2, 1).contiguous()}


def _checkpoint(z):
    """8-bit codes and float32 scales of every 64 columns of a row."""
    v = z.float().reshape(z.shape[0], -1, GROUP)
    top = v.abs().amax(-1, keepdim=True)
    r = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    return torch.round(v * r).clamp(-127, 127).to(torch.int8), top / 127.0


def _plain_act(s, case):
    z, dy, C = s["z"].float(), s["dy"].float(), case["C"]
    codes, scales = _checkpoint(s["z"])
    back = (codes.float() * scales).view(z.shape)
    if case["act"] == "gelu":
        y = z * 0.5 * torch.erfc(z * -math.sqrt(0.5))
        dz = dy * (0.5 * torch.erfc(back * -math.sqrt(0.5)) + back * torch.exp(back * back * -0.5) / math.sqrt(2 * math.pi))
    elif case["act"] == "gelu_tanh":
        # 0.5 (1 + tanh t) = sigmoid(2 t)
        a, b = 2 * math.sqrt(2 / math.pi), 0.044715
        y = z * torch.sigmoid(a * (z + b * z * z * z))
        p = torch.sigmoid(a * (back + b * back * back * back))
        dz = dy * (p + back * p * (1 - p) * a * (1 + 3 * b * back * back))
    else:
        y = z[:, :C] * torch.sigmoid(z[:, :C]) * z[:, C:]
        gate, lin = back[:, :C], back[:, C:]
        p = torch.sigmoid(gate)
        dz = torch.cat([dy * lin * p * (1 + gate * (1 - p)), dy * gate * p], 1)
    return {"y": y.to(torch.bfloat16), "dz": dz.to(torch.bfloat16)}


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["kind"] == "lora_forward":
        return _plain_forward(state, case)
    if case["kind"] == "lora_backward":
        return _plain_backward(state, case)
    return _plain_act(state, case)


def _own(s, case):
    import w4a8_rotated_quantized_amd as cr
    if case["kind"] == "act_step":
        act = {"gelu": cr.ACT.GELU, "gelu_tanh": cr.ACT.GELU_TANH, "swiglu": cr.ACT.SWIGLU}[case["act"]]
        y, codes, scales = cr.convrot_act_checkpoint(s["z"], act)
        return {"y": y, "dz": cr.convrot_act_backward(s["dy"], codes, scales, act)}
    kind = {"bf16": cr.OUT.BF16, "f32": cr.OUT.F32}[case["out"]]
    if case["kind"] == "lora_forward":
        out, la = cr.convrot_lora_forward(s["x"], s["down"], s["up"], s["off"], s["ids"], scale=s["scale"],
                                          base=s["base"], out_type=kind)
        return {"out": out, "lora_act": la}
    dx, d_down, d_up = cr.convrot_lora_backward(s["dy"], s["la"], s["x"], s["down"], s["up"], s["off"], s["ids"],
                                                scale=s["scale"], x_scales=s.get("x_scales"), rot_group=ROT,
                                                dx_base=s["base"], dx_type=kind)
    return {"dx": dx, "d_down": d_down, "d_up": d_up}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    M = case["M"]
    if case["kind"] == "act_step":
        wide = M * case["C"] * (2 if case["act"] == "swiglu" else 1)
        # z in, y out, codes and scales out and in again, dy in, dz out
        return {"bytes": wide * 2 + M * case["C"] * 2 + 2 * (wide + wide // GROUP * 4) + M * case["C"] * 2 + wide * 2,
                "flops": 40 * wide}
    N, K, R, A = (case[k] for k in ("N", "K", "R", "A"))
    off, ids = spans(case)
    used = np.unique(ids[(ids >= 0) & (np.diff(off) > 0)]).size
    rows = int(np.diff(off)[ids >= 0].sum())
    e = 2 if case["out"] == "bf16" else 4
    weights = used * R * (N + K) * 2
    if case["kind"] == "lora_forward":
        return {"bytes": rows * K * 2 + 2 * M * N * e + weights + M * R * 4, "flops": 2 * rows * R * (N + K)}
    saved = rows * K * 2 if case["saved"] == "bf16" else rows * (K + 4)
    return {"bytes": rows * N * 2 + rows * R * 4 + saved + 2 * M * K * e + weights + A * R * (N + K) * 4,
            "flops": 4 * rows * R * (N + K)}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "act_step":
        z, dy, C = s["z"].double(), s["dy"].double(), case["C"]
        kept = torch.empty_like(z)
        for c in range(0, z.shape[1], GROUP):
            v = z[:, c:c + GROUP]
            top = v.abs().max(1, keepdim=True).values
            # each quotient and product rounds once to float32: that is the quantizer's definition
            r = (127.0 / top).float().double()
            q = (v * r).float().double().round().clamp(-127, 127)
            kept[:, c:c + GROUP] = torch.where(top > 0, q * (top / 127.0).float().double(), 0.0)
        if case["act"] == "swiglu":
            g, u, kg, ku = z[:, :C], z[:, C:], kept[:, :C], kept[:, C:]
            e, ke = torch.exp(-g), torch.exp(-kg)
            dg = dy * ku * (1 + ke + kg * ke) / (1 + ke) ** 2
            return {"y": g * u / (1 + e), "dz": torch.cat([dg, dy * kg / (1 + ke)], 1)}
        if case["act"] == "gelu":
            rt = math.sqrt(2.0)
            slope = torch.special.erfc(-kept / rt) / 2 + kept * torch.exp(-kept * kept / 2) / math.sqrt(2 * math.pi)
            return {"y": z * torch.special.erfc(-z / rt) / 2, "dz": dy * slope}
        w = math.sqrt(2 / math.pi)
        t = torch.tanh(w * (kept + 0.044715 * kept ** 3))
        slope = (1 + t) / 2 + kept * (1 - t * t) / 2 * w * (1 + 3 * 0.044715 * kept ** 2)
        return {"y": z * (1 + torch.tanh(w * (z + 0.044715 * z ** 3))) / 2, "dz": dy * slope}
    off, ids = spans(case)
    M, N, K, R, A = (case[k] for k in ("M", "N", "K", "R", "A"))
    base = s["base"].double()
    if case["kind"] == "lora_forward":
        la = torch.zeros((M, R), dtype=torch.float64, device="cuda")
        out = base.clone()
        for a, lo, hi in zip(ids, off[:-1], off[1:]):
            if a >= 0 and hi > lo:
                la[lo:hi] = s["x"][lo:hi].double() @ s["down"][a].double().T
                out[lo:hi] += s["scale"][a].double() * (la[lo:hi] @ s["up"][a].double().T)
        return {"out": out, "lora_act": la}
    if case["saved"] == "codes":
        h4 = torch.tensor([[-1, 1, 1, 1], [1, 1, -1, 1], [1, -1, 1, 1], [1, 1, 1, -1]], dtype=torch.float64, device="cuda")
        h = h4
        while h.shape[0] < ROT:
            h = torch.kron(h, h4)
    dx = base.clone()
    d_down = torch.zeros((A, R, K), dtype=torch.float64, device="cuda")
    d_up = torch.zeros((A, N, R), dtype=torch.float64, device="cuda")
    for a, lo, hi in zip(ids, off[:-1], off[1:]):
        if a >= 0 and hi > lo:
            dy = s["dy"][lo:hi].double()
            dla = s["scale"][a].double() * (dy @ s["up"][a].double())
            dx[lo:hi] += dla @ s["down"][a].double()
            x = s["x"][lo:hi].double()
            if case["saved"] == "codes":
                x = ((x * s["x_scales"][lo:hi, None].double()).view(-1, ROT) @ h).view(hi - lo, K) / math.sqrt(ROT)
            d_down[a] += dla.T @ x
            d_up[a] += s["scale"][a].double() * (dy.T @ s["la"][lo:hi].double())
    return {"dx": dx, "d_down": d_down, "d_up": d_up}
