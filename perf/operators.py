"""Cases of the operators around the 4-bit layers of a transformer block: the
dense linear with a fused epilogue (16- and 8-bit operands), the RMS norm with
the residual's addition and an 8-bit output, and rotary positions with several
axes.

    plain form   elementary torch operations in fp32 (fp64 for rotary angles)
    own form     the calls of bit_diffusion_transformer_w4a4_b200.svdq
    exact        the definitions in fp64
"""
import math

import torch

own = False

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "int8": 1}
TOP = {"e4m3": 448.0, "int8": 127.0}       # largest code of an 8-bit type
TINY = 2.0 ** -118                         # rows whose largest value is below this become zero codes


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # attention's output projection of a 1024-px image (4096 image + 512 text tokens) kept in 16
        # bits: bias, the block's gate (one row of it: one image) and the residual stream
        _dense("dense_bf16_attn_out", "bf16", "bf16", 4608, 3072, 3072, "none", True, 4608, True),
        # the same block's first MLP layer in 8 bits
        _dense("dense_e4m3_fc1_gelu", "e4m3", "bf16", 4608, 3072, 12288, "gelu", True, 0, False),
        # the second MLP layer of a 2048-px image in 8 bits, two images' gates: the largest call
        _dense("dense_int8_fc2_2048px", "int8", "bf16", 16896, 12288, 3072, "none", True, 8448, True),
        # the modulation of two conditioning vectors (classifier-free guidance): one read of the weights
        _dense("dense_bf16_modulation", "bf16", "bf16", 2, 3072, 18432, "none", True, 0, False),
        # a text projection of odd length and width
        _dense("dense_fp16_ragged", "fp16", "fp16", 333, 1000, 1501, "silu", True, 0, True),
        # the norm before an 8-bit projection of a 1024-px block
        _rms("rms_e4m3_block", "bf16", "e4m3", 4608, 3072, True, True, True),
        # one token (a decoder's step or a pooled embedding): latency
        _rms("rms_int8_token", "bf16", "int8", 1, 4096, True, True, True),
        # quantising the activated MLP hidden state of a 2048-px image, without a norm
        _rms("rms_e4m3_hidden_2048px", "bf16", "e4m3", 16896, 12288, False, False, False),
        # odd rows of an odd length
        _rms("rms_int8_odd", "fp16", "int8", 517, 2047, True, True, True),
        # Q and K of an image block: text index, row and column axes, interleaved pairs
        _rope("rope_image_qk", "bf16", 1, 4608, 24, 24, 128, "16,56,56", 10000.0, True, False, False, 512),
        # Q and grouped K of a video: time, height and width sections of one frequency line, split halves
        _rope("rope_video_gqa", "bf16", 1, 32768, 24, 8, 128, "32,48,48", 1000000.0, False, True, False, 4096),
        # gradients of a partly rotated head in 32 bits, odd length, two sequences
        _rope("rope_inverse_fp32", "fp32", 2, 777, 10, 10, 80, "32,32", 10000.0, True, False, True, 100000),
    ]


def _dense(name, kind, out, M, K, N, act, bias, gate_rows, residual):
    c = {"op": "dense", "in": kind, "out": out, "M": M, "K": K, "N": N, "act": act, "bias": bias,
         "gate_rows": gate_rows, "residual": residual}
    return {"name": name, **c} if name else c


def _rms(name, kind, out, M, K, residual, weight, norm):
    c = {"op": "rms", "in": kind, "out": out, "M": M, "K": K, "residual": residual, "weight": weight, "norm": norm}
    return {"name": name, **c} if name else c


def _rope(name, kind, B, S, H, HK, D, axes, theta, interleaved, shared, inverse, far):
    c = {"op": "rope", "in": kind, "B": B, "S": S, "H": H, "HK": HK, "D": D, "axes": axes, "theta": theta,
         "interleaved": interleaved, "shared": shared, "inverse": inverse, "far": far}
    return {"name": name, **c} if name else c


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dense", "dense", "rms", "rope"])
    if op == "dense":
        kind = rng.choice(["bf16", "fp16", "e4m3", "int8"])
        out = kind if SIZE[kind] == 2 else rng.choice(["bf16", "fp16"])
        step = 16 // SIZE[kind]                    # a row is a whole number of 16-byte pieces
        M, N = _spread(rng, 1, 16896), _spread(rng, 17, 18432)
        K = step * _spread(rng, 4, 12288 // step)
        while M * N * K > 16896 * 12288 * 3072:
            M = max(1, M // 2)
        gate = rng.choice([0, 0, M, (M + 1) // 2])
        return _dense("", kind, out, M, K, N, rng.choice(["none", "gelu", "silu"]), rng.random() < 0.6, gate,
                      rng.random() < 0.5)
    if op == "rms":
        M, K = _spread(rng, 1, 16896), _spread(rng, 32, 12288)
        return _rms("", rng.choice(["bf16", "fp16", "fp32"]) if K <= 6144 else rng.choice(["bf16", "fp16"]),
                    rng.choice(["e4m3", "int8"]), M, K, rng.random() < 0.6, rng.random() < 0.7, rng.random() < 0.7)
    D = 2 * rng.randint(16, 64)
    n = rng.randint(1, 3)
    cut = sorted(rng.sample(range(1, D // 2), n))
    axes = [2 * (b - a) for a, b in zip([0] + cut[:-1], cut)]
    if rng.random() < 0.6:                         # most models rotate the whole head
        axes[-1] += D - sum(axes)
    H = rng.randint(1, 24)
    B = rng.randint(1, 3)
    S = _spread(rng, 1, 10922)
    return _rope("", rng.choice(["bf16", "fp16", "fp32"]) if S < 4096 else "bf16", B, S, H, rng.choice([0, H, 1]), D,
                 ",".join(map(str, axes)), rng.choice([10000.0, 256.0, 1000000.0]), rng.random() < 0.5,
                 rng.random() < 0.5, rng.random() < 0.4, rng.choice([64, 4096, 1000000]))


# ------------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"dense": _prepare_dense, "rms": _prepare_rms, "rope": _prepare_rope}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(x, kind):
    """Row-wise 8-bit codes of x and their scales."""
    s = x.abs().amax(dim=1) / TOP[kind]
    q = x / s[:, None]
    return (q.round().to(torch.int8) if kind == "int8" else q.to(torch.float8_e4m3fn)), s


def _prepare_dense(c, g):
    M, K, N, out = c["M"], c["K"], c["N"], TORCH[c["out"]]
    x, w = _randn(g, M, K), _randn(g, N, K) * K ** -0.5
    st = {"case": c, "a_scale": None, "w_scale": None, "bias": None, "gate": None, "residual": None}
    if SIZE[c["in"]] == 1:
        st["a"], st["a_scale"] = _codes(x, c["in"])
        st["w"], st["w_scale"] = _codes(w, c["in"])
    else:
        st["a"], st["w"] = x.to(out), w.to(out)
    if c["bias"]:
        st["bias"] = (0.5 * _randn(g, N)).to(out)
    if c["gate_rows"]:
        st["gate"] = _randn(g, -(-M // c["gate_rows"]), N).to(out)
    if c["residual"]:
        st["residual"] = _randn(g, M, N).to(out)
    st["y"] = torch.empty(M, N, device="cuda", dtype=out)
    return st


def _prepare_rms(c, g):
    M, K, t = c["M"], c["K"], TORCH[c["in"]]
    x = _randn(g, M, K)
    x[:, :: max(1, K // 8)] *= 20.0                # outlier channels
    st = {"case": c, "x": x.to(t), "residual": None, "h": None, "weight": None}
    if c["residual"]:
        st["residual"] = (4.0 * _randn(g, M, K)).to(t)
        st["h"] = torch.empty(M, K, device="cuda", dtype=t)
    if c["weight"]:
        st["weight"] = (1.0 + 0.2 * _randn(g, K)).to(t)
    st["codes"] = torch.empty(M, K, device="cuda", dtype=TORCH[c["out"]])
    st["scales"] = torch.empty(M, device="cuda", dtype=torch.float32)
    return st


def _axes(c):
    return [int(v) for v in c["axes"].split(",")]


def _prepare_rope(c, g):
    B, S, D, t, n = c["B"], c["S"], c["D"], TORCH[c["in"]], len(_axes(c))
    st = {"case": c, "q": _randn(g, B, S, c["H"], D).to(t), "k": None, "k_out": None}
    st["q_out"] = torch.empty_like(st["q"])
    if c["HK"]:
        st["k"] = _randn(g, B, S, c["HK"], D).to(t)
        st["k_out"] = torch.empty_like(st["k"])
    # every axis has a range of its own; the first reaches `far`
    hi = torch.tensor([c["far"]] + [64] * (n - 1), device="cuda", dtype=torch.float32)
    u = torch.rand(B * S, n, generator=g, device="cuda")
    st["pos"] = torch.floor(u * hi).to(torch.int32)
    if own:
        from bit_diffusion_transformer_w4a4_b200 import svdq
        st["plan"] = svdq.RopeAxes(D, _axes(c), c["theta"], interleaved=c["interleaved"], shared=c["shared"])
    else:
        st["axis"], st["freq"] = _plain_freq(c)
    return st


def _plain_freq(c):
    """The axis and the frequency (radians a position, fp64) of every pair."""
    axes = _axes(c)
    axis = torch.cat([torch.full((d // 2,), a) for a, d in enumerate(axes)]).cuda()
    if c["shared"]:
        e = torch.arange(sum(axes) // 2, dtype=torch.float64) * 2 / sum(axes)
    else:
        e = torch.cat([torch.arange(d // 2, dtype=torch.float64) * 2 / d for d in axes])
    return axis, torch.exp(-math.log(c["theta"]) * e).cuda()


# ------------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    if own:
        from bit_diffusion_transformer_w4a4_b200 import svdq
        if c["op"] == "dense":
            svdq.dense_forward(st["a"], st["w"], st["y"], a_scale=st["a_scale"], w_scale=st["w_scale"],
                               bias=st["bias"], act=c["act"], gate=st["gate"], gate_rows=c["gate_rows"],
                               residual=st["residual"])
            return st["y"]
        if c["op"] == "rms":
            svdq.rms_quantize8(st["x"], st["codes"], st["scales"], residual=st["residual"], h=st["h"],
                               weight=st["weight"], norm=c["norm"])
            return [st["codes"], st["scales"]] + ([st["h"]] if c["residual"] else [])
        st["plan"].apply(st["q"], st["pos"], k=st["k"], q_out=st["q_out"], k_out=st["k_out"], inverse=c["inverse"])
        return [st["q_out"]] + ([st["k_out"]] if c["HK"] else [])
    return {"dense": _plain_dense, "rms": _plain_rms, "rope": _plain_rope}[c["op"]](st, c)


def _plain_dense(st, c):
    y = st["a"].float() @ st["w"].float().t()
    if st["a_scale"] is not None:
        y = y * st["a_scale"][:, None] * st["w_scale"][None, :]
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    elif c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    if st["gate"] is not None:
        y = y * st["gate"].float().repeat_interleave(c["gate_rows"], dim=0)[:c["M"]]
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(TORCH[c["out"]])


def _plain_rms(st, c):
    h = st["x"]
    if c["residual"]:
        h = (h.float() + st["residual"].float()).to(h.dtype)   # the norm is of the residual stream as it is stored
    v = h.float()
    t = v * st["weight"].float() if c["weight"] else v
    top = t.abs().amax(dim=1)
    rstd = 1.0 / torch.sqrt((v * v).mean(dim=1) + 1e-6) if c["norm"] else 1.0
    live = top >= TINY
    inv = torch.where(live, torch.full_like(top, TOP[c["out"]]) / top, 0.0)   # the norm cancels in the codes
    q = t * inv[:, None]
    q = q.round().to(torch.int8) if c["out"] == "int8" else q.to(torch.float8_e4m3fn)
    scales = torch.where(live, top * rstd / TOP[c["out"]], 0.0)
    return [q, scales] + ([h] if c["residual"] else [])


def _plain_rope(st, c):
    ang = st["pos"].double()[:, st["axis"]] * st["freq"]
    ang = ang.view(c["B"], c["S"], 1, -1)
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    if c["inverse"]:
        sin = -sin
    r = sum(_axes(c))

    def turn(x):
        v = x.float()
        o = v.clone()
        if c["interleaved"]:
            a, b = v[..., 0:r:2], v[..., 1:r:2]
            o[..., 0:r:2], o[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = v[..., : r // 2], v[..., r // 2: r]
            o[..., : r // 2], o[..., r // 2: r] = a * cos - b * sin, a * sin + b * cos
        return o.to(x.dtype)

    return [turn(st["q"])] + ([turn(st["k"])] if c["HK"] else [])


# --------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "dense":
        return _exact_dense(st, case)
    return _exact_rms(st, case) if case["op"] == "rms" else _exact_rope(st, case)


def _exact_dense(st, c):
    y = torch.empty(c["M"], c["N"], dtype=torch.float64, device="cuda")
    w = st["w"].double()
    if st["w_scale"] is not None:
        w *= st["w_scale"].double().unsqueeze(1)
    torch.mm(st["a"].double(), w.T, out=y)
    if st["a_scale"] is not None:
        y *= st["a_scale"].double().unsqueeze(1)
    if st["bias"] is not None:
        y += st["bias"].double()
    if c["act"] == "gelu":                        # x sigmoid(2 u), u = sqrt(2/pi) (x + 0.044715 x^3)
        y = y * torch.sigmoid(math.sqrt(8.0 / math.pi) * (y + 0.044715 * y ** 3))
    elif c["act"] == "silu":
        y = y * torch.sigmoid(y)
    if st["gate"] is not None:
        rows = torch.arange(c["M"], device="cuda") // c["gate_rows"]
        y *= st["gate"].double()[rows]
    if st["residual"] is not None:
        y += st["residual"].double()
    return y


def _exact_rms(st, c):
    h = st["x"].double()
    if c["residual"]:
        h = h + st["residual"].double()
    v = h.to(st["x"].dtype).double()              # as it is stored
    n = v
    if c["norm"]:
        n = n / torch.sqrt(v.square().sum(dim=1, keepdim=True) / c["K"] + 1e-6)
    if c["weight"]:
        n = n * st["weight"].double()
    s = n.abs().max(dim=1).values / TOP[c["out"]]
    q = n / torch.where(s > 0, s, 1.0).unsqueeze(1)
    q = torch.round(q).to(torch.int8) if c["out"] == "int8" else q.to(torch.float8_e4m3fn).double()
    return [q, s] + ([h] if c["residual"] else [])


def _exact_rope(st, c):
    pairs = []                                    # (axis, frequency) of every pair, in order
    axes = _axes(c)
    for a, d in enumerate(axes):
        for i in range(d // 2):
            pairs.append((a, c["theta"] ** (-2.0 * len(pairs) / sum(axes) if c["shared"] else -2.0 * i / d)))
    f = torch.zeros(len(axes), len(pairs), dtype=torch.float64)
    for p, (a, w) in enumerate(pairs):
        f[a, p] = w
    ang = (st["pos"].double().unsqueeze(-1) * f.cuda()).sum(dim=1).view(c["B"], c["S"], 1, len(pairs))
    turn = torch.polar(torch.ones_like(ang), -ang if c["inverse"] else ang)
    n = len(pairs)

    def rotated(x):
        o = x.double()
        z = o[..., : 2 * n]
        z = z.unflatten(-1, (n, 2)) if c["interleaved"] else z.unflatten(-1, (2, n)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, o[..., 2 * n:]], dim=-1)

    return [rotated(st["q"])] + ([rotated(st["k"])] if c["HK"] else [])


# --------------------------------------------------------------------- the work
def work(case):
    c = case
    if c["op"] == "dense":
        M, K, N = c["M"], c["K"], c["N"]
        b = SIZE[c["in"]] * (M * K + N * K) + SIZE[c["out"]] * M * N
        if SIZE[c["in"]] == 1:
            b += 4 * (M + N)
        b += SIZE[c["out"]] * (N * c["bias"] + M * N * c["residual"])
        if c["gate_rows"]:
            b += SIZE[c["out"]] * N * -(-M // c["gate_rows"])
        return {"bytes": b, "flops": 2 * M * N * K}
    if c["op"] == "rms":
        M, K, e = c["M"], c["K"], SIZE[c["in"]]
        b = M * K * (e + 1) + 4 * M + (2 * M * K * e if c["residual"] else 0) + (K * e if c["weight"] else 0)
        return {"bytes": b, "flops": 6 * M * K}
    tokens = c["B"] * c["S"]
    n = tokens * (c["H"] + c["HK"])
    return {"bytes": 2 * SIZE[c["in"]] * n * c["D"] + 4 * tokens * len(_axes(c)), "flops": 3 * n * sum(_axes(c))}
