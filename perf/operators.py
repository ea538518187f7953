"""What is measured of the products on 4-bit weights and 8-bit activation checkpoints, and how.

Formats.  A 4-bit weight matrix is R x C codes 0 .. 15, two to a byte along each row (even columns
in the low half), with a scale of the activations' type T for every `group` columns of a row and, where
the weights are not symmetric, a zero point; a code stands for the number of type T nearest to
(code - zero) * scale, zero 8 without zero points.  An 8-bit checkpoint is E4M3 codes with one exponent
byte for every 32 columns of a row; a code stands for e4m3(code) * 2^(exponent - 127), which is a number
of type T.

Operators: `linear` x . W^T (a layer's forward pass), `dgrad` dy . W (its input gradient), `w4` (weights
rounded to 4 bits, and the weights these stand for), `x8` (activations saved in 8 bits, and restored),
`wgrad` dy^T . x8 (a layer's weight gradient from the saved activations).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEVICE = "cuda"

# Exponents of an 8-bit group: the smallest one kept, such that every value is a number of type T, and
# the largest magnitude that rounds to a number of type T.
X8_MIN_EXP = {"bf16": -117, "f16": -15}
X8_LIMIT = {"bf16": 240.0 * 2.0 ** 120, "f16": 240.0 * 2.0 ** 8}


def listed():
    return [
        # one token through a square projection of a 7B-parameter decoder: the smallest call of a
        # serving loop, where latency counts
        dict(name="linear 1x4096x4096 bf16", op="linear", M=1, N=4096, K=4096, dtype="bf16", group=128, zeros=False,
             out="bf16", bias=False, act="none"),
        # a decoding batch of 16 through the wide half of a feed-forward block, with zero points and bias
        dict(name="linear 16x11008x4096 f16", op="linear", M=16, N=11008, K=4096, dtype="f16", group=64, zeros=True,
             out="f16", bias=True, act="none"),
        # a ragged layer: odd extents, the last group and the last byte of a row partly filled
        dict(name="linear 37x4097x1023 bf16", op="linear", M=37, N=4097, K=1023, dtype="bf16", group=32, zeros=True,
             out="f32", bias=False, act="relu"),
        # a prompt of 2048 tokens through the wide half of a feed-forward block, activation fused
        dict(name="linear 2048x11008x4096 bf16", op="linear", M=2048, N=11008, K=4096, dtype="bf16", group=128,
             zeros=True, out="bf16", bias=True, act="gelu"),
        # fine-tuning over frozen weights: the gradient of 2048 tokens through the same layer
        dict(name="dgrad 2048x4096x11008 bf16", op="dgrad", M=2048, N=11008, K=4096, dtype="bf16", group=128,
             zeros=True, out="bf16"),
        # a short ragged sequence's gradient
        dict(name="dgrad 300x1000x1030 f16", op="dgrad", M=300, N=1030, K=1000, dtype="f16", group=64, zeros=False,
             out="f32"),
        # weights of a square projection, and of the feed-forward block's wide half, rounded when a model is loaded
        dict(name="w4 4096x4096 bf16", op="w4", R=4096, C=4096, dtype="bf16", group=128, zeros=True),
        dict(name="w4 11008x4096 f16", op="w4", R=11008, C=4096, dtype="f16", group=32, zeros=False),
        # a layer's input kept for its backward pass: one sequence of 2K tokens, and four at the block's width
        dict(name="x8 2048x4096 bf16", op="x8", R=2048, C=4096, dtype="bf16"),
        dict(name="x8 8192x11008 f16", op="x8", R=8192, C=11008, dtype="f16"),
        # the weight gradient of a square projection over 2K tokens, and one with odd extents
        dict(name="wgrad 4096x4096x2048 bf16", op="wgrad", N=4096, K=4096, T=2048, dtype="bf16", out="f32"),
        dict(name="wgrad 1030x1023x4095 f16", op="wgrad", N=1030, K=1023, T=4095, dtype="f16", out="f32"),
    ]


def _spread(rng, low, high):
    """A whole number of low .. high, even over its logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "dgrad", "w4", "x8", "wgrad"])
    case = dict(op=op, dtype=rng.choice(["bf16", "f16"]))

    def width(low):
        # model widths are mostly multiples of 8; some are anything
        n = _spread(rng, low, 11008 if case["op"] != "wgrad" else 4096)
        return n if rng.random() < 0.4 else min(11008, -(-n // 8) * 8)

    if op in ("linear", "dgrad"):
        case.update(M=_spread(rng, 1, 2048), N=width(64), K=width(64), group=rng.choice([32, 64, 128]),
                    zeros=rng.random() < 0.5, out=rng.choice([case["dtype"], "f32"]))
        if case["N"] * case["K"] > 11008 * 4096:
            case["N"] = 4096
        if op == "linear":
            case.update(bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "gelu"]))
    elif op == "w4":
        case.update(R=_spread(rng, 64, 4096), C=width(64), group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
    elif op == "x8":
        case.update(R=_spread(rng, 1, 8192), C=width(64))
    else:
        case.update(N=width(64), K=width(64), T=_spread(rng, 1, 2048), out="f32")
    return case


def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _normal(gen, rows, cols, std, dtype):
    return (torch.randn(rows, cols, generator=gen, device=DEVICE) * std).to(DTYPES[dtype])


def _activations(gen, rows, cols, dtype):
    """N(0, 1), with some columns of ten times that, as the inputs of a decoder's layers have."""
    loud = 1.0 + 9.0 * (torch.rand(cols, generator=gen, device=DEVICE) < 0.005).float()
    return (torch.randn(rows, cols, generator=gen, device=DEVICE) * loud).to(DTYPES[dtype])


def _groups(x, group, fill=0.0):
    """x [rows, cols] as [rows, groups, group], the last group filled up."""
    rows, cols = x.shape
    pad = -cols % group
    if pad:
        x = torch.cat([x, x.new_full((rows, pad), fill)], 1)
    return x.reshape(rows, -1, group)


def _w4_codes(w, group, zeros):
    """Codes [rows, cols], scales and zero points of 16-bit weights, by the nearest step of each group.
    In 32 bits: quotients of two 16-bit numbers are never so near to a border that this matters."""
    rows, cols = w.shape
    v = _groups(w.float(), group)
    if zeros:
        low, high = v.amin(2).clamp(max=0.0), v.amax(2).clamp(min=0.0)
        scales = ((high - low) / 15.0).to(w.dtype)
    else:
        scales = (v.abs().amax(2) / 7.0).to(w.dtype)
    s = scales.float()
    some = s != 0.0
    by = torch.where(some, s, torch.ones_like(s))
    if zeros:
        points = torch.where(some, torch.round(-low / by).clamp(0.0, 15.0), torch.full_like(s, 8.0))
    else:
        points = torch.full_like(s, 8.0)
    q = torch.where(some[..., None], torch.round(v / by[..., None]), torch.zeros_like(v))
    codes = (q + points[..., None]).clamp(0.0, 15.0).to(torch.uint8)
    return codes.reshape(rows, -1)[:, :cols], scales, points.to(torch.uint8) if zeros else None


def _pack(codes):
    """Two codes to a byte, even columns in the low half."""
    if codes.shape[1] % 2:
        codes = torch.cat([codes, codes.new_zeros(codes.shape[0], 1)], 1)
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpack(packed, cols):
    return torch.stack([packed & 15, packed >> 4], 2).reshape(packed.shape[0], -1)[:, :cols]


def _w4_values(codes, scales, zeros, group, dtype):
    """The numbers of type T that codes [rows, cols] stand for."""
    points = 8.0 if zeros is None else zeros.float()[..., None]
    v = (_groups(codes.float(), group) - points) * scales.float()[..., None]
    return v.reshape(codes.shape[0], -1)[:, : codes.shape[1]].to(DTYPES[dtype])


def _x8_codes(x, dtype):
    """E4M3 codes (as their values) [rows, groups, 32] and exponents [rows, groups] of 16-bit activations:
    the smallest exponent at which the group's largest finite magnitude is within E4M3's 448."""
    v = _groups(x.float(), 32)
    fine = torch.isfinite(v)
    kept = torch.where(fine, v, torch.zeros_like(v)).clamp(-X8_LIMIT[dtype], X8_LIMIT[dtype])
    top = kept.abs().amax(2)
    fraction, power = torch.frexp(top)
    e = torch.where(top > 0.0, power - 9 + (fraction > 0.875).int(), X8_MIN_EXP[dtype]).clamp(min=X8_MIN_EXP[dtype])
    codes = torch.ldexp(kept, -e[..., None]).to(torch.float8_e4m3fn).float()
    return torch.where(fine, codes, torch.full_like(codes, float("nan"))), e


def _x8_values(codes, e, cols):
    return torch.ldexp(codes, e[..., None]).reshape(codes.shape[0], -1)[:, :cols]


def _activation(y, act):
    if act == "relu":
        return torch.clamp(y, min=0.0)
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return y


def prepare(case, seed):
    gen, op, dtype = _gen(seed), case["op"], case["dtype"]
    state = dict(case=case)
    if op in ("linear", "dgrad"):
        M, N, K = case["M"], case["N"], case["K"]
        codes, scales, zeros = _w4_codes(_normal(gen, N, K, 0.02, dtype), case["group"], case["zeros"])
        state.update(codes=_pack(codes), scales=scales, zeros=zeros)
        if op == "linear":
            state.update(x=_activations(gen, M, K, dtype))
            state.update(bias=torch.randn(N, generator=gen, device=DEVICE) * 0.1 if case["bias"] else None)
        else:
            state.update(x=_normal(gen, M, N, 1e-2, dtype))
        if own:  # the weight's handle, and memory that a program keeps for its layers' outputs and scratch
            import gemm_f32_amd as g
            w = g.W4(state["codes"], state["scales"], state["zeros"], case["group"], K)
            size = g.w4_workspace_size(w, M, transposed=op == "dgrad")
            state.update(w=w, to=torch.empty(M, N if op == "linear" else K, dtype=DTYPES[case["out"]], device=DEVICE),
                         workspace=torch.empty(size, dtype=torch.uint8, device=DEVICE))
    elif op == "w4":
        state.update(weights=_normal(gen, case["R"], case["C"], 0.02, dtype))
    elif op == "x8":
        state.update(x=_activations(gen, case["R"], case["C"], dtype))
    else:
        N, K, T = case["N"], case["K"], case["T"]
        codes, e = _x8_codes(_activations(gen, T, K, dtype), dtype)
        state.update(codes=codes.reshape(T, -1)[:, :K].to(torch.float8_e4m3fn).view(torch.uint8),
                     exponents=(e + 127).to(torch.uint8), dy=_normal(gen, T, N, 1e-2, dtype))
        if own:
            import gemm_f32_amd as g
            q = g.X8(state["codes"], state["exponents"], DTYPES[dtype])
            state.update(q=q, to=torch.empty(N, K, dtype=DTYPES[case["out"]], device=DEVICE),
                         workspace=torch.empty(g.x8_wgrad_workspace_size(q, N), dtype=torch.uint8, device=DEVICE))
    return state


def _own(state):
    import gemm_f32_amd as g
    case = state["case"]
    if case["op"] == "linear":
        return g.w4_linear(state["x"], state["w"], bias=state["bias"], activation=g.Act[case["act"].upper()],
                           out=state["to"], workspace=state["workspace"])
    if case["op"] == "dgrad":
        return g.w4_dgrad(state["x"], state["w"], out=state["to"], workspace=state["workspace"])
    if case["op"] == "w4":
        w = g.w4_quantize(state["weights"], case["group"], zero_points=case["zeros"])
        return g.w4_dequantize(w), w.scales
    if case["op"] == "x8":
        q = g.x8_quantize(state["x"])
        return g.x8_dequantize(q), q.exponents
    return g.x8_wgrad(state["dy"], state["q"], out=state["to"], workspace=state["workspace"])


def _plain(state):
    case = state["case"]
    op, dtype = case["op"], case["dtype"]
    if op in ("linear", "dgrad"):
        codes = _unpack(state["codes"], case["K"])
        w = _w4_values(codes, state["scales"], state["zeros"], case["group"], dtype).float()
        if op == "dgrad":
            return (state["x"].float() @ w).to(DTYPES[case["out"]])
        y = state["x"].float() @ w.t()
        if state["bias"] is not None:
            y = y + state["bias"]
        return _activation(y, case["act"]).to(DTYPES[case["out"]])
    if op == "w4":
        codes, scales, zeros = _w4_codes(state["weights"], case["group"], case["zeros"])
        return _w4_values(_unpack(_pack(codes), case["C"]), scales, zeros, case["group"], dtype), scales
    if op == "x8":
        codes, e = _x8_codes(state["x"], dtype)
        return _x8_values(codes, e, case["C"]).to(DTYPES[dtype]), (e + 127).to(torch.uint8)
    codes = _groups(state["codes"].view(torch.float8_e4m3fn).float(), 32)
    x = _x8_values(codes, state["exponents"].int() - 127, case["K"])
    return (state["dy"].float().t() @ x).to(DTYPES[case["out"]])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """Each input read once, each output written once; of the round trips (w4, x8) the codes are written and read."""
    bits = {"bf16": 2, "f16": 2, "f32": 4}

    def packed(rows, cols):
        groups = -(-cols // case["group"])
        return rows * ((cols + 1) // 2 + groups * (2 + (1 if case["zeros"] else 0)))

    if case["op"] in ("linear", "dgrad"):
        M, N, K = case["M"], case["N"], case["K"]
        to, of = (N, K) if case["op"] == "linear" else (K, N)
        return dict(bytes=packed(N, K) + 2 * M * of + bits[case["out"]] * M * to + (4 * N if case.get("bias") else 0),
                    flops=2 * M * N * K)
    if case["op"] == "w4":
        return dict(bytes=4 * case["R"] * case["C"] + 2 * packed(case["R"], case["C"]), flops=4 * case["R"] * case["C"])
    if case["op"] == "x8":
        return dict(bytes=4 * case["R"] * case["C"] + 2 * case["R"] * (case["C"] + -(-case["C"] // 32)),
                    flops=4 * case["R"] * case["C"])
    N, K, T = case["N"], case["K"], case["T"]
    return dict(bytes=T * (K + -(-K // 32)) + 2 * T * N + bits[case["out"]] * N * K, flops=2 * N * K * T)


def _nearest(v, fraction_bits, least):
    """v in 64 bits at the nearest number of fraction_bits + 1 binary digits, ties to even, with no step
    below 2^least."""
    _, power = torch.frexp(v)
    step = torch.exp2((power - 1 - fraction_bits).clamp(min=least).double())
    return torch.round(v / step) * step


def _number(v, dtype):
    return _nearest(v, 7, -133) if dtype == "bf16" else _nearest(v, 10, -24)


def exact(case, seed):
    state = prepare(case, seed)
    op, dtype = case["op"], case["dtype"]
    if op in ("linear", "dgrad"):
        at = torch.arange(case["K"], device=DEVICE)
        byte = state["codes"][:, at // 2].long()
        code = torch.where(at % 2 == 0, byte % 16, byte // 16).double()
        zero = 8.0 if state["zeros"] is None else state["zeros"][:, at // case["group"]].double()
        w = _number((code - zero) * state["scales"][:, at // case["group"]].double(), dtype)
        if op == "dgrad":
            return torch.mm(state["x"].double(), w)
        y = torch.mm(state["x"].double(), w.t().contiguous())
        if state["bias"] is not None:
            y = y + state["bias"].double()
        if case["act"] == "relu":
            y = torch.where(y > 0.0, y, torch.zeros_like(y))
        if case["act"] == "gelu":
            y = y * torch.erfc(-y / math.sqrt(2.0)) / 2.0
        return y
    if op == "w4":
        w, group = state["weights"].double(), case["group"]
        values, scales = torch.empty_like(w), []
        for c in range(0, w.shape[1], group):
            part = w[:, c:c + group]
            if case["zeros"]:
                low, high = part.min(1).values.clamp(max=0.0), part.max(1).values.clamp(min=0.0)
                s = _number((high - low) / 15.0, dtype)
            else:
                s = _number(part.abs().max(1).values / 7.0, dtype)
            by = torch.where(s == 0.0, torch.ones_like(s), s)
            zero = torch.round(-low / by).clamp(0.0, 15.0) if case["zeros"] else torch.full_like(s, 8.0)
            code = (torch.round(part / by[:, None]) + zero[:, None]).clamp(0.0, 15.0)
            values[:, c:c + group] = _number((code - zero[:, None]) * s[:, None], dtype)
            scales.append(s)
        return values, torch.stack(scales, 1)
    if op == "x8":
        x = state["x"].double()
        values, exponents = torch.empty_like(x), []
        for c in range(0, x.shape[1], 32):
            part = x[:, c:c + 32].clamp(-X8_LIMIT[dtype], X8_LIMIT[dtype])
            top = part.abs().max(1).values
            e = torch.ceil(torch.log2(top / 448.0)).clamp(min=X8_MIN_EXP[dtype])
            e = e - (top <= 448.0 * torch.exp2(e - 1.0)).double() * (e > X8_MIN_EXP[dtype]).double()
            e = e + (top > 448.0 * torch.exp2(e)).double()
            unit = torch.exp2(e)[:, None]
            values[:, c:c + 32] = _nearest(part / unit, 3, -9) * unit
            exponents.append(e + 127.0)
        return values, torch.stack(exponents, 1).to(torch.uint8)
    at = torch.arange(case["K"], device=DEVICE)
    bits = state["codes"].long()
    size, fraction = bits // 8 % 16, bits % 8
    x = torch.where(size == 0, fraction.double() * 2.0 ** -9, (1.0 + fraction.double() / 8.0) * torch.exp2(size.double() - 7.0))
    x = torch.where(bits >= 128, -x, x) * torch.exp2(state["exponents"][:, at // 32].double() - 127.0)
    return torch.mm(state["dy"].double().t().contiguous(), x)
