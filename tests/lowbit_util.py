"""Plain float64 versions of the low-bit operands' definitions, for the tests."""
import numpy as np
import torch

import gemm_f32_amd as g

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
OUTS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
X8_MIN_EXP = {"bf16": -117, "f16": -15}
X8_LIMIT = {"bf16": 240.0 * 2.0 ** 120, "f16": 240.0 * 2.0 ** 8}


def to_type(v, dtype):
    """float64 -> the nearest T (as a torch tensor), ties to even, by numpy's own fp16 conversion or, for bf16,
    by rounding to 8 binary digits: every intermediate step is exact in float64."""
    v = np.asarray(v, dtype=np.float64)
    if dtype == "f16":
        with np.errstate(over="ignore"):
            return torch.from_numpy(v.astype(np.float16))
    _, power = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(power - 8, -133))
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.where(np.isfinite(v), np.rint(v / step) * step, v)
        r = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, r), r)
    return torch.from_numpy(r.astype(np.float32)).to(torch.bfloat16)      # a bf16 number: exact


def w4_reference(w, group, zeros, dtype):
    """(codes, scales, zeros) of a 16-bit matrix by the definition, in float64."""
    v = w.double().cpu().numpy()
    rows, cols = v.shape
    groups = -(-cols // group)
    codes = np.zeros((rows, cols), np.uint8)
    scales = torch.empty((rows, groups), dtype=DTYPES[dtype])
    points = np.zeros((rows, groups), np.uint8)
    for i in range(groups):
        part = v[:, i * group:(i + 1) * group]
        bad = ~np.isfinite(part).all(1)
        p = np.where(bad[:, None], 0.0, part)
        lo, hi = np.minimum(p.min(1), 0.0), np.maximum(p.max(1), 0.0)
        # the quotient is formed in FP32; its rounding to T is to_type's (see the C header)
        raw = (np.float32(hi) - np.float32(lo)) / np.float32(15.0) if zeros else \
            np.float32(np.abs(p).max(1)) / np.float32(7.0)
        s = to_type(raw, dtype)
        sv = s.double().numpy()
        some = (sv != 0.0) & ~bad
        by = np.where(some, sv, 1.0)
        z = np.where(some, np.clip(np.rint(-lo / by), 0, 15), 8.0) if zeros else np.full(rows, 8.0)
        q = np.where(some[:, None], np.rint(p / by[:, None]), 0.0)
        codes[:, i * group:(i + 1) * group] = np.clip(q + z[:, None], 0, 15)
        scales[:, i] = torch.where(torch.from_numpy(bad), torch.tensor(float("nan"), dtype=s.dtype), s)
        points[:, i] = z
    return codes, scales, points if zeros else None


def pack(codes):
    rows, cols = codes.shape
    c = np.zeros((rows, (cols + 1) // 2 * 2), np.uint8)
    c[:, :cols] = codes
    return c[:, 0::2] | (c[:, 1::2] << 4)


def w4_values(codes, scales, zeros, group, dtype):
    """The T (as torch, CPU) that codes (rows, cols) stand for."""
    at = np.arange(codes.shape[1]) // group
    s = scales.double().cpu().numpy()[:, at]
    z = 8.0 if zeros is None else np.asarray(zeros, dtype=np.float64)[:, at]
    return to_type((codes.astype(np.float64) - z) * s, dtype)


def x8_reference(x, dtype):
    """(values (float64, NaN where not finite), exponents) of a 16-bit matrix."""
    v = x.double().cpu().numpy()
    rows, cols = v.shape
    groups = -(-cols // 32)
    out, exps = np.empty_like(v), np.empty((rows, groups), np.int64)
    for i in range(groups):
        part = v[:, 32 * i:32 * i + 32]
        fine = np.isfinite(part)
        p = np.clip(np.where(fine, part, 0.0), -X8_LIMIT[dtype], X8_LIMIT[dtype])
        top = np.abs(p).max(1)
        e = np.full(rows, X8_MIN_EXP[dtype])
        for _ in range(300):                     # the smallest e from the least on with top <= 448 2^e
            e = np.where(top > 448.0 * np.exp2(e.astype(np.float64)), e + 1, e)
        q = p / np.exp2(e.astype(np.float64))[:, None]
        _, power = np.frexp(q)
        step = np.exp2(np.maximum(power - 4, -9).astype(np.float64))
        q = np.rint(q / step) * step
        out[:, 32 * i:32 * i + 32] = np.where(fine, q * np.exp2(e.astype(np.float64))[:, None], np.nan)
        exps[:, i] = e + 127
    return out, exps.astype(np.uint8)


E4M3 = np.array([((-1.0) ** (b >> 7)) * ((b & 7) * 2.0 ** -9 if (b >> 3) & 15 == 0 else
                                         (1 + (b & 7) / 8) * 2.0 ** (((b >> 3) & 15) - 7)) if b & 127 != 127
                 else np.nan for b in range(256)])


def gelu64(y):
    return 0.5 * y * torch.erfc(-y * 0.5 ** 0.5)


def sum_bound(k, d):
    """Bound of the error of a sum of k exact products in FP32, in any order: k - 1 additions, each within
    2^-24 of a partial sum that is at most the sum d of the magnitudes; 16 more for the epilogue's steps."""
    return (k + 16) * 2.0 ** -24 * d


def check_close(got, ref, bound):
    """|got - ref| <= bound + the rounding to got's type (half a step: eps / 2 of the value, or half of the
    type's smallest number), everywhere; non-finite where and as the reference is."""
    r = ref.to(got.device)
    fine = torch.isfinite(r)
    assert torch.equal(torch.isnan(got), torch.isnan(r))
    inf = torch.isinf(r)
    assert torch.equal(got[inf].double(), r[inf])
    info = torch.finfo(got.dtype)
    b = bound.to(got.device) + info.eps / 2 * (r.abs() + bound.to(got.device)) + info.smallest_normal * info.eps / 2
    over = ((got.double() - r).abs() > b) & fine
    assert not over.any(), (f"{int(over.sum())} of {got.numel()} outside, worst "
                            f"{float(((got.double() - r).abs() / b)[fine].max()):.3g} of the bound")


def make_w4(rows, cols, dtype, group, zeros, seed, pad=0, odd_high=True):
    """A random W4 on the GPU with padded rows, and the matrix it stands for (float64, CPU).  The half byte
    past an odd row's end and the padding hold codes that must not matter."""
    rng = np.random.default_rng([seed, rows, cols])
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    groups, width = -(-cols // group), (cols + 1) // 2
    scales = to_type(rng.uniform(0.5, 2.0, (rows, groups)) * 0.02, dtype)
    z = rng.integers(0, 16, (rows, groups)).astype(np.uint8) if zeros else None
    p = pack(codes)
    if odd_high and cols % 2:
        p[:, -1] |= 15 << 4
    buf = np.full((rows, width + pad), 0xa5, np.uint8)
    buf[:, :width] = p
    sbuf = torch.full((rows, groups + pad), float("nan"), dtype=DTYPES[dtype])
    sbuf[:, :groups] = scales
    w = g.W4(torch.from_numpy(buf).cuda()[:, :width], sbuf.cuda()[:, :groups],
             torch.from_numpy(z).cuda() if zeros else None, group, cols)
    return w, w4_values(codes, scales, z, group, dtype).double()
