"""4-bit weights and 8-bit activation checkpoints against their definitions in float64."""
import numpy as np
import pytest
import torch

import gemm_f32_amd as g
from lowbit_util import (DTYPES, E4M3, OUTS, check_close, gelu64, make_w4, pack, sum_bound, to_type, w4_reference,
                         w4_values, x8_reference)

pytestmark = pytest.mark.gpu

BOTH = ["bf16", "f16"]


def say(*a):
    print("[gpu]", *a, flush=True)


def randn(rows, cols, dtype, seed, scale=1.0, pad=0):
    """A (rows, cols) view of a matrix of cols + pad columns whose padding is NaN."""
    gen = torch.Generator().manual_seed(seed)
    t = torch.full((rows, cols + pad), float("nan"), dtype=DTYPES[dtype])
    t[:, :cols] = (torch.randn(rows, cols, generator=gen) * scale).to(DTYPES[dtype])
    return t.cuda()[:, :cols]


# ---- rounding weights to 4 bits ------------------------------------------------------------
W4_SHAPES = [(1, 1), (3, 31), (5, 32), (2, 33), (7, 128), (4, 1000), (9, 1023), (130, 257), (6, 2056)]


@pytest.mark.parametrize("shape", W4_SHAPES, ids=str)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", BOTH)
def test_w4_quantize_is_the_definition(dtype, group, zeros, shape):
    rows, cols = shape
    w = randn(rows, cols, dtype, 1, 0.02, pad=3)
    say("w4_quantize", dtype, group, zeros, shape)
    q = g.w4_quantize(w, group, zero_points=zeros)
    codes, scales, points = w4_reference(w, group, zeros, dtype)
    assert g.gemm_last_kernel() == f"{dtype}_w4_quantize"
    assert torch.equal(q.codes.cpu(), torch.from_numpy(pack(codes)))
    assert torch.equal(q.scales.cpu().view(torch.int16), scales.view(torch.int16))
    assert (q.zeros is None) == (points is None)
    if zeros:
        assert torch.equal(q.zeros.cpu(), torch.from_numpy(points))
    v = g.w4_dequantize(q)
    assert torch.equal(v.cpu().view(torch.int16), w4_values(codes, scales, points, group, dtype).view(torch.int16))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", BOTH)
def test_w4_quantize_special_groups(dtype, zeros):
    """Groups of zeros, of numbers too small for a scale, of one sign, of one value, with an infinity or a NaN,
    and of the type's largest numbers; the padding between rows stays as it was."""
    big = torch.finfo(DTYPES[dtype]).max
    tiny = torch.finfo(DTYPES[dtype]).smallest_normal * torch.finfo(DTYPES[dtype]).eps
    rows = [torch.zeros(64), torch.full((64,), tiny), torch.full((64,), -3.0), torch.linspace(0.1, 1.0, 64),
            -torch.linspace(0.1, 1.0, 64), torch.tensor([float("inf")] + [1.0] * 63),
            torch.tensor([1.0] * 40 + [float("nan")] * 24), torch.tensor([-float("inf")] * 64),
            torch.tensor([big] * 64), torch.tensor([big / 4, -big / 4] * 32), torch.tensor([0.0, -0.0] * 32)]
    w = torch.stack(rows).to(DTYPES[dtype]).cuda()
    codes, scales, points = w4_reference(w, 32, zeros, dtype)
    n = w.shape[0]
    cbuf = torch.full((n, 35), 0x5a, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((n, 3), 7.0, dtype=w.dtype, device="cuda")
    zbuf = torch.full((n, 4), 0x5a, dtype=torch.uint8, device="cuda") if zeros else None
    q = g.W4(cbuf[:, :32], sbuf[:, :2], zbuf[:, :2] if zeros else None, 32, 64)
    say("w4_quantize special", dtype, zeros)
    g.w4_quantize(w, 32, zero_points=zeros, out=q)
    assert torch.equal(cbuf[:, :32].cpu(), torch.from_numpy(pack(codes)))
    s = sbuf[:, :2].cpu()
    assert torch.equal(torch.isnan(s), torch.isnan(scales)) and torch.equal(torch.nan_to_num(s), torch.nan_to_num(scales))
    assert (cbuf[:, 32:] == 0x5a).all() and (sbuf[:, 2:] == 7.0).all()
    if zeros:
        assert torch.equal(zbuf[:, :2].cpu(), torch.from_numpy(points)) and (zbuf[:, 2:] == 0x5a).all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", BOTH)
def test_w4_quantize_every_magnitude(dtype, zeros):
    """Groups of every power of two that the type has, ties between two codes among their quotients, and a
    range whose width is past the type's largest number (an infinite scale)."""
    powers = torch.arange(-133, 127) if dtype == "bf16" else torch.arange(-24, 15)
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(len(powers), 64, generator=gen)
    x[:, 32:] = torch.arange(-16, 16) / 2.0          # scale 8/7 or 1: quotients at borders
    x[:, 63] = torch.where(torch.arange(len(powers)) % 2 == 0, 7.0, 7.5)
    w = torch.ldexp(x, powers[:, None] - 3).to(DTYPES[dtype])
    big = torch.finfo(w.dtype).max
    w = torch.cat([w, torch.tensor([big, -big] * 32)[None].to(w.dtype)]).cuda()
    say("w4_quantize magnitudes", dtype, zeros)
    q = g.w4_quantize(w, 32, zero_points=zeros)
    with np.errstate(over="ignore"):
        codes, scales, points = w4_reference(w, 32, zeros, dtype)
    assert torch.equal(q.scales.cpu().view(torch.int16), scales.view(torch.int16))
    assert torch.equal(q.codes.cpu(), torch.from_numpy(pack(codes)))
    if zeros:
        assert torch.equal(q.zeros.cpu(), torch.from_numpy(points))


@pytest.mark.parametrize("dtype", BOTH)
def test_w4_dequantize_every_code_and_zero_point(dtype):
    """All 16 codes by all 256 zero points, scales of every sign and size (subnormal results among them)."""
    rng = np.random.default_rng(2)
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 4))[:, :63]
    z = np.stack([np.arange(256), rng.integers(0, 256, 256)], 1).astype(np.uint8)
    s = to_type(rng.standard_normal((256, 2)) * np.exp2(rng.uniform(-22, 8, (256, 2))), dtype)
    s[3, 0] = float("nan")
    w = g.W4(torch.from_numpy(pack(codes)).cuda(), s.cuda(), torch.from_numpy(z).cuda(), 32, 63)
    out = torch.full((256, 70), 5.0, dtype=DTYPES[dtype], device="cuda")
    g.w4_dequantize(w, out=out[:, :63])
    ref = w4_values(codes, s, z, 32, dtype)
    got = out[:, :63].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(torch.nan_to_num(got, 9.0), torch.nan_to_num(ref, 9.0))
    assert (out[:, 63:] == 5.0).all()


# ---- products on 4-bit weights ----------------------------------------------------------------
# (M, stored rows of W, stored columns): one element, one row, odd extents, several blocks, K shorter than a
# group, a wavefront's step and its remainders, more rows than one block
PRODUCTS = [(1, 1, 1), (1, 17, 64), (1, 300, 1000), (2, 64, 31), (5, 33, 129), (16, 48, 256), (17, 100, 1023),
            (31, 130, 640), (33, 65, 127), (64, 128, 1152), (65, 50, 161), (130, 257, 383), (3, 8, 2048), (300, 400, 520),
            (600, 300, 257)]


def product_reference(x, wv, tr, alpha=1.0, beta=0.0, old=None, bias=None, act="none"):
    """(result, bound of its FP32 error), float64."""
    b = wv if tr else wv.t()
    y, d = alpha * (x @ b), abs(alpha) * (x.abs() @ b.abs())
    if beta != 0.0:
        y, d = y + beta * old, d + abs(beta) * old.abs()
    if bias is not None:
        y, d = y + bias, d + bias.abs()
    bound = sum_bound(x.shape[1], d)
    if act == "relu":
        y = torch.clamp(y, min=0.0)
    elif act == "gelu":      # |gelu'| < 1.13; the kernel's erf is within 5e-7 |x| of it, and 8 roundings
        y, bound = gelu64(y), 1.13 * bound + (5e-7 + 8 * 2.0 ** -24) * y.abs()
    return y, bound


def check_product(M, rows, cols, dtype, group, zeros, tr, out, seed, pad=0, workspace="none", **epi):
    w, wv = make_w4(rows, cols, dtype, group, zeros, seed, pad)
    k, n = (rows, cols) if tr else (cols, rows)
    x = randn(M, k, dtype, seed + 1, pad=pad)
    gen = torch.Generator().manual_seed(seed + 2)
    buf = torch.randn(M, n + pad, generator=gen).to(OUTS[out]).cuda()
    old = buf.clone()
    bias = torch.randn(n, generator=gen).cuda() if epi.get("bias") else None
    alpha, beta, act = epi.get("alpha", 1.0), epi.get("beta", 0.0), epi.get("act", "none")
    if beta == 0.0:
        buf[:, :n] = float("nan")
    ws = {"none": torch.empty(0, dtype=torch.uint8, device="cuda"), "own": None}[workspace]
    say("w4", dtype, f"group={group} zeros={zeros} tr={tr} M={M} W={rows}x{cols} out={out} pad={pad} ws={workspace}", epi)
    if tr:
        g.w4_dgrad(x, w, alpha=alpha, beta=beta, out=buf[:, :n], workspace=ws)
    else:
        g.w4_linear(x, w, bias=bias, activation=g.Act[act.upper()], alpha=alpha, beta=beta, out=buf[:, :n], workspace=ws)
    ref, bound = product_reference(x.cpu().double(), wv, tr, alpha, beta, old[:, :n].cpu().double(),
                                   bias.cpu().double() if bias is not None else None, act)
    check_close(buf[:, :n], ref, bound)
    assert torch.equal(buf[:, n:], old[:, n:]), "written past the rows of C"
    return buf[:, :n]


@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
@pytest.mark.parametrize("tr", [False, True], ids=["linear", "dgrad"])
@pytest.mark.parametrize("dtype", BOTH)
def test_w4_product(dtype, tr, shape):
    M, rows, cols = shape
    for i, (group, zeros, out, pad) in enumerate([(32, True, "f32", 0), (64, False, dtype, 3), (128, True, "f32", 8)]):
        check_product(M, rows, cols, dtype, group, zeros, tr, out, 10 + i, pad)
    short = (rows if tr else cols) < 32 or (tr and cols < 32)
    kernel = "w4_short" if short else "w4_tile_t" if tr else "w4_few" if M <= 16 else "w4_tile"
    assert g.gemm_last_kernel() == f"{dtype}_{kernel}"


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("tr", [False, True], ids=["linear", "dgrad"])
def test_w4_product_with_k_split_over_workgroups(dtype, tr):
    """With the workspace, few tiles of C take K in slices whose sums are added in order: the last slice
    shorter, K odd, every output type and step of the epilogue; with a workspace too small the call runs
    without the split."""
    for M, rows, cols, group, out, epi in [(17, 130, 2051, 32, "f32", {}), (33, 257, 4096, 128, dtype, dict(bias=True)),
                                           (64, 100, 2049, 64, "f32", dict(alpha=0.5, beta=-1.0, bias=True, act="gelu")),
                                           (200, 65, 1900, 32, "f16", dict(act="relu")), (500, 33, 4001, 64, "bf16", {})]:
        if tr:                             # (no bias and no activation)
            rows, cols, epi = cols, rows, {k: v for k, v in epi.items() if k in ("alpha", "beta")}
        check_product(M, rows, cols, dtype, group, True, tr, out, 40, pad=1, workspace="own", **epi)
        assert g.gemm_last_kernel() == f"{dtype}_w4_tile{'_t' if tr else ''}_splitk", (M, rows, cols)
    n, k = 130, 2051
    w, _ = make_w4(k if tr else n, n if tr else k, dtype, 32, False, 3)
    x = randn(17, k, dtype, 4)
    size = g.w4_workspace_size(w, 17, transposed=tr)
    assert size > 0 and size % (17 * n * 4) == 0
    small = torch.full((size,), 0x3f, dtype=torch.uint8, device="cuda")
    y = (g.w4_dgrad if tr else g.w4_linear)(x, w, workspace=small[:size - 16])
    assert g.gemm_last_kernel() == f"{dtype}_w4_tile{'_t' if tr else ''}" and (small == 0x3f).all()
    check_close(y, *product_reference(x.cpu().double(), g.w4_dequantize(w).cpu().double(), tr))


@pytest.mark.parametrize("epi", [dict(bias=True, act="relu"), dict(bias=True, act="gelu"), dict(alpha=-0.5, beta=2.0),
                                 dict(beta=1.0, bias=True), dict(alpha=0.0, beta=0.5, act="gelu")], ids=str)
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", BOTH)
def test_w4_linear_epilogue(dtype, out, epi):
    for shape in [(1, 130, 257), (20, 64, 512), (70, 90, 96)]:
        check_product(*shape, dtype, 64, True, False, out, 20, pad=1, **epi)


# enough columns for 1, 2, 3 and 4 column blocks a workgroup (4096 columns are one round of 256 CUs), few and many
# rows, K of one step, of several and of enough for 16 wavefronts a workgroup
FEW = [(1, 4112, 128), (4, 8208, 257), (5, 4112, 160), (16, 4112, 640), (16, 8208, 128), (9, 8208, 1023), (16, 12304, 96),
       (12, 12304, 300), (3, 4096, 8192), (16, 1000, 8200), (2, 5000, 11008)]


@pytest.mark.parametrize("shape", FEW, ids=str)
@pytest.mark.parametrize("dtype", BOTH)
def test_w4_linear_of_few_rows_and_many_columns(dtype, shape):
    M, rows, cols = shape
    for group, zeros, out in [(32, True, "f32"), (128, False, dtype)]:
        check_product(M, rows, cols, dtype, group, zeros, False, out, 50)
        assert g.gemm_last_kernel() == f"{dtype}_w4_few"


# (M, N, K) for which W is written as 16-bit numbers first, with a workspace for them
MANY = [(2100, 1001, 131), (1100, 2051, 136), (9000, 257, 131)]


@pytest.mark.parametrize("tr", [False, True], ids=["linear", "dgrad"])
@pytest.mark.parametrize("dtype", BOTH)
def test_w4_product_of_many_rows(dtype, tr):
    """With and without the workspace; odd extents, so that rows of the workspace are padded."""
    for (M, n, k), out, epi in zip(MANY, ["f32", dtype, "f16"], [{}, dict(alpha=0.5, beta=1.0), dict(beta=-1.0)]):
        rows, cols = (k, n) if tr else (n, k)
        check_product(M, rows, cols, dtype, 32, True, tr, out, 30, workspace="own", **epi)
        assert "_dma" in g.gemm_last_kernel()
        check_product(M, rows, cols, dtype, 32, True, tr, out, 30, workspace="none", **epi)
        assert g.gemm_last_kernel() == f"{dtype}_w4_tile" + ("_t" if tr else "")


@pytest.mark.parametrize("dtype", BOTH)
def test_w4_linear_of_many_rows_with_bias_and_activation(dtype):
    for act in ("none", "relu", "gelu"):
        check_product(2100, 1001, 131, dtype, 128, False, False, dtype, 31, workspace="own", bias=True, act=act)
        assert "_dma" in g.gemm_last_kernel()


@pytest.mark.parametrize("tr", [False, True], ids=["linear", "dgrad"])
@pytest.mark.parametrize("dtype", BOTH)
def test_w4_product_is_exact_on_small_integers(dtype, tr):
    """Integers whose sums FP32 holds exactly: every kernel gives the same bits."""
    rng = np.random.default_rng(5)
    for M, rows, cols in [(1, 70, 300), (40, 33, 640), (600, 130, 136), (1600, 900, 400)]:
        codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
        groups = -(-cols // 32)
        s = to_type(2.0 ** rng.integers(-1, 2, (rows, groups)), dtype)
        z = rng.integers(0, 16, (rows, groups)).astype(np.uint8)
        w = g.W4(torch.from_numpy(pack(codes)).cuda(), s.cuda(), torch.from_numpy(z).cuda(), 32, cols)
        wv = w4_values(codes, s, z, 32, dtype).double()
        x = torch.from_numpy(rng.integers(-4, 5, (M, rows if tr else cols))).to(DTYPES[dtype])
        ref = x.double() @ (wv if tr else wv.t())
        for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
            y = (g.w4_dgrad if tr else g.w4_linear)(x.cuda(), w, workspace=ws)
            assert torch.equal(y.cpu().double(), ref), (M, rows, cols, g.gemm_last_kernel())


@pytest.mark.parametrize("tr", [False, True], ids=["linear", "dgrad"])
def test_w4_product_with_non_finite_values(tr):
    """A NaN scale reaches only the outputs of its group, an infinite activation only its row; what lies past a
    row's end (NaN scales in the padding) reaches nothing."""
    rows, cols, M = 40, 100, 6
    w, wv = make_w4(rows, cols, "bf16", 32, True, 7, pad=2)
    w.scales[5, 1] = float("nan")
    wv[5, 32:64] = float("nan")
    x = randn(M, rows if tr else cols, "bf16", 8)
    x[2, 7] = float("inf")
    y = (g.w4_dgrad if tr else g.w4_linear)(x, w)
    ref = x.cpu().double() @ (wv if tr else wv.t())
    got = y.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf].double(), ref[inf])


def test_w4_empty_products():
    w, _ = make_w4(40, 64, "bf16", 32, False, 9)
    assert g.w4_linear(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w).shape == (0, 40)
    none = g.W4(torch.empty(0, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.bfloat16, device="cuda"),
                None, 32, 64)
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    assert g.w4_linear(x, none).shape == (3, 0)
    out = torch.full((3, 64), 2.0, device="cuda")
    g.w4_dgrad(torch.empty(3, 0, dtype=torch.bfloat16, device="cuda"), none, beta=0.5, out=out)
    assert (out == 1.0).all()
    q = g.w4_quantize(torch.empty(0, 64, dtype=torch.float16, device="cuda"), 32)
    assert g.w4_dequantize(q).shape == (0, 64)


def test_w4_far_offsets():
    """Rows of codes, activations and C more than 2^31 elements from their starts."""
    rows, cols = 2100, 64
    buf = torch.empty(rows << 20, dtype=torch.uint8, device="cuda")
    far = buf.as_strided((rows, cols // 2), (1 << 20, 1))
    w, wv = make_w4(rows, cols, "bf16", 32, False, 11)
    far.copy_(w.codes)
    f = g.W4(far, w.scales, None, 32, cols)
    x = randn(3, cols, "bf16", 12)
    say("w4 far offsets")
    assert torch.equal(g.w4_linear(x, f), g.w4_linear(x, w))
    dy = randn(2, rows, "bf16", 13)
    assert torch.equal(g.w4_dgrad(dy, f), g.w4_dgrad(dy, w))
    assert torch.equal(g.w4_dequantize(f), g.w4_dequantize(w))
    del buf, far, f
    wide = torch.empty(3 << 30, dtype=torch.bfloat16, device="cuda")
    xs, out = wide.as_strided((3, cols), (1 << 30, 1)), wide[1024:].as_strided((3, rows), (1 << 30, 1))
    xs.copy_(x)
    g.w4_linear(xs, w, out=out)
    ref, bound = product_reference(x.cpu().double(), wv, False)
    check_close(out, ref, bound)


# ---- activations in 8 bits --------------------------------------------------------------------
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (2, 32), (5, 33), (4, 257), (7, 1000), (130, 64), (3, 2056)], ids=str)
@pytest.mark.parametrize("dtype", BOTH)
def test_x8_round_trip_is_the_definition(dtype, shape):
    x = randn(*shape, dtype, 3, 5.0, pad=5)
    say("x8", dtype, shape)
    q = g.x8_quantize(x)
    assert g.gemm_last_kernel() == f"{dtype}_x8_quantize"
    values, exps = x8_reference(x, dtype)
    assert torch.equal(q.exponents.cpu(), torch.from_numpy(exps))
    out = torch.full((shape[0], shape[1] + 3), 7.0, dtype=DTYPES[dtype], device="cuda")
    g.x8_dequantize(q, out=out[:, :shape[1]])
    assert torch.equal(out[:, :shape[1]].cpu().double(), torch.from_numpy(values))
    assert (out[:, shape[1]:] == 7.0).all()


@pytest.mark.parametrize("dtype", BOTH)
def test_x8_every_number(dtype):
    """Every 16-bit pattern, once as the only number of its group (so that every magnitude is a group's largest) and
    once among its neighbours."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DTYPES[dtype])
    alone = torch.zeros(65536, 32, dtype=DTYPES[dtype])
    alone[:, 5] = bits
    mixed = bits[torch.randperm(65536, generator=torch.Generator().manual_seed(1))].view(2048, 32)
    for x in (alone, bits.view(2048, 32), mixed):
        q = g.x8_quantize(x.cuda())
        values, exps = x8_reference(x, dtype)
        assert torch.equal(q.exponents.cpu(), torch.from_numpy(exps))
        got = g.x8_dequantize(q).cpu().double().numpy()
        assert np.array_equal(got, values, equal_nan=True)
        assert np.array_equal(np.signbit(got[~np.isnan(values)]), np.signbit(x.double().numpy()[~np.isnan(values)]))
        # what the format promises: within 2^-4 of the value or half of the smallest step, where not held at the limit
        v = x.double().numpy()
        ok = np.isfinite(v) & (np.abs(v) <= {"bf16": 240.0 * 2.0 ** 120, "f16": 240.0 * 2.0 ** 8}[dtype])
        step = np.repeat(np.exp2(exps.astype(np.float64) - 127 - 10), 32, 1)
        assert (np.abs(got - v)[ok] <= np.maximum(2.0 ** -4 * np.abs(v), step)[ok]).all()


@pytest.mark.parametrize("dtype", BOTH)
def test_x8_dequantize_every_code(dtype):
    low, high = {"bf16": (10, 247), "f16": (112, 135)}[dtype]
    exps = torch.arange(low, high + 1).to(torch.uint8)[:, None].repeat(1, 8)
    codes = torch.arange(256).to(torch.uint8)[None].repeat(len(exps), 1)
    got = g.x8_dequantize(g.X8(codes.cuda(), exps.cuda(), DTYPES[dtype])).cpu().double().numpy()
    ref = E4M3[None, :] * np.exp2(exps[:, :1].double().numpy() - 127)
    # codes over 240 at the largest exponent are not written by quantize: they overflow T
    ok = np.isnan(ref) | (np.abs(ref) <= torch.finfo(DTYPES[dtype]).max)
    assert np.array_equal(got[ok], ref[ok], equal_nan=True)


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 8, 40), (7, 33, 65), (63, 16, 128), (64, 130, 257), (65, 264, 72),
                                   (200, 300, 100), (129, 7, 1000), (1000, 256, 512), (333, 513, 300)], ids=str)
@pytest.mark.parametrize("dtype", BOTH)
def test_x8_wgrad(dtype, shape):
    T, N, K = shape
    for out, alpha, beta, pad in [("f32", 1.0, 0.0, 0), (dtype, 0.5, 1.0, 3), ("f32", 1.0, 1.0, 8)]:
        dy, x = randn(T, N, dtype, 4, pad=pad), randn(T, K, dtype, 5, 3.0)
        q = g.x8_quantize(x)
        xv = g.x8_dequantize(q).cpu().double()
        buf = torch.randn(N, K + pad, generator=torch.Generator().manual_seed(6)).to(OUTS[out]).cuda()
        old = buf.clone()
        if beta == 0.0:
            buf[:, :K] = float("nan")
        say("x8_wgrad", dtype, shape, out, alpha, beta, pad)
        g.x8_wgrad(dy, q, alpha=alpha, beta=beta, out=buf[:, :K])
        d = dy.cpu().double()
        ref = alpha * (d.t() @ xv) + beta * old[:, :K].cpu().double()
        size = abs(alpha) * (d.abs().t() @ xv.abs()) + abs(beta) * old[:, :K].cpu().double().abs()
        check_close(buf[:, :K], ref, sum_bound(T, size))
        assert torch.equal(buf[:, K:], old[:, K:])


@pytest.mark.parametrize("shape", [(257, 300, 200), (1000, 129, 130), (2111, 520, 1030), (4096, 8, 8), (640, 256, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_x8_wgrad_few_tiles(shape):
    """Tokens split over workgroups: every slice count and last slice, twice the same bits."""
    T, N, K = shape
    dy, x = randn(T, N, "bf16", 11), randn(T, K, "bf16", 12)
    q = g.x8_quantize(x)
    d, xv = dy.cpu().double(), g.x8_dequantize(q).cpu().double()
    ws = torch.empty(g.x8_wgrad_workspace_size(q, N), dtype=torch.uint8, device="cuda")
    for out in ("f32", "bf16", "f16"):
        buf = torch.randn(N, K + 3, generator=torch.Generator().manual_seed(6)).to(OUTS[out]).cuda()
        old = buf.clone()
        ws.fill_(255)
        say("x8_wgrad few tiles", shape, out)
        g.x8_wgrad(dy, q, alpha=2.0, beta=0.5, out=buf[:, :K], workspace=ws)
        ref = 2.0 * (d.t() @ xv) + 0.5 * old[:, :K].cpu().double()
        size = 2.0 * (d.abs().t() @ xv.abs()) + 0.5 * old[:, :K].cpu().double().abs()
        check_close(buf[:, :K], ref, sum_bound(T, size))
        assert torch.equal(buf[:, K:], old[:, K:])
        again = old.clone()
        g.x8_wgrad(dy, q, alpha=2.0, beta=0.5, out=again[:, :K])
        assert torch.equal(again, buf)


def test_x8_wgrad_keeps_to_its_columns():
    """A NaN in one token's gradient or activation reaches its row or column of dW only."""
    dy, x = randn(70, 40, "bf16", 1), randn(70, 50, "bf16", 2)
    dy[3, 5] = float("nan")
    x[9, 45] = float("inf")
    dw = g.x8_wgrad(dy, g.x8_quantize(x)).cpu()
    bad = torch.zeros(40, 50, dtype=torch.bool)
    bad[5], bad[:, 45] = True, True
    assert torch.equal(torch.isnan(dw), bad)


def test_x8_no_tokens():
    q = g.x8_quantize(torch.empty(0, 40, dtype=torch.float16, device="cuda"))
    out = torch.full((8, 40), 3.0, device="cuda")
    g.x8_wgrad(torch.empty(0, 8, dtype=torch.float16, device="cuda"), q, beta=0.5, out=out)
    assert (out == 1.5).all()


# ---- together -----------------------------------------------------------------------------------
class AdapterLinear(torch.autograd.Function):
    """y = x . W^T + x . A^T . B^T over frozen 4-bit weights W, with the input kept in 8 bits: a layer as
    fine-tuning uses it."""

    @staticmethod
    def forward(ctx, x, w, a, b):
        saved = g.x8_quantize(x)
        h = g.matmul(x, a.t()).to(x.dtype)
        y = g.w4_linear(x, w)
        y += g.matmul(h, b.t())
        ctx.save_for_backward(h, a, b)
        ctx.w, ctx.saved = w, saved
        return y

    @staticmethod
    def backward(ctx, dy):
        h, a, b = ctx.saved_tensors
        dy16 = dy.to(h.dtype)
        dh = g.matmul(dy16, b).to(h.dtype)
        dx = g.w4_dgrad(dy16, ctx.w)
        dx += g.matmul(dh, a)
        return dx.to(h.dtype), None, g.x8_wgrad(dh, ctx.saved).to(h.dtype), g.matmul(dy16.t(), h).to(h.dtype)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("tokens", [1, 100, 600])
def test_fine_tuning_layer(dtype, tokens):
    """A layer's forward and backward pass through all of the calls, against the formulas in float64 on the
    numbers that each step reads."""
    w, wv = make_w4(96, 160, dtype, 32, True, 3)
    x = randn(tokens, 160, dtype, 4).requires_grad_()
    a, b = randn(16, 160, dtype, 5, 0.1).requires_grad_(), randn(96, 16, dtype, 6, 0.1).requires_grad_()
    y = AdapterLinear.apply(x, w, a, b)
    dy = randn(tokens, 96, dtype, 7, 0.01)
    y.backward(dy.float())
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    X, A, B, D = (t.detach().cpu().double() for t in (x, a, b, dy))
    h = X @ A.t()
    hr = eps * h.abs() + sum_bound(160, X.abs() @ A.abs().t()) * 2               # h as it is rounded
    ref = X @ wv.t() + h @ B.t()
    size = X.abs() @ wv.abs().t() + h.abs() @ B.abs().t()
    check_close(y.detach(), ref, hr @ B.abs().t() + sum_bound(180, size))
    dh = D @ B
    dhr = eps * dh.abs() + sum_bound(96, D.abs() @ B.abs()) * 2
    size = D.abs() @ wv.abs() + dh.abs() @ A.abs()
    check_close(x.grad, D @ wv + dh @ A, dhr @ A.abs() + sum_bound(120, size) * 2)
    # the adapter's gradient reads the activations as 8 bits hold them: within 2^-4 of each, or half a smallest step
    xq = g.x8_dequantize(g.x8_quantize(x.detach())).cpu().double()
    check_close(a.grad, dh.t() @ xq, dhr.t() @ xq.abs() + sum_bound(tokens, dh.abs().t() @ xq.abs()) * 2)
    check_close(b.grad, D.t() @ h, D.abs().t() @ hr + sum_bound(tokens, D.abs().t() @ h.abs()) * 2)
    rel = ((xq - X).norm() / X.norm()).item()
    assert rel <= 2.0 ** -4


def test_gradients_against_differences():
    """The linear map's gradient calls against differences of the forward call: with integers and steps that
    FP32 holds exactly the difference of a linear map is its derivative."""
    rng = np.random.default_rng(8)
    codes = rng.integers(0, 16, (24, 64)).astype(np.uint8)
    s = to_type(2.0 ** rng.integers(-1, 2, (24, 2)), "bf16")
    w = g.W4(torch.from_numpy(pack(codes)).cuda(), s.cuda(), None, 32, 64)
    x = torch.from_numpy(rng.integers(-4, 5, (5, 64))).to(torch.bfloat16).cuda()
    dy = torch.from_numpy(rng.integers(-3, 4, (5, 24))).to(torch.bfloat16).cuda()
    loss = lambda t: (g.w4_linear(t, w).double() * dy.double()).sum().item()  # noqa: E731
    dx = g.w4_dgrad(dy, w).cpu()
    for i, k in [(0, 0), (1, 31), (2, 32), (4, 63)]:
        up, down = x.clone(), x.clone()
        up[i, k] += 1
        down[i, k] -= 1
        assert dx[i, k].item() == (loss(up) - loss(down)) / 2
    # the weight gradient: differences of the product of a 16-bit layer over the same 8-bit activations
    q = g.x8_quantize(x)
    xq = g.x8_dequantize(q)
    assert torch.equal(xq, x)                      # small integers are E4M3 numbers
    dw = g.x8_wgrad(dy, q).cpu()
    wt = torch.from_numpy(rng.integers(-2, 3, (24, 64))).to(torch.bfloat16).cuda()
    loss = lambda t: (g.matmul(xq, t.t()).double() * dy.double()).sum().item()  # noqa: E731
    for n, k in [(0, 0), (23, 63), (11, 40)]:
        up, down = wt.clone(), wt.clone()
        up[n, k] += 1
        down[n, k] -= 1
        assert dw[n, k].item() == (loss(up) - loss(down)) / 2


# ---- streams, graphs, repeats -------------------------------------------------------------------
def every_call(dtype, rows=2100):
    """One call of each kind on fixed inputs: (call, outputs it writes)."""
    w, _ = make_w4(1000, 264, dtype, 32, True, 3)
    weights, x1, xm = randn(40, 130, dtype, 2), randn(1, 264, dtype, 4), randn(rows, 264, dtype, 5)
    x64, dy, dy9 = randn(64, 264, dtype, 7), randn(rows, 1000, dtype, 6), randn(9, 1000, dtype, 8)
    f = lambda *s, t=torch.float32: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    q4 = g.w4_quantize(weights, 64, zero_points=True)
    q8 = g.x8_quantize(xm)
    d4, d8 = f(40, 130, t=DTYPES[dtype]), f(rows, 264, t=DTYPES[dtype])
    y1, y64, ym, dx, dx9 = f(1, 1000), f(64, 1000), f(rows, 1000, t=DTYPES[dtype]), f(rows, 264), f(9, 264)
    dw = f(1000, 264)
    # (one workspace for all: they run one after the other)
    ws = torch.empty(max(*(g.w4_workspace_size(w, m, t) for m in (9, 64, rows) for t in (False, True)),
                         g.x8_wgrad_workspace_size(q8, 1000)), dtype=torch.uint8, device="cuda")

    def call():
        g.w4_quantize(weights, 64, zero_points=True, out=q4)
        g.w4_dequantize(q4, out=d4)
        g.w4_linear(x1, w, out=y1, workspace=ws)
        g.w4_linear(x64, w, out=y64, workspace=ws)
        g.w4_linear(xm, w, out=ym, workspace=ws)
        g.x8_quantize(xm, out=q8)
        g.x8_dequantize(q8, out=d8)
        g.w4_dgrad(dy, w, out=dx, workspace=ws)
        g.w4_dgrad(dy9, w, out=dx9, workspace=ws)
        g.x8_wgrad(dy, q8, out=dw, workspace=ws)
    outs = [q4.codes, q4.scales, q4.zeros, q8.codes, q8.exponents, d4, d8, y1, y64, ym, dx, dx9, dw]
    return call, outs


def spoil(outs):
    for t in outs:
        t.fill_(float("nan")) if t.is_floating_point() else t.fill_(0xee)


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", BOTH)
def test_lowbit_calls_captured_and_replayed(dtype):
    call, outs = every_call(dtype)
    say("graph", dtype)
    call()
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    torch.cuda.synchronize()
    for replay in range(4):
        spoil(outs)
        torch.cuda.synchronize()
        assert torch.isfinite((torch.ones(1 << 16, device="cuda") * 2.0).cumsum(0)).all()
        graph.replay()
        torch.cuda.synchronize()
        assert same(outs, eager), f"replay {replay} differs"


def test_lowbit_calls_on_another_stream_repeat_bit_for_bit():
    call, outs = every_call("bf16")
    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    for _ in range(3):
        spoil(outs)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert same(outs, first)
