"""Low-bit operands, host side: argument checks of the C calls (no kernel runs), workspace sizes, and the checks of
the torch-level wrappers."""
import ctypes

import pytest
import torch

import gemm_f32_amd as g
from conftest import gpu_available
from gemm_f32_amd.binding import EpilogueStruct, W4Struct, X8Struct

R, C_ = g.Order.ROW_MAJOR, g.Order.COL_MAJOR
INVALID, DEVICE = g.Status.ERR_INVALID_VALUE, g.Status.ERR_UNSUPPORTED_DEVICE
FAKE = 1 << 20          # a non-null, aligned address; never dereferenced by these calls
BIG = 2 ** 31 - 4095    # one past the largest extent

TYPES = ["bf16", "f16"]
W4_QUANTIZE = {"bf16": g.gemm_bf16_w4_quantize, "f16": g.gemm_f16_w4_quantize}
W4_DEQUANTIZE = {"bf16": g.gemm_bf16_w4_dequantize, "f16": g.gemm_f16_w4_dequantize}
W4_PRODUCT = {"bf16": g.gemm_bf16_w4, "f16": g.gemm_f16_w4}
X8_QUANTIZE = {"bf16": g.gemm_bf16_x8_quantize, "f16": g.gemm_f16_x8_quantize}
X8_DEQUANTIZE = {"bf16": g.gemm_bf16_x8_dequantize, "f16": g.gemm_f16_x8_dequantize}
WGRAD = {"bf16": g.gemm_bf16_x8_wgrad, "f16": g.gemm_f16_x8_wgrad}


def status(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except g.GemmError as e:
        return e.status
    return g.Status.OK


def named(d):
    return ",".join(f"{k}={v}" for k, v in d.items()) or "valid"


def w4(codes=FAKE, ld=32, scales=FAKE, lds=2, zeros=0, ldz=0, group=32):
    return W4Struct(codes or None, ld, scales or None, lds, zeros or None, ldz, group)


def x8(codes=FAKE, ld=64, exponents=FAKE, lde=2):
    return X8Struct(codes or None, ld, exponents or None, lde)


# a 16 x 64 matrix in 4 bits: rows of 32 bytes, 2 groups of 32
BAD_W4 = [dict(group=0), dict(group=16), dict(group=48), dict(group=256), dict(ld=31), dict(lds=1), dict(codes=0),
          dict(scales=0), dict(scales=FAKE + 1), dict(zeros=FAKE, ldz=1)]


def convert_w4(dtype, way, rows=16, cols=64, W=FAKE, ldw=64, **q):
    args = (w4(**q), W, ldw) if way == "dequantize" else (W, ldw, w4(**q))
    return status((W4_DEQUANTIZE if way == "dequantize" else W4_QUANTIZE)[dtype], rows, cols, *args)


@pytest.mark.parametrize("bad", BAD_W4 + [dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(W=0),
                                          dict(W=FAKE + 1), dict(ldw=63)], ids=named)
@pytest.mark.parametrize("way", ["quantize", "dequantize"])
@pytest.mark.parametrize("dtype", TYPES)
def test_w4_conversions_refuse(dtype, way, bad):
    assert convert_w4(dtype, way, **bad) == INVALID


@pytest.mark.skipif(gpu_available(), reason="checks the no-GPU path")
@pytest.mark.parametrize("good", [dict(), dict(group=128, lds=1), dict(zeros=FAKE, ldz=2), dict(zeros=0, ldz=-5),
                                  dict(cols=63), dict(cols=1, ldw=1, ld=1, lds=1), dict(codes=FAKE + 1)], ids=named)
@pytest.mark.parametrize("way", ["quantize", "dequantize"])
def test_w4_conversions_reach_the_device_check(way, good):
    assert convert_w4("bf16", way, **good) == DEVICE


@pytest.mark.parametrize("empty", [dict(rows=0, W=0, codes=0, scales=0), dict(cols=0, W=0, codes=0, scales=0)], ids=named)
@pytest.mark.parametrize("way", ["quantize", "dequantize"])
def test_w4_conversions_of_nothing(way, empty):
    assert convert_w4("f16", way, **empty) == g.Status.OK


def convert_x8(dtype, way, rows=16, cols=64, X=FAKE, ldx=64, **q):
    args = (x8(**q), X, ldx) if way == "dequantize" else (X, ldx, x8(**q))
    return status((X8_DEQUANTIZE if way == "dequantize" else X8_QUANTIZE)[dtype], rows, cols, *args)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(X=0),
                                 dict(X=FAKE + 1), dict(ldx=63), dict(ld=63), dict(lde=1), dict(codes=0),
                                 dict(exponents=0)], ids=named)
@pytest.mark.parametrize("way", ["quantize", "dequantize"])
@pytest.mark.parametrize("dtype", TYPES)
def test_x8_conversions_refuse(dtype, way, bad):
    assert convert_x8(dtype, way, **bad) == INVALID


@pytest.mark.skipif(gpu_available(), reason="checks the no-GPU path")
@pytest.mark.parametrize("good", [dict(), dict(cols=33), dict(codes=FAKE + 1, exponents=FAKE + 3)], ids=named)
@pytest.mark.parametrize("way", ["quantize", "dequantize"])
def test_x8_conversions_reach_the_device_check(way, good):
    assert convert_x8("f16", way, **good) == DEVICE


@pytest.mark.parametrize("empty", [dict(rows=0), dict(cols=0)], ids=named)
@pytest.mark.parametrize("way", ["quantize", "dequantize"])
def test_x8_conversions_of_nothing(way, empty):
    assert convert_x8("bf16", way, X=0, codes=0, exponents=0, **empty) == g.Status.OK


# x . W^T with W 16 x 64, or dy . W with W the same: M x 64 by 16, M x 16 by 64
def product(dtype, order=C_, M=4, A=FAKE, lda=64, C=FAKE, ldc=64, epi=None, workspace=0, nbytes=0, extents=None, **q):
    N, K = extents or ((16, 64) if order != R else (64, 16))
    e = ctypes.byref(EpilogueStruct(**epi)) if epi is not None else None
    return status(W4_PRODUCT[dtype], M, N, K, A, lda, w4(**q), int(order), C, ldc, e, workspace, nbytes)


def epi(alpha=1.0, beta=0.0, bias=None, activation=0, out_type=0):
    return dict(alpha=alpha, beta=beta, bias=bias, activation=activation, out_type=out_type)


BAD_PRODUCT = [dict(M=-1), dict(M=BIG), dict(A=0), dict(A=FAKE + 1), dict(lda=15), dict(C=0), dict(C=FAKE + 2),
               dict(ldc=15), dict(epi=epi(activation=3)), dict(epi=epi(out_type=3)), dict(epi=epi(out_type=-1)),
               dict(epi=epi(bias=FAKE + 2)), dict(epi=epi(out_type=1), C=FAKE + 1), dict(workspace=FAKE + 8, nbytes=64),
               dict(extents=(-1, 64)), dict(extents=(16, -1)), dict(extents=(BIG, 64)), dict(extents=(16, BIG))]


@pytest.mark.parametrize("bad", BAD_W4 + BAD_PRODUCT, ids=named)
@pytest.mark.parametrize("order", [C_, R], ids=["x.Wt", "dy.W"])
@pytest.mark.parametrize("dtype", TYPES)
def test_w4_products_refuse(dtype, order, bad):
    assert product(dtype, order, **bad) == INVALID


def test_w4_product_refuses_an_unknown_order():
    assert product("bf16", 2, extents=(16, 64)) == INVALID


def test_w4_calls_refuse_a_null_matrix():
    lib = g.lib_handle()
    assert lib.gemm_bf16_w4_quantize(4, 4, FAKE, 4, None, None) == INVALID
    assert lib.gemm_f16_w4(4, 4, 4, FAKE, 4, None, int(C_), FAKE, 4, None, None, 0, None) == INVALID
    assert lib.gemm_bf16_x8_dequantize(4, 4, None, FAKE, 4, None) == INVALID
    assert lib.gemm_f16_x8_wgrad(4, 4, 4, FAKE, 4, None, FAKE, 4, 1.0, 0.0, 0, FAKE, 1 << 20, None) == INVALID


@pytest.mark.skipif(gpu_available(), reason="checks the no-GPU path")
@pytest.mark.parametrize("good", [dict(), dict(epi=epi(beta=1.0, bias=FAKE, activation=2, out_type=2), C=FAKE + 2),
                                  dict(A=FAKE + 2), dict(workspace=FAKE, nbytes=1), dict(zeros=FAKE, ldz=2)], ids=named)
@pytest.mark.parametrize("order", [C_, R], ids=["x.Wt", "dy.W"])
@pytest.mark.parametrize("dtype", TYPES)
def test_w4_products_reach_the_device_check(dtype, order, good):
    assert product(dtype, order, **good) == DEVICE


@pytest.mark.parametrize("order", [C_, R], ids=["x.Wt", "dy.W"])
def test_w4_products_of_nothing(order):
    assert product("bf16", order, M=0, A=0, C=0) == g.Status.OK


def test_out_type_of_other_calls_stays_f32_or_bf16():
    args = (8, 8, 64, FAKE, 64, int(R), FAKE, 64, int(C_), FAKE, 8, int(R))
    assert status(g.gemm_bf16_f32acc_fused, *args, out_type=g.Out.F16) == INVALID


def test_w4_workspace_sizes():
    size = g.gemm_w4_workspace_size
    assert size(1, 4096, 4096, C_) == 0 and size(16, 11008, 4096, C_) == 0        # few rows: none
    assert size(2048, 11008, 4096, C_) == 2 * 11008 * 4096                        # W as 16-bit numbers
    assert size(2048, 4096, 11008, R) == 2 * 11008 * 4096
    for m, order in [(64, C_), (1, R), (128, R)]:                                 # the slices' FP32 sums
        assert size(m, 4096, 4096, order) > 0 and size(m, 4096, 4096, order) % (4 * m * 4096) == 0
    for bad in [(-1, 8, 8, C_), (8, -1, 8, C_), (8, 8, BIG, C_), (8, 8, 8, 2)]:
        assert size(*bad) == 0
    for nothing in [(0, 8, 8, C_), (8, 0, 8, R), (8, 8, 0, C_)]:
        assert size(*nothing) == 0


def wgrad(dtype, T=16, N=8, K=64, dY=FAKE, lddy=8, C=FAKE, ldc=64, out=0, workspace=FAKE, nbytes=1 << 30, **q):
    return status(WGRAD[dtype], T, N, K, dY, lddy, x8(**q), C, ldc, 1.0, 0.0, out, workspace, nbytes)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(N=-1), dict(K=-1), dict(T=BIG), dict(N=BIG), dict(K=BIG), dict(dY=0), dict(dY=FAKE + 1), dict(lddy=7),
    dict(C=0), dict(C=FAKE + 2), dict(C=FAKE + 1, out=1), dict(ldc=63), dict(out=3), dict(out=-1), dict(ld=63), dict(lde=1),
    dict(codes=0), dict(exponents=0), dict(workspace=0), dict(workspace=FAKE + 8), dict(nbytes=16 * 64 * 2 - 1),
    dict(N=7, lddy=7, nbytes=16 * 64 * 2 + 16 * 8 * 2 - 1),
    dict(T=(1 << 15) + 1, lddy=1 << 15, nbytes=1 << 40),                # dY's offsets reach 2^30
    dict(T=1 << 24, N=8, K=64, nbytes=1 << 40),                         # X's
], ids=named)
@pytest.mark.parametrize("dtype", TYPES)
def test_x8_wgrad_refuses(dtype, bad):
    assert wgrad(dtype, **bad) == INVALID


@pytest.mark.skipif(gpu_available(), reason="checks the no-GPU path")
@pytest.mark.parametrize("good", [dict(), dict(N=7, lddy=7), dict(out=2, C=FAKE + 2), dict(nbytes=16 * 64 * 2),
                                  dict(T=0, dY=0, codes=0, exponents=0, workspace=0, nbytes=0)], ids=named)
@pytest.mark.parametrize("dtype", TYPES)
def test_x8_wgrad_reaches_the_device_check(dtype, good):
    assert wgrad(dtype, **good) == DEVICE


def test_x8_wgrad_of_nothing():
    assert wgrad("bf16", N=0, dY=0, C=0, workspace=0, nbytes=0) == g.Status.OK
    assert wgrad("bf16", K=0, codes=0, exponents=0, C=0, workspace=0, nbytes=0) == g.Status.OK


def test_x8_wgrad_workspace_sizes():
    size = g.gemm_x8_wgrad_workspace_size
    assert size(2048, 4096, 4096) == 2048 * 4096 * 2                              # X as 16-bit numbers
    assert size(100, 4096, 60) == 100 * 64 * 2                                    # in rows of a multiple of 8
    assert size(100, 4097, 60) == 100 * (64 + 4104) * 2                           # and dY, N % 8 != 0
    split = size(4096, 1024, 1024) - 4096 * 1024 * 2                              # and the slices' sums
    assert split > 0 and split % (4 * 1024 * 1024) == 0
    for bad in [(-1, 8, 8), (8, BIG, 8), (0, 8, 8), (8, 0, 8), (8, 8, 0)]:
        assert size(*bad) == 0


# ---- the torch-level wrappers ---------------------------------------------------------------
def zeros(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("codes,scales,points,group,cols,error", [
    (zeros(4, 32), zeros(4, 2, dtype=torch.bfloat16), None, 48, 64, ValueError),
    (zeros(4, 31), zeros(4, 2, dtype=torch.bfloat16), None, 32, 64, ValueError),
    (zeros(4, 32, dtype=torch.int8), zeros(4, 2, dtype=torch.bfloat16), None, 32, 64, ValueError),
    (zeros(4, 32), zeros(4, 2, dtype=torch.float32), None, 32, 64, TypeError),
    (zeros(4, 32), zeros(4, 1, dtype=torch.float16), None, 32, 64, ValueError),
    (zeros(4, 32), zeros(4, 2, dtype=torch.float16), zeros(4, 1), 32, 64, ValueError),
    (zeros(4, 32), zeros(4, 2, dtype=torch.float16), zeros(4, 2, dtype=torch.int32), 32, 64, ValueError),
    (zeros(4, 32), zeros(4, 2, dtype=torch.float16), None, 32, 64, ValueError),         # not on a GPU
])
def test_w4_checks_its_tensors(codes, scales, points, group, cols, error):
    with pytest.raises(error):
        g.W4(codes, scales, points, group, cols)


@pytest.mark.parametrize("codes,exponents,dtype,error", [
    (zeros(4, 40, dtype=torch.int8), zeros(4, 2), torch.bfloat16, TypeError),
    (zeros(4, 40), zeros(4, 2, dtype=torch.int8), torch.bfloat16, TypeError),
    (zeros(4, 40), zeros(4, 1), torch.bfloat16, ValueError),
    (zeros(4, 40), zeros(4, 2), torch.float32, TypeError),
    (zeros(4, 40), zeros(4, 2), torch.float16, ValueError),                             # not on a GPU
])
def test_x8_checks_its_tensors(codes, exponents, dtype, error):
    with pytest.raises(error):
        g.X8(codes, exponents, dtype)


def test_quantize_checks_its_input():
    with pytest.raises(TypeError):
        g.w4_quantize(zeros(4, 64, dtype=torch.float32))
    with pytest.raises(TypeError):
        g.x8_quantize(zeros(4, 64, dtype=torch.float32))
    for f in (g.w4_quantize, g.x8_quantize):
        with pytest.raises(ValueError):
            f(zeros(4, 64, dtype=torch.bfloat16))          # not on a GPU
        with pytest.raises(ValueError):
            f(zeros(64, dtype=torch.bfloat16))
