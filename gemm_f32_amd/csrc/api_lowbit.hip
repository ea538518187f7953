// The C ABI of the low-bit operands (4-bit weights, 8-bit activations): argument checks, kernel
// choice and launch.  Formats and contracts are documented in include/gemm.h.
#include <climits>
#include <cstdint>

#include "gemm.h"
#include "api_internal.hpp"
#include "common.hpp"
#include "launch.hpp"
#include "lowbit.hpp"

namespace gemm {
namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }

int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }

bool extents_ok(int64_t a, int64_t b, int64_t c = 0) {
    for (int64_t v : {a, b, c})
        if (v < 0 || v > INT_MAX - 4095) return false;      // (rounded up to a kernel's block it is still an int)
    return true;
}

// A 4-bit matrix of rows x cols (extents already checked).
bool w4_ok(const gemm_w4_t* q, int64_t rows, int64_t cols, W4View& v) {
    if (q == nullptr || (q->group != 32 && q->group != 64 && q->group != 128)) return false;
    const int64_t groups = (cols + q->group - 1) / q->group;
    if (q->ld_codes < at_least_one((cols + 1) / 2) || q->ld_scales < at_least_one(groups)) return false;
    if (q->zeros != nullptr && q->ld_zeros < at_least_one(groups)) return false;
    if (rows > 0 && cols > 0 && (q->codes == nullptr || q->scales == nullptr)) return false;
    if (!aligned_to(q->scales, 2)) return false;
    v = W4View{q->codes, q->ld_codes, static_cast<const uint16_t*>(q->scales), q->ld_scales, q->zeros,
               q->zeros != nullptr ? q->ld_zeros : 0, q->group == 32 ? 5 : q->group == 64 ? 6 : 7};
    return true;
}

bool x8_ok(const gemm_x8_t* q, int64_t rows, int64_t cols, X8View& v) {
    if (q == nullptr || q->ld_codes < at_least_one(cols) || q->ld_exponents < at_least_one((cols + 31) / 32)) return false;
    if (rows > 0 && cols > 0 && (q->codes == nullptr || q->exponents == nullptr)) return false;
    v = X8View{q->codes, q->ld_codes, q->exponents, q->ld_exponents};
    return true;
}

// A 16-bit row-major matrix.
bool matrix_ok(const void* m, int64_t ld, int64_t rows, int64_t cols) {
    return ld >= at_least_one(cols) && (rows == 0 || cols == 0 || m != nullptr) && aligned_to(m, 2);
}

bool out_ok(const void* C, int64_t ldc, int64_t rows, int64_t cols, int out) {
    if (out != GEMM_OUT_F32 && out != GEMM_OUT_BF16 && out != GEMM_OUT_F16) return false;
    return ldc >= at_least_one(cols) && (rows == 0 || cols == 0 || C != nullptr) &&
           aligned_to(C, out == GEMM_OUT_F32 ? 4 : 2);
}

constexpr int out_kind(int out) { return out == GEMM_OUT_F32 ? kOutF32 : out == GEMM_OUT_BF16 ? kOutBf16 : kOutF16; }

// The conversions share their shape: check, nothing for an empty matrix, launch.
template <typename View, typename Launch>
gemm_status_t convert(int64_t rows, int64_t cols, bool ok, const View& v, const char* name, Launch launch) {
    if (!ok) return GEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0) return record_call(hipSuccess, "none");
    int cus = 0;
    if (!current_device(cus)) return GEMM_ERR_UNSUPPORTED_DEVICE;
    return record_call(launch(v), name);
}

gemm_status_t w4_quantize(bool f16, int64_t rows, int64_t cols, const uint16_t* W, int64_t ldw, const gemm_w4_t* Q,
                          hipStream_t stream) {
    W4View v{};
    const bool ok = extents_ok(rows, cols) && matrix_ok(W, ldw, rows, cols) && w4_ok(Q, rows, cols, v);
    return convert(rows, cols, ok, v, f16 ? "f16_w4_quantize" : "bf16_w4_quantize", [&](const W4View& q) {
        return launch_w4_quantize(W, ldw, (int)rows, (int)cols, q, f16, stream);
    });
}

gemm_status_t w4_dequantize(bool f16, int64_t rows, int64_t cols, const gemm_w4_t* Q, uint16_t* W, int64_t ldw,
                            hipStream_t stream) {
    W4View v{};
    const bool ok = extents_ok(rows, cols) && matrix_ok(W, ldw, rows, cols) && w4_ok(Q, rows, cols, v);
    return convert(rows, cols, ok, v, f16 ? "f16_w4_dequantize" : "bf16_w4_dequantize", [&](const W4View& q) {
        return launch_w4_dequantize(q, (int)rows, (int)cols, W, ldw, f16, stream);
    });
}

gemm_status_t x8_quantize(bool f16, int64_t rows, int64_t cols, const uint16_t* X, int64_t ldx, const gemm_x8_t* Q,
                          hipStream_t stream) {
    X8View v{};
    const bool ok = extents_ok(rows, cols) && matrix_ok(X, ldx, rows, cols) && x8_ok(Q, rows, cols, v);
    return convert(rows, cols, ok, v, f16 ? "f16_x8_quantize" : "bf16_x8_quantize", [&](const X8View& q) {
        return launch_x8_quantize(X, ldx, (int)rows, (int)cols, q, f16, stream);
    });
}

gemm_status_t x8_dequantize(bool f16, int64_t rows, int64_t cols, const gemm_x8_t* Q, uint16_t* X, int64_t ldx,
                            hipStream_t stream) {
    X8View v{};
    const bool ok = extents_ok(rows, cols) && matrix_ok(X, ldx, rows, cols) && x8_ok(Q, rows, cols, v);
    return convert(rows, cols, ok, v, f16 ? "f16_x8_dequantize" : "bf16_x8_dequantize", [&](const X8View& q) {
        return launch_x8_dequantize(q, (int)rows, (int)cols, X, ldx, f16, stream);
    });
}

// ---- products on 4-bit weights ----------------------------------------------------------
// The stored matrix (rows x cols of W) for a product's B.
void w4_shape(int64_t N, int64_t K, int order_b, int64_t& rows, int64_t& cols) {
    rows = order_b == GEMM_COL_MAJOR ? N : K;
    cols = order_b == GEMM_COL_MAJOR ? K : N;
}

// Bytes of W as 16-bit numbers (rows of a multiple of 8) where writing them and running the 16-bit
// direct-copy kernels is the faster way by the time model, else 0: so too where those kernels do not take the
// product (K too short, a W past their 31-bit offsets).
size_t w4_decoded(int64_t M, int64_t N, int64_t K, int order_b, int cus) {
    if (M < 256 || N <= 0 || K < 64) return 0;
    const bool tr = order_b == GEMM_ROW_MAJOR;
    int64_t rows, cols;
    w4_shape(N, K, order_b, rows, cols);
    const int64_t ld = round8(cols);
    if (tr && rows * ld * 2 >= (int64_t)1 << 31) return 0;
    if ((int64_t)64 * ld * 2 >= (int64_t)1 << 31) return 0;
    if ((!tr || N >= 32) && w4_split(M, N, K, tr, cus, true).us <= w4_decoded_us(M, N, K, cus)) return 0;
    return (size_t)rows * ld * 2;
}

// The workspace of a product: W as 16-bit numbers, else the slices' sums of a K split over workgroups.
size_t w4_workspace(int64_t M, int64_t N, int64_t K, int order_b) {
    int cus = 0;
    if (!current_device(cus)) cus = 256;
    const size_t decoded = w4_decoded(M, N, K, order_b, cus);
    const bool tr = order_b == GEMM_ROW_MAJOR;
    if (decoded > 0 || M <= (tr ? 0 : 16) || N < (tr ? 32 : 1) || K < 32) return decoded;
    return w4_split(M, N, K, tr, cus, true).bytes;
}

gemm_status_t w4_product(bool f16, int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const gemm_w4_t* W,
                         int order_b, void* C, int64_t ldc, const gemm_epilogue_t* epi, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
    if (order_b != GEMM_ROW_MAJOR && order_b != GEMM_COL_MAJOR) return GEMM_ERR_INVALID_VALUE;
    Epilogue e{1.f, 0.f, nullptr, 0, kActNone, kOutF32};
    int out = GEMM_OUT_F32;
    if (epi != nullptr) {
        if (epi->activation != GEMM_ACT_NONE && epi->activation != GEMM_ACT_RELU && epi->activation != GEMM_ACT_GELU)
            return GEMM_ERR_INVALID_VALUE;
        out = epi->out_type;
        e = Epilogue{epi->alpha, epi->beta, epi->bias, 0, (int)epi->activation, out_kind(out)};
    }
    W4View w{};
    int64_t rows, cols;
    w4_shape(N, K, order_b, rows, cols);
    if (!extents_ok(M, N, K) || !matrix_ok(A, lda, M, K) || !out_ok(C, ldc, M, N, out) || !w4_ok(W, rows, cols, w) ||
        !aligned_to(e.bias, 4) || !aligned_to(workspace, 16))
        return GEMM_ERR_INVALID_VALUE;
    // (a product over nothing reads neither operand)
    if (M == 0 || N == 0) return record_call(hipSuccess, "none");
    int cus = 0;
    if (!current_device(cus)) return GEMM_ERR_UNSUPPORTED_DEVICE;
    const int tr = order_b == GEMM_ROW_MAJOR ? 1 : 0;
    Problem p{(int)M, (int)N, (int)K, A, lda, kRow, workspace, round8(cols), tr ? kRow : kCol,
              static_cast<float*>(C), ldc};
    if (K == 0) return record_call(run_epilogue_fill(p, e, C, stream), "epilogue_fill");
    const size_t need = w4_decoded(M, N, K, order_b, cus);
    const bool reach = (int64_t)64 * lda * 2 < (int64_t)1 << 31;      // the direct-copy kernels' A
    const char* name = "none";
    hipError_t err = hipSuccess;
    const W4Problem wp{(int)M, (int)N, (int)K, A, lda, w, tr, C, ldc, e};
    if (need > 0 && workspace != nullptr && workspace_bytes >= need && reach) {
        err = launch_w4_dequantize(w, (int)rows, (int)cols, static_cast<uint16_t*>(workspace), round8(cols), f16, stream);
        if (err == hipSuccess) err = run_fused_tiles(f16 ? In::F16 : In::BF16, p, e, C, cus, stream, name);
    } else if (K < 32 || (tr && N < 32)) {
        err = launch_w4_short(wp, f16, stream, name);
    } else if (w4_few_applies(wp, cus)) {
        err = launch_w4_few(wp, f16, cus, stream, name);
    } else {
        W4Split sp = w4_split(M, N, K, tr != 0, cus, true);
        if (sp.slices > 1 && (workspace == nullptr || workspace_bytes < sp.bytes)) sp = w4_split(M, N, K, tr != 0, cus, false);
        err = launch_w4_tile(wp, sp, f16, static_cast<float*>(workspace), stream, name);
    }
    return record_call(err, name);
}

// ---- weight gradient from 8-bit activations -----------------------------------------------
// K (the tokens) split over workgroups where C has too few 256 x 128 tiles to fill the CUs: the number of slices
// by a time model fitted to 4095 tokens x 1030 x 1023 (40 tiles, fp16): unsplit 55 us, 0.85 us a k-tile of 64
// tokens; 4 slices 21.0 us (1.2 us a k-tile, the operands' traffic past the L2s among more workgroups) and 6.0 us
// for the second kernel, which reads the slices' sums at 3 TB/s.  Powers of two: the slices then divide the XCDs.
struct X8Split {
    int slices = 1, kslice = 0;
    size_t bytes = 0;
};

X8Split x8_split(int64_t T, int64_t N, int64_t K, int cus) {
    const int64_t tiles = ((N + 255) / 256) * ((K + 127) / 128), steps = (T + 63) / 64;
    X8Split best;
    double best_us = 0.85 * steps;
    for (int64_t s = 2; s <= 32 && s * tiles <= cus && s <= steps; s *= 2) {
        const int64_t each = (steps + s - 1) / s, used = (steps + each - 1) / each;
        const double us = 1.2 * each + 2.0 + used * N * K * 4 / 3e6;
        if (us >= best_us) continue;
        best_us = us;
        best = X8Split{(int)used, (int)(64 * each), (size_t)(used * N * ((K + 3) & ~3)) * 4};
    }
    return best;
}

// Bytes of the 16-bit numbers that the product reads: X, and dY where its rows are not whole chunks of 8.
size_t x8_decoded(int64_t T, int64_t N, int64_t K) {
    return (size_t)T * (round8(K) + (N % 8 != 0 ? round8(N) : 0)) * 2;
}

size_t x8_workspace(int64_t T, int64_t N, int64_t K) {
    if (T <= 0 || N <= 0 || K <= 0) return 0;
    int cus = 0;
    if (!current_device(cus)) cus = 256;
    return x8_decoded(T, N, K) + x8_split(T, N, K, cus).bytes;
}

gemm_status_t x8_wgrad(bool f16, int64_t T, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const gemm_x8_t* X,
                       void* C, int64_t ldc, float alpha, float beta, int out, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    X8View x{};
    if (!extents_ok(T, N, K) || !matrix_ok(dY, lddy, T, N) || !out_ok(C, ldc, N, K, out) || !x8_ok(X, T, K, x) ||
        !aligned_to(workspace, 16))
        return GEMM_ERR_INVALID_VALUE;
    const size_t need = x8_workspace(T, N, K);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GEMM_ERR_INVALID_VALUE;
    const Epilogue e{alpha, beta, nullptr, 0, kActNone, out_kind(out)};
    // rows of C: output features (dY's columns), columns: input features
    const bool copy = N % 8 != 0;
    uint16_t* xs = static_cast<uint16_t*>(workspace);
    uint16_t* ys = xs + (need > 0 ? T * round8(K) : 0);
    Problem p{(int)N, (int)K, (int)T, copy ? ys : dY, copy ? round8(N) : lddy, kCol, xs, round8(K), kRow,
              static_cast<float*>(C), ldc};
    if (T > 0 && N > 0 && K > 0 && !bf16_dma_tn_applies(p)) return GEMM_ERR_INVALID_VALUE;
    if (N == 0 || K == 0) return record_call(hipSuccess, "none");
    int cus = 0;
    if (!current_device(cus)) return GEMM_ERR_UNSUPPORTED_DEVICE;
    if (T == 0) return record_call(run_epilogue_fill(p, e, C, stream), "epilogue_fill");
    hipError_t err = copy ? launch_x8_operands(x, (int)T, (int)K, xs, round8(K), dY, lddy, (int)N, ys, round8(N), f16, stream)
                          : launch_x8_dequantize(x, (int)T, (int)K, xs, round8(K), f16, stream);
    const char* name = "none";
    if (err != hipSuccess) return record_call(err, name);
    const X8Split sp = x8_split(T, N, K, cus);
    if (sp.slices > 1) {
        name = f16 ? "f16_dma256x128_tn_splitk" : "bf16_dma256x128_tn_splitk";
        float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + x8_decoded(T, N, K));
        SplitProblem s{};
        static_cast<Problem&>(s) = p;
        // sums in rows of whole 16 bytes (the columns past K come from the padding of X's rows and are not read)
        s.N = (p.N + 3) & ~3;
        s.C = part;
        s.ldc = s.N;
        s.kslice = sp.kslice;
        s.part = part + N * s.N;
        Launch l{};
        l.stream = stream;
        l.vec_c = true;
        l.group_m = 1;
        err = launch_bf16_dma_tn_split(s, sp.slices, l, f16);
        EpiProblem ep{};
        static_cast<Problem&>(ep) = p;
        ep.C = static_cast<float*>(C);
        ep.e = e;
        if (err == hipSuccess) err = launch_join_slabs(ep, part, sp.slices, s.N, stream);
    } else {
        err = run_fused_tiles(f16 ? In::F16 : In::BF16, p, e, C, cus, stream, name);
    }
    return record_call(err, name);
}

}  // namespace
}  // namespace gemm

extern "C" {

gemm_status_t gemm_bf16_w4_quantize(int64_t rows, int64_t cols, const uint16_t* W, int64_t ldw, const gemm_w4_t* Q,
                                    hipStream_t stream) {
    return gemm::w4_quantize(false, rows, cols, W, ldw, Q, stream);
}

gemm_status_t gemm_f16_w4_quantize(int64_t rows, int64_t cols, const uint16_t* W, int64_t ldw, const gemm_w4_t* Q,
                                   hipStream_t stream) {
    return gemm::w4_quantize(true, rows, cols, W, ldw, Q, stream);
}

gemm_status_t gemm_bf16_w4_dequantize(int64_t rows, int64_t cols, const gemm_w4_t* Q, uint16_t* W, int64_t ldw,
                                      hipStream_t stream) {
    return gemm::w4_dequantize(false, rows, cols, Q, W, ldw, stream);
}

gemm_status_t gemm_f16_w4_dequantize(int64_t rows, int64_t cols, const gemm_w4_t* Q, uint16_t* W, int64_t ldw,
                                     hipStream_t stream) {
    return gemm::w4_dequantize(true, rows, cols, Q, W, ldw, stream);
}

size_t gemm_w4_workspace_size(int64_t M, int64_t N, int64_t K, gemm_order_t order_b) {
    if (!gemm::extents_ok(M, N, K) || (order_b != GEMM_ROW_MAJOR && order_b != GEMM_COL_MAJOR)) return 0;
    return gemm::w4_workspace(M, N, K, order_b);
}

gemm_status_t gemm_bf16_w4(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const gemm_w4_t* W,
                           gemm_order_t order_b, void* C, int64_t ldc, const gemm_epilogue_t* epilogue,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return gemm::w4_product(false, M, N, K, A, lda, W, order_b, C, ldc, epilogue, workspace, workspace_bytes, stream);
}

gemm_status_t gemm_f16_w4(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const gemm_w4_t* W,
                          gemm_order_t order_b, void* C, int64_t ldc, const gemm_epilogue_t* epilogue, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
    return gemm::w4_product(true, M, N, K, A, lda, W, order_b, C, ldc, epilogue, workspace, workspace_bytes, stream);
}

gemm_status_t gemm_bf16_x8_quantize(int64_t rows, int64_t cols, const uint16_t* X, int64_t ldx, const gemm_x8_t* Q,
                                    hipStream_t stream) {
    return gemm::x8_quantize(false, rows, cols, X, ldx, Q, stream);
}

gemm_status_t gemm_f16_x8_quantize(int64_t rows, int64_t cols, const uint16_t* X, int64_t ldx, const gemm_x8_t* Q,
                                   hipStream_t stream) {
    return gemm::x8_quantize(true, rows, cols, X, ldx, Q, stream);
}

gemm_status_t gemm_bf16_x8_dequantize(int64_t rows, int64_t cols, const gemm_x8_t* Q, uint16_t* X, int64_t ldx,
                                      hipStream_t stream) {
    return gemm::x8_dequantize(false, rows, cols, Q, X, ldx, stream);
}

gemm_status_t gemm_f16_x8_dequantize(int64_t rows, int64_t cols, const gemm_x8_t* Q, uint16_t* X, int64_t ldx,
                                     hipStream_t stream) {
    return gemm::x8_dequantize(true, rows, cols, Q, X, ldx, stream);
}

size_t gemm_x8_wgrad_workspace_size(int64_t tokens, int64_t N, int64_t K) {
    return gemm::extents_ok(tokens, N, K) ? gemm::x8_workspace(tokens, N, K) : 0;
}

gemm_status_t gemm_bf16_x8_wgrad(int64_t tokens, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy,
                                 const gemm_x8_t* X, void* C, int64_t ldc, float alpha, float beta, gemm_out_t out_type,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return gemm::x8_wgrad(false, tokens, N, K, dY, lddy, X, C, ldc, alpha, beta, out_type, workspace, workspace_bytes,
                          stream);
}

gemm_status_t gemm_f16_x8_wgrad(int64_t tokens, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy,
                                const gemm_x8_t* X, void* C, int64_t ldc, float alpha, float beta, gemm_out_t out_type,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return gemm::x8_wgrad(true, tokens, N, K, dY, lddy, X, C, ldc, alpha, beta, out_type, workspace, workspace_bytes,
                          stream);
}

}  // extern "C"
