// 4-bit weights and 8-bit activations: rounding 16-bit matrices to codes, and the 16-bit numbers
// that codes stand for (formats in lowbit.hpp).
//
// Every kernel reads its input once and writes its output once, so the time is that of the bytes.
// A lane owns 8 consecutive columns (16 bytes of the 16-bit side; a wavefront's access to a row is
// 1 KB contiguous) of kRows rows, all of whose loads are issued before the first is used.  A
// group's columns lie in 4 to 16 neighbouring lanes, which agree on its largest magnitude (or its
// extremes) by exchanging values; one of them writes the scale.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "lowbit.hpp"

namespace gemm {
namespace {

constexpr int kThreads = 256, kRows = 4;

// 8 elements of a row from column c on; zero past cols
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int cols) {
    if (c + 8 <= cols) return load16(row + c);
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? row[c + e] : 0u;
    return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

typedef unsigned int u32x4_u2 __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void store8(uint16_t* row, int c, int cols, const uint4& v) {
    if (c + 8 <= cols) {
        *reinterpret_cast<u32x4_u2*>(row + c) = u32x4_u2{v.x, v.y, v.z, v.w};
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < cols) row[c + e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
}

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = from16<F16>((uint16_t)(w[e / 2] >> (16 * (e % 2))));
}

// whether any of 8 packed numbers is an infinity or a NaN (the exponent field all ones)
template <bool F16>
__device__ __forceinline__ bool any_nonfinite(const uint4& v) {
    constexpr uint32_t E = F16 ? 0x7c00u : 0x7f80u;
    bool bad = false;
#pragma unroll
    for (uint32_t w : {v.x, v.y, v.z, v.w}) bad |= (w & E) == E || ((w >> 16) & E) == E;
    return bad;
}

// ---- 4-bit weights -----------------------------------------------------------------------
// Symmetric (no zeros): s = T(amax / 7), code = round(w / s) + 8.  With zero points: the range always
// includes 0, s = T((max - min) / 15), z = round(-min / s), code = round(w / s) + z; codes and z are held
// in 0 .. 15.  s == 0 (a group of zeros, or of numbers too small for a scale of type T): every code is
// the zero point 8.  A group with an infinity or a NaN gets a NaN scale: all of it stands for NaN.
// Quotients are correctly rounded divisions: no quotient of two T lies within FP32's rounding of a
// border between two codes unless it is that border.
template <bool F16>
__global__ __launch_bounds__(kThreads) void k_w4_quantize(const uint16_t* W, int64_t ldw, int rows, int cols,
                                                          uint8_t* codes, int64_t ld, uint16_t* scales, int64_t lds,
                                                          uint8_t* zeros, int64_t ldz, int gshift) {
    const int chunk = blockIdx.x * kThreads + threadIdx.x, c = 8 * chunk;
    const int lanes = 1 << (gshift - 3);          // lanes per group (4, 8 or 16, aligned)
    const bool first = (chunk & (lanes - 1)) == 0 && c < cols;
    for (int64_t r0 = (int64_t)blockIdx.y * kRows; r0 < rows; r0 += (int64_t)gridDim.y * kRows) {
        uint4 v[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r0 + i < rows && c < cols) v[i] = load8(W + (r0 + i) * ldw, c, cols);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float x[8];
            unpack8<F16>(v[i], x);
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                lo = fminf(lo, x[e]);
                hi = fmaxf(hi, x[e]);
            }
            if (zeros == nullptr) hi = fmaxf(hi, -lo);
            if (any_nonfinite<F16>(v[i])) hi = INFINITY;
            for (int d = 1; d < lanes; d *= 2) {
                hi = fmaxf(hi, __shfl_xor(hi, d));
                lo = fminf(lo, __shfl_xor(lo, d));
            }
            const bool bad = hi == INFINITY;
            const float raw = zeros == nullptr ? hi / 7.f : (hi - lo) / 15.f;
            const uint16_t s16 = bad ? (uint16_t)(F16 ? 0x7e00 : 0x7fc0) : to16<F16>(raw);
            const float s = from16<F16>(s16);
            const bool some = s != 0.f && !bad;
            const float by = some ? s : 1.f;
            float z = 8.f;
            if (zeros != nullptr && some) z = fminf(fmaxf(rintf(-lo / by), 0.f), 15.f);
            if (r0 + i >= rows || c >= cols) continue;
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float q = some ? rintf(x[e] / by) : 0.f;
                const uint32_t k = (uint32_t)(int)fminf(fmaxf(q + z, 0.f), 15.f);
                if (c + e < cols) w |= k << (4 * e);
            }
            uint8_t* dst = codes + (r0 + i) * ld + 4 * (int64_t)chunk;
            if (c + 8 <= cols) {
                *reinterpret_cast<u32_ua*>(dst) = w;
            } else {
                for (int b = 0; 2 * b < cols - c; ++b) dst[b] = (uint8_t)(w >> (8 * b));
            }
            if (first) {
                scales[(r0 + i) * lds + (c >> gshift)] = s16;
                if (zeros != nullptr) zeros[(r0 + i) * ldz + (c >> gshift)] = (uint8_t)z;
            }
        }
    }
}

template <bool F16>
__global__ __launch_bounds__(kThreads) void k_w4_dequantize(W4View q, int rows, int cols, uint16_t* out,
                                                            int64_t ldo) {
    const int chunk = blockIdx.x * kThreads + threadIdx.x, c = 8 * chunk;
    if (c >= cols) return;
    const int g = c >> q.gshift, bytes = min(4, (cols - c + 1) / 2);
    for (int64_t r0 = (int64_t)blockIdx.y * kRows; r0 < rows; r0 += (int64_t)gridDim.y * kRows) {
        uint32_t w[kRows];
        float s[kRows], zs[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + i < rows ? r0 + i : rows - 1;
            const uint8_t* src = q.codes + r * q.ld + 4 * (int64_t)chunk;
            if (bytes == 4) {
                w[i] = *reinterpret_cast<const u32_ua*>(src);
            } else {
                w[i] = 0;
                for (int b = 0; b < bytes; ++b) w[i] |= (uint32_t)src[b] << (8 * b);
            }
            s[i] = from16<F16>(q.scales[r * q.lds + g]);
            zs[i] = q.zeros == nullptr ? 8.f : (float)q.zeros[r * q.ldz + g];
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (r0 + i < rows) store8(out + (r0 + i) * ldo, c, cols, w4_eight<F16>(w[i], s[i], -zs[i] * s[i]));
    }
}

// ---- 8-bit activations -------------------------------------------------------------------
// A group's exponent e is the smallest, from kX8MinExp on, at which its largest finite magnitude is
// within E4M3's 448 = 1.75 2^8: the exponent of that magnitude less 8, one more where its fraction is
// over 1.75.  A power of two as the scale keeps every value a T (a larger one in the group never costs the
// others more than E4M3's own subnormals do), and dividing by it is exact.  At kX8MinExp the smallest
// code, 2^-9 2^e, is still a T: bf16 2^-126, fp16 2^-24.  Magnitudes that would round to 2^128 (bf16) or
// 2^16 (fp16), past T's largest number, are held at 240 2^e first.  NaN and infinities become NaN,
// the only non-finite code E4M3 has.
template <bool F16> constexpr int kX8MinExp = F16 ? -15 : -117;
template <bool F16> constexpr float kX8Limit = F16 ? 0x1.ep15f : 0x1.ep127f;

// the amax's group exponent (amax finite, >= 0)
template <bool F16>
__device__ __forceinline__ int x8_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, kX8MinExp<F16>);
}

template <bool F16>
__global__ __launch_bounds__(kThreads) void k_x8_quantize(const uint16_t* X, int64_t ldx, int rows, int cols,
                                                          uint8_t* codes, int64_t ld, uint8_t* exps, int64_t lde) {
    const int chunk = blockIdx.x * kThreads + threadIdx.x, c = 8 * chunk;
    for (int64_t r0 = (int64_t)blockIdx.y * kRows; r0 < rows; r0 += (int64_t)gridDim.y * kRows) {
        uint4 v[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r0 + i < rows && c < cols) v[i] = load8(X + (r0 + i) * ldx, c, cols);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float x[8], amax = 0.f;
            unpack8<F16>(v[i], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool fine = fabsf(x[e]) < INFINITY;
                x[e] = fine ? fminf(fmaxf(x[e], -kX8Limit<F16>), kX8Limit<F16>) : NAN;
                amax = fmaxf(amax, fine ? fabsf(x[e]) : 0.f);
            }
            amax = fmaxf(amax, __shfl_xor(amax, 1));
            amax = fmaxf(amax, __shfl_xor(amax, 2));
            const int e = x8_exponent<F16>(amax);
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);      // 2^-e, a normal number
            if (r0 + i >= rows || c >= cols) continue;
            int w0 = 0, w1 = 0;
            w0 = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * f, x[1] * f, w0, false);
            w0 = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * f, x[3] * f, w0, true);
            w1 = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * f, x[5] * f, w1, false);
            w1 = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * f, x[7] * f, w1, true);
            uint8_t* dst = codes + (r0 + i) * ld + c;
            if (c + 8 <= cols) {
                *reinterpret_cast<u32x2_ua*>(dst) = u32x2_ua{(uint32_t)w0, (uint32_t)w1};
            } else {
                const uint32_t w[2] = {(uint32_t)w0, (uint32_t)w1};
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (c + b < cols) dst[b] = (uint8_t)(w[b / 4] >> (8 * (b % 4)));
            }
            if ((chunk & 3) == 0) exps[(r0 + i) * lde + (c >> 5)] = (uint8_t)(e + 127);
        }
    }
}

template <bool F16>
__global__ __launch_bounds__(kThreads) void k_x8_dequantize(X8View q, int rows, int cols, uint16_t* out,
                                                            int64_t ldo) {
    const int chunk = blockIdx.x * kThreads + threadIdx.x, c = 8 * chunk;
    if (c >= cols) return;
    for (int64_t r0 = (int64_t)blockIdx.y * kRows; r0 < rows; r0 += (int64_t)gridDim.y * kRows) {
        uint32_t w[kRows][2];
        float f[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + i < rows ? r0 + i : rows - 1;
            const uint8_t* src = q.codes + r * q.ld + c;
            if (c + 8 <= cols) {
                const u32x2_ua v = *reinterpret_cast<const u32x2_ua*>(src);
                w[i][0] = v.x;
                w[i][1] = v.y;
            } else {
                w[i][0] = w[i][1] = 0u;
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (c + b < cols) w[i][b / 4] |= (uint32_t)src[b] << (8 * (b % 4));
            }
            f[i] = __uint_as_float((uint32_t)q.exps[r * q.lde + (c >> 5)] << 23);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (r0 + i >= rows) continue;
            const uint2 a = x8_four<F16>(w[i][0], f[i]), b = x8_four<F16>(w[i][1], f[i]);
            store8(out + (r0 + i) * ldo, c, cols, make_uint4(a.x, a.y, b.x, b.y));
        }
    }
}

__global__ __launch_bounds__(kThreads) void k_copy16(const uint16_t* in, int64_t ldi, int rows, int cols,
                                                     uint16_t* out, int64_t ldo) {
    const int c = 8 * (blockIdx.x * kThreads + threadIdx.x);
    if (c >= cols) return;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) store8(out + r * ldo, c, cols, load8(in + r * ldi, c, cols));
}

// a grid of 256 x 8 columns by `per` rows (65535 row blocks at most; the kernels stride over the rest)
dim3 grid_for(int rows, int cols, int per) {
    const unsigned gx = (unsigned)(((int64_t)cols + 8 * kThreads - 1) / (8 * kThreads));
    return dim3(gx, (unsigned)std::min<int64_t>(((int64_t)rows + per - 1) / per, 65535));
}

}  // namespace

hipError_t launch_w4_quantize(const uint16_t* W, int64_t ldw, int rows, int cols, const W4View& q, bool f16,
                              hipStream_t stream) {
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_for(rows, cols, kRows), dim3(kThreads), 0, stream, W, ldw, rows, cols,
                           const_cast<uint8_t*>(q.codes), q.ld, const_cast<uint16_t*>(q.scales), q.lds,
                           const_cast<uint8_t*>(q.zeros), q.ldz, q.gshift);
        return hipGetLastError();
    };
    return f16 ? go(k_w4_quantize<true>) : go(k_w4_quantize<false>);
}

hipError_t launch_w4_dequantize(const W4View& q, int rows, int cols, uint16_t* out, int64_t ldo, bool f16,
                                hipStream_t stream) {
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_for(rows, cols, kRows), dim3(kThreads), 0, stream, q, rows, cols, out, ldo);
        return hipGetLastError();
    };
    return f16 ? go(k_w4_dequantize<true>) : go(k_w4_dequantize<false>);
}

hipError_t launch_x8_quantize(const uint16_t* X, int64_t ldx, int rows, int cols, const X8View& q, bool f16,
                              hipStream_t stream) {
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_for(rows, cols, kRows), dim3(kThreads), 0, stream, X, ldx, rows, cols,
                           const_cast<uint8_t*>(q.codes), q.ld, const_cast<uint8_t*>(q.exps), q.lde);
        return hipGetLastError();
    };
    return f16 ? go(k_x8_quantize<true>) : go(k_x8_quantize<false>);
}

hipError_t launch_x8_dequantize(const X8View& q, int rows, int cols, uint16_t* out, int64_t ldo, bool f16,
                                hipStream_t stream) {
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_for(rows, cols, kRows), dim3(kThreads), 0, stream, q, rows, cols, out, ldo);
        return hipGetLastError();
    };
    return f16 ? go(k_x8_dequantize<true>) : go(k_x8_dequantize<false>);
}

hipError_t launch_copy16(const uint16_t* in, int64_t ldi, int rows, int cols, uint16_t* out, int64_t ldo,
                         hipStream_t stream) {
    hipLaunchKernelGGL(k_copy16, grid_for(rows, cols, 1), dim3(kThreads), 0, stream, in, ldi, rows, cols, out, ldo);
    return hipGetLastError();
}

}  // namespace gemm
