// 4-bit weights and 8-bit activations: rounding 16-bit matrices to codes, and the 16-bit numbers
// that codes stand for (formats in lowbit.hpp).
//
// Every kernel reads its input once and writes its output once, so the time is that of the bytes.
// A lane owns 8 consecutive columns (16 bytes of the 16-bit side; a wavefront's access to a row is
// 1 KB contiguous) of kRows rows, all of whose loads are issued before the first is used (2 rows: rounding 4096 x 4096 to 4 bits 12.3
// us against 13.4 with 4 and 12.8 with 1, 11008 x 4096 22.4, 21.8 and 26.0).  A
// group's columns lie in 4 to 16 neighbouring lanes, which agree on its largest magnitude (or its
// extremes) by exchanging values; one of them writes the scale.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "lowbit.hpp"

namespace gemm {
namespace {

constexpr int kThreads = 256, kRows = 2;

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

// ---- 4-bit weights -----------------------------------------------------------------------
// Symmetric (no zeros): s = T(amax / 7), code = round(w / s) + 8.  With zero points: the range always
// includes 0, s = T((max - min) / 15), z = round(-min / s), code = round(w / s) + z; codes and z are held
// in 0 .. 15.  s == 0 (a group of zeros, or of numbers too small for a scale of type T): every code is
// the zero point 8.  A group with an infinity or a NaN gets a NaN scale: all of it stands for NaN.
//
// Roundings are those of correctly rounded divisions, at 3 instructions a quotient: q = a y for y near
// 1 / b, then q + (a - b q) y, the residual exact.  No quotient of two T lies within FP32's rounding of a border
// between two codes unless it is that border, and there the second step is exact (all significands of both
// types and y up to 2 ulp off were tried: 59 million quotients); for b = 7 and 15 it is the correctly rounded
// quotient of every FP32 significand (tried too).  With the compiler's own divisions and an extreme at a time
// in FP32 the instructions, not the bytes, set the time: 19.9 us at 4096 x 4096 (bf16, group 128, zero
// points) and 37.2 at 11008 x 4096 (fp16, symmetric), 3.0 TB/s; so, with extremes of packed 16-bit keys exchanged by
// lane permutations of the register file, 12.3 (3.4 TB/s) and 22.4 us (5.1 TB/s).
__device__ __forceinline__ float quotient(float a, float b, float y) {
    const float q = a * y;
    return fmaf(fmaf(-q, b, a), y, q);
}

// d / (7 or 15), correctly rounded (subnormal results and infinity by the plain division)
template <int B>
__device__ __forceinline__ float over(float d) {
    if (!(d >= 0x1p-100f && d < INFINITY)) return d / B;
    return quotient(d, (float)B, 1.f / B);
}

// the integer nearest to a q of at most 2^22, ties to even
__device__ __forceinline__ int nearest(float q) { return (int)(__float_as_uint(q + 0x1.8p23f) - 0x4b400000u); }

typedef short i16x2 __attribute__((ext_vector_type(2)));

// the larger of each half among the 2^k lanes of a group (4, 8 or 16 lanes, all active)
__device__ __forceinline__ i16x2 group_max(i16x2 v, int lanes) {
    auto with = [&](auto dpp) {
        const int o = dpp(__builtin_bit_cast(int, v));
        v = __builtin_elementwise_max(v, __builtin_bit_cast(i16x2, o));
    };
    with([](int u) { return __builtin_amdgcn_mov_dpp(u, 0xb1, 0xf, 0xf, true); });       // lane ^ 1
    with([](int u) { return __builtin_amdgcn_mov_dpp(u, 0x4e, 0xf, 0xf, true); });       // lane ^ 2
    if (lanes > 4) with([](int u) { return __builtin_amdgcn_mov_dpp(u, 0x141, 0xf, 0xf, true); });   // 7 - lane
    if (lanes > 8) with([](int u) { return __builtin_amdgcn_mov_dpp(u, 0x140, 0xf, 0xf, true); });   // 15 - lane
    return v;
}

// ZP: with zero points
template <bool F16, bool ZP>
__global__ __launch_bounds__(kThreads) void k_w4_quantize(const uint16_t* W, int64_t ldw, int rows, int cols,
                                                          uint8_t* codes, int64_t ld, uint16_t* scales, int64_t lds,
                                                          uint8_t* zeros, int64_t ldz, int gshift) {
    constexpr short kInf = F16 ? 0x7c00 : 0x7f80;
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
            // Extremes of the bit patterns: magnitudes (no zero points), or keys that order as the numbers do
            // (negative numbers with the bits below the sign inverted; not-a-numbers beyond the infinities).
            // top: the largest in its second half, ~ the smallest key in its first.
            i16x2 most = {0, 0}, least = {0, 0};
#pragma unroll
            for (uint32_t w : {v[i].x, v[i].y, v[i].z, v[i].w}) {
                if constexpr (ZP) {
                    const i16x2 s = __builtin_bit_cast(i16x2, w);
                    const i16x2 key = s ^ ((s >> 15) & (short)0x7fff);
                    most = __builtin_elementwise_max(most, key);
                    least = __builtin_elementwise_min(least, key);
                } else {
                    most = __builtin_elementwise_max(most, __builtin_bit_cast(i16x2, w & 0x7fff7fffu));
                }
            }
            const i16x2 top = group_max(i16x2{(short)~min(least.x, least.y), max(most.x, most.y)}, lanes);
            const bool bad = top.y >= kInf || (ZP && top.x >= kInf);
            const float hi = from16<F16>((uint16_t)top.y);
            const float lo = ZP ? -from16<F16>((uint16_t)max(top.x, (short)0)) : 0.f;
            const uint16_t s16 = bad ? (uint16_t)(F16 ? 0x7e00 : 0x7fc0) : to16<F16>(ZP ? over<15>(hi - lo) : over<7>(hi));
            float s = from16<F16>(s16), x[8], low = lo;
            unpack8<F16>(v[i], x);
            const bool some = s > 0.f && s < INFINITY;
            if (!F16 && !(s >= 0x1p-100f && s <= 0x1p100f) && some) {
                // bf16 scales whose reciprocal or residuals could leave FP32's range: all by a power of two
                const float by = s < 1.f ? 0x1p64f : 0x1p-64f;
                s *= by;
                low *= by;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= by;
            }
            const float y = __builtin_amdgcn_rcpf(s);
            // (an infinite scale, from a range past FP32: zero point and codes 0, as quotients over it are)
            int z = 8;
            if (ZP) z = some ? min(max(nearest(quotient(-low, s, y)), 0), 15) : s == INFINITY ? 0 : 8;
            if (r0 + i >= rows || c >= cols) continue;
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w |= (uint32_t)min(max(nearest(quotient(x[e], s, y)) + z, 0), 15) << (4 * e);
            if (!some) w = 0x11111111u * (uint32_t)z;
            uint8_t* dst = codes + (r0 + i) * ld + 4 * (int64_t)chunk;
            if (c + 8 <= cols) {
                *reinterpret_cast<u32_ua*>(dst) = w;
            } else {
                w &= (1u << (4 * (cols - c))) - 1;       // (the half byte after an odd last column is 0)
                for (int b = 0; 2 * b < cols - c; ++b) dst[b] = (uint8_t)(w >> (8 * b));
            }
            if (first) {
                scales[(r0 + i) * lds + (c >> gshift)] = s16;
                if (ZP) zeros[(r0 + i) * ldz + (c >> gshift)] = (uint8_t)z;
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
__device__ __forceinline__ void x8_dequantize_rows(const X8View& q, int rows, int cols, uint16_t* out, int64_t ldo) {
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

template <bool F16>
__global__ __launch_bounds__(kThreads) void k_x8_dequantize(X8View q, int rows, int cols, uint16_t* out, int64_t ldo) {
    x8_dequantize_rows<F16>(q, rows, cols, out, ldo);
}

// The 16-bit operands of a weight gradient in one launch: X's numbers (grid z = 0), and dY in rows of whole
// chunks of 8 (z = 1; its columns past the end are left as they are, and give rows of C that do not exist).
template <bool F16>
__global__ __launch_bounds__(kThreads) void k_x8_operands(X8View q, int rows, int cols, uint16_t* out, int64_t ldo,
                                                          const uint16_t* dy, int64_t lddy, int n, uint16_t* dy_out,
                                                          int64_t ld_dy_out) {
    if (blockIdx.z == 0) {
        x8_dequantize_rows<F16>(q, rows, cols, out, ldo);
        return;
    }
    const int c = 8 * (blockIdx.x * kThreads + threadIdx.x);
    if (c >= n) return;
    for (int64_t r0 = (int64_t)blockIdx.y * kRows; r0 < rows; r0 += (int64_t)gridDim.y * kRows) {
        uint4 v[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) v[i] = load8(dy + min(r0 + i, (int64_t)rows - 1) * lddy, c, n);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (r0 + i < rows) store8(dy_out + (r0 + i) * ld_dy_out, c, n, v[i]);
    }
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
    if (q.zeros != nullptr) return f16 ? go(k_w4_quantize<true, true>) : go(k_w4_quantize<false, true>);
    return f16 ? go(k_w4_quantize<true, false>) : go(k_w4_quantize<false, false>);
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

hipError_t launch_x8_operands(const X8View& q, int rows, int cols, uint16_t* out, int64_t ldo, const uint16_t* dy,
                              int64_t lddy, int n, uint16_t* dy_out, int64_t ld_dy_out, bool f16, hipStream_t stream) {
    dim3 grid = grid_for(rows, std::max(cols, n), kRows);
    grid.z = 2;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, q, rows, cols, out, ldo, dy, lddy, n, dy_out, ld_dy_out);
        return hipGetLastError();
    };
    return f16 ? go(k_x8_operands<true>) : go(k_x8_operands<false>);
}

}  // namespace gemm
