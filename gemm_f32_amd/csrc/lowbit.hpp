// Low-bit operands: 4-bit weights with a scale (and a zero point) per group of columns, and 8-bit
// activations with an exponent per 32 columns.  Their formats, the conversions between codes and
// the 16-bit numbers they stand for, and the launchers of lowbit_codec.hip and w4_rows.hip.
//
// Both decode to a 16-bit number T (bf16 or fp16), and every product reads exactly these numbers: a
// 4-bit code c of a group with scale s and zero point z stands for the T nearest to (c - z) s (the
// product of an integer of at most 8 bits and an 8- or 11-bit fraction is exact in FP32, so this is
// one rounding, of half a step); an 8-bit code stands for e4m3(code) 2^e, which is a T.
#pragma once

#include "common.hpp"
#include "epilogue.hpp"

namespace gemm {

// A 4-bit matrix of rows x cols as kernels see it.  codes: two to a byte along a row, even columns
// in the low half; scales: T bit patterns; zeros: one byte per group, nullptr: 8 everywhere.  The
// group of column c is c >> gshift.
struct W4View {
    const uint8_t* codes;
    int64_t ld;
    const uint16_t* scales;
    int64_t lds;
    const uint8_t* zeros;
    int64_t ldz;
    int gshift;
};

// 8-bit activations: E4M3 codes and one exponent byte (e + 127) per group of 32 columns.
struct X8View {
    const uint8_t* codes;
    int64_t ld;
    const uint8_t* exps;
    int64_t lde;
};

// C (M x N, row-major) = epilogue(A . B), A 16-bit row-major, B 4-bit: stored N x K, groups along k
// (tr == 0: a layer's forward product x . W^T) or K x N, groups along n (tr == 1: dy . W).
struct W4Problem {
    int M, N, K;
    const uint16_t* A;
    int64_t lda;
    W4View w;
    int tr;
    void* C;
    int64_t ldc;
    Epilogue e;
};

hipError_t launch_w4_quantize(const uint16_t* W, int64_t ldw, int rows, int cols, const W4View& q, bool f16,
                              hipStream_t stream);
// out: T, leading dimension ldo
hipError_t launch_w4_dequantize(const W4View& q, int rows, int cols, uint16_t* out, int64_t ldo, bool f16,
                                hipStream_t stream);
hipError_t launch_x8_quantize(const uint16_t* X, int64_t ldx, int rows, int cols, const X8View& q, bool f16,
                              hipStream_t stream);
hipError_t launch_x8_dequantize(const X8View& q, int rows, int cols, uint16_t* out, int64_t ldo, bool f16,
                                hipStream_t stream);
// rows x cols 16-bit elements into rows of ldo elements
hipError_t launch_x8_operands(const X8View& q, int rows, int cols, uint16_t* out, int64_t ldo, const uint16_t* dy,
                              int64_t lddy, int n, uint16_t* dy_out, int64_t ld_dy_out, bool f16, hipStream_t stream);
// The products (w4_rows.hip, w4_tile.hip); each sets the name that gemm_last_kernel() reports.
// Fewer than 32 k (or, dy . W, 32 columns): any M, N, either order.
hipError_t launch_w4_short(const W4Problem& p, bool f16, hipStream_t stream, const char*& name);
// x . W^T, M <= 16, K >= 32, within the offsets and LDS that w4_few_applies checks.
bool w4_few_applies(const W4Problem& p, int cus);
hipError_t launch_w4_few(const W4Problem& p, bool f16, int cus, hipStream_t stream, const char*& name);
// Either order, any M, N, K >= 32 (dy . W: N >= 32 too); K in `slices` slices of `kslice`, whose sums (dense M x N, FP32) take `bytes` at
// `part` (slices == 1: none).  fm: 32-row blocks of a workgroup, wv: its wavefronts, of 32 columns each.
struct W4Split {
    int fm = 1, wv = 4, slices = 1, kslice = 0;
    size_t bytes = 0;
    double us = 0;               // the model's time
};
W4Split w4_split(int64_t M, int64_t N, int64_t K, bool tr, int cus, bool workspace);
// The model's time of writing W as 16-bit numbers and multiplying these.
double w4_decoded_us(int64_t M, int64_t N, int64_t K, int cus);
hipError_t launch_w4_tile(const W4Problem& p, const W4Split& sp, bool f16, float* part, hipStream_t stream,
                          const char*& name);

#ifdef __HIPCC__
typedef float lb_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 lb_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 lb_f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32_ua __attribute__((aligned(1)));
typedef uint16_t u16_ua __attribute__((aligned(1)));
typedef unsigned int u32x2_ua __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned int u32x4_ub __attribute__((ext_vector_type(4), aligned(1)));

// word i (a constant) of four
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// two FP32 values -> two T, each to nearest, ties to even (one conversion instruction)
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    const lb_f32x2 v = {a, b};
    if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, lb_f16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, lb_bf16x2));
}

template <bool F16>
__device__ __forceinline__ float from16(uint16_t u) {
    if constexpr (F16) return (float)__builtin_bit_cast(_Float16, u);
    else return __uint_as_float((uint32_t)u << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t to16(float y) {
    if constexpr (F16) return to_f16(y);
    else return to_bf16(y);
}

// Eight codes of one group (nibble i of w: column i) as T, in column order.  c s - z s is formed in
// FP32: both products and their difference are exact, so the conversion's rounding is the only one.
// A code as a byte is an E4M3 pattern of value c 2^-9 (subnormal up to 7, then exponent 1), so the
// 8-bit conversion with scale 2^9 turns two codes into floats in one instruction: 19 vector
// instructions for 8 codes (field extraction and integer conversion took 28).
template <bool F16>
__device__ __forceinline__ uint4 w4_eight(uint32_t w, float s, float minus_zs) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    const lb_f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.f, false),
                   e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.f, true),
                   o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.f, false),
                   o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.f, true);
    uint4 r;
    r.x = pack16<F16>(fmaf(e0.x, s, minus_zs), fmaf(o0.x, s, minus_zs));
    r.y = pack16<F16>(fmaf(e0.y, s, minus_zs), fmaf(o0.y, s, minus_zs));
    r.z = pack16<F16>(fmaf(e1.x, s, minus_zs), fmaf(o1.x, s, minus_zs));
    r.w = pack16<F16>(fmaf(e1.y, s, minus_zs), fmaf(o1.y, s, minus_zs));
    return r;
}

// Four E4M3 codes times 2^e, f = 2^e, as T (exact for codes and exponents that launch_x8_quantize writes)
template <bool F16>
__device__ __forceinline__ uint2 x8_four(uint32_t w, float f) {
    const lb_f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return make_uint2(pack16<F16>(a.x * f, a.y * f), pack16<F16>(b.x * f, b.y * f));
}
// The 16 bytes v shifted down by n bytes (n >= 0; 16 and more leave nothing), zero from above.  By whole
// words, then by bytes within them: selections, no branch on the lane.
__device__ __forceinline__ uint4 shift_down(uint4 v, int n) {
    if (n & 8) v = make_uint4(v.z, v.w, 0u, 0u);
    if (n & 4) v = make_uint4(v.y, v.z, v.w, 0u);
    v = make_uint4(__builtin_amdgcn_alignbyte(v.y, v.x, n & 3), __builtin_amdgcn_alignbyte(v.z, v.y, n & 3),
                   __builtin_amdgcn_alignbyte(v.w, v.z, n & 3), __builtin_amdgcn_alignbyte(0u, v.w, n & 3));
    return n < 16 ? v : make_uint4(0u, 0u, 0u, 0u);
}

// The end of a row of n >= 16 bytes: where the 16 bytes from byte i on would run past it, the row's last
// 16 are loaded instead (load_end), and shifted into place once they are there (shift_down by end_shift).
__device__ __forceinline__ uint4 load_end(const uint8_t* row, int64_t i, int64_t n) {
    const u32x4_ub v = *reinterpret_cast<const u32x4_ub*>(row + min(i, n - 16));
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ int end_shift(int64_t i, int64_t n) { return (int)max((int64_t)0, min(i - (n - 16), (int64_t)16)); }

// keep the first n of 8 packed elements (n may be negative or over 8)
__device__ __forceinline__ uint4 keep_first(uint4 v, int n) {
    auto mask = [n](int i) { return (n > 2 * i ? 0xffffu : 0u) | (n > 2 * i + 1 ? 0xffff0000u : 0u); };
    return make_uint4(v.x & mask(0), v.y & mask(1), v.z & mask(2), v.w & mask(3));
}

#endif

}  // namespace gemm
