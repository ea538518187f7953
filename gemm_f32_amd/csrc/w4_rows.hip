// Few rows times a 4-bit matrix: C = epilogue(A . B), A 16-bit row-major, B in 4-bit codes with a scale
// per group of columns (lowbit.hpp), decoded in registers on the way to the matrix instructions.
//
// With few rows the product is bound by reading B, a quarter of the bytes of a 16-bit B, so B goes
// from memory straight to the lane that decodes it, and each code is read and decoded once per
// 16 FM rows.  Two orders of B:
//  * TR = false, B stored N x K (x . W^T): lane l of a 16 x 16 x 32 matrix instruction supplies
//    column l % 16 with 8 consecutive k.  It loads the 16 bytes of 32 consecutive codes, one group's
//    (groups are 32 or more, aligned), which are the operands of four instructions: a wavefront's
//    load is 64 contiguous bytes of each of 16 rows of W.
//  * TR = true, B stored K x N (dy . W): k runs over the rows of W.  Lane l loads two bytes, columns
//    4 (l % 16) .. + 3, of each of the 8 rows 8 (l / 16) ..: code j of each is the operand of
//    instruction j, which computes columns 4 i + j.  No transposition in LDS.
// The workgroup's 8 wavefronts take k in turn and add their sums through LDS in a fixed order
// (deterministic; no workspace).
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "lowbit.hpp"
#include "mma16.hpp"

namespace gemm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;

// 8 elements of a row of A from k on; zero past K
__device__ __forceinline__ uint4 load_a(const uint16_t* row, int k, int K, bool whole) {
    if (whole || k + 8 <= K) return load16(row + k);
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < K ? row[k + e] : 0u;
    return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

// keep the first n of 8 packed elements (n may be negative or over 8)
__device__ __forceinline__ uint4 keep_first(uint4 v, int n) {
    uint32_t* w = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= (n > 2 * i ? 0xffffu : 0u) | (n > 2 * i + 1 ? 0xffff0000u : 0u);
    return v;
}

template <bool F16, int FM, int FN, bool TR>
__global__ __launch_bounds__(64 * kWaves) void k_w4_rows(W4Problem p) {
    static_assert(!TR || FN == 4, "two bytes of a row of W are four columns");
    constexpr int BM = 16 * FM, BN = 16 * FN;
    constexpr int KU = TR ? 32 : 128;               // k per wavefront and step
    __shared__ f32x4 red[kWaves][FM][FN][64];

    const int slabs = (p.N + BN - 1) / BN, rblocks = (p.M + BM - 1) / BM;
    int rb, slab;
    tile_coords(blockIdx.x, rblocks, slabs, rblocks, rb, slab);
    const int n0 = slab * BN, m0 = rb * BM;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lq = lane >> 4;
    const int K = p.K;

    // rows of A past M are read as the last one: their products are never stored
    const uint16_t* arow[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) arow[f] = p.A + (int64_t)min(m0 + 16 * f + li, p.M - 1) * p.lda;

    f32x4 acc[FM][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto mma = [&](int f, int j, const uint4& a, const uint4& b) {
        acc[f][j] = mma_16x16x32<F16>(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc[f][j]);
    };

    const int steps = (K + KU - 1) / KU;
    if constexpr (!TR) {
        // this lane's column of each block (the last one past N) and its row of W
        const uint8_t* crow[FN];
        const uint16_t* srow[FN];
        const uint8_t* zrow[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int64_t n = min(n0 + 16 * j + li, p.N - 1);
            crow[j] = p.w.codes + n * p.w.ld;
            srow[j] = p.w.scales + n * p.w.lds;
            zrow[j] = p.w.zeros == nullptr ? nullptr : p.w.zeros + n * p.w.ldz;
        }
        for (int u = wave; u < steps; u += kWaves) {
            const int k = u * KU + 32 * lq;             // this lane's 32 k
            const bool whole = (u + 1) * KU <= K;       // uniform
            uint4 c[FN], a[FM][4];
            float s[FN], zs[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                c[j] = make_uint4(0u, 0u, 0u, 0u);
                s[j] = zs[j] = 0.f;
                if (whole || k + 32 <= K) {
                    const u32x4_ub v = *reinterpret_cast<const u32x4_ub*>(crow[j] + k / 2);
                    c[j] = make_uint4(v.x, v.y, v.z, v.w);
                } else if (k < K) {                     // the row's last bytes
                    uint32_t* w = &c[j].x;
#pragma unroll
                    for (int b = 0; b < 16; ++b)
                        if (k + 2 * b < K) w[b / 4] |= (uint32_t)crow[j][k / 2 + b] << (8 * (b % 4));
                }
                if (whole || k < K) {
                    s[j] = from16<F16>(srow[j][k >> p.w.gshift]);
                    zs[j] = -s[j] * (zrow[j] == nullptr ? 8.f : (float)zrow[j][k >> p.w.gshift]);
                }
            }
#pragma unroll
            for (int f = 0; f < FM; ++f)
#pragma unroll
                for (int t = 0; t < 4; ++t) a[f][t] = load_a(arow[f], k + 8 * t, K, whole);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    uint4 b = w4_eight<F16>((&c[j].x)[t], s[j], zs[j]);
                    if (!whole) b = keep_first(b, K - (k + 8 * t));
#pragma unroll
                    for (int f = 0; f < FM; ++f) mma(f, j, a[f][t], b);
                }
            }
        }
    } else {
        // this lane's four columns (the last ones where they lie past N)
        const int c = min(n0 + 4 * li, (p.N - 1) & ~3), g = c >> p.w.gshift;
        const bool two = c + 3 <= p.N;                  // both bytes exist (N odd: the last half byte does)
        for (int u = wave; u < steps; u += kWaves) {
            const int k = u * KU + 8 * lq;              // this lane's 8 k
            const bool whole = (u + 1) * KU <= K;       // uniform
            uint32_t w[8];
            float s[8], zs[8];
            uint4 a[FM];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t r = min(k + e, K - 1);
                const uint8_t* src = p.w.codes + r * p.w.ld + c / 2;
                w[e] = two ? (uint32_t)*reinterpret_cast<const u16_ua*>(src) : (uint32_t)*src;
                s[e] = from16<F16>(p.w.scales[r * p.w.lds + g]);
                zs[e] = -s[e] * (p.w.zeros == nullptr ? 8.f : (float)p.w.zeros[r * p.w.ldz + g]);
            }
#pragma unroll
            for (int f = 0; f < FM; ++f) a[f] = load_a(arow[f], k, K, whole);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = fmaf((float)((w[e] >> (4 * j)) & 15u), s[e], zs[e]);
                uint4 b = make_uint4(pack16<F16>(x[0], x[1]), pack16<F16>(x[2], x[3]), pack16<F16>(x[4], x[5]),
                                     pack16<F16>(x[6], x[7]));
                if (!whole) b = keep_first(b, K - k);
#pragma unroll
                for (int f = 0; f < FM; ++f) mma(f, j, a[f], b);
            }
        }
    }

    // ---- the wavefronts' sums, added in their order; then the epilogue ----
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int j = 0; j < FN; ++j) red[wave][f][j][lane] = acc[f][j];
    __syncthreads();
    for (int i = wave; i < FM * FN; i += kWaves) {
        const int f = i / FN, j = i % FN;
        f32x4 sum = red[0][f][j][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += red[w][f][j][lane];
        const int col = TR ? n0 + 4 * li + j : n0 + 16 * j + li;
        if (col >= p.N) continue;
        const float bias = p.e.bias == nullptr ? 0.f : p.e.bias[col];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = m0 + 16 * f + 4 * lq + r;
            if (row >= p.M) continue;
            const int64_t off = (int64_t)row * p.ldc + col;
            const float old = p.e.beta != 0.f ? epi_load(p.e, p.C, off) : 0.f;
            epi_store(p.e, p.C, off, epi_apply(p.e, sum[r], old, bias));
        }
    }
}

template <bool F16, int FM>
hipError_t launch_fm(const W4Problem& p, int fn, hipStream_t stream) {
    auto go = [&](auto kernel, int bn) {
        const int64_t blocks = (((int64_t)p.N + bn - 1) / bn) * (((int64_t)p.M + 16 * FM - 1) / (16 * FM));
        if (blocks > INT32_MAX) return hipErrorInvalidValue;
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * kWaves), 0, stream, p);
        return hipGetLastError();
    };
    if (p.tr) return go(k_w4_rows<F16, FM, 4, true>, 64);
    if (fn == 4) return go(k_w4_rows<F16, FM, 4, false>, 64);
    if (fn == 2) return go(k_w4_rows<F16, FM, 2, false>, 32);
    return go(k_w4_rows<F16, FM, 1, false>, 16);
}

template <bool F16>
hipError_t launch_type(const W4Problem& p, int fm, int fn, hipStream_t stream) {
    if (fm == 1) return launch_fm<F16, 1>(p, fn, stream);
    if (fm == 2) return launch_fm<F16, 2>(p, fn, stream);
    return launch_fm<F16, 4>(p, fn, stream);
}

}  // namespace

hipError_t launch_w4_rows(const W4Problem& p, bool f16, int cus, hipStream_t stream, const char*& name) {
    const int fm = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
    const int64_t rblocks = ((int64_t)p.M + 16 * fm - 1) / (16 * fm);
    int fn = 4;
    while (!p.tr && fn > 1 && rblocks * ((p.N + 16 * fn - 1) / (16 * fn)) < cus) fn /= 2;
    static const char* names[2][2] = {{"bf16_w4_rows", "f16_w4_rows"}, {"bf16_w4_rows_t", "f16_w4_rows_t"}};
    name = names[p.tr ? 1 : 0][f16 ? 1 : 0];
    return f16 ? launch_type<true>(p, fm, fn, stream) : launch_type<false>(p, fm, fn, stream);
}

}  // namespace gemm
