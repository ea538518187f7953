// At most 16 rows times a 4-bit matrix, x . W^T, and the products too short for any matrix instruction:
// C = epilogue(A . B), A 16-bit row-major, B stored N x K in 4-bit codes with a scale per group of columns
// (lowbit.hpp), decoded in registers on the way to the matrix instructions.
//
// With few rows the product is bound by reading W, a quarter of the bytes of a 16-bit W, so the codes go
// from memory straight to the lane that decodes them, each once: lane l of a 16 x 16 x 32 matrix
// instruction supplies column l % 16 with 8 consecutive k; it loads the 16 bytes of 32 consecutive codes, one
// group's (groups are 32 or more, aligned), the operands of four instructions, and a wavefront's load is 64
// contiguous bytes of each of 16 rows of W.  The workgroup's wavefronts take k in turn and add their sums
// through LDS in a fixed order (deterministic; no workspace).
//
// 1 x 4096 x 4096 (bf16): 5.1 us, 1.7 TB/s of W; of them 1.5 are an empty launch, and reading these 8.6 MB at
// the rate of a large copy would take 1.8.  16 x 11008 x 4096 (fp16): 10.7 to 12.6 us, 2.2 TB/s; a step's loads of A
// from L2 (as many as W's at three column blocks) and decoding are what it waits for.  Rows of A at odd multiples
// of 2 bytes cost the loads of A twice their time: 16 x 4096 x 4096 7.8 us, x 4095 16.2.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "lowbit.hpp"
#include "mma16.hpp"

namespace gemm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---- at most 16 rows, x . W^T ---------------------------------------------------------------
// Bound by the bytes of W, at the smallest sizes by latency, and in between by the number of load
// instructions a CU can issue: so W's codes are all that the loop loads when it can be.
//  * A workgroup owns 16 FN columns; its NW wavefronts take steps of 128 k in turn.  Latency is hidden by
//    the other wavefronts of the CU, not by loading further ahead: two or four steps in flight per
//    wavefront were slower everywhere (1 x 4096 x 4096 by 0.4 and 0.7 us, 1 x 11008 x 4096 by 1.0 and 1.8,
//    16 x 11008 x 4096 by 2.0), as all of a CU's data then arrives before any is decoded.
//  * Scales and zero points of the workgroup's columns are staged in LDS first, one word a group, while
//    the first codes are on their way (two scattered loads a step otherwise).
//  * XL: so is A, where it is small (a load of A from L2 carries 16 bytes for each of 16 rows, whether
//    or not there are as many); else A's fragments come from L2 with the codes.
//  * Loads are buffer loads, a per-lane offset fixed for the whole kernel plus a scalar one.  Lanes of
//    rows past M (columns past N) read past the buffer's end, which returns zero and moves nothing.
constexpr int kBufWord3 = 0x00020000;            // 32-bit unformatted data, no swizzle
constexpr unsigned kPastEnd = 0x80000000u;       // an offset past any of the buffers below (the host checks)

__device__ __forceinline__ uint4 buf16(__amdgpu_buffer_rsrc_t r, unsigned voff, int soff) {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

// words between the groups of two columns in LDS: odd, so that 16 columns fall on 16 banks
__host__ __device__ constexpr int few_stride(int groups) { return groups | 1; }
// bytes between two rows of A in LDS: the 16 rows read together 16 bytes apart in the banks
__host__ __device__ constexpr int few_row(int K) { return (K * 2 + 255) / 256 * 256 + 16; }

template <bool F16, int FN, int NW, bool XL>
__global__ __launch_bounds__(64 * NW) void k_w4_few(W4Problem p) {
    constexpr int BN = 16 * FN, KU = 128, T = 64 * NW;
    extern __shared__ __align__(16) unsigned char lds[];
    uint32_t* sz = reinterpret_cast<uint32_t*>(lds);                 // [BN][few_stride]: scale | zero << 16

    const int n0 = blockIdx.x * BN, tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lq = lane >> 4;
    const int K = p.K, gs = p.w.gshift, cols = min(BN, p.N - n0);
    const int kb = (K + 1) / 2, groups = ((K - 1) >> gs) + 1, gw = few_stride(groups);
    unsigned char* xl = lds + (BN * gw * 4 + 15) / 16 * 16;
    // (each buffer ends with its last row's last element)
    const int ea = (int)(((int64_t)(p.M - 1) * p.lda + K) * 2), ec = (int)((int64_t)(cols - 1) * p.w.ld + kb);
    const uint8_t* codes = p.w.codes + (int64_t)n0 * p.w.ld;
    auto buffer = [](const void* base, int bytes) {
        return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, bytes, kBufWord3);
    };
    // this lane's 32 k of a step start at 32 lq
    const unsigned avoff = li < p.M ? (unsigned)(li * (int)p.lda * 2 + 64 * lq) : kPastEnd;
    unsigned cvoff[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j)
        cvoff[j] = 16 * j + li < cols ? (unsigned)((16 * j + li) * (int)p.w.ld + 16 * lq) : kPastEnd;

    uint4 c[FN], a[4];
    const int whole = K / KU;
    const __amdgpu_buffer_rsrc_t rc = buffer(codes, ec), ra = buffer(p.A, ea);
    // (readfirstlane: otherwise the compiler takes the step for a lane's own and steps through the lanes' values of
    // it around every load)
    auto load = [&](int step) {
        const int u = __builtin_amdgcn_readfirstlane(step);
#pragma unroll
        for (int j = 0; j < FN; ++j) c[j] = buf16(rc, cvoff[j], u * 64);
        if constexpr (!XL) {
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = buf16(ra, avoff + 16 * t, u * 256);
        }
    };
    // (Every path to a use of the loaded registers writes them, here and in the loop: with undefined values on
    // one path this compiler gave a decoded operand the registers of codes still to be read.  Wavefronts beyond the
    // last step load the last, and do not use it.)
    load(max(0, min(wave, whole - 1)));

    // the scales and zero points of this workgroup's columns, and A
    for (int i = tid; i < cols * groups; i += T) {
        const int nn = i / groups, g = i - nn * groups;
        const uint32_t sc = p.w.scales[(n0 + nn) * p.w.lds + g];
        const uint32_t zz = p.w.zeros != nullptr ? p.w.zeros[(n0 + nn) * p.w.ldz + g] : 8u;
        sz[nn * gw + g] = sc | zz << 16;
    }
    const int xrow = few_row(K);
    if constexpr (XL) {
        const int chunks = (K + 7) / 8;
        for (int m = 0; m < p.M; ++m) {
            const uint8_t* row = reinterpret_cast<const uint8_t*>(p.A + (int64_t)m * p.lda);
            for (int i = tid; i < chunks; i += T)
                *reinterpret_cast<uint4*>(xl + m * xrow + 16 * i) =
                    shift_down(load_end(row, 16 * (int64_t)i, 2 * (int64_t)K), end_shift(16 * (int64_t)i, 2 * (int64_t)K));
        }
    }
    __syncthreads();

    f32x4 acc[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // columns past N take the last one's scales: what they give is never stored
    const uint32_t* szl[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) szl[j] = sz + min(16 * j + li, cols - 1) * gw;
    const unsigned char* xrd = xl + min(li, p.M - 1) * xrow;
    // this lane's 32 k from k0 on; `last`: only the first `left` of them lie before K
    auto multiply = [&](int k0, bool last, int left) {
        uint4 x[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if constexpr (XL) {
                x[t] = *reinterpret_cast<const uint4*>(xrd + (last ? min(k0 + 8 * t, (K - 1) & ~7) : k0 + 8 * t) * 2);
                if (last && left <= 8 * t) x[t] = make_uint4(0u, 0u, 0u, 0u);
            } else
                x[t] = a[t];
        }
        const int g = (last ? min(k0, K - 1) : k0) >> gs;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t v = szl[j][g];
            const float sc = from16<F16>((uint16_t)v), zs = -sc * (float)(v >> 16);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint4 b = w4_eight<F16>(word(c[j], t), sc, zs);
                if (last) b = keep_first(b, left - 8 * t);
                acc[j] = mma_16x16x32<F16>(__builtin_bit_cast(bf16x8, x[t]), __builtin_bit_cast(bf16x8, b), acc[j]);
            }
        }
    };
    for (int u = wave; u < whole; u += NW) {            // (uniform)
        if (u != wave) load(u);
        multiply(u * KU + 32 * lq, false, 0);
    }
    if (K % KU != 0 && whole % NW == wave) {            // the step that K ends in (uniform)
        const int k = whole * KU + 32 * lq;
#pragma unroll
        for (int j = 0; j < FN; ++j)
            c[j] = load_end(codes + (int64_t)min(16 * j + li, cols - 1) * p.w.ld, k / 2, kb);
        if constexpr (!XL) {
            const uint8_t* row = reinterpret_cast<const uint8_t*>(p.A + (int64_t)min(li, p.M - 1) * p.lda);
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = load_end(row, 2 * (k + 8 * t), 2 * (int64_t)K);
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = shift_down(a[t], end_shift(2 * (k + 8 * t), 2 * (int64_t)K));
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) c[j] = shift_down(c[j], end_shift(k / 2, kb));
        multiply(k, true, K - k);
    }

    // ---- the wavefronts' sums, added in their order (a thread per output); then the epilogue ----
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(lds);                      // [NW][FN][64]
#pragma unroll
    for (int j = 0; j < FN; ++j) red[(wave * FN + j) * 64 + lane] = acc[j];
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(lds);
    for (int i = tid; i < FN * 256; i += T) {
        // value i: fragment i / 256, its lane (i / 4) % 64, register i % 4
        const int row = 4 * ((i >> 6) & 3) + (i & 3), col = n0 + 16 * (i >> 8) + ((i >> 2) & 15);
        float sum = sums[i];
#pragma unroll
        for (int w = 1; w < NW; ++w) sum += sums[w * FN * 256 + i];
        if (row >= p.M || col >= p.N) continue;
        const int64_t off = (int64_t)row * p.ldc + col;
        const float old = p.e.beta != 0.f ? epi_load(p.e, p.C, off) : 0.f;
        epi_store(p.e, p.C, off, epi_apply(p.e, sum, old, p.e.bias == nullptr ? 0.f : p.e.bias[col]));
    }
}

// Fewer than 32 k, or 32 columns of dy . W (rows of codes shorter than a lane's 16 bytes): a thread per
// element of C.
template <bool F16>
__global__ __launch_bounds__(256) void k_w4_short(W4Problem p) {
    const int64_t total = (int64_t)p.M * p.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / p.N), col = (int)(i % p.N);
        float sum = 0.f;
        for (int k = 0; k < p.K; ++k) {
            const int64_t r = p.tr ? k : col;
            const int c = p.tr ? col : k, g = c >> p.w.gshift;
            const uint32_t code = (p.w.codes[r * p.w.ld + c / 2] >> (4 * (c & 1))) & 15u;
            const float s = from16<F16>(p.w.scales[r * p.w.lds + g]);
            const float z = p.w.zeros == nullptr ? 8.f : (float)p.w.zeros[r * p.w.ldz + g];
            sum = fmaf(from16<F16>(p.A[row * p.lda + k]), from16<F16>(to16<F16>(fmaf((float)code, s, -z * s))), sum);
        }
        const int64_t off = row * p.ldc + col;
        const float old = p.e.beta != 0.f ? epi_load(p.e, p.C, off) : 0.f;
        epi_store(p.e, p.C, off, epi_apply(p.e, sum, old, p.e.bias == nullptr ? 0.f : p.e.bias[col]));
    }
}

// LDS of a workgroup of k_w4_few: scales, and A where it is staged, then the wavefronts' sums over both.
constexpr int64_t kFewLds = 64 << 10;
int64_t few_lds(const W4Problem& p, int fn, int nw, bool xl) {
    const int64_t groups = ((p.K - 1) >> p.w.gshift) + 1;
    const int64_t stage = (16 * fn * (groups | 1) * 4 + 15) / 16 * 16 + (xl ? p.M * ((int64_t)p.K * 2 + 272) : 0);
    return std::max<int64_t>(stage, (int64_t)nw * fn * 1024);
}

// Column blocks of 16 per workgroup.  With A in LDS one: more workgroups a CU, some of which load while
// others decode (1 x 11008 x 4096: 8.7 us; two and three were 1.7 and 1.4 slower).  Else the fewest columns
// on the busiest CU, then the widest, since every workgroup reads A (16 x 11008 x 4096: three 10.7 us, one
// 16.4, two 15.0; 16 x 4096 x 4096: one 7.8, two 9.2).  0: the staged operands do not fit.
bool few_in_lds(const W4Problem& p) { return p.M <= 4 && few_lds(p, 1, 16, true) <= kFewLds; }

int few_blocks(const W4Problem& p, int cus, bool xl) {
    if (xl) return 1;
    int best = 0;
    int64_t cost = INT64_MAX;
    for (int fn = 1; fn <= 4; ++fn) {
        if (few_lds(p, fn, 16, false) > kFewLds) break;
        const int64_t blocks = ((int64_t)p.N + 16 * fn - 1) / (16 * fn), c = (blocks + cus - 1) / cus * fn;
        if (c <= cost) { cost = c; best = fn; }
    }
    return best;
}

template <bool F16, int FN, int NW, bool XL>
hipError_t launch_few_one(const W4Problem& p, hipStream_t stream) {
    const int64_t blocks = ((int64_t)p.N + 16 * FN - 1) / (16 * FN);
    hipLaunchKernelGGL((k_w4_few<F16, FN, NW, XL>), dim3((unsigned)blocks), dim3(64 * NW),
                       (unsigned)few_lds(p, FN, NW, XL), stream, p);
    return hipGetLastError();
}

// 16 wavefronts a workgroup, or 8 where a CU gets several workgroups or K has few steps for each.
template <bool F16>
hipError_t launch_few(const W4Problem& p, int fn, bool xl, int cus, hipStream_t stream) {
    const bool wide = ((int64_t)p.N + 15) / 16 <= cus && p.K >= 64 * 128;
    if (xl) return wide ? launch_few_one<F16, 1, 16, true>(p, stream) : launch_few_one<F16, 1, 8, true>(p, stream);
    switch (fn) {
        case 1: return wide ? launch_few_one<F16, 1, 16, false>(p, stream) : launch_few_one<F16, 1, 8, false>(p, stream);
        case 2: return launch_few_one<F16, 2, 16, false>(p, stream);
        case 3: return launch_few_one<F16, 3, 16, false>(p, stream);
        default: return launch_few_one<F16, 4, 16, false>(p, stream);
    }
}

}  // namespace

bool w4_few_applies(const W4Problem& p, int cus) {
    // offsets within a block's rows that buffer loads can hold
    const int64_t lim = (int64_t)1 << 30;
    return !p.tr && p.M <= 16 && p.K >= 32 && 16 * p.lda < lim / 2 && 64 * p.w.ld < lim && 64 * p.w.lds < lim / 2 &&
           64 * p.w.ldz < lim && few_blocks(p, cus, few_in_lds(p)) > 0;
}

hipError_t launch_w4_few(const W4Problem& p, bool f16, int cus, hipStream_t stream, const char*& name) {
    const bool xl = few_in_lds(p);
    const int fn = few_blocks(p, cus, xl);
    name = f16 ? "f16_w4_few" : "bf16_w4_few";
    return f16 ? launch_few<true>(p, fn, xl, cus, stream) : launch_few<false>(p, fn, xl, cus, stream);
}

hipError_t launch_w4_short(const W4Problem& p, bool f16, hipStream_t stream, const char*& name) {
    const int64_t blocks = ((int64_t)p.M * p.N + 255) / 256;
    name = f16 ? "f16_w4_short" : "bf16_w4_short";
    hipLaunchKernelGGL(f16 ? k_w4_short<true> : k_w4_short<false>, dim3((unsigned)std::min<int64_t>(blocks, 65536)),
                       dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace gemm
