// 16-bit rows times a 4-bit matrix, x . W^T, from about 16 rows to the size at which W is worth writing as
// 16-bit numbers: C = epilogue(A . B), B stored N x K in 4-bit codes (lowbit.hpp).
//
// Between the few-row product, bound by W's bytes, and the large one, bound by matrix instructions, the
// costs are decoding W (19 vector instructions for the 8 codes of a lane's operand, once per
// wavefront) and moving A from L2 (once per workgroup).  So a wavefront decodes 32 FN columns of W into
// registers, never through LDS, and multiplies each operand with 32 FM rows of A, which all wavefronts of
// the workgroup share in LDS:
//  * v_mfma_f32_32x32x16: lane l supplies column l % 32 of a block and, of a step of 64 k, the 32
//    consecutive k from 32 (l / 32) on: one 16-byte load of codes, one group's, the operands of four
//    instructions.  A's lanes read the same k.
//  * A's tile of a step (32 FM rows of 64 k, 128 bytes each) is loaded into registers a step ahead and
//    stored to the other of two LDS buffers, one barrier a step; 16-byte chunk c of row r at
//    c ^ (r mod 8) ^ (bit 3 of r), so that the rows read together fall on different banks.
//  * K is divided among workgroups where the tiles alone would leave CUs idle (grid y): each
//    slice's sums go to the workspace, and a second kernel adds them in slice order and applies the
//    epilogue (deterministic).
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "lowbit.hpp"
#include "mma16.hpp"

namespace gemm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kWavesN = 4, kThreads = 64 * kWavesN, kStep = 64;

__device__ __forceinline__ int chunk_at(int row, int c) { return c ^ (row & 7) ^ ((row >> 3) & 1); }

// part != nullptr: slice blockIdx.y's sums, dense M x N, to part + blockIdx.y M N, without the epilogue.
// vec: rows of C (of the slices' sums) allow 16-byte FP32 or 8-byte 16-bit accesses.
template <bool F16, int FM, int FN, bool ZP>
__global__ __launch_bounds__(kThreads, 2) void k_w4_tile(W4Problem p, int kslice, float* part, int vec) {
    constexpr int BM = 32 * FM, BN = 32 * FN * kWavesN, ROW = 2 * kStep;     // LDS row bytes
    constexpr int XL = BM * 8 / kThreads;                                    // 16-byte chunks of A per thread and step
    constexpr int EP = 32 * FN + 4;                                          // epilogue: floats per staged row
    constexpr int XBYTES = BM * ROW, EBYTES = kWavesN * 32 * EP * 4;
    static_assert(XL >= 1 && BM * 8 % kThreads == 0, "whole chunks per thread");
    __shared__ __align__(16) unsigned char lds[2 * XBYTES > EBYTES ? 2 * XBYTES : EBYTES];

    const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, tiles_m, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, h = lane >> 5;
    const int k_begin = blockIdx.y * kslice, K = min(p.K, k_begin + kslice);
    const int wn = n0 + wave * 32 * FN;

    // this lane's columns of W from k 32 h on, and the chunks of A that this thread stages: chunk t % 8 of
    // rows t / 8 + 32 i.  Rows of A past M and columns past N are read as the last one: their products are
    // never stored.
    const uint8_t* crow[FN];
    const uint16_t* srow[FN];
    const uint8_t* zrow[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int64_t n = min(wn + 32 * j + l32, p.N - 1);
        crow[j] = p.w.codes + n * p.w.ld;
        srow[j] = p.w.scales + n * p.w.lds;
        zrow[j] = ZP ? p.w.zeros + n * p.w.ldz : nullptr;
    }
    const int xc = threadIdx.x & 7, xr = threadIdx.x >> 3;
    const uint8_t* arow[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i)
        arow[i] = reinterpret_cast<const uint8_t*>(p.A + (int64_t)min(m0 + xr + 32 * i, p.M - 1) * p.lda);

    f32x16 acc[FM][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[f][j][r] = 0.f;

    uint4 c[2][FN], x[XL];
    uint16_t s[2][FN];
    uint8_t z[2][FN];
    auto load = [&](int b, int k0) {                    // a step wholly inside K
        const int k = k0 + 32 * h, g = k >> p.w.gshift;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const u32x4_ub v = *reinterpret_cast<const u32x4_ub*>(crow[j] + k / 2);
            c[b][j] = make_uint4(v.x, v.y, v.z, v.w);
            s[b][j] = srow[j][g];
            if constexpr (ZP) z[b][j] = zrow[j][g];
        }
#pragma unroll
        for (int i = 0; i < XL; ++i) x[i] = load16(arow[i] + 2 * (k0 + 8 * xc));
    };
    unsigned char* xst = lds + xr * ROW + 16 * chunk_at(xr, xc);             // (rows 32 apart swizzle alike)
    auto store = [&](int b) {
#pragma unroll
        for (int i = 0; i < XL; ++i) *reinterpret_cast<uint4*>(xst + b * XBYTES + 32 * i * ROW) = x[i];
    };
    auto multiply = [&](int b, bool end, int left) {    // end: only `left` of this lane's k lie before K
        float sc[FN], zs[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            sc[j] = from16<F16>(s[b][j]);
            zs[j] = -sc[j] * (ZP ? (float)z[b][j] : 8.f);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint4 a[FM];
#pragma unroll
            for (int f = 0; f < FM; ++f)
                a[f] = *reinterpret_cast<const uint4*>(lds + b * XBYTES + (32 * f + l32) * ROW + 16 * chunk_at(l32, 4 * h + t));
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                uint4 w = w4_eight<F16>((&c[b][j].x)[t], sc[j], zs[j]);
                if (end) w = keep_first(w, left - 8 * t);
#pragma unroll
                for (int f = 0; f < FM; ++f)
                    acc[f][j] = mma_32x32x16<F16>(__builtin_bit_cast(bf16x8, a[f]), __builtin_bit_cast(bf16x8, w), acc[f][j]);
            }
        }
    };

    // whole steps, the next one's loads under the current one's products (past the last, the last again:
    // no branch, so that the compiler can count the loads in flight)
    const int n = (K - k_begin) / kStep;
    if (n > 0) {
        load(0, k_begin);
        store(0);
        __syncthreads();
        for (int i = 0; i < n; i += 2) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (b == 1 && i + 1 >= n) break;        // uniform
                load(b ^ 1, k_begin + min(i + b + 1, n - 1) * kStep);
                multiply(b, false, 0);
                store(b ^ 1);
                __syncthreads();
            }
        }
    }
    // the step that K ends in: the rows' last 16 bytes, shifted into place (the host makes sure that rows
    // have 32 k)
    if (K - k_begin > n * kStep) {
        const int k0 = k_begin + n * kStep, k = k0 + 32 * h, g = min(k, p.K - 1) >> p.w.gshift;
        const int64_t cb = (p.K + 1) / 2, ab = 2 * (int64_t)p.K, ak = 2 * ((int64_t)k0 + 8 * xc);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            c[0][j] = load_end(crow[j], k / 2, cb);
            s[0][j] = srow[j][g];
            if constexpr (ZP) z[0][j] = zrow[j][g];
        }
#pragma unroll
        for (int i = 0; i < XL; ++i) x[i] = load_end(arow[i], ak, ab);
#pragma unroll
        for (int j = 0; j < FN; ++j) c[0][j] = shift_down(c[0][j], end_shift(k / 2, cb));
#pragma unroll
        for (int i = 0; i < XL; ++i) x[i] = shift_down(x[i], end_shift(ak, ab));
        store(0);
        __syncthreads();
        multiply(0, true, p.K - k);
        __syncthreads();
    }

    // ---- epilogue: a 32-row band at a time through this wavefront's part of LDS, whole rows stored ----
    const bool split = part != nullptr;
    const Epilogue e = split ? Epilogue{1.f, 0.f, nullptr, 0, kActNone, kOutF32} : p.e;
    void* C = split ? static_cast<void*>(part + (int64_t)blockIdx.y * p.M * p.N) : p.C;
    const int64_t ldc = split ? p.N : p.ldc;
    constexpr int LPR = 8 * FN, RPI = 64 / LPR;          // lanes per row, rows per store
    float* band = reinterpret_cast<float*>(lds) + wave * 32 * EP;
    const int cc = 4 * (lane % LPR), col = wn + cc;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (e.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < p.N) bias[i] = e.bias[col + i];
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        // accumulator layout: lane l, register r holds row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) band[(8 * (r >> 2) + 4 * h + (r & 3)) * EP + 32 * j + l32] = acc[f][j][r];
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int q = 0; q < 32 / RPI; ++q) {
            const int rr = q * RPI + lane / LPR, row = m0 + 32 * f + rr;
            if (row >= p.M || col >= p.N) continue;
            const float4 v = *reinterpret_cast<const float4*>(band + rr * EP + cc);
            const float a[4] = {v.x, v.y, v.z, v.w};
            const int64_t off = (int64_t)row * ldc + col;
            float old[4] = {0.f, 0.f, 0.f, 0.f}, y[4];
            const bool four = vec != 0 && col + 3 < p.N;
            if (e.beta != 0.f) {
                if (four) {
                    epi_load4(e, C, off, old);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (col + i < p.N) old[i] = epi_load(e, C, off + i);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = epi_apply(e, a[i], old[i], bias[i]);
            if (four) {
                epi_store4(e, C, off, y);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + i < p.N) epi_store(e, C, off + i, y[i]);
            }
        }
    }
}

// C = epilogue(slab 0 + slab 1 + ...), the slabs dense M x N, added in order.
__global__ __launch_bounds__(256) void k_w4_join(W4Problem p, const float* part, int slices) {
    const int64_t total = (int64_t)p.M * p.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / p.N), col = (int)(i % p.N);
        float sum = part[i];
        for (int s = 1; s < slices; ++s) sum += part[s * total + i];
        const int64_t off = (int64_t)row * p.ldc + col;
        const float old = p.e.beta != 0.f ? epi_load(p.e, p.C, off) : 0.f;
        epi_store(p.e, p.C, off, epi_apply(p.e, sum, old, p.e.bias == nullptr ? 0.f : p.e.bias[col]));
    }
}

template <bool F16, int FM, int FN>
hipError_t launch_tile(const W4Problem& p, const W4Split& sp, float* part, hipStream_t stream) {
    constexpr int BM = 32 * FM, BN = 32 * FN * kWavesN;
    const int64_t tiles = (((int64_t)p.M + BM - 1) / BM) * (((int64_t)p.N + BN - 1) / BN);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles, (unsigned)sp.slices);
    float* out = sp.slices > 1 ? part : nullptr;
    // 16-byte FP32 or 8-byte 16-bit groups of four columns (the slices' sums start 16-byte aligned)
    const uintptr_t align = p.e.out == kOutF32 ? 16 : 8;
    const int vec = out != nullptr ? p.N % 4 == 0 : p.ldc % 4 == 0 && reinterpret_cast<uintptr_t>(p.C) % align == 0;
    if (p.w.zeros != nullptr)
        hipLaunchKernelGGL((k_w4_tile<F16, FM, FN, true>), grid, dim3(kThreads), 0, stream, p, sp.kslice, out, vec);
    else
        hipLaunchKernelGGL((k_w4_tile<F16, FM, FN, false>), grid, dim3(kThreads), 0, stream, p, sp.kslice, out, vec);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || sp.slices == 1) return err;
    const int64_t blocks = ((int64_t)p.M * p.N + 255) / 256;
    hipLaunchKernelGGL(k_w4_join, dim3((unsigned)std::min<int64_t>(blocks, 4096)), dim3(256), 0, stream, p, part,
                       sp.slices);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_type(const W4Problem& p, const W4Split& sp, float* part, hipStream_t stream) {
    if (sp.fm == 1) return launch_tile<F16, 1, 1>(p, sp, part, stream);
    if (sp.fm == 2) return sp.fn == 2 ? launch_tile<F16, 2, 2>(p, sp, part, stream) : launch_tile<F16, 2, 1>(p, sp, part, stream);
    return launch_tile<F16, 4, 2>(p, sp, part, stream);
}

}  // namespace

W4Split w4_split(int64_t M, int64_t N, int64_t K, int cus) {
    W4Split s;
    s.fm = M <= 32 ? 1 : M <= 64 ? 2 : 4;
    s.fn = s.fm == 4 ? 2 : 1;
    const int64_t bm = 32 * s.fm, bn = 128 * s.fn, tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
    const int64_t steps = (K + kStep - 1) / kStep;
    // as many slices as give every CU a workgroup, of at least four steps each
    int64_t slices = std::max<int64_t>(1, std::min<int64_t>(cus / std::max<int64_t>(1, tiles), steps / 4));
    const int64_t per = (steps + slices - 1) / slices;
    slices = (steps + per - 1) / per;
    s.kslice = (int)(per * kStep);
    s.slices = (int)slices;
    s.bytes = slices > 1 ? (size_t)slices * M * N * 4 : 0;
    return s;
}

hipError_t launch_w4_tile(const W4Problem& p, const W4Split& sp, bool f16, float* part, hipStream_t stream,
                          const char*& name) {
    static const char* names[2][2] = {{"bf16_w4_tile", "f16_w4_tile"}, {"bf16_w4_tile_splitk", "f16_w4_tile_splitk"}};
    name = names[sp.slices > 1 ? 1 : 0][f16 ? 1 : 0];
    return f16 ? launch_type<true>(p, sp, part, stream) : launch_type<false>(p, sp, part, stream);
}

}  // namespace gemm
