// 16-bit rows times a 4-bit matrix, x . W^T, from about 16 rows to the size at which W is worth writing as
// 16-bit numbers: C = epilogue(A . B), B stored N x K in 4-bit codes (lowbit.hpp).
//
// Between the few-row product, bound by W's bytes, and the large one, bound by matrix instructions, the
// costs are decoding W (19 vector instructions for the 8 codes of a lane's operand, once per
// wavefront) and moving A from L2 (once per workgroup).  So a wavefront decodes 32 columns of W into
// registers, never through LDS, and multiplies each operand with 32 FM rows of A, which all WV wavefronts of
// the workgroup share in LDS:
//  * v_mfma_f32_32x32x16: lane l supplies column l % 32 and, of a step of 128 k, the 64 consecutive k from
//    64 (l / 32) on, the operands of eight instructions, from 32 bytes of codes; A's lanes read the same
//    k.  The next operand is decoded between the matrix instructions of the current one (one of them keeps
//    the matrix unit busy for 32 cycles, in which the wavefront can issue seven vector instructions).
//  * A's tiles (a step: 32 FM rows of 128 k, 256 bytes each) are copied from memory straight into a ring of
//    three LDS stages, two steps ahead, as are W's codes, scales and zero points into registers; one
//    barrier a step.  16-byte chunk c of row r lies at c ^ (r mod 16), so that the rows read together fall
//    on different banks.
//  * K is divided among workgroups where the tiles alone would leave CUs idle (grid y): each
//    slice's sums go to the workspace, and a second kernel adds them in slice order and applies the
//    epilogue (deterministic).
#include <algorithm>
#include <cmath>

#include "common.hpp"
#include "launch.hpp"
#include "lowbit.hpp"
#include "mma16.hpp"

namespace gemm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kStep = 128, kRing = 3;
constexpr int kBufWord3 = 0x00020000;            // 32-bit unformatted data, no swizzle
typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes a lane straight into LDS.  (A function of its own: with the builtin inside the kernel's lambda the
// host pass of this compiler silently drops the kernel's launch stub.)
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t r, lds_void* dst, unsigned voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, voff, soff, 0, 0);
}

__device__ __forceinline__ int chunk_at(int row, int c) { return c ^ (row & 15); }

// The 32 FM x 32 sums of a wavefront through the epilogue (part != nullptr: as they are, to the slice's dense
// M x N), a 32-row band at a time through `band`, this wavefront's 32 rows of kEpRow floats in LDS, so that whole rows
// are stored.  vec: rows of C (of the slices' sums) allow 16-byte FP32 or 8-byte 16-bit accesses.
constexpr int kEpRow = 32 + 4;
template <int FM>
__device__ __forceinline__ void store_tile(const W4Problem& p, float* part, int vec, const f32x16 (&acc)[FM], float* band,
                                           int m0, int wn, int lane) {
    const int l32 = lane & 31, h = lane >> 5;
    const bool split = part != nullptr;
    const Epilogue e = split ? Epilogue{1.f, 0.f, nullptr, 0, kActNone, kOutF32} : p.e;
    void* C = split ? static_cast<void*>(part + (int64_t)blockIdx.y * p.M * p.N) : p.C;
    const int64_t ldc = split ? p.N : p.ldc;
    constexpr int LPR = 8, RPI = 64 / LPR;               // lanes per row, rows per store
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
        for (int r = 0; r < 16; ++r) band[(8 * (r >> 2) + 4 * h + (r & 3)) * kEpRow + l32] = acc[f][r];
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int q = 0; q < 32 / RPI; ++q) {
            const int rr = q * RPI + lane / LPR, row = m0 + 32 * f + rr;
            if (row >= p.M || col >= p.N) continue;
            const float4 v = *reinterpret_cast<const float4*>(band + rr * kEpRow + cc);
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

// part != nullptr: slice blockIdx.y's sums, dense M x N, to part + blockIdx.y M N, without the epilogue.
// G32: groups of 32 (a lane's 64 k of a step lie in two).
// FAR: the rows of A of a workgroup span more than a buffer's 31 bits; every step is then staged through
// registers, as the step that K ends in always is.
template <bool F16, int FM, int WV, bool ZP, bool G32, bool FAR>
__global__ __launch_bounds__(64 * WV, 2) void k_w4_tile(W4Problem p, int kslice, float* part, int vec) {
    constexpr int BM = 32 * FM, BN = 32 * WV, ROW = 2 * kStep, T = 64 * WV;     // ROW: LDS row bytes
    constexpr int EP = kEpRow;                                               // epilogue: floats per staged row
    constexpr int XBYTES = BM * ROW, EBYTES = WV * 32 * EP * 4, NG = G32 ? 2 : 1;
    // of a wavefront and step, copies into LDS and the loads that at least follow the step before's copies (the
    // codes'; the compiler makes one load of a lane's two scales or zero points)
    constexpr int COPIES = BM / 4 / WV, LOADS = COPIES + 2;
    static_assert(COPIES >= 1 && BM % (4 * WV) == 0, "whole copies per wavefront");
    __shared__ __align__(16) unsigned char lds[kRing * XBYTES > EBYTES ? kRing * XBYTES : EBYTES];

    const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, tiles_m, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, h = lane >> 5;
    const int k_begin = blockIdx.y * kslice, K = min(p.K, k_begin + kslice);
    const int wn = n0 + wave * 32, gs = p.w.gshift;

    // this lane's column of W (the last one past N: its products are never stored)
    const int64_t n = min(wn + l32, p.N - 1);
    const uint8_t* crow = p.w.codes + n * p.w.ld;
    const uint16_t* srow = p.w.scales + n * p.w.lds;
    const uint8_t* zrow = ZP ? p.w.zeros + n * p.w.ldz : nullptr;

    f32x16 acc[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[f][r] = 0.f;

    uint4 c[kRing][2];
    uint16_t s[kRing][NG];
    uint8_t z[kRing][NG];
    // a wavefront copies rows 4 (COPIES wave + i) .. + 3, lane l row l / 16's chunk for position l % 16; rows
    // past M are read as the last one
    const int abytes = FAR ? 0 : (int)((min(p.M - m0, BM) - 1) * p.lda * 2 + 2 * (int64_t)p.K);
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.A + (int64_t)m0 * p.lda), (short)0, abytes, kBufWord3);
    unsigned avoff[COPIES];
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int r = 4 * (COPIES * wave + i) + (lane >> 4);
        avoff[i] = FAR ? 0u : (unsigned)(min(r, p.M - 1 - m0) * (int)p.lda * 2 + 16 * chunk_at(r, lane & 15));
    }
    auto load = [&](int b, int k0) {                    // a step wholly inside K
        const int k = k0 + 64 * h;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            s[b][j] = srow[(k >> gs) + j];
            if constexpr (ZP) z[b][j] = zrow[(k >> gs) + j];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const u32x4_ub v = *reinterpret_cast<const u32x4_ub*>(crow + k / 2 + 16 * j);
            c[b][j] = make_uint4(v.x, v.y, v.z, v.w);
        }
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            lds_void* dst = (lds_void*)(lds + b * XBYTES + (COPIES * wave + i) * 1024);
            copy_to_lds(ra, dst, avoff[i], 2 * k0);
        }
    };
    auto multiply = [&](int b, bool end, int left) {    // end: only `left` of this lane's k lie before K
        float sc[NG], zs[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            sc[j] = from16<F16>(s[b][j]);
            zs[j] = -sc[j] * (ZP ? (float)z[b][j] : 8.f);
        }
        // operand t: 8 k of W, and of A's rows (read as 16-bit vectors: with that type the compiler adds no
        // wait for the copies in flight)
        auto decode = [&](int t) -> uint4 {
            const uint32_t w = word(c[b][t / 4], t % 4);
            const uint4 v = w4_eight<F16>(w, sc[G32 ? t / 4 : 0], zs[G32 ? t / 4 : 0]);
            return end ? keep_first(v, left - 8 * t) : v;
        };
        auto rows = [&](int t, int f) -> bf16x8 {
            return *reinterpret_cast<const bf16x8*>(lds + b * XBYTES + (32 * f + l32) * ROW + 16 * chunk_at(l32, 8 * h + t));
        };
        // A's operands are read AHEAD - 1 instructions' worth ahead (an LDS read takes as long as four matrix
        // instructions)
        constexpr int AHEAD = FM == 1 ? 8 : FM == 2 ? 4 : 3;
        uint4 w[2];
        bf16x8 a[AHEAD][FM];
#pragma unroll
        for (int t = 0; t < AHEAD - 1; ++t)
#pragma unroll
            for (int f = 0; f < FM; ++f) a[t][f] = rows(t, f);
        w[0] = decode(0);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t + AHEAD - 1 < 8) {
#pragma unroll
                for (int f = 0; f < FM; ++f) a[(t + AHEAD - 1) % AHEAD][f] = rows(t + AHEAD - 1, f);
            }
            if (t < 7) w[(t + 1) & 1] = decode(t + 1);
#pragma unroll
            for (int f = 0; f < FM; ++f)
                acc[f] = mma_32x32x16<F16>(a[t % AHEAD][f], __builtin_bit_cast(bf16x8, w[t & 1]), acc[f]);
#pragma unroll
            for (int f = 0; f < FM; ++f) {              // a matrix instruction, a read, a share of the decoding
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, (20 + FM - 1) / FM, 0);
            }
        }
    };

    // Whole steps.  At the barrier of step i every wavefront has waited for its own copies of step i (all but the
    // LOADS newest loads are then there, and step i + 1 has issued at least as many) and is done with step i - 1, whose stage then takes step i + 2.  Past the
    // last step the last is loaded again, into a stage that nobody reads: no branch.
    const int whole = FAR ? 0 : (K - k_begin) / kStep;
    if (!FAR && whole > 0) {                            // uniform
#pragma unroll
        for (int r = 0; r < kRing - 1; ++r) load(r, k_begin + min(r, whole - 1) * kStep);
        for (int i = 0; i < whole; i += kRing) {
#pragma unroll
            for (int r = 0; r < kRing; ++r) {
                if (r > 0 && i + r >= whole) break;     // uniform
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"((kRing - 2) * LOADS) : "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                load((r + kRing - 1) % kRing, k_begin + min(i + r + kRing - 1, whole - 1) * kStep);
                multiply(r, false, 0);
            }
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");      // the surplus copies land before LDS is reused
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
    // The step that K ends in (FAR: every step): where the 16 bytes would run past a row's end, its last 16
    // shifted into place (the host makes sure that rows have 32 k).  Thread t stages chunk t % 16 of rows
    // t / 16 + T / 16 i.
    constexpr int XL = BM * 16 / T;
    for (int k0 = k_begin + whole * kStep; k0 < K; k0 += kStep) {
        const int xc = threadIdx.x & 15, xr = threadIdx.x >> 4;
        const int k = k0 + 64 * h;
        const int64_t cb = (p.K + 1) / 2, ab = 2 * (int64_t)p.K, ak = 2 * ((int64_t)k0 + 8 * xc);
        uint4 x[XL];
#pragma unroll
        for (int j = 0; j < 2; ++j) c[0][j] = load_end(crow, k / 2 + 16 * j, cb);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int g = min(k + 32 * j, p.K - 1) >> gs;
            s[0][j] = srow[g];
            if constexpr (ZP) z[0][j] = zrow[g];
        }
#pragma unroll
        for (int i = 0; i < XL; ++i)
            x[i] = load_end(reinterpret_cast<const uint8_t*>(p.A + (int64_t)min(m0 + xr + T / 16 * i, p.M - 1) * p.lda), ak, ab);
#pragma unroll
        for (int j = 0; j < 2; ++j) c[0][j] = shift_down(c[0][j], end_shift(k / 2 + 16 * j, cb));
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int r = xr + T / 16 * i;
            *reinterpret_cast<uint4*>(lds + r * ROW + 16 * chunk_at(r, xc)) = shift_down(x[i], end_shift(ak, ab));
        }
        __syncthreads();
        multiply(0, true, p.K - k);
        __syncthreads();
    }

    store_tile<FM>(p, part, vec, acc, reinterpret_cast<float*>(lds) + wave * 32 * EP, m0, wn, lane);
}

// dy . W: k runs over the rows of W.  A thread decodes 32 codes of one row (16 bytes, one group) and stores
// them as T to one of two LDS tiles of 64 k by 128 columns, a step ahead; gfx950's transposing LDS read then
// hands each lane 8 consecutive k of a column.  Row r of the tile is 256 bytes in four groups of 32 columns,
// group q at q ^ (r mod 4), so that the four rows that one read takes lie on different banks.  A as in the
// kernel above, 64 k a step: 128-byte rows, chunk c at c ^ (r mod 8) ^ (bit 3 of r).
constexpr int kStepT = 64, kRingT = 4, kWavesT = 4, kColsT = 32 * kWavesT;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// (through a restrict-qualified parameter: the inlined read then carries alias information, without which the
// compiler makes it wait for every copy into LDS in flight)
__device__ __forceinline__ s16x4 lds_read_tr(lds_s16x4* __restrict__ p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p); }
__device__ __forceinline__ int chunk64_at(int row, int c) { return c ^ (row & 7) ^ ((row >> 3) & 1); }

template <bool F16, int FM, bool ZP, bool FAR>
__global__ __launch_bounds__(64 * kWavesT, 2) void k_w4_tile_t(W4Problem p, int kslice, float* part, int vec) {
    constexpr int BM = 32 * FM, ROW = 2 * kStepT, T = 64 * kWavesT;
    constexpr int XBYTES = BM * ROW, WROW = 2 * kColsT, WBYTES = kStepT * WROW, EBYTES = kWavesT * 32 * kEpRow * 4;
    constexpr int COPIES = BM / 8 / kWavesT, LOADS = COPIES + (ZP ? 3 : 2);
    constexpr int STAGES = kRingT * XBYTES + 2 * WBYTES;
    static_assert(T * 32 == kStepT * kColsT, "32 codes per thread and step");
    __shared__ __align__(16) unsigned char lds[STAGES > EBYTES ? STAGES : EBYTES];
    unsigned char* wl = lds + kRingT * XBYTES;

    const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + kColsT - 1) / kColsT;
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, tiles_m, tm, tn);
    const int m0 = tm * BM, n0 = tn * kColsT;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, h = lane >> 5;
    const int k_begin = blockIdx.y * kslice, K = min(p.K, k_begin + kslice);

    // this thread's 32 columns of row kr of a step; where their 16 bytes would run past the row's end, its last
    // 16 are loaded and shifted into place (columns past N: their products are never stored)
    const int kr = threadIdx.x >> 2, q = threadIdx.x & 3, nb = (p.N + 1) / 2;
    const int off = min(n0 / 2 + 16 * q, nb - 16), shift = min(n0 / 2 + 16 * q - off, 16);
    const bool edge = n0 + kColsT > 2 * nb;             // uniform
    const int g = min(n0 + 32 * q, p.N - 1) >> p.w.gshift;
    unsigned char* wst = wl + kr * WROW + ((q ^ (kr & 3)) << 6);

    f32x16 acc[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[f][r] = 0.f;

    uint4 c[kRingT];
    uint16_t s[kRingT];
    uint8_t z[kRingT];
    const int abytes = FAR ? 0 : (int)((min(p.M - m0, BM) - 1) * p.lda * 2 + 2 * (int64_t)p.K);
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.A + (int64_t)m0 * p.lda), (short)0, abytes, kBufWord3);
    unsigned avoff[COPIES];
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int r = 8 * (COPIES * wave + i) + (lane >> 3);
        avoff[i] = FAR ? 0u : (unsigned)(min(r, p.M - 1 - m0) * (int)p.lda * 2 + 16 * chunk64_at(r, lane & 7));
    }
    auto load_w = [&](int b, int k0) {
        const int64_t r = min(k0 + kr, p.K - 1);
        const u32x4_ub v = *reinterpret_cast<const u32x4_ub*>(p.w.codes + r * p.w.ld + off);
        c[b] = make_uint4(v.x, v.y, v.z, v.w);
        s[b] = p.w.scales[r * p.w.lds + g];
        if constexpr (ZP) z[b] = p.w.zeros[r * p.w.ldz + g];
    };
    auto load_x = [&](int b, int k0) {
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            lds_void* dst = (lds_void*)(lds + b * XBYTES + (COPIES * wave + i) * 1024);
            copy_to_lds(ra, dst, avoff[i], 2 * k0);
        }
    };
    // ring slot b's codes as T into tile w; rows past K as zeros (stored as 16-bit vectors: with that type the
    // compiler adds no wait for the copies in flight)
    auto decode = [&](int b, int w, bool keep) {
        const float sc = from16<F16>(s[b]), zs = -sc * (ZP ? (float)z[b] : 8.f);
        uint4 v = c[b];
        if (edge) v = shift_down(v, shift);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 t = w4_eight<F16>(u[i], sc, zs);
            if (!keep) t = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<bf16x8*>(wst + w * WBYTES + 16 * i) = __builtin_bit_cast(bf16x8, t);
        }
    };
    const int l16 = lane & 15, rr = 8 * h + (l16 >> 2);
    const unsigned wrd = (unsigned)(rr * WROW + ((wave ^ (rr & 3)) << 6) + 32 * ((lane >> 4) & 1) + 8 * (l16 & 3));
    auto multiply = [&](int b, int w) {
#pragma unroll
        for (int t = 0; t < kStepT / 16; ++t) {
            const unsigned char* src = wl + w * WBYTES + wrd + 16 * t * WROW;
            const s16x4 lo = lds_read_tr((lds_s16x4*)src);
            const s16x4 hi = lds_read_tr((lds_s16x4*)(src + 4 * WROW));
            const bf16x8 v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const bf16x8 a = *reinterpret_cast<const bf16x8*>(lds + b * XBYTES + (32 * f + l32) * ROW +
                                                                  16 * chunk64_at(l32, 2 * t + h));
                acc[f] = mma_32x32x16<F16>(a, v, acc[f]);
            }
        }
    };

    // Whole steps.  Step i is decoded during step i - 1, into the tile that step i - 2 was read from; A's stages
    // as in the kernel above.
    const int whole = FAR ? 0 : (K - k_begin) / kStepT;
    if (!FAR && whole > 0) {                            // uniform
        auto load = [&](int b, int i) {
            load_w(b, k_begin + min(i, whole - 1) * kStepT);
            load_x(b, k_begin + min(i, whole - 1) * kStepT);
        };
#pragma unroll
        for (int r = 0; r < kRingT - 1; ++r) load(r, r);
        decode(0, 0, true);
        constexpr int TURN = kRingT;                     // (even: both rings' indices are constants in a turn)
        for (int i = 0; i < whole; i += TURN) {
#pragma unroll
            for (int r = 0; r < TURN; ++r) {
                if (r > 0 && i + r >= whole) break;     // uniform
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"((kRingT - 2) * LOADS) : "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                load((r + kRingT - 1) % kRingT, i + r + kRingT - 1);
                decode((r + 1) % kRingT, (r + 1) & 1, true);      // (past the last step: a tile that nobody reads)
                multiply(r % kRingT, r & 1);
            }
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");      // the surplus copies land before LDS is reused
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
    // the step that K ends in (FAR: every step)
    constexpr int XL = BM * 8 / T;
    for (int k0 = k_begin + whole * kStepT; k0 < K; k0 += kStepT) {
        const int xc = threadIdx.x & 7, xr = threadIdx.x >> 3;
        const int64_t ab = 2 * (int64_t)p.K, ak = 2 * ((int64_t)k0 + 8 * xc);
        uint4 x[XL];
        load_w(0, k0);
#pragma unroll
        for (int i = 0; i < XL; ++i)
            x[i] = load_end(reinterpret_cast<const uint8_t*>(p.A + (int64_t)min(m0 + xr + T / 8 * i, p.M - 1) * p.lda), ak, ab);
        decode(0, 0, k0 + kr < p.K);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int r = xr + T / 8 * i;
            *reinterpret_cast<uint4*>(lds + r * ROW + 16 * chunk64_at(r, xc)) = shift_down(x[i], end_shift(ak, ab));
        }
        __syncthreads();
        multiply(0, 0);
        __syncthreads();
    }
    store_tile<FM>(p, part, vec, acc, reinterpret_cast<float*>(lds) + wave * 32 * kEpRow, m0, n0 + 32 * wave, lane);
}

template <bool F16, int FM, int WV, bool TR>
hipError_t launch_tile(const W4Problem& p, const W4Split& sp, float* part, hipStream_t stream) {
    constexpr int BM = 32 * FM, BN = 32 * WV;
    const int64_t tiles = (((int64_t)p.M + BM - 1) / BM) * (((int64_t)p.N + BN - 1) / BN);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles, (unsigned)sp.slices);
    float* out = sp.slices > 1 ? part : nullptr;
    // 16-byte FP32 or 8-byte 16-bit groups of four columns (the slices' sums start 16-byte aligned)
    const uintptr_t align = p.e.out == kOutF32 ? 16 : 8;
    const int vec_c = p.ldc % 4 == 0 && reinterpret_cast<uintptr_t>(p.C) % align == 0;
    const int vec = out != nullptr ? p.N % 4 == 0 : vec_c;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(64 * WV), 0, stream, p, sp.kslice, out, vec);
        return hipGetLastError();
    };
    const bool zp = p.w.zeros != nullptr, g32 = p.w.gshift == 5, far = (int64_t)BM * p.lda * 2 >= (int64_t)1 << 31;
    if (far && FM != 1) return hipErrorInvalidValue;     // (launch_w4_tile gives far rows tiles of 32)
    constexpr bool F = FM == 1;
    hipError_t err;
    if constexpr (TR) {
        static_assert(WV == kWavesT, "128 columns");
        err = far ? zp ? go(k_w4_tile_t<F16, FM, true, F>) : go(k_w4_tile_t<F16, FM, false, F>)
                  : zp ? go(k_w4_tile_t<F16, FM, true, false>) : go(k_w4_tile_t<F16, FM, false, false>);
    } else {
        err = far ? g32 ? zp ? go(k_w4_tile<F16, FM, WV, true, true, F>) : go(k_w4_tile<F16, FM, WV, false, true, F>)
                        : zp ? go(k_w4_tile<F16, FM, WV, true, false, F>) : go(k_w4_tile<F16, FM, WV, false, false, F>)
            : g32 ? zp ? go(k_w4_tile<F16, FM, WV, true, true, false>) : go(k_w4_tile<F16, FM, WV, false, true, false>)
                  : zp ? go(k_w4_tile<F16, FM, WV, true, false, false>) : go(k_w4_tile<F16, FM, WV, false, false, false>);
    }
    if (err != hipSuccess || sp.slices == 1) return err;
    EpiProblem ep{};
    ep.M = p.M;
    ep.N = p.N;
    ep.C = static_cast<float*>(p.C);
    ep.ldc = p.ldc;
    ep.e = p.e;
    return launch_join_slabs(ep, part, sp.slices, p.N, stream);
}

template <bool F16>
hipError_t launch_type(const W4Problem& p, const W4Split& sp, float* part, hipStream_t stream) {
    if (p.tr) {
        if (sp.fm == 1) return launch_tile<F16, 1, 4, true>(p, sp, part, stream);
        if (sp.fm == 2) return launch_tile<F16, 2, 4, true>(p, sp, part, stream);
        return launch_tile<F16, 4, 4, true>(p, sp, part, stream);
    }
    if (sp.fm == 1) return launch_tile<F16, 1, 4, false>(p, sp, part, stream);
    if (sp.fm == 2) return launch_tile<F16, 2, 4, false>(p, sp, part, stream);
    return sp.wv == 4 ? launch_tile<F16, 4, 4, false>(p, sp, part, stream) : launch_tile<F16, 4, 8, false>(p, sp, part, stream);
}

// Tile and K split by a time model fitted to the kernels' times at N 4096 and 11008, K 4096 and 11008, M 32
// to 2048 (HIP events, bf16, zero points, operands rotating over three sets).  A step (128 k; 64 of dy . W)
// takes a workgroup alone on its CU `alone` us, up to `busy` where every CU has one (the power limit lowers the
// clock), and n workgroups that share a CU n `shared` together.  A split adds a second kernel (4 us) and
// the slices' sums, written and read once each at 3 TB/s.  Best and second-best measured, x . W^T: 64 x 4096 x
// 4096 15.6 us (32 x 128 tiles, 4 slices) and 17.3 (64 x 128, 8 slices), unsplit 25.2; 512 x 4096 x 4096 32.1
// (64 x 128) and 36.4 (128 x 256, 4 slices); 512 x 11008 x 4096 62.9 (128 x 256) and 75.6 (64 x 128); dy . W:
// 128 x 4096 x 4096 22.2 (64 x 128, 4 slices) and 25.0 (32 x 128, 4 slices), unsplit 37.2.
struct TileTime {
    int fm, wv;
    double alone, busy, shared;
    int per_cu;
};
constexpr TileTime kTiles[] = {{1, 4, 0.69, 0.73, 0.65, 4}, {2, 4, 0.82, 0.96, 0.83, 3}, {4, 4, 1.25, 1.5, 1.5, 1},
                               {4, 8, 1.65, 2.2, 2.2, 1}};
constexpr TileTime kTilesT[] = {{1, 4, 0.53, 0.55, 0.42, 3}, {2, 4, 0.66, 0.70, 0.54, 2}, {4, 4, 0.97, 1.02, 1.02, 1}};

double tile_us(const TileTime& t, double tiles, int64_t steps, int cus) {
    // workgroups on the busiest CU: whole rounds of `per_cu`, and what is left
    const double load = std::ceil(tiles / cus), full = std::floor(load / t.per_cu) * t.per_cu, rest = load - full;
    const double fill = std::min(1.0, tiles / cus), one = t.alone + (t.busy - t.alone) * fill * fill;
    return 3.0 + steps * (full * t.shared + (rest == 0 ? 0 : rest == 1 ? one : rest * t.shared));
}

}  // namespace

W4Split w4_split(int64_t M, int64_t N, int64_t K, bool tr, int cus, bool workspace) {
    const int64_t deep = tr ? kStepT : kStep, steps = (K + deep - 1) / deep;
    W4Split best;
    best.us = 1e300;
    auto consider = [&](const TileTime& t) {
        const int64_t bm = 32 * t.fm, bn = 32 * t.wv;
        const double tiles = (double)((M + bm - 1) / bm) * (double)((N + bn - 1) / bn);
        for (int64_t want = 1; want == 1 || (workspace && want <= 16 && (tr ? 4 : 2) * want <= steps); ++want) {
            const int64_t per = (steps + want - 1) / want, slices = (steps + per - 1) / per;
            double us = tile_us(t, tiles * slices, per, cus);
            if (slices > 1) us += 4.0 + 8.0 * slices * M * N / 3e6;
            if (us < best.us)
                best = W4Split{t.fm, t.wv, (int)slices, (int)(per * deep), slices > 1 ? (size_t)slices * M * N * 4 : 0, us};
        }
    };
    if (tr) {
        for (const TileTime& t : kTilesT) consider(t);
    } else {
        for (const TileTime& t : kTiles) consider(t);
    }
    return best;
}

// W written as 16-bit numbers (2.6 bytes a weight at 4.5 TB/s), then the 16-bit direct-copy kernels: a k-tile of 64
// takes a round of 256 x 128 tiles 0.70 us, up to 1.17 where it fills the chip, one of 256 x 256 tiles 1.1 to
// 1.66; many rounds run at 1.07 PFLOP/s.  (2048 x 11008 x 4096, x . W^T: 199 us measured, 208 by the model, the
// tile kernel 211; 1024 x 4096 x 4096, dy . W: 61, 66, 68.)
double w4_decoded_us(int64_t M, int64_t N, int64_t K, int cus) {
    const double m = std::ceil(M / 256.0), t256 = m * std::ceil(N / 256.0), t128 = m * std::ceil(N / 128.0);
    auto rounds = [&](double tiles, double low, double high) {
        const double u = std::min(1.0, tiles / cus);
        return std::ceil(tiles / cus) * (low + (high - low) * u * u) * K / 64.0;
    };
    double us = std::min(rounds(t256, 1.1, 1.66), rounds(t128, 0.70, 1.17));
    if (t128 > 2.0 * cus) us = std::min(us, 2.0 * M * N * K / 1.07e9 + 5.0);
    return 2.6 * N * K / 4.5e6 + us + 4.0;
}

hipError_t launch_w4_tile(const W4Problem& p, const W4Split& sp, bool f16, float* part, hipStream_t stream,
                          const char*& name) {
    static const char* names[2][2][2] = {
        {{"bf16_w4_tile", "f16_w4_tile"}, {"bf16_w4_tile_splitk", "f16_w4_tile_splitk"}},
        {{"bf16_w4_tile_t", "f16_w4_tile_t"}, {"bf16_w4_tile_t_splitk", "f16_w4_tile_t_splitk"}}};
    W4Split s = sp;
    if ((int64_t)32 * s.fm * p.lda * 2 >= (int64_t)1 << 31) s = W4Split{1, 4, 1, p.K, 0, 0};      // FAR, without a split
    name = names[p.tr ? 1 : 0][s.slices > 1 ? 1 : 0][f16 ? 1 : 0];
    return f16 ? launch_type<true>(p, s, part, stream) : launch_type<false>(p, s, part, stream);
}

}  // namespace gemm
