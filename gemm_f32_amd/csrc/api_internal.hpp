// What the host sources of the C ABI share (api.hip defines, api_lowbit.hip uses).
#pragma once

#include "gemm.h"
#include "common.hpp"
#include "epilogue.hpp"

namespace gemm {

enum class In { F32, BF16, F16, FP8 };

// The current device is a gfx950: its compute units.
bool current_device(int& cus);

// The end of a call: keeps the HIP error or the kernel's name (a static string) for this thread.
gemm_status_t record_call(hipError_t err, const char* name);

// C = epilogue(A.B) on the 16-bit or FP32 direct-copy kernels: p normalised (row-major C, whose memory
// is `C`), within their layouts (bf16_dma_applies, or bf16_dma_tn_applies for a column-major A), K >= 1.
hipError_t run_fused_tiles(In in, const Problem& p, const Epilogue& e, void* C, int cus, hipStream_t stream,
                           const char*& name);

// C = act(beta * C + bias): the epilogue of an empty sum.
hipError_t run_epilogue_fill(const Problem& p, const Epilogue& e, void* C, hipStream_t stream);

}  // namespace gemm
