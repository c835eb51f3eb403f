// seq_dev.cuh -- device helpers shared by the sequence operators: which
// sequence a packed row belongs to, the e4m3 rows of a cache and their E8M0
// scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace wanvae {

// The last s in [0, n) with start[s] <= row, for 0 = start[0] <= start[1] ..:
// the sequence that holds `row` (empty sequences hold none).  A whole warp
// asks for the same row: 32 probes a step, so 1024 sequences take two.
__device__ __forceinline__ int seq_of_row(const int32_t *start, int n, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int width = (hi - lo + 31) / 32;
        const int at = lo + lane * width;
        const bool below = at < hi && __ldg(start + at) <= row;
        const int c = __popc(__ballot_sync(0xffffffffu, below));
        if (c == 0) return lo;
        lo += (c - 1) * width;
        hi = min(hi, lo + width);
    }
    return lo;
}

// An E8M0 scale as a float: 2^(code - 127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
    return code == 255u ? __uint_as_float(0x7fc00000u)
                        : __uint_as_float(code == 0u ? 0x00400000u : code << 23);
}

// Two e4m3 values (the low 16 bits of w) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}

// a -> bits 0-7, b -> bits 8-15, each the nearest e4m3 value (ties to even).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

}  // namespace wanvae
