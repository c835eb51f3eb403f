// seq_ptx.cuh -- inline-PTX wrappers that the sequence operators need beyond
// ptx.cuh: a tensor-core operand read along its rows, TMEM stores.
#pragma once

#include "ptx.cuh"

namespace wanvae {

// Instruction descriptor as idesc_bf16_f32, B stored [K][N] (N contiguous:
// bit 16), for O = P V with V as it lies in memory.
__host__ __device__ constexpr uint32_t idesc_bf16_f32_bt(int M, int N) {
    return idesc_bf16_f32(M, N) | (1u << 16);
}

// Descriptor of an operand [K][N] in 128-byte swizzled rows of 64 bf16 of N:
// 8-row (K) groups lie 1024 bytes apart (the stride offset), 64-wide pieces of
// N `piece` bytes apart (the leading offset).
__device__ __forceinline__ uint64_t sdesc_rows_sw128(uint32_t saddr, uint32_t piece) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((piece >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)kLayoutSw128 << 61;
    return d;
}

// 32 columns of this warp's TMEM lane quarter <- r (then wait for the store).
__device__ __forceinline__ void tmem_st_cols32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

}  // namespace wanvae
