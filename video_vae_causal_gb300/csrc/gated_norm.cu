// gated_norm.cu -- the norms after and before a block fused with its gate, its
// residual scale and the residual add:
//
//     y = x + s * gate (.) RMS_norm(f; g_post)     f = the block's output
//     n = RMS_norm(y; g_pre)                       the next block's input
//
// RMS_norm as in norm_act.cuh (the L2 norm over a token's channels, clamped
// below by eps, divides the token, scaled by sqrt(C) * gamma).  Without
// g_post f enters as it is, without a gate the gate is one, without g_pre n is
// not written.  Everything between the loads and the two stores stays in
// fp32 registers: n is the norm of y before y is rounded.
//
// The pass moves 4 C elements a token and computes about 10 C operations, so
// it is bound by HBM.  A row belongs to a group of TPR threads (a power of
// two, the fewest that leave a thread at most 4 16-byte vectors of x and of
// f), whose vectors lie TPR apart so that neighbouring threads read
// neighbouring vectors; the loads of both tensors are in flight before the
// first reduction.  Threads past the row's end hold zeros, so C need only be
// a multiple of 16.
//
// Measured: 131040 tokens of 384 channels in bf16, a gate for every 6240 of them: 70 us,
// 5.7 TB/s, 0.85 of the measured copy rate.  One resident wave of blocks that step through
// the rows: a block for every 16 rows takes 80 us, five resident blocks in place of three
// (fewer registers, fewer loads in flight) 77; streaming loads and stores change
// nothing (70).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "norm_act.cuh"
#include "ptx.cuh"
#include "seq_ops.h"

namespace wanvae {
namespace {

constexpr int kThreads = 256;

struct GatedArgs {
    const uint4 *x, *f;
    const float *g_post, *gate, *g_pre;
    uint4 *y, *n;
    uint32_t rows, per_gate;
    int V, tpr;  // 16-byte vectors and threads of a row
    float scale, eps, sqrt_c;
};

// Sum over the TPR threads of a row.  Rows wider than a warp go through
// `part` (one slot a warp); every thread of the block takes part.
__device__ __forceinline__ float row_sum(float v, int tpr, float *part) {
    v = nact_group_sum(v, tpr < 32 ? tpr : 32);
    if (tpr <= 32) return v;
    const int warp = threadIdx.x >> 5, warps = tpr >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    float s = 0.f;
    const int first = warp / warps * warps;
    for (int w = 0; w < warps; ++w) s += part[first + w];
    return s;
}

// What a row of sum of squares `ss` is multiplied by: NaN where the row holds one (the
// clamp's maximum would drop it, and give the row's other channels a norm of eps).
__device__ __forceinline__ float row_scale(float ss, float sqrt_c, float eps) {
    const float s = nact_scale(ss, sqrt_c, eps);
    return ss == ss ? s : ss;
}

template <bool F32>
struct Vec {
    static constexpr int E = F32 ? 4 : 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *o) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (F32) {
                o[k] = __uint_as_float(w[k]);
            } else {
                o[2 * k] = nact_lo(w[k]);
                o[2 * k + 1] = nact_hi(w[k]);
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *o) {
        if (F32)
            return make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                              __float_as_uint(o[3]));
        return make_uint4(nact_pack(o[0], o[1]), nact_pack(o[2], o[3]),
                          nact_pack(o[4 % E], o[5 % E]), nact_pack(o[6 % E], o[7 % E]));
    }
};

template <int E>
__device__ __forceinline__ void load_f32(const float *p, float *o) {
#pragma unroll
    for (int k = 0; k < E; k += 4)
        *reinterpret_cast<float4 *>(o + k) = __ldg(reinterpret_cast<const float4 *>(p + k));
}

template <bool F32, int VPT>
__global__ void __launch_bounds__(kThreads)
gated_norm_kernel(const GatedArgs a) {
    constexpr int E = Vec<F32>::E;
    __shared__ float part[2][kThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int sub = threadIdx.x & (a.tpr - 1);
    const uint32_t rpb = kThreads / a.tpr, grp = threadIdx.x / a.tpr;
    // every thread of a block makes the same number of turns (row_sum's barriers)
    for (uint32_t r0 = blockIdx.x * rpb; r0 < a.rows; r0 += gridDim.x * rpb) {
        const uint32_t row = r0 + grp;
        const bool there = row < a.rows;
        const uint64_t at = (uint64_t)row * a.V;
        uint4 xv[VPT], fv[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = sub + i * a.tpr;
            xv[i] = fv[i] = make_uint4(0u, 0u, 0u, 0u);
            if (there && j < a.V) {
                fv[i] = __ldg(a.f + at + j);
                xv[i] = __ldg(a.x + at + j);
            }
        }
        float scale = a.scale;
        if (a.g_post) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float t[E];
                Vec<F32>::unpack(fv[i], t);
#pragma unroll
                for (int k = 0; k < E; ++k) ss = fmaf(t[k], t[k], ss);
            }
            ss = row_sum(ss, a.tpr, part[0]);
            scale *= row_scale(ss, a.sqrt_c, a.eps);
        }
        const float *gate = a.gate && there ? a.gate + (uint64_t)(row / a.per_gate) * a.V * E
                                            : nullptr;
        float y[VPT][E];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = sub + i * a.tpr;
            float t[E], w[E];
            Vec<F32>::unpack(fv[i], t);
            Vec<F32>::unpack(xv[i], y[i]);
#pragma unroll
            for (int k = 0; k < E; ++k) t[k] *= scale;
            if (a.g_post && j < a.V) {
                load_f32<E>(a.g_post + j * E, w);
#pragma unroll
                for (int k = 0; k < E; ++k) t[k] *= w[k];
            }
            if (gate && j < a.V) {
                load_f32<E>(gate + j * E, w);
#pragma unroll
                for (int k = 0; k < E; ++k) t[k] *= w[k];
            }
#pragma unroll
            for (int k = 0; k < E; ++k) {
                y[i][k] += t[k];
                ss = fmaf(y[i][k], y[i][k], ss);
            }
            if (there && j < a.V) a.y[at + j] = Vec<F32>::pack(y[i]);
        }
        if (a.g_pre) {
            ss = row_sum(ss, a.tpr, part[1]);
            const float rn = row_scale(ss, a.sqrt_c, a.eps);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int j = sub + i * a.tpr;
                if (!there || j >= a.V) continue;
                float w[E];
                load_f32<E>(a.g_pre + j * E, w);
#pragma unroll
                for (int k = 0; k < E; ++k) w[k] *= y[i][k] * rn;
                a.n[at + j] = Vec<F32>::pack(w);
            }
        }
        if (a.tpr > 32) __syncthreads();  // the slots are free for the next row
    }
}

template <bool F32, int VPT>
cudaError_t launch(const GatedArgs &a, const LaunchCtx &ctx) {
    const uint32_t rpb = kThreads / a.tpr;
    const uint32_t blocks = (a.rows + rpb - 1) / rpb;
    // one resident wave, grid-stride beyond it
    static std::atomic<int> per_sm{0};
    int occ = per_sm.load(std::memory_order_relaxed);
    if (!occ) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &occ, gated_norm_kernel<F32, VPT>, kThreads, 0);
        if (e != cudaSuccess) return e;
        per_sm.store(occ = std::max(1, occ), std::memory_order_relaxed);
    }
    const uint32_t grid = std::min(blocks, (uint32_t)(ctx.num_sms * occ));
    return launch_pdl(gated_norm_kernel<F32, VPT>, dim3(grid), dim3(kThreads), 0, ctx, a);
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormSpec &s, const LaunchCtx &ctx) {
    GatedArgs a;
    a.x = static_cast<const uint4 *>(s.x);
    a.f = static_cast<const uint4 *>(s.f);
    a.g_post = s.g_post;
    a.gate = s.gate;
    a.g_pre = s.g_pre;
    a.y = static_cast<uint4 *>(s.y);
    a.n = static_cast<uint4 *>(s.n);
    a.rows = (uint32_t)s.tokens;
    a.per_gate = (uint32_t)std::min<int64_t>(s.per_gate, s.tokens);
    a.V = s.C / (s.f32 ? 4 : 8);
    a.tpr = 1;
    while (a.tpr * 4 < a.V) a.tpr *= 2;  // C <= 4096: at most 256
    a.scale = s.scale;
    a.eps = s.eps;
    a.sqrt_c = sqrtf((float)s.C);
    const int vpt = (a.V + a.tpr - 1) / a.tpr;
    switch (vpt) {
        case 1: return s.f32 ? launch<true, 1>(a, ctx) : launch<false, 1>(a, ctx);
        case 2: return s.f32 ? launch<true, 2>(a, ctx) : launch<false, 2>(a, ctx);
        case 3: return s.f32 ? launch<true, 3>(a, ctx) : launch<false, 3>(a, ctx);
        case 4: return s.f32 ? launch<true, 4>(a, ctx) : launch<false, 4>(a, ctx);
    }
    return cudaErrorInvalidValue;
}

}  // namespace wanvae
