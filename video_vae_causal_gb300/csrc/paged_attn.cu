// paged_attn.cu -- attention of one new token for each sequence over a paged
// key-value cache (kv_cache.cu), split over the cache's length and joined:
//
//     out[b, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q[b, h] . k_j)
//
// over the lens[b] cached rows of kv head h / G.  Every row is read once for
// the G query heads that share it, so the work is G multiply-adds a cache
// byte or less and the bound is HBM.
//
// Split.  The rows of one (sequence, kv head) are cut into units of 64 or 128; the
// units of the whole batch, laid end to end, are dealt to the CTAs in equal
// contiguous shares, so a ragged batch and a single long sequence load every
// multiprocessor alike.  A share may begin or end inside an item: then its
// CTA leaves a partial result (the running maximum, the sum and the
// unnormalised output) in the workspace, two slots a CTA, and a second small
// kernel joins them in the order of the CTAs.  Which CTA left what follows from the
// lengths alone, so nothing is counted, reset or raced for.
//
// A warp takes 16 or 32 rows of a unit.  Its threads copy (cp.async) exactly the
// bytes that they will multiply: thread (g, t) = (lane / 4, lane % 4) needs, as the
// B operand of S = Q K^T, a quarter of key rows g and g + 8, and as the A
// operand of O^T = V^T P^T an eighth of value rows 2t, 2t + 1, 2t + 8 and
// 2t + 9.  The order of the elements along the summed dimension is free, so
// these are whole 16-byte pieces; shared memory is a private queue of each
// thread (no barrier, no bank conflict), kStages units deep.
//
// 8-bit rows become fp16 exactly; queries become fp16 with a power of two taken
// out so that the largest has exponent 14 (bf16's 8 bits fit in fp16's 11;
// what falls below fp16's range is 2^-39 of the largest).  A key row's scale
// multiplies its score; a value row's scale 2^e joins the exponent of its
// weight, w_j = 2^(s_j + e_j - m) with m the running maximum of s_j + e_j, while the sum
// takes 2^(s_j - m) in fp32, so that weights stay in fp16's upper range
// whatever the scales are (weights round once, to 2^-12 relative).
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "norm_act.cuh"
#include "seq_dev.cuh"
#include "seq_ops.h"
#include "seq_ptx.cuh"

namespace wanvae {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kMaxCtas = 640;       // CTAs of a launch (sizes the workspace)

struct PagedArgs {
    const __nv_bfloat16 *q;
    int64_t q_stride;
    const uint8_t *k, *v, *k_exp, *v_exp;
    int n_pages, log2_page, H;
    const int32_t *table, *lens;
    int max_pages, n_seq;
    int G, HB;  // query heads of a kv head; blocks of heads that a kv head is read for
    float scale_log2;
    __nv_bfloat16 *out;
    int64_t out_stride;
    float *part_o;   // [2 CTAs][heads of a block][D]
    float2 *part_ml; // [2 CTAs][heads of a block]: maximum, sum
    unsigned *err;
};

// A sequence's length as far as the page table reaches.
__device__ __forceinline__ int seq_len(const PagedArgs &p, int b, bool tell) {
    const int len = __ldg(p.lens + b);
    const int64_t most = (int64_t)p.max_pages << p.log2_page;
    if (len >= 0 && len <= most) return len;
    if (tell) atomicOr(p.err, kDevErrAlign);
    return len < 0 ? 0 : (int)most;
}
template <int kUnit>
__device__ __forceinline__ int units_of(int len) {
    return (len + kUnit - 1) / kUnit;
}

// Units before sequence b (all of them for b = n_seq) of one head; whole warp.
template <int kUnit>
__device__ __forceinline__ int units_before(const PagedArgs &p, int b) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int i = lane; i < b; i += 32) n += units_of<kUnit>(seq_len(p, i, false));
    return __reduce_add_sync(0xffffffffu, n);
}

__device__ __forceinline__ int share_begin(int total, int cta, int ctas) {
    return (int)((int64_t)total * cta / ctas);
}
__device__ __forceinline__ int share_of(int total, int unit, int ctas) {
    return (int)((((int64_t)unit + 1) * ctas - 1) / total);
}

template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
    if (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// Same, or zeros where the source is not there.
template <int kBytes>
__device__ __forceinline__ void cp_async_part(uint32_t dst, const void *src, bool there) {
    const int n = there ? kBytes : 0;  // bytes that are read
    if (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// D += A B, 16 x 8 x 16, fp16 or bf16 in, fp32 out.
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    return nact_pack(lo, hi);
}

// D: head width; Q8: e4m3 cache; NH: blocks of 8 query heads read together.
template <int D, bool Q8, int NH>
struct Shape {
    static constexpr int EB = Q8 ? 1 : 2;                // bytes of an element
    static constexpr int RB = D * EB;                    // bytes of a row
    static constexpr int KC = RB / 64;                   // 16-byte pieces of a key row, a thread
    static constexpr int VB = RB / 8 < 16 ? 8 : 16;      // bytes of a value piece
    static constexpr int VC = RB / 8 / VB;               // pieces of a value row, a thread
    // Groups of 16 rows of a warp's turn: two share one maximum and give the
    // tensor core twice the independent products; rows of 256 bytes take one
    // so that three CTAs' queues fit a multiprocessor.
    static constexpr int NG = RB >= 256 ? 1 : 2;
    static constexpr int kUnit = 16 * NG * kWarps;       // cache rows of a unit
    static constexpr int kStages = RB == 64 ? 4 : 2;
    static constexpr int kGroup = 32 * RB;               // bytes of a group, k and v
    static constexpr int kWarpStage = NG * kGroup;
    static constexpr int kExpOff = kStages * kWarps * kWarpStage;  // 32 bytes a group
    static constexpr int kMetaOff = kExpOff + kStages * kWarps * NG * 32;
    static constexpr int kMlOff = kMetaOff + kStages * kWarps * 4;
    static constexpr int kSmem = kMlOff + kWarps * NH * 8 * 8;
    // a warp's outputs wait for the join in its part of the stage just read:
    // [D][8] floats for each 8 heads, 8 more behind every 16 rows where there is
    // room (bank conflicts)
    static constexpr int kPad = (D + D / 16) * 8 * 4 * NH <= kWarpStage ? 8 : 0;
    static constexpr int kJoinHeads = (D * 8 + D / 16 * kPad);  // floats of 8 heads
    static_assert(kJoinHeads * 4 * NH <= kWarpStage, "join buffer");
};

// Where a share stands: unit u of the U units of (sequence b, head block hh).
template <int kUnit>
struct Cursor {
    int b, hh, u, U, len;
    // On to the next unit; true where the item changed.
    __device__ __forceinline__ bool next(const PagedArgs &p, int HH) {
        if (++u < U) return false;
        u = 0;
        if (++hh < HH) return true;
        hh = 0;
        do {
            if (++b >= p.n_seq) return true;
            len = seq_len(p, b, false);
            U = units_of<kUnit>(len);
        } while (U == 0);
        return true;
    }
};

template <int D, bool Q8, int NH>
__global__ void __launch_bounds__(kThreads, 3)
paged_attn_kernel(const PagedArgs p) {
    using S = Shape<D, Q8, NH>;
    constexpr int NG = S::NG;
    constexpr int kSteps = D / 16;  // 16-wide steps along D of a score; 16-row tiles of O^T
    extern __shared__ __align__(16) uint8_t smem[];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int HH = p.H * p.HB;

    // this CTA's share
    const int total = units_before<S::kUnit>(p, p.n_seq) * HH;
    const int ctas = min((int)gridDim.x, total);  // no share is empty
    if ((int)blockIdx.x >= ctas) return;
    const int u0 = share_begin(total, blockIdx.x, ctas);
    const int u1 = share_begin(total, blockIdx.x + 1, ctas);
    Cursor<S::kUnit> at;  // the unit to compute next
    {
        int b0 = 0, before = 0;  // (in units of one head)
        while (true) {
            const int i = b0 + lane;
            const int U = i < p.n_seq
                              ? units_of<S::kUnit>(seq_len(p, i, blockIdx.x == 0 && warp == 0))
                              : 0;
            int incl = U;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            const bool beyond = (int64_t)(before + incl) * HH > u0;
            const unsigned m = __ballot_sync(0xffffffffu, beyond);
            if (m) {
                const int l = __ffs(m) - 1;
                at.b = b0 + l;
                at.U = __shfl_sync(0xffffffffu, U, l);
                const int rest = u0 - (before + __shfl_sync(0xffffffffu, incl - U, l)) * HH;
                at.hh = rest / at.U;
                at.u = rest % at.U;
                break;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
            b0 += 32;
        }
        at.len = seq_len(p, at.b, false);
    }

    const uint32_t base = smem_u32(smem);
    int *meta = reinterpret_cast<int *>(smem + S::kMetaOff);
    // ---- copies: `ahead` is the unit to copy next, `page` its pages (loaded one
    // unit early), `kvh` its kv head
    Cursor<S::kUnit> ahead = at;
    int left = u1 - u0;  // units not yet copied
    int kvh_ahead = ahead.hh / p.HB;
    int page[NG];
    auto find_pages = [&]() {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int tok = ahead.u * S::kUnit + (warp * NG + i) * 16;
            page[i] = -1;
            if (tok < ahead.len)
                page[i] = __ldg(p.table + (int64_t)ahead.b * p.max_pages + (tok >> p.log2_page));
        }
    };
    find_pages();
    auto copy = [&](int stage) {
        if (left > 0) {
            int told = 0;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int tok = ahead.u * S::kUnit + (warp * NG + i) * 16;
                int rows = min(max(ahead.len - tok, 0), 16);
                if ((unsigned)page[i] >= (unsigned)p.n_pages) {
                    if (rows && lane == 0) atomicOr(p.err, kDevErrAlign);
                    rows = 0;
                }
                told |= rows << (8 * i);
                const int64_t row = rows ? ((((int64_t)page[i] * p.H + kvh_ahead) << p.log2_page) +
                                            (tok & ((1 << p.log2_page) - 1)))
                                         : 0;
                const uint32_t dst = base + (uint32_t)((stage * kWarps + warp) * S::kWarpStage +
                                                       i * S::kGroup);
                const uint32_t kd = dst + lane * 16, vd = dst + 2 * S::KC * 512 + lane * S::VB;
                const uint8_t *kr = p.k + row * S::RB + g * S::RB + 16 * t;
                const uint8_t *vr = p.v + row * S::RB + 2 * t * S::RB + g * S::VB;
                if (rows == 16) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < S::KC; ++c)
                            cp_async<16>(kd + (j * S::KC + c) * 512, kr + 8 * j * S::RB + 64 * c);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int c = 0; c < S::VC; ++c)
                            cp_async<S::VB>(vd + (j * S::VC + c) * (32 * S::VB),
                                            vr + ((j & 1) + 8 * (j >> 1)) * S::RB + c * 8 * S::VB);
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < S::KC; ++c) {
                            const bool in = 8 * j + g < rows;
                            cp_async_part<16>(kd + (j * S::KC + c) * 512,
                                              in ? kr + 8 * j * S::RB + 64 * c : p.k, in);
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int c = 0; c < S::VC; ++c) {
                            const int r = (j & 1) + 8 * (j >> 1);
                            const bool in = 2 * t + r < rows;
                            cp_async_part<S::VB>(vd + (j * S::VC + c) * (32 * S::VB),
                                                 in ? vr + r * S::RB + c * 8 * S::VB : p.v, in);
                        }
                }
                if (Q8 && lane < 2)
                    cp_async_part<16>(base + S::kExpOff +
                                          ((stage * kWarps + warp) * NG + i) * 32 + lane * 16,
                                      (lane ? p.v_exp : p.k_exp) + row, rows > 0);
            }
            if (lane == 0) meta[stage * kWarps + warp] = told;
            if (--left > 0) {
                if (ahead.next(p, HH)) kvh_ahead = ahead.hh / p.HB;
                find_pages();
            }
        }
        cp_async_commit();  // (an empty group keeps the count)
    };
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) copy(s);

    // ---- one item after another
    int stage = 0;
    bool first = true;
    for (int u = u0; u < u1;) {
        const int units = min(at.U - at.u, u1 - u);  // of this item, in this share
        const bool whole = at.u == 0 && units == at.U;
        const int kvh = at.hh / p.HB, h0 = kvh * p.G + (at.hh % p.HB) * 8 * NH;
        const int heads = min(8 * NH, (kvh + 1) * p.G - h0);
        // the queries as A operands: step s of piece c covers elements
        // d = c * 64 / EB + t * 16 / EB + 4 s .. + 3 of heads g and g + 8
        uint32_t qa[kSteps][2][NH];
        float qs[NH];  // what a score of head g + 8 i is multiplied by, in log2 units
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            const int h = g + 8 * i;
            const __nv_bfloat16 *src = p.q + (int64_t)at.b * p.q_stride + (int64_t)(h0 + h) * D;
            constexpr int kPer = 16 / S::EB;  // elements of a piece
            uint32_t raw[kSteps][2];
            uint32_t amax = 0;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int c = s / (kPer / 4), w = s % (kPer / 4);
                uint2 x = make_uint2(0u, 0u);
                if (h < heads)
                    x = __ldg(reinterpret_cast<const uint2 *>(src + c * 4 * kPer + t * kPer + 4 * w));
                raw[s][0] = x.x;
                raw[s][1] = x.y;
                if (Q8) {
                    amax = max(amax, max(x.x & 0x7fffu, (x.x >> 16) & 0x7fffu));
                    amax = max(amax, max(x.y & 0x7fffu, (x.y >> 16) & 0x7fffu));
                }
            }
            qs[i] = p.scale_log2;
            if (Q8) {
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^(14 - exponent of the largest); both powers stay in fp32's range
                const int ex = min(max((int)(amax >> 7), 15), 254) - 127 - 14;
                const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
                qs[i] *= __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        qa[s][w][i] = pack16<true>(nact_lo(raw[s][w]) * down,
                                                   nact_hi(raw[s][w]) * down);
            } else {
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int w = 0; w < 2; ++w) qa[s][w][i] = raw[s][w];
            }
        }
        float m[NH], l[NH];  // of head g + 8 i; the sum over this thread's rows alone
        float o[NH][kSteps][4];
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][s][k] = 0.f;
        }

        for (int n = 0; n < units; ++n) {
            cp_async_wait<S::kStages - 2>();
            __syncwarp();  // the other lanes' copies (exponents, meta) too; stage - 1 is read
            copy(stage == 0 ? S::kStages - 1 : stage - 1);
            const uint8_t *src = smem + (stage * kWarps + warp) * S::kWarpStage;
            const int rows = meta[stage * kWarps + warp];
            // S = Q K^T for rows 8 j + 2 t, + 1 of a group and heads g, g + 8
            float sc[NG][2][4] = {};
#pragma unroll
            for (int c = 0; c < S::KC; ++c) {
                uint4 w4[NG][2];
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        w4[i][j] = *reinterpret_cast<const uint4 *>(
                            src + i * S::kGroup + (j * S::KC + c) * 512 + lane * 16);
                constexpr int kPiece = Q8 ? 4 : 2;  // steps of a piece
#pragma unroll
                for (int k = 0; k < kPiece; ++k) {
                    const int s = c * kPiece + k;
#pragma unroll
                    for (int i = 0; i < NG; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t w[4] = {w4[i][j].x, w4[i][j].y, w4[i][j].z, w4[i][j].w};
                            const uint32_t b0 = Q8 ? e4m3x2_to_f16x2(w[k % 4]) : w[(2 * k) % 4];
                            const uint32_t b1 = Q8 ? e4m3x2_to_f16x2(w[k % 4] >> 16)
                                                   : w[(2 * k + 1) % 4];
                            mma_16816<Q8>(sc[i][j], qa[s][0][0], NH > 1 ? qa[s][0][NH - 1] : 0u,
                                          qa[s][1][0], NH > 1 ? qa[s][1][NH - 1] : 0u, b0, b1);
                        }
                }
            }
            // the rows' scales: keys' as factors, values' as exponents
            float kf[NG][2][2], ve[NG][2][2];
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    kf[i][j][0] = kf[i][j][1] = 1.f;
                    ve[i][j][0] = ve[i][j][1] = 0.f;
                    if (!Q8) continue;
                    const uint8_t *ex =
                        smem + S::kExpOff + ((stage * kWarps + warp) * NG + i) * 32 + 8 * j + 2 * t;
                    const uint32_t kx = *reinterpret_cast<const uint16_t *>(ex);
                    const uint32_t vx = *reinterpret_cast<const uint16_t *>(ex + 16);
                    kf[i][j][0] = __uint_as_float((kx << 23) & 0x7f800000u);
                    kf[i][j][1] = __uint_as_float((kx << 15) & 0x7f800000u);
                    // 2^23 + code, less 2^23 + 127
                    ve[i][j][0] = __uint_as_float(__byte_perm(vx, 0x4b000000u, 0x7440)) - 8388735.f;
                    ve[i][j][1] = __uint_as_float(__byte_perm(vx, 0x4b000000u, 0x7441)) - 8388735.f;
                }
            uint32_t pb[NH][NG][2];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                float s[NG][2][2], mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            s[i][j][c] = sc[i][j][2 * h + c] * (qs[h] * kf[i][j][c]);
                if (rows != (NG == 2 ? 0x1010 : 0x10)) {
#pragma unroll
                    for (int i = 0; i < NG; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (8 * j + 2 * t + c >= ((rows >> (8 * i)) & 0xff))
                                    s[i][j][c] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        mx = max3(mx, s[i][j][0] + ve[i][j][0], s[i][j][1] + ve[i][j][1]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // the maximum moves only by more than 2^4: weights stay below 16,
                // their sums below fp16's products' fp32 range, and O is seldom rescaled
                if (__any_sync(0xffffffffu, mx > m[h] + 4.f)) {
                    const float mn = fmaxf(m[h], mx);
                    const float f = mn == -INFINITY ? 0.f : exp2_fast(m[h] - mn);
                    m[h] = mn;
                    l[h] *= f;
                    const float f0 = __shfl_sync(0xffffffffu, f, 8 * t);
                    const float f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        o[h][k][0] *= f0;
                        o[h][k][1] *= f1;
                        o[h][k][2] *= f0;
                        o[h][k][3] *= f1;
                    }
                }
                const float ms = m[h] == -INFINITY ? 0.f : m[h];  // nothing seen yet: weights 0
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    float w[2][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float x = s[i][j][c] - ms;
                            const float e = exp2_fast(x);
                            l[h] += e;
                            w[j][c] = Q8 ? exp2_fast(x + ve[i][j][c]) : e;
                        }
                    pb[h][i][0] = pack16<Q8>(w[0][0], w[0][1]);
                    pb[h][i][1] = pack16<Q8>(w[1][0], w[1][1]);
                }
            }
            // O^T += V^T P^T: tile s holds elements 2 s (rows g) and 2 s + 1
            // (rows g + 8) of this thread's piece of the value rows
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const uint8_t *vsrc = src + i * S::kGroup + 2 * S::KC * 512 + lane * S::VB;
#pragma unroll
                for (int c = 0; c < S::VC; ++c) {
                    uint32_t r[4][S::VB / 4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint8_t *a = vsrc + (j * S::VC + c) * (32 * S::VB);
                        if (S::VB == 16) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(a);
                            r[j][0] = x.x;
                            r[j][1] = x.y;
                            r[j][2 % (S::VB / 4)] = x.z;
                            r[j][3 % (S::VB / 4)] = x.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2 *>(a);
                            r[j][0] = x.x;
                            r[j][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < S::VB / 4; ++x) {
                        if (Q8) {
                            const uint32_t lo0 = __byte_perm(r[0][x], r[1][x], 0x5140);
                            const uint32_t hi0 = __byte_perm(r[0][x], r[1][x], 0x7362);
                            const uint32_t lo1 = __byte_perm(r[2][x], r[3][x], 0x5140);
                            const uint32_t hi1 = __byte_perm(r[2][x], r[3][x], 0x7362);
                            const uint32_t a0 = e4m3x2_to_f16x2(lo0);
                            const uint32_t a1 = e4m3x2_to_f16x2(lo0 >> 16);
                            const uint32_t a2 = e4m3x2_to_f16x2(lo1);
                            const uint32_t a3 = e4m3x2_to_f16x2(lo1 >> 16);
                            const uint32_t c0 = e4m3x2_to_f16x2(hi0);
                            const uint32_t c1 = e4m3x2_to_f16x2(hi0 >> 16);
                            const uint32_t c2 = e4m3x2_to_f16x2(hi1);
                            const uint32_t c3 = e4m3x2_to_f16x2(hi1 >> 16);
#pragma unroll
                            for (int h = 0; h < NH; ++h) {
                                mma_16816<Q8>(o[h][(2 * x) % kSteps], a0, a1, a2, a3, pb[h][i][0],
                                              pb[h][i][1]);
                                mma_16816<Q8>(o[h][(2 * x + 1) % kSteps], c0, c1, c2, c3,
                                              pb[h][i][0], pb[h][i][1]);
                            }
                        } else {
                            const uint32_t a0 = __byte_perm(r[0][x], r[1][x], 0x5410);
                            const uint32_t a1 = __byte_perm(r[0][x], r[1][x], 0x7632);
                            const uint32_t a2 = __byte_perm(r[2][x], r[3][x], 0x5410);
                            const uint32_t a3 = __byte_perm(r[2][x], r[3][x], 0x7632);
#pragma unroll
                            for (int h = 0; h < NH; ++h)
                                mma_16816<Q8>(o[h][(c * 4 + x) % kSteps], a0, a1, a2, a3,
                                              pb[h][i][0], pb[h][i][1]);
                        }
                    }
                }
            }
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
        }

        // ---- join the warps, then leave the result or a partial one.  A warp's
        // outputs go to its part of the stage that it has just read (the next copy
        // into it comes after the second barrier).
        uint8_t *last = smem + (stage == 0 ? S::kStages - 1 : stage - 1) * kWarps * S::kWarpStage;
        float2 *ml = reinterpret_cast<float2 *>(smem + S::kMlOff);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (t == 0) ml[(warp * NH + i) * 8 + g] = make_float2(m[i], l[i]);
            float *dst = reinterpret_cast<float *>(last + warp * S::kWarpStage) + i * S::kJoinHeads;
            constexpr int kEl = S::VB / S::EB;  // elements of a value piece
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int c = 2 * s / kEl, e = 2 * s % kEl;
                const int d = c * 8 * kEl + g * kEl + e;
                float *a = dst + d * 8 + (d >> 4) * S::kPad + 2 * t;
                float *b = dst + (d + 1) * 8 + ((d + 1) >> 4) * S::kPad + 2 * t;
                *reinterpret_cast<float2 *>(a) = make_float2(o[i][s][0], o[i][s][1]);
                *reinterpret_cast<float2 *>(b) = make_float2(o[i][s][2], o[i][s][3]);
            }
        }
        __syncthreads();
        const int slot = 2 * blockIdx.x + (first ? 0 : 1);
        for (int e = threadIdx.x; e < heads * D; e += kThreads) {
            const int h = e / D, d = e % D;
            const int i = h >> 3, hr = h & 7;
            float mw[kWarps], top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                mw[w] = ml[(w * NH + i) * 8 + hr].x;
                top = fmaxf(top, mw[w]);
            }
            float sum = 0.f, acc = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = mw[w] == -INFINITY ? 0.f : exp2_fast(mw[w] - top);
                sum += f * ml[(w * NH + i) * 8 + hr].y;
                acc += f * reinterpret_cast<const float *>(last + w * S::kWarpStage)
                               [i * S::kJoinHeads + d * 8 + (d >> 4) * S::kPad + hr];
            }
            if (whole) {
                p.out[(int64_t)at.b * p.out_stride + (int64_t)(h0 + h) * D + d] =
                    __float2bfloat16(sum > 0.f || sum != sum ? acc / sum : 0.f);
            } else {
                p.part_o[((int64_t)slot * (8 * NH) + h) * D + d] = acc;
                if (d == 0) p.part_ml[slot * (8 * NH) + h] = make_float2(top, sum);
            }
        }
        __syncthreads();  // the join buffers are free for the next item
        first = false;
        // on to the next item of the share
        u += units;
        at.u += units - 1;
        if (u < u1) at.next(p, HH);
    }
    cp_async_wait<0>();
}

// Joins the partial results of the items that were cut between CTAs, and
// writes zeros for sequences without rows.  One block of D threads for each
// (query head, sequence): the parts' weights side by side, then the sum of the
// parts in their order.
template <int D, int kUnit>
__global__ void __launch_bounds__(D)
paged_join_kernel(const PagedArgs p, int most_ctas, int block_heads) {
    __shared__ float weight[kMaxCtas];
    __shared__ float2 warp_ml[D / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
    __nv_bfloat16 *out = p.out + (int64_t)b * p.out_stride + (int64_t)h * D + d;
    const int U = units_of<kUnit>(seq_len(p, b, false));
    if (U == 0) {
        *out = __float2bfloat16(0.f);
        return;
    }
    const int HH = p.H * p.HB;
    const int kvh = h / p.G, hb = (h % p.G) / block_heads, hr = (h % p.G) % block_heads;
    const int total = units_before<kUnit>(p, p.n_seq) * HH;
    const int ctas = min(most_ctas, total);
    const int i0 = units_before<kUnit>(p, b) * HH + (kvh * p.HB + hb) * U;
    const int c0 = share_of(total, i0, ctas), c1 = share_of(total, i0 + U - 1, ctas);
    if (c0 == c1) return;  // one CTA held the whole item and wrote it
    // the item lies in the first slot of its CTAs, but for one that began before it
    const int s0 = 2 * c0 + (share_begin(total, c0, ctas) < i0 ? 1 : 0);
    auto slot_of = [&](int c) { return (c == c0 ? s0 : 2 * c) * block_heads + hr; };
    float top = -INFINITY;
    for (int c = c0 + d; c <= c1; c += D) top = fmaxf(top, p.part_ml[slot_of(c)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if ((d & 31) == 0) warp_ml[d >> 5].x = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; ++w) top = fmaxf(top, warp_ml[w].x);
    float sum = 0.f;
    for (int c = c0 + d; c <= c1; c += D) {
        const float2 ml = p.part_ml[slot_of(c)];
        const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top);
        weight[c - c0] = f;
        sum += f * ml.y;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if ((d & 31) == 0) warp_ml[d >> 5].y = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) sum += warp_ml[w].y;
    float acc = weight[0] * p.part_o[(int64_t)slot_of(c0) * D + d];
#pragma unroll 8
    for (int c = c0 + 1; c <= c1; ++c) acc += weight[c - c0] * p.part_o[(int64_t)slot_of(c) * D + d];
    *out = __float2bfloat16(sum > 0.f || sum != sum ? acc / sum : 0.f);
}

int head_block(int G) { return G <= 8 ? 8 : 16; }

template <int D, bool Q8, int NH>
cudaError_t launch(const PagedArgs &a, const LaunchCtx &ctx) {
    using S = Shape<D, Q8, NH>;
    const int64_t most_units =
        (((int64_t)a.max_pages << a.log2_page) + S::kUnit - 1) / S::kUnit * a.n_seq * a.H * a.HB;
    if (most_units > INT32_MAX) return cudaErrorInvalidValue;
    auto *kern = paged_attn_kernel<D, Q8, NH>;
    // resident CTAs, and the shared-memory opt-in, once per device
    constexpr int kMaxDev = 64;
    static std::atomic<int> per_sm[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    int occ = per_sm[dev].load(std::memory_order_acquire);
    if (!occ) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, kThreads, S::kSmem);
        if (e != cudaSuccess) return e;
        if (occ < 1) return cudaErrorInvalidConfiguration;
        per_sm[dev].store(occ, std::memory_order_release);
    }
    const int ctas = (int)std::max<int64_t>(
        1, std::min<int64_t>(most_units, std::min(kMaxCtas, occ * ctx.num_sms)));
    e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), S::kSmem, ctx, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_join_kernel<D, S::kUnit>, dim3((unsigned)(a.H * a.G), (unsigned)a.n_seq),
                      dim3(D), 0, ctx, a, ctas, 8 * NH);
}

}  // namespace

size_t paged_attention_workspace(int Hq, int Hkv, int D) {
    const size_t rows = (size_t)2 * kMaxCtas * head_block(Hq / Hkv);
    return rows * (D * sizeof(float) + sizeof(float2));
}

cudaError_t launch_paged_attention(const KvCacheSpec &c, const void *q, int64_t q_stride,
                                   const int32_t *lens, const int32_t *table, int max_pages,
                                   int n_seq, int Hq, float scale, void *out, int64_t out_stride,
                                   void *workspace, const LaunchCtx &ctx) {
    PagedArgs a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.k = static_cast<const uint8_t *>(c.k);
    a.v = static_cast<const uint8_t *>(c.v);
    a.k_exp = c.k_exp;
    a.v_exp = c.v_exp;
    a.n_pages = c.n_pages;
    a.log2_page = c.log2_page;
    a.H = c.H;
    a.table = table;
    a.lens = lens;
    a.max_pages = max_pages;
    a.n_seq = n_seq;
    a.G = Hq / c.H;
    const int hb = head_block(a.G);
    a.HB = (a.G + hb - 1) / hb;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.out_stride = out_stride;
    const size_t rows = (size_t)2 * kMaxCtas * hb;
    a.part_ml = static_cast<float2 *>(workspace);
    a.part_o = reinterpret_cast<float *>(a.part_ml + rows);
    a.err = ctx.err;
    if (c.D == 64) {
        if (c.e4m3) return hb == 8 ? launch<64, true, 1>(a, ctx) : launch<64, true, 2>(a, ctx);
        return hb == 8 ? launch<64, false, 1>(a, ctx) : launch<64, false, 2>(a, ctx);
    }
    if (c.D == 128) {
        if (c.e4m3)
            return hb == 8 ? launch<128, true, 1>(a, ctx) : launch<128, true, 2>(a, ctx);
        return hb == 8 ? launch<128, false, 1>(a, ctx) : launch<128, false, 2>(a, ctx);
    }
    return cudaErrorInvalidValue;
}

}  // namespace wanvae
