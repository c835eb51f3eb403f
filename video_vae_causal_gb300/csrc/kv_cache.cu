// kv_cache.cu -- the paged key-value cache: rows quantised as they are
// written, and read back.
//
// A cache row is the key (or value) of one token and one kv head, D elements.
// In 8 bits it is stored as x[d] = 2^e q[d], q e4m3 and e one byte (E8M0) for
// the row: e is the smallest exponent that brings the row's largest
// magnitude to 448 (e4m3's largest value) or below, so nothing saturates,
// dividing by the scale is exact, and a row rounds once, by at most half a
// step of e4m3 (2^-4 relative, above e4m3's subnormals).  e stays in
// [-100, 120]: 2^120 * 448 covers every finite bf16 value, and rows below 2^-100
// round on the grid of 2^-100 (so that attention can carry scales as
// exponents without leaving fp32's range).  Magnitudes from 1.9375 * 2^127 on round to
// 256 * 2^120 = 2^128, which reads back as the largest bf16 value.  Infinities and NaN become
// e4m3's NaN and do not count for the scale.
//
// Rows lie [page][head][slot][D]: the rows of one head and page are
// contiguous, which is how attention over the cache reads them.  Both passes
// move each row once (2 D bytes on one side, D + 1 on the other) and are bound
// by HBM: 73513 tokens of 8 heads of 128 read back take 78 us (5.8 TB/s, 0.86 of
// the measured copy rate), 16384 tokens written 27 us (3.7 TB/s, 0.55: 2.7 tokens a
// warp, so that some have two and some three, and it waits for their places, loads and
// rows' maxima one token after another; loading the next pass's rows as each is used
// spilled and took 29 us).  A row takes D / 8 lanes with
// one 16-byte vector of bf16 each; a warp keeps the rows of a token's heads together and
// takes tokens in a row, so that a token's page is looked up once for all heads and its
// sequence once for the tokens that follow it.
#include <cuda_bf16.h>

#include <algorithm>

#include "norm_act.cuh"
#include "ptx.cuh"
#include "seq_dev.cuh"
#include "seq_ops.h"

namespace wanvae {
namespace {

constexpr int kThreads = 256;
// Rows of a lane's that are loaded before the first is used, and resident blocks that
// leave the registers for them.  Sixteen sequences, 73513 tokens of 8 heads of 128,
// read back, in us: 8 rows and 3 blocks 81.7, 4 and 4 79.6, 4 and 5 77.7, 4 and 6 87
// (spills), 2 and 6 82.3, 2 and 8 81.6.
constexpr int kFlight = 4;
constexpr int kBlocks = 5;
constexpr int kExpMin = -100, kExpMax = 120;

struct CacheArgs {
    uint8_t *k, *v;
    uint8_t *k_exp, *v_exp;
    int n_pages, log2_page, H;
    const int32_t *table;
    int max_pages;
    unsigned *err;
};

// Where a token lies in the cache: the row of head 0 (rows of later heads
// follow a page's height apart); -1 where the page table has no such page.
__device__ __forceinline__ int64_t cache_row(const CacheArgs &c, int seq, int pos) {
    const int page_no = pos >> c.log2_page;
    int page = -1;
    if (pos >= 0 && page_no < c.max_pages) page = __ldg(c.table + (int64_t)seq * c.max_pages + page_no);
    if ((unsigned)page >= (unsigned)c.n_pages) return -1;
    return (((int64_t)page * c.H) << c.log2_page) + (pos & ((1 << c.log2_page) - 1));
}

// The scale's exponent of a row whose largest finite magnitude has the bf16 bits
// amax: ceil(log2(amax / 448)) (448 = 1.75 * 2^8).
__device__ __forceinline__ int row_exponent(uint32_t amax) {
    if (amax == 0u) return 0;
    const int e = (int)(amax >> 7) - 127 - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
    return min(max(e, kExpMin), kExpMax);
}

// Largest of two pairs of 16-bit magnitudes over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1)
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
    return max(m & 0xffffu, m >> 16);
}

// 8 bf16 values -> e4m3 with the row's scale; kLanes lanes hold the row, the whole
// warp takes part.  Magnitudes compare as integers, two at a time; infinities and
// NaN, the largest of them, are looked for only where a row has any.
template <int kLanes>
__device__ __forceinline__ uint2 quantise8(const uint4 &v, int &e) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    uint32_t amax = row_max<kLanes>(m);
    if (__any_sync(0xffffffffu, amax >= 0x7f80u)) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t bad = __vcmpgeu2(w[i] & 0x7fff7fffu, 0x7f807f80u);
            m = __vmaxu2(m, w[i] & 0x7fff7fffu & ~bad);
            w[i] = (w[i] & ~bad) | (bad & 0x7fc07fc0u);
        }
        amax = row_max<kLanes>(m);
    }
    e = row_exponent(amax);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = f32x2_to_e4m3x2(nact_lo(w[i]) * inv, nact_hi(w[i]) * inv);
    return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}

// nact_pack, with what passes the largest value as that value (a NaN stays one; tested).
__device__ __forceinline__ uint32_t pack_finite(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 e4m3 values of a row -> bf16 (exact for scales that leave bf16's range alone; what
// passes its largest value is that value, as nothing that is stored is infinite).
__device__ __forceinline__ uint4 dequantise8(const uint2 &q, uint32_t code) {
    const float s = e8m0_value(code);
    const uint32_t w[2] = {q.x, q.y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = e4m3x2_to_f16x2(w[i >> 1] >> (16 * (i & 1)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        o[i] = pack_finite(f.x * s, f.y * s);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The first token of this warp (ahead 0) or of the next one: `total` tokens over
// `warps` warps, in order, to within one of each other.
__device__ __forceinline__ int first_token(int total, int warps, int ahead) {
    const int64_t id = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) + ahead;
    return (int)(min(id, (int64_t)warps) * total / warps);
}

// Rows cu_new[s] .. of k and v to the last positions of sequence s.
template <int D, bool kQuant>
__global__ void __launch_bounds__(kThreads, kBlocks)
kv_append_kernel(const CacheArgs c, const __nv_bfloat16 *__restrict__ k, int64_t k_stride,
                 const __nv_bfloat16 *__restrict__ v, int64_t v_stride,
                 const int32_t *__restrict__ lens, const int32_t *__restrict__ cu_new, int n_seq,
                 int total, int warps) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes a row, rows a warp holds
    const int lane = threadIdx.x & 31, sub = lane % kLanes, grp = lane / kLanes;
    const int t1 = first_token(total, warps, 1);
    int seq = 0, first = 0, end = 0, len = 0;
    for (int t = first_token(total, warps, 0); t < t1; ++t) {
        // the token's H key rows, then its H value rows, kFlight turns' loads at a time; the
        // first are in flight while the token's place is looked up
        const int64_t kt = t * k_stride, vt = t * v_stride;
        uint4 x[kFlight];
        auto load = [&](int r0) {
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int r = r0 + i * kRows;
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < 2 * c.H)
                    x[i] = __ldg(reinterpret_cast<const uint4 *>(
                                     r >= c.H ? v + vt + (r - c.H) * D : k + kt + r * D) +
                                 sub);
            }
        };
        load(grp);
        if (!cu_new) {
            seq = first = t;
            end = t + 1;
            len = __ldg(lens + seq);
        } else if (t >= end) {
            seq = seq_of_row(cu_new, n_seq, t);
            first = __ldg(cu_new + seq);
            end = __ldg(cu_new + seq + 1);
            len = __ldg(lens + seq);
        }
        if (t < first || t >= end) continue;  // a row behind the last sequence
        const int64_t row0 = end > total ? -1 : cache_row(c, seq, len - (end - t));
        if (row0 < 0) {
            if (lane == 0) atomicOr(c.err, kDevErrAlign);
            continue;
        }
        for (int r0 = grp; r0 < 2 * c.H + grp; r0 += kFlight * kRows) {
            if (r0 >= kFlight * kRows) load(r0);
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int r = r0 + i * kRows;
                if (r - grp >= 2 * c.H) break;
                const bool there = r < 2 * c.H, is_v = r >= c.H;
                const int h = is_v ? r - c.H : r;
                const int64_t row = row0 + ((int64_t)h << c.log2_page);
                uint8_t *dst = (is_v ? c.v : c.k) + row * (kQuant ? D : 2 * D);
                if (kQuant) {
                    int e;
                    const uint2 q = quantise8<kLanes>(x[i], e);
                    if (!there) continue;
                    reinterpret_cast<uint2 *>(dst)[sub] = q;
                    if (sub == 0) (is_v ? c.v_exp : c.k_exp)[row] = (uint8_t)(e + 127);
                } else if (there) {
                    reinterpret_cast<uint4 *>(dst)[sub] = x[i];
                }
            }
        }
    }
}

// Positions 0 .. of sequence s to rows cu[s] .. of k and v.
template <int D, bool kQuant>
__global__ void __launch_bounds__(kThreads, kBlocks)
kv_gather_kernel(const CacheArgs c, const int32_t *__restrict__ cu, int n_seq, int total,
                 int warps, __nv_bfloat16 *__restrict__ k, int64_t k_stride, __nv_bfloat16 *__restrict__ v,
                 int64_t v_stride) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, sub = lane % kLanes, grp = lane / kLanes;
    const int t1 = first_token(total, warps, 1);
    int seq = 0, first = 0, end = 0;
    for (int t = first_token(total, warps, 0); t < t1; ++t) {
        if (t >= end) {
            seq = seq_of_row(cu, n_seq, t);
            first = __ldg(cu + seq);
            end = __ldg(cu + seq + 1);
        }
        if (t < first || t >= end) continue;
        const int64_t row0 = end > total ? -1 : cache_row(c, seq, t - first);
        if (row0 < 0) {
            if (lane == 0) atomicOr(c.err, kDevErrAlign);
            continue;
        }
        const int64_t kt = t * k_stride, vt = t * v_stride;
        for (int r0 = grp; r0 < 2 * c.H; r0 += kFlight * kRows) {
            uint4 x[kFlight];
            uint32_t code[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int r = r0 + i * kRows;
                if (r >= 2 * c.H) break;
                const bool is_v = r >= c.H;
                const int64_t row = row0 + ((int64_t)(is_v ? r - c.H : r) << c.log2_page);
                const uint8_t *src = (is_v ? c.v : c.k) + row * (kQuant ? D : 2 * D);
                if (kQuant) {
                    const uint2 q = __ldg(reinterpret_cast<const uint2 *>(src) + sub);
                    x[i].x = q.x;
                    x[i].y = q.y;
                    code[i] = __ldg((is_v ? c.v_exp : c.k_exp) + row);
                } else {
                    x[i] = __ldg(reinterpret_cast<const uint4 *>(src) + sub);
                }
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int r = r0 + i * kRows;
                if (r >= 2 * c.H) break;
                __nv_bfloat16 *dst = r >= c.H ? v + vt + (r - c.H) * D : k + kt + r * D;
                reinterpret_cast<uint4 *>(dst)[sub] =
                    kQuant ? dequantise8(make_uint2(x[i].x, x[i].y), code[i]) : x[i];
            }
        }
    }
}

CacheArgs cache_args(const KvCacheSpec &c, const int32_t *table, int max_pages,
                     const LaunchCtx &ctx) {
    CacheArgs a;
    a.k = static_cast<uint8_t *>(c.k);
    a.v = static_cast<uint8_t *>(c.v);
    a.k_exp = c.k_exp;
    a.v_exp = c.v_exp;
    a.n_pages = c.n_pages;
    a.log2_page = c.log2_page;
    a.H = c.H;
    a.table = table;
    a.max_pages = max_pages;
    a.err = ctx.err;
    return a;
}

// Warps of a launch: one resident wave, or one for each token.
int warps_for(int total, const LaunchCtx &ctx) {
    return std::min(total, ctx.num_sms * kBlocks * (kThreads / 32));
}
unsigned blocks_for(int warps) { return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)); }

}  // namespace

cudaError_t launch_kv_append(const KvCacheSpec &c, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const int32_t *lens, const int32_t *table,
                             int max_pages, const int32_t *cu_new, int n_seq, int total,
                             const LaunchCtx &ctx) {
    const CacheArgs a = cache_args(c, table, max_pages, ctx);
    auto *kp = static_cast<const __nv_bfloat16 *>(k);
    auto *vp = static_cast<const __nv_bfloat16 *>(v);
    const int warps = warps_for(total, ctx);
    const dim3 grid(blocks_for(warps)), block(kThreads);
    auto go = [&](auto kern) {
        return launch_pdl(kern, grid, block, 0, ctx, a, kp, k_stride, vp, v_stride, lens, cu_new,
                          n_seq, total, warps);
    };
    if (c.D == 64) return c.e4m3 ? go(kv_append_kernel<64, true>) : go(kv_append_kernel<64, false>);
    if (c.D == 128)
        return c.e4m3 ? go(kv_append_kernel<128, true>) : go(kv_append_kernel<128, false>);
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_gather(const KvCacheSpec &c, const int32_t *table, int max_pages,
                             const int32_t *cu, int n_seq, int total, void *k, int64_t k_stride,
                             void *v, int64_t v_stride, const LaunchCtx &ctx) {
    const CacheArgs a = cache_args(c, table, max_pages, ctx);
    auto *kp = static_cast<__nv_bfloat16 *>(k);
    auto *vp = static_cast<__nv_bfloat16 *>(v);
    const int warps = warps_for(total, ctx);
    const dim3 grid(blocks_for(warps)), block(kThreads);
    auto go = [&](auto kern) {
        return launch_pdl(kern, grid, block, 0, ctx, a, cu, n_seq, total, warps, kp, k_stride,
                          vp, v_stride);
    };
    if (c.D == 64) return c.e4m3 ? go(kv_gather_kernel<64, true>) : go(kv_gather_kernel<64, false>);
    if (c.D == 128)
        return c.e4m3 ? go(kv_gather_kernel<128, true>) : go(kv_gather_kernel<128, false>);
    return cudaErrorInvalidValue;
}

}  // namespace wanvae
