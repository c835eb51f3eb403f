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
// In 4 bits it is x[d] = 2^(e - off) q[d], q e2m1, with e as above for e2m1's largest
// value, 6, and off, four bits, for each block of 16 elements: how far the block's own
// smallest exponent lies below the row's, at most 14.  (A row whose blocks' magnitudes
// differ keeps its small ones; a scale a block of its own would cost four more bits and
// would not let a row be read as one of e4m3 elements and one scale: seq_dev.cuh.)  e is
// in [-94, 126], 6 above the range of 8 bits, as those elements reach 2^6 times further.
// Elements round to nearest, ties to even: half a step is 2^-2 of the value.  A row of zeros
// has the smallest scale, so that attention's weights for it (which carry the scale) are
// nothing, and need not be looked for.  A row with an
// infinity or a NaN has the scale code 255 and reads as NaN throughout.
//
// In 4 bits 16384 tokens are written in 24 us (3.5 TB/s, 0.52: 3.4 tokens a warp, so that some have
// four, and a token's place, loads, maxima and stores one after another; the 50 or so instructions
// for 8 elements are a quarter of it; a lane with 8 of a block's 16, which then needs the other's
// maximum: 32 us), 73513 read back in 70.5 (5.4 TB/s, 0.80; a block a lane there: 72 to 83).
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
#include <type_traits>

#include "norm_act.cuh"
#include "ptx.cuh"
#include "seq_dev.cuh"
#include "seq_ops.h"
#include "seq_ptx.cuh"

namespace wanvae {
namespace {

constexpr int kThreads = 256;
// Rows of a lane's that are loaded before the first is used, and resident blocks that
// leave the registers for them.  Sixteen sequences, 73513 tokens of 8 heads of 128,
// read back, in us: 8 rows and 3 blocks 81.7, 4 and 4 79.6, 4 and 5 77.7, 4 and 6 87
// (spills), 2 and 6 82.3, 2 and 8 81.6.
// In 4 bits, whose rows are half as long: 8 and 4 70.5 (16384 tokens written: 24.3; there a
// turn counts twice, as a lane has two vectors), 8 and 3 74.2, 4 and 5 73.7 (23.8), 6 and 4 77,
// 12 and 4 - (28.8), 8 and 5 94 (27.8).
template <int F>
constexpr int kFlight = F == kKvE2M1 ? 8 : 4;
template <int F>
constexpr int kBlocks = F == kKvE2M1 ? 4 : 5;
constexpr int kExpMin = -100, kExpMax = 120;
constexpr uint32_t kNanRow = 255;  // scale code of an e2m1 row that is not finite

struct CacheArgs {
    uint8_t *k, *v;
    uint8_t *k_exp, *v_exp;
    uint8_t *k_off, *v_off;
    int n_pages, log2_page, H;
    const int32_t *table;
    int max_pages;
    unsigned *err;
};

// The row of head 0 of a slot of a page (rows of later heads follow a page's height
// apart); -1 where there is no such page.
__device__ __forceinline__ int64_t page_row(const CacheArgs &c, int64_t page, int slot) {
    if (page < 0 || page >= c.n_pages) return -1;
    return ((page * c.H) << c.log2_page) + slot;
}

// That of a token; -1 where the page table has no such page.
__device__ __forceinline__ int64_t cache_row(const CacheArgs &c, int seq, int pos) {
    const int page_no = pos >> c.log2_page;
    int page = -1;
    if (pos >= 0 && page_no < c.max_pages) page = __ldg(c.table + (int64_t)seq * c.max_pages + page_no);
    return page_row(c, page, pos & ((1 << c.log2_page) - 1));
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

// The exponent of a row, or block, of e2m1 elements: ceil(log2(amax / 6)) (6 = 1.5 * 2^2);
// zero for zeros, not yet in its range.
__device__ __forceinline__ int e2m1_exponent(uint32_t amax) {
    return amax == 0u ? 0 : (int)(amax >> 7) - 127 - 2 + ((amax & 0x7fu) > 0x40u ? 1 : 0);
}

// x[j] -> bits 4 j .. 4 j + 3, each the nearest e2m1 value (ties to even).
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// A block of 16 bf16 values -> two words of e2m1 elements (seq_dev.cuh), the row's scale code
// and, in the lanes of a row alike, its blocks' offsets; kLanes lanes hold the row.
template <int kLanes>
__device__ __forceinline__ uint2 quantise4(const uint4 (&v)[2], uint32_t &code, uint32_t &offs) {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    const uint32_t most = max(m & 0xffffu, m >> 16);  // of the block
    uint32_t amax = most;
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1)
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const bool bad = amax >= 0x7f80u;
    int e = min(max(e2m1_exponent(amax), kExpMin + kE2m1Lift), kExpMax + kE2m1Lift);
    if (amax == 0u) e = kExpMin + kE2m1Lift;
    if (bad) e = 0;
    const int off = most == 0u || bad ? 0 : min(max(e - e2m1_exponent(most), 0), kE2m1OffMax);
    code = bad ? kNanRow : (uint32_t)(e + 127);
    offs = (uint32_t)off << (threadIdx.x % kLanes * 4);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) offs |= __shfl_xor_sync(0xffffffffu, offs, o);
    const float inv = __uint_as_float((uint32_t)(127 + off - e) << 23);
    uint32_t r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float x[8];  // magnitudes
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = w[4 * h + i] & 0x7fff7fffu;
            f32x2_split(mul_f32x2(f32x2(nact_lo(two), nact_hi(two)), f32x2(inv, inv)), x[2 * i],
                        x[2 * i + 1]);
        }
        r[h] = f32x8_to_e2m1x8(x);
        // the signs of elements 0 .. 3 (two words) to bits 7, 15, .., of 4 .. 7 to 3, 11, ..
        r[h] |= __byte_perm(w[4 * h], w[4 * h + 1], 0x7531) & kByteSigns;
        r[h] |= (__byte_perm(w[4 * h + 2], w[4 * h + 3], 0x7531) & kByteSigns) >> 4;
    }
    return bad ? make_uint2(0u, 0u) : make_uint2(r[0], r[1]);
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

// 8 e2m1 values of a row -> bf16 (exact, but for what passes its largest value).
__device__ __forceinline__ uint4 dequantise4(uint32_t w, uint32_t code, int off) {
    // as 2^6 times their values in fp16, the offset in the scale
    uint32_t h[2];
    e2m1_bytes(w, e2m1_table_f16(0), h[0], h[1]);
    const float s = code == kNanRow
                        ? __uint_as_float(0x7fc00000u)
                        : __uint_as_float((uint32_t)max((int)code - kE2m1Lift - off, 1) << 23);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = __byte_perm(h[i >> 1], 0u, i & 1 ? 0x3424 : 0x1404);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&two));
        float lo, hi;
        f32x2_split(mul_f32x2(f32x2(f.x, f.y), f32x2(s, s)), lo, hi);
        o[i] = pack_finite(lo, hi);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The first token of this warp (ahead 0) or of the next one: `total` tokens over
// `warps` warps, in order, to within one of each other.
__device__ __forceinline__ int first_token(int total, int warps, int ahead) {
    const int64_t id = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) + ahead;
    return (int)(min(id, (int64_t)warps) * total / warps);
}

// Rows cu_new[s] .. of k and v to the last positions of sequence s, or row i to slot
// slots[i].
template <int D, int F>
__global__ void __launch_bounds__(kThreads, kBlocks<F>)
kv_append_kernel(const CacheArgs c, const __nv_bfloat16 *__restrict__ k, int64_t k_stride,
                 const __nv_bfloat16 *__restrict__ v, int64_t v_stride,
                 const int32_t *__restrict__ lens, const int32_t *__restrict__ cu_new,
                 const int64_t *__restrict__ slots, int n_seq, int total, int warps) {
    griddep_launch_dependents();
    griddep_wait();
    // lanes of a row, each with 8 elements or (4 bits) a block of 16; rows a warp holds; turns
    // that are loaded together
    constexpr int kVecs = F == kKvE2M1 ? 2 : 1, kLanes = D / 8 / kVecs, kRows = 32 / kLanes;
    constexpr int kTurns = kFlight<F> / kVecs;
    const int lane = threadIdx.x & 31, sub = lane % kLanes, grp = lane / kLanes;
    const int t1 = first_token(total, warps, 1);
    int seq = 0, first = 0, end = 0, len = 0;
    for (int t = first_token(total, warps, 0); t < t1; ++t) {
        // the token's H key rows, then its H value rows, kTurns turns' loads at a time; the
        // first are in flight while the token's place is looked up
        const int64_t kt = t * k_stride, vt = t * v_stride;
        uint4 x[kTurns][kVecs];
        auto load = [&](int r0) {
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int r = r0 + i * kRows;
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    x[i][j] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < 2 * c.H)
                        x[i][j] = __ldg(reinterpret_cast<const uint4 *>(
                                            r >= c.H ? v + vt + (r - c.H) * D : k + kt + r * D) +
                                        sub * kVecs + j);
                }
            }
        };
        load(grp);
        int64_t row0;
        if (slots) {
            const int64_t slot = __ldg(slots + t);
            if (slot < 0) continue;  // a row of no sequence
            row0 = page_row(c, slot >> c.log2_page, (int)(slot & ((1 << c.log2_page) - 1)));
        } else {
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
            row0 = end > total ? -1 : cache_row(c, seq, len - (end - t));
        }
        if (row0 < 0) {
            if (lane == 0) atomicOr(c.err, kDevErrAlign);
            continue;
        }
        for (int r0 = grp; r0 < 2 * c.H + grp; r0 += kTurns * kRows) {
            if (r0 >= kTurns * kRows) load(r0);
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int r = r0 + i * kRows;
                if (r - grp >= 2 * c.H) break;
                const bool there = r < 2 * c.H, is_v = r >= c.H;
                const int h = is_v ? r - c.H : r;
                const int64_t row = row0 + ((int64_t)h << c.log2_page);
                uint8_t *dst = (is_v ? c.v : c.k) + row * kv_row_bytes(F, D);
                if constexpr (F == kKvE2M1) {
                    uint32_t code, offs;
                    const uint2 q = quantise4<kLanes>(x[i], code, offs);
                    if (!there) continue;
                    reinterpret_cast<uint2 *>(dst)[sub] = q;
                    if (sub == 0) {
                        (is_v ? c.v_exp : c.k_exp)[row] = (uint8_t)code;
                        uint8_t *o = (is_v ? c.v_off : c.k_off) + row * kv_off_bytes(D);
                        if (D == 128) *reinterpret_cast<uint32_t *>(o) = offs;
                        else *reinterpret_cast<uint16_t *>(o) = (uint16_t)offs;
                    }
                } else if constexpr (F == kKvE4M3) {
                    int e;
                    const uint2 q = quantise8<kLanes>(x[i][0], e);
                    if (!there) continue;
                    reinterpret_cast<uint2 *>(dst)[sub] = q;
                    if (sub == 0) (is_v ? c.v_exp : c.k_exp)[row] = (uint8_t)(e + 127);
                } else if (there) {
                    reinterpret_cast<uint4 *>(dst)[sub] = x[i][0];
                }
            }
        }
    }
}

// Positions 0 .. of sequence s to rows cu[s] .. of k and v.
template <int D, int F>
__global__ void __launch_bounds__(kThreads, kBlocks<F>)
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
        for (int r0 = grp; r0 < 2 * c.H; r0 += kFlight<F> * kRows) {
            uint4 x[kFlight<F>];
            uint32_t code[kFlight<F>];
#pragma unroll
            for (int i = 0; i < kFlight<F>; ++i) {
                const int r = r0 + i * kRows;
                if (r >= 2 * c.H) break;
                const bool is_v = r >= c.H;
                const int64_t row = row0 + ((int64_t)(is_v ? r - c.H : r) << c.log2_page);
                const uint8_t *src = (is_v ? c.v : c.k) + row * kv_row_bytes(F, D);
                if (F == kKvE2M1) {
                    x[i].x = __ldg(reinterpret_cast<const uint32_t *>(src) + sub);
                    x[i].y = __ldg((is_v ? c.v_off : c.k_off) + row * kv_off_bytes(D) + sub / 4);
                    code[i] = __ldg((is_v ? c.v_exp : c.k_exp) + row);
                } else if (F == kKvE4M3) {
                    const uint2 q = __ldg(reinterpret_cast<const uint2 *>(src) + sub);
                    x[i].x = q.x;
                    x[i].y = q.y;
                    code[i] = __ldg((is_v ? c.v_exp : c.k_exp) + row);
                } else {
                    x[i] = __ldg(reinterpret_cast<const uint4 *>(src) + sub);
                }
            }
#pragma unroll
            for (int i = 0; i < kFlight<F>; ++i) {
                const int r = r0 + i * kRows;
                if (r >= 2 * c.H) break;
                __nv_bfloat16 *dst = r >= c.H ? v + vt + (r - c.H) * D : k + kt + r * D;
                reinterpret_cast<uint4 *>(dst)[sub] =
                    F == kKvE2M1 ? dequantise4(x[i].x, code[i], (int)(x[i].y >> (sub & 2 ? 4 : 0) & 15u))
                    : F == kKvE4M3 ? dequantise8(make_uint2(x[i].x, x[i].y), code[i])
                                   : x[i];
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
    a.k_off = c.k_off;
    a.v_off = c.v_off;
    a.n_pages = c.n_pages;
    a.log2_page = c.log2_page;
    a.H = c.H;
    a.table = table;
    a.max_pages = max_pages;
    a.err = ctx.err;
    return a;
}

// Warps of a launch: one resident wave, or one for each token.
int warps_for(int total, int fmt, const LaunchCtx &ctx) {
    const int blocks = fmt == kKvE2M1 ? kBlocks<kKvE2M1> : kBlocks<kKvE4M3>;
    return std::min(total, ctx.num_sms * blocks * (kThreads / 32));
}
unsigned blocks_for(int warps) { return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)); }

}  // namespace

cudaError_t launch_kv_append(const KvCacheSpec &c, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const int32_t *lens, const int32_t *table,
                             int max_pages, const int32_t *cu_new, const int64_t *slots,
                             int n_seq, int total, const LaunchCtx &ctx) {
    const CacheArgs a = cache_args(c, table, max_pages, ctx);
    auto *kp = static_cast<const __nv_bfloat16 *>(k);
    auto *vp = static_cast<const __nv_bfloat16 *>(v);
    const int warps = warps_for(total, c.fmt, ctx);
    const dim3 grid(blocks_for(warps)), block(kThreads);
    auto go = [&](auto kern) {
        return launch_pdl(kern, grid, block, 0, ctx, a, kp, k_stride, vp, v_stride, lens, cu_new,
                          slots, n_seq, total, warps);
    };
    auto pick = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return c.fmt == kKvE2M1   ? go(kv_append_kernel<D, kKvE2M1>)
               : c.fmt == kKvE4M3 ? go(kv_append_kernel<D, kKvE4M3>)
                                  : go(kv_append_kernel<D, kKv16>);
    };
    if (c.D == 64) return pick(std::integral_constant<int, 64>());
    if (c.D == 128) return pick(std::integral_constant<int, 128>());
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_gather(const KvCacheSpec &c, const int32_t *table, int max_pages,
                             const int32_t *cu, int n_seq, int total, void *k, int64_t k_stride,
                             void *v, int64_t v_stride, const LaunchCtx &ctx) {
    const CacheArgs a = cache_args(c, table, max_pages, ctx);
    auto *kp = static_cast<__nv_bfloat16 *>(k);
    auto *vp = static_cast<__nv_bfloat16 *>(v);
    const int warps = warps_for(total, c.fmt, ctx);
    const dim3 grid(blocks_for(warps)), block(kThreads);
    auto go = [&](auto kern) {
        return launch_pdl(kern, grid, block, 0, ctx, a, cu, n_seq, total, warps, kp, k_stride,
                          vp, v_stride);
    };
    auto pick = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return c.fmt == kKvE2M1   ? go(kv_gather_kernel<D, kKvE2M1>)
               : c.fmt == kKvE4M3 ? go(kv_gather_kernel<D, kKvE4M3>)
                                  : go(kv_gather_kernel<D, kKv16>);
    };
    if (c.D == 64) return pick(std::integral_constant<int, 64>());
    if (c.D == 128) return pick(std::integral_constant<int, 128>());
    return cudaErrorInvalidValue;
}

}  // namespace wanvae
