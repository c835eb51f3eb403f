// paged_attn.cuh -- what the two kernels of attention over the cache share: the
// cut of a batch's cached rows into ranges (see paged_attn.cu) and where a range's
// rows lie.
#pragma once

#include <cuda_bf16.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "seq_dev.cuh"
#include "seq_ops.h"
#include "seq_ptx.cuh"

namespace wanvae {

constexpr int kMaxWays = 152 * 2;  // CTAs of a launch
constexpr uint64_t kPagedDrainNs = 200ull * 1000 * 1000;

struct PagedArgs {
    const __nv_bfloat16 *q;
    int64_t q_stride;
    const uint8_t *k_exp, *v_exp;
    int n_pages, log2_page, H;
    const int32_t *table, *lens;
    int max_pages, n_seq;
    int G, HB;  // query heads of a kv head; blocks of heads that a kv head is read for
    float scale_log2;
    __nv_bfloat16 *out;
    int64_t out_stride;
    int ways;        // CTAs that share the units; 0: an item a CTA
    float *part_o;   // [2 CTAs][heads of a block][D]
    float4 *part_ml; // [2 CTAs][heads of a block]: m and r (below; 8 bits alone), sum
    unsigned *err;
    uint64_t wait_ns;
};

// A sequence's length as far as the page table reaches.
__device__ __forceinline__ int seq_len(const PagedArgs &p, int b, bool tell) {
    const int len = __ldg(p.lens + b);
    const int64_t most = (int64_t)p.max_pages << p.log2_page;
    if (len >= 0 && len <= most) return len;
    if (tell) atomicOr(p.err, kDevErrAlign);
    return len < 0 ? 0 : (int)most;
}

// A kernel's units: kRows cached rows of one kv head, and what an item (a sequence
// and a block of heads) costs besides them, in units.  Shares are cut in these,
// places: an item of U units has kExtra + U, its units the last ones.
template <int kRows_, int kExtra_>
struct Units {
    static constexpr int kRows = kRows_, kExtra = kExtra_;
    static __device__ __forceinline__ int of(int len) { return (len + kRows - 1) / kRows; }
    static __device__ __forceinline__ int places(int len) {
        return len > 0 ? of(len) + kExtra : 0;
    }
    // Places before sequence b (all of them for b = n_seq) of one head; whole warp.
    static __device__ __forceinline__ int before(const PagedArgs &p, int b, bool tell) {
        int n = 0;
        for (int i = threadIdx.x & 31; i < b; i += 32) n += places(seq_len(p, i, tell));
        return __reduce_add_sync(0xffffffffu, n);
    }
};

// How `total` places are cut: one share for each of `ways` CTAs, in order.
struct Split {
    int ways, q, rem;
    __device__ __forceinline__ Split(int total, int most) {
        ways = max(1, min(most, total));  // (no share is empty)
        q = total / ways;
        rem = total - q * ways;
    }
    __device__ __forceinline__ int begin(int w) const { return q * w + min(w, rem); }
    __device__ __forceinline__ int of(int place) const {  // (q is at least 1)
        const int big = rem * (q + 1);
        return place < big ? place / (q + 1) : rem + (place - big) / q;
    }
};

// 16 bytes or a multiple of global memory to shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Where a share stands: unit u of the U units of (sequence b, head block hh), `left`
// places of the share from it on.
template <class U_>
struct Cursor {
    int b, hh, u, U, len, left;
    // The item's units from here on that the share holds.
    __device__ __forceinline__ int units() const { return min(U - u, left); }
    // On to unit u + n of the item (n at most units()), or to the next item's first;
    // true where the item changed.  The share has ended where left is 0.
    __device__ __forceinline__ bool next(const PagedArgs &p, int HH, int n) {
        u += n;
        left -= n;
        if (u < U) return false;
        u = 0;
        left = max(left - U_::kExtra, 0);
        if (left == 0 || ++hh < HH) return true;
        hh = 0;
        do {
            if (++b >= p.n_seq) {
                left = 0;
                return true;
            }
            len = seq_len(p, b, false);
            U = U_::of(len);
        } while (U == 0);
        return true;
    }
};

// The first unit of a share that begins at `place` of the batch and has `left`
// places (whole warp).
template <class U_>
__device__ __forceinline__ Cursor<U_> locate(const PagedArgs &p, int HH, int place, int left) {
    const int lane = threadIdx.x & 31;
    Cursor<U_> at = {0, 0, 0, 1, 0, 0};
    int before = 0;  // (of one head)
    for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
        const int i = b0 + lane;
        const int len = i < p.n_seq ? seq_len(p, i, false) : 0;
        const int n = U_::places(len);
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const unsigned m = __ballot_sync(0xffffffffu, (before + incl) * HH > place);
        if (m) {
            const int l = __ffs(m) - 1;
            at.b = b0 + l;
            at.len = __shfl_sync(0xffffffffu, len, l);
            at.U = U_::of(at.len);
            const int rest = place - (before + __shfl_sync(0xffffffffu, incl - n, l)) * HH;
            const int each = at.U + U_::kExtra;
            at.hh = rest / each;
            const int j = rest - at.hh * each;  // place of the item
            at.u = max(j - U_::kExtra, 0);
            at.left = max(left - max(U_::kExtra - j, 0), 0);
            break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return at;
}

// Two references in log2 units belong to a head's output and sum: m, a little below or at the
// largest s + e (a row's score, and the exponent of its value row's scale), which the
// output's weights 2^(s + e - m) are relative to, and r, at most kSumLag below the largest s
// and never above it, for the sum of 2^(s - r).  One reference for both would not do: scales
// reach from 2^-100 to 2^120, and a sum relative to m lost every row more than 2^6 below the
// largest under scales of 2^120, or all rows but some where scales lie 2^126 apart.  Both
// begin at kLowest, which any score passes.
constexpr float kLowest = -FLT_MAX;
constexpr float kSumLag = 60.f;  // (2^31 rows of 2^60 stay in fp32's range)

// The output from sums relative to m and r, zero where no row counted: acc / sum *
// 2^(m - r), this last in two factors, as m - r is up to 120 + kSumLag.  (Rows of 16 bits have
// no scales, and one reference.)
__device__ __forceinline__ float half_factor(float m, float r) { return exp2_fast(0.5f * (m - r)); }
template <bool Q8>
__device__ __forceinline__ float output_of(float acc, float sum, float half) {
    const float o = sum > 0.f || sum != sum ? acc / sum : 0.f;
    return Q8 ? o * half * half : o;
}

// An output as bf16.  What 8-bit rows hold is finite or NaN, so a sum that passes bf16's
// largest value is that value (rows near it round to 2^128; read back they saturate too).
template <bool Q8>
__device__ __forceinline__ __nv_bfloat16 to_output(float v) {
    const float most = __uint_as_float(0x7f7f0000u);
    if (Q8 && v == v) v = fminf(fmaxf(v, -most), most);
    return __float2bfloat16(v);
}

// That no s lies more than kSumLag above r is seen from the value rows' exponents alone: s + e
// is at most m and a lag of m's, so that e >= least_e = m - r - (kSumLag - that lag) will do,
// one comparison a row for all heads.  Where it does not hold, or m moves, r moves up:
__device__ __forceinline__ void raise_sum(float top, float &r, float &l) {
    const float rn = fmaxf(r, top);
    l *= exp2_fast(r - rn);
    r = rn;
}

// The CTAs of a launch: as many as there can be units, at most `most`.
int paged_ways(const PagedArgs &a, int rows, int most);

// The tcgen05 kernel (paged_attn_tc.cu): 8-bit rows of 128 elements, at most 8 query
// heads a kv head.  An item costs about two units besides its own: the queries' way into
// shared memory, the first maximum, the joined output (64 sequences of 17 to 8192
// rows, 8 kv heads of 8 query heads: 118, 113 and 113 us with 1, 2 and 3 counted).
// *block_heads: the heads of a partial result.
using TcUnits = Units<256, 2>;
cudaError_t launch_paged_tc(PagedArgs &a, const KvCacheSpec &cache, const LaunchCtx &ctx,
                            int *block_heads);

}  // namespace wanvae
