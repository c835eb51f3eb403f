// paged_attn.cuh -- what the two kernels of attention over the cache share: the
// cut of a batch's cached rows into ranges (see paged_attn.cu) and where a range's
// rows lie.
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "seq_dev.cuh"
#include "seq_ops.h"
#include "seq_ptx.cuh"

namespace wanvae {

constexpr int kMaxWays = 152 * 2;  // CTAs of a launch
constexpr int kPieces = 2;         // ranges of a share that any CTA may take
constexpr int kMaxRanges = (1 + kPieces) * kMaxWays;
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
    int ways;        // CTAs
    int *taken;      // ranges taken beyond the shares; NULL: shares alone
    float *part_o;   // [2 ranges][heads of a block][D]
    float2 *part_ml; // [2 ranges][heads of a block]: maximum, sum
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
template <int kUnit>
__device__ __forceinline__ int units_of(int len) {
    return (len + kUnit - 1) / kUnit;
}

// Units before sequence b (all of them for b = n_seq) of one head; whole warp.
template <int kUnit>
__device__ __forceinline__ int units_before(const PagedArgs &p, int b, bool tell) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int i = lane; i < b; i += 32) n += units_of<kUnit>(seq_len(p, i, tell));
    return __reduce_add_sync(0xffffffffu, n);
}

// How `total` units are cut: one share for each of `ways` CTAs, in order.  Where
// ranges are taken, a share ends in kPieces pieces of `small` units, each a range
// of its own, and what is left of it is its first range.
struct Split {
    static constexpr int kOf = 1 + kPieces;  // ranges of a share
    int ways, ranges, q, rem, small;
    __device__ __forceinline__ Split(int total, int most, bool takes) {
        ways = max(1, min(most, total));  // (no share is empty)
        q = total / ways;
        rem = total - q * ways;
        small = takes ? q / 16 : 0;
        ranges = small ? kOf * ways : ways;
    }
    __device__ __forceinline__ int share(int w) const { return q * w + min(w, rem); }
    // The first range of CTA w, and the range taken as number n (first pieces first).
    __device__ __forceinline__ int own(int w) const { return small ? kOf * w : w; }
    __device__ __forceinline__ int taken(int n) const {
        return n < kPieces * ways ? kOf * (n % ways) + 1 + n / ways : ranges;
    }
    __device__ __forceinline__ int begin(int r) const {
        if (!small) return share(r);
        const int w = r / kOf, j = r - w * kOf;
        return j ? share(w + 1) - small * (kOf - j) : share(w);
    }
    __device__ __forceinline__ int of(int unit) const {  // (q is at least 1)
        const int big = rem * (q + 1);
        const int w = unit < big ? unit / (q + 1) : rem + (unit - big) / q;
        if (!small) return w;
        const int behind = unit - (share(w + 1) - small * kPieces);
        return kOf * w + (behind < 0 ? 0 : 1 + behind / small);
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

// Where a range stands: unit u of the U units of (sequence b, head block hh).
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

// The cursor of a unit of the whole batch (whole warp).
template <int kUnit>
__device__ __forceinline__ Cursor<kUnit> locate(const PagedArgs &p, int HH, int unit) {
    const int lane = threadIdx.x & 31;
    Cursor<kUnit> at = {0, 0, 0, 1, 0};
    int before = 0;  // (in units of one head)
    for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
        const int i = b0 + lane;
        const int len = i < p.n_seq ? seq_len(p, i, false) : 0;
        const int U = units_of<kUnit>(len);
        int incl = U;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const unsigned m = __ballot_sync(0xffffffffu, (before + incl) * HH > unit);
        if (m) {
            const int l = __ffs(m) - 1;
            at.b = b0 + l;
            at.U = __shfl_sync(0xffffffffu, U, l);
            at.len = __shfl_sync(0xffffffffu, len, l);
            const int rest = unit - (before + __shfl_sync(0xffffffffu, incl - U, l)) * HH;
            at.hh = rest / at.U;
            at.u = rest - at.hh * at.U;
            break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return at;
}

// Sets a.ways for units of `unit` rows and at most `most` CTAs; false (and a.taken
// NULL) where every CTA keeps to its share.
bool paged_ways(PagedArgs &a, int unit, int most);
cudaError_t launch_paged_begin(const PagedArgs &a, const LaunchCtx &ctx);

// The tcgen05 kernel (paged_attn_tc.cu): 8-bit rows of 128 elements.  *block_heads:
// the heads of a partial result.
constexpr int kPagedTcUnit = 128;
cudaError_t launch_paged_tc(PagedArgs &a, const KvCacheSpec &cache, const LaunchCtx &ctx,
                            int *block_heads);

}  // namespace wanvae
