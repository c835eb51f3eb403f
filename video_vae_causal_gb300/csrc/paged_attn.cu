// paged_attn.cu -- attention of one new token for each sequence over a paged
// key-value cache (kv_cache.cu), split over the cache's length and joined:
//
//     out[b, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q[b, h] . k_j)
//
// over the lens[b] cached rows of kv head h / G.  Every row is read once for up to
// 16 of the G query heads that share it (once more for every 16 after that), so the work
// is 16 multiply-adds a cache byte or less and the bound is HBM.
//
// Split.  The rows of one (sequence, kv head) are cut into units of 64 or 128; the
// units of the whole batch, laid end to end, are dealt to the CTAs in equal
// contiguous shares, so a ragged batch and a single long sequence load every
// multiprocessor alike (behind short page tables each item is a CTA's own: kApartBytes).
// A share may begin or end inside an item: then its CTA
// leaves a partial result (the running maximum, the sum and the unnormalised output) in
// the workspace, two slots a CTA, and a second small kernel joins them in the order of
// the CTAs.  Which CTA left what follows from the lengths alone, so nothing is
// counted, reset or raced for.  (Shares whose last tenth any CTA could take, by a
// counter, ended within 5 % of each other instead of 10, but each piece so taken cost
// its CTA 4 us to begin: 61 -> 67 us for 131040 rows of 8 heads.)
//
// A warp takes 16 or 32 rows of a unit, for which one lane starts two TMA loads of
// 16 rows each (keys, values) into the warp's own queue, kStages turns deep; no
// warp waits for another until an item ends.  Thread (g, t) = (lane / 4, lane % 4)
// needs, as the B operand of S = Q K^T, a quarter of two key rows and, as the A operand
// of O^T = V^T P^T, an eighth of four value rows.  The order of the elements along
// the summed dimension is free, so these are whole 16-byte pieces, and the order of
// the rows is chosen so that with TMA's swizzle eight lanes read eight banks' pieces
// (rows of 128 bytes: column g of S is row g / 2 + 4 (g % 2)).
//
// 8-bit elements become fp16, exactly, on their way into the MMA (mma.sync of e4m3 operands
// has no rate of its own here).  A query is scaled by a power of two that brings its
// largest element to exponent 14, where bf16's 8 bits stay whole down to 2^-31 of it
// and below that round to within 2^-39 of it; weights round once to fp16.  A key row's
// scale multiplies its score; a value row's scale 2^e joins the exponent of its weight,
// w_j = 2^(s_j + e_j - m) with m the running maximum of s_j + e_j, so that weights stay in
// fp16's upper range whatever the scales are, while the sum takes 2^(s_j - r) in fp32, r the
// running maximum of the scores alone (see paged_attn.cuh).  A weight is off by 2^-11 of
// itself or, where that is more, by 2^-25 of the largest 2^(s + e); rows of zeros (scale 1) do
// not count there.  They are looked for where m would move, which is seldom, among rows of
// e = 0 alone (as in the tcgen05 kernel, where the values may still be on their way).
//
// Over 16-bit rows the weights round to bf16, the type that the values have (an MMA's operands
// share one), and carry no scales: r is m.
//
// What bounds it: HBM for 16-bit rows (64 sequences of 17 to 8192 rows, 8 kv heads of 4 query
// heads of 128: 174 us, 6.2 TB/s, 0.91 of the measured copy rate; of 64: 93 us, 5.8 TB/s),
// the conversions for 8-bit ones (of 64: 91 us, 3.0 TB/s; one sequence of 131040 rows, 8
// heads of 8 of 128: 60 us, 4.5 TB/s, of 16: 67 us; about 470 warp instructions for 16 rows of
// 128, half as many for 64).  Where a long 8-bit cache of 128-element heads
// would wait for those, the tensor core reads it as it is: paged_attn_tc.cu.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "norm_act.cuh"
#include "paged_attn.cuh"

namespace wanvae {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kJoinThreads = 128;
constexpr float kLag = 4.f;  // how far a score may pass m before m moves
// Keys of an item (a sequence and a block of heads), as far as the page table reaches, up
// to which a CTA takes an item whole and no join follows; twice this where a quarter of
// the CTAs have one, four times where all have.  Shared / apart, in us with the host's call,
// tables of 16-row pages, 8-bit rows of 128: 8 items of 256 rows 10.8 / 8.9, of 512 11.3 /
// 9.4, of 1024 11.0 / 14.9; 128 of 1024 19.4 / 18.8, of 2048 25.9 / 33.6; 320 of 1 to 2000
// 31.3 / 33.0, 512 42.3 / 48.3, 1600 116 / 108 (four times is early for a few hundred ragged
// items); 16-bit rows of 128: 8 of 256 11.2 / 8.7, 128 of 512 15.3 / 12.5, 512 of 1 to 1000
// 32.7 / 31.9.
constexpr int64_t kApartBytes = 64 << 10;

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
    static constexpr int EB = Q8 ? 1 : 2;            // bytes of an element
    static constexpr int RB = D * EB;                // bytes of a row
    static constexpr int SB = RB < 128 ? RB : 128;   // bytes of a row of a TMA box
    static constexpr int NS = RB / SB;               // boxes of 16 rows
    static constexpr int KC = RB / 64;               // 16-byte pieces of a key row, a thread
    static constexpr int VB = RB / 8 < 16 ? 8 : 16;  // bytes of a value piece
    static constexpr int VC = RB / 8 / VB;           // pieces of a value row, a thread
    // Groups of 16 rows of a warp's turn, and resident CTAs.
    static constexpr int NG = RB >= 256 ? 1 : 2;
    static constexpr int kCtas = 2;
    static constexpr int kUnit = 16 * NG * kWarps;   // cache rows of a unit
    // An item's queries, first loads and join cost about two units: 32 sequences of 50 to
    // 6000 rows, 4 kv heads, 16-bit rows of 128, take 44.1, 40.7 and 40.8 us with 0, 2 and
    // 4 counted, 64 of 17 to 8192 rows, 8 kv heads, 178, 174 and 175 (8-bit rows of 64: 100,
    // 89 and 91).
    using U = Units<kUnit, 2>;
    static constexpr int kHalf = 16 * RB;            // bytes of a group's keys, or values
    static constexpr int kTurn = NG * 2 * kHalf;     // bytes of a warp's turn
    static constexpr int kRoom = (220 / kCtas - 2) * 1024 / (kWarps * kTurn);
    static constexpr int kStages = kRoom > 6 ? 6 : kRoom;
    static constexpr int kExpOff = kStages * kWarps * kTurn;  // 32 bytes a group
    static constexpr int kBarOff = kExpOff + kStages * kWarps * NG * 32;
    static constexpr int kMetaOff = kBarOff + kStages * kWarps * 8;
    static constexpr int kMlOff = kMetaOff + kStages * kWarps * 4;
    static constexpr int kAbortOff = kMlOff + kWarps * NH * 8 * 16;
    static constexpr int kSmem = 1024 + kAbortOff + 16;
    static_assert(kStages >= 2, "queue");
    // A warp's outputs wait for the join in its part of the turn just read:
    // [D][8] floats for each 8 heads, 8 more behind every 16 rows where there is
    // room (bank conflicts).
    static constexpr int kPad = (D + D / 16) * 8 * 4 * NH <= kTurn ? 8 : 0;
    static constexpr int kJoinHeads = (D * 8 + D / 16 * kPad);  // floats of 8 heads
    static_assert(kJoinHeads * 4 * NH <= kTurn, "join buffer");
    // The cache row that column n of S's 8 stands for, and the byte in a box of
    // 16-byte piece x of row r (TMA's swizzle of 128- and 64-byte rows).
    static __device__ __forceinline__ int row_of(int n) {
        return SB == 128 ? (n >> 1) + 4 * (n & 1) : n;
    }
    static __device__ __forceinline__ int piece(int r, int x) {
        return r * SB + ((x ^ (SB == 128 ? r & 7 : (r >> 1) & 3)) << 4);
    }
};

template <int D, bool Q8, int NH>
__global__ void __launch_bounds__(kThreads, Shape<D, Q8, NH>::kCtas)
paged_attn_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                  const PagedArgs p) {
    using S = Shape<D, Q8, NH>;
    constexpr int NG = S::NG;
    constexpr int kSteps = D / 16;  // 16-row tiles of O^T
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t base = smem_u32(smem);
    const uint32_t bars = base + S::kBarOff + warp * S::kStages * 8;
    uint8_t *turns = smem + warp * S::kStages * S::kTurn;  // this warp's queue
    uint8_t *exps = smem + S::kExpOff + warp * S::kStages * NG * 32;
    int *meta = reinterpret_cast<int *>(smem + S::kMetaOff) + warp * S::kStages;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kAbortOff);
    if (lane == 0) {
        for (int s = 0; s < S::kStages; ++s) mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
        if (warp == 0) {
            tma_prefetch_desc(&mK);
            tma_prefetch_desc(&mV);
            *abort_flag = 0;
        }
    }
    __syncthreads();
    griddep_wait();
    const int HH = p.H * p.HB;
    Cursor<typename S::U> at;  // the unit to compute next
    if (p.ways == 0) {         // an item a CTA
        at.b = blockIdx.x / HH;
        at.hh = blockIdx.x - at.b * HH;
        at.u = 0;
        at.len = seq_len(p, at.b, at.hh == 0 && warp == 0);
        at.U = at.left = S::U::of(at.len);
        if (at.len == 0) {
            const int kvh = at.hh / p.HB, h0 = kvh * p.G + (at.hh % p.HB) * 8 * NH;
            const int n = min(8 * NH, (kvh + 1) * p.G - h0) * D;
            for (int e = threadIdx.x; e < n; e += kThreads)
                p.out[(int64_t)at.b * p.out_stride + (int64_t)h0 * D + e] = __float2bfloat16(0.f);
            return;
        }
    } else {
        const int total = S::U::before(p, p.n_seq, blockIdx.x == 0 && warp == 0) * HH;
        const Split split(total, p.ways);
        if ((int)blockIdx.x >= split.ways || total == 0) return;
        const int begin = split.begin(blockIdx.x);
        at = locate<typename S::U>(p, HH, begin, split.begin(blockIdx.x + 1) - begin);
    }
    const WaitCtl wc{p.wait_ns, p.err, abort_flag, 0u};
    bool ok = true;       // no wait of this warp has run out
    int fills = 0;        // turns copied, and the place in the queue of the next
    int put = 0, stage = 0;
    uint32_t phase = 0;   // of the turn to read next, at `stage`

    // ---- copies, by lane 0: `ahead` is the unit to copy next, `page` its pages
    // (loaded one unit early), `kvh_ahead` its kv head
    Cursor<typename S::U> ahead = at;
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
    if (lane == 0) find_pages();
    auto copy = [&]() {
        if (lane == 0 && ahead.left > 0 && ok) {
            const uint32_t bar = bars + 8 * put;
            int rows[NG], told = 0, groups = 0;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int tok = ahead.u * S::kUnit + (warp * NG + i) * 16;
                rows[i] = min(max(ahead.len - tok, 0), 16);
                if ((unsigned)page[i] >= (unsigned)p.n_pages) {
                    if (rows[i]) atomicOr(p.err, kDevErrAlign);
                    rows[i] = 0;
                }
                told |= rows[i] << (8 * i);
                groups += rows[i] > 0;
            }
            meta[put] = told;
            mbar_arrive_expect_tx(bar, groups * (2 * S::kHalf + (Q8 ? 32 : 0)));
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                if (rows[i] == 0) continue;
                const int slot = (kvh_ahead << p.log2_page) +
                                 ((ahead.u * S::kUnit + (warp * NG + i) * 16) &
                                  ((1 << p.log2_page) - 1));
                const uint32_t dst = smem_u32(turns) + put * S::kTurn + i * 2 * S::kHalf;
#pragma unroll
                for (int c = 0; c < S::NS; ++c) {
                    tma_load_3d(dst + c * 16 * S::SB, &mK, bar, c * S::SB / 2, slot, page[i]);
                    tma_load_3d(dst + S::kHalf + c * 16 * S::SB, &mV, bar, c * S::SB / 2, slot,
                                page[i]);
                }
                if (Q8) {
                    const int64_t row = (((int64_t)page[i] * p.H) << p.log2_page) + slot;
                    const uint32_t ex = smem_u32(exps) + (put * NG + i) * 32;
                    bulk_load(ex, p.k_exp + row, 16, bar);
                    bulk_load(ex + 16, p.v_exp + row, 16, bar);
                }
            }
            ++fills;
            put = put + 1 == S::kStages ? 0 : put + 1;
            if (ahead.next(p, HH, 1)) kvh_ahead = ahead.hh / p.HB;
            if (ahead.left > 0) find_pages();
        }
    };
#pragma unroll 1
    for (int s = 0; s < S::kStages - 1; ++s) copy();

    // ---- one item after another
    bool first = true;
    while (at.left > 0) {
        const int units = at.units();  // of this item, in this share
        const bool whole = at.u == 0 && units == at.U;
        const int kvh = at.hh / p.HB, h0 = kvh * p.G + (at.hh % p.HB) * 8 * NH;
        const int heads = min(8 * NH, (kvh + 1) * p.G - h0);
        // the queries as A operands: word w of piece c goes with elements
        // d = (64 c + 16 t) / EB + 4 w .. + 3 of heads g + 8 h
        uint32_t qa[kSteps][2][NH];
        float qs[NH];  // what a score of head g + 8 h is multiplied by, in log2 units
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const __nv_bfloat16 *src =
                p.q + (int64_t)at.b * p.q_stride + (int64_t)(h0 + g + 8 * h) * D;
            uint2 raw[kSteps];
            uint32_t amax = 0;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                constexpr int kPer = 16 / S::EB / 4;  // words of a piece
                const int d = (64 * (s / kPer) + 16 * t) / S::EB + 4 * (s % kPer);
                raw[s] = make_uint2(0u, 0u);
                if (g + 8 * h < heads) raw[s] = __ldg(reinterpret_cast<const uint2 *>(src + d));
                amax = max(amax, max(raw[s].x & 0x7fffu, (raw[s].x >> 16) & 0x7fffu));
                amax = max(amax, max(raw[s].y & 0x7fffu, (raw[s].y >> 16) & 0x7fffu));
            }
            qs[h] = p.scale_log2;
            float down = 1.f;
            if (Q8) {
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^(14 - exponent of the largest); both powers stay in fp32's range
                const int ex = min(max((int)(amax >> 7), 15), 254) - 127 - 14;
                down = __uint_as_float((uint32_t)(127 - ex) << 23);
                qs[h] *= __uint_as_float((uint32_t)(127 + ex) << 23);
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                qa[s][0][h] = Q8 ? pack16<true>(nact_lo(raw[s].x) * down, nact_hi(raw[s].x) * down)
                                 : raw[s].x;
                qa[s][1][h] = Q8 ? pack16<true>(nact_lo(raw[s].y) * down, nact_hi(raw[s].y) * down)
                                 : raw[s].y;
            }
        }
        // of head g + 8 i; the sum, and r of an 8-bit cache, of this thread's rows alone
        float m[NH], r[NH], l[NH];
        float o[NH][kSteps][4];
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            m[i] = r[i] = kLowest;
            l[i] = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][s][k] = 0.f;
        }

        float least_e = INFINITY;
        for (int n = 0; n < units; ++n) {
            __syncwarp();  // the turn before this one is read: its place is free
            copy();
            ok = ok && mbar_wait_warp<false>(bars + 8 * stage, phase, wc);
            if (!ok) continue;  // (on to the barriers of the join)
            const uint8_t *src = turns + stage * S::kTurn;
            const int rows = meta[stage];
            // S = Q K^T: columns 2 t and 2 t + 1 of each 8 rows of a group, heads g, g + 8
            float sc[NG][2][4] = {};
#pragma unroll
            for (int c = 0; c < S::KC; ++c) {
                uint4 w4[NG][2];
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        w4[i][j] = *reinterpret_cast<const uint4 *>(
                            src + i * 2 * S::kHalf + c * 64 / S::SB * 16 * S::SB +
                            S::piece(8 * j + S::row_of(g), c * 4 % (S::SB / 16) + t));
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
            // the rows' scales: keys' as factors, values' as exponents.  Column c of
            // this thread's two is byte t of the 4 rows 4 c .. of 8 (rows of 128 bytes)
            // or byte 2 t + c.
            float kf[NG][2][2], ve[NG][2][2];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
                if (Q8) {
                    kx = *reinterpret_cast<const uint4 *>(exps + (stage * NG + i) * 32);
                    vx = *reinterpret_cast<const uint4 *>(exps + (stage * NG + i) * 32 + 16);
                }
                const uint32_t kw[4] = {kx.x, kx.y, kx.z, kx.w}, vw[4] = {vx.x, vx.y, vx.z, vx.w};
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        kf[i][j][c] = 1.f;
                        ve[i][j][c] = 0.f;
                        if (!Q8) continue;
                        const uint32_t ka = S::SB == 128 ? kw[2 * j + c] : t < 2 ? kw[2 * j] : kw[2 * j + 1];
                        const uint32_t va = S::SB == 128 ? vw[2 * j + c] : t < 2 ? vw[2 * j] : vw[2 * j + 1];
                        const uint32_t at_byte = S::SB == 128 ? t : (2 * t + c) & 3;
                        // the code to an exponent; 2^23 + code, less 2^23 + 127
                        kf[i][j][c] =
                            __uint_as_float(__byte_perm(ka, 0u, 0x0444u | (at_byte << 12)) >> 1);
                        ve[i][j][c] = __uint_as_float(__byte_perm(va, 0x4b000000u, 0x7440u | at_byte)) -
                                      8388735.f;
                    }
            }
            uint32_t pb[NH][NG][2];
            // (least_e: see paged_attn.cuh; rows that are not there, whose scales are whatever
            // lay in the queue's place, ask for nothing)
            bool low = false;
            if (Q8) {
                if (rows != (NG == 2 ? 0x1010 : 0x10)) {
#pragma unroll
                    for (int i = 0; i < NG; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (8 * j + S::row_of(2 * t + c) >= ((rows >> (8 * i)) & 0xff))
                                    ve[i][j][c] = 128.f;
                }
                float x = INFINITY;
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) x = min3(x, ve[i][j][0], ve[i][j][1]);
                low = x < least_e;
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                float s[NG][2][2], mx;
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
                                if (8 * j + S::row_of(2 * t + c) >= ((rows >> (8 * i)) & 0xff))
                                    s[i][j][c] = -INFINITY;
                }
                float sv[NG][2][2];  // with the value rows' exponents
                auto largest = [&]() {
                    mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NG; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            sv[i][j][0] = s[i][j][0] + ve[i][j][0];
                            sv[i][j][1] = s[i][j][1] + ve[i][j][1];
                            mx = max3(mx, sv[i][j][0], sv[i][j][1]);
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                };
                largest();
                // the maximum moves only by more than 2^4: weights stay below 16,
                // their sums below fp16's products' fp32 range, and O is seldom rescaled
                if (__any_sync(0xffffffffu, mx > m[h] + kLag || low)) {
                    if (Q8) {
                        // A value row of zeros (scale 1: e = 0) has no part in the maximum:
                        // it would take the bits of the weights that count.  The eight
                        // lanes of a t look at a row together.
                        bool unsure = false;
#pragma unroll
                        for (int i = 0; i < NG; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                unsure |= ve[i][j][0] == 0.f || ve[i][j][1] == 0.f;
                        if (__any_sync(0xffffffffu, unsure)) {
#pragma unroll
                            for (int i = 0; i < NG; ++i)
#pragma unroll
                                for (int j = 0; j < 2; ++j)
#pragma unroll
                                    for (int c = 0; c < 2; ++c) {
                                        const int row = 8 * j + S::row_of(2 * t + c);
                                        const uint2 *a = reinterpret_cast<const uint2 *>(
                                            src + i * 2 * S::kHalf + S::kHalf +
                                            S::piece(row, S::VB == 16 ? g : g >> 1));
                                        uint2 x = a[S::VB == 16 ? 0 : g & 1];
                                        if (S::VB == 16) {
                                            const uint2 y = a[1];
                                            x.x |= y.x;
                                            x.y |= y.y;
                                        }
                                        const bool some = ((x.x | x.y) & 0x7f7f7f7fu) != 0u;
                                        const unsigned any = __ballot_sync(0xffffffffu, some);
                                        if (!(any & (0x11111111u << t)) && ve[i][j][c] == 0.f) {
                                            ve[i][j][c] = -INFINITY;
                                            low = true;  // (for the other 8 heads)
                                        }
                                    }
                            largest();
                        }
                        float top = -INFINITY;
#pragma unroll
                        for (int i = 0; i < NG; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) top = max3(top, s[i][j][0], s[i][j][1]);
                        raise_sum(top, r[h], l[h]);
                    }
                    const float mn = fmaxf(m[h], mx);
                    const float f = exp2_fast(m[h] - mn);
                    m[h] = mn;
                    if (!Q8) l[h] *= f;
                    const float f0 = __shfl_sync(0xffffffffu, f, 8 * t);
                    const float f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        o[h][k][0] *= f0;
                        o[h][k][1] *= f1;
                        o[h][k][2] *= f0;
                        o[h][k][3] *= f1;
                    }
                    if (Q8)
                        least_e = fmaxf(m[0] - r[0], m[NH - 1] - r[NH - 1]) - (kSumLag - kLag);
                }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    float w[2][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float e = exp2_fast(s[i][j][c] - (Q8 ? r[h] : m[h]));
                            l[h] += e;
                            w[j][c] = Q8 ? exp2_fast(sv[i][j][c] - m[h]) : e;
                        }
                    pb[h][i][0] = pack16<Q8>(w[0][0], w[0][1]);
                    pb[h][i][1] = pack16<Q8>(w[1][0], w[1][1]);
                }
            }
            // O^T += V^T P^T: tile s holds elements 2 s (rows g) and 2 s + 1
            // (rows g + 8) of this thread's piece of the value rows
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const uint8_t *vsrc = src + i * 2 * S::kHalf + S::kHalf;
                const int have = (rows >> (8 * i)) & 0xff;
#pragma unroll
                for (int c = 0; c < S::VC; ++c) {
                    uint32_t r[4][S::VB / 4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = S::row_of(2 * t + (j & 1)) + 8 * (j >> 1);
                        const uint8_t *a = vsrc + c * 16 * S::SB +
                                           S::piece(row, S::VB == 16 ? g : g >> 1) +
                                           (S::VB == 16 ? 0 : (g & 1) * 8);
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
                    if (have != 16) {  // what lies behind the length may be anything
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int x = 0; x < S::VB / 4; ++x)
                                if (S::row_of(2 * t + (j & 1)) + 8 * (j >> 1) >= have) r[j][x] = 0u;
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
            if (++stage == S::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }

        // ---- join the warps, then leave the result or a partial one.  A warp's
        // outputs go to the turn that it has just read (the next copy into it comes
        // after the second barrier).
        const int last = (stage == 0 ? S::kStages : stage) - 1;
        float4 *ml = reinterpret_cast<float4 *>(smem + S::kMlOff);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            if (Q8) {
                float top = fmaxf(r[i], __shfl_xor_sync(0xffffffffu, r[i], 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                l[i] *= exp2_fast(r[i] - top);
                r[i] = top;
            }
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (t == 0)
                ml[(warp * NH + i) * 8 + g] = make_float4(m[i], Q8 ? r[i] : 0.f, l[i], 0.f);
            float *dst = reinterpret_cast<float *>(turns + last * S::kTurn) + i * S::kJoinHeads;
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
        if (threadIdx.x < heads) {
            // a thread for each head: the warps' factors in place of their m, and with the
            // first the head's sum and half_factor
            const int h = threadIdx.x, i = h >> 3, hr = h & 7;
            float4 mw[kWarps];
            float top = kLowest, rtop = kLowest, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                mw[w] = ml[(w * NH + i) * 8 + hr];
                top = fmaxf(top, mw[w].x);
                if (Q8) rtop = fmaxf(rtop, mw[w].y);
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2_fast(mw[w].x - top);
                sum += (Q8 ? exp2_fast(mw[w].y - rtop) : f) * mw[w].z;
                ml[(w * NH + i) * 8 + hr].x = f;
            }
            ml[i * 8 + hr].y = Q8 ? half_factor(top, rtop) : 1.f;
            ml[i * 8 + hr].z = sum;
            if (!whole) p.part_ml[slot * (8 * NH) + h] = make_float4(top, rtop, sum, 0.f);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < heads * D; e += kThreads) {
            const int h = e / D, d = e % D;
            const int i = h >> 3, hr = h & 7;
            float acc = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                acc += ml[(w * NH + i) * 8 + hr].x *
                       reinterpret_cast<const float *>(
                           smem + (w * S::kStages + last) * S::kTurn)
                           [i * S::kJoinHeads + d * 8 + (d >> 4) * S::kPad + hr];
            const float4 all = ml[i * 8 + hr];
            if (whole) {
                p.out[(int64_t)at.b * p.out_stride + (int64_t)(h0 + h) * D + d] =
                    to_output<Q8>(output_of<Q8>(acc, all.z, all.y));
            } else {
                p.part_o[((int64_t)slot * (8 * NH) + h) * D + d] = acc;
            }
        }
        fence_proxy_async_smem();  // the buffers' next writer is the TMA
        __syncthreads();           // and they are free for the next item
        first = false;
        at.next(p, HH, units);  // on to the next item of the share
    }
    if (!ok && lane == 0) {
        // Aborted: let every copy in flight land before shared memory goes away.
        volatile int no_abort = 0;
        const WaitCtl dc{kPagedDrainNs, p.err, &no_abort, kDevErrTimeout | kDevErrDrain};
        for (int i = fills > S::kStages ? fills - S::kStages : 0; i < fills; ++i)
            mbar_wait<false>(bars + 8 * (i % S::kStages), (uint32_t)(i / S::kStages) & 1u, dc);
    }
}

// Joins the partial results of the items that were cut between CTAs, and
// writes zeros for sequences without rows.  One block for each (query head,
// sequence): the parts' weights side by side, then a warp for every fourth part.
template <int D, bool Q8, class U>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(const PagedArgs p, int block_heads) {
    constexpr int kW = kJoinThreads / 32, E = D / 32;
    __shared__ float weight[kMaxWays];
    __shared__ float warp_m[kW], warp_r[kW], warp_l[kW];
    __shared__ float acc_w[kW][D];
    griddep_launch_dependents();
    griddep_wait();
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    __nv_bfloat16 *out = p.out + (int64_t)b * p.out_stride + (int64_t)h * D;
    const int units = U::of(seq_len(p, b, false));
    if (units == 0) {
        if (tid < D) out[tid] = __float2bfloat16(0.f);
        return;
    }
    const int HH = p.H * p.HB;
    const int kvh = h / p.G, hb = (h % p.G) / block_heads, hr = (h % p.G) % block_heads;
    const Split split(U::before(p, p.n_seq, false) * HH, p.ways);
    // the item's first place; its units are the last of its places
    const int i0 = U::before(p, b, false) * HH + (kvh * p.HB + hb) * (units + U::kExtra);
    const int w0 = split.of(i0 + U::kExtra), n = split.of(i0 + U::kExtra + units - 1) - w0 + 1;
    if (n == 1) return;  // one CTA held the whole item: it is written
    // the item lies in the first slot of its CTAs, but for one with units before it
    const int s0 = 2 * w0 + (split.begin(w0) < i0 ? 1 : 0);
    auto slot_of = [&](int i) { return (i == 0 ? s0 : 2 * (w0 + i)) * block_heads + hr; };
    float top = kLowest, rtop = kLowest;
    for (int i = tid; i < n; i += kJoinThreads) {
        const float4 ml = p.part_ml[slot_of(i)];
        top = fmaxf(top, ml.x);
        if (Q8) rtop = fmaxf(rtop, ml.y);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (Q8) rtop = fmaxf(rtop, __shfl_xor_sync(0xffffffffu, rtop, off));
    }
    if (lane == 0) {
        warp_m[warp] = top;
        if (Q8) warp_r[warp] = rtop;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        top = fmaxf(top, warp_m[w]);
        if (Q8) rtop = fmaxf(rtop, warp_r[w]);
    }
    float sum = 0.f;
    for (int i = tid; i < n; i += kJoinThreads) {
        const float4 ml = p.part_ml[slot_of(i)];
        const float f = exp2_fast(ml.x - top);
        weight[i] = f;
        sum += (Q8 ? exp2_fast(ml.y - rtop) : f) * ml.z;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) warp_l[warp] = sum;
    __syncthreads();
    float acc[E] = {};
    constexpr int kBatch = 8;  // loads in flight
    for (int at = warp; at < n; at += kW * kBatch) {
        float2 x[kBatch][E / 2];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = at + k * kW;
            const float *src = p.part_o + (int64_t)slot_of(min(i, n - 1)) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) x[k][e] = reinterpret_cast<const float2 *>(src)[e];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            // (behind the last part: 0 times 0, not times what was loaded, which may be infinite)
            const bool in = at + k * kW < n;
            const float f = in ? weight[at + k * kW] : 0.f;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                acc[2 * e] = fmaf(f, in ? x[k][e].x : 0.f, acc[2 * e]);
                acc[2 * e + 1] = fmaf(f, in ? x[k][e].y : 0.f, acc[2 * e + 1]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc_w[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (tid < D) {
        float a = 0.f;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            a += acc_w[w][tid];
            sum += warp_l[w];
        }
        out[tid] =
            to_output<Q8>(output_of<Q8>(a, sum, Q8 ? half_factor(top, rtop) : 1.f));
    }
}

int head_block(int G) { return G <= 8 ? 8 : 16; }

// Whether the tcgen05 kernel takes the call: 8-bit rows of 128 elements.  It reads faster but
// begins an item later, and its threads' work grows with the query heads of a kv head.
// Measured, here / there, in us, 8 kv heads: long tables (here in shares), one sequence of
// 16384 rows 16.9 / 14.7 (4 query heads a kv head) and 17.5 / 18.7 (8), of 131040 59.4 / 48.8
// and 60.2 / 53.1, 64 of 17 to 8192 114 / 94 and 120 / 113; short ones (an item a CTA), 64 of
// 300 rows 19.7 / 30.8 and 22.0 / 39.9, 64 of 1000 37.6 / 41.5 and 39.7 / 54.3, one of 300
// 9.1 / 10.8; 16 query heads, one of 131040 68.4 / 79.8 when it was tried (8 of them a turn
// there would read the cache twice).  The host knows how far the page table reaches, not
// the lengths.
bool on_tc(const KvCacheSpec &c, int G, int max_pages, int n_seq) {
    const int64_t rows = (int64_t)max_pages << c.log2_page;
    return c.e4m3 && c.D == 128 && G <= 8 && rows > 2048 &&
           (rows + TcUnits::kRows - 1) / TcUnits::kRows * n_seq * c.H >= 512;
}

template <int D, bool Q8, class U>
cudaError_t launch_join(const PagedArgs &a, int block_heads, const LaunchCtx &ctx) {
    count_launches(1);
    return launch_pdl(paged_join_kernel<D, Q8, U>, dim3((unsigned)(a.H * a.G), (unsigned)a.n_seq),
                      dim3(kJoinThreads), 0, ctx, a, block_heads);
}

template <int D, bool Q8, int NH>
cudaError_t launch(PagedArgs a, const KvCacheSpec &cache, const LaunchCtx &ctx) {
    using S = Shape<D, Q8, NH>;
    // the cache as (bytes of a row, in pairs; rows of a page; pages), 16 rows a box
    CUtensorMap mK, mV;
    const cuuint64_t rows = (cuuint64_t)cache.H << cache.log2_page;
    const cuuint64_t dims[3] = {S::RB / 2, rows, (cuuint64_t)cache.n_pages};
    const cuuint64_t strides[2] = {S::RB, rows * S::RB};
    const cuuint32_t box[3] = {S::SB / 2, 16, 1};
    if (!encode_tiled_bf16(&mK, 3, cache.k, dims, strides, box, S::SB) ||
        !encode_tiled_bf16(&mV, 3, cache.v, dims, strides, box, S::SB))
        return cudaErrorInvalidValue;
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
    const int most = std::min(kMaxWays, occ * ctx.num_sms);
    const int64_t items = (int64_t)a.n_seq * a.H * a.HB;
    const int64_t bytes = ((int64_t)a.max_pages << a.log2_page) * S::RB;
    const bool apart = bytes <= kApartBytes * (items >= most ? 4 : 4 * items >= most ? 2 : 1);
    a.ways = apart ? 0 : paged_ways(a, S::kUnit, most);
    count_launches(1);
    e = launch_pdl(kern, dim3((unsigned)(apart ? items : a.ways)), dim3(kThreads), S::kSmem, ctx,
                   mK, mV, a);
    if (e != cudaSuccess || apart) return e;
    return launch_join<D, Q8, typename S::U>(a, 8 * NH, ctx);
}

}  // namespace

int paged_ways(const PagedArgs &a, int rows, int most) {
    const int64_t len = (int64_t)a.max_pages << a.log2_page;
    const int64_t units = (len + rows - 1) / rows * a.n_seq * a.H * a.HB;
    return (int)std::max<int64_t>(1, std::min<int64_t>(units, most));
}

// The parts' references and sums, then their outputs.
size_t paged_attention_workspace(int Hq, int Hkv, int D) {
    const size_t rows = (size_t)2 * kMaxWays * head_block(Hq / Hkv);
    return rows * (D * sizeof(float) + sizeof(float4));
}

cudaError_t launch_paged_attention(const KvCacheSpec &c, const void *q, int64_t q_stride,
                                   const int32_t *lens, const int32_t *table, int max_pages,
                                   int n_seq, int Hq, float scale, void *out, int64_t out_stride,
                                   void *workspace, const LaunchCtx &ctx) {
    PagedArgs a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
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
    const size_t rows = (size_t)2 * kMaxWays * hb;
    a.ways = 0;
    a.part_ml = static_cast<float4 *>(workspace);
    a.part_o = reinterpret_cast<float *>(a.part_ml + rows);
    a.err = ctx.err;
    a.wait_ns = ctx.wait_ns;
    if (on_tc(c, a.G, max_pages, n_seq)) {
        int heads = 0;
        const cudaError_t e = launch_paged_tc(a, c, ctx, &heads);
        return e != cudaSuccess ? e : launch_join<128, true, TcUnits>(a, heads, ctx);
    }
    if (c.D == 64) {
        if (c.e4m3) return hb == 8 ? launch<64, true, 1>(a, c, ctx) : launch<64, true, 2>(a, c, ctx);
        return hb == 8 ? launch<64, false, 1>(a, c, ctx) : launch<64, false, 2>(a, c, ctx);
    }
    if (c.D == 128) {
        if (c.e4m3)
            return hb == 8 ? launch<128, true, 1>(a, c, ctx) : launch<128, true, 2>(a, c, ctx);
        return hb == 8 ? launch<128, false, 1>(a, c, ctx) : launch<128, false, 2>(a, c, ctx);
    }
    return cudaErrorInvalidValue;
}

}  // namespace wanvae
