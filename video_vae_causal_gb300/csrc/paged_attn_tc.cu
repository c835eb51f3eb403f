// paged_attn_tc.cu -- attention of one token over an 8-bit cache of 128-element
// heads on tcgen05 (the split and the join: paged_attn.cu).
//
// Reading the cache at HBM's rate leaves an SM about 1400 cycles for a unit of 128
// rows of one kv head (32 KB), too few to convert 8-bit elements for a 16-bit MMA
// in registers: that took about 470 warp instructions for every 16 rows, and was
// what bounded the kernel.  Here the tensor core reads the elements as TMA left
// them in shared memory (kind::f8f6f4), and the threads see scores and weights alone:
//   S[row, col]  = K[row, :] . Qt[col, :]     128 rows, 16 or 32 columns
//   Ot[d, col]  += sum_row V[row, d] Pt[col, row]
// Both other operands become several e4m3 terms, each in columns of its own:
//   a query, scaled by a power of two so that its largest element has exponent 7, is
//   a + b / 32, a the nearest e4m3 value and b what is left: exact for bf16's 8
//   bits down to 2^-14 of the largest element, within 2^-22 of it below;
//   a weight, times 2^7, is a + b / 16 + c / 256: within 2^-12 of it, or 2^-25 of the
//   largest weight where that is more (as fp16 would hold it).
// A key row's scale multiplies its score; a value row's scale 2^e joins the exponent
// of its weight, w = 2^(s + e - m), with m the running maximum of s + e, while the sum
// takes 2^(s - m) in fp32.  m moves only by more than 1, so weights stay below 2.
//
// Roles: warps 0-3 softmax and output (thread = cache row of a unit, then = element of
// O); warp 4 looks up pages, starts the loads (a queue of kStages units, which keeps
// 160 KB in flight) and lays out the next item's queries; warp 5 issues the MMAs, the
// scores of unit i + 1 before the product of unit i, so that softmax never waits for
// them.  What a unit is goes along with it in the queue, so only warp 4 knows the
// split.  Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "norm_act.cuh"
#include "paged_attn.cuh"

namespace wanvae {
namespace {

constexpr int kThreads = 192;
constexpr int kStages = 6;
constexpr int kUnit = kPagedTcUnit;
constexpr uint32_t kTileBytes = kUnit * 128;  // keys, or values, of a unit

// What the queue tells of a unit.
struct Unit {
    int b, head0, heads;  // sequence, first query head, heads of the item
    int rows;             // rows that count (the unit's first)
    uint32_t missing;     // groups of 16 rows whose page is not there
    int slot;             // of the partial result
    int flags;
    int pad;
};
enum : int { kFirst = 1, kLast = 2, kWhole = 4, kEnd = 8 };

// HP: query heads of an item, at most (4, 8 or 16).
template <int HP>
struct Cfg {
    static constexpr int N1 = 2 * HP < 16 ? 16 : 2 * HP;         // columns of S
    static constexpr int N2 = (3 * HP + 15) / 16 * 16;           // columns of O
    static constexpr uint32_t kP = kStages * 2 * kTileBytes;     // [2][N2][128 rows]
    static constexpr uint32_t kPBytes = N2 * 128;
    static constexpr uint32_t kQ = kP + 2 * kPBytes;             // [2][N1][128 elements]
    static constexpr uint32_t kQBytes = N1 * 128;
    static constexpr uint32_t kExp = kQ + 2 * kQBytes;           // [stages][2][128]
    static constexpr uint32_t kMeta = kExp + kStages * 256;
    static constexpr uint32_t kQs = kMeta + kStages * sizeof(Unit);  // [2][16] floats
    static constexpr uint32_t kRed = kQs + 128;                  // [2][4][16] floats
    static constexpr uint32_t kBars = kRed + 512;
    static constexpr uint32_t kSlots = kBars + 8 * (2 * kStages + 13);
    static constexpr uint32_t kSmem = 1024 + kSlots + 16;
    static constexpr uint32_t kTmemO = 64;  // S at columns 0 and 32, O behind
};

struct Bars {
    uint32_t base;
    __device__ uint32_t full(int s) const { return base + 8 * s; }
    __device__ uint32_t empty(int s) const { return base + 8 * (kStages + s); }
    __device__ uint32_t q_ready(int i) const { return base + 8 * (2 * kStages + i); }
    __device__ uint32_t q_free(int i) const { return base + 8 * (2 * kStages + 2 + i); }
    __device__ uint32_t s_full(int i) const { return base + 8 * (2 * kStages + 4 + i); }
    __device__ uint32_t s_free(int i) const { return base + 8 * (2 * kStages + 6 + i); }
    __device__ uint32_t p_full(int i) const { return base + 8 * (2 * kStages + 8 + i); }
    __device__ uint32_t pv_done(int i) const { return base + 8 * (2 * kStages + 10 + i); }
    __device__ uint32_t drain() const { return base + 8 * (2 * kStages + 12); }
};

// A place in a ring of n, and the parity of its turn.
template <int n>
struct Turn {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == n) {
            i = 0;
            phase ^= 1u;
        }
    }
};

// kind::f8f6f4, e4m3 in, fp32 out; A [K][M] (bit 15) for O = V^T P^T.
__device__ __forceinline__ constexpr uint32_t idesc_e4m3(int N, bool a_rows) {
    return (1u << 4) | (a_rows ? 1u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 columns of TMEM, without the wait.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
template <int n>
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[n]) {
#pragma unroll
    for (int c = 0; c < n; c += 16) tmem_ld16_async(taddr + c, r + c);
#pragma unroll
    for (int c = 0; c < n; c += 16) tmem_ld_wait16(r + c);
}
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void bar_softmax() {
    asm volatile("bar.sync 1, 128;" ::: "memory");
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w) {
    const uint32_t h = e4m3x2_to_f16x2(w);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Warp 4: units into the queue, range after range.
template <int HP>
__device__ void feed(const CUtensorMap *mK, const CUtensorMap *mV, const PagedArgs &p,
                     int log2_box, uint8_t *smem, const Bars &bars, const WaitCtl &wc) {
    using C = Cfg<HP>;
    const int lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    const int HH = p.H * p.HB;
    const int total = units_before<kUnit>(p, p.n_seq, blockIdx.x == 0) * HH;
    const Split split(total, p.ways, p.taken != nullptr);
    Unit *queue = reinterpret_cast<Unit *>(smem + C::kMeta);
    Turn<kStages> put;
    Turn<2> item;
    int fills = 0;
    bool ok = true;
    int range = (int)blockIdx.x < split.ways && total > 0 ? split.own(blockIdx.x) : split.ranges;
    while (ok && range < split.ranges) {
        int left = split.begin(range + 1) - split.begin(range);
        Cursor<kUnit> at = locate<kUnit>(p, HH, split.begin(range));
        bool first_item = true, starts = true, whole = false;
        // the page of box `lane` of the unit to come
        const int boxes = kUnit >> log2_box;
        auto find_page = [&]() -> int {
            const int tok = at.u * kUnit + (lane << log2_box);
            if (lane >= boxes || tok >= at.len) return -2;
            return __ldg(p.table + (int64_t)at.b * p.max_pages + (tok >> p.log2_page));
        };
        int page = find_page();
        while (left > 0) {
            const int kvh = at.hh / p.HB, head0 = kvh * p.G + (at.hh - kvh * p.HB) * HP;
            const int heads = min(HP, (kvh + 1) * p.G - head0);
            if (starts) whole = at.u == 0 && at.U <= left;  // the range holds the item
            ok = mbar_wait_warp<false>(bars.empty(put.i), put.phase ^ 1u, wc);
            if (!ok) break;
            const bool wanted = page != -2, there = (unsigned)page < (unsigned)p.n_pages;
            if (wanted && !there) atomicOr(p.err, kDevErrAlign);
            const uint32_t gone = __ballot_sync(0xffffffffu, wanted && !there);
            const int loads = __popc(__ballot_sync(0xffffffffu, there));
            if (lane == 0) {
                Unit u;
                u.b = at.b;
                u.head0 = head0;
                u.heads = heads;
                u.rows = min(at.len - at.u * kUnit, kUnit);
                u.missing = gone;
                u.slot = (2 * range + (first_item ? 0 : 1)) * HP;
                u.flags = (starts ? kFirst : 0) | (at.u + 1 == at.U || left == 1 ? kLast : 0) |
                          (whole ? kWhole : 0);
                u.pad = 0;
                queue[put.i] = u;
                mbar_arrive_expect_tx(bars.full(put.i), (uint32_t)loads * (258u << log2_box));
            }
            __syncwarp();
            if (there) {
                const int row = (kvh << p.log2_page) +
                                ((at.u * kUnit + (lane << log2_box)) & ((1 << p.log2_page) - 1));
                const uint32_t dst = sbase + put.i * 2 * kTileBytes + ((uint32_t)lane << (log2_box + 7));
                const uint32_t ex = sbase + C::kExp + put.i * 256 + (lane << log2_box);
                const uint32_t bar = bars.full(put.i);
                tma_load_3d(dst, mK, bar, 0, row, page);
                tma_load_3d(dst + kTileBytes, mV, bar, 0, row, page);
                const int64_t at_row = (((int64_t)page * p.H) << p.log2_page) + row;
                bulk_load(ex, p.k_exp + at_row, 1u << log2_box, bar);
                bulk_load(ex + 128, p.v_exp + at_row, 1u << log2_box, bar);
            }
            ++fills;
            put.next();
            if (starts) {
                // the item's queries, as e4m3 terms: rows h and HP + h of its buffer
                uint2 raw[HP];
                const __nv_bfloat16 *src =
                    p.q + (int64_t)at.b * p.q_stride + (int64_t)head0 * 128 + lane * 4;
#pragma unroll
                for (int h = 0; h < HP; ++h)
                    raw[h] = h < heads ? __ldg(reinterpret_cast<const uint2 *>(src + h * 128))
                                       : make_uint2(0u, 0u);
                ok = mbar_wait_warp<false>(bars.q_free(item.i), item.phase ^ 1u, wc);
                if (!ok) break;
                uint8_t *dst = smem + C::kQ + item.i * C::kQBytes;
                float *qs = reinterpret_cast<float *>(smem + C::kQs) + item.i * 16;
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    uint32_t amax = max(max(raw[h].x & 0x7fffu, (raw[h].x >> 16) & 0x7fffu),
                                        max(raw[h].y & 0x7fffu, (raw[h].y >> 16) & 0x7fffu));
                    amax = __reduce_max_sync(0xffffffffu, amax);
                    // 2^(7 - exponent of the largest); both powers stay in fp32's range
                    const int ex = min(max((int)(amax >> 7), 8), 254) - 127 - 7;
                    const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
                    const float x[4] = {nact_lo(raw[h].x) * down, nact_hi(raw[h].x) * down,
                                        nact_lo(raw[h].y) * down, nact_hi(raw[h].y) * down};
                    const uint32_t a = f32x2_to_e4m3x2(x[0], x[1]), b = f32x2_to_e4m3x2(x[2], x[3]);
                    const float2 ya = e4m3x2_to_f32(a), yb = e4m3x2_to_f32(b);
                    const uint32_t ra = f32x2_to_e4m3x2(32.f * (x[0] - ya.x), 32.f * (x[1] - ya.y));
                    const uint32_t rb = f32x2_to_e4m3x2(32.f * (x[2] - yb.x), 32.f * (x[3] - yb.y));
                    auto place = [&](int n) {
                        return dst + n * 128 + (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4;
                    };
                    *reinterpret_cast<uint32_t *>(place(h)) = a | (b << 16);
                    *reinterpret_cast<uint32_t *>(place(HP + h)) = ra | (rb << 16);
                    if (lane == 0)  // (a query that is not finite has no scores)
                        qs[h] = amax >= 0x7f80u ? __uint_as_float(0x7fc00000u)
                                                : p.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.q_ready(item.i));
                item.next();
                starts = false;
            }
            if (--left > 0) {
                if (at.next(p, HH)) {
                    starts = true;
                    first_item = false;
                }
                page = find_page();
            }
        }
        if (!ok) break;
        range = split.ranges;
        if (split.small) {
            if (lane == 0) range = split.taken(atomicAdd(p.taken, 1));
            range = __shfl_sync(0xffffffffu, range, 0);
        }
    }
    if (ok) ok = mbar_wait_warp<false>(bars.empty(put.i), put.phase ^ 1u, wc);
    if (ok) {
        if (lane == 0) {
            queue[put.i].flags = kEnd;
            mbar_arrive(bars.full(put.i));
        }
    } else if (lane == 0) {
        // Aborted: let every copy in flight land before shared memory goes away.
        volatile int no_abort = 0;
        const WaitCtl dc{kPagedDrainNs, wc.err, &no_abort, kDevErrTimeout | kDevErrDrain};
        for (int i = fills > kStages ? fills - kStages : 0; i < fills; ++i)
            mbar_wait<false>(bars.full(i % kStages), (uint32_t)(i / kStages) & 1u, dc);
    }
}

// Warp 5, one thread: the MMAs.
template <int HP>
__device__ void issue(uint8_t *smem, uint32_t tmem, const Bars &bars, const WaitCtl &wc) {
    using C = Cfg<HP>;
    const uint32_t sbase = smem_u32(smem);
    const Unit *queue = reinterpret_cast<const Unit *>(smem + C::kMeta);
    const uint32_t id_s = idesc_e4m3(C::N1, false), id_o = idesc_e4m3(C::N2, true);
    const uint64_t k0 = sdesc_kmajor(sbase, 128u, kLayoutSw128);
    const uint64_t v0 = sdesc_rows_sw128(sbase + kTileBytes, kTileBytes);
    const uint64_t q0 = sdesc_kmajor(sbase + C::kQ, 128u, kLayoutSw128);
    const uint64_t p0 = sdesc_kmajor(sbase + C::kP, 128u, kLayoutSw128);
    Turn<kStages> get;
    Turn<2> item, buf, last_buf;
    int last_stage = -1, last_first = 0;
    bool ok = true;
    auto product = [&]() -> bool {  // of the unit before
        if (!mbar_wait<false>(bars.p_full(last_buf.i), last_buf.phase, wc)) return false;
        tc_fence_after();
        const uint64_t a = v0 + (uint32_t)last_stage * (2 * kTileBytes >> 4);
        const uint64_t b = p0 + (uint32_t)last_buf.i * (C::kPBytes >> 4);
#pragma unroll
        for (int k = 0; k < kUnit / 32; ++k)
            mma_e4m3_ss(tmem + C::kTmemO, a + k * (32 * 128 >> 4), b + k * 2, id_o,
                        !last_first || k > 0);
        mma_commit(bars.empty(last_stage));
        mma_commit(bars.pv_done(last_buf.i));
        last_buf.next();
        return true;
    };
    while (true) {
        ok = mbar_wait<false>(bars.full(get.i), get.phase, wc);
        if (!ok) break;
        const int flags = queue[get.i].flags;
        if (flags & kEnd) {
            if (last_stage >= 0) ok = product();
            break;
        }
        if (flags & kFirst) ok = mbar_wait<false>(bars.q_ready(item.i), item.phase, wc);
        ok = ok && mbar_wait<false>(bars.s_free(buf.i), buf.phase ^ 1u, wc);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = k0 + (uint32_t)get.i * (2 * kTileBytes >> 4);
        const uint64_t b = q0 + (uint32_t)item.i * (C::kQBytes >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_e4m3_ss(tmem + 32u * buf.i, a + k * 2, b + k * 2, id_s, k > 0);
        mma_commit(bars.s_full(buf.i));
        if (flags & kLast) {
            mma_commit(bars.q_free(item.i));
            item.next();
        }
        if (last_stage >= 0) ok = product();
        if (!ok) break;
        last_stage = get.i;
        last_first = flags & kFirst;
        buf.next();
        get.next();
    }
    // Every MMA issued above completes before TMEM is released.
    volatile int no_abort = 0;
    const WaitCtl dc{kPagedDrainNs, wc.err, &no_abort, kDevErrTimeout | kDevErrDrain};
    mma_commit(bars.drain());
    mbar_wait<false>(bars.drain(), 0u, dc);
}

// Warps 0-3.  Thread r: row r of a unit, and element r of the outputs.  A warp
// whose wait runs out does no more work, but keeps to the barriers until all four
// learn of it and leave together.
template <int HP>
__device__ void softmax(const PagedArgs &p, uint8_t *smem, uint32_t tmem, const Bars &bars,
                        const WaitCtl &wc) {
    using C = Cfg<HP>;
    const int r = threadIdx.x, warp = r >> 5, lane = r & 31;
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const Unit *queue = reinterpret_cast<const Unit *>(smem + C::kMeta);
    float *red = reinterpret_cast<float *>(smem + C::kRed);
    // the place of this row in P's rows n (128-byte swizzle)
    uint32_t place[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) place[n] = n * 128 + (((r >> 4) ^ n) << 4) + (r & 15);
    Turn<kStages> get;
    Turn<2> item, buf;
    float qs[HP], m[HP], l[HP], s[HP];
#pragma unroll
    for (int h = 0; h < HP; ++h) qs[h] = m[h] = l[h] = s[h] = 0.f;
    bool ok = true;
    while (true) {
        ok = ok && mbar_wait_warp<false>(bars.full(get.i), get.phase, wc);
        Unit u = {0, 0, 0, 0, 0u, 0, 0, 0};
        if (ok) u = queue[get.i];
        const bool end = (u.flags & kEnd) != 0;
        float ve = 0.f;
        bool there = false, moves = false;
        if (ok && !end) {
            if (u.flags & kFirst) {
                ok = mbar_wait_warp<false>(bars.q_ready(item.i), item.phase, wc);
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    qs[h] = reinterpret_cast<const float *>(smem + C::kQs)[item.i * 16 + h];
                    m[h] = -INFINITY;
                    l[h] = 0.f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.q_free(item.i));
                item.next();
            }
            ok = ok && mbar_wait_warp<false>(bars.s_full(buf.i), buf.phase, wc);
        }
        if (ok && !end) {
            const uint8_t *ex = smem + C::kExp + get.i * 256 + r;
            const float kf = __uint_as_float((uint32_t)ex[0] << 23);
            ve = (float)ex[128] - 127.f;
            there = r < u.rows && !((u.missing >> (r >> p.log2_page)) & 1u);
            tc_fence_after();
            uint32_t raw[C::N1];
            tmem_read(trow + 32u * buf.i, raw);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.s_free(buf.i));
            // scores in log2 units
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                const float x = fmaf(__uint_as_float(raw[HP + h]), 0.03125f, __uint_as_float(raw[h]));
                s[h] = there ? x * (qs[h] * kf) : -INFINITY;
                moves |= s[h] + ve > m[h] + 1.f;
            }
        }
        if (bar_any(1, 128, moves || !ok)) {
            if (bar_any(1, 128, !ok)) return;
            if (!end) {
                float f[HP];
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    const float top = warp_max(s[h] + ve);
                    if (lane == 0) red[warp * 16 + h] = top;
                }
                bar_softmax();
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    float mn = m[h];
#pragma unroll
                    for (int w = 0; w < 4; ++w) mn = fmaxf(mn, red[w * 16 + h]);
                    f[h] = mn == -INFINITY ? 0.f : exp2_fast(m[h] - mn);
                    m[h] = mn;
                    l[h] *= f[h];
                }
                if (!(u.flags & kFirst)) {
                    // O is whole once the product of the unit before is done
                    ok = mbar_wait_warp<false>(bars.pv_done(buf.i ^ 1),
                                               buf.i ? buf.phase : buf.phase ^ 1u, wc);
                    tc_fence_after();
                    uint32_t o[C::N2];
                    tmem_read(trow + C::kTmemO, o);
#pragma unroll
                    for (int c = 0; c < C::N2; ++c)
                        if (c < 3 * HP) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c % HP]);
#pragma unroll
                    for (int c = 0; c < C::N2; c += 16)
                        tmem_st16_async(trow + C::kTmemO + c, o + c);
                    tmem_st_wait();
                    tc_fence_before();
                }
            }
        }
        if (end) return;
        // weights, times 2^7, as three terms; P's buffer is free once the product of
        // the unit before the last is done
        ok = ok && mbar_wait_warp<false>(bars.pv_done(buf.i), buf.phase ^ 1u, wc);
        uint8_t *pb = smem + C::kP + buf.i * C::kPBytes;
#pragma unroll
        for (int h = 0; h < HP; h += 2) {
            float x[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float ms = m[h + c] == -INFINITY ? 0.f : m[h + c];
                const float y = s[h + c] - ms;
                l[h + c] += exp2_fast(y);
                x[c] = exp2_fast(y + (ve + 7.f));
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t a = f32x2_to_e4m3x2(x[0], x[1]);
                pb[(k * HP + h) / 8 * 1024 + place[(k * HP + h) & 7]] = (uint8_t)a;
                pb[(k * HP + h) / 8 * 1024 + place[(k * HP + h + 1) & 7]] = (uint8_t)(a >> 8);
                if (k < 2) {
                    const float2 y = e4m3x2_to_f32(a);
                    x[0] = 16.f * (x[0] - y.x);
                    x[1] = 16.f * (x[1] - y.y);
                }
            }
        }
        if (!there) {  // what lies in a row that does not count may be anything
            uint4 *v = reinterpret_cast<uint4 *>(smem + get.i * 2 * kTileBytes + kTileBytes + r * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();  // P and V are read by the tensor core (async proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.p_full(buf.i));
        if (u.flags & kLast) {
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                float t = l[h];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
                if (lane == 0) red[64 + warp * 16 + h] = t;
            }
            ok = ok && mbar_wait_warp<false>(bars.pv_done(buf.i), buf.phase, wc);
            tc_fence_after();
            uint32_t o[C::N2];
            tmem_read(trow + C::kTmemO, o);
            tc_fence_before();
            bar_softmax();
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                if (h >= u.heads || !ok) break;
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) sum += red[64 + w * 16 + h];
                const float x = 0.0078125f *
                                fmaf(fmaf(__uint_as_float(o[2 * HP + h]), 0.0625f,
                                          __uint_as_float(o[HP + h])),
                                     0.0625f, __uint_as_float(o[h]));
                if (u.flags & kWhole) {
                    p.out[(int64_t)u.b * p.out_stride + (int64_t)(u.head0 + h) * 128 + r] =
                        __float2bfloat16(sum > 0.f || sum != sum ? x / sum : 0.f);
                } else {
                    p.part_o[(int64_t)(u.slot + h) * 128 + r] = x;
                    if (r == 0) p.part_ml[u.slot + h] = make_float2(m[h], sum);
                }
            }
            bar_softmax();  // the sums are read
        }
        buf.next();
        get.next();
    }
}

template <int HP>
__global__ void __launch_bounds__(kThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                const PagedArgs p, int log2_box) {
    using C = Cfg<HP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const Bars bars{smem_u32(smem) + C::kBars};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kSlots);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kSlots + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bars.full(s), 1);
            mbar_init(bars.empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.q_ready(i), 1);
            mbar_init(bars.q_free(i), 5);  // the MMAs that read it, and four warps
            mbar_init(bars.s_full(i), 1);
            mbar_init(bars.s_free(i), 4);
            mbar_init(bars.p_full(i), 4);
            mbar_init(bars.pv_done(i), 1);
        }
        mbar_init(bars.drain(), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mK);
        tma_prefetch_desc(&mV);
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(tmem_slot), 128u);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{p.wait_ns, p.err, abort_flag, 0u};
    griddep_wait();
    if (warp < 4) {
        softmax<HP>(p, smem, tmem, bars, wc);
    } else if (warp == 4) {
        feed<HP>(&mK, &mV, p, log2_box, smem, bars, wc);
    } else if ((threadIdx.x & 31) == 0) {
        issue<HP>(smem, tmem, bars, wc);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, 128u);
}

template <int HP>
cudaError_t launch(PagedArgs &a, const KvCacheSpec &cache, const LaunchCtx &ctx) {
    using C = Cfg<HP>;
    static_assert(C::kSmem <= 227 * 1024, "shared memory");
    static_assert(C::N1 <= 32 && C::kTmemO + C::N2 <= 128, "TMEM");
    const int log2_box = std::min(cache.log2_page, 7);
    CUtensorMap mK, mV;
    const cuuint64_t rows = (cuuint64_t)cache.H << cache.log2_page;
    const cuuint64_t dims[3] = {64, rows, (cuuint64_t)cache.n_pages};
    const cuuint64_t strides[2] = {128, rows * 128};
    const cuuint32_t box[3] = {64, 1u << log2_box, 1};
    if (!encode_tiled_bf16(&mK, 3, cache.k, dims, strides, box, 128) ||
        !encode_tiled_bf16(&mV, 3, cache.v, dims, strides, box, 128))
        return cudaErrorInvalidValue;
    constexpr int kMaxDev = 64;
    static std::atomic<bool> attr_set[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(paged_tc_kernel<HP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    const bool takes = paged_ways(a, kUnit, std::min(kMaxWays, ctx.num_sms));
    count_launches(takes ? 3 : 2);
    if (takes) {
        e = launch_paged_begin(a, ctx);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(paged_tc_kernel<HP>, dim3((unsigned)a.ways), dim3(kThreads), C::kSmem, ctx,
                      mK, mV, a, log2_box);
}

}  // namespace

cudaError_t launch_paged_tc(PagedArgs &a, const KvCacheSpec &cache, const LaunchCtx &ctx,
                            int *block_heads) {
    const int hp = a.G <= 4 ? 4 : a.G <= 8 ? 8 : 16;
    a.HB = (a.G + hp - 1) / hp;
    *block_heads = hp;
    if (hp == 4) return launch<4>(a, cache, ctx);
    if (hp == 8) return launch<8>(a, cache, ctx);
    return launch<16>(a, cache, ctx);
}

}  // namespace wanvae
