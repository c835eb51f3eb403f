// paged_attn_tc.cu -- attention of one token over an 8-bit cache of 128-element
// heads, or a 4-bit one, on tcgen05 (the split and the join: paged_attn.cu).
//
// Reading the cache at HBM's rate leaves an SM about 1400 cycles for 128 rows of one kv
// head (32 KB), too few to convert 8-bit elements for a 16-bit MMA in registers: that
// took about 470 warp instructions for every 16 rows, and was what bounded the
// kernel.  Here the tensor core reads the elements as TMA left them in shared memory
// (kind::f8f6f4), and the threads see scores and weights alone:
//   S[row, col]  = K[row, :] . Qt[col, :]     128 rows, 16 columns
//   Ot[d, col]  += sum_row V[row, d] Pt[col, row]
// Both other operands become several e4m3 terms, each in columns of its own (the weights'
// columns lie together for each row, so that a row's are one or two 16-byte stores):
//   a query, scaled by a power of two so that its largest element has exponent 7, is
//   a + b / 32, a the nearest e4m3 value and b what is left: exact for bf16's 8
//   bits down to 2^-14 of the largest element, within 2^-22 of it below;
//   a weight, times 2^7, is a + b / 16 + c / 256: within 2^-12 of it, or 2^-25 of the
//   largest weight where that is more (as fp16 would hold it).
// A key row's scale multiplies its score; a value row's scale 2^e joins the exponent
// of its weight, w = 2^(s + e - m), with m the running maximum of s + e, while the sum
// takes 2^(s - r) in fp32, r that of s alone (see paged_attn.cuh).  m moves only by more
// than 1, so weights stay below 2; rows of zeros do not move it.
//
// A unit is 256 rows, two MMAs' worth: each role's waits and bookkeeping take it about
// 1000 cycles a unit, whatever its size.
//
// Roles: warps 0-3 and 4-7 softmax and output, two groups that take turns (thread = two
// cache rows of a unit, then = element of O), since a unit's chain of dependent
// instructions is longer than its share of HBM.  Each group has its own m, sum and
// O; where an item ends they are joined.  Warp 8 looks up pages, starts the loads of
// keys and lays out the next item's queries; warp 11 starts the loads of scales and values
// (a TMA instruction takes its lanes one after another, about 100 cycles each); warp 9
// issues the MMAs of the scores, up to four units ahead of the products, which warp 10
// issues.  Keys' places are free once their scores are done, values are waited for
// where the product needs them, not before, so that most of the queue's bytes are in
// flight.  What a unit is goes along with it in the queue, so only warp 8 knows the
// split.  Every wait is bounded.
//
// Rows of 4 bits become rows of e4m3 elements on their way, exactly (seq_dev.cuh): TMA
// leaves a unit's packed rows in a queue of their own, and eight more warps look their
// elements up, eight to seven instructions: 12-15 write keys to TMEM, where the
// scores' MMA takes them from, 16-19 values to shared memory.  (Both through shared
// memory would move 768 bytes of it for each row of 136, more than it has in the time that
// HBM takes for the row; so it is 512.)  The rest of the kernel sees rows of 8 bits
// with scales 2^6 smaller.  Values of 64-element heads lie in rows of 128 with zeros behind
// them: the MMA's 128 rows of O^T take the same time half empty.
//
// What bounds it: HBM, behind what each item costs besides its units.  64 sequences of 17
// to 8192 rows, 8 kv heads of 4 query heads: 94 us (5.7 TB/s, 0.84 of the measured copy
// rate); one of 131040 rows, 8 heads of 8: 50 us (5.4 TB/s, 0.80; about 8 us of it
// the launches, the first loads' latency and the join).
//
// Over 4 bits, the look-up's instructions and the chain from one role to the next: the batch takes
// 90 us (3.2 TB/s, 0.48), the one sequence 55 (2.7 TB/s, 0.40), with 0.56 instructions issued a
// quarter of an SM and cycle, half of them for the look-up, and the longest waits those for
// barriers and TMEM.  Without the look-up's arithmetic (timing alone) they take 74 and 44, without
// the softmax's 89 and 52.
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

constexpr int kUnit = TcUnits::kRows, kHalves = kUnit / 128;
constexpr uint32_t kHalfBytes = 128 * 128;              // 128 rows of keys, or values
constexpr uint32_t kTileBytes = kHalves * kHalfBytes;   // of a unit
constexpr int kBoxes = kUnit / 16;                      // boxes of a unit, at most

// mbar_wait_warp with all but the first look out of line.  A role's code for a unit is
// walked through by one or two warps of a scheduler: beyond what its instruction cache
// holds, they wait for instructions (with every wait's loop in line, and both halves
// of a unit unrolled, that was most of a unit's time).
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                         unsigned *err, volatile int *abort) {
    return mbar_wait_warp<false>(bar, parity, WaitCtl{limit_ns, err, abort, 0u});
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, const WaitCtl &wc) {
    if (wc.limit_ns != 0 && __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_longer(bar, parity, wc.limit_ns, wc.err, wc.abort);
}

// What the queue tells of a unit.
struct Unit {
    int b, head0, heads;  // sequence, first query head, heads of the item
    int rows;             // rows that count (the unit's first)
    uint32_t missing;     // boxes whose page is not there
    int slot;             // of the partial result
    int flags;
    int item;             // number of the item in this CTA
};
// The item's first two units (each group's first), its last two (each group's last;
// kLast alone where it has one), whether a range holds it whole, the end of all.
enum : int { kFirst = 1, kSecond = 2, kLast = 4, kLastBut1 = 8, kWhole = 16, kEnd = 32 };

// How far a score may pass m in one unit, over 4 bits, without the sum's reference r moving too
// (2^31 rows of 2^(kSumLag + kStep) stay in fp32's range).
constexpr float kStep = 30.f;

// What a softmax warp keeps for the heads of its item, in shared memory (own[kind + head]):
// the queries' factors; the largest s + e where m moves; m and r (paged_attn.cuh; m is the
// group's, r the warp's); the factors that O and the sums go on with; the sum at the item's
// end and its r.  (Other warps read the fourth kind no more: a warp may have begun the next item.)
enum : int { kOwnQs = 0, kOwnTop = 8, kOwnM = 16, kOwnR = 24, kOwnF = 32, kOwnFl = 40, kOwnL = 48,
             kOwnRl = 56, kOwnSize = 64 };

// HP: query heads of an item, at most (4 or 8: a thread's work grows with them, and
// with 8 in place of 4 the batch above takes 108 us instead of 94).  Q4: rows of 4 bits.
// (Sixteen warps that unpack, with 72 registers a thread, in place of eight: 94 us for 90.)
template <int HP_, int D_, bool Q4_>
struct Cfg {
    static constexpr int HP = HP_, D = D_;
    static constexpr bool Q4 = Q4_;
    static constexpr int kThreads = Q4 ? 640 : 384;
    static constexpr int N1 = 2 * HP < 16 ? 16 : 2 * HP;         // columns of S
    static constexpr int N2 = (3 * HP + 15) / 16 * 16;           // columns of O
    // Places for keys, which the scores free, and for values and what is told of a
    // unit, which the products free.  Of 4 bits: places for packed keys and values, which
    // the warps that unpack them free; two for values unpacked; and more for what is
    // told of a unit.
    static constexpr int kKeys = Q4 ? 3 : 2, kStages = Q4 ? 8 : 4, kValues = Q4 ? 2 : kStages;
    static constexpr int kRawValues = Q4 ? 4 : 0;
    static constexpr int kRowBytes = kv_row_bytes(Q4 ? kKvE2M1 : kKvE4M3, D);
    // How far m is set above the largest s + e where it moves (4 bits), so that the next
    // units' a little larger ones do not move it again, at the price of the weights' two
    // lowest bits (64 sequences 103 -> 99 us, one of 131040 rows 63.4 -> 60.5 when it was tried;
    // a move takes a group some three units' time).
    static constexpr float kAhead = Q4 ? 2.f : 0.f;
    static constexpr uint32_t kRawBytes = kUnit * kRowBytes;     // keys, or values, as they come
    static constexpr uint32_t kV = (kKeys + kRawValues) * kRawBytes;
    static constexpr uint32_t kP = kV + kValues * kTileBytes;    // [groups][halves][N2 / 16][128 rows][16]
    static constexpr uint32_t kPBytes = N2 * 128;
    static constexpr uint32_t kQ = kP + 2 * kHalves * kPBytes;   // [2][N1][128 elements]
    static constexpr uint32_t kQBytes = N1 * 128;
    static constexpr uint32_t kExp = kQ + 2 * kQBytes;           // [stages][2][rows]
    static constexpr uint32_t kOffBytes = Q4 ? kUnit * kv_off_bytes(D) : 0;
    static constexpr uint32_t kOff = kExp + kStages * 2 * kUnit;  // [stages][2][rows] offsets
    static constexpr uint32_t kTable = kOff + kStages * 2 * kOffBytes;  // [16] of 8 bytes
    static constexpr uint32_t kMeta = kTable + (Q4 ? 128 : 0);
    static constexpr uint32_t kPages = kMeta + kStages * sizeof(Unit);  // [stages][page, row]
    static constexpr uint32_t kQs = kPages + kStages * kBoxes * 8;  // [2][16] floats
    static constexpr uint32_t kOwn = kQs + 128;                  // [8 warps][kOwnSize] floats
    static constexpr uint32_t kJoin = kOwn + 8 * kOwnSize * 4;         // [HP][128], [HP][m, r, sum, -]
    static constexpr uint32_t kBars = kJoin + HP * 132 * 4;
    static constexpr uint32_t kSlots = kBars + 8 * (2 * kKeys + 4 * kStages + 20 + 2 * kRawValues + 6);
    static constexpr uint32_t kSmem = 1024 + kSlots + 16;
    // TMEM: S of half h of units i % 4 at columns 64 (i % 4) + 32 h, then each group's O,
    // then keys unpacked, of units i % 2 at 64 (i % 2) + 32 h
    static __device__ __forceinline__ uint32_t s_col(int i) { return 64u * i; }
    static __device__ __forceinline__ uint32_t o_col(int w) { return 256u + 48u * w; }
    static __device__ __forceinline__ uint32_t k_col(int i) { return 352u + 64u * i; }
    // Places of packed keys and values.
    static __device__ __forceinline__ uint32_t raw_key(int i) { return i * kRawBytes; }
    static __device__ __forceinline__ uint32_t raw_value(int i) { return (kKeys + i) * kRawBytes; }
};

template <class C>
struct Bars {
    static constexpr int kKeys = C::kKeys, kStages = C::kStages;
    uint32_t base;
    __device__ uint32_t at(int i) const { return base + 8 * i; }
    __device__ uint32_t k_full(int s) const { return at(s); }
    __device__ uint32_t k_empty(int s) const { return at(kKeys + s); }
    __device__ uint32_t v_full(int s) const { return at(2 * kKeys + s); }
    __device__ uint32_t v_empty(int s) const { return at(2 * kKeys + kStages + s); }
    __device__ uint32_t posted(int s) const { return at(2 * kKeys + 2 * kStages + s); }
    __device__ uint32_t told(int s) const { return at(2 * kKeys + 3 * kStages + s); }
    __device__ uint32_t more(int i) const { return at(2 * kKeys + 4 * kStages + i); }
    __device__ uint32_t q_ready(int i) const { return more(i); }
    __device__ uint32_t q_free(int i) const { return more(2 + i); }
    __device__ uint32_t s_full(int i) const { return more(4 + i); }
    __device__ uint32_t s_free(int i) const { return more(8 + i); }
    __device__ uint32_t p_full(int w) const { return more(12 + w); }
    __device__ uint32_t pv_done(int w) const { return more(14 + w); }
    __device__ uint32_t join_full() const { return more(16); }
    __device__ uint32_t join_free() const { return more(17); }
    __device__ uint32_t drain(int i) const { return more(18 + i); }
    // 4 bits: keys and values unpacked, and read; packed values are there, and unpacked
    __device__ uint32_t kt_full(int i) const { return more(20 + i); }
    __device__ uint32_t kt_empty(int i) const { return more(22 + i); }
    __device__ uint32_t vt_empty(int i) const { return more(24 + i); }
    __device__ uint32_t raw_full(int s) const { return more(26 + s); }
    __device__ uint32_t raw_empty(int s) const { return more(26 + C::kRawValues + s); }
};

// A place in a ring of n, and the parity of its turn.
template <int n>
struct Turn {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int by = 1) {
        i += by;
        if (i >= n) {
            i -= n;
            phase ^= 1u;
        }
    }
};

// kind::f8f6f4, e4m3 in, fp32 out; by rows: A [K][M] (bit 15) and B [K][N] (bit 16), for
// O = V^T P^T.
__device__ __forceinline__ constexpr uint32_t idesc_e4m3(int N, bool rows) {
    return (1u << 4) | (rows ? 3u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
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

// The same with A [128][K] in TMEM (lane = row, four elements a 32-bit column).
__device__ __forceinline__ void mma_e4m3_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
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

__device__ __forceinline__ void tmem_st8_async(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

__device__ __forceinline__ void bar_group(int w) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory");
}

// The largest of a warp (a NaN loses to a number).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w) {
    const uint32_t h = e4m3x2_to_f16x2(w);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Two fp32 values as fp16, two fp16 ones as e4m3 (each to nearest, ties to even), and 16 (y - a),
// which is exact where a is y rounded to e4m3.
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t y) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(y));
    return r;
}
__device__ __forceinline__ uint32_t times16_less(uint32_t y, uint32_t a) {
    const __half2 d = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&y),
                                      *reinterpret_cast<const __half2 *>(&a)),
                              __float2half2_rn(16.f));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// 8 bytes of global memory to shared memory, and this thread's arrival on `bar` once
// its copies so far are done.
__device__ __forceinline__ void copy8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

// Aborted: lets every copy in flight land before shared memory goes away.
template <class C>
__device__ __forceinline__ void drain_loads(int fills, const Bars<C> &bars, bool values,
                                            const WaitCtl &wc) {
    volatile int no_abort = 0;
    const WaitCtl dc{kPagedDrainNs, wc.err, &no_abort, kDevErrTimeout | kDevErrDrain};
    const int n = !values ? C::kKeys : C::Q4 ? C::kRawValues : C::kStages;
    for (int i = fills > n ? fills - n : 0; i < fills; ++i)
        mbar_wait<false>(!values ? bars.k_full(i % n)
                         : C::Q4 ? bars.raw_full(i % n)
                                 : bars.v_full(i % n),
                         (uint32_t)(i / n) & 1u, dc);
}

// Warp 8: the share's units into the queue (their keys; the rest is warp 11's).
template <class C>
__device__ void feed(const CUtensorMap *mK, const PagedArgs &p, int log2_box,
                     uint8_t *smem, const Bars<C> &bars, const WaitCtl &wc) {
    constexpr int HP = C::HP, kLog2Row = C::kRowBytes == 128 ? 7 : C::kRowBytes == 64 ? 6 : 5;
    const int lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    const int HH = p.H * p.HB;
    const int total = TcUnits::before(p, p.n_seq, blockIdx.x == 0) * HH;
    const Split split(total, p.ways);
    Unit *queue = reinterpret_cast<Unit *>(smem + C::kMeta);
    Turn<C::kStages> put;
    Turn<C::kKeys> key;
    Turn<2> item;
    int fills = 0, items = 0, nth = 0;  // nth: of the item's units
    bool ok = true;
    const int begin = split.begin(blockIdx.x);
    Cursor<TcUnits> at = {0, 0, 0, 1, 0, 0};
    if ((int)blockIdx.x < split.ways && total > 0)
        at = locate<TcUnits>(p, HH, begin, split.begin(blockIdx.x + 1) - begin);
    bool first_item = true, starts = true, whole = false;
    // The pages of the item's boxes `base` .. + 31 and of the 32 behind them, one a
    // lane: looked up this far ahead, the loop does not wait for them unit by unit.
    const int boxes = kUnit >> log2_box;
    auto look_up = [&](int box) -> int {
        const int64_t tok = (int64_t)(box + lane) << log2_box;
        if (tok >= at.len) return -2;
        return __ldg(p.table + (int64_t)at.b * p.max_pages + (tok >> p.log2_page));
    };
    int base = (at.u * boxes) & ~31;
    int pages = look_up(base), more_pages = look_up(base + 32);
    Unit u = {};  // (what an item's units have alike is set where it starts)
    int row0 = 0;
    while (at.left > 0) {
        if (starts) {
            const int kvh = at.hh / p.HB;
            row0 = kvh << p.log2_page;
            u.b = at.b;
            u.head0 = kvh * p.G + (at.hh - kvh * p.HB) * HP;
            u.heads = min(HP, (kvh + 1) * p.G - u.head0);
            u.slot = (2 * blockIdx.x + (first_item ? 0 : 1)) * HP;
            u.item = items;
            whole = at.u == 0 && at.U <= at.left;  // the share holds the item
        }
        // box `lane` of this unit
        const int box0 = at.u * boxes - base + lane;
        int page = __shfl_sync(0xffffffffu, pages, box0 & 31);
        if (lane >= boxes) page = -2;
        const int row = row0 + ((at.u * kUnit + (lane << log2_box)) & ((1 << p.log2_page) - 1));
        const bool wanted = page != -2, there = (unsigned)page < (unsigned)p.n_pages;
        if (wanted && !there) atomicOr(p.err, kDevErrAlign);
        const uint32_t gone = __ballot_sync(0xffffffffu, wanted && !there);
        const int loads = __popc(__ballot_sync(0xffffffffu, there));
        const int more = at.units() - 1;  // units of the item behind it
        u.rows = min(at.len - at.u * kUnit, kUnit);
        u.missing = gone;
        u.flags = (nth == 0 ? kFirst : 0) | (nth == 1 ? kSecond : 0) |
                  (more == 0 ? kLast : 0) | (more == 1 ? kLastBut1 : 0) | (whole ? kWhole : 0);
        ok = wait_for(bars.k_empty(key.i), key.phase ^ 1u, wc) &&
             wait_for(bars.v_empty(put.i), put.phase ^ 1u, wc);
        if (!ok) break;
        if (lane < boxes)
            reinterpret_cast<int2 *>(smem + C::kPages)[put.i * kBoxes + lane] =
                make_int2(there ? page : -1, row);
        if (lane == 0) {
            queue[put.i] = u;
            mbar_arrive_expect_tx(bars.k_full(key.i), (uint32_t)loads << (log2_box + kLog2Row));
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bars.posted(put.i));
            mbar_arrive(bars.told(put.i));
        }
        if (there)
            tma_load_3d(sbase + key.i * C::kRawBytes +
                            ((uint32_t)lane << (log2_box + kLog2Row)),
                        mK, bars.k_full(key.i), 0, row, page);
        ++fills;
        ++nth;
        put.next();
        key.next();
        if (starts) {
            // the item's queries, as e4m3 terms: rows h and HP + h of its buffer
            uint2 raw[HP];
            const __nv_bfloat16 *src =
                p.q + (int64_t)u.b * p.q_stride + (int64_t)u.head0 * C::D + lane * 4;
#pragma unroll
            for (int h = 0; h < HP; ++h)
                raw[h] = h < u.heads && lane < C::D / 4
                             ? __ldg(reinterpret_cast<const uint2 *>(src + h * C::D))
                             : make_uint2(0u, 0u);
            ok = wait_for(bars.q_free(item.i), item.phase ^ 1u, wc);
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
        if (at.next(p, HH, 1)) {
            starts = true;
            first_item = false;
            nth = 0;
            ++items;
            base = 0;
            if (at.left > 0) {
                pages = look_up(0);
                more_pages = look_up(32);
            }
        } else if (at.u * boxes >= base + 32) {
            base += 32;
            pages = more_pages;
            more_pages = look_up(base + 32);
        }
    }
    for (int w = 0; ok && w < 2; ++w) {  // both groups are told
        ok = wait_for(bars.k_empty(key.i), key.phase ^ 1u, wc) &&
             wait_for(bars.v_empty(put.i), put.phase ^ 1u, wc);
        if (ok) {
            if (lane == 0) {
                queue[put.i].flags = kEnd;
                mbar_arrive(bars.posted(put.i));
                mbar_arrive(bars.k_full(key.i));
                mbar_arrive(bars.told(put.i));
            }
        }
        put.next();
        key.next();
    }
    if (!ok && lane == 0) drain_loads(fills, bars, false, wc);
}

// Warp 11: the scales and values of the units that warp 8 posts.
template <class C>
__device__ void feed_values(const CUtensorMap *mV, const PagedArgs &p, int log2_box, uint8_t *smem,
                            const Bars<C> &bars, const WaitCtl &wc) {
    const int lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    const Unit *queue = reinterpret_cast<const Unit *>(smem + C::kMeta);
    constexpr int kLog2Row = C::kRowBytes == 128 ? 7 : C::kRowBytes == 64 ? 6 : 5;
    Turn<C::kStages> put;
    Turn<C::Q4 ? C::kRawValues : 1> raw;
    int fills = 0, ends = 0;
    bool ok = true;
    while (ends < 2) {
        ok = wait_for(bars.posted(put.i), put.phase, wc);
        if (!ok) break;
        const uint32_t bar = C::Q4 ? bars.raw_full(raw.i) : bars.v_full(put.i);
        if (queue[put.i].flags & kEnd) {
            if (!C::Q4 && lane == 0) mbar_arrive(bar);
            mbar_arrive(bars.told(put.i));  // (as many arrivals as a unit has)
            ++ends;
        } else {
            const int2 *said = reinterpret_cast<const int2 *>(smem + C::kPages) + put.i * kBoxes;
            const int2 box = lane < (kUnit >> log2_box) ? said[lane] : make_int2(-1, 0);
            const int2 box8 = said[(lane * 8) >> log2_box];  // of rows 8 lane .. + 7
            if (box8.x >= 0) {
                const int64_t at_row = (((int64_t)box8.x * p.H) << p.log2_page) + box8.y +
                                       ((lane * 8) & ((1 << log2_box) - 1));
                const uint32_t ex = sbase + C::kExp + put.i * 2 * kUnit + lane * 8;
                copy8(ex, p.k_exp + at_row);
                copy8(ex + kUnit, p.v_exp + at_row);
                if (C::Q4) {
                    constexpr int kEight = 8 * kv_off_bytes(C::D);  // bytes of 8 rows' offsets
                    const uint32_t off = sbase + C::kOff + put.i * 2 * C::kOffBytes + lane * kEight;
                    const uint8_t *ko = p.k_off + at_row * kv_off_bytes(C::D);
                    const uint8_t *vo = p.v_off + at_row * kv_off_bytes(C::D);
#pragma unroll
                    for (int i = 0; i < kEight; i += 16) {
                        copy16(off + i, ko + i);
                        copy16(off + C::kOffBytes + i, vo + i);
                    }
                }
            }
            arrive_after_copies(bars.told(put.i));
            if (C::Q4) {
                ok = wait_for(bars.raw_empty(raw.i), raw.phase ^ 1u, wc);
                if (!ok) break;
            }
            const int loads = __popc(__ballot_sync(0xffffffffu, box.x >= 0));
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)loads << (log2_box + kLog2Row));
            __syncwarp();
            if (box.x >= 0)
                tma_load_3d(sbase + (C::Q4 ? C::raw_value(raw.i) : C::kV + put.i * kTileBytes) +
                                ((uint32_t)lane << (log2_box + kLog2Row)),
                            mV, bar, 0, box.y, box.x);
            ++fills;
        }
        put.next();
        if (C::Q4) raw.next();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) drain_loads(fills, bars, true, wc);
}

// Every MMA that this warp issued completes before TMEM is released.
__device__ __forceinline__ void drain_mmas(uint32_t bar, const WaitCtl &wc) {
    volatile int no_abort = 0;
    const WaitCtl dc{kPagedDrainNs, wc.err, &no_abort, kDevErrTimeout | kDevErrDrain};
    if (elect_one()) {
        mma_commit(bar);
        mbar_wait<false>(bar, 0u, dc);
    }
    __syncwarp();
}

// Warp 9: the scores.
template <class C>
__device__ void issue_scores(uint8_t *smem, uint32_t tmem, const Bars<C> &bars, const WaitCtl &wc) {
    const uint32_t sbase = smem_u32(smem);
    const Unit *queue = reinterpret_cast<const Unit *>(smem + C::kMeta);
    const uint32_t id = idesc_e4m3(C::N1, false);
    const uint64_t k0 = sdesc_kmajor(sbase, 128u, kLayoutSw128);
    const uint64_t q0 = sdesc_kmajor(sbase + C::kQ, 128u, kLayoutSw128);
    Turn<C::kStages> get;
    Turn<C::Q4 ? 2 : C::kKeys> key;  // (keys unpacked in TMEM, or as they came)
    Turn<4> buf;
    while (wait_for(C::Q4 ? bars.kt_full(key.i) : bars.k_full(key.i), key.phase, wc)) {
        const int flags = __shfl_sync(0xffffffffu, queue[get.i].flags, 0);
        const int item = __shfl_sync(0xffffffffu, queue[get.i].item, 0);
        if (flags & kEnd) break;
        if ((flags & kFirst) &&
            !wait_for(bars.q_ready(item & 1), (uint32_t)(item >> 1) & 1u, wc))
            break;
        if (!wait_for(bars.s_free(buf.i), buf.phase ^ 1u, wc)) break;
        tc_fence_after();
        if (elect_one()) {
            const uint64_t a = k0 + (uint32_t)key.i * (kTileBytes >> 4);
            const uint64_t b = q0 + (uint32_t)(item & 1) * (C::kQBytes >> 4);
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int k = 0; k < C::D / 32; ++k)
                    if (C::Q4)
                        mma_e4m3_ts(tmem + C::s_col(buf.i) + 32u * h,
                                    tmem + C::k_col(key.i) + 32u * h + 8u * k, b + k * 2, id, k > 0);
                    else
                        mma_e4m3_ss(tmem + C::s_col(buf.i) + 32u * h,
                                    a + h * (kHalfBytes >> 4) + k * 2, b + k * 2, id, k > 0);
            mma_commit(bars.s_full(buf.i));
            mma_commit(C::Q4 ? bars.kt_empty(key.i) : bars.k_empty(key.i));
            if (flags & kLast) mma_commit(bars.q_free(item & 1));
        }
        __syncwarp();
        buf.next();
        get.next();
        key.next();
    }
    drain_mmas(bars.drain(0), wc);
}

// Warp 10: the products.
template <class C>
__device__ void issue_products(uint8_t *smem, uint32_t tmem, const Bars<C> &bars, const WaitCtl &wc) {
    const uint32_t sbase = smem_u32(smem);
    const Unit *queue = reinterpret_cast<const Unit *>(smem + C::kMeta);
    const uint32_t id = idesc_e4m3(C::N2, true);
    const uint64_t v0 = sdesc_rows_sw128(sbase + C::kV, kHalfBytes);
    // (rows of 16 columns; eight rows, the leading offset, are 128 bytes, 16 more columns,
    // the stride offset, 128 rows on)
    const uint64_t p0 = sdesc_plain(sbase + C::kP, 128u, 128u * 16u);
    Turn<C::kStages> get;
    Turn<2> w;
    while (wait_for(C::Q4 ? bars.v_full(w.i) : bars.v_full(get.i),
                                 C::Q4 ? w.phase : get.phase, wc)) {
        const int flags = __shfl_sync(0xffffffffu, queue[get.i].flags, 0);
        if ((flags & kEnd) || !wait_for(bars.p_full(w.i), w.phase, wc)) break;
        tc_fence_after();
        if (elect_one()) {
            const uint32_t more = (flags & (kFirst | kSecond)) ? 0u : 1u;
            const uint64_t a = v0 + (uint32_t)(C::Q4 ? w.i : get.i) * (kTileBytes >> 4);
            const uint64_t b = p0 + (uint32_t)w.i * (kHalves * C::kPBytes >> 4);
            const uint32_t d = tmem + C::o_col(w.i);
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_e4m3_ss(d, a + h * (kHalfBytes >> 4) + k * (32 * 128 >> 4),
                                b + h * (C::kPBytes >> 4) + k * (32 * 16 >> 4), id,
                                h + k > 0 ? 1u : more);
            mma_commit(bars.pv_done(w.i));
            if (C::Q4) mma_commit(bars.vt_empty(w.i));
            mma_commit(bars.v_empty(get.i));
        }
        __syncwarp();
        w.next();
        get.next();
    }
    drain_mmas(bars.drain(1), wc);
}

// The bytes that magnitudes stand for under each offset, in e4m3; in place of the one that
// there is none of, 15, those of a row that is not finite: NaN throughout.
template <class C>
__device__ __forceinline__ void write_tables(uint8_t *smem) {
    const int t = threadIdx.x;
    if (t >= 16) return;
    const float unit = __uint_as_float((uint32_t)(127 + kE2m1Lift - t) << 23);
    uint2 v = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    if (t <= kE2m1OffMax) {
        v.x = f32x2_to_e4m3x2(0.f, 0.5f * unit) | (f32x2_to_e4m3x2(unit, 1.5f * unit) << 16);
        v.y = f32x2_to_e4m3x2(2.f * unit, 3.f * unit) | (f32x2_to_e4m3x2(4.f * unit, 6.f * unit) << 16);
    }
    reinterpret_cast<uint2 *>(smem + C::kTable)[t] = v;
}

// A packed row, where TMA left it, as e4m3 elements in order: put(c, x) takes its 32
// elements c 32 .. as eight words.
// (A row whole, in code of its own for keys and for values: one loop for both, 16 bytes at a
// time, takes the batch above 97 to 107 us in place of 90, two rows side by side 113.)
template <class C, class Put>
__device__ __forceinline__ void unpack_row(const uint8_t *raw, int row, uint32_t offs,
                                           const uint8_t *tables, Put put) {
    constexpr int kRow = C::kRowBytes, kChunks = kRow / 16;
    const uint8_t *src = raw + row * kRow;
    const uint32_t sw = (kRow == 64 ? (row >> 1) & 3 : (row >> 2) & 1) << 4;
    uint4 x[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) x[c] = *reinterpret_cast<const uint4 *>(src + (sw ^ (c << 4)));
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        // (a table has 8 bytes: block b's lies at 8 times its offset)
        const uint32_t i0 = (c == 0 ? offs << 3 : offs >> (8 * c - 3)) & 0x78u;
        const uint32_t i1 = (offs >> (8 * c + 1)) & 0x78u;
        const uint2 t0 = *reinterpret_cast<const uint2 *>(tables + i0);
        const uint2 t1 = *reinterpret_cast<const uint2 *>(tables + i1);
        uint32_t out[8];
        e2m1_bytes(x[c].x, t0, out[0], out[1]);
        e2m1_bytes(x[c].y, t0, out[2], out[3]);
        e2m1_bytes(x[c].z, t1, out[4], out[5]);
        e2m1_bytes(x[c].w, t1, out[6], out[7]);
        put(c, out);
    }
}

// The offsets of a row's blocks; all 15 where its scale says that it is not finite.  A row
// that does not count (which may hold anything) becomes one of zeros.
template <class C>
__device__ __forceinline__ uint32_t row_offsets(uint8_t *smem, const Unit &u, int log2_box,
                                                uint8_t *raw, int stage, int which, int row) {
    if (row >= u.rows || ((u.missing >> (row >> log2_box)) & 1u)) {
#pragma unroll
        for (int c = 0; c < C::kRowBytes; c += 16)
            *reinterpret_cast<uint4 *>(raw + row * C::kRowBytes + c) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();  // its next writer is the TMA
        return 0u;
    }
    const uint8_t *o = smem + C::kOff + (2 * stage + which) * C::kOffBytes + row * kv_off_bytes(C::D);
    const uint32_t offs = C::D == 128 ? *reinterpret_cast<const uint32_t *>(o)
                                      : (uint32_t) * reinterpret_cast<const uint16_t *>(o);
    return smem[C::kExp + (2 * stage + which) * kUnit + row] == 255 ? ~0u : offs;
}

// Warps 12-15 (4 bits): packed keys to e4m3 elements in TMEM.  Thread r: rows r and r + 128.
template <class C>
__device__ void unpack_keys(int log2_box, uint8_t *smem, uint32_t tmem, const Bars<C> &bars,
                            const WaitCtl &wc) {
    const int r = threadIdx.x & 127, lane = r & 31;
    const uint32_t trow = tmem + ((uint32_t)(r & 96) << 16);
    const Unit *queue = reinterpret_cast<const Unit *>(smem + C::kMeta);
    const uint8_t *tables = smem + C::kTable;
    Turn<C::kStages> get;
    Turn<C::kKeys> key;
    Turn<2> out;
    // (the place's last unit is read, at the end too: a phase may not pass its waiters)
    while (wait_for(bars.told(get.i), get.phase, wc) &&
           wait_for(bars.kt_empty(out.i), out.phase ^ 1u, wc)) {
        if (queue[get.i].flags & kEnd) {
            if (lane == 0) mbar_arrive(bars.kt_full(out.i));
            break;
        }
        if (!wait_for(bars.k_full(key.i), key.phase, wc)) break;
        tc_fence_after();
#pragma unroll 1
        for (int h = 0; h < kHalves; ++h) {
            const int row = 128 * h + r;
            uint8_t *raw = smem + C::raw_key(key.i);
            const uint32_t offs = row_offsets<C>(smem, queue[get.i], log2_box, raw, get.i, 0, row);
            __syncwarp();
            const uint32_t col = trow + C::k_col(out.i) + 32u * h;
            unpack_row<C>(raw, row, offs, tables,
                          [&](int c, const uint32_t *x) { tmem_st8_async(col + 8u * c, x); });
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bars.kt_full(out.i));
            mbar_arrive(bars.k_empty(key.i));
        }
        get.next();
        key.next();
        out.next();
    }
}

// Warps 16-19 (4 bits): packed values to e4m3 elements in shared memory, zeros in place of
// rows that do not count.  Thread r: rows r and r + 128.
template <class C>
__device__ void unpack_values(int log2_box, uint8_t *smem, const Bars<C> &bars, const WaitCtl &wc) {
    const int r = threadIdx.x & 127, lane = r & 31;
    const Unit *queue = reinterpret_cast<const Unit *>(smem + C::kMeta);
    const uint8_t *tables = smem + C::kTable;
    if (C::D == 64) {  // the elements that 64-element rows do not have
#pragma unroll 1
        for (int i = 0; i < C::kValues * kHalves; ++i)
#pragma unroll
            for (int c = 4; c < 8; ++c)
                *reinterpret_cast<uint4 *>(smem + C::kV + (i * 128 + r) * 128 + ((c ^ (r & 7)) << 4)) =
                    make_uint4(0u, 0u, 0u, 0u);
    }
    Turn<C::kStages> get;
    Turn<C::kRawValues> key;
    Turn<2> out;
    while (wait_for(bars.told(get.i), get.phase, wc) &&
           wait_for(bars.vt_empty(out.i), out.phase ^ 1u, wc)) {
        if (queue[get.i].flags & kEnd) {
            if (lane == 0) mbar_arrive(bars.v_full(out.i));
            break;
        }
        if (!wait_for(bars.raw_full(key.i), key.phase, wc)) break;
#pragma unroll 1
        for (int h = 0; h < kHalves; ++h) {
            const int row = 128 * h + r;
            uint8_t *raw = smem + C::raw_value(key.i);
            const uint32_t offs = row_offsets<C>(smem, queue[get.i], log2_box, raw, get.i, 1, row);
            uint8_t *dst = smem + C::kV + out.i * kTileBytes + row * 128;
            const uint32_t sw = (row & 7) << 4;
            unpack_row<C>(raw, row, offs, tables, [&](int c, const uint32_t *x) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4 *>(dst + (sw ^ ((2 * c + i) << 4))) =
                        make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            });
        }
        fence_proxy_async_smem();  // read by the tensor core (async proxy)
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bars.v_full(out.i));
            mbar_arrive(bars.raw_empty(key.i));
        }
        get.next();
        key.next();
        out.next();
    }
}

template <int HP>
__device__ __forceinline__ void read_own(const float *own, float (&v)[HP]) {
#pragma unroll
    for (int h = 0; h < HP; h += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(own + h);
        v[h] = x.x;
        v[h + 1] = x.y;
        v[h + 2] = x.z;
        v[h + 3] = x.w;
    }
}

// The sum over the warp of v[h], in the lanes h, h + HP, ..
template <int HP>
__device__ __forceinline__ float warp_sums(float (&v)[HP], int lane) {
#pragma unroll
    for (int b = HP / 2; b > 0; b >>= 1) {
        const bool up = (lane & b) != 0;
#pragma unroll
        for (int j = 0; j < b; ++j) {
            const float give = up ? v[j] : v[j + b];
            v[j] = (up ? v[j + b] : v[j]) + __shfl_xor_sync(0xffffffffu, give, b);
        }
    }
#pragma unroll
    for (int off = HP; off < 32; off <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    return v[0];
}

// The weights of one row of a unit of 4 bits, as P's words, and its part of the sums, and the
// thread's largest s + e + 7 - m, above 8 where m has to move first; true where r has to.  A
// weight is rounded to fp16 (2^-11 of itself, where the terms of the 8-bit cache's hold 2^-12;
// an eighth of what the bf16 output rounds by); from there on two heads take an instruction, and the
// three e4m3 terms hold its 11 bits.
template <class C>
__device__ __forceinline__ bool weights4(const uint8_t *smem, const float *own,
                                         const float (&m)[C::HP], float (&l)[C::HP],
                                         const float (&rs)[C::HP], float (&tops)[C::HP],
                                         uint32_t (&pw)[C::N2 / 4],
                                         uint32_t scores, int stage, int row, bool there,
                                         float least_e) {
    constexpr int HP = C::HP;
    const uint8_t *ex = smem + C::kExp + stage * 2 * kUnit + row;
    // (rows that do not count have scores of zero: see row_offsets)
    const float kf = there ? __uint_as_float((uint32_t)max((int)ex[0] - kE2m1Lift, 0) << 23) : 0.f;
    const float ve = (float)ex[kUnit] - (127.f + kE2m1Lift);
    const float none = there ? 0.f : -INFINITY;
    const uint64_t kf2 = f32x2(kf, kf), none2 = f32x2(none, none);
    const uint64_t ve2 = f32x2(ve + 7.f, ve + 7.f), minus2 = f32x2(-1.f, -1.f);
    const uint64_t low2 = f32x2(0.03125f, 0.03125f);
    float qs[HP];
    read_own<HP>(own + kOwnQs, qs);
    uint32_t raw[C::N1];
    tmem_read(scores, raw);
#pragma unroll
    for (int h = 0; h < HP; h += 2) {
        const auto raw2 = [&](int i) {
            return f32x2(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1]));
        };
        const uint64_t x = fma_f32x2(raw2(HP + h), low2, raw2(h));
        const uint64_t s = fma_f32x2(x, mul_f32x2(f32x2(qs[h], qs[h + 1]), kf2), none2);
        float e0, e1, t0, t1;
        f32x2_split(fma_f32x2(f32x2(rs[h], rs[h + 1]), minus2, s), e0, e1);
        f32x2_split(add_f32x2(s, fma_f32x2(f32x2(m[h], m[h + 1]), minus2, ve2)), t0, t1);
        tops[h] = fmaxf(tops[h], t0);
        tops[h + 1] = fmaxf(tops[h + 1], t1);
        f32x2_split(add_f32x2(f32x2(l[h], l[h + 1]), f32x2(exp2_fast(e0), exp2_fast(e1))), l[h],
                    l[h + 1]);
        uint32_t y = f32x2_to_f16x2(exp2_fast(t0), exp2_fast(t1));
#pragma unroll
        for (int t = 0; t < 3; ++t) {
            const uint32_t a = f16x2_to_e4m3x2(y);
            const int n = t * HP + h;
            if (n % 4) pw[n / 4] = __byte_perm(pw[n / 4], a, 0x5410);
            else pw[n / 4] = a;
            if (t < 2) y = times16_less(y, e4m3x2_to_f16x2(a));
        }
    }
    return there && ve < least_e;
}

// Group w (warps 4 w .. 4 w + 3): every second unit.  Thread r: rows r and r + 128 of a
// unit, and element r of the outputs.  A warp whose wait runs out does no more work, but keeps
// to the group's barriers until all four learn of it and leave together.
//
// What a head needs once in a while -- moving m and r, joining the warps' sums and the groups'
// outputs -- is done by one lane for each head: a single long sequence passes through
// here a few times only, and what it waits for is the instructions themselves (all heads'
// worth in every thread: 57 us in place of 53 for 131040 rows, 8 heads of 8).
template <class C>
__device__ void softmax(const PagedArgs &p, int w, uint8_t *smem, uint32_t tmem,
                        const Bars<C> &bars, const WaitCtl &wc) {
    constexpr int HP = C::HP;
    const int r = threadIdx.x & 127, warp = r >> 5, lane = r & 31;
    const int hl = lane & (HP - 1);  // this lane's head
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t to = trow + C::o_col(w);
    const Unit *queue = reinterpret_cast<const Unit *>(smem + C::kMeta);
    float *group = reinterpret_cast<float *>(smem + C::kOwn) + w * 4 * kOwnSize;
    float *own = group + warp * kOwnSize;
    float *join = reinterpret_cast<float *>(smem + C::kJoin), *join_stat = join + HP * 128;
    Turn<C::kStages> get;
    get.i = w;
    Turn<4> buf;
    buf.i = w;
    Turn<1> turn, joins;  // parities alone
    const int log2_box = min(p.log2_page, 7);
    // (an e2m1 row's scale is read 2^6 smaller: seq_dev.cuh)
    constexpr int kLift = C::Q4 ? kE2m1Lift : 0;
    float m[HP], l[HP];
#pragma unroll
    for (int h = 0; h < HP; ++h) m[h] = l[h] = 0.f;
    // While the rows' e are at least this, no s is more than kSumLag above its r, as no
    // s + e is more than m + 1: one comparison a row stands for those of all heads.
    float least_e = INFINITY;
    bool ok = true;
    while (true) {
        ok = ok && wait_for(bars.told(get.i), get.phase, wc);
        Unit u = {0, 0, 0, 0, 0u, 0, 0, 0};
        if (ok) u = queue[get.i];
        const bool end = (u.flags & kEnd) != 0, fresh = (u.flags & (kFirst | kSecond)) != 0;
        // Half k of the unit: this thread's row in it, its scores in log2 units (read from TMEM
        // where they are needed: both halves' would take more code and registers), its value
        // row's exponent, and whether it counts.
        uint32_t zeros = 0;  // halves whose value row is known to be zeros
        auto counts = [&](int row) -> bool {
            return row < u.rows && !((u.missing >> (row >> log2_box)) & 1u);
        };
        auto half = [&](int k, float (&s)[HP], float &ve) -> bool {
            const int row = k * 128 + r;
            const uint8_t *ex = smem + C::kExp + get.i * 2 * kUnit + row;
            const float kf = C::Q4 ? __uint_as_float((uint32_t)max((int)ex[0] - kLift, 0) << 23)
                                   : __uint_as_float((uint32_t)ex[0] << 23);
            ve = (float)ex[kUnit] - (127.f + kLift);
            const bool there = counts(row);
            float qs[HP];
            read_own<HP>(own + kOwnQs, qs);
            uint32_t raw[C::N1];
            tmem_read(trow + C::s_col(buf.i) + 32u * k, raw);
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                const float x = fmaf(__uint_as_float(raw[HP + h]), 0.03125f, __uint_as_float(raw[h]));
                s[h] = there ? x * (qs[h] * kf) : -INFINITY;
            }
            if ((zeros >> k) & 1u) ve = -INFINITY;
            return there;
        };
        if (ok && !end) {
            if (fresh) {
                const int q = u.item & 1;
                ok = wait_for(bars.q_ready(q), (uint32_t)(u.item >> 1) & 1u, wc);
                __syncwarp();
                if (lane < HP) {
                    own[kOwnQs + lane] = reinterpret_cast<const float *>(smem + C::kQs)[q * 16 + lane];
                    own[kOwnM + lane] = own[kOwnR + lane] = kLowest;
                }
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    m[h] = kLowest;
                    l[h] = 0.f;
                }
                least_e = INFINITY;
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bars.q_free(q));
                    // (the other group has no part in an item of one unit)
                    if ((u.flags & kFirst) && (u.flags & kLast)) mbar_arrive(bars.q_free(q));
                }
            }
            ok = ok && wait_for(bars.s_full(buf.i), buf.phase, wc);
            tc_fence_after();
        }
        // P and O are free, and O whole, once the product of the group's unit before is done
        ok = ok && wait_for(bars.pv_done(w), turn.phase ^ 1u, wc);
        // The weights are worked out as if m and r could stay (but for an item's first unit);
        // where they cannot, which is seldom, they move and the weights are made once more.
        float ln[HP];  // the sums with this unit's part
        float tops[HP];    // (4 bits) this thread's largest s + e + 7 - m
        bool low = false;  // (4 bits) its r has to move
        for (bool moved = false;; moved = true) {
            bool moves = fresh && !moved;
            if (!end && !moves) {
                float rs[HP];
                read_own<HP>(own + kOwnR, rs);
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    ln[h] = l[h];
                    tops[h] = -INFINITY;
                }
#pragma unroll 1
                for (int k = 0; k < kHalves; ++k) {
                    // weights, times 2^7, as three terms: columns t HP + head of P's row
                    uint32_t pw[C::N2 / 4] = {};
                    if constexpr (C::Q4) {
                        low |= weights4<C>(smem, own, m, ln, rs, tops, pw, trow + C::s_col(buf.i) + 32u * k,
                                             get.i, k * 128 + r, counts(k * 128 + r),
                                             least_e);
                    } else {
                        float s[HP], ve;
                        moves |= half(k, s, ve) && ve < least_e;
#pragma unroll
                        for (int h = 0; h < HP; h += 2) {
                            float x[2];
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                ln[h + c] += exp2_fast(s[h + c] - rs[h + c]);
                                moves |= s[h + c] + ve > m[h + c] + 1.f;
                                x[c] = exp2_fast(s[h + c] + ((ve + 7.f) - m[h + c]));
                            }
#pragma unroll
                            for (int t = 0; t < 3; ++t) {
                                const uint32_t a = f32x2_to_e4m3x2(x[0], x[1]);
                                const int n = t * HP + h;
                                if (n % 4) pw[n / 4] = __byte_perm(pw[n / 4], a, 0x5410);
                                else pw[n / 4] = a;
                                if (t < 2) {
                                    const float2 y = e4m3x2_to_f32(a);
                                    x[0] = 16.f * (x[0] - y.x);
                                    x[1] = 16.f * (x[1] - y.y);
                                }
                            }
                        }
                    }
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        smem + C::kP + (w * kHalves + k) * C::kPBytes + r * 16);
#pragma unroll
                    for (int i = 0; i < C::N2 / 16; ++i)
                        dst[i * 128] = make_uint4(pw[4 * i], pw[4 * i + 1], pw[4 * i + 2], pw[4 * i + 3]);
                }
                if (C::Q4) {
                    moves |= low;
#pragma unroll
                    for (int h = 0; h < HP; ++h) moves |= tops[h] > 8.f;
                }
            }
            if (moved || !bar_any(1 + w, 128, moves || !ok)) break;
            if (bar_any(1 + w, 128, !ok)) return;
            // A value row of zeros (scale 1) has no part in m: it would take the bits of the
            // weights that count.  Rows of other scales are not looked at, as the values may
            // still be on their way: 3 us of 94 for 64 sequences.  (Of 4 bits, they have the
            // smallest scale, and no part in m.)
            bool ready = false;
#pragma unroll 1
            for (int k = 0; !C::Q4 && k < kHalves; ++k) {
                const int row = k * 128 + r;
                const bool unsure =
                    (float)smem[C::kExp + (get.i * 2 + 1) * kUnit + row] == 127.f && row < u.rows;
                if (!__any_sync(0xffffffffu, unsure)) continue;
                if (!ready)
                    ok = ok && wait_for(bars.v_full(get.i), get.phase, wc);
                ready = true;
                const uint4 *v = reinterpret_cast<const uint4 *>(
                    smem + C::kV + get.i * kTileBytes + row * 128);
                uint32_t some = 0;
                if (ok)
#pragma unroll
                    for (int c = 0; c < 8; ++c) {  // (each of eight lanes another piece)
                        const uint4 x = v[c ^ (r & 7)];
                        some |= x.x | x.y | x.z | x.w;
                    }
                if (unsure && !(some & 0x7f7f7f7fu)) zeros |= 1u << k;
            }
            float top = -INFINITY, stop = -INFINITY;  // of s + e, of s; head hl's
            // (4 bits: m alone moves, as a rule, and the weights have shown how far.  The warp's
            // r may stay behind, where no row asks for it and no row's s + e passes m by more than
            // 1 + kStep: with e >= least_e = m - r - (kSumLag - 1), s - r is at most kSumLag +
            // kStep then, and m - r at most 120 more.  From the next unit on least_e goes by
            // the new m.  A higher step would take the sum to infinity: r moves with m.)
            bool far = false;
            if (C::Q4 && !fresh)
#pragma unroll
                for (int h = 0; h < HP; ++h) far |= tops[h] > 8.f + kStep;
            const bool known = C::Q4 && !__any_sync(0xffffffffu, low || far || fresh ||
                                                                     own[kOwnM + hl] == kLowest ||
                                                                     own[kOwnR + hl] == kLowest);
            if (known) {
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    const float y = warp_max(tops[h]);
                    if (hl == h) top = y;
                }
                top += own[kOwnM + hl] - 7.f;
            } else {
#pragma unroll 1
                for (int k = 0; k < kHalves; ++k) {
                    float s[HP], ve;
                    half(k, s, ve);
#pragma unroll
                    for (int h = 0; h < HP; ++h) {
                        const float x = warp_max(s[h]), y = warp_max(s[h] + ve);
                        if (hl == h) {
                            stop = fmaxf(stop, x);
                            top = fmaxf(top, y);
                        }
                    }
                }
            }
            if (lane < HP) own[kOwnTop + lane] = top;
            bar_group(w);
            float e = -INFINITY;
            if (lane < HP) {
                const float m0 = own[kOwnM + lane], r0 = own[kOwnR + lane];
                float mn = m0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mn = fmaxf(mn, group[k * kOwnSize + kOwnTop + lane] + C::kAhead);
                const float rn = fmaxf(r0, stop);
                own[kOwnM + lane] = mn;
                own[kOwnR + lane] = rn;
                own[kOwnF + lane] = exp2_fast(m0 - mn);
                own[kOwnFl + lane] = exp2_fast(r0 - rn);
                e = mn - rn - (kSumLag - 1.f);
            }
            least_e = warp_max(e);
            __syncwarp();
            float f[HP];
            read_own<HP>(own + kOwnFl, f);
#pragma unroll
            for (int h = 0; h < HP; ++h) l[h] *= f[h];
            read_own<HP>(own + kOwnM, m);
            if (!fresh) {
                read_own<HP>(own + kOwnF, f);
                tc_fence_after();
                uint32_t o[C::N2];
                tmem_read(to, o);
#pragma unroll
                for (int c = 0; c < C::N2; ++c)
                    if (c < 3 * HP) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c % HP]);
#pragma unroll
                for (int c = 0; c < C::N2; c += 16) tmem_st16_async(to + c, o + c);
                tmem_st_wait();
                tc_fence_before();
            }
        }
        if (end) return;
#pragma unroll
        for (int h = 0; h < HP; ++h) l[h] = ln[h];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.s_free(buf.i));
        if (!C::Q4 && (u.rows < kUnit || u.missing)) {  // (the values have to be there)
            ok = ok && wait_for(bars.v_full(get.i), get.phase, wc);
#pragma unroll
            for (int k = 0; k < kHalves; ++k) {
                const int row = k * 128 + r;
                if (!ok || (row < u.rows && !((u.missing >> (row >> log2_box)) & 1u))) continue;
                // what lies in other rows may be anything
                uint4 *v = reinterpret_cast<uint4 *>(smem + C::kV + get.i * kTileBytes + row * 128);
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        fence_proxy_async_smem();  // P and V are read by the tensor core (async proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.p_full(w));
        if (u.flags & (kLast | kLastBut1)) {
            // the group's last unit of the item
            const float mine = warp_sums<HP>(l, lane);
            if (lane < HP) {
                own[kOwnL + lane] = mine;
                own[kOwnRl + lane] = own[kOwnR + lane];
            }
            ok = ok && wait_for(bars.pv_done(w), turn.phase, wc);
            tc_fence_after();
            uint32_t o[C::N2];
            tmem_read(to, o);
            tc_fence_before();
            bar_group(w);
            float x[HP];
#pragma unroll
            for (int h = 0; h < HP; ++h)
                x[h] = 0.0078125f * fmaf(fmaf(__uint_as_float(o[2 * HP + h]), 0.0625f,
                                              __uint_as_float(o[HP + h])),
                                         0.0625f, __uint_as_float(o[h]));
            // m, r and the sum of head hl over the group
            float mh = own[kOwnM + hl], rh = kLowest, sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) rh = fmaxf(rh, group[k * kOwnSize + kOwnRl + hl]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum += group[k * kOwnSize + kOwnL + hl] *
                       exp2_fast(group[k * kOwnSize + kOwnRl + hl] - rh);
            if (u.flags & kLastBut1) {  // the other group has the item's last
                ok = ok && wait_for(bars.join_free(), joins.phase ^ 1u, wc);
                if (ok) {
#pragma unroll
                    for (int h = 0; h < HP; ++h) join[h * 128 + r] = x[h];
                    if (r < HP)
                        *reinterpret_cast<float4 *>(join_stat + r * 4) = make_float4(mh, rh, sum, 0.f);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.join_full());
                joins.next();
            } else {
                float f[HP];
                if (!(u.flags & kFirst)) {
                    ok = ok && wait_for(bars.join_full(), joins.phase, wc);
                    const float4 o1 = *reinterpret_cast<const float4 *>(join_stat + hl * 4);
                    const float mn = fmaxf(mh, o1.x), rn = fmaxf(rh, o1.y);
                    if (lane < HP) {
                        own[kOwnF + lane] = exp2_fast(mh - mn);
                        own[kOwnFl + lane] = exp2_fast(o1.x - mn);
                    }
                    sum = sum * exp2_fast(rh - rn) + o1.z * exp2_fast(o1.y - rn);
                    mh = mn;
                    rh = rn;
                    __syncwarp();
                    read_own<HP>(own + kOwnF, f);
#pragma unroll
                    for (int h = 0; h < HP; ++h) x[h] *= f[h];
                    read_own<HP>(own + kOwnFl, f);
#pragma unroll
                    for (int h = 0; h < HP; ++h) x[h] = fmaf(join[h * 128 + r], f[h], x[h]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars.join_free());
                    joins.next();
                }
                if (u.flags & kWhole) {
                    if (lane < HP) {
                        const float half = half_factor(mh, rh);
                        own[kOwnF + lane] = sum > 0.f || sum != sum ? half / sum : 0.f;
                        own[kOwnFl + lane] = half;
                    }
                    __syncwarp();
                    read_own<HP>(own + kOwnF, f);
#pragma unroll
                    for (int h = 0; h < HP; ++h) x[h] *= f[h];
                    read_own<HP>(own + kOwnFl, f);
                }
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    if (h >= u.heads || !ok || r >= C::D) break;
                    if (u.flags & kWhole)
                        p.out[(int64_t)u.b * p.out_stride + (int64_t)(u.head0 + h) * C::D + r] =
                            to_output<true>(x[h] * f[h]);
                    else
                        p.part_o[(int64_t)(u.slot + h) * C::D + r] = x[h];
                }
                if (!(u.flags & kWhole) && ok && r < u.heads)
                    p.part_ml[u.slot + r] = make_float4(mh, rh, sum, 0.f);
            }
        }
        buf.next(2);
        get.next(2);
        turn.next();
    }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                const PagedArgs p, int log2_box) {
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded address: the compiler then knows that it is shared memory, and
    // its accesses do not go through the generic path)
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    griddep_launch_dependents();
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const Bars<C> bars{smem_u32(smem) + C::kBars};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kSlots);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kSlots + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kKeys; ++s) {
            mbar_init(bars.k_full(s), 1);
            mbar_init(bars.k_empty(s), C::Q4 ? 4 : 1);  // (the warps that unpack)
        }
        for (int s = 0; s < C::kRawValues; ++s) {
            mbar_init(bars.raw_full(s), 1);
            mbar_init(bars.raw_empty(s), 4);
        }
        for (int i = 0; C::Q4 && i < 2; ++i) {
            mbar_init(bars.kt_full(i), 4);
            mbar_init(bars.kt_empty(i), 1);
            mbar_init(bars.vt_empty(i), 1);
        }
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bars.v_full(s), C::Q4 ? 4 : 1);
            mbar_init(bars.v_empty(s), 1);
            mbar_init(bars.posted(s), 1);
            mbar_init(bars.told(s), 1 + 32);  // what the unit is, and 32 lanes' copies of scales
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.q_ready(i), 1);
            mbar_init(bars.q_free(i), 9);  // the MMAs that read it, and eight warps
            mbar_init(bars.p_full(i), 4);
            mbar_init(bars.pv_done(i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bars.s_full(i), 1);
            mbar_init(bars.s_free(i), 4);
        }
        mbar_init(bars.join_full(), 4);
        mbar_init(bars.join_free(), 4);
        mbar_init(bars.drain(0), 1);
        mbar_init(bars.drain(1), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mK);
        tma_prefetch_desc(&mV);
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512u);
        tmem_relinquish();
    }
    if (C::Q4) write_tables<C>(smem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{p.wait_ns, p.err, abort_flag, 0u};
    griddep_wait();
    if (warp < 8) {
        softmax<C>(p, warp >> 2, smem, tmem, bars, wc);
    } else if (C::Q4 && warp >= 16) {
        unpack_values<C>(log2_box, smem, bars, wc);
    } else if (C::Q4 && warp >= 12) {
        unpack_keys<C>(log2_box, smem, tmem, bars, wc);
    } else if (warp == 8) {
        feed<C>(&mK, p, log2_box, smem, bars, wc);
    } else if (warp == 11) {
        feed_values<C>(&mV, p, log2_box, smem, bars, wc);
    } else if (warp == 9) {
        issue_scores<C>(smem, __shfl_sync(0xffffffffu, tmem, 0), bars, wc);
    } else {
        issue_products<C>(smem, __shfl_sync(0xffffffffu, tmem, 0), bars, wc);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512u);
}

template <class C>
cudaError_t launch(PagedArgs &a, const KvCacheSpec &cache, const LaunchCtx &ctx) {
    static_assert(C::kSmem <= 227 * 1024, "shared memory");
    static_assert(C::N1 <= 32 && C::N2 <= 48, "TMEM");
    constexpr int RB = C::kRowBytes;
    const int log2_box = std::min(cache.log2_page, 7);
    CUtensorMap mK, mV;
    const cuuint64_t rows = (cuuint64_t)cache.H << cache.log2_page;
    const cuuint64_t dims[3] = {RB / 2, rows, (cuuint64_t)cache.n_pages};
    const cuuint64_t strides[2] = {RB, rows * RB};
    const cuuint32_t box[3] = {RB / 2, 1u << log2_box, 1};
    if (!encode_tiled_bf16(&mK, 3, cache.k, dims, strides, box, RB) ||
        !encode_tiled_bf16(&mV, 3, cache.v, dims, strides, box, RB))
        return cudaErrorInvalidValue;
    constexpr int kMaxDev = 64;
    static std::atomic<bool> attr_set[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(paged_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    a.ways = paged_ways(a, kUnit, std::min(kMaxWays, ctx.num_sms));
    count_launches(1);
    return launch_pdl(paged_tc_kernel<C>, dim3((unsigned)a.ways), dim3(C::kThreads), C::kSmem, ctx,
                      mK, mV, a, log2_box);
}

}  // namespace

cudaError_t launch_paged_tc(PagedArgs &a, const KvCacheSpec &cache, const LaunchCtx &ctx,
                            int *block_heads) {
    a.HB = 1;
    const bool few = a.G <= 4;
    *block_heads = few ? 4 : 8;
    if (cache.fmt == kKvE4M3)
        return few ? launch<Cfg<4, 128, false>>(a, cache, ctx)
                   : launch<Cfg<8, 128, false>>(a, cache, ctx);
    if (cache.D == 128)
        return few ? launch<Cfg<4, 128, true>>(a, cache, ctx)
                   : launch<Cfg<8, 128, true>>(a, cache, ctx);
    return few ? launch<Cfg<4, 64, true>>(a, cache, ctx) : launch<Cfg<8, 64, true>>(a, cache, ctx);
}

}  // namespace wanvae
