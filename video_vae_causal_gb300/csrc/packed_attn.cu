// packed_attn.cu -- attention over packed sequences of different lengths,
// causal or full, query heads in groups that share a kv head, on tcgen05:
//
//     out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j)
//
// over the keys j of query i's own sequence and, where causal, j <= i + Lk - Lq
// (the last query sees every key).  A query that sees none gives zeros.
//
// A CTA owns one kv head and two tiles of 128 rows of one sequence, each 128 / G
// consecutive queries times the G query heads of the group, so that short
// prompts fill the tensor core's rows, keys are read once for the group, and
// a causal tile's diagonal is G times shorter.  It sweeps the visible keys, and for
// each tile, turn by turn,
//   S = Q K_u^T       (tcgen05, S in TMEM)
//   P = exp2(S' - m)  (a warpgroup of its own, one row a thread; P in TMEM)
//   O += P V_u        (tcgen05, P from TMEM, V as it lies in memory, read along its rows)
// Each tile has an issuing warp of its own (one warp for both, which waits for one
// tile while the other's P is there: 324 and 1319 us for the two examples below) and
// its next S is under way while the warpgroup computes exponentials:
//   D = 128: O of both tiles takes half of TMEM, S and P the rest.  A turn is 64
//     keys, with two places for S a tile; P lies over its S, and the place's next S is
//     issued behind the product that reads P (MMAs of one thread run in order).  Turns of 128
//     keys with one place, where S waits for P's product: 318 us.
//   D = 64: a turn is 128 keys with one place for S and columns of its own for P
//     (kApart); the next S is issued as soon as the warpgroup has read the last one.
//     Turns of 64 keys as above: 1440 us, their waits and Q's reads counting twice.
// The running maximum m moves only by more than 2^8, as in the mid-block's core, so P
// stays <= 256 and O is rarely rescaled, by the tile's own warpgroup.  P rounds to
// bf16, the type that V has (an MMA's operands share one); the sum is of the
// unrounded P.  (Taking the first half's weights from the maximum so far while the
// turn's is found changed nothing: 333 us.)
//
// What bounds it: for D = 128 the tensor core, 2048 cycles of arithmetic for 128 keys of both
// tiles of about 2900 (the tensor pipe is 61 % active; Q K^T, half of it, also reads both
// operands from shared memory); 16 query and 4 kv heads over causal prompts of 8192, 5003,
// 188 and 3001 tokens: 301 us, 1.38 PFLOP/s, 0.71 of the measured matrix rate.  For D = 64
// nothing alone: 128 keys of both tiles take about 2300 cycles, of which an SM quarter issues
// 1460 (exponentials, sums, maxima and roundings, 1024 of them MUFU's) and the tensor core
// works 1024; the rest is what two warps a scheduler leave bare of the chain from S in TMEM
// over the maximum and the exponentials back to TMEM.  21 frames of 6240 tokens, 6 heads,
// full: 1195 us, 1.05 PFLOP/s, 0.54.
//
// Masked scores are replaced, never added to, so nothing in a masked key
// reaches a row.  A masked value's weight is zero, but 0 * NaN is not: of the blocks
// that some row of the CTA sees in part (the last three at most) the value rows
// behind the last key are zeroed in shared memory, and so are elements that are
// not finite; those are added afterwards to the rows that see them, key by key.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <atomic>

#include "norm_act.cuh"
#include "seq_dev.cuh"
#include "seq_ops.h"
#include "seq_ptx.cuh"

namespace wanvae {
namespace {

constexpr int kThreads = 384;  // two softmax warpgroups; two issuers, producer, an idle warp
// Registers: 384 threads launch with 168 (64512 in all); the third warpgroup
// gives back what the softmax warpgroups take: 2 * 128 * 216 + 128 * 72 = 64512.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kRows = 128;                 // rows of a tile, keys of a block
constexpr uint32_t kAtom = kRows * 128u;   // 128 rows x 64 bf16, 128-byte swizzled
constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;

struct PackedArgs {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *out;
    int64_t q_stride, k_stride, v_stride, out_stride;
    const int32_t *cu_q, *cu_k;
    int n_seq, total_q, total_k;
    int Hkv, G, nt;    // kv heads; query heads of one; queries of a tile
    float scale_log2;  // scale * log2(e)
    int causal;
    unsigned *err;
    uint64_t wait_ns;
};

// A CTA's queries [q0, q0 + nq) of the packed rows (tile w holds p.nt of them
// from q0 + w nt); its sequence's keys [k0, k0 + Lk).  Query i of the CTA sees
// the first see0 + i keys where causal, else all.
struct Tile {
    int q0, nq, k0, Lk, see0;
};

template <int D>
struct Layout {
    static constexpr uint32_t kTile = (D / 64) * kAtom;  // a tile of Q, a block of K or V
    static constexpr int kStages = D == 64 ? 8 : 5;      // blocks of K and V in flight
    static constexpr uint32_t kQ = 0, kRing = 2 * kTile;
    static constexpr uint32_t kBars = kRing + kStages * kTile;
    static constexpr uint32_t kSmem = 1024 + kBars + 272;
    // Keys of a turn, turns of a block.  TMEM columns of tile w: S of turn u, its P over S or
    // (kApart) in columns of its own, O.
    static constexpr bool kApart = D == 64;
    static constexpr int kTurn = kApart ? 128 : 64, kPer = kRows / kTurn;
    static __device__ __forceinline__ int block_of(int u) { return kApart ? u : u >> 1; }
    static __device__ __forceinline__ int place_of(int u) { return kApart ? 0 : u & 1; }
    static __device__ __forceinline__ uint32_t s_col(int w, int u) {
        return 128u * w + (kApart ? 0u : 64u * (u & 1));
    }
    static __device__ __forceinline__ uint32_t p_col(int w, int u) {
        return kApart ? 256u + 64u * w : s_col(w, u);
    }
    static __device__ __forceinline__ uint32_t o_col(int w) {
        return kApart ? 384u + 64u * w : 256u + 128u * w;
    }
};

// The ring holds K_0, V_0, K_1, V_1, ..
__device__ __forceinline__ int fill_k(int j) { return 2 * j; }
__device__ __forceinline__ int fill_v(int j) { return 2 * j + 1; }

template <int D>
struct Bars {
    static constexpr int kStages = Layout<D>::kStages;
    uint32_t base;
    __device__ uint32_t q_full() const { return base; }
    __device__ uint32_t drain(int w) const { return base + 8 + 8 * w; }
    __device__ uint32_t o_done(int w) const { return base + 24 + 8 * w; }
    // of a turn's S and P (phase_of_turn): two turns' worth, or one and S read (kApart)
    static constexpr bool kApart = Layout<D>::kApart;
    static __device__ int buf(int u) { return kApart ? 0 : u & 1; }
    __device__ uint32_t s_full(int w, int u) const { return base + 40 + 16 * w + 8 * buf(u); }
    __device__ uint32_t p_full(int w, int u) const { return base + 72 + 16 * w + 8 * buf(u); }
    __device__ uint32_t s_free(int w) const { return base + 48 + 16 * w; }
    __device__ uint32_t o_full(int w) const { return base + 104 + 8 * w; }
    __device__ uint32_t full(int fill) const { return base + 120 + 8 * (fill % kStages); }
    __device__ uint32_t empty(int fill) const {
        return base + 120 + 8 * (kStages + fill % kStages);
    }
    static __device__ uint32_t phase(int fill) { return (uint32_t)(fill / kStages) & 1u; }
    static __device__ uint32_t phase_of_turn(int u) {
        return (uint32_t)(kApart ? u : u >> 1) & 1u;
    }
};

// Tile pair `x` of the launch, counting the pairs of every sequence in order;
// whole warp.  nq = 0: no such pair.  `tell`: report offsets that leave the tensors (the
// launch's last pair does: one more than sequences in order can have, it comes by all of them
// up to the first that is out of order).
__device__ Tile find_tile(const PackedArgs &p, int x, bool tell) {
    const int lane = threadIdx.x & 31;
    Tile r = {0, 0, 0, 0, 0};
    int before = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += 32) {
        const int s = s0 + lane;
        int qa = 0, qb = 0, ka = 0, kb = 0, tiles = 0;
        if (s < p.n_seq) {
            qa = __ldg(p.cu_q + s);
            qb = __ldg(p.cu_q + s + 1);
            ka = __ldg(p.cu_k + s);
            kb = __ldg(p.cu_k + s + 1);
            // offsets that leave the tensors count for nothing
            const bool ok = qa >= 0 && qb >= qa && qb <= p.total_q && ka >= 0 && kb >= ka &&
                            kb <= p.total_k;
            if (!ok && tell) atomicOr(p.err, kDevErrAlign);
            tiles = ok ? (qb - qa + 2 * p.nt - 1) / (2 * p.nt) : 0;
        }
        int incl = tiles;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const unsigned m = __ballot_sync(0xffffffffu, before + incl > x);
        if (m) {
            const int l = __ffs(m) - 1;
            // the last queries first: where causal they see the most keys
            const int t = before + __shfl_sync(0xffffffffu, incl, l) - 1 - x;
            qa = __shfl_sync(0xffffffffu, qa, l);
            qb = __shfl_sync(0xffffffffu, qb, l);
            ka = __shfl_sync(0xffffffffu, ka, l);
            kb = __shfl_sync(0xffffffffu, kb, l);
            const int Lq = qb - qa, i0 = t * 2 * p.nt;
            r.q0 = qa + i0;
            r.nq = min(2 * p.nt, Lq - i0);
            r.k0 = ka;
            r.Lk = kb - ka;
            r.see0 = i0 + r.Lk - Lq + 1;
            return r;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return r;
}

// The bf16 pairs of w that are not finite, as masks of 16 bits.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return __vcmpgeu2(w & 0x7fff7fffu, 0x7f807f80u);
}

// A value row of a block in shared memory (row `row` of 128, the blocks of 64
// elements kAtom apart): zeros where `behind`, else without its elements that are
// not finite, and *odd set where it had any.  The row's 16-byte pieces are taken in any
// order (the swizzle stays within a row), a different one by each of eight lanes.
template <int D>
__device__ __forceinline__ void clean_row(uint8_t *block, int row, bool behind, int *odd) {
    uint32_t m = 0;
    uint4 *v = reinterpret_cast<uint4 *>(block) + row * 8;
#pragma unroll
    for (int a = 0; a < D / 64; ++a)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint4 *at = v + a * (kAtom / 16) + (c ^ (row & 7));
            if (behind) {
                *at = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            const uint4 x = *at;
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                     __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
        }
    if (!not_finite(m)) return;
    *odd = 1;
    __threadfence_block();  // who finds the zeros finds this too
    for (int a = 0; a < D / 64; ++a)
        for (int c = 0; c < 8; ++c) {
            uint4 x = v[a * (kAtom / 16) + c];
            x.x &= ~not_finite(x.x);
            x.y &= ~not_finite(x.y);
            x.z &= ~not_finite(x.z);
            x.w &= ~not_finite(x.w);
            v[a * (kAtom / 16) + c] = x;
        }
}

// Adds to a row that is written the value elements that clean_row took out of the keys
// [from, keys) (they are not finite, so their sum is the output, whatever l is); m:
// the row's maximum in log2 units.  Whole warp, lane l holds outputs l * D / 32 ..
template <int D>
__device__ __noinline__ void put_back(const PackedArgs &p, int q, int head, int kvh, int k0,
                                      int from, int keys, float m) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16 *qr = p.q + (int64_t)q * p.q_stride + (int64_t)head * D + lane * E;
    float qv[E], o[E] = {};
#pragma unroll
    for (int e = 0; e < E; ++e) qv[e] = __bfloat162float(qr[e]);
    bool any = false;
    for (int j = from; j < keys; ++j) {
        const int64_t at = (int64_t)kvh * D + lane * E;
        const __nv_bfloat16 *vr = p.v + (int64_t)(k0 + j) * p.v_stride + at;
        float v[E];
        bool bad = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[e] = __bfloat162float(vr[e]);
            bad |= !isfinite(v[e]);
        }
        if (!__any_sync(0xffffffffu, bad)) continue;
        const __nv_bfloat16 *kr = p.k + (int64_t)(k0 + j) * p.k_stride + at;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(qv[e], __bfloat162float(kr[e]), s);
        s = nact_group_sum(s, 32) * p.scale_log2;
        const float w = s == -INFINITY ? 0.f : exp2f(s - m);
        if (w == 0.f) continue;
        any = true;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (!isfinite(v[e])) o[e] += w * v[e];
    }
    if (!any) return;
    __nv_bfloat16 *dst = p.out + (int64_t)q * p.out_stride + (int64_t)head * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (o[e] != 0.f) dst[e] = __float2bfloat16(__bfloat162float(dst[e]) + o[e]);
}

// Keys that a query of tile w sees (0: none, or no such tile).
__device__ __forceinline__ int keys_of(const PackedArgs &p, const Tile &tl, int w) {
    const int nq = min(tl.nq - w * p.nt, p.nt);
    if (nq <= 0) return 0;
    return p.causal ? min(tl.Lk, max(0, tl.see0 + w * p.nt + nq - 1)) : tl.Lk;
}
template <int D>
__device__ __forceinline__ int turns_of(int keys) {
    return (keys + Layout<D>::kTurn - 1) / Layout<D>::kTurn;
}

// TMA producer (one thread): Q, then K_0, V_0, K_1, ..
template <int D>
__device__ void producer(const CUtensorMap *mQ, const CUtensorMap *mK, const CUtensorMap *mV,
                         const PackedArgs &p, const Tile &tl, int kvh, int blocks, uint32_t sbase,
                         const Bars<D> &bars, const WaitCtl &wc) {
    using L = Layout<D>;
    const int tiles = tl.nq > p.nt ? 2 : 1;
    mbar_arrive_expect_tx(bars.q_full(), (uint32_t)(tiles * (D / 64) * p.G * p.nt) * 128u);
    for (int w = 0; w < tiles; ++w)
        for (int a = 0; a < D / 64; ++a)
            tma_load_3d(sbase + L::kQ + w * L::kTile + a * kAtom, mQ, bars.q_full(), a * 64,
                        kvh * p.G, tl.q0 + w * p.nt);
    int f = 0;
    for (; f < 2 * blocks; ++f) {
        if (!mbar_wait<false>(bars.empty(f), bars.phase(f) ^ 1u, wc)) break;
        mbar_arrive_expect_tx(bars.full(f), L::kTile);
        const CUtensorMap *m = f & 1 ? mV : mK;
        for (int a = 0; a < D / 64; ++a)
            tma_load_3d(sbase + L::kRing + (f % L::kStages) * L::kTile + a * kAtom, m, bars.full(f),
                        a * 64, kvh, tl.k0 + (f >> 1) * kRows);
    }
    if (f < 2 * blocks) {
        // Aborted: let every copy in flight land before shared memory goes away.
        volatile int no_abort = 0;
        const WaitCtl dc{kDrainNs, wc.err, &no_abort, kDevErrTimeout | kDevErrDrain};
        mbar_wait<false>(bars.q_full(), 0u, dc);
        for (int i = f > L::kStages ? f - L::kStages : 0; i < f; ++i)
            mbar_wait<false>(bars.full(i), bars.phase(i), dc);
    }
}

// MMA issuer of tile w (one warp), which has n turns in the first of the CTA's blocks.
template <int D>
__device__ void issuer(int w, int n, int blocks, uint32_t sbase, uint32_t tmem,
                       const Bars<D> &bars, const WaitCtl &wc) {
    using L = Layout<D>;
    constexpr int kTurn = L::kTurn, kPer = L::kPer, kAhead = L::kApart ? 1 : 2;
    const uint32_t id_s = idesc_bf16_f32(128, kTurn), id_o = idesc_bf16_f32_bt(128, D);
    const uint64_t q0 = sdesc_kmajor(sbase + L::kQ + w * L::kTile, 128u, kLayoutSw128);
    const uint64_t k0 = sdesc_kmajor(sbase + L::kRing, 128u, kLayoutSw128);
    const uint64_t v0 = sdesc_rows_sw128(sbase + L::kRing, kAtom);
    const uint32_t to = tmem + L::o_col(w);
    auto part_of = [](int f, int u) {  // a turn's rows of a block in the ring
        return (uint32_t)(f % L::kStages) * (L::kTile >> 4) +
               (uint32_t)L::place_of(u) * (kTurn * 128 >> 4);
    };
    auto ends_block = [&](int u) { return L::place_of(u) == kPer - 1 || u + 1 == n; };
    auto scores = [&](int u) {  // S = Q K^T of a turn (in the elected lane)
        const int f = fill_k(L::block_of(u));
        const uint64_t b = k0 + part_of(f, u);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (uint32_t)(kk >> 2) * (kAtom >> 4) + (kk & 3) * 2;
            mma_bf16_ss(tmem + L::s_col(w, u), q0 + off, b + off, id_s, kk > 0);
        }
        mma_commit(bars.s_full(w, u));
        if (ends_block(u)) mma_commit(bars.empty(f));
    };
    bool ok = n == 0 || (mbar_wait_warp<false>(bars.q_full(), 0u, wc) &&
                         mbar_wait_warp<false>(bars.full(fill_k(0)), 0u, wc));
    if (ok && n > 0) {
        tc_fence_after();
        if (elect_one()) {
            scores(0);
            if (kAhead > 1 && n > 1) scores(1);
        }
        __syncwarp();
    }
    for (int u = 0; ok && u < n; ++u) {
        const int f = fill_v(L::block_of(u));  // (the next block's keys are fill f + 1)
        const bool more = u + kAhead < n;
        if (L::place_of(u) == 0) {
            if (!L::kApart)
                ok = mbar_wait_warp<false>(bars.full(f), bars.phase(f), wc);
            if (more) ok = ok && mbar_wait_warp<false>(bars.full(f + 1), bars.phase(f + 1), wc);
            if (L::kApart && more) {
                ok = ok && mbar_wait_warp<false>(bars.s_free(w), bars.phase_of_turn(u), wc);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) scores(u + 1);
                __syncwarp();
            }
            if (L::kApart)
                ok = ok && mbar_wait_warp<false>(bars.full(f), bars.phase(f), wc);
        }
        ok = ok && mbar_wait_warp<false>(bars.p_full(w, u), bars.phase_of_turn(u), wc);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            const uint64_t b = v0 + part_of(f, u);
#pragma unroll
            for (int kk = 0; kk < kTurn / 16; ++kk)
                mma_bf16_ts(to, tmem + L::p_col(w, u) + kk * 8, b + kk * (2048u >> 4), id_o,
                            u > 0 || kk > 0);
            mma_commit(u + 1 < n ? bars.o_done(w) : bars.o_full(w));
            if (ends_block(u)) mma_commit(bars.empty(f));
            if (!L::kApart && more) scores(u + 2);
        }
        __syncwarp();
    }
    // the other tile's blocks (a place is given back once a turn: not before it is full)
    for (int f = 2 * ((n + kPer - 1) / kPer); ok && f < 2 * blocks; ++f) {
        ok = mbar_wait_warp<false>(bars.full(f), bars.phase(f), wc);
        if (ok && elect_one()) mbar_arrive(bars.empty(f));
        __syncwarp();
    }
    // Every MMA issued above completes before TMEM is released.
    volatile int no_abort = 0;
    const WaitCtl dc{kDrainNs, wc.err, &no_abort, kDevErrTimeout | kDevErrDrain};
    if (elect_one()) {
        mma_commit(bars.drain(w));
        mbar_wait<false>(bars.drain(w), 0u, dc);
    }
    __syncwarp();
}

// Softmax and epilogue of tile w (4 warps, one row a thread: the TMEM lane
// quarter that the warp may access).  Decisions before warp-wide TMEM accesses
// are uniform.
template <int D>
__device__ void softmax(const PackedArgs &p, const Tile &tl, int w, int kvh, int n, int keys_cta,
                        uint8_t *smem, uint32_t tmem, int *odd_values,
                        const Bars<D> &bars, const WaitCtl &wc) {
    using L = Layout<D>;
    constexpr int kTurn = L::kTurn;
    const int qd = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int row = qd * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(qd * 32) << 16);
    const uint32_t to = trow + L::o_col(w);
    const int r = row / p.G, head = kvh * p.G + row % p.G;
    const int i = w * p.nt + r;  // query of the CTA
    const bool there = row < p.G * p.nt && i < tl.nq;
    const int see = p.causal ? min(tl.Lk, max(0, tl.see0 + i)) : tl.Lk;
    // The first block that some row of the CTA does not see whole.
    const int part = (p.causal ? min(tl.Lk, max(0, tl.see0)) : tl.Lk) / kRows;
    float m = -INFINITY;  // of the raw scores
    float l = 0.f;
    for (int u = 0; u < n; ++u) {
        if (!mbar_wait_warp<false>(bars.s_full(w, u), bars.phase_of_turn(u), wc)) return;
        tc_fence_after();
        const uint32_t ts = trow + L::s_col(w, u), tp = trow + L::p_col(w, u);
        uint32_t s[kTurn];
#pragma unroll
        for (int c0 = 0; c0 < kTurn; c0 += 32) tmem_ld32_async(ts + (uint32_t)c0, s + c0);
#pragma unroll
        for (int c0 = 0; c0 < kTurn; c0 += 32) tmem_ld_wait32(s + c0);
        if (L::kApart) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.s_free(w));
        }
        const int kvalid = see - u * kTurn;
        if (__any_sync(0xffffffffu, kvalid < kTurn)) {
#pragma unroll
            for (int c = 0; c < kTurn; ++c)
                if (c >= kvalid) s[c] = 0xff800000u;  // -inf
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            mx[c] = fmaxf(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
#pragma unroll
        for (int c = 8; c < kTurn; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mx[k] = max3(mx[k], __uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        float f = 1.f;
        if ((top - m) * p.scale_log2 > 8.f) {  // (also the first turn's, from -inf)
            if (m != -INFINITY) f = exp2_fast((m - top) * p.scale_log2);
            m = top;
        }
        if (u > 0 && __any_sync(0xffffffffu, f != 1.f)) {
            l *= f;
            // once the last turn's product is in O (the one before it was there before S,
            // or, kApart, before the last P)
            if (!mbar_wait_warp<false>(bars.o_done(w), (uint32_t)(u - 1) & 1u, wc)) return;
            tc_fence_after();
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tmem_ld32_async(to + (uint32_t)c0, o);
                tmem_ld_wait32(o);
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                tmem_st32_async(to + (uint32_t)c0, o);
            }
        }
        const float ms = m == -INFINITY ? 0.f : m * p.scale_log2;
        const uint64_t sc2 = f32x2(p.scale_log2, p.scale_log2), ms2 = f32x2(-ms, -ms);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int h = 0; h < kTurn / 64; ++h) {  // 64 keys, 32 columns of P at a time
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const int e = h * 64 + 2 * c;
                float a, b;
                f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2,
                                      ms2), a, b);
                a = exp2_fast(a);
                b = exp2_fast(b);
                sum[c & 1] = add_f32x2(sum[c & 1], f32x2(a, b));
                pk[c] = nact_pack(a, b);
            }
            if (L::kApart && h == 0 && u > 0) {  // the last turn's product has read P
                if (!mbar_wait_warp<false>(bars.o_done(w), (uint32_t)(u - 1) & 1u, wc)) return;
                tc_fence_after();
            }
            tmem_st32_async(tp + 32u * h, pk);
        }
        float s0, s1;
        f32x2_split(add_f32x2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        // a block seen in part (both tiles' warpgroups clean it: the same zeros)
        if (L::place_of(u) == 0 && L::block_of(u) >= part) {
            const int fv = fill_v(L::block_of(u));
            if (!mbar_wait_warp<false>(bars.full(fv), bars.phase(fv), wc)) return;
            const bool behind = u * kTurn + row >= keys_cta;
            if (p.causal || behind)
                clean_row<D>(smem + L::kRing + (fv % L::kStages) * L::kTile, row, behind,
                             odd_values);
            fence_proxy_async_smem();  // read by the tensor core (async proxy)
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.p_full(w, u));
    }
    if (n > 0) {
        if (!mbar_wait_warp<false>(bars.o_full(w), 0u, wc)) return;
        tc_fence_after();
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    __nv_bfloat16 *dst = p.out + (int64_t)(tl.q0 + i) * p.out_stride + (int64_t)head * D;
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t acc[32];
        if (n > 0) {
            tmem_ld32_async(to + (uint32_t)c0, acc);
            tmem_ld_wait32(acc);
        } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) acc[c] = 0u;
        }
        float o[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = see > 0 ? __uint_as_float(acc[c]) * inv : 0.f;
        if (there) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4 *>(dst + c0 + 8 * c) =
                    make_uint4(nact_pack(o[8 * c], o[8 * c + 1]), nact_pack(o[8 * c + 2], o[8 * c + 3]),
                               nact_pack(o[8 * c + 4], o[8 * c + 5]),
                               nact_pack(o[8 * c + 6], o[8 * c + 7]));
        }
    }
    // (set before the last p_full that o_full came after)
    if (*reinterpret_cast<volatile int *>(odd_values)) {
        __syncwarp();
        unsigned rows = __ballot_sync(0xffffffffu, there && see > part * kRows);
        const float ms = m == -INFINITY ? 0.f : m * p.scale_log2;
        while (rows) {
            const int b = __ffs(rows) - 1;
            rows &= rows - 1;
            put_back<D>(p, tl.q0 + __shfl_sync(0xffffffffu, i, b),
                        __shfl_sync(0xffffffffu, head, b), kvh, tl.k0, part * kRows,
                        __shfl_sync(0xffffffffu, see, b), __shfl_sync(0xffffffffu, ms, b));
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
packed_attn_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                   const __grid_constant__ CUtensorMap mV, const __grid_constant__ PackedArgs p) {
    using L = Layout<D>;
    griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const Bars<D> bars{sbase + L::kBars};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kBars + 256);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kBars + 260);
    int *odd_values = reinterpret_cast<int *>(smem + L::kBars + 264);
    if (threadIdx.x == 0) {
        mbar_init(bars.q_full(), 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(bars.drain(w), 1);
            mbar_init(bars.o_done(w), 1);
            mbar_init(bars.o_full(w), 1);
            for (int u = 0; u < L::kPer; ++u) {
                mbar_init(bars.s_full(w, u), 1);
                mbar_init(bars.p_full(w, u), 4);
            }
            if (L::kApart) mbar_init(bars.s_free(w), 4);
        }
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bars.full(s), 1);
            mbar_init(bars.empty(s), 2);
        }
        *abort_flag = 0;
        *odd_values = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mQ);
        tma_prefetch_desc(&mK);
        tma_prefetch_desc(&mV);
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512u);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{p.wait_ns, p.err, abort_flag, 0u};
    griddep_wait();
    const int kvh = blockIdx.x % p.Hkv;
    const Tile tl = find_tile(p, blockIdx.x / p.Hkv,
                              blockIdx.x == gridDim.x - 1);
    const int keys[2] = {keys_of(p, tl, 0), keys_of(p, tl, 1)};
    const int n0 = turns_of<D>(keys[0]), n1 = turns_of<D>(keys[1]);
    const int keys_cta = max(keys[0], keys[1]), blocks = (max(n0, n1) + L::kPer - 1) / L::kPer;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        if (tl.nq > 0)
            softmax<D>(p, tl, warp >> 2, kvh, warp >> 2 ? n1 : n0, keys_cta, smem, tmem, odd_values, bars, wc);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        const int w = warp - 8;
        if (w < 2 && blocks > 0)
            issuer<D>(w, __shfl_sync(0xffffffffu, w ? n1 : n0, 0),
                      __shfl_sync(0xffffffffu, blocks, 0), sbase,
                      __shfl_sync(0xffffffffu, tmem, 0), bars, wc);
        if (w == 2 && lane == 0 && blocks > 0)
            producer<D>(&mQ, &mK, &mV, p, tl, kvh, blocks, sbase, bars, wc);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512u);
}

template <int D>
cudaError_t launch(const PackedAttnSpec &s, const LaunchCtx &ctx) {
    using L = Layout<D>;
    PackedArgs a;
    memset(&a, 0, sizeof(a));
    a.q = static_cast<const __nv_bfloat16 *>(s.q);
    a.k = static_cast<const __nv_bfloat16 *>(s.k);
    a.v = static_cast<const __nv_bfloat16 *>(s.v);
    a.out = static_cast<__nv_bfloat16 *>(s.out);
    a.q_stride = s.q_stride;
    a.k_stride = s.k_stride;
    a.v_stride = s.v_stride;
    a.out_stride = s.out_stride;
    a.cu_q = s.cu_q;
    a.cu_k = s.cu_k;
    a.n_seq = s.n_seq;
    a.total_q = s.total_q;
    a.total_k = s.total_k;
    a.Hkv = s.Hkv;
    a.G = s.Hq / s.Hkv;
    a.nt = kRows / a.G;
    a.scale_log2 = s.scale * 1.4426950408889634f;
    a.causal = s.causal;
    a.err = ctx.err;
    a.wait_ns = ctx.wait_ns;
    CUtensorMap mQ, mK, mV;
    // [token][head][D] as (D, heads, tokens): a tile of Q is 64 elements of
    // the group's heads of nt tokens (rows in that order), a block of K or V 64
    // elements of one head of 128 tokens
    const cuuint64_t dq[3] = {(cuuint64_t)D, (cuuint64_t)s.Hq, (cuuint64_t)s.total_q};
    const cuuint64_t sq[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.q_stride * 2};
    const cuuint32_t bq[3] = {64, (cuuint32_t)a.G, (cuuint32_t)a.nt};
    const cuuint64_t dk[3] = {(cuuint64_t)D, (cuuint64_t)s.Hkv, (cuuint64_t)s.total_k};
    const cuuint64_t sk[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.k_stride * 2};
    const cuuint64_t sv[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.v_stride * 2};
    const cuuint32_t bk[3] = {64, 1, (cuuint32_t)kRows};
    if (!encode_tiled_bf16(&mQ, 3, s.q, dq, sq, bq, 128) ||
        !encode_tiled_bf16(&mK, 3, s.k, dk, sk, bk, 128) ||
        !encode_tiled_bf16(&mV, 3, s.v, dk, sv, bk, 128))
        return cudaErrorInvalidValue;
    constexpr int kMaxDev = 64;
    static std::atomic<bool> attr_set[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(packed_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 L::kSmem);
        if (e != cudaSuccess) return e;
        // the register split waits forever on a launch with fewer
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, packed_attn_kernel<D>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
        attr_set[dev].store(true, std::memory_order_release);
    }
    // at most this many pairs of tiles, whatever the lengths (the rest finds none)
    const int64_t pairs = ((int64_t)s.total_q + 2 * a.nt - 1) / (2 * a.nt) + s.n_seq;
    if (pairs * s.Hkv > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(packed_attn_kernel<D>, dim3((unsigned)(pairs * s.Hkv)), dim3(kThreads),
                      L::kSmem, ctx, mQ, mK, mV, a);
}

}  // namespace

cudaError_t launch_packed_attention(const PackedAttnSpec &s, const LaunchCtx &ctx) {
    if (s.D == 64) return launch<64>(s, ctx);
    if (s.D == 128) return launch<128>(s, ctx);
    return cudaErrorInvalidValue;
}

}  // namespace wanvae
