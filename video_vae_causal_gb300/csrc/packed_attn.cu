// packed_attn.cu -- attention over packed sequences of different lengths,
// causal or full, query heads in groups that share a kv head, on tcgen05:
//
//     out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j)
//
// over the keys j of query i's own sequence and, where causal, j <= i + Lk - Lq
// (the last query sees every key).  A query that sees none gives zeros.
//
// A CTA owns one kv head and a tile of 128 rows of one sequence: 128 / G
// consecutive queries times the G query heads of the group, so that short
// prompts fill the tensor core's rows, keys are read once for the group, and
// a causal tile's diagonal is G times shorter.  It sweeps the visible keys in
// blocks of 128:
//   S = Q K_j^T       (tcgen05, S in TMEM)
//   P = exp2(S' - m)  (4 softmax warps, one row a thread; P in shared memory)
//   O += P V_j        (tcgen05, O in TMEM; V as it lies in memory, read along its rows)
// The running maximum m moves only by more than 2^8, as in the mid-block's
// core, so P stays <= 256 and O is rarely rescaled.  P rounds to bf16, the type
// that V has (an MMA's operands share one); the sum is of the unrounded P.
//
// Masked scores are replaced, never added to, so nothing in a masked key
// reaches a row.  A masked value's weight is zero, but 0 * NaN is not: the value
// rows behind the last key that the tile sees are zeroed in shared memory, and a
// causal row that comes out non-finite is computed again over the keys that it
// sees, key by key (only non-finite inputs lead there).
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

constexpr int kThreads = 192;
constexpr int kRows = 128;                 // rows of a tile, keys of a block
constexpr uint32_t kAtom = kRows * 128u;   // 128 rows x 64 bf16, 128-byte swizzled
constexpr int kStages = 2;                 // blocks of K and of V in flight
constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;

struct PackedArgs {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *out;
    int64_t q_stride, k_stride, v_stride, out_stride;
    const int32_t *cu_q, *cu_k;
    int n_seq, total_q, total_k;
    int G, nt;         // query heads of a kv head, queries of a tile
    float scale_log2;  // scale * log2(e)
    int causal;
    unsigned *err;
    uint64_t wait_ns;
};

// A CTA's tile: queries [q0, q0 + nq) of the packed rows; keys [k0, k0 + kend)
// are seen by one of them or more, query i (in the tile) sees the first
// min(kend, see + i) of them (see: see0 where causal, kend elsewhere).
struct Tile {
    int q0, nq, k0, kend, see0;
};

template <int D>
struct Layout {
    static constexpr uint32_t kTile = (D / 64) * kAtom;  // Q, a block of K, a block of V
    static constexpr uint32_t kQ = 0, kP = kTile, kK = kP + 2 * kAtom, kV = kK + kStages * kTile;
    static constexpr uint32_t kBars = kV + kStages * kTile;
    static constexpr uint32_t kSmem = 1024 + kBars + 256;
};

struct Bars {
    uint32_t base;
    __device__ uint32_t q_full() const { return base; }
    __device__ uint32_t s_full() const { return base + 8; }
    __device__ uint32_t s_free() const { return base + 16; }
    __device__ uint32_t p_full() const { return base + 24; }
    __device__ uint32_t o_done() const { return base + 32; }
    __device__ uint32_t drain() const { return base + 40; }
    __device__ uint32_t k_full(int s) const { return base + 48 + 8 * s; }
    __device__ uint32_t k_empty(int s) const { return base + 48 + 8 * (kStages + s); }
    __device__ uint32_t v_full(int s) const { return base + 48 + 8 * (2 * kStages + s); }
    __device__ uint32_t v_empty(int s) const { return base + 48 + 8 * (3 * kStages + s); }
};

// Tile `x` of the launch, counting the tiles of every sequence in order;
// whole warp.  nq = 0: no such tile.
__device__ Tile find_tile(const PackedArgs &p, int x) {
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
            if (!ok && x == 0) atomicOr(p.err, kDevErrAlign);
            tiles = ok ? (qb - qa + p.nt - 1) / p.nt : 0;
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
            const int t = x - before - __shfl_sync(0xffffffffu, incl - tiles, l);
            qa = __shfl_sync(0xffffffffu, qa, l);
            qb = __shfl_sync(0xffffffffu, qb, l);
            ka = __shfl_sync(0xffffffffu, ka, l);
            kb = __shfl_sync(0xffffffffu, kb, l);
            const int Lq = qb - qa, Lk = kb - ka;
            r.q0 = qa + t * p.nt;
            r.nq = min(p.nt, Lq - t * p.nt);
            r.k0 = ka;
            r.see0 = p.causal ? t * p.nt + Lk - Lq + 1 : Lk;
            r.kend = p.causal ? min(Lk, max(0, r.see0 + r.nq - 1)) : Lk;
            return r;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return r;
}

// A row that met a non-finite value, over the keys that it sees alone; whole
// warp, lane l holds outputs l * D / 32 ...
template <int D>
__device__ __noinline__ void slow_row(const PackedArgs &p, int q, int head, int kvh, int k0,
                                      int keys) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16 *qr = p.q + (int64_t)q * p.q_stride + (int64_t)head * D + lane * E;
    float qv[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) qv[e] = __bfloat162float(qr[e]);
    for (int j = 0; j < keys; ++j) {
        const __nv_bfloat16 *kr = p.k + (int64_t)(k0 + j) * p.k_stride + (int64_t)kvh * D + lane * E;
        const __nv_bfloat16 *vr = p.v + (int64_t)(k0 + j) * p.v_stride + (int64_t)kvh * D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(qv[e], __bfloat162float(kr[e]), s);
        s = nact_group_sum(s, 32) * p.scale_log2;
        const float mn = fmaxf(m, s);
        const float f = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float w = mn == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * f + (w == 0.f ? 0.f : w * __bfloat162float(vr[e]));
    }
    __nv_bfloat16 *dst = p.out + (int64_t)q * p.out_stride + (int64_t)head * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16(o[e] / l);
}

// TMA producer (one thread): Q, then K_j and V_j of every block.
template <int D>
__device__ void producer(const CUtensorMap *mQ, const CUtensorMap *mK, const CUtensorMap *mV,
                         const PackedArgs &p, const Tile &tl, int kvh, int nkb, uint32_t sbase,
                         const Bars &bars, const WaitCtl &wc) {
    using L = Layout<D>;
    uint32_t kf = 0, vf = 0;
    bool ok = true;
    mbar_arrive_expect_tx(bars.q_full(), (uint32_t)(D / 64) * p.G * p.nt * 128u);
    for (int a = 0; a < D / 64; ++a)
        tma_load_3d(sbase + L::kQ + a * kAtom, mQ, bars.q_full(), a * 64, kvh * p.G, tl.q0);
    for (int j = 0; ok && j < nkb; ++j) {
        const int s = j % kStages;
        const uint32_t ph = (uint32_t)(j / kStages) & 1u;
        ok = mbar_wait<false>(bars.k_empty(s), ph ^ 1u, wc);
        if (!ok) break;
        mbar_arrive_expect_tx(bars.k_full(s), L::kTile);
        for (int a = 0; a < D / 64; ++a)
            tma_load_3d(sbase + L::kK + s * L::kTile + a * kAtom, mK, bars.k_full(s), a * 64, kvh,
                        tl.k0 + j * kRows);
        ++kf;
        ok = mbar_wait<false>(bars.v_empty(s), ph ^ 1u, wc);
        if (!ok) break;
        mbar_arrive_expect_tx(bars.v_full(s), L::kTile);
        for (int a = 0; a < D / 64; ++a)
            tma_load_3d(sbase + L::kV + s * L::kTile + a * kAtom, mV, bars.v_full(s), a * 64, kvh,
                        tl.k0 + j * kRows);
        ++vf;
    }
    if (!ok) {
        // Aborted: let every copy in flight land before shared memory goes away.
        volatile int no_abort = 0;
        const WaitCtl dc{kDrainNs, wc.err, &no_abort, kDevErrTimeout | kDevErrDrain};
        mbar_wait<false>(bars.q_full(), 0u, dc);
        for (uint32_t f = kf > kStages ? kf - kStages : 0; f < kf; ++f)
            mbar_wait<false>(bars.k_full(f % kStages), (f / kStages) & 1u, dc);
        for (uint32_t f = vf > kStages ? vf - kStages : 0; f < vf; ++f)
            mbar_wait<false>(bars.v_full(f % kStages), (f / kStages) & 1u, dc);
    }
}

// MMA issuer (one thread): S_0, then S_{j+1} and O += P_j V_j for every block.
template <int D>
__device__ void issuer(int nkb, uint32_t sbase, uint32_t tmem, const Bars &bars,
                       const WaitCtl &wc) {
    using L = Layout<D>;
    const uint32_t id_s = idesc_bf16_f32(128, 128), id_o = idesc_bf16_f32_bt(128, D);
    const uint64_t q0 = sdesc_kmajor(sbase + L::kQ, 128u, kLayoutSw128);
    const uint64_t p0 = sdesc_kmajor(sbase + L::kP, 128u, kLayoutSw128);
    const uint64_t k0 = sdesc_kmajor(sbase + L::kK, 128u, kLayoutSw128);
    const uint64_t v0 = sdesc_rows_sw128(sbase + L::kV, kAtom);
    auto issue_s = [&](int j) -> bool {
        const int s = j % kStages;
        if (j > 0 && !mbar_wait<false>(bars.s_free(), (uint32_t)(j - 1) & 1u, wc)) return false;
        if (!mbar_wait<false>(bars.k_full(s), (uint32_t)(j / kStages) & 1u, wc)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (uint32_t)(kk >> 2) * (kAtom >> 4) + (kk & 3) * 2;
            mma_bf16_ss(tmem, q0 + off, k0 + (uint32_t)s * (L::kTile >> 4) + off, id_s, kk > 0);
        }
        mma_commit(bars.k_empty(s));
        mma_commit(bars.s_full());
        return true;
    };
    bool ok = mbar_wait<false>(bars.q_full(), 0u, wc);
    if (ok) tc_fence_after();
    ok = ok && issue_s(0);
    for (int j = 0; ok && j < nkb; ++j) {
        if (j + 1 < nkb) ok = issue_s(j + 1);
        const int s = j % kStages;
        ok = ok && mbar_wait<false>(bars.v_full(s), (uint32_t)(j / kStages) & 1u, wc) &&
             mbar_wait<false>(bars.p_full(), (uint32_t)j & 1u, wc);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
            mma_bf16_ss(tmem + 128u,
                        p0 + (uint32_t)(kk >> 2) * (kAtom >> 4) + (kk & 3) * 2,
                        v0 + (uint32_t)s * (L::kTile >> 4) + kk * (2048u >> 4), id_o,
                        j > 0 || kk > 0);
        mma_commit(bars.v_empty(s));
        mma_commit(bars.o_done());
    }
    // Every MMA issued above completes before TMEM is released.
    volatile int no_abort = 0;
    const WaitCtl dc{kDrainNs, wc.err, &no_abort, kDevErrTimeout | kDevErrDrain};
    mma_commit(bars.drain());
    mbar_wait<false>(bars.drain(), 0u, dc);
}

// Softmax and epilogue (4 warps, one row a thread: the TMEM lane quarter that
// the warp may access).  Decisions before warp-wide TMEM accesses are uniform.
template <int D>
__device__ void softmax(const PackedArgs &p, const Tile &tl, int kvh, int nkb, uint8_t *smem,
                        uint32_t tmem, const Bars &bars, const WaitCtl &wc) {
    using L = Layout<D>;
    const int qd = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int row = qd * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(qd * 32) << 16);
    const int i = row / p.G, head = kvh * p.G + row % p.G;
    const bool there = row < p.G * p.nt && i < tl.nq;
    const int see = min(tl.kend, max(0, p.causal ? tl.see0 + i : tl.kend));
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < nkb; ++j) {
        if (!mbar_wait_warp<false>(bars.s_full(), (uint32_t)j & 1u, wc)) return;
        tc_fence_after();
        float s[kRows];
#pragma unroll
        for (int c0 = 0; c0 < kRows; c0 += 32) {
            uint32_t r[32];
            tmem_ld_cols(trow + (uint32_t)c0, 32, r);
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c0 + c] = __uint_as_float(r[c]);
        }
        tc_fence_before();
        mbar_arrive(bars.s_free());
        const int kvalid = see - j * kRows;
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < kRows; ++c) {
            s[c] = c < kvalid ? s[c] * p.scale_log2 : -INFINITY;
            mx = fmaxf(mx, s[c]);
        }
        float f = 1.f;
        if (mx > m + 8.f) {
            if (m != -INFINITY) f = exp2f(m - mx);
            m = mx;
        }
        const float ms = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
        uint32_t pk[kRows / 2];
#pragma unroll
        for (int c = 0; c < kRows; c += 2) {
            const float a = exp2f(s[c] - ms), b = exp2f(s[c + 1] - ms);
            sum += a + b;
            pk[c / 2] = nact_pack(a, b);
        }
        l = l * f + sum;
        // P's buffer and O are free once the previous block's product is done
        if (j > 0 && !mbar_wait_warp<false>(bars.o_done(), (uint32_t)(j - 1) & 1u, wc)) return;
        tc_fence_after();
        if (__any_sync(0xffffffffu, f != 1.f)) {
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t r[32];
                tmem_ld_cols(trow + 128u + (uint32_t)c0, 32, r);
#pragma unroll
                for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * f);
                tmem_st_cols32(trow + 128u + (uint32_t)c0, r);
            }
        }
#pragma unroll
        for (int ch = 0; ch < kRows / 8; ++ch)
            *reinterpret_cast<uint4 *>(smem + L::kP + (ch >> 3) * kAtom + row * 128 +
                                       (((ch & 7) ^ (row & 7)) << 4)) =
                make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
        // values behind the last visible key become zeros (the last block alone)
        const int left = tl.kend - j * kRows;
        if (left < kRows) {
            const int st = j % kStages;
            if (!mbar_wait_warp<false>(bars.v_full(st), (uint32_t)(j / kStages) & 1u, wc)) return;
            uint4 *v = reinterpret_cast<uint4 *>(smem + L::kV + st * L::kTile);
            for (int e = left * 8 + row; e < kRows * 8; e += 128)
#pragma unroll
                for (int a = 0; a < D / 64; ++a) v[a * (kAtom / 16) + e] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // P and V are read by the tensor core (async proxy)
        tc_fence_before();
        mbar_arrive(bars.p_full());
    }
    if (nkb > 0) {
        if (!mbar_wait_warp<false>(bars.o_done(), (uint32_t)(nkb - 1) & 1u, wc)) return;
        tc_fence_after();
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    __nv_bfloat16 *dst = p.out + (int64_t)(tl.q0 + i) * p.out_stride + (int64_t)head * D;
    float probe = 0.f;  // NaN once an output is not finite
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t r[32];
        if (nkb > 0) {
            tmem_ld_cols(trow + 128u + (uint32_t)c0, 32, r);
        } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = 0u;
        }
        float o[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            o[c] = see > 0 ? __uint_as_float(r[c]) * inv : 0.f;
            probe = fmaf(o[c], 0.f, probe);
        }
        if (there) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4 *>(dst + c0 + 8 * c) =
                    make_uint4(nact_pack(o[8 * c], o[8 * c + 1]), nact_pack(o[8 * c + 2], o[8 * c + 3]),
                               nact_pack(o[8 * c + 4], o[8 * c + 5]),
                               nact_pack(o[8 * c + 6], o[8 * c + 7]));
        }
    }
    if (p.causal) {
        unsigned bad = __ballot_sync(0xffffffffu, there && see > 0 && probe != probe);
        while (bad) {
            const int b = __ffs(bad) - 1;
            bad &= bad - 1;
            slow_row<D>(p, tl.q0 + __shfl_sync(0xffffffffu, i, b),
                        __shfl_sync(0xffffffffu, head, b), kvh, tl.k0,
                        __shfl_sync(0xffffffffu, see, b));
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
packed_attn_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                   const __grid_constant__ CUtensorMap mV, const PackedArgs p) {
    using L = Layout<D>;
    griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Bars bars{sbase + L::kBars};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kBars + 240);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kBars + 244);
    if (threadIdx.x == 0) {
        mbar_init(bars.q_full(), 1);
        mbar_init(bars.s_full(), 1);
        mbar_init(bars.s_free(), 128);
        mbar_init(bars.p_full(), 128);
        mbar_init(bars.o_done(), 1);
        mbar_init(bars.drain(), 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bars.k_full(s), 1);
            mbar_init(bars.k_empty(s), 1);
            mbar_init(bars.v_full(s), 1);
            mbar_init(bars.v_empty(s), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mQ);
        tma_prefetch_desc(&mK);
        tma_prefetch_desc(&mV);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 256u);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{p.wait_ns, p.err, abort_flag, 0u};
    griddep_wait();
    const int kvh = blockIdx.y;
    const Tile tl = find_tile(p, blockIdx.x);
    const int nkb = (tl.kend + kRows - 1) / kRows;
    if (tl.nq > 0) {
        if (warp == 0) {
            if (lane == 0 && nkb > 0)
                producer<D>(&mQ, &mK, &mV, p, tl, kvh, nkb, sbase, bars, wc);
        } else if (warp == 1) {
            if (lane == 0 && nkb > 0) issuer<D>(nkb, sbase, tmem, bars, wc);
        } else {
            softmax<D>(p, tl, kvh, nkb, smem, tmem, bars, wc);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 256u);
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
        attr_set[dev].store(true, std::memory_order_release);
    }
    // at most this many tiles, whatever the lengths (the rest finds none)
    const int tiles = (s.total_q + a.nt - 1) / a.nt + s.n_seq;
    return launch_pdl(packed_attn_kernel<D>, dim3((unsigned)tiles, (unsigned)s.Hkv), dim3(kThreads),
                      L::kSmem, ctx, mQ, mK, mV, a);
}

}  // namespace

cudaError_t launch_packed_attention(const PackedAttnSpec &s, const LaunchCtx &ctx) {
    if (s.D == 64) return launch<64>(s, ctx);
    if (s.D == 128) return launch<128>(s, ctx);
    return cudaErrorInvalidValue;
}

}  // namespace wanvae
