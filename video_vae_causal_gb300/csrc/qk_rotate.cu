// qk_rotate.cu -- the norm of every query and key head and the rotation by the token's
// position, in one pass:
//
//     n = RMS_norm(x; gamma) over the D elements of a head (or x, without gamma)
//     (y_a, y_b) = (n_a cos t - n_b sin t, n_b cos t + n_a sin t)   for each pair (a, b)
//     t = position[axis of the pair] * inv_freq[pair]
//
// RMS_norm as in norm_act.cuh.  The pairs are the first 2 P elements of a head, neighbours
// (2 p, 2 p + 1) or halves apart (p, p + P); the other elements are normed alone.
//
// Angles.  A position of 10^5 times a frequency near one leaves 32-bit floats seven bits of
// the turn, fewer than bf16 has.  A frequency is therefore held as a 64-bit fraction of a
// turn (its whole turns do not matter, positions being whole numbers), and the product with
// the position, modulo 2^64, is the angle's fraction of a turn, its upper half within 2^-31 of a
// turn: one integer multiplication, no table, any position.
//
// A head is D / 8 lanes of four pairs each, so the two elements of a pair are in one
// thread; a warp holds the same head of 256 / D tokens at a time, each lane with the sines and
// cosines of its pairs for all of the token's heads, times the weights: with A = gamma_a cos t
// and so on, a head is
//     y_a = (x_a A_c - x_b B_s) / |x|,  y_b = (x_b B_c + x_a A_s) / |x|
// two elements an instruction (packed fp32).  Tokens, cut into as many pieces of their heads
// as it takes to keep the warps busy, go to the warps in turn.
//
// Sines and cosines of bf16 rows are the fast ones, off by less than 2^-20 (absolute: the
// functions' 2^-21.19 over half a turn, and pi 2^-23 of the angle's rounding and its product
// with pi), 2^-12 of what a result of the pair's size rounds by; fp32 rows take the exact ones,
// 2^-22 off with the angle's rounding.
//
// What bounds it: HBM, behind the chain of a head's sum (four shuffles, a root) with 24 warps a
// multiprocessor: 16384 tokens of 32 + 8 heads of 128 in bf16 take 68.7 us (4.9 TB/s, 0.72 of
// the measured copy rate), 131040 of 6 + 6 heads of 64 turned by three positions 76.1 (5.3 TB/s,
// 0.78).  The other order of the pairs: 67.5 and 79.7; in fp32 131 and 134 (5.1 and 6.0 TB/s;
// floors of 99.5 and 119.5).  Heads one by one, a warp holding several of one token: 77 and
// 100 us; loads through shared memory, eight deep: 82 and 131.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "norm_act.cuh"
#include "ptx.cuh"
#include "seq_ops.h"
#include "seq_ptx.cuh"

namespace wanvae {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 4;    // pieces of work for each warp, where there are few tokens
// Heads of a lane that are loaded together, while those before them are worked on, and
// resident blocks.  16384 tokens of 32 + 8 heads of 128 and 131040 of 6 + 6 of 64, bf16, in us:
// 2 heads and 3 blocks 68.7 and 76.1, 3 and 3 73 and 81, 4 and 2 65 and 92, 4 and 3 79 and 88
// (spills), 6 and 2 69 and 81, 2 and 4 75 and 81.  One pair of numbers for all variants: with 2 and
// 3 each has 80 registers and spills a little (8 to 28 bytes in bf16, 40 to 80 in fp32), with 4 and
// 2 those of bf16 spill nothing, which pays for heads of 128 and costs those of 64.
constexpr int kFlight = 2;
constexpr int kBlocks = 3;

struct RotateArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // bytes
    const float *g_q, *g_k;
    const int32_t *positions;
    int axes, pairs, Hq, Hk;
    int tokens, pieces;      // pieces that a token's heads are cut into
    int64_t warps;
    float most, sqrt_d;      // 1 / eps
    uint64_t turn[64];       // of each pair: 2^64 = a whole turn for each position
    uint8_t axis[64];
};

// Eight elements of a head as they lie in memory: two runs of four (of neighbours, pairs one
// after the other; of halves, the pairs' first elements, then their second), as packed pairs.
template <bool F32>
struct Run {
    using V = uint2;
    static __device__ __forceinline__ void unpack(const V &v, uint64_t &x0, uint64_t &x1) {
        x0 = f32x2(nact_lo(v.x), nact_hi(v.x));
        x1 = f32x2(nact_lo(v.y), nact_hi(v.y));
    }
    static __device__ __forceinline__ V pack(uint64_t x0, uint64_t x1) {
        float a, b, c, d;
        f32x2_split(x0, a, b);
        f32x2_split(x1, c, d);
        return make_uint2(nact_pack(a, b), nact_pack(c, d));
    }
};
template <>
struct Run<true> {
    using V = float4;
    static __device__ __forceinline__ void unpack(const V &v, uint64_t &x0, uint64_t &x1) {
        x0 = f32x2(v.x, v.y);
        x1 = f32x2(v.z, v.w);
    }
    static __device__ __forceinline__ V pack(uint64_t x0, uint64_t x1) {
        float4 v;
        f32x2_split(x0, v.x, v.y);
        f32x2_split(x1, v.z, v.w);
        return v;
    }
};

__device__ __forceinline__ uint64_t swapped(uint64_t v) {
    float a, b;
    f32x2_split(v, a, b);
    return f32x2(b, a);
}

// Sine and cosine of x half turns, x in [-1, 1).
template <bool F32>
__device__ __forceinline__ void half_turns(float x, float &s, float &c) {
    if (F32) {
        sincospif(x, &s, &c);
    } else {
        s = __sinf(x * 3.14159265f);
        c = __cosf(x * 3.14159265f);
    }
}

// N heads of the batch, from its i0-th: norms, rotation, stores.
template <int D, bool F32, bool kNear, int N>
__device__ __forceinline__ void heads(const typename Run<F32>::V (&raw)[kFlight][2], int i0, bool norm,
                                      float most, const uint64_t (&own)[4], const uint64_t (&other)[4],
                                      bool turns, bool there, char *dst, int e0, int e1) {
    using Vec = typename Run<F32>::V;
    constexpr int L = D / 8, ES = F32 ? 4 : 2;
    uint64_t x[N][4];
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        Run<F32>::unpack(raw[i0 + i][0], x[i][0], x[i][1]);
        Run<F32>::unpack(raw[i0 + i][1], x[i][2], x[i][3]);
        f[i] = 1.f;
    }
    if (norm) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint64_t ss = mul_f32x2(x[i][0], x[i][0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) ss = fma_f32x2(x[i][e], x[i][e], ss);
            float rest;
            f32x2_split(ss, f[i], rest);
            f[i] += rest;
        }
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] += __shfl_xor_sync(0xffffffffu, f[i], off);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // 1 / max(|x|, eps); a NaN in a head makes it NaN (it fails the test)
            const float r = rsqrtf(f[i]);
            f[i] = r > most ? most : r;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint64_t f2 = f32x2(f[i], f[i]);
        uint64_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = mul_f32x2(x[i][e], own[e]);
            if (turns)
                y[e] = fma_f32x2(kNear ? swapped(x[i][e]) : x[i][e ^ 2], other[e], y[e]);
            y[e] = mul_f32x2(y[e], f2);
        }
        if (there) {
            char *to = dst + (i0 + i) * (D * ES);
            const Vec v0 = Run<F32>::pack(y[0], y[1]), v1 = Run<F32>::pack(y[2], y[3]);
            if (kNear && !F32) {
                const uint2 w0 = *reinterpret_cast<const uint2 *>(&v0);
                const uint2 w1 = *reinterpret_cast<const uint2 *>(&v1);
                *reinterpret_cast<uint4 *>(to + e0 * ES) = make_uint4(w0.x, w0.y, w1.x, w1.y);
            } else {
                *reinterpret_cast<Vec *>(to + e0 * ES) = v0;
                *reinterpret_cast<Vec *>(to + e1 * ES) = v1;
            }
        }
    }
}

// kNear: the elements of a pair are neighbours.
template <int D, bool F32, bool kNear>
__global__ void __launch_bounds__(kThreads, kBlocks)
qk_rotate_kernel(const __grid_constant__ RotateArgs a) {
    using Vec = typename Run<F32>::V;
    constexpr int L = D / 8, G = 32 / L;  // lanes of a head, tokens of a warp
    constexpr int ES = F32 ? 4 : 2;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
    const int64_t id = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    if (id >= a.warps) return;
    // this lane's two runs (pairs behind the P that turn are the elements behind 2 P, in
    // halves too)
    const int p0 = 4 * sub;
    const bool turns = p0 < a.pairs;
    const int e0 = kNear ? 8 * sub : turns ? p0 : p0 + a.pairs;
    const int e1 = kNear ? 8 * sub + 4 : turns ? p0 + a.pairs : p0 + D / 2;
    const int H = a.Hq + a.Hk;
    const int64_t units = (a.tokens + (int64_t)G - 1) / G * a.pieces;
    for (int64_t u = id; u < units; u += a.warps) {
        const int64_t first = u / a.pieces;  // G tokens, and heads h .. end - 1 of them
        const int piece = (int)(u - first * a.pieces);
        int h = (int)((int64_t)piece * H / a.pieces);
        const int end = (int)((int64_t)(piece + 1) * H / a.pieces);
        const bool there = first * G + grp < a.tokens;
        const int64_t t = min(first * G + grp, (int64_t)a.tokens - 1);
        const char *q = static_cast<const char *>(a.q) + t * a.q_stride;
        const char *k = static_cast<const char *>(a.k) + t * a.k_stride;
        // kFlight heads at a time, of queries or of keys
        auto batch = [&](int at) { return min(kFlight, (at < a.Hq ? min(end, a.Hq) : end) - at); };
        auto load = [&](int at, int n, Vec (&raw)[kFlight][2]) {
            const char *src = at < a.Hq ? q + (int64_t)at * (D * ES)
                                        : k + (int64_t)(at - a.Hq) * (D * ES);
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                if (i >= n) continue;
                if (kNear && !F32) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + i * (D * ES) + e0 * ES);
                    *reinterpret_cast<uint2 *>(&raw[i][0]) = make_uint2(v.x, v.y);
                    *reinterpret_cast<uint2 *>(&raw[i][1]) = make_uint2(v.z, v.w);
                } else {
                    raw[i][0] = *reinterpret_cast<const Vec *>(src + i * (D * ES) + e0 * ES);
                    raw[i][1] = *reinterpret_cast<const Vec *>(src + i * (D * ES) + e1 * ES);
                }
            }
        };
        Vec raw[kFlight][2] = {}, more[kFlight][2] = {};
        int n = batch(h);
        load(h, n, raw);
        float c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = 1.f;
            s[j] = 0.f;
            if (turns) {
                const int64_t pos = __ldg(a.positions + t * a.axes + a.axis[p0 + j]);
                // the upper half, to nearest, as a signed fraction of half a turn
                const uint64_t turn = (uint64_t)pos * a.turn[p0 + j] + 0x80000000ull;
                half_turns<F32>((float)(int32_t)(turn >> 32) * 0x1p-31f, s[j], c[j]);
            }
        }
        uint64_t own[4], other[4];
        int kind = -1;
        while (true) {
            const int next = h + n, n_next = next < end ? batch(next) : 0;
            load(next, n_next, more);
            const bool is_k = h >= a.Hq;
            const float *g = is_k ? a.g_k : a.g_q;
            if (kind != (is_k ? 1 : 0)) {
                kind = is_k ? 1 : 0;
                float w[8], x[8], y[8];
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 v = g ? __ldg(reinterpret_cast<const float4 *>(g + (e ? e1 : e0)))
                                       : make_float4(1.f, 1.f, 1.f, 1.f);
                    const float by = g ? a.sqrt_d : 1.f;
                    w[e] = v.x * by;
                    w[e + 1] = v.y * by;
                    w[e + 2] = v.z * by;
                    w[e + 3] = v.w * by;
                }
                // element e of eight: pair, and whether it is the pair's second
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int pair = kNear ? e / 2 : e % 4, mate = kNear ? e ^ 1 : e ^ 4;
                    const bool second = kNear ? e % 2 : e / 4;
                    x[e] = w[e] * c[pair];
                    y[e] = w[mate] * (second ? s[pair] : -s[pair]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    own[i] = f32x2(x[2 * i], x[2 * i + 1]);
                    other[i] = f32x2(y[2 * i], y[2 * i + 1]);
                }
            }
            char *dst = is_k ? static_cast<char *>(a.k_out) + t * a.k_out_stride +
                                   (int64_t)(h - a.Hq) * (D * ES)
                             : static_cast<char *>(a.q_out) + t * a.q_out_stride +
                                   (int64_t)h * (D * ES);
            // (whole batches without a branch between their heads, whose sums would wait for each
            // other; the rest one by one)
            if (n == kFlight) {
                heads<D, F32, kNear, kFlight>(raw, 0, g != nullptr, a.most, own, other, turns, there,
                                              dst, e0, e1);
            } else {
#pragma unroll
                for (int i = 0; i < kFlight - 1; ++i)
                    if (i < n)
                        heads<D, F32, kNear, 1>(raw, i, g != nullptr, a.most, own, other, turns, there,
                                                dst, e0, e1);
            }
            if (n_next == 0) break;
            h = next;
            n = n_next;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                raw[i][0] = more[i][0];
                raw[i][1] = more[i][1];
            }
        }
    }
}

template <int D, bool F32, bool kNear>
cudaError_t launch(RotateArgs &a, const LaunchCtx &ctx) {
    constexpr int kMaxDev = 64;
    static std::atomic<int> per_sm[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    int occ = per_sm[dev].load(std::memory_order_relaxed);
    if (!occ) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, qk_rotate_kernel<D, F32, kNear>,
                                                          kThreads, 0);
        if (e != cudaSuccess) return e;
        per_sm[dev].store(occ = std::max(1, occ), std::memory_order_relaxed);
    }
    constexpr int G = 256 / D, kWarps = kThreads / 32;
    // whole tokens, where each warp has some; else pieces, of a head at the least
    const int64_t groups = ((int64_t)a.tokens + G - 1) / G, most = (int64_t)ctx.num_sms * occ * kWarps;
    a.pieces = (int)std::min<int64_t>(a.Hq + a.Hk, (kEach * most + groups - 1) / groups);
    a.warps = std::min(groups * a.pieces, most);
    return launch_pdl(qk_rotate_kernel<D, F32, kNear>,
                      dim3((unsigned)((a.warps + kWarps - 1) / kWarps)), dim3(kThreads), 0, ctx, a);
}

template <int D>
cudaError_t pick(RotateArgs &a, bool f32, bool near, const LaunchCtx &ctx) {
    if (f32) return near ? launch<D, true, true>(a, ctx) : launch<D, true, false>(a, ctx);
    return near ? launch<D, false, true>(a, ctx) : launch<D, false, false>(a, ctx);
}

// f radians in turns, without the whole ones, times 2^64, off by less than 2 (f up to 2^20; 1 / (2 pi)
// in two parts): a position of 31 bits then leaves the angle within 2^-31 of a turn.  A negative
// f is its magnitude turned back, as the fraction of a small negative product lies near 1,
// where 53 bits hold 1024 times less of it.
uint64_t fraction_of_turn(double f) {
    const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    const double a = fabs(f), p = a * hi, rest = fma(a, hi, -p) + a * lo;
    const double frac = p - floor(p);  // (exact)
    const uint64_t turn = (uint64_t)(frac * 0x1p64) + (uint64_t)(int64_t)(rest * 0x1p64);
    return f < 0.0 ? 0 - turn : turn;
}

}  // namespace

cudaError_t launch_qk_rotate(const QkRotateSpec &s, const LaunchCtx &ctx) {
    RotateArgs a = {};
    const int es = s.f32 ? 4 : 2;
    a.q = s.q;
    a.k = s.k;
    a.q_out = s.q_out;
    a.k_out = s.k_out;
    a.q_stride = s.q_stride * es;
    a.k_stride = s.k_stride * es;
    a.q_out_stride = s.q_out_stride * es;
    a.k_out_stride = s.k_out_stride * es;
    a.g_q = s.g_q;
    a.g_k = s.g_k;
    a.positions = s.positions;
    a.axes = s.axes;
    a.pairs = s.pairs;
    a.Hq = s.Hq;
    a.Hk = s.Hk;
    a.tokens = s.tokens;
    a.most = 1.f / s.eps;    // (infinite for none)
    a.sqrt_d = sqrtf((float)s.D);
    for (int p = 0; p < s.pairs; ++p) {
        a.turn[p] = fraction_of_turn(s.inv_freq[p]);
        a.axis[p] = s.axis[p];
    }
    if (s.D == 64) return pick<64>(a, s.f32, s.near, ctx);
    if (s.D == 128) return pick<128>(a, s.f32, s.near, ctx);
    return cudaErrorInvalidValue;
}

}  // namespace wanvae
