// seq_api.cu -- the C ABI of the sequence operators declared in
// include/wanvae.h: argument checks, then one launch (two for attention over
// the cache).  What only the device knows (lengths, offsets, pages) is checked
// by the kernels.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/wanvae.h"
#include "seq_ops.h"

using namespace wanvae;

namespace {

bool misaligned(const void *p, uintptr_t to = 16) {
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Bytes from the first to the last element of n tokens, `stride` elements apart.
size_t span(int64_t n, int64_t stride, int64_t width) {
    return n < 1 ? 0 : ((size_t)(n - 1) * stride + width) * 2;
}

// Bytes of n int32 values.
size_t ints(int64_t n) { return (size_t)n * 4; }

// Whether rows of two tensors collide: n tokens of `width` elements each, which may
// lie side by side in one buffer where their strides are equal.
bool rows_collide(const void *a, int64_t a_stride, const void *b, int64_t b_stride, int64_t n,
                  int64_t width) {
    if (!overlap(a, span(n, a_stride, width), b, span(n, b_stride, width))) return false;
    if (a_stride != b_stride) return true;
    const int64_t s = a_stride * 2, w = width * 2;
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    const int64_t off = (d % s + s) % s;  // from a row of a to the next row of b
    return off < w || off > s - w;
}

wanvae_status from_cuda(cudaError_t e) { return e == cudaSuccess ? WANVAE_OK : WANVAE_ERR_CUDA; }

// Tokens and widths as the kernels count them (int32), strides within a tensor
// map's reach.
constexpr int64_t kMaxStride = int64_t(1) << 36;
bool count_ok(int64_t n) { return n >= 0 && n < INT32_MAX; }
bool stride_ok(int64_t stride, int64_t width) {
    return stride >= width && stride % 8 == 0 && stride < kMaxStride;
}

wanvae_status check_cache(const wanvae_kv_cache *c, KvCacheSpec &s) {
    if (!c || !c->k || !c->v) return WANVAE_ERR_INVALID_ARG;
    if (c->dt != WANVAE_BF16 && c->dt != WANVAE_E4M3) return WANVAE_ERR_INVALID_ARG;
    s.e4m3 = c->dt == WANVAE_E4M3;
    if (s.e4m3 != (c->k_exp != nullptr) || s.e4m3 != (c->v_exp != nullptr))
        return WANVAE_ERR_INVALID_ARG;
    if (c->n_pages < 1 || !count_ok(c->n_pages) || c->n_kv_heads < 1 || c->page_size < 1)
        return WANVAE_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return WANVAE_ERR_UNSUPPORTED;
    if (c->n_kv_heads > 4096) return WANVAE_ERR_UNSUPPORTED;
    s.log2_page = 4;
    while (s.log2_page < 10 && (int64_t(1) << s.log2_page) < c->page_size) ++s.log2_page;
    if ((int64_t(1) << s.log2_page) != c->page_size) return WANVAE_ERR_UNSUPPORTED;
    if (misaligned(c->k) || misaligned(c->v) || misaligned(c->k_exp) || misaligned(c->v_exp))
        return WANVAE_ERR_MISALIGNED;
    s.k = c->k;
    s.v = c->v;
    s.k_exp = c->k_exp;
    s.v_exp = c->v_exp;
    s.n_pages = (int)c->n_pages;
    s.H = (int)c->n_kv_heads;
    s.D = (int)c->head_dim;
    const size_t rows = ((size_t)s.n_pages * s.H) << s.log2_page;
    const size_t bytes = rows * s.D * (s.e4m3 ? 1 : 2);
    if (overlap(s.k, bytes, s.v, bytes) || (s.e4m3 && overlap(s.k_exp, rows, s.v_exp, rows)))
        return WANVAE_ERR_INVALID_ARG;
    return WANVAE_OK;
}

size_t cache_bytes(const KvCacheSpec &s) {
    return (((size_t)s.n_pages * s.H) << s.log2_page) * s.D * (s.e4m3 ? 1 : 2);
}

// Whether [p, p + n) touches the cache's elements or scales.
bool touches(const KvCacheSpec &s, const void *p, size_t n) {
    const size_t b = cache_bytes(s), rows = ((size_t)s.n_pages * s.H) << s.log2_page;
    return overlap(p, n, s.k, b) || overlap(p, n, s.v, b) ||
           (s.e4m3 && (overlap(p, n, s.k_exp, rows) || overlap(p, n, s.v_exp, rows)));
}

}  // namespace

extern "C" {

wanvae_status wanvae_packed_attention(const void *q, int64_t q_stride, const void *k,
                                      int64_t k_stride, const void *v, int64_t v_stride, void *out,
                                      int64_t out_stride, const int32_t *cu_q,
                                      const int32_t *cu_k, int64_t n_seq, int64_t total_q,
                                      int64_t total_k, int64_t n_heads, int64_t n_kv_heads,
                                      int64_t head_dim, float scale, int causal,
                                      wanvae_stream stream) {
    if (!q || !k || !v || !out || !cu_q || !cu_k) return WANVAE_ERR_INVALID_ARG;
    if (n_seq < 1 || total_q < 1 || total_k < 1 || !count_ok(n_seq) || !count_ok(total_q) ||
        !count_ok(total_k))
        return WANVAE_ERR_INVALID_ARG;
    if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads) return WANVAE_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY)) return WANVAE_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return WANVAE_ERR_UNSUPPORTED;
    const int64_t G = n_heads / n_kv_heads;
    if (n_kv_heads > 4096 || G > 128) return WANVAE_ERR_UNSUPPORTED;
    // pairs of tiles of 128 / G queries, one more a sequence, of every kv head in one grid
    if ((total_q / (2 * (128 / G)) + 1 + n_seq) * n_kv_heads > INT32_MAX)
        return WANVAE_ERR_UNSUPPORTED;
    const int64_t wq = n_heads * head_dim, wk = n_kv_heads * head_dim;
    if (!stride_ok(q_stride, wq) || !stride_ok(out_stride, wq) || !stride_ok(k_stride, wk) ||
        !stride_ok(v_stride, wk))
        return WANVAE_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(out) ||
        misaligned(cu_q, 4) || misaligned(cu_k, 4))
        return WANVAE_ERR_MISALIGNED;
    const size_t ob = span(total_q, out_stride, wq);
    if (overlap(out, ob, q, span(total_q, q_stride, wq)) ||
        overlap(out, ob, k, span(total_k, k_stride, wk)) ||
        overlap(out, ob, v, span(total_k, v_stride, wk)) ||
        overlap(out, ob, cu_q, ints(n_seq + 1)) || overlap(out, ob, cu_k, ints(n_seq + 1)))
        return WANVAE_ERR_INVALID_ARG;
    PackedAttnSpec s;
    s.q = q;
    s.k = k;
    s.v = v;
    s.out = out;
    s.q_stride = q_stride;
    s.k_stride = k_stride;
    s.v_stride = v_stride;
    s.out_stride = out_stride;
    s.cu_q = cu_q;
    s.cu_k = cu_k;
    s.n_seq = (int)n_seq;
    s.total_q = (int)total_q;
    s.total_k = (int)total_k;
    s.Hq = (int)n_heads;
    s.Hkv = (int)n_kv_heads;
    s.D = (int)head_dim;
    s.scale = scale;
    s.causal = causal != 0;
    LaunchCtx ctx;
    if (!make_launch_ctx(ctx, stream)) return WANVAE_ERR_CUDA;
    count_launches(1);
    return from_cuda(launch_packed_attention(s, ctx));
}

wanvae_status wanvae_kv_cache_append(const wanvae_kv_cache *cache, const void *k,
                                     int64_t k_stride, const void *v, int64_t v_stride,
                                     const int32_t *lens, const int32_t *page_table,
                                     int64_t max_pages, const int32_t *cu_new, int64_t n_seq,
                                     int64_t total, wanvae_stream stream) {
    KvCacheSpec s;
    const wanvae_status st = check_cache(cache, s);
    if (st != WANVAE_OK) return st;
    if (!k || !v || !lens || !page_table) return WANVAE_ERR_INVALID_ARG;
    if (n_seq < 1 || !count_ok(n_seq) || total < 1 || !count_ok(total) || max_pages < 1 ||
        !count_ok(max_pages))
        return WANVAE_ERR_INVALID_ARG;
    if (!cu_new && total != n_seq) return WANVAE_ERR_INVALID_ARG;
    const int64_t w = (int64_t)s.H * s.D;
    if (!stride_ok(k_stride, w) || !stride_ok(v_stride, w)) return WANVAE_ERR_INVALID_ARG;
    if (misaligned(k) || misaligned(v) || misaligned(lens, 4) || misaligned(page_table, 4) ||
        misaligned(cu_new, 4))
        return WANVAE_ERR_MISALIGNED;
    if (touches(s, k, span(total, k_stride, w)) || touches(s, v, span(total, v_stride, w)) ||
        touches(s, lens, ints(n_seq)) || touches(s, page_table, ints(n_seq * max_pages)) ||
        (cu_new && touches(s, cu_new, ints(n_seq + 1))))
        return WANVAE_ERR_INVALID_ARG;
    LaunchCtx ctx;
    if (!make_launch_ctx(ctx, stream)) return WANVAE_ERR_CUDA;
    count_launches(1);
    return from_cuda(launch_kv_append(s, k, k_stride, v, v_stride, lens, page_table,
                                      (int)max_pages, cu_new, (int)n_seq, (int)total, ctx));
}

wanvae_status wanvae_kv_cache_gather(const wanvae_kv_cache *cache, const int32_t *page_table,
                                     int64_t max_pages, const int32_t *cu, int64_t n_seq,
                                     int64_t total, void *k, int64_t k_stride, void *v,
                                     int64_t v_stride, wanvae_stream stream) {
    KvCacheSpec s;
    const wanvae_status st = check_cache(cache, s);
    if (st != WANVAE_OK) return st;
    if (!k || !v || !cu || !page_table) return WANVAE_ERR_INVALID_ARG;
    if (n_seq < 1 || !count_ok(n_seq) || total < 1 || !count_ok(total) || max_pages < 1 ||
        !count_ok(max_pages))
        return WANVAE_ERR_INVALID_ARG;
    const int64_t w = (int64_t)s.H * s.D;
    if (!stride_ok(k_stride, w) || !stride_ok(v_stride, w)) return WANVAE_ERR_INVALID_ARG;
    if (misaligned(k) || misaligned(v) || misaligned(cu, 4) || misaligned(page_table, 4))
        return WANVAE_ERR_MISALIGNED;
    const size_t kb = span(total, k_stride, w), vb = span(total, v_stride, w);
    const size_t cb = ints(n_seq + 1), tb = ints(n_seq * max_pages);
    if (rows_collide(k, k_stride, v, v_stride, total, w) || touches(s, k, kb) ||
        touches(s, v, vb) || overlap(k, kb, cu, cb) || overlap(v, vb, cu, cb) ||
        overlap(k, kb, page_table, tb) || overlap(v, vb, page_table, tb))
        return WANVAE_ERR_INVALID_ARG;
    LaunchCtx ctx;
    if (!make_launch_ctx(ctx, stream)) return WANVAE_ERR_CUDA;
    count_launches(1);
    return from_cuda(launch_kv_gather(s, page_table, (int)max_pages, cu, (int)n_seq, (int)total, k,
                                      k_stride, v, v_stride, ctx));
}

size_t wanvae_paged_attention_workspace_size(int64_t n_heads, int64_t n_kv_heads,
                                             int64_t head_dim) {
    if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || n_kv_heads > 4096 ||
        n_heads > 65535 || (head_dim != 64 && head_dim != 128))
        return 0;
    return (paged_attention_workspace((int)n_heads, (int)n_kv_heads, (int)head_dim) + 255) &
           ~size_t(255);
}

wanvae_status wanvae_paged_attention(const void *q, int64_t q_stride,
                                     const wanvae_kv_cache *cache, const int32_t *lens,
                                     const int32_t *page_table, int64_t max_pages, int64_t n_seq,
                                     int64_t n_heads, float scale, void *out, int64_t out_stride,
                                     void *workspace, size_t ws_bytes, wanvae_stream stream) {
    KvCacheSpec s;
    const wanvae_status st = check_cache(cache, s);
    if (st != WANVAE_OK) return st;
    if (!q || !out || !lens || !page_table) return WANVAE_ERR_INVALID_ARG;
    if (n_seq < 1 || n_seq > 65535 || max_pages < 1 || !count_ok(max_pages))
        return WANVAE_ERR_INVALID_ARG;
    if (n_heads < 1 || n_heads % s.H) return WANVAE_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY)) return WANVAE_ERR_INVALID_ARG;
    const size_t need = wanvae_paged_attention_workspace_size(n_heads, s.H, s.D);
    if (need == 0) return WANVAE_ERR_UNSUPPORTED;
    // rows of a sequence, and units of 64 rows that the page table could hold (two more
    // an item, an item for each kv head and 8 query heads), are counted in 32 bits
    const int64_t units = ((max_pages << s.log2_page) + 63) / 64 + 2;
    const int64_t items = n_seq * s.H * ((n_heads / s.H + 7) / 8);
    if (units > INT32_MAX / 256 || units * items > INT32_MAX) return WANVAE_ERR_UNSUPPORTED;
    const int64_t w = n_heads * s.D;
    if (!stride_ok(q_stride, w) || !stride_ok(out_stride, w)) return WANVAE_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(out) || misaligned(lens, 4) || misaligned(page_table, 4))
        return WANVAE_ERR_MISALIGNED;
    if (!workspace || ws_bytes < need) return WANVAE_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return WANVAE_ERR_MISALIGNED;
    const size_t qb = span(n_seq, q_stride, w), ob = span(n_seq, out_stride, w);
    const size_t lb = ints(n_seq), tb = ints(n_seq * max_pages);
    if (overlap(q, qb, out, ob) || touches(s, out, ob) || touches(s, workspace, need) ||
        overlap(workspace, need, q, qb) || overlap(workspace, need, out, ob) ||
        overlap(out, ob, lens, lb) || overlap(out, ob, page_table, tb) ||
        overlap(workspace, need, lens, lb) || overlap(workspace, need, page_table, tb))
        return WANVAE_ERR_INVALID_ARG;
    LaunchCtx ctx;
    if (!make_launch_ctx(ctx, stream)) return WANVAE_ERR_CUDA;
    return from_cuda(launch_paged_attention(s, q, q_stride, lens, page_table, (int)max_pages,
                                            (int)n_seq, (int)n_heads, scale, out, out_stride,
                                            workspace, ctx));
}

wanvae_status wanvae_gated_residual_norm(const void *x, const void *f, const float *gamma_post,
                                         const float *gate, int64_t tokens_per_gate,
                                         const float *gamma_pre, void *y, void *n,
                                         wanvae_dtype dt, int64_t n_tokens, int64_t C,
                                         float residual_scale, float eps, wanvae_stream stream) {
    if (!x || !f || !y || (gamma_pre != nullptr) != (n != nullptr)) return WANVAE_ERR_INVALID_ARG;
    if (dt != WANVAE_BF16 && dt != WANVAE_F32) return WANVAE_ERR_INVALID_ARG;
    if (n_tokens < 1 || n_tokens >= INT32_MAX || C < 16 || C % 16 || C > 4096)
        return WANVAE_ERR_INVALID_ARG;
    if (gate && tokens_per_gate < 1) return WANVAE_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !(residual_scale > -INFINITY && residual_scale < INFINITY))
        return WANVAE_ERR_INVALID_ARG;
    if (misaligned(x) || misaligned(f) || misaligned(gamma_post) || misaligned(gate) ||
        misaligned(gamma_pre) || misaligned(y) || misaligned(n))
        return WANVAE_ERR_MISALIGNED;
    const size_t bytes = (size_t)n_tokens * C * (dt == WANVAE_F32 ? 4 : 2);
    const size_t row = (size_t)C * 4;
    const size_t gates = gate ? (size_t)((n_tokens - 1) / tokens_per_gate + 1) * row : 0;
    for (const void *o : {static_cast<const void *>(y), static_cast<const void *>(n)})
        if (o && (overlap(gamma_post, gamma_post ? row : 0, o, bytes) ||
                  overlap(gate, gates, o, bytes) || overlap(gamma_pre, gamma_pre ? row : 0, o, bytes)))
            return WANVAE_ERR_INVALID_ARG;
    if (overlap(x, bytes, y, bytes) || overlap(f, bytes, y, bytes) ||
        (n && (overlap(x, bytes, n, bytes) || overlap(f, bytes, n, bytes) ||
               overlap(y, bytes, n, bytes))))
        return WANVAE_ERR_INVALID_ARG;
    GatedNormSpec s;
    s.x = x;
    s.f = f;
    s.g_post = gamma_post;
    s.gate = gate;
    s.g_pre = gamma_pre;
    s.y = y;
    s.n = n;
    s.tokens = n_tokens;
    s.per_gate = gate ? tokens_per_gate : n_tokens;
    s.C = (int)C;
    s.scale = residual_scale;
    s.eps = eps;
    s.f32 = dt == WANVAE_F32;
    LaunchCtx ctx;
    if (!make_launch_ctx(ctx, stream)) return WANVAE_ERR_CUDA;
    count_launches(1);
    return from_cuda(launch_gated_norm(s, ctx));
}

}  // extern "C"
