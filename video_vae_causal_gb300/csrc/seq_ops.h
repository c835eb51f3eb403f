// seq_ops.h -- internal launch interface between the C ABI (seq_api.cu) and
// the sequence operators' kernels: attention over packed sequences
// (packed_attn.cu), the paged key-value cache (kv_cache.cu), attention of one
// token over it (paged_attn.cu) and the gated residual with the norms around
// it (gated_norm.cu).  Not installed, not exported.
#pragma once

#include "kernels.h"

namespace wanvae {

// softmax(scale q k^T) v of packed sequences: sequence s holds the queries
// [cu_q[s], cu_q[s+1]) and the keys [cu_k[s], cu_k[s+1]).  Strides are in
// elements between tokens; heads are D apart.
struct PackedAttnSpec {
    const void *q, *k, *v;  // bf16 [total_q][Hq][D], [total_k][Hkv][D] twice
    void *out;              // bf16 [total_q][Hq][D]
    int64_t q_stride, k_stride, v_stride, out_stride;
    const int32_t *cu_q, *cu_k;
    int n_seq, total_q, total_k;
    int Hq, Hkv, D;  // D = 64 or 128
    float scale;
    bool causal;
};
cudaError_t launch_packed_attention(const PackedAttnSpec &s, const LaunchCtx &ctx);

// A paged cache: pages of `page` (1 << log2_page) rows for each kv head,
// [n_pages][H][page][D], 16-bit or e4m3 with one E8M0 scale per row.
struct KvCacheSpec {
    void *k, *v;
    uint8_t *k_exp, *v_exp;  // [n_pages][H][page], e4m3 only
    int n_pages, log2_page, H, D;
    bool e4m3;
};
// Rows cu_new[s] .. cu_new[s+1] - 1 of k and v (row s alone where cu_new is
// NULL) become the last positions of sequence s, of length lens[s] with them.
cudaError_t launch_kv_append(const KvCacheSpec &c, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const int32_t *lens, const int32_t *table,
                             int max_pages, const int32_t *cu_new, int n_seq, int total,
                             const LaunchCtx &ctx);
// Positions 0 .. of every sequence to rows cu[s] .. cu[s+1] - 1 of k and v.
cudaError_t launch_kv_gather(const KvCacheSpec &c, const int32_t *table, int max_pages,
                             const int32_t *cu, int n_seq, int total, void *k, int64_t k_stride,
                             void *v, int64_t v_stride, const LaunchCtx &ctx);

// One query token for each sequence against its cached positions.
size_t paged_attention_workspace(int Hq, int Hkv, int D);
cudaError_t launch_paged_attention(const KvCacheSpec &c, const void *q, int64_t q_stride,
                                   const int32_t *lens, const int32_t *table, int max_pages,
                                   int n_seq, int Hq, float scale, void *out, int64_t out_stride,
                                   void *workspace, const LaunchCtx &ctx);

// y = x + s gate (.) RMS_norm(f; g_post), n = RMS_norm(y; g_pre); see gated_norm.cu.
struct GatedNormSpec {
    const void *x, *f;
    const float *g_post, *gate, *g_pre;  // each may be NULL (n too, with g_pre)
    void *y, *n;
    int64_t tokens, per_gate;
    int C;
    float scale, eps;
    bool f32;
};
cudaError_t launch_gated_norm(const GatedNormSpec &s, const LaunchCtx &ctx);

}  // namespace wanvae
