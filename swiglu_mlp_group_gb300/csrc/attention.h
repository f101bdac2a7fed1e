// attention.h -- what the attention entry points (attention_api.cu) pass to
// their kernels.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace ck {

// bf16 data is passed as its 16-bit patterns.
struct NormRopeArgs {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    int64_t ldq, ldk, ldqo, ldko;
    const void *wq, *wk;  // null: no norm
    const float *cos_sin;
    const int32_t *positions;
    int64_t T, max_pos;
    int Hq, Hk, D, rot;  // rot 0: no rotation
    float eps, inv_d;
    bool w_f32;
    unsigned int *status;
};
cudaError_t launch_qk_norm_rope(const NormRopeArgs &a, bool interleaved, const LaunchCtx &ctx);

struct KvAppendArgs {
    const uint16_t *k, *v;
    uint16_t *k_cache, *v_cache;
    int64_t ldk, ldv;
    const void *wk;
    const float *cos_sin;
    const int32_t *positions;
    const int64_t *slots;
    int64_t T, max_pos, pages, page_size;
    int Hkv, D, rot;
    float eps, inv_d;
    bool w_f32;
    unsigned int *status;
};
cudaError_t launch_kv_append(const KvAppendArgs &a, bool interleaved, const LaunchCtx &ctx);

// Attention of B x Lq query tokens over keys in two places: a prefix that
// every sequence sees, and each sequence's own keys.
//   paged: both in pages of a cache [pages, Hkv, page_size, D].
//   dense: own keys only, k and v [B * Lk tokens] with leading dimensions.
struct AttentionArgs {
    const uint16_t *q;
    uint16_t *out;
    int64_t ldq, ldo;
    int64_t B, Lq;
    int Hq, Hkv, G, D;
    bool ragged;  // lengths of own keys may differ; the workspace is sized for that
    const uint16_t *k, *v;  // the cache, or the dense states
    int64_t ldk, ldv;       // dense
    int64_t pages;          // paged; 0: dense
    int page_size;
    const int32_t *prefix_pages;
    int64_t prefix_len;
    const int32_t *block_table;
    int64_t table_stride;
    const int32_t *lens;  // null: max_len for every sequence
    int64_t max_len;      // longest own length (dense: Lk)
    bool causal;          // own key j is seen by query i when j <= len - Lq + i
    float scale;
    void *ws;
};
// kAttentionTooLarge: more key tiles over all heads and sequences than a call
// can count (2^30 of 128 keys).
constexpr size_t kAttentionTooLarge = ~size_t{0};
size_t attention_workspace_bytes(const AttentionArgs &a);
cudaError_t launch_attention(const AttentionArgs &a, const LaunchCtx &ctx);

}  // namespace ck
