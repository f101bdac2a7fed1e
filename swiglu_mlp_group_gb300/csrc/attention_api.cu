// attention_api.cu -- the C ABI of the attention operators (include/ck.h):
// argument validation and launches, nothing else.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention.h"
#include "ck.h"
#include "internal.h"
#include "trace.h"

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxHeads = 1 << 16;
constexpr int64_t kMaxKeys = int64_t{1} << 30;  // longest prefix, sequence or encoder length

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
const uint16_t *bits(const void *p) { return static_cast<const uint16_t *>(p); }
uint16_t *bits(void *p) { return static_cast<uint16_t *>(p); }

ck_status device(unsigned int **status) { return static_cast<ck_status>(ck::device_ready_status(status)); }

ck::LaunchCtx context(ck_stream_t stream, unsigned int *status) {
    ck::LaunchCtx c;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    c.status = status;
    c.timeout_ns = ck::wait_timeout_ns();
    c.pdl = true;
    return c;
}

// Tokens of `heads` heads of D elements, ld elements apart.
bool token_rows(int64_t ld, int64_t heads, int64_t D) { return ld % 8 == 0 && ld >= heads * D && ld <= kMaxRows; }

// The norm and rotation arguments that qk_norm_rope and kv_append share.
ck_status check_norm_rope(int64_t T, int64_t D, ck_dtype wdt, float eps, const float *cos_sin, int64_t max_pos,
                          int64_t rot_dim, ck_rope_mode mode, const int32_t *positions) {
    if ((rot_dim != 0) != (cos_sin != nullptr) || (rot_dim != 0 && !positions)) return CK_ERR_NULL;
    if (mode != CK_ROPE_HALF && mode != CK_ROPE_INTERLEAVED) return CK_ERR_INVALID;
    if (!isfinite(eps) || eps < 0.f) return CK_ERR_INVALID;
    if (wdt != CK_F32 && wdt != CK_BF16) return CK_ERR_DTYPE;
    if (T < 1 || T > kMaxRows || D < 16 || D > 256 || D % 16 != 0) return CK_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0) return CK_ERR_SHAPE;
    if (rot_dim != 0 && (max_pos < 1 || max_pos > kMaxRows)) return CK_ERR_SHAPE;
    if (cos_sin && !aligned16(cos_sin)) return CK_ERR_ALIGN;
    return CK_OK;
}

// Sizes of an attention call.
bool attention_sizes(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D) {
    if (B < 1 || Lq < 1 || Hkv < 1 || Hq < 1 || Hkv > kMaxHeads || Hq > kMaxHeads) return false;
    if (Hq % Hkv != 0 || Hq / Hkv > 128 || (D != 64 && D != 128)) return false;
    return B <= kMaxRows && Lq <= kMaxRows && B * Lq <= kMaxRows && B * Lq * Hq <= kMaxRows;
}

ck::AttentionArgs attention_sizes_only(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D) {
    ck::AttentionArgs a = {};
    a.ragged = true;
    a.B = B, a.Lq = Lq;
    a.Hq = static_cast<int>(Hq), a.Hkv = static_cast<int>(Hkv), a.G = static_cast<int>(Hq / Hkv);
    a.D = static_cast<int>(D);
    return a;
}

ck::AttentionArgs prefix_sizes(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix_len,
                               int64_t max_seq_len) {
    ck::AttentionArgs a = attention_sizes_only(B, Lq, Hq, Hkv, D);
    a.prefix_len = prefix_len, a.max_len = max_seq_len;
    a.causal = true;
    a.pages = 1;  // paged
    return a;
}

ck::AttentionArgs cross_sizes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t D) {
    ck::AttentionArgs a = attention_sizes_only(B, Lq, Hq, Hkv, D);
    a.max_len = Lk;
    return a;
}

ck_status run_attention(ck::AttentionArgs &a, const void *q, int64_t ldq, void *out, int64_t ldo, float scale,
                        void *ws, size_t ws_bytes, ck_stream_t stream) {
    const size_t need = ck::attention_workspace_bytes(a);
    if (need == ck::kAttentionTooLarge) return CK_ERR_SHAPE;
    if (need > 0 && (!ws || ws_bytes < need)) return CK_ERR_WORKSPACE;
    if (need > 0 && !aligned16(ws)) return CK_ERR_ALIGN;
    unsigned int *status = nullptr;
    if (ck_status st = device(&status); st != CK_OK) return st;
    a.q = bits(q), a.ldq = ldq, a.out = bits(out), a.ldo = ldo;
    a.scale = scale, a.ws = ws;
    return ck::launch_attention(a, context(stream, status)) == cudaSuccess ? CK_OK : CK_ERR_CUDA;
}

}  // namespace

extern "C" {

CK_API ck_status ck_qk_norm_rope(const void *q, int64_t ldq, int64_t Hq, const void *wq, const void *k,
                                 int64_t ldk, int64_t Hk, const void *wk, ck_dtype wdt, int64_t T,
                                 int64_t D, float eps, const float *cos_sin, int64_t max_pos,
                                 int64_t rot_dim, ck_rope_mode mode, const int32_t *positions,
                                 void *q_out, int64_t ldqo, void *k_out, int64_t ldko,
                                 ck_stream_t stream) {
    CK_TRACE("ck_qk_norm_rope");
    if (!q || !q_out || (k != nullptr) != (Hk != 0) || (k != nullptr) != (k_out != nullptr)) return CK_ERR_NULL;
    if (ck_status st = check_norm_rope(T, D, wdt, eps, cos_sin, max_pos, rot_dim, mode, positions); st != CK_OK)
        return st;
    if (Hq < 1 || Hk < 0 || Hq > kMaxHeads || Hk > kMaxHeads || T * (Hq + Hk) > kMaxRows) return CK_ERR_SHAPE;
    if (!token_rows(ldq, Hq, D) || !token_rows(ldqo, Hq, D)) return CK_ERR_SHAPE;
    if (k && (!token_rows(ldk, Hk, D) || !token_rows(ldko, Hk, D))) return CK_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out) || !aligned16(wq) || !aligned16(wk))
        return CK_ERR_ALIGN;
    unsigned int *status = nullptr;
    if (ck_status st = device(&status); st != CK_OK) return st;
    ck::NormRopeArgs a = {};
    a.q = bits(q), a.k = bits(k), a.q_out = bits(q_out), a.k_out = bits(k_out);
    a.ldq = ldq, a.ldk = ldk, a.ldqo = ldqo, a.ldko = ldko;
    a.wq = wq, a.wk = wk, a.w_f32 = wdt == CK_F32;
    a.cos_sin = cos_sin, a.positions = positions, a.max_pos = max_pos;
    a.T = T, a.Hq = static_cast<int>(Hq), a.Hk = static_cast<int>(Hk);
    a.D = static_cast<int>(D), a.rot = static_cast<int>(rot_dim);
    a.eps = eps, a.inv_d = 1.f / static_cast<float>(D), a.status = status;
    return ck::launch_qk_norm_rope(a, mode == CK_ROPE_INTERLEAVED, context(stream, status)) == cudaSuccess
               ? CK_OK
               : CK_ERR_CUDA;
}

CK_API ck_status ck_kv_append(const void *k, int64_t ldk, const void *v, int64_t ldv, int64_t T,
                              int64_t Hkv, int64_t D, const void *wk, ck_dtype wdt, float eps,
                              const float *cos_sin, int64_t max_pos, int64_t rot_dim,
                              ck_rope_mode mode, const int32_t *positions, const int64_t *slots,
                              void *k_cache, void *v_cache, int64_t pages, int64_t page_size,
                              ck_stream_t stream) {
    CK_TRACE("ck_kv_append");
    if (!k || !v || !slots || !k_cache || !v_cache) return CK_ERR_NULL;
    if (ck_status st = check_norm_rope(T, D, wdt, eps, cos_sin, max_pos, rot_dim, mode, positions); st != CK_OK)
        return st;
    if (Hkv < 1 || Hkv > kMaxHeads || T * Hkv > kMaxRows) return CK_ERR_SHAPE;
    if (pages < 1 || pages > kMaxRows || page_size < 1 || page_size > 65536) return CK_ERR_SHAPE;
    if (!token_rows(ldk, Hkv, D) || !token_rows(ldv, Hkv, D)) return CK_ERR_SHAPE;
    if (!aligned16(k) || !aligned16(v) || !aligned16(wk) || !aligned16(k_cache) || !aligned16(v_cache))
        return CK_ERR_ALIGN;
    unsigned int *status = nullptr;
    if (ck_status st = device(&status); st != CK_OK) return st;
    ck::KvAppendArgs a = {};
    a.k = bits(k), a.v = bits(v), a.k_cache = bits(k_cache), a.v_cache = bits(v_cache);
    a.ldk = ldk, a.ldv = ldv, a.wk = wk, a.w_f32 = wdt == CK_F32;
    a.cos_sin = cos_sin, a.positions = positions, a.slots = slots, a.max_pos = max_pos;
    a.T = T, a.pages = pages, a.page_size = page_size;
    a.Hkv = static_cast<int>(Hkv), a.D = static_cast<int>(D), a.rot = static_cast<int>(rot_dim);
    a.eps = eps, a.inv_d = 1.f / static_cast<float>(D), a.status = status;
    return ck::launch_kv_append(a, mode == CK_ROPE_INTERLEAVED, context(stream, status)) == cudaSuccess
               ? CK_OK
               : CK_ERR_CUDA;
}

CK_API size_t ck_prefix_attention_workspace_bytes(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D,
                                                  int64_t prefix_len, int64_t max_seq_len) {
    if (!attention_sizes(B, Lq, Hq, Hkv, D) || prefix_len < 0 || max_seq_len < 0 || prefix_len > kMaxKeys ||
        max_seq_len > kMaxKeys)
        return 0;
    const size_t n = ck::attention_workspace_bytes(prefix_sizes(B, Lq, Hq, Hkv, D, prefix_len, max_seq_len));
    return n == ck::kAttentionTooLarge ? 0 : n;
}

CK_API ck_status ck_prefix_attention(const void *q, int64_t ldq, int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv,
                                     int64_t D, const void *k_cache, const void *v_cache, int64_t pages,
                                     int64_t page_size, const int32_t *prefix_pages, int64_t prefix_len,
                                     const int32_t *block_table, int64_t table_stride,
                                     const int32_t *seq_lens, int64_t max_seq_len, float scale, void *out,
                                     int64_t ldo, void *ws, size_t ws_bytes, ck_stream_t stream) {
    CK_TRACE("ck_prefix_attention");
    if (!q || !out || !k_cache || !v_cache) return CK_ERR_NULL;
    if ((prefix_len > 0 && !prefix_pages) || (max_seq_len > 0 && (!block_table || !seq_lens))) return CK_ERR_NULL;
    if (!(scale > 0.f) || !isfinite(scale)) return CK_ERR_INVALID;
    if (!attention_sizes(B, Lq, Hq, Hkv, D)) return CK_ERR_SHAPE;
    if (!token_rows(ldq, Hq, D) || !token_rows(ldo, Hq, D)) return CK_ERR_SHAPE;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return CK_ERR_SHAPE;
    if (pages < 1 || pages > kMaxRows || pages * page_size > kMaxRows || pages * page_size * Hkv > kMaxRows)
        return CK_ERR_SHAPE;
    if (prefix_len < 0 || max_seq_len < 0 || prefix_len > kMaxKeys || max_seq_len > kMaxKeys) return CK_ERR_SHAPE;
    if (max_seq_len > 0 && (table_stride < 1 || table_stride > kMaxRows || max_seq_len > table_stride * page_size))
        return CK_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache)) return CK_ERR_ALIGN;
    ck::AttentionArgs a = prefix_sizes(B, Lq, Hq, Hkv, D, prefix_len, max_seq_len);
    a.k = bits(k_cache), a.v = bits(v_cache), a.pages = pages, a.page_size = static_cast<int>(page_size);
    a.prefix_pages = prefix_pages, a.block_table = block_table, a.table_stride = table_stride;
    a.lens = seq_lens;
    return run_attention(a, q, ldq, out, ldo, scale, ws, ws_bytes, stream);
}

CK_API size_t ck_cross_attention_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv,
                                                 int64_t D) {
    if (!attention_sizes(B, Lq, Hq, Hkv, D) || Lk < 0 || Lk > kMaxKeys || B * Lk > kMaxRows) return 0;
    const size_t n = ck::attention_workspace_bytes(cross_sizes(B, Lq, Lk, Hq, Hkv, D));
    return n == ck::kAttentionTooLarge ? 0 : n;
}

CK_API ck_status ck_cross_attention(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                                    int64_t ldv, int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv,
                                    int64_t D, const int32_t *kv_lens, float scale, void *out, int64_t ldo,
                                    void *ws, size_t ws_bytes, ck_stream_t stream) {
    CK_TRACE("ck_cross_attention");
    if (!q || !out || (Lk > 0 && (!k || !v))) return CK_ERR_NULL;
    if (!(scale > 0.f) || !isfinite(scale)) return CK_ERR_INVALID;
    if (!attention_sizes(B, Lq, Hq, Hkv, D)) return CK_ERR_SHAPE;
    if (Lk < 0 || Lk > kMaxKeys || B * Lk > kMaxRows) return CK_ERR_SHAPE;
    if (!token_rows(ldq, Hq, D) || !token_rows(ldo, Hq, D)) return CK_ERR_SHAPE;
    if (Lk > 0 && (!token_rows(ldk, Hkv, D) || !token_rows(ldv, Hkv, D))) return CK_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(out) || !aligned16(k) || !aligned16(v)) return CK_ERR_ALIGN;
    ck::AttentionArgs a = cross_sizes(B, Lq, Lk, Hq, Hkv, D);
    a.k = bits(k), a.v = bits(v), a.ldk = ldk, a.ldv = ldv;
    a.lens = kv_lens;
    a.ragged = a.lens != nullptr;
    return run_attention(a, q, ldq, out, ldo, scale, ws, ws_bytes, stream);
}

}  // extern "C"
