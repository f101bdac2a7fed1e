// head_norm_rope.cu -- the two passes between the qkv linear and attention:
// the norm and rotation of query and key heads, and the append of keys (normed
// and rotated on the way) and values to a paged cache.  Each reads a head's
// row once into registers and writes it once; the bound is HBM bandwidth.
#include "head_norm_rope.cuh"
#include "attention.h"
#include "internal.h"
#include "launch_util.h"
#include "ptx.cuh"

namespace ck {
namespace {

constexpr int kThreads = 256;
// Head rows a group of lanes has in flight at once: their 16-byte loads are all
// issued before the first is used, and share the token's rotation factors.
constexpr int kRowsAhead = 4;

// How a block's groups of L lanes are dealt out: 2^gp_log2 of them share a
// token, the g-th taking its heads g, g + 2^gp_log2, ...
struct Deal {
    int gp_log2;
};

template <int L, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormRopeArgs a, const Deal deal) {
    pdl_launch_dependents();
    const int gl = threadIdx.x % L;
    const int d0 = gl * 8;
    const bool lane_on = d0 < a.D;
    const int heads = a.Hq + a.Hk;
    const int group = threadIdx.x / L;
    const int gp = 1 << deal.gp_log2;
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * ((kThreads / L) >> deal.gp_log2) + (group >> deal.gp_log2);
    const bool tok_on = tok < a.T;
    const int64_t t = tok_on ? tok : 0;
    const int h0 = group & (gp - 1);
    pdl_wait();
    const int pos = a.rot > 0 ? a.positions[t] : 0;
    float w[2][8] = {};
    if (lane_on) {
        if (a.wq) load_weight8(a.wq, a.w_f32, d0, w[0]);
        if (a.wk) load_weight8(a.wk, a.w_f32, d0, w[1]);
    }
    bool ok = tok_on;
    Rotation r;
    r.on = false, r.partner = gl;
    // heads in rounds of kRowsAhead a group; uniform over the block
    for (int base = 0; base < heads; base += gp * kRowsAhead) {
        uint4 in[kRowsAhead];
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            const int h = base + i * gp + h0;
            in[i] = make_uint4(0, 0, 0, 0);
            if (tok_on && lane_on && h < heads) {
                const uint16_t *src = h < a.Hq ? a.q + t * a.ldq + static_cast<int64_t>(h) * a.D
                                               : a.k + t * a.ldk + static_cast<int64_t>(h - a.Hq) * a.D;
                in[i] = *reinterpret_cast<const uint4 *>(src + d0);
            }
        }
        if (base == 0 && a.rot > 0) {
            const bool in_table = pos >= 0 && pos < a.max_pos;
            if (in_table)
                load_rotation<INTERLEAVED>(r, a.cos_sin + static_cast<int64_t>(pos) * a.rot, a.rot, d0, gl);
            else if (gl == 0 && tok_on)
                atomicOr(a.status, kDeviceStatusIndex);
            ok = ok && in_table;
        }
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            if (base + i * gp >= heads) break;  // uniform over the block
            const int h = base + i * gp + h0;
            const bool is_q = h < a.Hq;
            float x[8], wv[8];
            unpack8(in[i], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) wv[j] = is_q ? w[0][j] : w[1][j];
            norm_rotate<L, INTERLEAVED>(x, a.wq || a.wk, (is_q ? a.wq : a.wk) != nullptr, wv, a.inv_d, a.eps, a.rot > 0, r);
            if (ok && lane_on && h < heads) {
                uint16_t *dst = is_q ? a.q_out + t * a.ldqo + static_cast<int64_t>(h) * a.D
                                     : a.k_out + t * a.ldko + static_cast<int64_t>(h - a.Hq) * a.D;
                *reinterpret_cast<uint4 *>(dst + d0) = pack8(x);
            }
        }
    }
}

template <int L, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a, const Deal deal) {
    pdl_launch_dependents();
    const int gl = threadIdx.x % L;
    const int d0 = gl * 8;
    const bool lane_on = d0 < a.D;
    const int group = threadIdx.x / L;
    const int gp = 1 << deal.gp_log2;
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * ((kThreads / L) >> deal.gp_log2) + (group >> deal.gp_log2);
    const bool tok_on = tok < a.T;
    const int64_t t = tok_on ? tok : 0;
    const int h0 = group & (gp - 1);
    pdl_wait();
    const int64_t slot = tok_on ? a.slots[t] : -1;
    const int pos = a.rot > 0 ? a.positions[t] : 0;
    float w[8] = {};
    if (lane_on && a.wk) load_weight8(a.wk, a.w_f32, d0, w);
    bool ok = slot >= 0 && slot < a.pages * a.page_size;
    if (slot >= 0 && !ok && gl == 0) atomicOr(a.status, kDeviceStatusIndex);
    const int64_t page = ok ? slot / a.page_size : 0;
    const int64_t at0 = (page * a.Hkv * a.page_size + (slot - page * a.page_size)) * a.D + d0;
    Rotation r;
    r.on = false, r.partner = gl;
    constexpr int kAhead = kRowsAhead / 2;  // keys and values
    for (int base = 0; base < a.Hkv; base += gp * kAhead) {
        uint4 kin[kAhead], vin[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int h = base + i * gp + h0;
            kin[i] = vin[i] = make_uint4(0, 0, 0, 0);
            if (ok && lane_on && h < a.Hkv) {
                kin[i] = *reinterpret_cast<const uint4 *>(a.k + t * a.ldk + static_cast<int64_t>(h) * a.D + d0);
                vin[i] = *reinterpret_cast<const uint4 *>(a.v + t * a.ldv + static_cast<int64_t>(h) * a.D + d0);
            }
        }
        if (base == 0 && a.rot > 0 && ok) {
            ok = pos >= 0 && pos < a.max_pos;
            if (ok)
                load_rotation<INTERLEAVED>(r, a.cos_sin + static_cast<int64_t>(pos) * a.rot, a.rot, d0, gl);
            else if (gl == 0)
                atomicOr(a.status, kDeviceStatusIndex);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (base + i * gp >= a.Hkv) break;  // uniform over the block
            const int h = base + i * gp + h0;
            float x[8];
            unpack8(kin[i], x);
            norm_rotate<L, INTERLEAVED>(x, a.wk != nullptr, true, w, a.inv_d, a.eps, a.rot > 0, r);
            if (ok && lane_on && h < a.Hkv) {
                const int64_t at = at0 + static_cast<int64_t>(h) * a.page_size * a.D;
                *reinterpret_cast<uint4 *>(a.k_cache + at) = pack8(x);
                *reinterpret_cast<uint4 *>(a.v_cache + at) = vin[i];
            }
        }
    }
}

// Lanes that hold a row: the power of two of at least D / 8.
int group_lanes(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

template <typename Args>
cudaError_t launch_rows(void (*const (&kernels)[3][2])(const Args, const Deal), const Args &a, int64_t T, int heads,
                        bool interleaved, const LaunchCtx &ctx) {
    const int L = group_lanes(a.D);
    // Groups that share a token: each takes at least two of its heads, so that
    // the token's rotation factors serve more than one row.  A few tokens leave
    // SMs idle, so there a token's heads are spread as far as they go.
    int gp_log2 = 0;
    const int groups = kThreads / L;
    const bool few = T * heads <= 4 * sm_count() * groups;
    while ((1 << gp_log2) < groups && (2 << gp_log2) <= (few ? 2 * heads - 1 : heads / 2)) ++gp_log2;
    const int64_t per = groups >> gp_log2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((T + per - 1) / per));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernels[L == 8 ? 0 : (L == 16 ? 1 : 2)][interleaved ? 1 : 0], a, Deal{gp_log2});
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs &a, bool interleaved, const LaunchCtx &ctx) {
    static void (*const kernels[3][2])(const NormRopeArgs, const Deal) = {
        {qk_norm_rope_kernel<8, false>, qk_norm_rope_kernel<8, true>},
        {qk_norm_rope_kernel<16, false>, qk_norm_rope_kernel<16, true>},
        {qk_norm_rope_kernel<32, false>, qk_norm_rope_kernel<32, true>}};
    return launch_rows(kernels, a, a.T, a.Hq + a.Hk, interleaved, ctx);
}

cudaError_t launch_kv_append(const KvAppendArgs &a, bool interleaved, const LaunchCtx &ctx) {
    static void (*const kernels[3][2])(const KvAppendArgs, const Deal) = {
        {kv_append_kernel<8, false>, kv_append_kernel<8, true>},
        {kv_append_kernel<16, false>, kv_append_kernel<16, true>},
        {kv_append_kernel<32, false>, kv_append_kernel<32, true>}};
    return launch_rows(kernels, a, a.T, a.Hkv, interleaved, ctx);
}

}  // namespace ck
