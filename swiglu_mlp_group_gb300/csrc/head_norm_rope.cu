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

template <int L, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormRopeArgs a) {
    pdl_launch_dependents();
    const int gl = threadIdx.x % L;
    const int d0 = gl * 8;
    const bool lane_on = d0 < a.D;
    const int heads = a.Hq + a.Hk;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
    const bool row_on = row < a.T * heads;
    const int64_t t = row_on ? row / heads : 0;
    const int h = row_on ? static_cast<int>(row - t * heads) : 0;
    const bool is_q = h < a.Hq;
    const void *w = is_q ? a.wq : a.wk;
    const uint16_t *src = is_q ? a.q + t * a.ldq + static_cast<int64_t>(h) * a.D
                               : a.k + t * a.ldk + static_cast<int64_t>(h - a.Hq) * a.D;
    uint16_t *dst = is_q ? a.q_out + t * a.ldqo + static_cast<int64_t>(h) * a.D
                         : a.k_out + t * a.ldko + static_cast<int64_t>(h - a.Hq) * a.D;
    pdl_wait();
    float x[8] = {}, wv[8] = {};
    if (row_on && lane_on) {
        unpack8(*reinterpret_cast<const uint4 *>(src + d0), x);
        if (w) load_weight8(w, a.w_f32, d0, wv);
    }
    bool ok = true;
    Rotation r;
    r.on = false, r.partner = gl;
    if (a.rot > 0) {
        const int pos = a.positions[t];
        ok = pos >= 0 && pos < a.max_pos;
        if (ok)
            load_rotation<INTERLEAVED>(r, a.cos_sin + static_cast<int64_t>(pos) * a.rot, a.rot, d0, gl);
        else if (gl == 0 && row_on)
            atomicOr(a.status, kDeviceStatusIndex);
    }
    norm_rotate<L, INTERLEAVED>(x, w != nullptr, wv, a.inv_d, a.eps, a.rot > 0, r);
    if (row_on && lane_on && ok) *reinterpret_cast<uint4 *>(dst + d0) = pack8(x);
}

template <int L, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a) {
    pdl_launch_dependents();
    const int gl = threadIdx.x % L;
    const int d0 = gl * 8;
    const bool lane_on = d0 < a.D;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
    const bool row_on = row < a.T * a.Hkv;
    const int64_t t = row_on ? row / a.Hkv : 0;
    const int h = row_on ? static_cast<int>(row - t * a.Hkv) : 0;
    pdl_wait();
    const int64_t slot = row_on ? a.slots[t] : -1;
    bool ok = slot >= 0 && slot < a.pages * a.page_size;
    if (slot >= 0 && !ok && gl == 0) atomicOr(a.status, kDeviceStatusIndex);
    Rotation r;
    r.on = false, r.partner = gl;
    if (a.rot > 0 && ok) {
        const int pos = a.positions[t];
        ok = pos >= 0 && pos < a.max_pos;
        if (ok)
            load_rotation<INTERLEAVED>(r, a.cos_sin + static_cast<int64_t>(pos) * a.rot, a.rot, d0, gl);
        else if (gl == 0)
            atomicOr(a.status, kDeviceStatusIndex);
    }
    float x[8] = {}, wv[8] = {};
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok && lane_on) {
        unpack8(*reinterpret_cast<const uint4 *>(a.k + t * a.ldk + static_cast<int64_t>(h) * a.D + d0), x);
        v = *reinterpret_cast<const uint4 *>(a.v + t * a.ldv + static_cast<int64_t>(h) * a.D + d0);
        if (a.wk) load_weight8(a.wk, a.w_f32, d0, wv);
    }
    norm_rotate<L, INTERLEAVED>(x, a.wk != nullptr, wv, a.inv_d, a.eps, a.rot > 0, r);
    if (ok && lane_on) {
        const int64_t page = slot / a.page_size;
        const int64_t at = ((page * a.Hkv + h) * a.page_size + (slot - page * a.page_size)) * a.D + d0;
        *reinterpret_cast<uint4 *>(a.k_cache + at) = pack8(x);
        *reinterpret_cast<uint4 *>(a.v_cache + at) = v;
    }
}

// Lanes that hold a row: the power of two of at least D / 8.
int group_lanes(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

template <typename Args>
cudaError_t launch_rows(void (*const (&kernels)[3][2])(const Args), const Args &a, int64_t rows, bool interleaved,
                        const LaunchCtx &ctx) {
    const int L = group_lanes(a.D);
    const int64_t per = kThreads / L;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows + per - 1) / per));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernels[L == 8 ? 0 : (L == 16 ? 1 : 2)][interleaved ? 1 : 0], a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs &a, bool interleaved, const LaunchCtx &ctx) {
    static void (*const kernels[3][2])(const NormRopeArgs) = {
        {qk_norm_rope_kernel<8, false>, qk_norm_rope_kernel<8, true>},
        {qk_norm_rope_kernel<16, false>, qk_norm_rope_kernel<16, true>},
        {qk_norm_rope_kernel<32, false>, qk_norm_rope_kernel<32, true>}};
    return launch_rows(kernels, a, a.T * (a.Hq + a.Hk), interleaved, ctx);
}

cudaError_t launch_kv_append(const KvAppendArgs &a, bool interleaved, const LaunchCtx &ctx) {
    static void (*const kernels[3][2])(const KvAppendArgs) = {
        {kv_append_kernel<8, false>, kv_append_kernel<8, true>},
        {kv_append_kernel<16, false>, kv_append_kernel<16, true>},
        {kv_append_kernel<32, false>, kv_append_kernel<32, true>}};
    return launch_rows(kernels, a, a.T * a.Hkv, interleaved, ctx);
}

}  // namespace ck
