// attention.cu -- attention over a shared prefix and each sequence's own keys
// (paged), or over an encoder's states (dense): one warp a query row.
//
//   x_j = scale * q . k_j,   m = max_j x_j,   out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m)
// in one pass over the keys: m and the sum are carried, and the sums so far are
// scaled by e^(m_old - m_new) where m grows.  A lane scores one key of 32, then
// the warp adds the 32 value rows, each lane its own elements.
#include <math.h>

#include "attention.h"
#include "head_norm_rope.cuh"
#include "ptx.cuh"

namespace ck {
namespace {

constexpr int kRowsPerBlock = 4;

template <int D>
__global__ void __launch_bounds__(32 * kRowsPerBlock) attention_rows_kernel(const AttentionArgs a) {
    __shared__ float sq[kRowsPerBlock][D];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + warp;
    if (row >= a.B * a.Lq * a.Hq) return;
    const int64_t t = row / a.Hq;
    const int hq = static_cast<int>(row - t * a.Hq), h = hq / a.G;
    const int64_t b = t / a.Lq, i = t - b * a.Lq;
    constexpr int E = D / 32;
    for (int e = 0; e < E; ++e) {
        const uint32_t u = a.q[t * a.ldq + static_cast<int64_t>(hq) * D + lane * E + e];
        sq[warp][lane * E + e] = __uint_as_float(u << 16) * a.scale;
    }
    __syncwarp();
    int64_t len = a.max_len;
    if (a.lens) {
        len = a.lens[b];
        if (len < 0 || len > a.max_len) {
            if (lane == 0) atomicOr(a.status, kDeviceStatusIndex);
            len = len < 0 ? 0 : a.max_len;
        }
    }
    float m = -INFINITY, l = 0.f, o[E] = {};
    auto pass = [&](int64_t n, bool prefix) {
        for (int64_t j0 = 0; j0 < n; j0 += 32) {
            const int64_t j = j0 + lane;
            int64_t ko = -1, vo = -1;  // offsets of this lane's key and value row (-1: a row of zeros)
            if (j < n) {
                if (a.pages > 0) {
                    const int32_t page = prefix ? a.prefix_pages[j / a.page_size]
                                                : a.block_table[b * a.table_stride + j / a.page_size];
                    if (page >= 0 && page < a.pages)
                        ko = vo = ((static_cast<int64_t>(page) * a.Hkv + h) * a.page_size + j % a.page_size) * D;
                    else
                        atomicOr(a.status, kDeviceStatusIndex);
                } else {
                    ko = (b * a.max_len + j) * a.ldk + static_cast<int64_t>(h) * D;
                    vo = (b * a.max_len + j) * a.ldv + static_cast<int64_t>(h) * D;
                }
            }
            float x = -INFINITY;
            if (j < n) {
                x = 0.f;
                if (ko >= 0)
                    for (int d = 0; d < D; d += 8) {
                        float kv[8];
                        unpack8(*reinterpret_cast<const uint4 *>(a.k + ko + d), kv);
                        for (int e = 0; e < 8; ++e) x = fmaf(sq[warp][d + e], kv[e], x);
                    }
            }
            float top = x;
            for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float m_new = fmaxf(m, top);
            const float base = m_new == -INFINITY ? 0.f : m_new;
            const float p = expf(x - base), f = expf(m - base);
            float sum = p;
            for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            l = l * f + sum;
            m = m_new;
            for (int e = 0; e < E; ++e) o[e] *= f;
            for (int s = 0; s < 32 && j0 + s < n; ++s) {
                const float ps = __shfl_sync(0xffffffffu, p, s);
                const int64_t at = __shfl_sync(0xffffffffu, vo, s);
                if (at < 0) continue;
                for (int e = 0; e < E; ++e) {
                    const uint32_t u = a.v[at + lane * E + e];
                    o[e] = fmaf(ps, __uint_as_float(u << 16), o[e]);
                }
            }
        }
    };
    if (a.prefix_len > 0) pass(a.prefix_len, true);
    int64_t own = a.causal ? len - a.Lq + i + 1 : len;
    pass(own < 0 ? 0 : own, false);
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    for (int e = 0; e < E; ++e) {
        const __nv_bfloat16 r = __float2bfloat16_rn(o[e] * inv);
        a.out[t * a.ldo + static_cast<int64_t>(hq) * D + lane * E + e] = *reinterpret_cast<const uint16_t *>(&r);
    }
}

}  // namespace

size_t attention_workspace_bytes(const AttentionArgs &) { return 0; }

cudaError_t launch_attention(const AttentionArgs &a, const LaunchCtx &ctx) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.B * a.Lq * a.Hq + kRowsPerBlock - 1) / kRowsPerBlock));
    cfg.blockDim = dim3(32 * kRowsPerBlock);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 1 : 0;
    return a.D == 64 ? cudaLaunchKernelEx(&cfg, attention_rows_kernel<64>, a)
                     : cudaLaunchKernelEx(&cfg, attention_rows_kernel<128>, a);
}

}  // namespace ck
