// block_norm.cu -- what stands between a block's branch and the next linear, in
// one pass over the residual stream:
//
//   b = branch [* rsqrt(mean(branch^2) + eps) * post_weight]
//   h = x_factor * x + branch_factor * gate * b                (stored as bf16)
//   n = norm(h) * weight + bias,  then  n * (1 + scale) + shift
//
// norm: h * rsqrt(mean(h^2) + eps), or of h less its mean.  f32 throughout: n is
// formed from h before its rounding, and rounded once, to bf16 or to the 4-bit
// codes and block scales that the next product reads (fp4_core.cuh).
#include <cuda_bf16.h>

#include "fp4_core.cuh"
#include "launch_util.h"

namespace ck {
namespace {

enum class Out : int { kBf16, kMx, kNv };

constexpr int kMaxThreads = 512;

__device__ __forceinline__ void unpack8(const uint4 &u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8]) {
    unpack8(__ldg(reinterpret_cast<const uint4 *>(p)), v);
}
// Eight weights of the norms' type.
__device__ __forceinline__ void load_weight(const void *p, bool f32, int col, float (&v)[8]) {
    if (f32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + col);
        const float4 a = __ldg(q), b = __ldg(q + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        load8(static_cast<const uint16_t *>(p) + col, v);
    }
}

// The sum of v over the `warps` warps of a row's team; every thread of the block
// takes part.  `red` has a float for each warp of the block, and the caller
// alternates between two of them.
__device__ __forceinline__ float team_sum(float v, float *red, int warps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const float *mine = red + warp / warps * warps;
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += mine[i];
    return s;
}

// A row belongs to a team of `warps` warps, a thread of which has V times eight
// columns; the teams of a block take rows in turn.  While a row is worked on, the
// next one's x and branch are on their way.
template <int V, Out OUT>
__global__ void __launch_bounds__(kMaxThreads, V == 4 ? 1 : 2)
block_norm_kernel(const __grid_constant__ BlockNorm a, int warps, int rows_per_block, fp4::Scale t) {
    __shared__ float red[2][kMaxThreads / 32];
    pdl_launch_dependents();
    const int team = threadIdx.x / (32 * warps), tt = threadIdx.x - team * 32 * warps, lane = threadIdx.x & 31;
    const int tw = 32 * warps;  // threads of a team
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_block;
    const float inv_h = 1.f / static_cast<float>(a.H);
    const int words = static_cast<int>(fp4_words(a.H, OUT == Out::kNv));
    pdl_wait();
    uint4 rx[V], rb[V];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (j * tw + tt) * 8;
            rx[j] = rb[j] = make_uint4(0, 0, 0, 0);
            if (row < a.T && col < a.H) {
                rx[j] = *reinterpret_cast<const uint4 *>(a.x + row * a.ldx + col);
                if (a.branch) rb[j] = *reinterpret_cast<const uint4 *>(a.branch + row * a.ldb + col);
            }
        }
    };
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + team;
    fetch(row);
    int turn = 0;
    // every team of a block makes the same rounds
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * rows_per_block; first < a.T; first += step, row += step) {
        const bool on = row < a.T;
        const uint32_t group = a.tokens_per_group > 0 && on
                                   ? static_cast<uint32_t>(row) / static_cast<uint32_t>(a.tokens_per_group) : 0u;
        const int64_t mod = group * a.ldm;
        float h[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) unpack8(rb[j], h[j]);
        uint4 cx[V];
#pragma unroll
        for (int j = 0; j < V; ++j) cx[j] = rx[j];
        fetch(row + step);
        if (a.post_weight) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += h[j][e] * h[j][e];
            const float r = rsqrtf(team_sum(s, red[turn], warps) * inv_h + a.eps);
            turn ^= 1;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int col = (j * tw + tt) * 8;
                if (col < a.H) {
                    float w[8];
                    load_weight(a.post_weight, a.w_f32, col, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[j][e] = h[j][e] * r * w[e];
                }
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (j * tw + tt) * 8;
            if (col < a.H) {
                if (a.gate) {
                    float g[8];
                    load8(a.gate + mod + col, g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[j][e] *= g[e];
                }
                float x[8];
                unpack8(cx[j], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[j][e] = a.branch ? a.x_factor * x[e] + a.branch_factor * h[j][e] : a.x_factor * x[e];
                if (a.h && on) *reinterpret_cast<uint4 *>(a.h + row * a.ldh + col) = pack8(h[j]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += a.norm == Norm::kLayer ? h[j][e] : h[j][e] * h[j][e];
        }
        sum = team_sum(sum, red[turn], warps);
        turn ^= 1;
        if (a.norm == Norm::kLayer) {
            const float mean = sum * inv_h;
            sum = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if ((j * tw + tt) * 8 >= a.H) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    h[j][e] -= mean;
                    sum += h[j][e] * h[j][e];
                }
            }
            sum = team_sum(sum, red[turn], warps);
            turn ^= 1;
        }
        const float r = rsqrtf(sum * inv_h + a.eps);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (j * tw + tt) * 8;
            const bool in = col < a.H;
            float n[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] = h[j][e] * r;
            if (in) {
                float w[8];
                if (a.weight) {
                    load_weight(a.weight, a.w_f32, col, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) n[e] *= w[e];
                }
                if (a.bias) {
                    load_weight(a.bias, a.w_f32, col, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) n[e] += w[e];
                }
                if (a.scale) {
                    load8(a.scale + mod + col, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) n[e] *= 1.f + w[e];
                }
                if (a.shift) {
                    load8(a.shift + mod + col, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) n[e] += w[e];
                }
            }
            if constexpr (OUT == Out::kBf16) {
                if (in && on) *reinterpret_cast<uint4 *>(a.n + row * a.ldn + col) = pack8(n);
            } else {
                constexpr bool kNv = OUT == Out::kNv;
                constexpr int kGroup = kNv ? 8 : 16;  // lanes of a word
                uint64_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = f32x2(n[2 * i], n[2 * i + 1]);
                uint32_t scale;
                const uint32_t q = fp4::quantize8<kNv>(v, t, scale);
                const uint32_t word = fp4::scale_word<kNv>(in ? scale : 0u, lane);
                if (in && on) {
                    *reinterpret_cast<uint32_t *>(a.codes + row * (a.H / 2) + col / 2) = q;
                    if (lane % kGroup == 0)
                        *reinterpret_cast<uint32_t *>(a.scales + fp4::scale_word_at(row, col / (8 * kGroup), words)) = word;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNorm &b, const LaunchCtx &ctx) {
    using Kernel = void (*)(const BlockNorm, int, int, fp4::Scale);
    static const Kernel kernels[3][3] = {
        {block_norm_kernel<1, Out::kBf16>, block_norm_kernel<1, Out::kMx>, block_norm_kernel<1, Out::kNv>},
        {block_norm_kernel<2, Out::kBf16>, block_norm_kernel<2, Out::kMx>, block_norm_kernel<2, Out::kNv>},
        {block_norm_kernel<4, Out::kBf16>, block_norm_kernel<4, Out::kMx>, block_norm_kernel<4, Out::kNv>}};
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const int v = b.H <= 2048 ? 0 : (b.H <= 8192 ? 1 : 2);
    const int per_warp = 256 << v;  // columns
    const int warps = (b.H + per_warp - 1) / per_warp;
    int rows = warps >= 8 ? 1 : 8 / warps;  // of a block
    while (rows > 1 && (b.T + rows - 1) / rows < sms) rows /= 2;
    const int threads = 32 * warps * rows;
    const Kernel kernel = kernels[v][b.n ? 0 : (b.nv ? 2 : 1)];
    const int resident = resident_blocks_per_sm(reinterpret_cast<const void *>(kernel), threads, 0);
    if (resident < 1) return cudaErrorInvalidConfiguration;
    const int64_t blocks = (b.T + rows - 1) / rows;
    const int64_t most = static_cast<int64_t>(resident) * sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, b, warps, rows, fp4::scale_of(b.n_scale));
}

}  // namespace ck
