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

__device__ __forceinline__ void unpack8(const uint4 &u, uint64_t (&v)[4]) {
    v[0] = fp4::unpack2(u.x), v[1] = fp4::unpack2(u.y), v[2] = fp4::unpack2(u.z), v[3] = fp4::unpack2(u.w);
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
    float lo, hi;
    f32x2_split(v, lo, hi);
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) {
    return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3]));
}
// The sum of v over a row's team of `tw` threads (8, 16 or whole warps); every thread of
// the block takes part.  `red` has the team's slots, a multiple of four floats of which
// those past its warps hold 0; the caller alternates between two sets of them.
__device__ __forceinline__ float team_sum(uint64_t v, float *red, int tt, int tw) {
    float s, t;
    f32x2_split(v, s, t);
    s += t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o < tw) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tw <= 32) return s;
    if ((threadIdx.x & 31) == 0) red[tt >> 5] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxThreads / 32; i += 4)
        if (32 * i < tw) {
            const float4 q = *reinterpret_cast<const float4 *>(red + i);
            s += (q.x + q.y) + (q.z + q.w);
        }
    return s;
}

// A row belongs to a team of `tw` threads, a warp of which has V times 256 columns (the
// parts of its columns at offsets known to the compiler); the teams of a block take rows
// in turn.  While a row is worked on, the next one's x and branch are on their way.
// FULL: every thread has all its columns.
//
// Read once, written once: HBM's rate is the floor, and what holds it off is a row's
// chain (load, one to three sums over the row, store) and the instructions: arithmetic
// is on pairs, an operand's presence is asked once a row and not once a part, a warp's
// parts are 256 columns apart so that a row's addresses are made once (all three: from
// 218 us to 193 with a norm behind the branch, from 36 to 25 modulated to codes).
// 30011 x 5120 in 188 us (6.5 TB/s, 0.97 of the measured copy), with a norm behind the
// branch too 193 us; 4096 x 4096 22.6 us (5.9 TB/s), with layer norm, gate, scale and
// shift 24.9 us, these to MX codes 25.2 us.
template <int V, Out OUT, bool FULL>
__global__ void __launch_bounds__(kMaxThreads, V >= 2 ? 1 : 2)
block_norm_kernel(const __grid_constant__ BlockNorm a, int tw, int rows_per_block, fp4::Scale t) {
    __shared__ alignas(16) float red[2][kMaxThreads / 32];
    pdl_launch_dependents();
    const int team = threadIdx.x / tw, tt = threadIdx.x - team * tw, lane = threadIdx.x & 31;
    if (threadIdx.x < kMaxThreads / 32) red[0][threadIdx.x] = red[1][threadIdx.x] = 0.f;
    __syncthreads();
    // (teams of five warps and more are alone in their block)
    float *mine = red[0] + team * 4;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_block;
    const float inv_h = 1.f / static_cast<float>(a.H);
    const int col0 = (tt >> 5) * (256 * V) + (tt & 31) * 8;
    bool in[V];
#pragma unroll
    for (int j = 0; j < V; ++j) in[j] = FULL || col0 + j * 256 < a.H;
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + team;
    const uint16_t *px = a.x + row * a.ldx + col0, *pb = a.branch + (a.branch ? row * a.ldb + col0 : 0);
    const int64_t sx = step * a.ldx, sb = step * a.ldb;
    pdl_wait();
    uint4 rx[V], rb[V];
#pragma unroll
    for (int j = 0; j < V; ++j) rx[j] = rb[j] = make_uint4(0, 0, 0, 0);  // and so they, and h, stay where no column is
    auto fetch = [&]() {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (in[j]) rx[j] = fp4::load_stream(px + j * 256);
        px += sx;
        if (a.branch) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (in[j]) rb[j] = fp4::load_stream(pb + j * 256);
            pb += sb;
        }
    };
    // f(j, its weights) for each part that has columns
    auto each = [&](const void *p, bool f32, auto f) {
        if (f32) {
            const float *q = static_cast<const float *>(p) + col0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (in[j]) {
                    const ulonglong2 *u = reinterpret_cast<const ulonglong2 *>(q + j * 256);
                    const ulonglong2 lo = __ldg(u), hi = __ldg(u + 1);
                    const uint64_t w[4] = {lo.x, lo.y, hi.x, hi.y};
                    f(j, w);
                }
        } else {
            const uint16_t *q = static_cast<const uint16_t *>(p) + col0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (in[j]) {
                    uint64_t w[4];
                    unpack8(__ldg(reinterpret_cast<const uint4 *>(q + j * 256)), w);
                    f(j, w);
                }
        }
    };
    // the same of gate, scale and shift: what a kernel ahead may still have been writing when
    // this one was let in, so not by loads for data that nobody writes
    auto each_mod = [&](const uint16_t *p, auto f) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (in[j]) {
                uint64_t w[4];
                unpack8(*reinterpret_cast<const uint4 *>(p + col0 + j * 256), w);
                f(j, w);
            }
    };
    if (row < a.T) fetch();
    const uint64_t fx = f32x2(a.x_factor, a.x_factor), fb = f32x2(a.branch_factor, a.branch_factor);
    const uint64_t one = f32x2(1.f, 1.f);
    const bool layer = a.norm == Norm::kLayer;
    auto sum_of = [&](uint64_t s) {
        const float r = team_sum(s, mine, tt, tw);
        mine = mine == red[0] + team * 4 ? red[1] + team * 4 : red[0] + team * 4;
        return r * inv_h;
    };
    // every team of a block makes the same rounds
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * rows_per_block; first < a.T; first += step, row += step) {
        const bool on = row < a.T;
        int64_t mod = 0;
        if (a.tokens_per_group > 0 && on)
            mod = static_cast<uint32_t>(row) / static_cast<uint32_t>(a.tokens_per_group) * a.ldm;
        uint64_t h[V][4];
        uint4 cx[V];
        if (a.branch) {
#pragma unroll
            for (int j = 0; j < V; ++j) unpack8(rb[j], h[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = 0;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) cx[j] = rx[j];
        if (row + step < a.T) fetch();
        if (a.post_weight) {
            uint64_t s = 0;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s = fma_f32x2(h[j][e], h[j][e], s);
            const float r = rsqrtf(sum_of(s) + a.eps);
            const uint64_t r2 = f32x2(r, r);
            each(a.post_weight, a.w_f32, [&](int j, const uint64_t (&w)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = mul_f32x2(mul_f32x2(h[j][e], r2), w[e]);
            });
        }
        if (a.gate)
            each_mod(a.gate + mod, [&](int j, const uint64_t (&w)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = mul_f32x2(h[j][e], w[e]);
            });
        if (a.branch) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                uint64_t x[4];
                unpack8(cx[j], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = fma_f32x2(h[j][e], fb, mul_f32x2(x[e], fx));
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                uint64_t x[4];
                unpack8(cx[j], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = mul_f32x2(x[e], fx);
            }
        }
        if (a.h && on) {
            uint16_t *p = a.h + row * a.ldh + col0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (in[j]) *reinterpret_cast<uint4 *>(p + j * 256) = pack8(h[j]);
        }
        uint64_t s = 0;
        if (layer) {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s = add_f32x2(s, h[j][e]);
            const float mean = sum_of(s);
            const uint64_t nm = f32x2(-mean, -mean);
            s = 0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (in[j]) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[j][e] = add_f32x2(h[j][e], nm);
                        s = fma_f32x2(h[j][e], h[j][e], s);
                    }
                }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s = fma_f32x2(h[j][e], h[j][e], s);
        }
        const float r = rsqrtf(sum_of(s) + a.eps);
        const uint64_t r2 = f32x2(r, r);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) h[j][e] = mul_f32x2(h[j][e], r2);
        if (a.weight)
            each(a.weight, a.w_f32, [&](int j, const uint64_t (&w)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = mul_f32x2(h[j][e], w[e]);
            });
        if (a.bias)
            each(a.bias, a.w_f32, [&](int j, const uint64_t (&w)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = add_f32x2(h[j][e], w[e]);
            });
        if (a.scale)
            each_mod(a.scale + mod, [&](int j, const uint64_t (&w)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = mul_f32x2(h[j][e], add_f32x2(w[e], one));
            });
        if (a.shift)
            each_mod(a.shift + mod, [&](int j, const uint64_t (&w)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = add_f32x2(h[j][e], w[e]);
            });
        if constexpr (OUT == Out::kBf16) {
            if (on) {
                uint16_t *p = a.n + row * a.ldn + col0;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (in[j]) *reinterpret_cast<uint4 *>(p + j * 256) = pack8(h[j]);
            }
        } else {
            constexpr bool kNv = OUT == Out::kNv;
            constexpr int kBlock = fp4::block_lanes(kNv), kWord = fp4::word_lanes(kNv);
            const int words = static_cast<int>(fp4_words(a.H, kNv)), word = col0 / (8 * kWord);
            uint8_t *code = a.codes + row * (a.H / 2) + col0 / 2;
            uint8_t *scales = a.scales + fp4::scale_word_at(row, word, words) + (lane / kBlock & 3);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                uint64_t n[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) n[e] = in[j] ? h[j][e] ^ 0x8000000080000000ull : 0ull;
                uint32_t scale;
                const uint32_t q = fp4::quantize8<kNv>(n, t, scale);
                if (on) {
                    if (in[j]) *reinterpret_cast<uint32_t *>(code + j * 128) = q;
                    if ((FULL || word + j * (32 / kWord) < words) && lane % kBlock == 0)
                        scales[j * (32 / kWord) * 512] = static_cast<uint8_t>(scale);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNorm &b, const LaunchCtx &ctx) {
    using Kernel = void (*)(const BlockNorm, int, int, fp4::Scale);
#define CK_KERNELS(V, FULL) \
    { block_norm_kernel<V, Out::kBf16, FULL>, block_norm_kernel<V, Out::kMx, FULL>, block_norm_kernel<V, Out::kNv, FULL> }
    static const Kernel kernels[3][2][3] = {{CK_KERNELS(1, false), CK_KERNELS(1, true)},
                                            {CK_KERNELS(2, false), CK_KERNELS(2, true)},
                                            {CK_KERNELS(4, false), CK_KERNELS(4, true)}};
#undef CK_KERNELS
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    // Columns of a thread, 8 << v.  Where all the columns fit the machine's threads at
    // once, as many threads a row as there are, for its chain (16 x 4096 2.0 us with 8
    // columns, 3.3 with 32).  Else few and wide threads, which share a row's sums and
    // addresses (4096 x 4096, modulated, to codes: 25.2 us with 32, 29.3 with 16, 34.1
    // with 8; 600 x 4096 5.4 and 6.9 with 8), but no more than a third without columns
    // (14463 x 1160, modulated: 35 us with 32, 33 with 16).
    const bool few = b.T * b.H < static_cast<int64_t>(sms) * 1024 * 8;
    int v = 2;
    if (few)
        v = b.H <= 4096 ? 0 : (b.H <= 8192 ? 1 : 2);
    else
        while (v > 0 && (b.H + (256 << v) - 1) / (256 << v) * (256 << v) * 2 > 3 * b.H) --v;
    const int per_warp = 256 << v;  // columns
    // (to codes whole warps: a word of scales is up to 16 lanes')
    const int tw = b.n && b.H <= 64 ? 8 : (b.n && b.H <= 128 ? 16 : (b.H + per_warp - 1) / per_warp * 32);
    int rows = tw >= 256 ? 1 : 256 / tw;  // of a block
    while (rows * tw > 32 && rows % 2 == 0 && (b.T + rows - 1) / rows < sms) rows /= 2;
    const int threads = (tw * rows + 31) / 32 * 32;
    const Kernel kernel = kernels[v][b.H % per_warp == 0][b.n ? 0 : (b.nv ? 2 : 1)];
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
    return cudaLaunchKernelEx(&cfg, kernel, b, tw, rows, fp4::scale_of(b.n_scale));
}

}  // namespace ck
