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
__device__ __forceinline__ void load8(const uint16_t *p, uint64_t (&v)[4]) {
    unpack8(__ldg(reinterpret_cast<const uint4 *>(p)), v);
}
// A stream's 16 bytes: read once, so they do not displace the weights in L1 (they may
// be written later in the kernel, by the thread that reads them).
__device__ __forceinline__ uint4 load_stream(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
// Eight weights of the norms' type.
__device__ __forceinline__ void load_weight(const void *p, bool f32, int col, uint64_t (&v)[4]) {
    if (f32) {
        const ulonglong2 *q = reinterpret_cast<const ulonglong2 *>(static_cast<const float *>(p) + col);
        const ulonglong2 a = __ldg(q), b = __ldg(q + 1);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
        load8(static_cast<const uint16_t *>(p) + col, v);
    }
}

// The sum of v over a row's team of `tw` threads (8, 16 or whole warps, the first of
// which is the block's `first`); every thread of the block takes part.  `red` has a
// float for each warp, and the caller alternates between two of them.
__device__ __forceinline__ float team_sum(uint64_t v, float *red, int first, int tw) {
    float s, t;
    f32x2_split(v, s, t);
    s += t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o < tw) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tw <= 32) return s;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
    for (int i = 0; i < tw / 32; ++i) s += red[first + i];
    return s;
}

// A row belongs to a team of `tw` threads, each with V times eight columns; the teams
// of a block take rows in turn.  While a row is worked on, the next one's x and branch
// are on their way.
//
// Read once, written once: HBM's rate is the floor, and what holds it off is a row's
// chain (load, one to three sums over the row, store) and, with modulation, the
// instructions: arithmetic is on pairs.  30011 x 5120 in 192 us (6.4 TB/s, 0.94 of the
// measured copy), with a norm behind the branch too 214 us, 4096 x 4096 24 us (5.6
// TB/s), with layer norm, gate, scale and shift 33 us.
template <int V, Out OUT>
__global__ void __launch_bounds__(kMaxThreads, V == 4 ? 1 : 2)
block_norm_kernel(const __grid_constant__ BlockNorm a, int tw, int rows_per_block, fp4::Scale t) {
    __shared__ float red[2][kMaxThreads / 32];
    pdl_launch_dependents();
    const int team = threadIdx.x / tw, tt = threadIdx.x - team * tw, lane = threadIdx.x & 31;
    const int first_warp = team * (tw / 32);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_block;
    const float inv_h = 1.f / static_cast<float>(a.H);
    const int col0 = tt * 8, col_step = tw * 8;
    bool in[V];
#pragma unroll
    for (int j = 0; j < V; ++j) in[j] = col0 + j * col_step < a.H;
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + team;
    const uint16_t *px = a.x + row * a.ldx + col0, *pb = a.branch + (a.branch ? row * a.ldb + col0 : 0);
    const int64_t sx = step * a.ldx, sb = step * a.ldb;
    pdl_wait();
    uint4 rx[V], rb[V];
    auto fetch = [&](bool on) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            rx[j] = rb[j] = make_uint4(0, 0, 0, 0);
            if (on && in[j]) {
                rx[j] = load_stream(px + j * col_step);
                if (a.branch) rb[j] = load_stream(pb + j * col_step);
            }
        }
        px += sx;
        if (a.branch) pb += sb;
    };
    fetch(row < a.T);
    const uint64_t fx = f32x2(a.x_factor, a.x_factor), fb = f32x2(a.branch_factor, a.branch_factor);
    int turn = 0;
    // every team of a block makes the same rounds
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * rows_per_block; first < a.T; first += step, row += step) {
        const bool on = row < a.T;
        int64_t mod = 0;
        if (a.tokens_per_group > 0 && on)
            mod = static_cast<uint32_t>(row) / static_cast<uint32_t>(a.tokens_per_group) * a.ldm;
        uint64_t h[V][4];
        uint4 cx[V];
#pragma unroll
        for (int j = 0; j < V; ++j) unpack8(rb[j], h[j]), cx[j] = rx[j];
        fetch(row + step < a.T);
        if (a.post_weight) {
            uint64_t s = 0;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s = fma_f32x2(h[j][e], h[j][e], s);
            const float r = rsqrtf(team_sum(s, red[turn], first_warp, tw) * inv_h + a.eps);
            const uint64_t r2 = f32x2(r, r);
            turn ^= 1;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (in[j]) {
                    uint64_t w[4];
                    load_weight(a.post_weight, a.w_f32, col0 + j * col_step, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[j][e] = mul_f32x2(mul_f32x2(h[j][e], r2), w[e]);
                }
        }
        uint64_t s = 0;
        const bool layer = a.norm == Norm::kLayer;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (in[j]) {
                const int col = col0 + j * col_step;
                if (a.gate) {
                    uint64_t g[4];
                    load8(a.gate + mod + col, g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[j][e] = mul_f32x2(h[j][e], g[e]);
                }
                uint64_t x[4];
                unpack8(cx[j], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t y = mul_f32x2(x[e], fx);
                    h[j][e] = a.branch ? fma_f32x2(h[j][e], fb, y) : y;
                }
                if (a.h && on) *reinterpret_cast<uint4 *>(a.h + row * a.ldh + col) = pack8(h[j]);
#pragma unroll
                for (int e = 0; e < 4; ++e) s = layer ? add_f32x2(s, h[j][e]) : fma_f32x2(h[j][e], h[j][e], s);
            }
        }
        float sum = team_sum(s, red[turn], first_warp, tw);
        turn ^= 1;
        if (layer) {
            const float mean = sum * inv_h;
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
            sum = team_sum(s, red[turn], first_warp, tw);
            turn ^= 1;
        }
        const float r = rsqrtf(sum * inv_h + a.eps);
        const uint64_t r2 = f32x2(r, r);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = col0 + j * col_step;
            uint64_t n[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) n[e] = mul_f32x2(h[j][e], r2);
            if (in[j]) {
                uint64_t w[4];
                if (a.weight) {
                    load_weight(a.weight, a.w_f32, col, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) n[e] = mul_f32x2(n[e], w[e]);
                }
                if (a.bias) {
                    load_weight(a.bias, a.w_f32, col, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) n[e] = add_f32x2(n[e], w[e]);
                }
                if (a.scale) {
                    load8(a.scale + mod + col, w);
                    const uint64_t one = f32x2(1.f, 1.f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) n[e] = mul_f32x2(n[e], add_f32x2(w[e], one));
                }
                if (a.shift) {
                    load8(a.shift + mod + col, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) n[e] = add_f32x2(n[e], w[e]);
                }
            }
            if constexpr (OUT == Out::kBf16) {
                if (in[j] && on) *reinterpret_cast<uint4 *>(a.n + row * a.ldn + col) = pack8(n);
            } else {
                constexpr bool kNv = OUT == Out::kNv;
                constexpr int kBlock = fp4::block_lanes(kNv), kWord = fp4::word_lanes(kNv);
#pragma unroll
                for (int e = 0; e < 4; ++e) n[e] = in[j] ? n[e] ^ 0x8000000080000000ull : 0ull;
                uint32_t scale;
                const uint32_t q = fp4::quantize8<kNv>(n, t, scale);
                const int words = static_cast<int>(fp4_words(a.H, kNv)), word = col / (8 * kWord);
                if (on) {
                    if (in[j]) *reinterpret_cast<uint32_t *>(a.codes + row * (a.H / 2) + col / 2) = q;
                    if (word < words && lane % kBlock == 0)
                        a.scales[fp4::scale_word_at(row, word, words) + (lane / kBlock & 3)] = static_cast<uint8_t>(scale);
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
    // Columns of a thread, 8 << v.  Few rows: as many threads a row as there are, for its
    // chain (16 x 4096 2.3 us with 8 columns, 2.7 with 16, 3.3 with 32).  Many: fewer and
    // wider threads, which share a row's sums (30011 x 5120 192 us with 32, 207 with 16;
    // 4096 x 4096 to codes, modulated, 39 us with 16, 41 with 32, 46 with 8).
    const bool few = b.T < 8 * sms;
    const int v = few ? (b.H <= 4096 ? 0 : (b.H <= 8192 ? 1 : 2)) : (b.H <= 2048 ? 0 : (b.H <= 4096 ? 1 : 2));
    const int per_warp = 256 << v;  // columns
    // (to codes whole warps: a word of scales is up to 16 lanes')
    const int tw = b.n && b.H <= 64 ? 8 : (b.n && b.H <= 128 ? 16 : (b.H + per_warp - 1) / per_warp * 32);
    int rows = tw >= 256 ? 1 : 256 / tw;  // of a block
    while (rows * tw > 32 && rows % 2 == 0 && (b.T + rows - 1) / rows < sms) rows /= 2;
    const int threads = (tw * rows + 31) / 32 * 32;
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
    return cudaLaunchKernelEx(&cfg, kernel, b, tw, rows, fp4::scale_of(b.n_scale));
}

}  // namespace ck
