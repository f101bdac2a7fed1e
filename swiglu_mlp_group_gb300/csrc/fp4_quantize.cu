// fp4_quantize.cu -- bf16 (or f32) rows to microscaled 4-bit floats, and the
// block scales of a checkpoint into the tiles that the tensor cores read.
#include <cuda_bf16.h>

#include "fp4_core.cuh"
#include "launch_util.h"
#include "quant_core.cuh"

namespace ck {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerWarp = 4;

// Read once, written once: 2 bytes in and 0.56 (NV) or 0.53 (MX) out an element.
// A lane has 8 columns, 16 bytes to load and 4 to store, so that a warp's load is
// 512 bytes in a row; a warp takes 256 columns of 4 rows, whose loads are on
// their way together and whose scales lie next to each other.  What counts then is
// instructions, of the ALU above all: addresses are worked out once for the four
// rows, and each block's first lane stores its scale byte itself.  16384 x 4096: bf16
// 30.7 us NV (5.6 TB/s) and 27 MX (6.3 to 6.6), f32 45.7 (6.7) and 44.9 (6.8), silu(gate)
// * up 49.5 (6.2) and 45.4 (6.7): with twice the bytes to load, HBM.
enum class In : int { kBf16, kF32, kSwiglu };

template <bool NV, In IN>
__global__ void __launch_bounds__(kThreads)
fp4_quantize_kernel(const void *__restrict__ x, int64_t M, int K, int64_t ldx, fp4::Scale t,
                    uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, bool early_trigger) {
    if (early_trigger) pdl_launch_dependents();
    pdl_wait();
    if (!early_trigger) pdl_launch_dependents();
    constexpr int kBlock = fp4::block_lanes(NV), kWord = fp4::word_lanes(NV);
    const int lane = threadIdx.x & 31;
    const uint32_t segs = (static_cast<uint32_t>(K) + 255) / 256;
    const int words = static_cast<int>(fp4_words(K, NV));
    const int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    // (tasks are fewer than 2^35 and segs at most 128: 32 bits for calls of a usual size)
    const int64_t quad = task <= 0xffffffffll ? static_cast<uint32_t>(task) / segs : task / segs;
    const int64_t row0 = quad * kRowsPerWarp;
    const int col = static_cast<int>(task - quad * segs) * 256 + lane * 8;
    if (row0 >= M) return;
    const int rows = M - row0 < kRowsPerWarp ? static_cast<int>(M - row0) : kRowsPerWarp;
    const bool in = col < K;
    uint4 a[kRowsPerWarp], b[kRowsPerWarp];
    const char *src = static_cast<const char *>(x) + (row0 * ldx + col) * (IN == In::kF32 ? 4 : 2);
    const int64_t src_step = ldx * (IN == In::kF32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        if (in && i < rows) {
            a[i] = fp4::load_stream(src);
            if constexpr (IN == In::kF32) b[i] = fp4::load_stream(src + 16);
            if constexpr (IN == In::kSwiglu) b[i] = fp4::load_stream(src + 2 * K);
        }
        src += src_step;
    }
    uint8_t *code = codes + row0 * (K / 2) + col / 2;
    // four rows from a multiple of four on: their words 16 bytes apart
    const int word = col / (8 * kWord);
    uint8_t *scale_at = scales + fp4::scale_word_at(row0, word, words) + (lane / kBlock & 3);
    const bool has_scale = word < words && lane % kBlock == 0;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        if (i >= rows) break;
        const uint32_t ra[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, rb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
        uint64_t n[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (IN == In::kF32) {
                const uint32_t *r = j < 2 ? ra : rb;
                n[j] = f32x2(-__uint_as_float(r[2 * (j & 1)]), -__uint_as_float(r[2 * (j & 1) + 1]));
            } else if constexpr (IN == In::kSwiglu) {
                n[j] = f32x2(-qc::silu_mul(__uint_as_float(ra[j] << 16), __uint_as_float(rb[j] << 16)),
                             -qc::silu_mul(__uint_as_float(ra[j] & 0xffff0000u), __uint_as_float(rb[j] & 0xffff0000u)));
            } else {
                n[j] = fp4::unpack2_neg(ra[j]);
            }
        }
        uint32_t scale;
        const uint32_t q = fp4::quantize8<NV>(n, t, scale);
        if (in) *reinterpret_cast<uint32_t *>(code) = q;
        if (has_scale) scale_at[16 * i] = static_cast<uint8_t>(scale);
        code += K / 2;
    }
}

// One word a thread.
__global__ void __launch_bounds__(kThreads)
fp4_tile_scales_kernel(const uint8_t *__restrict__ in, int64_t rows, int words, int blocks, uint8_t *__restrict__ out) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t row = i / words;
    if (row >= rows) return;
    const int word = static_cast<int>(i - row * words);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (4 * word + j < blocks) w |= static_cast<uint32_t>(in[row * blocks + 4 * word + j]) << (8 * j);
    *reinterpret_cast<uint32_t *>(out + fp4::scale_word_at(row, word, words)) = w;
}

template <typename... A, typename... B>
cudaError_t launch(void (*kernel)(A...), int64_t blocks, const LaunchCtx &ctx, B... args) {
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_fp4_quantize(const void *x, bool x_f32, Act act, int64_t M, int64_t K, int64_t ldx, bool nv,
                                float tensor_scale, uint8_t *codes, uint8_t *scales, const LaunchCtx &ctx) {
    using Kernel = void (*)(const void *, int64_t, int, int64_t, fp4::Scale, uint8_t *, uint8_t *, bool);
    static const Kernel kernels[2][3] = {
        {fp4_quantize_kernel<false, In::kBf16>, fp4_quantize_kernel<false, In::kF32>,
         fp4_quantize_kernel<false, In::kSwiglu>},
        {fp4_quantize_kernel<true, In::kBf16>, fp4_quantize_kernel<true, In::kF32>,
         fp4_quantize_kernel<true, In::kSwiglu>}};
    const In in = x_f32 ? In::kF32 : act == Act::kSwiglu ? In::kSwiglu : In::kBf16;
    const int64_t tasks = (M + kRowsPerWarp - 1) / kRowsPerWarp * ((K + 255) / 256);
    constexpr int kWarps = kThreads / 32;
    return launch(kernels[nv ? 1 : 0][static_cast<int>(in)], (tasks + kWarps - 1) / kWarps, ctx, x, M,
                  static_cast<int>(K), ldx, fp4::scale_of(tensor_scale), codes, scales,
                  ctx.early_trigger);
}

cudaError_t launch_fp4_tile_scales(const uint8_t *scales, int64_t rows, int64_t K, bool nv, uint8_t *tiled,
                                   const LaunchCtx &ctx) {
    const int words = static_cast<int>(fp4_words(K, nv));
    return launch(fp4_tile_scales_kernel, (rows * words + kThreads - 1) / kThreads, ctx, scales, rows, words,
                  static_cast<int>(K / fp4_block(nv)), tiled);
}

}  // namespace ck
