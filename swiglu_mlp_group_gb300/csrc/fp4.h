// fp4.h -- launchers of the microscaled 4-bit operators and of the block norm,
// shared between their kernels and the C-ABI layer (fp4_api.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace ck {

// Scales of a row that stand in one 32-bit word, and the K they cover.
constexpr int fp4_block(bool nv) { return nv ? 16 : 32; }
constexpr int fp4_word(bool nv) { return nv ? 64 : 128; }

// Words of scales a row has.
constexpr int64_t fp4_words(int64_t K, bool nv) { return (K + fp4_word(nv) - 1) / fp4_word(nv); }
// Bytes of the tiled scales of `rows` rows: tiles of 128 rows x one word.
constexpr size_t fp4_scale_bytes(int64_t rows, int64_t K, bool nv) {
    return static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>(fp4_words(K, nv)) * 512;
}

// x (bf16, or f32 with x_f32) [M, ldx] -> codes [M, K / 2], tiled scales.
// act kSwiglu: x holds [gate | up] (bf16).
cudaError_t launch_fp4_quantize(const void *x, bool x_f32, Act act, int64_t M, int64_t K, int64_t ldx, bool nv,
                                float tensor_scale, uint8_t *codes, uint8_t *scales, const LaunchCtx &ctx);

// Scales by row [rows, K / block] -> tiled.
cudaError_t launch_fp4_tile_scales(const uint8_t *scales, int64_t rows, int64_t K, bool nv, uint8_t *tiled,
                                   const LaunchCtx &ctx);

// y bf16 [M, N] = bf16(alpha * X W^T + bias[n] + residual[m, n]).  X: codes [M, K / 2]
// and tiled scales; or (few tokens) bf16 x [M, ldx] that the kernel quantizes with
// tensor scale x_scale (swiglu: of [gate | up]).  W: [N, K / 2] codes and tiled
// scales.  weights_settled: nothing in flight writes W or its scales once the kernel
// has been let in.
struct Fp4Gemm {
    const uint8_t *x = nullptr, *xs = nullptr;
    const void *x_bf16 = nullptr;
    int64_t ldx = 0;
    bool swiglu = false;
    float x_scale = 1.f;
    const uint8_t *w = nullptr, *ws = nullptr;
    int64_t M = 0, N = 0, K = 0;
    bool nv = false;
    float alpha = 1.f;
    const void *bias = nullptr, *residual = nullptr;
    void *y = nullptr;
    bool weights_settled = false;
    // launch_fp4_gemm_glu's result
    uint8_t *a_codes = nullptr, *a_scales = nullptr;
    float a_scale = 1.f;
};
cudaError_t launch_fp4_gemm(const Fp4Gemm &g, const LaunchCtx &ctx);
// Most tokens that a product quantizes itself.
constexpr int64_t kFp4QuantizeInside = 8;
// Most tokens of its kernel for few.
constexpr int64_t kFp4Few = 32;
// its kernels for few tokens and for many
cudaError_t launch_fp4_gemm_few(const Fp4Gemm &g, const LaunchCtx &ctx);
cudaError_t launch_fp4_gemm_pair(const Fp4Gemm &g, const LaunchCtx &ctx);
// The product with W = [gate | up] of 2 N rows, N a multiple of 64, and from the bf16
// gate and up (with bias; no residual) silu(gate) * up, quantized with tensor scale
// a_scale: a_codes [M, N / 2] and tiled a_scales, the same as a linear, then the
// quantizer, would leave.
cudaError_t launch_fp4_gemm_glu(const Fp4Gemm &g, const LaunchCtx &ctx);

enum class Norm : int { kRms = 0, kLayer = 1 };

// h = x_factor * x + branch_factor * gate * post(branch);
// n = norm(h) * weight + bias, then * (1 + scale) + shift.
struct BlockNorm {
    const uint16_t *x, *branch;
    int64_t ldx, ldb;
    const void *post_weight, *weight, *bias;  // [H] of one type
    bool w_f32;
    const uint16_t *gate, *scale, *shift;  // a row for each group of tokens, ldm apart
    int64_t ldm, tokens_per_group;
    float x_factor, branch_factor, eps;
    Norm norm;
    int64_t T;
    int H;
    uint16_t *h;  // may be null
    int64_t ldh;
    uint16_t *n;  // bf16, or null: codes and tiled scales
    int64_t ldn;
    bool nv;
    float n_scale;
    uint8_t *codes, *scales;
};
cudaError_t launch_block_norm(const BlockNorm &b, const LaunchCtx &ctx);

}  // namespace ck
