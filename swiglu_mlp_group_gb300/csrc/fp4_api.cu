// fp4_api.cu -- the C ABI of the microscaled 4-bit operators and of the block
// norm (include/ck.h): argument validation and launches, nothing else.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ck.h"
#include "fp4.h"
#include "internal.h"
#include "trace.h"

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxK = 32768;
constexpr int64_t kMaxNorm = 16384;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round_up(size_t v) { return (v + 255) / 256 * 256; }
ck_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CK_OK : CK_ERR_CUDA; }
bool known(ck_fp4_format f) { return f == CK_FP4_MX || f == CK_FP4_NV; }

// A tensor's scale: 1 of an MX tensor; such that its products with block scales
// and codes are normal f32 numbers.
bool scale_ok(ck_fp4_format f, float s) { return f == CK_FP4_MX ? s == 1.f : s >= 0x1p-60f && s <= 0x1p60f; }
bool codes_shape(int64_t rows, int64_t K) { return rows >= 1 && rows <= kMaxRows && K >= 32 && K <= kMaxK && K % 32 == 0; }
// Columns of y.  Tiles of many tokens have up to 384 of them, and count those past N in
// 32 bits, too.
bool columns_ok(int64_t M, int64_t N) {
    return N >= 1 && N % 8 == 0 && N <= (M > ck::kFp4Few ? kMaxRows - 383 : kMaxRows);
}

ck::LaunchCtx context(ck_stream_t stream, unsigned int *status) {
    ck::LaunchCtx c;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    c.status = status;
    c.timeout_ns = ck::wait_timeout_ns();
    c.pdl = true;
    return c;
}

// The quantizer in front of a call's product lets it in behind its own wait, so
// that the product may read the weight at once; with overlapped launches, where
// the caller vouches for the weight, earlier.
ck::LaunchCtx quantizer_context(ck_stream_t stream, unsigned int *status) {
    ck::LaunchCtx c = context(stream, status);
    c.early_trigger = ck::launch_overlap();
    return c;
}

struct Codes {
    size_t codes, scales, end;
};
Codes codes_at(size_t off, int64_t M, int64_t K, bool nv) {
    Codes c;
    c.codes = off;
    c.scales = off + round_up(static_cast<size_t>(M) * K / 2);
    c.end = c.scales + round_up(ck::fp4_scale_bytes(M, K, nv));
    return c;
}
struct MlpWs {
    Codes x, a;
    size_t h, total;
};
MlpWs mlp_ws(int64_t M, int64_t H, int64_t I, bool nv) {
    MlpWs w;
    w.x = codes_at(0, M, H, nv);
    w.h = w.x.end;
    w.a = codes_at(w.h + round_up(static_cast<size_t>(M) * 2 * I * 2), M, I, nv);
    w.total = w.a.end;
    return w;
}

uint8_t *at(void *base, size_t off) { return static_cast<uint8_t *>(base) + off; }

ck_status check_rows(const void *x, int64_t M, int64_t K, int64_t ldx, ck_input_act act, int per16) {
    if (act != CK_ACT_NONE && act != CK_ACT_SWIGLU) return CK_ERR_INVALID;
    if (!codes_shape(M, K)) return CK_ERR_SHAPE;
    if (ldx < (act == CK_ACT_SWIGLU ? 2 * K : K) || ldx % per16 != 0 || ldx > kMaxRows) return CK_ERR_SHAPE;
    return aligned16(x) ? CK_OK : CK_ERR_ALIGN;
}

ck::Fp4Gemm gemm(const uint8_t *x, const uint8_t *xs, int64_t M, int64_t K, bool nv, const void *W, const void *ws,
                 int64_t N, float alpha, const void *bias, const void *residual, void *y, bool settled) {
    ck::Fp4Gemm g;
    g.x = x, g.xs = xs, g.w = static_cast<const uint8_t *>(W), g.ws = static_cast<const uint8_t *>(ws);
    g.M = M, g.N = N, g.K = K, g.nv = nv, g.alpha = alpha;
    g.bias = bias, g.residual = residual, g.y = y;
    g.weights_settled = settled;
    return g;
}

// Whether [p, p + n) and [q, q + m) share a byte.
bool overlap(const void *p, size_t n, const void *q, size_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

// One linear: with few tokens a single kernel, which quantizes x in every CTA (and so
// while others write y), else the quantizer and the product.  settled: the kernel ahead
// is this call's, let this one in behind its own wait, and does not write W.
ck_status run_linear(const void *x, int64_t M, int64_t K, int64_t ldx, ck_input_act act, bool nv, float x_scale,
                     const void *W, const void *w_scales, float w_scale, int64_t N, const void *bias,
                     const void *residual, void *y, void *ws, const Codes &c, bool settled, unsigned int *status,
                     ck_stream_t stream) {
    const size_t x_bytes = (static_cast<size_t>(M - 1) * ldx + (act == CK_ACT_SWIGLU ? 2 * K : K)) * 2;
    if (M <= ck::kFp4QuantizeInside && !overlap(x, x_bytes, y, static_cast<size_t>(M) * N * 2)) {
        ck::Fp4Gemm g = gemm(nullptr, nullptr, M, K, nv, W, w_scales, N, x_scale * w_scale, bias, residual, y,
                             settled || ck::launch_overlap());
        g.x_bf16 = x, g.ldx = ldx, g.swiglu = act == CK_ACT_SWIGLU, g.x_scale = x_scale;
        return from_cuda(ck::launch_fp4_gemm_few(g, quantizer_context(stream, status)));
    }
    if (ck::launch_fp4_quantize(x, false, act == CK_ACT_SWIGLU ? ck::Act::kSwiglu : ck::Act::kNone, M, K, ldx, nv,
                                x_scale, at(ws, c.codes), at(ws, c.scales),
                                quantizer_context(stream, status)) != cudaSuccess)
        return CK_ERR_CUDA;
    return from_cuda(ck::launch_fp4_gemm(gemm(at(ws, c.codes), at(ws, c.scales), M, K, nv, W, w_scales, N,
                                              x_scale * w_scale, bias, residual, y, true),
                                         context(stream, status)));
}

// The arguments that both forms of the block norm share.
ck_status check_norm(const ck::BlockNorm &b, ck_norm norm, ck_dtype wdt, const void *h_out, int64_t ldh) {
    if (!b.x) return CK_ERR_NULL;
    if (!b.branch && (b.post_weight || b.gate)) return CK_ERR_NULL;
    if (norm != CK_NORM_RMS && norm != CK_NORM_LAYER) return CK_ERR_INVALID;
    if (!isfinite(b.x_factor) || !isfinite(b.branch_factor) || !isfinite(b.eps) || b.eps < 0.f) return CK_ERR_INVALID;
    if (wdt != CK_F32 && wdt != CK_BF16) return CK_ERR_DTYPE;
    auto rows = [&](int64_t ld) { return ld >= b.H && ld % 8 == 0 && ld <= kMaxRows; };
    if (b.T < 1 || b.T > kMaxRows || b.H < 8 || b.H % 8 != 0) return CK_ERR_SHAPE;
    if (!rows(b.ldx) || (b.branch && !rows(b.ldb)) || (h_out && !rows(ldh))) return CK_ERR_SHAPE;
    if (b.tokens_per_group < 0 || b.tokens_per_group > kMaxRows) return CK_ERR_SHAPE;
    if ((b.gate || b.scale || b.shift) && b.tokens_per_group > 0 && b.tokens_per_group < b.T && !rows(b.ldm))
        return CK_ERR_SHAPE;
    if (!aligned16(b.x) || !aligned16(b.branch) || !aligned16(b.post_weight) || !aligned16(b.weight) ||
        !aligned16(b.bias) || !aligned16(b.gate) || !aligned16(b.scale) || !aligned16(b.shift) || !aligned16(h_out))
        return CK_ERR_ALIGN;
    return CK_OK;
}

ck::BlockNorm norm_args(const void *x, int64_t ldx, const void *branch, int64_t ldb, int64_t T, int64_t H,
                        const void *post_weight, const void *gate, const void *scale, const void *shift, int64_t ldm,
                        int64_t tokens_per_group, float x_factor, float branch_factor, ck_norm norm,
                        const void *weight, const void *bias, ck_dtype wdt, float eps, void *h_out, int64_t ldh) {
    ck::BlockNorm b = {};
    auto bits = [](const void *p) { return static_cast<const uint16_t *>(p); };
    b.x = bits(x), b.ldx = ldx, b.branch = bits(branch), b.ldb = ldb;
    b.T = T, b.H = H < 1 || H > kMaxNorm ? 0 : static_cast<int>(H);
    b.post_weight = post_weight, b.weight = weight, b.bias = bias, b.w_f32 = wdt == CK_F32;
    b.gate = bits(gate), b.scale = bits(scale), b.shift = bits(shift);
    b.ldm = ldm;
    // one group: every token reads the first row
    b.tokens_per_group = tokens_per_group >= T ? 0 : tokens_per_group;
    b.x_factor = x_factor, b.branch_factor = branch_factor, b.eps = eps;
    b.norm = norm == CK_NORM_LAYER ? ck::Norm::kLayer : ck::Norm::kRms;
    b.h = static_cast<uint16_t *>(h_out), b.ldh = ldh;
    return b;
}

}  // namespace

extern "C" {

CK_API size_t ck_fp4_scale_bytes(ck_fp4_format format, int64_t rows, int64_t K) {
    return known(format) && codes_shape(rows, K) ? ck::fp4_scale_bytes(rows, K, format == CK_FP4_NV) : 0;
}

CK_API ck_status ck_fp4_quantize(const void *x, ck_dtype xdt, int64_t M, int64_t K, int64_t ldx, ck_input_act act,
                                 ck_fp4_format format, float tensor_scale, void *codes, void *scales,
                                 ck_stream_t stream) {
    CK_TRACE("ck_fp4_quantize");
    if (!x || !codes || !scales) return CK_ERR_NULL;
    if (!known(format) || !scale_ok(format, tensor_scale)) return CK_ERR_INVALID;
    if (xdt != CK_BF16 && xdt != CK_F32) return CK_ERR_DTYPE;
    if (xdt == CK_F32 && act == CK_ACT_SWIGLU) return CK_ERR_DTYPE;
    if (ck_status st = check_rows(x, M, K, ldx, act, xdt == CK_F32 ? 4 : 8); st != CK_OK) return st;
    if (!aligned16(codes) || !aligned16(scales)) return CK_ERR_ALIGN;
    unsigned int *status = nullptr;
    if (int st = ck::device_ready_status(&status); st != CK_OK) return static_cast<ck_status>(st);
    return from_cuda(ck::launch_fp4_quantize(x, xdt == CK_F32, act == CK_ACT_SWIGLU ? ck::Act::kSwiglu : ck::Act::kNone,
                                             M, K, ldx, format == CK_FP4_NV, tensor_scale,
                                             static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales),
                                             context(stream, status)));
}

CK_API ck_status ck_fp4_tile_scales(const void *scales, int64_t rows, int64_t K, ck_fp4_format format, void *tiled,
                                    ck_stream_t stream) {
    CK_TRACE("ck_fp4_tile_scales");
    if (!scales || !tiled) return CK_ERR_NULL;
    if (!known(format)) return CK_ERR_INVALID;
    if (!codes_shape(rows, K)) return CK_ERR_SHAPE;
    if (!aligned16(tiled)) return CK_ERR_ALIGN;
    unsigned int *status = nullptr;
    if (int st = ck::device_ready_status(&status); st != CK_OK) return static_cast<ck_status>(st);
    return from_cuda(ck::launch_fp4_tile_scales(static_cast<const uint8_t *>(scales), rows, K, format == CK_FP4_NV,
                                                static_cast<uint8_t *>(tiled), context(stream, status)));
}

CK_API ck_status ck_fp4_gemm(const void *codes, const void *scales, int64_t M, int64_t K, ck_fp4_format format,
                             const void *W, const void *w_scales, int64_t N, float alpha, const void *bias,
                             const void *residual, void *y, ck_stream_t stream) {
    CK_TRACE("ck_fp4_gemm");
    if (!codes || !scales || !W || !w_scales || !y) return CK_ERR_NULL;
    if (!known(format) || !isfinite(alpha)) return CK_ERR_INVALID;
    if (!codes_shape(M, K) || !columns_ok(M, N)) return CK_ERR_SHAPE;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(W) || !aligned16(w_scales) || !aligned16(y) ||
        !aligned16(bias) || !aligned16(residual))
        return CK_ERR_ALIGN;
    unsigned int *status = nullptr;
    if (int st = ck::device_ready_status(&status); st != CK_OK) return static_cast<ck_status>(st);
    return from_cuda(ck::launch_fp4_gemm(
        gemm(static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), M, K, format == CK_FP4_NV, W,
             w_scales, N, alpha, bias, residual, y, ck::launch_overlap()),
        context(stream, status)));
}

CK_API size_t ck_fp4_linear_workspace_bytes(int64_t M, int64_t K, ck_fp4_format format) {
    return known(format) && codes_shape(M, K) ? codes_at(0, M, K, format == CK_FP4_NV).end : 0;
}

CK_API ck_status ck_fp4_linear(const void *x, int64_t M, int64_t K, int64_t ldx, ck_input_act act,
                               ck_fp4_format format, float x_scale, const void *W, const void *w_scales,
                               float w_scale, int64_t N, const void *bias, const void *residual, void *y, void *ws,
                               size_t ws_bytes, ck_stream_t stream) {
    CK_TRACE("ck_fp4_linear");
    if (!x || !W || !w_scales || !y) return CK_ERR_NULL;
    if (!known(format) || !scale_ok(format, x_scale) || !scale_ok(format, w_scale)) return CK_ERR_INVALID;
    if (ck_status st = check_rows(x, M, K, ldx, act, 8); st != CK_OK) return st;
    if (!columns_ok(M, N)) return CK_ERR_SHAPE;
    if (!aligned16(W) || !aligned16(w_scales) || !aligned16(y) || !aligned16(bias) || !aligned16(residual))
        return CK_ERR_ALIGN;
    const bool nv = format == CK_FP4_NV;
    const Codes c = codes_at(0, M, K, nv);
    if (!ws || ws_bytes < c.end) return CK_ERR_WORKSPACE;
    if (!aligned16(ws)) return CK_ERR_ALIGN;
    unsigned int *status = nullptr;
    if (int st = ck::device_ready_status(&status); st != CK_OK) return static_cast<ck_status>(st);
    return run_linear(x, M, K, ldx, act, nv, x_scale, W, w_scales, w_scale, N, bias, residual, y, ws, c, false, status,
                      stream);
}

CK_API size_t ck_fp4_swiglu_mlp_workspace_bytes(int64_t M, int64_t H, int64_t I, ck_fp4_format format) {
    return known(format) && codes_shape(M, H) && codes_shape(M, I) ? mlp_ws(M, H, I, format == CK_FP4_NV).total : 0;
}

CK_API ck_status ck_fp4_swiglu_mlp(const void *x, int64_t M, int64_t H, int64_t I, ck_fp4_format format, float x_scale,
                                   const void *Wgu, const void *gu_scales, float gu_scale, const void *bgu,
                                   float a_scale, const void *Wd, const void *d_scales, float d_scale, const void *bd,
                                   const void *residual, void *y, void *ws, size_t ws_bytes, ck_stream_t stream) {
    CK_TRACE("ck_fp4_swiglu_mlp");
    if (!x || !Wgu || !gu_scales || !Wd || !d_scales || !y) return CK_ERR_NULL;
    if (!known(format) || !scale_ok(format, x_scale) || !scale_ok(format, gu_scale) || !scale_ok(format, a_scale) ||
        !scale_ok(format, d_scale))
        return CK_ERR_INVALID;
    if (ck_status st = check_rows(x, M, H, H, CK_ACT_NONE, 8); st != CK_OK) return st;
    if (!codes_shape(M, I)) return CK_ERR_SHAPE;
    if (!aligned16(Wgu) || !aligned16(gu_scales) || !aligned16(bgu) || !aligned16(Wd) || !aligned16(d_scales) ||
        !aligned16(bd) || !aligned16(residual) || !aligned16(y))
        return CK_ERR_ALIGN;
    const bool nv = format == CK_FP4_NV;
    const MlpWs w = mlp_ws(M, H, I, nv);
    if (!ws || ws_bytes < w.total) return CK_ERR_WORKSPACE;
    if (!aligned16(ws)) return CK_ERR_ALIGN;
    unsigned int *status = nullptr;
    if (int st = ck::device_ready_status(&status); st != CK_OK) return static_cast<ck_status>(st);
    if (M > ck::kFp4Few && I % 64 == 0) {
        // gate and up never leave the chip as such: the first product's epilogue
        // quantizes silu(gate) * up (up's rows of a tile begin at a half or a whole of
        // 128 rows of scales for such I)
        if (ck::launch_fp4_quantize(x, false, ck::Act::kNone, M, H, H, nv, x_scale, at(ws, w.x.codes), at(ws, w.x.scales),
                                    quantizer_context(stream, status)) != cudaSuccess)
            return CK_ERR_CUDA;
        ck::Fp4Gemm g = gemm(at(ws, w.x.codes), at(ws, w.x.scales), M, H, nv, Wgu, gu_scales, I, x_scale * gu_scale, bgu,
                             nullptr, nullptr, true);
        g.a_codes = at(ws, w.a.codes), g.a_scales = at(ws, w.a.scales), g.a_scale = a_scale;
        if (ck::launch_fp4_gemm_glu(g, context(stream, status)) != cudaSuccess) return CK_ERR_CUDA;
        return from_cuda(ck::launch_fp4_gemm(gemm(at(ws, w.a.codes), at(ws, w.a.scales), M, I, nv, Wd, d_scales, H,
                                                  a_scale * d_scale, bd, residual, y, true),
                                             context(stream, status)));
    }
    if (ck_status st = run_linear(x, M, H, H, CK_ACT_NONE, nv, x_scale, Wgu, gu_scales, gu_scale, 2 * I, bgu, nullptr,
                                  at(ws, w.h), ws, w.x, false, status, stream);
        st != CK_OK)
        return st;
    return run_linear(at(ws, w.h), M, I, 2 * I, CK_ACT_SWIGLU, nv, a_scale, Wd, d_scales, d_scale, H, bd, residual, y,
                      ws, w.a, true, status, stream);
}

CK_API ck_status ck_block_norm(const void *x, int64_t ldx, const void *branch, int64_t ldb, int64_t T, int64_t H,
                               const void *post_weight, const void *gate, const void *scale, const void *shift,
                               int64_t ldm, int64_t tokens_per_group, float x_factor, float branch_factor,
                               ck_norm norm, const void *weight, const void *bias, ck_dtype wdt, float eps,
                               void *h_out, int64_t ldh, void *n_out, int64_t ldn, ck_stream_t stream) {
    CK_TRACE("ck_block_norm");
    if (!n_out) return CK_ERR_NULL;
    ck::BlockNorm b = norm_args(x, ldx, branch, ldb, T, H, post_weight, gate, scale, shift, ldm, tokens_per_group,
                                x_factor, branch_factor, norm, weight, bias, wdt, eps, h_out, ldh);
    if (ck_status st = check_norm(b, norm, wdt, h_out, ldh); st != CK_OK) return st;
    if (ldn < H || ldn % 8 != 0 || ldn > kMaxRows) return CK_ERR_SHAPE;
    if (!aligned16(n_out)) return CK_ERR_ALIGN;
    b.n = static_cast<uint16_t *>(n_out), b.ldn = ldn, b.n_scale = 1.f;
    unsigned int *status = nullptr;
    if (int st = ck::device_ready_status(&status); st != CK_OK) return static_cast<ck_status>(st);
    return from_cuda(ck::launch_block_norm(b, context(stream, status)));
}

CK_API ck_status ck_block_norm_fp4(const void *x, int64_t ldx, const void *branch, int64_t ldb, int64_t T, int64_t H,
                                   const void *post_weight, const void *gate, const void *scale, const void *shift,
                                   int64_t ldm, int64_t tokens_per_group, float x_factor, float branch_factor,
                                   ck_norm norm, const void *weight, const void *bias, ck_dtype wdt, float eps,
                                   void *h_out, int64_t ldh, ck_fp4_format format, float n_scale, void *codes,
                                   void *scales, ck_stream_t stream) {
    CK_TRACE("ck_block_norm_fp4");
    if (!codes || !scales) return CK_ERR_NULL;
    if (!known(format) || !scale_ok(format, n_scale)) return CK_ERR_INVALID;
    ck::BlockNorm b = norm_args(x, ldx, branch, ldb, T, H, post_weight, gate, scale, shift, ldm, tokens_per_group,
                                x_factor, branch_factor, norm, weight, bias, wdt, eps, h_out, ldh);
    if (ck_status st = check_norm(b, norm, wdt, h_out, ldh); st != CK_OK) return st;
    if (H % 32 != 0) return CK_ERR_SHAPE;
    if (!aligned16(codes) || !aligned16(scales)) return CK_ERR_ALIGN;
    b.nv = format == CK_FP4_NV, b.n_scale = n_scale;
    b.codes = static_cast<uint8_t *>(codes), b.scales = static_cast<uint8_t *>(scales);
    unsigned int *status = nullptr;
    if (int st = ck::device_ready_status(&status); st != CK_OK) return static_cast<ck_status>(st);
    return from_cuda(ck::launch_block_norm(b, context(stream, status)));
}

}  // extern "C"
