// fp4_gemm_few.cu -- the 4-bit product for few tokens:
//
//   y[m, n] = bf16( alpha * sum_k X[m, k] W[n, k] + bias[n] + residual[m, n] )
//
// X, W: E2M1 codes times the scales of their blocks (fp4_core.cuh).  The weight's
// bytes are the floor, so the weight is the operand that the tensor cores walk:
// a CTA has 128 rows of W as tcgen05.mma's A and TN tokens as its B, D[n, m] in
// TMEM, and the scales' multiplication is the instruction's own -- nothing is
// decoded.  K is split over the S CTAs of a cluster so that every SM has weight to
// fetch; each CTA sends the columns of its partial sums to the CTA that finishes
// them through distributed shared memory, which adds them in the order of the
// CTAs' ranks (f32: the result does not depend on timing).
//
// Roles (6 warps): warp 0 TMA producer, warp 1 TMEM and MMA issue, warps 2..5 the
// epilogue (one 32-lane quarter of TMEM each).  Up to 8 tokens can come as bf16: these
// four and four more then quantize, every CTA its own columns of x into the stages
// while the weight is on its way, instead of a kernel ahead (a block needs nothing
// beyond itself, so a CTA does with its share of K).
#include <cuda_bf16.h>

#include "fp4_core.cuh"
#include "launch_util.h"
#include "quant_core.cuh"

namespace ck {
namespace {

constexpr int kThreads = 192;            // without the four more
constexpr int kQuantWarps = 8;
constexpr int kRows = 128;               // rows of W a CTA
constexpr int kStageK = 256;             // 128 bytes of codes a row
constexpr int kABytes = kRows * kStageK / 2;
constexpr int kCtaBytes = 112 * 1024 + 256;  // two CTAs an SM

// Where X comes from: codes, or bf16 x (or [gate | up]) to quantize.
enum class From : int { kCodes, kBf16, kSwiglu };

template <int TN, bool NV>
struct Cfg {
    static constexpr int kWords = kStageK / fp4_word(NV);  // scale words of a stage
    static constexpr int kSfBytes = kWords * 512;
    static constexpr int kBBytes = TN * kStageK / 2;
    static constexpr int kStageBytes = kABytes + kBBytes + 2 * kSfBytes;
    // partial sums, beside the stages: a CTA may send its own while another multiplies
    static constexpr int kRedBytes = TN * kRows * 4;
    static constexpr int kStages = (kCtaBytes - 1024 - 256 - kRedBytes) / kStageBytes;
    static constexpr int kTmemSf = 32;  // first column of the scales
    static constexpr int kTmemCols = 64;
    static constexpr size_t kSmemBytes = static_cast<size_t>(kStages) * kStageBytes + kRedBytes + 256 + 1024;
    static_assert(kTmemSf + 32 <= kTmemCols, "TMEM");
    static_assert(kStageBytes % 1024 == 0 && kStages >= 3 && 8 * (2 * kStages + 1) + 8 <= 256, "stage");
};

struct Args {
    const uint8_t *xs, *ws;
    const __nv_bfloat16 *x;  // to quantize
    int64_t ldx;
    fp4::Scale t;
    int M, N, K, words, splits;  // words: scale words a row
    float alpha;
    const __nv_bfloat16 *bias, *residual;
    __nv_bfloat16 *y;
    bool weights_settled, early_trigger;
    unsigned int *status;
    unsigned long long timeout_ns;
};

template <int TN, bool NV, From FROM>
__global__ void __launch_bounds__(FROM == From::kCodes ? kThreads : kThreads + 128, 2)
fp4_gemm_few_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ Args a) {
    using C = Cfg<TN, NV>;
    constexpr int kStages = C::kStages;
    constexpr bool kQuant = FROM != From::kCodes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t smem_s = (raw_s + 1023u) & ~1023u;
    const uint32_t red_s = smem_s + kStages * C::kStageBytes;
    const float *red = reinterpret_cast<const float *>(smem_raw + (red_s - raw_s));
    const uint32_t bars_s = red_s + C::kRedBytes;
    uint8_t *bars = smem_raw + (bars_s - raw_s);
    auto full = [&](int s) { return bars_s + 8u * s; };
    auto empty = [&](int s) { return bars_s + 8u * (kStages + s); };
    const uint32_t done = bars_s + 8u * (2 * kStages);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 8 * (2 * kStages + 1));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    // a stage: W codes, X codes, W scales, X scales
    auto stage = [&](int s) { return smem_s + s * C::kStageBytes; };
    constexpr int kOffB = kABytes, kOffSfa = kABytes + C::kBBytes, kOffSfb = kOffSfa + C::kSfBytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int n_tile = blockIdx.x / a.splits;
    const int n0 = n_tile * kRows;
    const int num_kb = (a.K + kStageK - 1) / kStageK;
    const int kb0 = num_kb * rank / a.splits, kbs = num_kb * (rank + 1) / a.splits - kb0;
    const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), kQuant ? 1 + kQuantWarps : 1);  // the copies, and the quantizers' warps
            mbar_init(empty(s), 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    cluster_arrive();  // waited for before another CTA's shared memory is written
    const uint32_t tmem = *tmem_slot;
    // A kernel behind this one that reads what settles before it (a weight) may do so
    // once let in: with x quantized here, no kernel ahead has waited for it.
    if (!kQuant || a.early_trigger) pdl_launch_dependents();

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int issued = 0;
        if (elect_one()) {
            tma_prefetch_desc(&tm_w);
            if constexpr (!kQuant) tma_prefetch_desc(&tm_x);
            const uint8_t *ws = a.ws + (static_cast<int64_t>(n_tile) * a.words) * 512;
            auto sf_bytes = [&](int kb) {
                const int left = a.words - kb * C::kWords;
                return static_cast<uint32_t>((left < C::kWords ? left : C::kWords) * 512);
            };
            auto load_w = [&](int s, int kb) {
                const uint32_t sf = sf_bytes(kb);
                mbar_arrive_expect_tx(full(s), kABytes + sf + (kQuant ? 0 : C::kBBytes + sf));
                tma_load_2d(stage(s), &tm_w, full(s), kb * (kStageK / 2), n0);
                bulk_load_1d(stage(s) + kOffSfa, ws + static_cast<int64_t>(kb) * C::kSfBytes, sf, full(s));
            };
            auto load_x = [&](int s, int kb) {
                if constexpr (!kQuant) {
                    tma_load_2d(stage(s) + kOffB, &tm_x, full(s), kb * (kStageK / 2), 0);
                    bulk_load_1d(stage(s) + kOffSfb, a.xs + static_cast<int64_t>(kb) * C::kSfBytes, sf_bytes(kb), full(s));
                }
            };
            if (!a.weights_settled) pdl_wait();
            const int pre = kbs < kStages ? kbs : kStages;
            for (int i = 0; i < pre; ++i) load_w(i, kb0 + i);
            if (a.weights_settled) pdl_wait();
            for (int i = 0; i < pre; ++i) load_x(i, kb0 + i);
            issued = pre;
            int s = 0;
            uint32_t ph = 0;
            for (int i = pre; i < kbs; ++i) {
                if (!mbar_wait_spin(empty(s), ph, ctl)) break;
                load_w(s, kb0 + i);
                load_x(s, kb0 + i);
                issued = i + 1;
                if (++s == kStages) s = 0, ph ^= 1u;
            }
            if (*abort_flag) {
                const int first = issued > kStages ? issued - kStages : 0;
                for (int i = first; i < issued; ++i)
                    mbar_wait_drain(full(i % kStages), (i / kStages) & 1, a.timeout_ns, a.status);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        const uint32_t sfa = tmem + C::kTmemSf, sfb = sfa + 16;
        if (elect_one()) {
            bool ok = true;
            int s = 0;
            uint32_t ph = 0;
            for (int i = 0; i < kbs; ++i) {
                ok = mbar_wait_spin(full(s), ph, ctl);
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t ad = sdesc_kmajor_sw128(stage(s)), bd = sdesc_kmajor_sw128(stage(s) + kOffB);
                const int words = a.words - (kb0 + i) * C::kWords;
#pragma unroll
                for (int w = 0; w < C::kWords; ++w)
                    if (w < words) {
                        tmem_copy_scales(sfa + 4 * w, sdesc_scales(stage(s) + kOffSfa + 512 * w));
                        tmem_copy_scales(sfb + 4 * w, sdesc_scales(stage(s) + kOffSfb + 512 * w));
                    }
                const int left = a.K - (kb0 + i) * kStageK;  // columns of K from here on
#pragma unroll
                for (int k = 0; k < kStageK / 64; ++k)
                    if (64 * k < left) {
                        const int w = NV ? k : k / 2;
                        mma_fp4<NV, false>(tmem, ad + 2 * k, bd + 2 * k, idesc_fp4(kRows, TN, NV, NV ? 0 : k & 1),
                                           sfa + 4 * w, sfb + 4 * w, i > 0 || k > 0 ? 1u : 0u);
                    }
                mma_commit(empty(s));
                if (++s == kStages) s = 0, ph ^= 1u;
            }
            mma_commit(done);
            if (!ok) mbar_wait_drain(done, 0, a.timeout_ns, a.status);
        }
        __syncwarp();
    } else if constexpr (kQuant) {
        // ------------------------------------------------------------ quantizers
        // Items (a token's 256 columns of a stage, 8 a lane) go round the warps, stage
        // after stage; a warp quantizes four at a time, the next four on their way: one
        // alone is some 500 clocks from its load to its codes, most of them latency.
        constexpr int kBatch = 4;
        constexpr int kBlock = fp4::block_lanes(NV);
        const int step_kb = kQuantWarps / a.M, step_t = kQuantWarps - step_kb * a.M;
        pdl_wait();
        if (!a.early_trigger) pdl_launch_dependents();
        struct Item {
            int kb, t;
        };
        auto forward = [&](Item &it) {
            it.kb += step_kb, it.t += step_t;
            if (it.t >= a.M) it.t -= a.M, ++it.kb;
        };
        uint4 u[kBatch], v[FROM == From::kSwiglu ? kBatch : 1];
        Item ahead{(warp - 2) / a.M, (warp - 2) % a.M}, now = ahead;
        auto fetch = [&] {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int col = (kb0 + ahead.kb) * kStageK + lane * 8;
                u[j] = make_uint4(0, 0, 0, 0);
                if constexpr (FROM == From::kSwiglu) v[j] = u[j];
                if (ahead.kb < kbs && col < a.K) {
                    const __nv_bfloat16 *p = a.x + ahead.t * a.ldx + col;
                    u[j] = *reinterpret_cast<const uint4 *>(p);
                    if constexpr (FROM == From::kSwiglu) v[j] = *reinterpret_cast<const uint4 *>(p + a.K);
                }
                forward(ahead);
            }
        };
        fetch();
        int kb = 0, s = 0;  // the stage that is being filled
        uint32_t ph = 1;
        bool waited = false, ok = true;
        auto wait = [&] {  // (the first round's is over at once)
            if (!waited) {
                int got = 0;
                if (lane == 0) got = mbar_wait_spin(empty(s), ph, ctl) ? 1 : 0;
                ok = __shfl_sync(0xffffffffu, got, 0) != 0;
                waited = true;
            }
            return ok;
        };
        // Hands the stages before `to` over.
        auto hand_over = [&](int to) {
            for (; kb < to; ++kb) {
                if (!wait()) return;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full(s));
                waited = false;
                if (++s == kStages) s = 0, ph ^= 1u;
            }
        };
        while (now.kb < kbs && ok) {
            uint32_t codes[kBatch], scale[kBatch];
            uint64_t q[kBatch][4];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const uint32_t ru[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (FROM == From::kSwiglu) {
                        const uint32_t rv[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                        q[j][e] = f32x2(-qc::silu_mul(__uint_as_float(ru[e] << 16), __uint_as_float(rv[e] << 16)),
                                        -qc::silu_mul(__uint_as_float(ru[e] & 0xffff0000u), __uint_as_float(rv[e] & 0xffff0000u)));
                    } else {
                        q[j][e] = fp4::unpack2_neg(ru[e]);
                    }
                }
            }
            fetch();
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                codes[j] = fp4::quantize8<NV>(q[j], a.t, scale[j]);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (now.kb < kbs && ok) {
                    hand_over(now.kb);
                    if (ok && wait()) {
                        // 128-byte rows, their 16-byte pieces swizzled by the row
                        const int t = now.t;
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(stage(s) + kOffB + t * 128 + (((lane >> 2) ^ (t & 7)) << 4) +
                                                                     (lane & 3) * 4),
                                     "r"(codes[j])
                                     : "memory");
                        if (lane % kBlock == 0)
                            asm volatile("st.shared.u8 [%0], %1;" ::"r"(stage(s) + kOffSfb + lane / (4 * kBlock) * 512 + t * 16 +
                                                                      (lane / kBlock & 3)),
                                         "r"(scale[j])
                                         : "memory");
                    }
                }
                forward(now);
            }
        }
        if (ok) hand_over(kbs);
    }
    // ---------------------------------------------------------------- epilogue
    // Column c of the tile is finished by the CTA of rank c / own.
    const int own = TN / a.splits;
    bool ok = true;
    const bool finishes = warp >= 2 && warp < 6;
    if (finishes) {
        int got = 0;
        if (lane == 0) got = mbar_wait(done, 0, ctl) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        tc_fence_after_sync();
    }
    __syncwarp();
    cluster_wait();  // every CTA of the cluster has begun
    if (finishes) {
        const int q = warp & 3;
        if (ok) {
            const int r = q * 32 + lane;
            constexpr int kStep = TN < 16 ? 8 : 16;
#pragma unroll
            for (int c0 = 0; c0 < TN; c0 += kStep) {
                if (c0 >= a.M) break;
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c0, v);
                tmem_wait_ld16(v);
#pragma unroll
                for (int j = 0; j < kStep; ++j) {
                    const int c = c0 + j, owner = c / own;
                    if (c >= a.M) break;
                    const uint32_t at = red_s + 4u * ((rank * own + c - owner * own) * kRows + r);
                    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapa_shared(at, owner)), "r"(v[j]) : "memory");
                }
            }
        }
        tc_fence_before_sync();
    }
    cluster_sync();
    if (finishes && !*abort_flag) {
        const int t = threadIdx.x - 64;
        const int n = n0 + 2 * (t & 63);
        if (n < a.N) {
            float b0 = 0.f, b1 = 0.f;
            if (a.bias != nullptr) {
                const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162 *>(a.bias + n);
                b0 = __low2float(b), b1 = __high2float(b);
            }
            if constexpr (!kQuant) pdl_wait();  // the residual may come from the kernel ahead
            for (int c = t >> 6; c < own; c += 2) {
                const int m = rank * own + c;
                if (m >= a.M) break;
                const int64_t at = static_cast<int64_t>(m) * a.N + n;
                float r0 = 0.f, r1 = 0.f;
                if (a.residual != nullptr) {
                    const __nv_bfloat162 r = *reinterpret_cast<const __nv_bfloat162 *>(a.residual + at);
                    r0 = __low2float(r), r1 = __high2float(r);
                }
                float s0 = 0.f, s1 = 0.f;
                for (int src = 0; src < a.splits; ++src) {
                    const float2 p = *reinterpret_cast<const float2 *>(red + (src * own + c) * kRows + 2 * (t & 63));
                    s0 += p.x, s1 += p.y;
                }
                *reinterpret_cast<__nv_bfloat162 *>(a.y + at) =
                    __floats2bfloat162_rn(a.alpha * s0 + b0 + r0, a.alpha * s1 + b1 + r1);
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int TN, bool NV, From FROM>
cudaError_t launch_t(const Fp4Gemm &g, const LaunchCtx &ctx) {
    using C = Cfg<TN, NV>;
    CUtensorMap mw, mx;
    const int row_bytes = static_cast<int>(g.K / 2);
    if (!tensor_map_2d(&mw, g.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.N, row_bytes, kStageK / 2, kRows,
                       CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if constexpr (FROM == From::kCodes) {
        if (!tensor_map_2d(&mx, g.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.M, row_bytes, kStageK / 2, TN,
                           CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    } else {
        mx = mw;  // not used
    }
    auto kern = fp4_gemm_few_kernel<TN, NV, FROM>;
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), static_cast<int>(C::kSmemBytes));
        e != cudaSuccess)
        return e;
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const int64_t n_tiles = (g.N + kRows - 1) / kRows;
    const int64_t num_kb = (g.K + kStageK - 1) / kStageK;
    if (g.M > TN) return cudaErrorInvalidValue;  // one tile of tokens
    // as many parts of K as leave all CTAs resident at once
    int splits = 1;
    while (splits < 8 && n_tiles * splits * 2 <= 2 * sms && splits * 2 <= num_kb) splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n_tiles * splits));
    cfg.blockDim = dim3(FROM == From::kCodes ? kThreads : kThreads + 128);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 2 : 1;
    Args a = {};
    a.xs = g.xs, a.ws = g.ws;
    a.x = static_cast<const __nv_bfloat16 *>(g.x_bf16), a.ldx = g.ldx;
    a.t = fp4::scale_of(g.x_scale);
    a.M = static_cast<int>(g.M), a.N = static_cast<int>(g.N), a.K = static_cast<int>(g.K);
    a.words = static_cast<int>(fp4_words(g.K, g.nv));
    a.splits = splits;
    a.alpha = g.alpha;
    a.bias = static_cast<const __nv_bfloat16 *>(g.bias), a.residual = static_cast<const __nv_bfloat16 *>(g.residual);
    a.y = static_cast<__nv_bfloat16 *>(g.y);
    a.weights_settled = g.weights_settled, a.early_trigger = ctx.early_trigger;
    a.status = ctx.status, a.timeout_ns = ctx.timeout_ns;
    return cudaLaunchKernelEx(&cfg, kern, mw, mx, a);
}

template <bool NV>
cudaError_t launch_n(const Fp4Gemm &g, const LaunchCtx &ctx) {
    if (g.x_bf16 != nullptr) {
        if (g.M > kFp4QuantizeInside) return cudaErrorInvalidValue;
        return g.swiglu ? launch_t<8, NV, From::kSwiglu>(g, ctx) : launch_t<8, NV, From::kBf16>(g, ctx);
    }
    if (g.M <= 8) return launch_t<8, NV, From::kCodes>(g, ctx);
    if (g.M <= 16) return launch_t<16, NV, From::kCodes>(g, ctx);
    return launch_t<32, NV, From::kCodes>(g, ctx);
}

}  // namespace

cudaError_t launch_fp4_gemm_few(const Fp4Gemm &g, const LaunchCtx &ctx) {
    return g.nv ? launch_n<true>(g, ctx) : launch_n<false>(g, ctx);
}

// Up to 32 tokens the weight's bytes count, and a tile of 256 tokens leaves most SMs
// without any (32 x 4096 -> 4096: 6.5 us against 8.1); with a second tile of tokens here,
// 33 took 7.4 against 8.2, but 12.4 against the other's 8.6 at -> 12288.
cudaError_t launch_fp4_gemm(const Fp4Gemm &g, const LaunchCtx &ctx) {
    return g.M > kFp4Few ? launch_fp4_gemm_pair(g, ctx) : launch_fp4_gemm_few(g, ctx);
}

}  // namespace ck
