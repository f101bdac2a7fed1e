// fp4_gemm_pair.cu -- the 4-bit product for many tokens:
//
//   y[m, n] = bf16( alpha * sum_k X[m, k] W[n, k] + bias[n] + residual[m, n] )
//
// X, W: E2M1 codes times the scales of their blocks (fp4_core.cuh).  CTA pairs
// (tcgen05.mma.cta_group::2): a tile of 256 tokens x PN rows of W on two SMs, each
// holding its 128 tokens, half of W's rows, and the scales of its tokens and of all
// of W's rows; f32 accumulators in TMEM, two of them, so that a tile's epilogue runs
// under the next one's products.  PN is at most 192: two accumulators of 256 columns
// would leave TMEM no room for scales.
//
// Roles (each CTA, 10 warps): warp 0 TMA producer, warp 1 TMEM and, in the leader,
// the issue of the scales' copies to TMEM and of the MMAs (both run in the order of
// their issue), warps 2..9 the epilogue on this CTA's 128 tokens.
#include <cuda_bf16.h>

#include "fp4_core.cuh"
#include "gemm_epilogue.cuh"
#include "launch_util.h"

namespace ck {
namespace {

constexpr int kThreads = 320;
constexpr int kRows = 128;     // tokens a CTA
constexpr int kStageK = 256;   // 128 bytes of codes a row
constexpr int kABytes = kRows * kStageK / 2;

template <int PN, bool NV>
struct Cfg {
    static constexpr int kWords = kStageK / fp4_word(NV);  // scale words of a stage
    static constexpr int kSfaBytes = kWords * 512;
    static constexpr int kBTiles = (PN + 127) / 128;       // 128-row tiles of W's scales
    static constexpr int kSfBytes = kSfaBytes * (1 + kBTiles);
    static constexpr int kBBytes = PN / 2 * kStageK / 2;
    static constexpr int kStageBytes = kABytes + kBBytes + kSfBytes;
    static constexpr int kBarBytes = 256;
    static constexpr int kStages = (225 * 1024 - kBarBytes) / kStageBytes;
    static constexpr int kTmemSf = 2 * PN;                 // the scales' first column
    static constexpr int kSfCols = 4 * kWords * (1 + kBTiles);
    static constexpr int kTmemCols = 512;
    static constexpr size_t kSmemBytes = static_cast<size_t>(kStages) * kStageBytes + kBarBytes + 1024;
    static_assert(kStageBytes % 1024 == 0 && kTmemSf + 2 * kSfCols <= kTmemCols, "layout");
    static_assert(8 * (2 * kStages + 5) + 8 <= kBarBytes && kSmemBytes <= 227 * 1024, "shared memory");
};

struct Args {
    int M, N, K, words, m_pairs;
    float alpha;
    const __nv_bfloat16 *bias, *residual;
    __nv_bfloat16 *y;
    bool weights_settled;
    unsigned int *status;
    unsigned long long timeout_ns;
};

// Eight columns of a row, packed to bf16: alpha * acc + bias + residual.
__device__ __forceinline__ void finish8(const uint32_t *acc, float alpha, const uint4 &b, const uint4 &r, uint32_t *pk) {
    const uint32_t bw[4] = {b.x, b.y, b.z, b.w}, rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float y0 = __uint_as_float(acc[2 * e]) * alpha + __uint_as_float(bw[e] << 16) + __uint_as_float(rw[e] << 16);
        const float y1 = __uint_as_float(acc[2 * e + 1]) * alpha + __uint_as_float(bw[e] & 0xffff0000u) +
                         __uint_as_float(rw[e] & 0xffff0000u);
        const __nv_bfloat162 v = __floats2bfloat162_rn(y0, y1);
        pk[e] = *reinterpret_cast<const uint32_t *>(&v);
    }
}

template <int PN, bool NV>
__global__ void __launch_bounds__(kThreads, 1)
fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws,
                     const __grid_constant__ Args a) {
    using C = Cfg<PN, NV>;
    constexpr int kStages = C::kStages;
    constexpr int kOffB = kABytes, kOffSfa = kABytes + C::kBBytes, kOffSfb = kOffSfa + C::kSfaBytes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t smem_s = (raw_s + 1023u) & ~1023u;
    const uint32_t bars_s = smem_s + kStages * C::kStageBytes;
    uint8_t *bars = smem_raw + (bars_s - raw_s);
    auto full = [&](int s) { return bars_s + 8u * s; };
    auto empty = [&](int s) { return bars_s + 8u * (kStages + s); };
    auto accf = [&](int b) { return bars_s + 8u * (2 * kStages + b); };
    auto acce = [&](int b) { return bars_s + 8u * (2 * kStages + 2 + b); };
    const uint32_t done = bars_s + 8u * (2 * kStages + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 8 * (2 * kStages + 5));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    auto stage = [&](int s) { return smem_s + s * C::kStageBytes; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());  // 0: leader (issues), 1: peer
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int total = a.m_pairs * ((a.N + PN - 1) / PN);
    const int my_tiles = pair < total ? (total - 1 - pair) / npairs + 1 : 0;
    const int num_kb = (a.K + kStageK - 1) / kStageK;
    const int total_kb = my_tiles * num_kb;
    const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 16);  // 8 epilogue warps in each CTA
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int issued = 0;
        if (elect_one()) {
            tma_prefetch_desc(&tm_x);
            tma_prefetch_desc(&tm_w);
            tma_prefetch_desc(&tm_xs);
            tma_prefetch_desc(&tm_ws);
            // both CTAs' copies complete on the leader's barrier, which counts the pair's bytes
            auto load_w = [&](int s, int kb, int tile) {
                if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * C::kStageBytes);
                const uint32_t bar = mapa_shared(full(s), 0);
                const int n0 = tile / a.m_pairs * PN;
                tma_load_2d_pair(stage(s) + kOffB, &tm_w, bar, kb * (kStageK / 2), n0 + rank * (PN / 2));
#pragma unroll
                for (int i = 0; i < C::kBTiles; ++i)
                    tma_load_2d_pair(stage(s) + kOffSfb + i * C::kSfaBytes, &tm_ws, bar, 0,
                                     (((n0 >> 7) + i) * a.words + kb * C::kWords) * 4);
            };
            auto load_x = [&](int s, int kb, int tile) {
                const uint32_t bar = mapa_shared(full(s), 0);
                const int m0 = tile % a.m_pairs * (2 * kRows) + rank * kRows;
                tma_load_2d_pair(stage(s), &tm_x, bar, kb * (kStageK / 2), m0);
                tma_load_2d_pair(stage(s) + kOffSfa, &tm_xs, bar, 0, ((m0 >> 7) * a.words + kb * C::kWords) * 4);
            };
            if (!a.weights_settled) pdl_wait();
            const int pre = total_kb > 0 ? min(kStages, num_kb) : 0;
            for (int i = 0; i < pre; ++i) load_w(i, i, pair);
            if (a.weights_settled) pdl_wait();
            for (int i = 0; i < pre; ++i) load_x(i, i, pair);
            issued = pre;
            int s = pre % kStages, kb = pre == num_kb ? 0 : pre, tile = pre == num_kb ? pair + npairs : pair;
            uint32_t ph = pre / kStages;
            for (int i = pre; i < total_kb; ++i) {
                if (!mbar_wait_spin(empty(s), (ph & 1) ^ 1, ctl)) break;
                load_w(s, kb, tile);
                load_x(s, kb, tile);
                issued = i + 1;
                if (++s == kStages) s = 0, ++ph;
                if (++kb == num_kb) kb = 0, tile += npairs;
            }
            if (*abort_flag) {
                if (rank == 0) {
                    const int first = issued > kStages ? issued - kStages : 0;
                    for (int i = first; i < issued; ++i)
                        mbar_wait_drain(full(i % kStages), (i / kStages) & 1, a.timeout_ns, a.status);
                } else {
                    // copies in flight into this CTA land within microseconds
                    const uint64_t t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < 50000ull) {
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        if (rank == 0) {
            const uint64_t ad0 = sdesc_kmajor_sw128(stage(0)), bd0 = sdesc_kmajor_sw128(stage(0) + kOffB);
            const uint64_t sa0 = sdesc_scales(stage(0) + kOffSfa), sb0 = sdesc_scales(stage(0) + kOffSfb);
            int kb = 0, tile = pair, gc = 0, s = 0, parity = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = 0; i < total_kb; ++i) {
                const int buf = gc & 1;
                if (kb == 0 && gc >= 2) {
                    // the epilogue has read what this accumulator held two tiles ago
                    ok = __all_sync(0xffffffffu, mbar_wait_spin(acce(buf), ((gc >> 1) - 1) & 1, ctl));
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                ok = __all_sync(0xffffffffu, mbar_wait_spin(full(s), ph, ctl));
                if (!ok) break;
                tc_fence_after_sync();
                const bool last = kb + 1 == num_kb;
                if (elect_one()) {
                    const uint64_t step = static_cast<uint64_t>(s) * (C::kStageBytes / 16);
                    const uint32_t sfa = tmem + C::kTmemSf + parity * C::kSfCols, sfb = sfa + 4 * C::kWords;
                    // where W's rows of this tile begin in their scales' 128-row tile
                    const uint32_t sfb_tile = sfb + ((tile / a.m_pairs * PN & 127) >> 5);
#pragma unroll
                    for (int w = 0; w < C::kWords; ++w) {
                        tmem_copy_scales_pair(sfa + 4 * w, sa0 + step + 32 * w);
#pragma unroll
                        for (int t = 0; t < C::kBTiles; ++t)
                            tmem_copy_scales_pair(sfb + 4 * (C::kBTiles * w + t), sb0 + step + t * (C::kSfaBytes / 16) + 32 * w);
                    }
                    const int left = a.K - kb * kStageK;
#pragma unroll
                    for (int k = 0; k < kStageK / 64; ++k)
                        if (64 * k < left) {
                            const int w = NV ? k : k / 2;
                            mma_fp4<NV, true>(tmem + buf * PN, ad0 + step + 2 * k, bd0 + step + 2 * k,
                                              idesc_fp4(2 * kRows, PN, NV, NV ? 0 : k & 1), sfa + 4 * w,
                                              sfb_tile + 4 * C::kBTiles * w, kb > 0 || k > 0 ? 1u : 0u);
                        }
                    mma_commit_pair(empty(s), 0x3);
                    if (last) mma_commit_pair(accf(buf), 0x3);
                }
                __syncwarp();
                parity ^= 1;
                if (++s == kStages) s = 0, ph ^= 1;
                if (++kb == num_kb) kb = 0, ++gc, tile += npairs;
            }
            if (elect_one()) {
                mma_commit_pair(done, 0x1);
                mbar_wait_drain(done, 0, a.timeout_ns, a.status);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        constexpr int kCols = PN / 2;
        const int q = warp & 3, h = (warp - 2) >> 2;
        const int qi = lane & 3;
        pdl_wait();  // the residual may come from the kernel ahead
        int gc = 0;
        for (int tile = pair; tile < total; tile += npairs, ++gc) {
            const int buf = gc & 1;
            int got = 0;
            if (lane == 0) got = mbar_wait(accf(buf), (gc >> 1) & 1, ctl) ? 1 : 0;
            got = __shfl_sync(0xffffffffu, got, 0);
            if (!got) break;
            tc_fence_after_sync();
            const int row0 = tile % a.m_pairs * (2 * kRows) + rank * kRows + q * 32;
            const int m = row0 + lane;
            const int n0 = tile / a.m_pairs * PN + h * kCols;
            const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * PN + h * kCols;
#pragma unroll
            for (int grp = 0; grp < kCols / 32; ++grp) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tbase + 32 * grp, r);
                tmem_wait_ld(r);
                if (grp == kCols / 32 - 1) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(acce(buf), 0));
                }
                const int n1 = n0 + 32 * grp;
                uint32_t P[16];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int n = n1 + 8 * p;
                    uint4 b = make_uint4(0, 0, 0, 0), res = b;
                    if (a.bias != nullptr && n < a.N) b = __ldg(reinterpret_cast<const uint4 *>(a.bias + n));
                    if (a.residual != nullptr && n < a.N && m < a.M)
                        res = *reinterpret_cast<const uint4 *>(a.residual + static_cast<int64_t>(m) * a.N + n);
                    finish8(r + 8 * p, a.alpha, b, res, P + 4 * p);
                }
                ep::quad_transpose(P, qi);
                const int n = n1 + 8 * qi;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int mr = row0 + (lane & ~3) + k;
                    if (mr < a.M && n < a.N)
                        *reinterpret_cast<uint4 *>(a.y + static_cast<int64_t>(mr) * a.N + n) =
                            make_uint4(P[4 * k], P[4 * k + 1], P[4 * k + 2], P[4 * k + 3]);
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // the leader's MMAs and both CTAs' barrier traffic are over
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, C::kTmemCols);
    }
}

// The scales of `rows` rows as a tensor of 128-byte rows, four of them a word tile.
bool scale_map(CUtensorMap *map, const uint8_t *scales, int64_t rows, int64_t words, int box_words) {
    return tensor_map_2d(map, scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (rows + 127) / 128 * words * 4, 128, 128,
                         4 * box_words, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int PN, bool NV>
cudaError_t launch_t(const Fp4Gemm &g, const LaunchCtx &ctx) {
    using C = Cfg<PN, NV>;
    CUtensorMap mx, mw, mxs, mws;
    const int row_bytes = static_cast<int>(g.K / 2);
    const int64_t words = fp4_words(g.K, NV);
    if (!tensor_map_2d(&mx, g.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.M, row_bytes, kStageK / 2, kRows,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tensor_map_2d(&mw, g.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.N, row_bytes, kStageK / 2, PN / 2,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
        !scale_map(&mxs, g.xs, g.M, words, C::kWords) || !scale_map(&mws, g.ws, g.N, words, C::kWords))
        return cudaErrorInvalidValue;
    auto kern = fp4_gemm_pair_kernel<PN, NV>;
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), static_cast<int>(C::kSmemBytes));
        e != cudaSuccess)
        return e;
    const int sms = sm_count();
    if (sms < 2) return cudaErrorInvalidDevice;
    const int64_t m_pairs = (g.M + 2 * kRows - 1) / (2 * kRows);
    const int64_t tiles = m_pairs * ((g.N + PN - 1) / PN);
    if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
    const int pairs = static_cast<int>(tiles < sms / 2 ? tiles : sms / 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 2 : 1;
    Args a = {};
    a.M = static_cast<int>(g.M), a.N = static_cast<int>(g.N), a.K = static_cast<int>(g.K);
    a.words = static_cast<int>(words), a.m_pairs = static_cast<int>(m_pairs);
    a.alpha = g.alpha;
    a.bias = static_cast<const __nv_bfloat16 *>(g.bias), a.residual = static_cast<const __nv_bfloat16 *>(g.residual);
    a.y = static_cast<__nv_bfloat16 *>(g.y);
    a.weights_settled = g.weights_settled;
    a.status = ctx.status, a.timeout_ns = ctx.timeout_ns;
    return cudaLaunchKernelEx(&cfg, kern, mx, mw, mxs, mws, a);
}

}  // namespace

cudaError_t launch_fp4_gemm_pair(const Fp4Gemm &g, const LaunchCtx &ctx) {
    return g.nv ? launch_t<192, true>(g, ctx) : launch_t<192, false>(g, ctx);
}

}  // namespace ck
