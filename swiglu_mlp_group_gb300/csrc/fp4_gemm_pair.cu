// fp4_gemm_pair.cu -- the 4-bit product for many tokens:
//
//   y[m, n] = bf16( alpha * sum_k X[m, k] W[n, k] + bias[n] + residual[m, n] )
//
// X, W: E2M1 codes times the scales of their blocks (fp4_core.cuh).  CTA pairs
// (tcgen05.mma.cta_group::2): a tile of 256 tokens x 192 rows of W on two SMs, each
// holding its 128 tokens, half of W's rows, and the scales of its tokens and of all of
// W's rows; two f32 accumulators in TMEM, so that a tile's epilogue runs under the next
// one's products (two of 256 columns would leave no room for the scales).
//
// Roles (each CTA, 12 warps): warps 0 and 2 TMA producers of the tokens' and of the
// weight's codes and scales, warp 1 TMEM and, in the leader, the issue of the scales'
// copies to TMEM and of the MMAs (both run in the order of their issue), warps 4..11
// the epilogue.
//
// What bounds it.  The MMAs of a stage (256 columns of K) take 384 clocks, 9.5 PFLOP/s
// in all, with or without the scales' copies between them (timed alone, from shared
// memory).  On zeros, which draw little power, the kernel runs at 7.3 (MX) and 6.9 (NV)
// PFLOP/s at 16384 x 4096 -> 12288, without its stores at 8.3 and 7.7, without its
// epilogue at 9.1 and 8.2: operands come in at some 77 bytes a clock and SM of the 81 and
// 89 that the MMAs would take, and y's bytes go the same way.  On random codes power takes
// another tenth.  What it took: one lane that polls and issues, of a warp of its own (32
// lanes polling a barrier cost the issuer a third of its time), a producer for each
// operand (one for both took longer to issue than the MMAs to run), y through shared
// memory and TMA (exchanged between lanes and stored by them: 252 us against 240, NV).
// Tried and slower: tiles of 512 tokens on both accumulators (22 % less operand traffic,
// but no accumulator to spare: 252 us against 240), the stages unrolled in the issuer
// (no gain), tiles in bands of 8 and 16 rows of tiles (no gain), y in pieces of 64
// columns (250).
#include <cuda_bf16.h>

#include "fp4_core.cuh"
#include "launch_util.h"
#include "quant_core.cuh"

namespace ck {
namespace {

constexpr int kThreads = 384;
constexpr int kRows = 128;     // tokens of an accumulator
constexpr int kStageK = 256;   // 128 bytes of codes a row
constexpr int kPN = 192;       // rows of W a tile

// GLU: a tile is 192 rows of gate and the 192 rows of up that go with them.
template <bool NV, bool GLU>
struct Cfg {
    static constexpr int kWords = kStageK / fp4_word(NV);  // scale words of a stage
    static constexpr int kSfaBytes = kWords * 512;
    static constexpr int kBTiles = 2;                      // 128-row tiles of W's scales
    static constexpr int kABytes = kRows * kStageK / 2;
    static constexpr int kBBytes = kPN / 2 * kStageK / 2;
    static constexpr int kParts = GLU ? 2 : 1;             // accumulators of a tile
    static constexpr int kXBytes = kABytes + kSfaBytes, kWBytes = kParts * (kBBytes + kBTiles * kSfaBytes);
    static constexpr int kStageBytes = kXBytes + kWBytes;
    static constexpr int kBarBytes = 256;
    static constexpr int kOutBytes = GLU ? 0 : 8 * 2048;   // a 32 x 32 piece of y a warp of the epilogue
    static constexpr int kStages = (227 * 1024 - kBarBytes - kOutBytes - 1024) / kStageBytes;
    static constexpr int kTmemSf = 2 * kPN;                // the scales' first column
    static constexpr int kSfCols = 4 * kWords * (1 + kParts * kBTiles);
    static constexpr int kTmemCols = 512;
    static constexpr int kSets = kTmemSf + 2 * kSfCols <= kTmemCols ? 2 : 1;  // of scales, taken in turn
    static constexpr size_t kSmemBytes = static_cast<size_t>(kStages) * kStageBytes + kOutBytes + kBarBytes + 1024;
    static_assert(kStageBytes % 1024 == 0 && kTmemSf + kSets * kSfCols <= kTmemCols, "layout");
    static_assert(8 * (2 * kStages + 5) + 8 <= kBarBytes && kSmemBytes <= 227 * 1024, "shared memory");
};

struct Args {
    int M, N, K, m_tiles;  // N: rows of W (GLU: of gate, and of up)
    float alpha;
    const __nv_bfloat16 *bias, *residual;
    uint8_t *codes, *scales;  // GLU: out
    fp4::Scale t;
    bool weights_settled;
    unsigned int *status;
    unsigned long long timeout_ns;
};

// Eight columns of a row, packed to bf16: alpha * acc + bias + residual.
__device__ __forceinline__ uint4 finish8(const uint32_t *acc, uint64_t alpha, const __nv_bfloat16 *bias,
                                         const __nv_bfloat16 *residual) {
    uint64_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = mul_f32x2(f32x2(__uint_as_float(acc[2 * e]), __uint_as_float(acc[2 * e + 1])), alpha);
    auto add = [&](const uint4 &u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = add_f32x2(v[e], f32x2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)));
    };
    if (bias != nullptr) add(__ldg(reinterpret_cast<const uint4 *>(bias)));
    if (residual != nullptr) add(*reinterpret_cast<const uint4 *>(residual));
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        f32x2_split(v[e], lo, hi);
        const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
        p[e] = *reinterpret_cast<const uint32_t *>(&t);
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
}

template <bool NV, bool GLU>
__global__ void __launch_bounds__(kThreads, 1)
fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws,
                     const __grid_constant__ CUtensorMap tm_y,
                     const __grid_constant__ Args a) {
    using C = Cfg<NV, GLU>;
    constexpr int kStages = C::kStages;
    constexpr int kOffB = C::kABytes, kOffSfa = kOffB + C::kParts * C::kBBytes, kOffSfb = kOffSfa + C::kSfaBytes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t smem_s = (raw_s + 1023u) & ~1023u;
    const uint32_t out_s = smem_s + kStages * C::kStageBytes;
    const uint32_t bars_s = out_s + C::kOutBytes;
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
    const int total = a.m_tiles * ((a.N + kPN - 1) / kPN);
    const int num_kb = (a.K + kStageK - 1) / kStageK;
    const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 2);  // the leader's two producers
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

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ producers
        // Both CTAs' copies complete on the leader's barrier of the stage, where
        // the leader's producers announce the pair's bytes.
        const bool weight = warp == 2;
        int issued = 0;
        if (elect_one()) {
            const CUtensorMap *codes = weight ? &tm_w : &tm_x, *scales = weight ? &tm_ws : &tm_xs;
            tma_prefetch_desc(codes);
            tma_prefetch_desc(scales);
            if (!weight || !a.weights_settled) pdl_wait();
            const uint32_t to_codes = stage(0) + (weight ? kOffB : 0), to_scales = stage(0) + (weight ? kOffSfb : kOffSfa);
            const uint32_t bytes = 2 * (weight ? C::kWBytes : C::kXBytes);
            const uint32_t lead = mapa_shared(full(0), 0);
            int s = 0;
            uint32_t ph = 1;
            for (int tile = pair; tile < total; tile += npairs) {
                const int n0 = tile / a.m_tiles * kPN, m0 = tile % a.m_tiles * (2 * kRows) + rank * kRows;
                const int row = weight ? n0 + rank * (kPN / 2) : m0, sf_tile = (weight ? n0 : m0) >> 7;
                bool ok = true;
                for (int kb = 0; kb < num_kb; ++kb) {
                    ok = mbar_wait_spin(empty(s), ph, ctl);  // (the first round's wait is over at once)
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(full(s), bytes);
                    const uint32_t dst = to_codes + s * C::kStageBytes, sf_dst = to_scales + s * C::kStageBytes;
                    tma_load_2d_pair(dst, codes, lead + 8 * s, kb * (kStageK / 2), row);
                    tma_load_2d_pair(sf_dst, scales, lead + 8 * s, kb * (C::kWords * 64), sf_tile);
                    if (GLU && weight) {
                        tma_load_2d_pair(dst + C::kBBytes, codes, lead + 8 * s, kb * (kStageK / 2), a.N + row);
                        tma_load_2d_pair(sf_dst + C::kBTiles * C::kSfaBytes, scales, lead + 8 * s, kb * (C::kWords * 64),
                                         (a.N + n0) >> 7);
                    }
                    ++issued;
                    if (++s == kStages) s = 0, ph ^= 1;
                }
                if (!ok) break;
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
            const int tail = (a.K - (num_kb - 1) * kStageK + 63) / 64;  // MMAs of a tile's last k-block
            if (elect_one()) {
            int gc = 0, s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += npairs, ++gc) {
                // where W's rows of this tile begin in their scales' 128-row tile
                const int n0 = tile / a.m_tiles * kPN;
                const uint32_t sfb_off[2] = {static_cast<uint32_t>((n0 & 127) >> 5), static_cast<uint32_t>(((a.N + n0) & 127) >> 5)};
                for (int kb = 0; kb < num_kb; ++kb) {
                    ok = mbar_wait_spin(full(s), ph, ctl);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t step = static_cast<uint64_t>(s) * (C::kStageBytes / 16);
                    const uint64_t ad = ad0 + step, bd = bd0 + step, sa = sa0 + step, sb = sb0 + step;
                    const uint32_t sfa = tmem + C::kTmemSf + s % C::kSets * C::kSfCols, sfb = sfa + 4 * C::kWords;
                    constexpr int kPartCols = 4 * C::kWords * C::kBTiles;
                    const bool last = kb + 1 == num_kb;
                    const int n = last ? tail : 4;
#pragma unroll
                    for (int w = 0; w < C::kWords; ++w) {
                        tmem_copy_scales_pair(sfa + 4 * w, sa + 32 * w);
#pragma unroll
                        for (int p = 0; p < C::kParts; ++p)
#pragma unroll
                            for (int t = 0; t < C::kBTiles; ++t)
                                tmem_copy_scales_pair(sfb + p * kPartCols + 4 * (C::kBTiles * w + t),
                                                      sb + (p * C::kBTiles + t) * (C::kSfaBytes / 16) + 32 * w);
                    }
#pragma unroll
                    for (int p = 0; p < C::kParts; ++p) {
                        const int acc = GLU ? p : gc & 1, use = GLU ? gc : gc >> 1;
                        // the epilogue has read what this accumulator held before
                        if (kb == 0 && use > 0) {
                            ok = mbar_wait_spin(acce(acc), (use - 1) & 1, ctl);
                            if (!ok) break;
                            tc_fence_after_sync();
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < n) {
                                const int w = NV ? k : k / 2;
                                mma_fp4<NV, true>(tmem + acc * kPN, ad + 2 * k, bd + p * (C::kBBytes / 16) + 2 * k,
                                                  idesc_fp4(2 * kRows, kPN, NV, NV ? 0 : k & 1), sfa + 4 * w,
                                                  sfb + p * kPartCols + sfb_off[p] + 4 * C::kBTiles * w,
                                                  kb > 0 || k > 0 ? 1u : 0u);
                            }
                        if (p == C::kParts - 1) mma_commit_pair(empty(s), 0x3);
                        if (last) mma_commit_pair(accf(acc), 0x3);
                    }
                    if (!ok) break;
                    if (++s == kStages) s = 0, ph ^= 1;
                }
            }
                mma_commit_pair(done, 0x1);
                mbar_wait_drain(done, 0, a.timeout_ns, a.status);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        constexpr int kCols = kPN / 2, kGroups = kCols / 32;
        const int q = warp & 3, c0 = (warp - 4) / 4 * kCols;
        const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + c0;
        pdl_wait();  // the residual may come from the kernel ahead
        // This thread's row of an accumulator into registers; the accumulator is free.
        auto read = [&](int acc, int use, uint32_t (&r)[kGroups][32]) {
            int got = 0;
            if (lane == 0) got = mbar_wait(accf(acc), use & 1, ctl) ? 1 : 0;
            if (!__shfl_sync(0xffffffffu, got, 0)) return false;
            tc_fence_after_sync();
#pragma unroll
            for (int g = 0; g < kGroups; ++g) tmem_ld_32x32b_x32(tbase + acc * kPN + 32 * g, r[g]);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) tmem_wait_ld(r[g]);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(acce(acc), 0));
            return true;
        };
        const uint64_t alpha = f32x2(a.alpha, a.alpha);
        if constexpr (GLU) {
            // gate and up, as bf16 as a linear of its own would leave them, and from
            // them silu(gate) * up in f32, quantized: a thread has 96 columns of a row,
            // whole blocks.  Both accumulators go back before that.
            constexpr int kBlock = fp4_block(NV);
            const int words = static_cast<int>(fp4_words(a.N, NV));
            int gc = 0;
            for (int tile = pair; tile < total; tile += npairs, ++gc) {
                const int n0 = tile / a.m_tiles * kPN + c0;
                const int m = tile % a.m_tiles * (2 * kRows) + rank * kRows + q * 32 + lane;
                uint32_t r[kGroups][32];
                uint4 gate[4 * kGroups], up[4 * kGroups];
                auto take = [&](int part, uint4 (&v)[4 * kGroups]) {
                    if (!read(part, gc, r)) return false;
                    const __nv_bfloat16 *bias = a.bias != nullptr ? a.bias + part * a.N + n0 : nullptr;
#pragma unroll
                    for (int p = 0; p < 4 * kGroups; ++p)
                        v[p] = finish8(r[p / 4] + 8 * (p % 4), alpha, bias != nullptr && n0 + 8 * p < a.N ? bias + 8 * p : nullptr,
                                       nullptr);
                    return true;
                };
                if (!take(0, gate) || !take(1, up)) break;
                if (m < a.M) {
                    uint8_t *code = a.codes + static_cast<int64_t>(m) * (a.N / 2) + n0 / 2;
#pragma unroll
                    for (int b = 0; b < kCols / kBlock; ++b) {
                        const int col = n0 + b * kBlock;
                        uint32_t scale = 0;
                        if (col < a.N) {  // (a.N is a multiple of both blocks)
                            uint64_t n[kBlock / 8][4];
                            float top = 0.f;
#pragma unroll
                            for (int i = 0; i < kBlock / 8; ++i) {
                                const uint4 g = gate[b * (kBlock / 8) + i], u = up[b * (kBlock / 8) + i];
                                const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    n[i][e] = f32x2(-qc::silu_mul(__uint_as_float(gw[e] << 16), __uint_as_float(uw[e] << 16)),
                                                    -qc::silu_mul(__uint_as_float(gw[e] & 0xffff0000u),
                                                                  __uint_as_float(uw[e] & 0xffff0000u)));
                                top = fp4::amax8(n[i], top);
                            }
                            const fp4::Divisor d = fp4::divisor<NV>(top, a.t, scale);
                            uint32_t c[kBlock / 8];
#pragma unroll
                            for (int i = 0; i < kBlock / 8; ++i) c[i] = fp4::codes8<NV>(n[i], d);
                            if constexpr (NV)
                                *reinterpret_cast<uint2 *>(code + b * 8) = make_uint2(c[0], c[1]);
                            else
                                *reinterpret_cast<uint4 *>(code + b * 16) = make_uint4(c[0], c[1], c[2], c[3]);
                        }
                        const int block = col / kBlock;
                        if (block < 4 * words)
                            a.scales[fp4::scale_word_at(m, block / 4, words) + (block & 3)] = static_cast<uint8_t>(scale);
                    }
                    // the last word's blocks past the last tile
                    if (n0 + kCols >= (a.N + kPN - 1) / kPN * kPN)
                        for (int block = (n0 + kCols) / kBlock; block < 4 * words; ++block)
                            a.scales[fp4::scale_word_at(m, block / 4, words) + (block & 3)] = 0;
                }
                __syncwarp();
            }
        } else {
            // 32 rows x 32 columns at a time through shared memory (64-byte rows, swizzled as
            // the map has it) and out by TMA.
            const uint32_t piece = out_s + (warp - 4) * 2048;
            const uint32_t mine = piece + lane * 64, turn = (lane >> 1) & 3;
            int gc = 0;
            for (int tile = pair; tile < total; tile += npairs, ++gc) {
                const int n0 = tile / a.m_tiles * kPN + c0;
                const int row0 = tile % a.m_tiles * (2 * kRows) + rank * kRows + q * 32;
                const bool in = row0 + lane < a.M;
                uint32_t r[kGroups][32];
                if (!read(gc & 1, gc >> 1, r)) break;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int n1 = n0 + 32 * g;
                    if (n1 >= a.N || row0 >= a.M) break;
                    if (lane == 0) bulk_wait_read();  // the piece before has left
                    __syncwarp();
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int n = n1 + 8 * p;
                        const uint4 v = finish8(r[g] + 8 * p, alpha, a.bias != nullptr && n < a.N ? a.bias + n : nullptr,
                                                a.residual != nullptr && n < a.N && in
                                                    ? a.residual + static_cast<int64_t>(row0 + lane) * a.N + n : nullptr);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((p ^ turn) << 4)), "r"(v.x),
                                     "r"(v.y), "r"(v.z), "r"(v.w)
                                     : "memory");
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tm_y, piece, n1, row0);
                        bulk_commit();
                    }
                }
            }
            if (lane == 0) bulk_wait();
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

template <bool NV, bool GLU>
cudaError_t launch_t(const Fp4Gemm &g, const LaunchCtx &ctx) {
    using C = Cfg<NV, GLU>;
    CUtensorMap mx, mw, mxs, mws, my;
    const int row_bytes = static_cast<int>(g.K / 2);
    const int64_t words = fp4_words(g.K, NV), w_rows = GLU ? 2 * g.N : g.N;
    if (!tensor_map_2d(&mx, g.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.M, row_bytes, kStageK / 2, kRows,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tensor_map_2d(&mw, g.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w_rows, row_bytes, kStageK / 2, kPN / 2,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tensor_map_scales(&mxs, g.xs, (g.M + 127) / 128, words, C::kWords, 1) ||
        !tensor_map_scales(&mws, g.ws, (w_rows + 127) / 128, words, C::kWords, C::kBTiles))
        return cudaErrorInvalidValue;
    if constexpr (GLU)
        my = mx;  // not used
    else if (!tensor_map_2d(&my, g.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.M, g.N, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    auto kern = fp4_gemm_pair_kernel<NV, GLU>;
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), static_cast<int>(C::kSmemBytes));
        e != cudaSuccess)
        return e;
    const int sms = sm_count();
    if (sms < 2) return cudaErrorInvalidDevice;
    const int64_t m_tiles = (g.M + 2 * kRows - 1) / (2 * kRows);
    const int64_t tiles = m_tiles * ((g.N + kPN - 1) / kPN);
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
    a.m_tiles = static_cast<int>(m_tiles);
    a.alpha = g.alpha;
    a.bias = static_cast<const __nv_bfloat16 *>(g.bias), a.residual = static_cast<const __nv_bfloat16 *>(g.residual);
    a.codes = g.a_codes, a.scales = g.a_scales, a.t = fp4::scale_of(g.a_scale);
    a.weights_settled = g.weights_settled;
    a.status = ctx.status, a.timeout_ns = ctx.timeout_ns;
    return cudaLaunchKernelEx(&cfg, kern, mx, mw, mxs, mws, my, a);
}

}  // namespace

cudaError_t launch_fp4_gemm_pair(const Fp4Gemm &g, const LaunchCtx &ctx) {
    return g.nv ? launch_t<true, false>(g, ctx) : launch_t<false, false>(g, ctx);
}

cudaError_t launch_fp4_gemm_glu(const Fp4Gemm &g, const LaunchCtx &ctx) {
    return g.nv ? launch_t<true, true>(g, ctx) : launch_t<false, true>(g, ctx);
}

}  // namespace ck
