// fp4_gemm_pair.cu -- the 4-bit product for many tokens:
//
//   y[m, n] = bf16( alpha * sum_k X[m, k] W[n, k] + bias[n] + residual[m, n] )
//
// X, W: E2M1 codes times the scales of their blocks (fp4_core.cuh).  CTA pairs
// (tcgen05.mma.cta_group::2): a tile of 256 tokens x one or two parts of 192 rows of W
// on two SMs, each holding its 128 tokens, half of W's rows, and the scales of its
// tokens and of all of W's rows; an f32 accumulator in TMEM for each part, two of them
// in all (of 256 columns they would leave no room for the scales).
//
// One part a tile: the accumulators in turn, so that a tile's epilogue runs under the
// next one's products.  Two: X's bytes once for both, and the epilogue first reads both
// accumulators into registers and hands them back before it does anything else; a
// tile's first and last two k-blocks go to the first part together, then to the second,
// so that the tensor cores have 768 clocks of work while an accumulator is read.
//
// SPLIT: few tiles and long K, so a tile has a cluster of up to four pairs, each with its
// share of K; the pairs' sums meet through distributed shared memory.
//
// GLU: the parts are rows of gate and the rows of up that go with them, and the
// epilogue makes silu(gate) * up of them and quantizes it: what the next linear of a
// SwiGLU MLP reads, without gate and up ever leaving the chip.
//
// Roles (each CTA, 12 warps): warps 0 and 2 TMA producers of the tokens' and of the
// weight's codes and scales, warp 1 TMEM and, in the leader, the issue of the scales'
// copies to TMEM and of the MMAs (both run in the order of their issue), warps 4..11
// the epilogue.
#include <cuda_bf16.h>

#include <type_traits>

#include "fp4_core.cuh"
#include "launch_util.h"
#include "quant_core.cuh"

namespace ck {
namespace {

constexpr int kThreads = 384;
// Registers of a thread of warps 0..3 and of the epilogue's; together what the block is
// launched with (168 a thread).
constexpr int kOtherRegs = 56, kEpilogueRegs = 224;
static_assert(128 * kOtherRegs + 256 * kEpilogueRegs <= kThreads * 168, "registers");
constexpr int kRows = 128;     // tokens of an accumulator
constexpr int kStageK = 256;   // 128 bytes of codes a row
constexpr int kPN = 192;       // rows of W a part

template <bool NV, int PARTS, bool GLU, bool SPLIT = false>
struct Cfg {
    static constexpr int kWords = kStageK / fp4_word(NV);  // scale words of a stage
    static constexpr int kSfaBytes = kWords * 512;
    static constexpr int kBTiles = 2;                      // 128-row tiles of a part's scales
    static constexpr int kABytes = kRows * kStageK / 2;
    static constexpr int kBBytes = kPN / 2 * kStageK / 2;
    static constexpr int kXBytes = kABytes + kSfaBytes, kWBytes = PARTS * (kBBytes + kBTiles * kSfaBytes);
    static constexpr int kStageBytes = kXBytes + kWBytes;
    // a 32 x 32 piece of y a warp of the epilogue; SPLIT: the other pairs' sums, a CTA's rows
    // of at most three quarters of the columns
    static constexpr int kOutBytes = SPLIT ? kRows * kPN * 3 : (GLU ? 0 : 8 * 2048);
    static constexpr int kBarBytes = 256;
    static constexpr int kStages = (227 * 1024 - kBarBytes - kOutBytes - 1024) / kStageBytes;
    static constexpr int kTmemSf = 2 * kPN;                // the scales' first column
    static constexpr int kSfCols = 4 * kWords * (1 + kBTiles);
    static constexpr int kTmemCols = 512;
    static constexpr size_t kSmemBytes = static_cast<size_t>(kStages) * kStageBytes + kOutBytes + kBarBytes + 1024;
    static_assert(kStageBytes % 1024 == 0 && kTmemSf + 2 * kSfCols <= kTmemCols, "layout");
    static_assert(8 * (2 * kStages + 5) + 8 <= kBarBytes && kSmemBytes <= 227 * 1024, "shared memory");
};

struct Args {
    int M, N, K, m_tiles, n_tiles;  // N: rows of W (GLU: of gate, and of up)
    int splits;                     // SPLIT: pairs of a tile
    __nv_bfloat16 *y;               // SPLIT
    float alpha;
    const __nv_bfloat16 *bias, *residual;
    uint8_t *codes, *scales;  // GLU: out
    fp4::Scale t;
    bool weights_settled;
    unsigned int *status;
    unsigned long long timeout_ns;
};

// Eight columns of a row, packed to bf16: alpha * acc (+ bias) (+ residual).
template <bool BIAS, bool RESIDUAL>
__device__ __forceinline__ uint4 finish8(const uint32_t *acc, uint64_t alpha, const uint4 &bias, const uint4 &residual) {
    const uint32_t b[4] = {bias.x, bias.y, bias.z, bias.w}, r[4] = {residual.x, residual.y, residual.z, residual.w};
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint64_t v = mul_f32x2(f32x2(__uint_as_float(acc[2 * e]), __uint_as_float(acc[2 * e + 1])), alpha);
        if constexpr (BIAS) v = add_f32x2(v, fp4::unpack2(b[e]));
        if constexpr (RESIDUAL) v = add_f32x2(v, fp4::unpack2(r[e]));
        float lo, hi;
        f32x2_split(v, lo, hi);
        const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
        p[e] = *reinterpret_cast<const uint32_t *>(&t);
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, const uint4 &v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster_v4(uint32_t at, const uint4 &v) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// silu(gate) * up of whole blocks of a row, quantized: codes from `code` on (a
// thread's 96 columns from `col` on), scale bytes to row m of `scales`.
template <bool NV, int COLS>
__device__ __forceinline__ void quantize_glu(const uint4 (&gate)[COLS / 8], const uint4 (&up)[COLS / 8], int col, int N,
                                             const fp4::Scale &t, uint8_t *code, uint8_t *scales, int64_t m, int words) {
    constexpr int kBlock = fp4_block(NV);
#pragma unroll
    for (int b = 0; b < COLS / kBlock; ++b) {
        uint32_t scale = 0;
        if (col + b * kBlock < N) {  // (N is a multiple of both blocks)
            uint64_t n[kBlock / 8][4];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < kBlock / 8; ++i) {
                const uint4 g = gate[b * (kBlock / 8) + i], u = up[b * (kBlock / 8) + i];
                const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    n[i][e] = f32x2(-qc::silu_mul(__uint_as_float(gw[e] << 16), __uint_as_float(uw[e] << 16)),
                                    -qc::silu_mul(__uint_as_float(gw[e] & 0xffff0000u), __uint_as_float(uw[e] & 0xffff0000u)));
                top = fp4::amax8(n[i], top);
            }
            const fp4::Divisor d = fp4::divisor<NV>(top, t, scale);
            uint32_t c[kBlock / 8];
#pragma unroll
            for (int i = 0; i < kBlock / 8; ++i) c[i] = fp4::codes8<NV>(n[i], d);
            if constexpr (NV)
                *reinterpret_cast<uint2 *>(code + b * 8) = make_uint2(c[0], c[1]);
            else
                *reinterpret_cast<uint4 *>(code + b * 16) = make_uint4(c[0], c[1], c[2], c[3]);
        }
        const int block = col / kBlock + b;
        if (block < 4 * words)
            scales[fp4::scale_word_at(m, block / 4, words) + (block & 3)] = static_cast<uint8_t>(scale);
    }
}

// What bounds it.  The MMAs of a part's stage (256 columns of K) take 384 clocks, 9.5
// PFLOP/s in all, with or without the scales' copies between them (timed alone, from
// shared memory; of the instruction's K = 64 form, the one used: sm_103a has a K = 96 form,
// too, by the chip's published rate half as fast again, which is not measured here).  Their
// operands: 81 (MX) and 89 (NV) bytes a clock and SM with one part, of which some 70 come
// in, 59 and 65 with two, which then wait for the issue (28 instructions a k-block, NV, at
// some 30 clocks each, MX 18) and between tiles.
// Random codes draw so much power that the clock gives another 5 %.  16384 x 4096 ->
// 12288: 223 us (NV) and 217 (MX), on zeros 213 and 208 (7.7 and 7.9 PFLOP/s), with a
// residual 272 and 264; gate and up of as many tokens with 6144 rows each, where no y is
// stored, 209 and 200, on zeros 196 and 188 (8.4 and 8.8).
//
// What it took: one lane that polls and issues, of a warp of its own (32 lanes polling a
// barrier, or walking together and issuing by predicate, 259 us against 205), a producer
// for each operand (one for both took longer to issue than the MMAs to run), y through
// shared memory and TMA (exchanged between lanes and stored by them 252 us against 240,
// from shared memory by coalesced stores 212 against 208), no branches between the
// columns of an accumulator's reading (1450 clocks for 96 columns with them, 650
// without), the residual read in whole sectors, four lanes a row, and turned to rows in
// shared memory (a lane its own row: 300 us against 265), with two parts more registers
// for the epilogue than for the rest (222 us against 218; one part does not need them:
// 247 against 242), the k-blocks' order at a tile's ends (gate and up 206 us without, MX;
// for every k-block NV 205 against 196), in a loop that is not unrolled (278).  With two
// parts and a y the epilogue spills 48 bytes a thread (132 loaded), with gate and up NV 8
// (20); with one part, and with gate and up MX, nothing.
//
// Few tokens (33 to 256): a tile has 256 rows, most of them zeros, and there are as many
// tiles as for 256 tokens: 64 x 4096 -> 12288 10.2 us NV and 9.7 MX, 256 10.9 and 10.4,
// where the weight's bytes take 4.2 of HBM.  64 tiles for 76 pairs, a tile each, so a
// call is one tile's chain: beginning, 16 k-blocks, epilogue.  1000 x 2080 -> 1544 8.0 and
// 7.6: 36 tiles of nine k-blocks, too short a K to split.
// Tried and slower, one part: 512 tokens x 192 rows (252 us against 240), the issuer's
// stages unrolled, tiles in bands of 8 and 16 rows of tiles, y in pieces of 64 columns
// (250), the next tile's first k-blocks prefetched to L2 (264 against 249); two parts, the
// last round's tiles part by part where that is one round less (61 us against 59 of one
// part for 4096 x 12288 -> 4096).
template <bool NV, int PARTS, bool GLU, bool SPLIT = false>
__global__ void __launch_bounds__(kThreads, 1)
fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws,
                     const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ Args a) {
    static_assert(PARTS == 2 ? !SPLIT : !GLU, "gate and up in two parts, K split for one");
    using C = Cfg<NV, PARTS, GLU, SPLIT>;
    constexpr int kStages = C::kStages;
    constexpr int kOffB = C::kABytes, kOffSfa = kOffB + PARTS * C::kBBytes, kOffSfb = kOffSfa + C::kSfaBytes;
    constexpr int kTileN = GLU ? kPN : PARTS * kPN;  // columns of y, or of the product, a tile
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
    const int crank = static_cast<int>(cluster_ctarank()), rank = SPLIT ? crank & 1 : crank;  // 0: leader (issues), 1: peer
    const int lead_rank = SPLIT ? crank & ~1 : 0;
    const uint16_t both = static_cast<uint16_t>(0x3 << lead_rank);
    // SPLIT: a cluster a tile, the pairs of which have a share of K each
    const int share = crank >> 1;
    const int pair = SPLIT ? blockIdx.x / (2 * a.splits) : blockIdx.x >> 1, npairs = SPLIT ? 1 << 30 : gridDim.x >> 1;
    const int total = a.m_tiles * a.n_tiles;
    const int num_kb = (a.K + kStageK - 1) / kStageK;
    const int kb0 = SPLIT ? num_kb * share / a.splits : 0, kb1 = SPLIT ? num_kb * (share + 1) / a.splits : num_kb;
    const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};
    // first row of W of a tile's part (GLU: up's rows follow gate's N)
    auto part_row = [&](int tile, int p) { return tile / a.m_tiles * kTileN + p * (GLU ? a.N : kPN); };

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

    if (warp < 4) {
        if constexpr (PARTS == 2) setmaxnreg_dec<kOtherRegs>();  // by all four warps at once
        if (warp == 0 || warp == 2) {
            // -------------------------------------------------------- producers
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
                const uint32_t lead = mapa_shared(full(0), lead_rank);
                int s = 0;
                uint32_t ph = 1;
                for (int tile = pair; tile < total; tile += npairs) {
                    const int m0 = tile % a.m_tiles * (2 * kRows) + rank * kRows;
                    const int w0 = part_row(tile, 0), w1 = part_row(tile, PARTS - 1);
                    const int row = weight ? w0 + rank * (kPN / 2) : m0, sf_tile = (weight ? w0 : m0) >> 7;
                    bool ok = true;
                    for (int kb = kb0; kb < kb1; ++kb) {
                        ok = mbar_wait_spin(empty(s), ph, ctl);  // (the first round's wait is over at once)
                        if (!ok) break;
                        if (rank == 0) mbar_arrive_expect_tx(full(s), bytes);
                        const uint32_t dst = to_codes + s * C::kStageBytes, sf_dst = to_scales + s * C::kStageBytes;
                        const int x = kb * (kStageK / 2), sf_x = kb * (C::kWords * 64);
                        tma_load_2d_pair(dst, codes, lead + 8 * s, x, row);
                        tma_load_2d_pair(sf_dst, scales, lead + 8 * s, sf_x, sf_tile);
                        if (PARTS == 2 && weight) {
                            tma_load_2d_pair(dst + C::kBBytes, codes, lead + 8 * s, x, w1 + rank * (kPN / 2));
                            tma_load_2d_pair(sf_dst + C::kBTiles * C::kSfaBytes, scales, lead + 8 * s, sf_x, w1 >> 7);
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
            // (rank == 0 in this branch's own condition made the issuer a tenth slower)
            if (rank == 0) {
                // -------------------------------------------------------- MMA issue
                const uint64_t ad0 = sdesc_kmajor_sw128(stage(0)), bd0 = sdesc_kmajor_sw128(stage(0) + kOffB);
                const uint64_t sa0 = sdesc_scales(stage(0) + kOffSfa), sb0 = sdesc_scales(stage(0) + kOffSfb);
                const int tail = (a.K - (num_kb - 1) * kStageK + 63) / 64;  // MMAs of a tile's last k-block
                if (elect_one()) {
                    int gc = 0, s = 0;
                    uint32_t ph = 0;
                    bool ok = true;
                    // Stage st's share of a part: its scales' copies to set `set`, its MMAs.
                    auto unit = [&](int st, int set, int acc, int p, uint32_t sfb_off, int n, bool first) {
                        const uint64_t step = static_cast<uint64_t>(st) * (C::kStageBytes / 16);
                        const uint64_t ad = ad0 + step, bd = bd0 + step + p * (C::kBBytes / 16);
                        const uint64_t sa = sa0 + step, sb = sb0 + step + p * (C::kBTiles * C::kSfaBytes / 16);
                        const uint32_t sfa = tmem + C::kTmemSf + set * C::kSfCols, sfb = sfa + 4 * C::kWords;
#pragma unroll
                        for (int w = 0; w < C::kWords; ++w) {
                            if (p == 0) tmem_copy_scales_pair(sfa + 4 * w, sa + 32 * w);
#pragma unroll
                            for (int t = 0; t < C::kBTiles; ++t)
                                tmem_copy_scales_pair(sfb + 4 * (C::kBTiles * w + t), sb + t * (C::kSfaBytes / 16) + 32 * w);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < n) {
                                const int w = NV ? k : k / 2;
                                mma_fp4<NV, true>(tmem + acc * kPN, ad + 2 * k, bd + 2 * k,
                                                  idesc_fp4(2 * kRows, kPN, NV, NV ? 0 : k & 1), sfa + 4 * w,
                                                  sfb + sfb_off + 4 * C::kBTiles * w, !first || k > 0 ? 1u : 0u);
                            }
                    };
                    for (int tile = pair; tile < total && ok; tile += npairs, ++gc) {
                        // where a part's rows begin in their scales' 128-row tile
                        const uint32_t sfb_off[2] = {static_cast<uint32_t>(part_row(tile, 0) & 127) >> 5,
                                                     static_cast<uint32_t>(part_row(tile, 1) & 127) >> 5};
                        for (int kb = kb0; kb < kb1;) {
                            const int group = PARTS == 2 && (kb == 0 || kb + 2 == num_kb) && kb + 1 < num_kb ? 2 : 1;
                            int st = s;
                            uint32_t sph = ph;
#pragma unroll
                            for (int p = 0; p < PARTS; ++p) {
                                const int acc = PARTS == 2 ? p : gc & 1, use = PARTS == 2 ? gc : gc >> 1;
                                st = s, sph = ph;
#pragma unroll 1
                                for (int j = 0; j < group; ++j) {
                                    if (p == 0) {
                                        ok = mbar_wait_spin(full(st), sph, ctl);
                                        if (!ok) break;
                                    }
                                    // the epilogue has read what this accumulator held before
                                    if (kb + j == kb0 && use > 0) {
                                        ok = mbar_wait_spin(acce(acc), (use - 1) & 1, ctl);
                                        if (!ok) break;
                                    }
                                    tc_fence_after_sync();
                                    const bool last = kb + j + 1 == kb1;
                                    unit(st, PARTS == 2 ? j : st & 1, acc, p, sfb_off[p], kb + j + 1 == num_kb ? tail : 4, kb + j == kb0);
                                    if (p == PARTS - 1) mma_commit_pair(empty(st), both);
                                    if (last) mma_commit_pair(accf(acc), both);
                                    if (++st == kStages) st = 0, sph ^= 1;
                                }
                                if (!ok) break;
                            }
                            if (!ok) break;
                            kb += group, s = st, ph = sph;
                        }
                    }
                    mma_commit_pair(done, static_cast<uint16_t>(0x1 << lead_rank));
                    mbar_wait_drain(done, 0, a.timeout_ns, a.status);
                }
            }
            __syncwarp();
        }
    } else {
        if constexpr (PARTS == 2) setmaxnreg_inc<kEpilogueRegs>();
        // ------------------------------------------------------------ epilogue
        constexpr int kCols = kPN / 2, kGroups = kCols / 32, kPieces = kCols / 8;
        const int q = warp & 3, c0 = (warp - 4) / 4 * kCols;
        const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + c0;
        const uint64_t alpha = f32x2(a.alpha, a.alpha);
        pdl_wait();  // the residual may come from the kernel ahead
        // This thread's row of an accumulator into registers, in two steps: when both are
        // done the accumulator is free.
        auto begin_read = [&](int acc, int use, uint32_t (&r)[kGroups][32]) {
            int got = 0;
            if (lane == 0) got = mbar_wait(accf(acc), use & 1, ctl) ? 1 : 0;
            if (!__shfl_sync(0xffffffffu, got, 0)) return false;
            tc_fence_after_sync();
#pragma unroll
            for (int g = 0; g < kGroups; ++g) tmem_ld_32x32b_x32(tbase + acc * kPN + 32 * g, r[g]);
            return true;
        };
        auto end_read = [&](int acc, uint32_t (&r)[kGroups][32]) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) tmem_wait_ld(r[g]);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(acce(acc), 0));
        };
        // 32 rows x 32 columns of y at a time through shared memory (64-byte rows,
        // swizzled as the map has it) and out by TMA.
        const uint32_t piece = out_s + (warp - 4) * 2048;
        const uint32_t mine = piece + lane * 64, turn = (lane >> 1) & 3;
        const uint32_t turned = piece + lane / 4 * 64 + (((lane ^ (lane >> 3)) & 3) << 4);  // row lane / 4, its piece lane % 4
        auto store = [&](int row0, int n0, const uint4 (&v)[kPieces]) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                if (n0 + 32 * g >= a.N || row0 >= a.M) break;
                if (lane == 0) bulk_wait_read();  // the piece before has left
                __syncwarp();
#pragma unroll
                for (int p = 0; p < 4; ++p) st_shared_v4(mine + ((p ^ turn) << 4), v[4 * g + p]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&tm_y, piece, n0 + 32 * g, row0);
                    bulk_commit();
                }
            }
        };
        // All of this CTA's tiles.  Pieces past the last column or row read the bias and
        // the residual of the last one there is, and are not stored.
        auto run = [&](auto bias_tag, auto residual_tag) {
            constexpr bool kBias = decltype(bias_tag)::value, kResidual = decltype(residual_tag)::value;
            int gc = 0;
            for (int tile = pair; tile < total; tile += npairs, ++gc) {
                const int row0 = tile % a.m_tiles * (2 * kRows) + rank * kRows + q * 32;
                uint4 v[PARTS][kPieces], res[kResidual ? PARTS : 1][kPieces];
                int n0[PARTS];
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    n0[p] = tile / a.m_tiles * kTileN + (GLU ? 0 : p * kPN) + c0;
                    if constexpr (kResidual) {  // four lanes a row: its turn to rows comes below
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat16 *r = a.residual + static_cast<int64_t>(min(row0 + 8 * i + lane / 4, a.M - 1)) * a.N;
#pragma unroll
                            for (int g = 0; g < kGroups; ++g)
                                res[p][4 * g + i] =
                                    *reinterpret_cast<const uint4 *>(r + min(n0[p] + 32 * g + 8 * (lane % 4), a.N - 8));
                        }
                    }
                }
                auto finish = [&](int p, const uint32_t (&r)[kGroups][32]) {
                    if constexpr (kResidual) {
                        if (lane == 0) bulk_wait_read();
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) {
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i) st_shared_v4(turned + i * 512, res[p][4 * g + i]);
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i) res[p][4 * g + i] = ld_shared_v4(mine + ((i ^ turn) << 4));
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        uint4 b = make_uint4(0, 0, 0, 0);
                        if constexpr (kBias)
                            b = __ldg(reinterpret_cast<const uint4 *>(a.bias + (GLU ? p * a.N : 0) + min(n0[p] + 8 * i, a.N - 8)));
                        v[p][i] = finish8<kBias, kResidual>(r[i / 4] + 8 * (i % 4), alpha, b, res[kResidual ? p : 0][i]);
                    }
                };
                uint32_t r[kGroups][32];
                if (!begin_read(PARTS == 2 ? 0 : gc & 1, PARTS == 2 ? gc : gc >> 1, r)) break;
                end_read(PARTS == 2 ? 0 : gc & 1, r);
                if constexpr (PARTS == 1 || kResidual) finish(0, r);
                if constexpr (PARTS == 2) {
                    // (with a residual there are no registers for both)
                    uint32_t r1[kGroups][32];
                    if (!begin_read(1, gc, r1)) break;
                    if constexpr (!kResidual) finish(0, r);
                    end_read(1, r1);
                    finish(1, r1);
                }
                if constexpr (GLU) {
                    const int words = static_cast<int>(fp4_words(a.N, NV)), m = row0 + lane;
                    if (m < a.M) {
                        quantize_glu<NV, kCols>(v[0], v[PARTS - 1], n0[0], a.N, a.t,
                                                a.codes + static_cast<int64_t>(m) * (a.N / 2) + n0[0] / 2, a.scales, m, words);
                        // the last word's blocks past the last tile
                        if (n0[0] + kCols >= a.n_tiles * kPN)
                            for (int block = a.n_tiles * kPN / fp4_block(NV); block < 4 * words; ++block)
                                a.scales[fp4::scale_word_at(m, block / 4, words) + (block & 3)] = 0;
                    }
                    __syncwarp();
                } else {
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) store(row0, n0[p], v[p]);
                }
            }
        };
        using std::false_type;
        using std::true_type;
        if constexpr (SPLIT) {
            if (lane == 0) mbar_wait(accf(0), 0, ctl);  // (a wait that gives up leaves the abort flag)
            __syncwarp();
            tc_fence_after_sync();
        } else if constexpr (GLU) {
            if (a.bias != nullptr) run(true_type(), false_type());
            else run(false_type(), false_type());
        } else {
            if (a.bias != nullptr && a.residual != nullptr) run(true_type(), true_type());
            else if (a.bias != nullptr) run(true_type(), false_type());
            else if (a.residual != nullptr) run(false_type(), true_type());
            else run(false_type(), false_type());
            if (lane == 0) bulk_wait();
        }
    }
    if constexpr (SPLIT) {
        // Each pair finishes its share of the columns: the other pairs send it their sums of
        // them, which it adds in the order of K.
        const int q = warp & 3, half = (warp - 4) / 4, row = q * 32 + lane, own = kPN / a.splits;
        const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
        // where four columns of this thread's row lie, of those that the from-th other pair sent
        auto at = [&](int from, int c) { return static_cast<uint32_t>(((from * own + c) / 4 * kRows + row) * 16); };
        if (warp >= 4) {
            uint32_t v[3][32];
#pragma unroll
            for (int g = 0; g < 3; ++g) tmem_ld_32x32b_x32(acc + half * 96 + 32 * g, v[g]);
#pragma unroll
            for (int g = 0; g < 3; ++g) tmem_wait_ld(v[g]);
#pragma unroll
            for (int g = 0; g < 6; ++g) {
                const int c = half * 96 + 16 * g, owner = (c >= own) + (c >= 2 * own) + (c >= 3 * own);
                if (owner != share) {
                    const uint32_t to = mapa_shared(out_s, 2 * owner + rank) + at(share < owner ? share : share - 1, c - owner * own);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st_cluster_v4(to + i * kRows * 16, make_uint4(v[g / 2][g % 2 * 16 + 4 * i], v[g / 2][g % 2 * 16 + 4 * i + 1],
                                                                     v[g / 2][g % 2 * 16 + 4 * i + 2], v[g / 2][g % 2 * 16 + 4 * i + 3]));
                }
            }
        }
        __syncwarp();
        cluster_sync();  // the sums are there
        const int m = pair % a.m_tiles * (2 * kRows) + rank * kRows + row;
        if (warp >= 4 && !*abort_flag) {
#pragma unroll 1
            for (int g = half; g < own / 16; g += 2) {
                uint32_t mine[16];
                tmem_ld_32x32b_x16(acc + share * own + 16 * g, mine);
                tmem_wait_ld16(mine);
                float sum[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i] = 0.f;
                for (int src = 0; src < a.splits; ++src)
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const uint4 v = src == share ? make_uint4(mine[i], mine[i + 1], mine[i + 2], mine[i + 3])
                                                     : ld_shared_v4(out_s + at(src < share ? src : src - 1, 16 * g + i));
                        sum[i] += __uint_as_float(v.x), sum[i + 1] += __uint_as_float(v.y);
                        sum[i + 2] += __uint_as_float(v.z), sum[i + 3] += __uint_as_float(v.w);
                    }
#pragma unroll
                for (int i = 0; i < 16; i += 8) {
                    const int n = pair / a.m_tiles * kPN + share * own + 16 * g + i;
                    if (m >= a.M || n >= a.N) continue;
                    const int64_t off = static_cast<int64_t>(m) * a.N + n;
                    uint4 b = make_uint4(0, 0, 0, 0), r = b;
                    if (a.bias != nullptr) b = __ldg(reinterpret_cast<const uint4 *>(a.bias + n));
                    if (a.residual != nullptr) r = *reinterpret_cast<const uint4 *>(a.residual + off);
                    uint32_t bits[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) bits[e] = __float_as_uint(sum[i + e]);
                    *reinterpret_cast<uint4 *>(a.y + off) = finish8<true, true>(bits, f32x2(a.alpha, a.alpha), b, r);
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

// splits: pairs that share a tile's K
template <bool NV, int PARTS, bool GLU, bool SPLIT = false>
cudaError_t launch_t(const Fp4Gemm &g, const LaunchCtx &ctx, int splits = 1) {
    using C = Cfg<NV, PARTS, GLU, SPLIT>;
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
    auto kern = fp4_gemm_pair_kernel<NV, PARTS, GLU, SPLIT>;
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), static_cast<int>(C::kSmemBytes));
        e != cudaSuccess)
        return e;
    const int sms = sm_count();
    if (sms < 2) return cudaErrorInvalidDevice;
    constexpr int kTileN = GLU ? kPN : PARTS * kPN;
    const int64_t m_tiles = (g.M + 2 * kRows - 1) / (2 * kRows), n_tiles = (g.N + kTileN - 1) / kTileN;
    const int64_t tiles = m_tiles * n_tiles;
    if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
    const int pairs = static_cast<int>(tiles < sms / 2 ? tiles : sms / 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(SPLIT ? 2 * splits * tiles : 2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(2 * splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 2 : 1;
    Args a = {};
    a.M = static_cast<int>(g.M), a.N = static_cast<int>(g.N), a.K = static_cast<int>(g.K);
    a.m_tiles = static_cast<int>(m_tiles), a.n_tiles = static_cast<int>(n_tiles);
    a.splits = splits, a.y = static_cast<__nv_bfloat16 *>(g.y);
    a.alpha = g.alpha;
    a.bias = static_cast<const __nv_bfloat16 *>(g.bias), a.residual = static_cast<const __nv_bfloat16 *>(g.residual);
    a.codes = g.a_codes, a.scales = g.a_scales, a.t = fp4::scale_of(g.a_scale);
    a.weights_settled = g.weights_settled;
    a.status = ctx.status, a.timeout_ns = ctx.timeout_ns;
    return cudaLaunchKernelEx(&cfg, kern, mx, mw, mxs, mws, my, a);
}

}  // namespace

// How many pairs share a tile's K: as many as find room at once, with ten k-blocks each
// at least, as the exchange takes some 2 us (linears of 64 tokens 16384 -> 2048 14.3 us
// against 19.6, 12288 -> 4096 17.0 against 18.3, their product alone 11.3 against 13.8;
// 4096 -> 4096, not split, 7.4 against 8.6 with three pairs).
template <bool NV>
int pairs_of_a_tile(const Fp4Gemm &g) {
    using C = Cfg<NV, 1, false, true>;
    const void *kern = reinterpret_cast<const void *>(fp4_gemm_pair_kernel<NV, 1, false, true>);
    const int64_t tiles = (g.M + 2 * kRows - 1) / (2 * kRows) * ((g.N + kPN - 1) / kPN), kbs = (g.K + kStageK - 1) / kStageK;
    if (kbs < 20 || ensure_dynamic_smem(kern, static_cast<int>(C::kSmemBytes)) != cudaSuccess) return 1;
    for (int n = 4; n > 1; --n)
        if (kbs >= 10 * n && tiles <= max_active_clusters(kern, kThreads, C::kSmemBytes, 2 * n)) return n;
    return 1;
}

cudaError_t launch_fp4_gemm_pair(const Fp4Gemm &g, const LaunchCtx &ctx) {
    const int64_t pairs = sm_count() / 2;
    if (pairs < 1) return cudaErrorInvalidDevice;
    // Two parts a tile take 1.75 times one part's time where K is long, and twice it where
    // the stores bound both, so they pay when they take half the rounds of tiles: 213 us
    // against 240 for 16384 x 4096 -> 12288 (27 rounds against 54; NV, zeros), 60.5
    // against 65 for 4096 x 4096 -> 12288 (7, 14), but 34.3 against 33.5 for 8192 x 1024
    // -> 8192 (10, 19), 67 against 60 for 4096 x 12288 -> 4096 (3, 5) and 19.5 against
    // 15.7 for 2048 x 4096 -> 4096 (2, 3).
    const int share = g.nv ? pairs_of_a_tile<true>(g) : pairs_of_a_tile<false>(g);
    if (share > 1)
        return g.nv ? launch_t<true, 1, false, true>(g, ctx, share) : launch_t<false, 1, false, true>(g, ctx, share);
    auto rounds = [&](int n) { return ((g.M + 2 * kRows - 1) / (2 * kRows) * ((g.N + n - 1) / n) + pairs - 1) / pairs; };
    if (2 * rounds(2 * kPN) <= rounds(kPN))
        return g.nv ? launch_t<true, 2, false>(g, ctx) : launch_t<false, 2, false>(g, ctx);
    return g.nv ? launch_t<true, 1, false>(g, ctx) : launch_t<false, 1, false>(g, ctx);
}

cudaError_t launch_fp4_gemm_glu(const Fp4Gemm &g, const LaunchCtx &ctx) {
    return g.nv ? launch_t<true, 2, true>(g, ctx) : launch_t<false, 2, true>(g, ctx);
}

}  // namespace ck
