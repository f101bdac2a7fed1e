// attention.cu -- attention over a shared prefix and each sequence's own keys
// (paged), or over an encoder's states (dense), on tcgen05.
//
//   x_j = scale * q . k_j,   m = max_j x_j,   out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m)
// in one pass over the keys: a running maximum and sum per query row, and an
// accumulator in TMEM that is scaled where the maximum grows.
//
// Rows.  The G query heads of a key head read the same keys, so a tile of 128
// MMA rows holds 128 / G query tokens x G heads.  Against the prefix the tokens
// of all sequences are rows of the same product: each prefix key is read once
// for the whole batch, which is what makes the shared part a matrix product
// instead of B vector ones.
//
// Items.  The work is a list of items -- rows of one key head x a chunk of keys
// -- that a persistent grid walks with a stride.  More than one row tile makes
// a wide item: two row tiles against the same key tiles.  Otherwise an item is
// narrow: one row tile, its key tiles taken alternately by the two halves of
// the pipeline.  Chunks (and the halves of a narrow item) leave partial sums
// with their maximum in the workspace; a second kernel joins them.
//
// Pipeline (one CTA per SM, 11 warps).  Two streams, each with its own S and O
// in TMEM and four softmax warps, so that the tensor core works on one while
// the other is in its softmax:
//   warps 0..3, 4..7 : softmax of stream 0 / 1, a thread per row: S from TMEM,
//                      maximum, exponentials, P back to TMEM (over S) as bf16.
//   warp 8           : TMA: query tiles, and K and V tiles into a ring.
//   warps 9, 10      : MMA issue: S = Q K^T, O += P V.  Their steps alternate
//                      between the streams.
// P is rounded to bf16 for the second product, the operand type of V; its sum
// is taken in f32 before that rounding.
#include <math.h>

#include "attention.h"
#include "gemm_epilogue.cuh"
#include "head_norm_rope.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace ck {
namespace {

constexpr int kRows = 128;     // rows of a query tile
constexpr int kKeys = 128;     // keys of a key tile
constexpr int kTmaWarp = 8, kQkWarp = 9, kPvWarp = 10;
constexpr int kThreads = 384;  // 8 softmax warps, TMA, 2 MMA, 1 idle (register shares go by 4 warps)
// Registers a thread: 168 at launch; the softmax holds a row of 128 scores.
// 256 x 208 + 128 x 88 = 384 x 168.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
// Keys of a tile whose P is handed over first: P V of them runs while the last
// exponentials are taken.
constexpr int kFirstKeys = 96;
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
// The accumulator is rescaled only when a row's maximum has grown by more than
// 2^8: until then its exponentials are taken against the old maximum, at most
// 256 instead of 1, which f32 sums and bf16's exponent range take unharmed.
constexpr float kRescaleLog2 = 8.f;

template <int D>
struct Cfg {
    static constexpr int kHalves = D / 64;         // 128-byte swizzle columns of a tile
    static constexpr int kHalfBytes = kKeys * 128;
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    static constexpr int kSlots = D == 128 ? 5 : 10;  // ring of K and V tiles: 160 KB
    static constexpr int kBarBytes = 512;
    static constexpr size_t kSmemBytes = static_cast<size_t>(2 + kSlots) * kTileBytes + kBarBytes + 1024;
};

// What the kernels take: sizes, pointers and the split of the work.
struct Work {
    uint16_t *out;
    int64_t ldo;
    int B, Lq, Hkv, G, T;  // T = B * Lq tokens
    int page_size;         // 0: dense
    int pages;
    const int32_t *prefix_pages, *block_table, *lens;
    int64_t table_stride;
    int prefix_len, max_len;
    bool causal;
    float scale_log2;  // scale * log2(e)
    // prefix items: rt_p row items x Hkv x split_p chunks; own: rt_o x Hkv x B x split_o
    int wide_p, wide_o, tok_p, tok_o;  // tok: query tokens of one tile
    int rt_p, rt_o, chunk_p, chunk_o;  // chunk: keys
    int items_p, items;
    int slots_p, slots;                // partial results of a row; slots = 0: written to out directly
    float *part_o;                     // [slots][T * Hq][D]
    float2 *part_ml;                   // [slots][T * Hq]: log2-scaled maximum, sum
    unsigned int *status;
    unsigned long long timeout_ns;
};

struct Item {
    int b;             // sequence; -1: prefix
    int h;             // key head
    int tok0, tok_end; // its query tokens
    int tok;           // tokens of one tile
    int key0, nkeys;   // its keys
    int lim0, lim_step;  // token t sees the keys below lim0 + lim_step * t
    int slot;
    bool wide;
};

// The length of sequence b; out of range: the nearer end (`bad` is set).
__device__ __forceinline__ int own_len(const Work &w, int b, bool &bad) {
    if (!w.lens) return w.max_len;
    const int n = w.lens[b];
    bad = n < 0 || n > w.max_len;
    return min(max(n, 0), w.max_len);
}

__device__ __forceinline__ Item decode(const Work &w, int idx, bool &bad_len) {
    Item it;
    bad_len = false;
    if (idx < w.items_p) {
        const int rt = idx % w.rt_p;
        int r = idx / w.rt_p;
        it.h = r % w.Hkv;
        r /= w.Hkv;
        it.b = -1;
        it.wide = w.wide_p;
        it.tok = w.tok_p;
        it.tok0 = rt * it.tok * (it.wide ? 2 : 1);
        it.tok_end = min(w.T, it.tok0 + it.tok * (it.wide ? 2 : 1));
        it.key0 = r * w.chunk_p;
        it.nkeys = min(w.chunk_p, w.prefix_len - it.key0);
        it.lim0 = w.prefix_len, it.lim_step = 0;
        it.slot = it.wide ? r : 2 * r;
    } else {
        idx -= w.items_p;
        const int rt = idx % w.rt_o;
        int r = idx / w.rt_o;
        it.h = r % w.Hkv;
        r /= w.Hkv;
        it.b = r % w.B;
        r /= w.B;
        it.wide = w.wide_o;
        it.tok = w.tok_o;
        const int first = it.b * w.Lq;
        it.tok0 = first + rt * it.tok * (it.wide ? 2 : 1);
        it.tok_end = min(first + w.Lq, it.tok0 + it.tok * (it.wide ? 2 : 1));
        const int len = own_len(w, it.b, bad_len);
        it.lim_step = w.causal ? 1 : 0;
        it.lim0 = w.causal ? len - w.Lq + 1 - first : len;
        it.key0 = r * w.chunk_o;
        const int last = min(len, it.lim0 + it.lim_step * (it.tok_end - 1));
        it.nkeys = max(0, min(w.chunk_o, last - it.key0));
        it.slot = w.slots_p + (it.wide ? r : 2 * r);
    }
    return it;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of 32 scores (keys 32 Q .. of a tile), those from key `vis` on
// first set to -inf, into four running maxima.
template <int Q>
__device__ __forceinline__ void row_max(uint32_t (&x)[32], bool masked, int vis, float (&mx)[4]) {
    if (masked) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (32 * Q + i >= vis) x[i] = 0xff800000u;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        mx[i / 2 & 3] = max3(mx[i / 2 & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
}

// P of 32 keys: 2^(x c - mc), added to `sum` in f32 and stored as bf16.
__device__ __forceinline__ void weights(const uint32_t (&x)[32], float c, float mc, uint64_t (&sum)[2],
                                        uint32_t taddr) {
    const uint64_t cc = f32x2(c, c), mm = f32x2(-mc, -mc);
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float a, b;
        f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cc, mm), a, b);
        a = ex2(a), b = ex2(b);
        sum[i & 1] = add_f32x2(sum[i & 1], f32x2(a, b));
        p[i] = pack2(a, b);
    }
    tmem_st_32x32b_x16(taddr, p);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap qmap_p, const __grid_constant__ CUtensorMap qmap_o,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ Work w) {
    using C = Cfg<D>;
    constexpr int NS = C::kSlots;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t smem_s = raw_s + pad;
    auto sQ = [&](int i) { return smem_s + i * C::kTileBytes; };
    auto sKV = [&](int s) { return smem_s + (2 + s) * C::kTileBytes; };
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + (2 + NS) * C::kTileBytes);
    const uint32_t bars_s = smem_s + (2 + NS) * C::kTileBytes;
    auto kv_full = [&](int s) { return bars_s + 8u * s; };
    auto kv_empty = [&](int s) { return bars_s + 8u * (NS + s); };
    auto q_full = [&](int i) { return bars_s + 8u * (2 * NS + i); };
    auto q_empty = [&](int i) { return bars_s + 8u * (2 * NS + 2 + i); };
    auto s_full = [&](int i) { return bars_s + 8u * (2 * NS + 4 + i); };  // S of a step is in TMEM
    // P of a step is in TMEM: its first kFirstKeys keys, the others
    auto p_full = [&](int i, int half) { return bars_s + 8u * (2 * NS + 6 + 2 * i + half); };
    auto o_full = [&](int i) { return bars_s + 8u * (2 * NS + 10 + i); };  // its P V is in O
    auto pv_issued = [&](int i) { return bars_s + 8u * (2 * NS + 12 + i); };
    const uint32_t done_bar = bars_s + 8u * (2 * NS + 14);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * NS + 15);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert(8 * (2 * NS + 15) + 8 <= C::kBarBytes);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform for the compiler too
    const int lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, w.status, w.timeout_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i, 0), 4);
            mbar_init(p_full(i, 1), 4);
            mbar_init(o_full(i), 1);
            mbar_init(pv_issued(i), 1);
        }
        mbar_init(done_bar, 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kQkWarp) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto tS = [&](int st) { return tmem + 128u * st; };
    auto tO = [&](int st) { return tmem + 256u + static_cast<uint32_t>(D) * st; };
    pdl_launch_dependents();
    pdl_wait();

    // Every role walks the same items and key tiles with the same counters:
    // J, key tiles so far (K in ring position 2 J, V in 2 J + 1); step, S tiles
    // so far (its parity is the stream); narrow items so far (their query
    // buffer), and the uses of each query buffer.
    if (warp >= kTmaWarp) {
        setmaxnreg_dec<kOtherRegs>();  // by all four warps at once
        if (warp == kTmaWarp) {
            // ------------------------------------------------------------ TMA
            uint32_t seq = 0, nar = 0;
            uint32_t qpar = 0, qused = 0;  // bit i: parity of query buffer i's next use, used at all
            bool ok = true;
            if (elect_one()) {
                tma_prefetch_desc(&qmap_p);
                tma_prefetch_desc(&qmap_o);
                tma_prefetch_desc(&kmap);
                tma_prefetch_desc(&vmap);
            }
            __syncwarp();
#pragma unroll 1
            for (int idx = blockIdx.x; idx < w.items && ok; idx += gridDim.x) {
                bool bad = false;
                const Item it = decode(w, idx, bad);
                if (bad && lane == 0) atomicOr(w.status, kDeviceStatusIndex);
                const int ntiles = (it.nkeys + kKeys - 1) / kKeys;
                const int32_t *table = it.b < 0 ? w.prefix_pages : w.block_table + it.b * w.table_stride;
#pragma unroll 1
                for (int j = 0; j < ntiles && ok; ++j) {
                    const int key = it.key0 + j * kKeys;
                    const int valid = min(kKeys, it.nkeys - j * kKeys);
                    int npages = 0, row = 0;
                    if (w.page_size > 0) {
                        npages = (valid + w.page_size - 1) / w.page_size;
                        if (lane < npages) {
                            const int page = table[key / w.page_size + lane];
                            const bool in = page >= 0 && page < w.pages;
                            if (!in) atomicOr(w.status, kDeviceStatusIndex);
                            // past the cache's rows: TMA fills zeros
                            row = ((in ? page : w.pages) * w.Hkv + (in ? it.h : 0)) * w.page_size;
                        }
                    }
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        const int s = seq % NS;
                        ok = __all_sync(0xffffffffu, mbar_wait_spin(kv_empty(s), ((seq / NS) & 1) ^ 1, ctl));
                        if (!ok) break;
                        const CUtensorMap *map = kv == 0 ? &kmap : &vmap;
                        if (w.page_size > 0) {
                            if (elect_one())
                                mbar_arrive_expect_tx(kv_full(s), npages * w.page_size * 128 * C::kHalves);
                            __syncwarp();
                            if (lane < npages) {
#pragma unroll 1
        #pragma unroll 1
                            for (int hf = 0; hf < C::kHalves; ++hf)
                                    tma_load_2d(sKV(s) + hf * C::kHalfBytes + lane * w.page_size * 128, map, kv_full(s),
                                                hf * 64, row);
                            }
                            __syncwarp();
                        } else if (elect_one()) {
                            mbar_arrive_expect_tx(kv_full(s), C::kTileBytes);
#pragma unroll 1
                            for (int hf = 0; hf < C::kHalves; ++hf)
                                tma_load_2d(sKV(s) + hf * C::kHalfBytes, map, kv_full(s), it.h * D + hf * 64,
                                            it.b * w.max_len + key);
                        }
                        __syncwarp();
                        ++seq;
                        if (kv == 0 && j == 0) {
                            // the item's query tiles, behind its first K tile: the
                            // buffers are free once the last item's S are done
                            const CUtensorMap *qm = it.b < 0 ? &qmap_p : &qmap_o;
#pragma unroll 1
                            for (int i = 0; i < (it.wide ? 2 : 1) && ok; ++i) {
                                const int buf = it.wide ? i : static_cast<int>(nar & 1);
                                ok = __all_sync(0xffffffffu, mbar_wait_spin(q_empty(buf), ((qpar >> buf) & 1) ^ 1, ctl));
                                if (!ok) break;
                                if (elect_one()) {
                                    mbar_arrive_expect_tx(q_full(buf), it.tok * w.G * 128 * C::kHalves);
        #pragma unroll 1
        #pragma unroll 1
                            for (int hf = 0; hf < C::kHalves; ++hf)
                                        tma_load_3d(sQ(buf) + hf * C::kHalfBytes, qm, q_full(buf), hf * 64, it.h * w.G,
                                                    it.tok0 + i * it.tok);
                                }
                                __syncwarp();
                                qpar ^= 1u << buf;
                                qused |= 1u << buf;
                            }
                        }
                    }
                }
                if (!it.wide && ntiles > 0) ++nar;
            }
            if (*abort_flag && elect_one()) {
                // let the copies still in flight land before the CTA exits
                for (uint32_t q = seq > NS ? seq - NS : 0; q < seq; ++q)
                    mbar_wait_drain(kv_full(q % NS), (q / NS) & 1, w.timeout_ns, w.status);
                for (int i = 0; i < 2; ++i)
                    if ((qused >> i) & 1) mbar_wait_drain(q_full(i), ((qpar >> i) & 1) ^ 1, w.timeout_ns, w.status);
            }
            __syncwarp();
        } else if (warp == kQkWarp || warp == kPvWarp) {
            // ------------------------------------------------------------ MMA
            // One warp issues S = Q K^T of every step, one O += P V; both take
            // the steps in the same order, which alternates between the streams
            // and so keeps one in its softmax while the other's products run.
            // (A poll of a barrier takes some 120 cycles, and a commit returns
            // when the products before it have nearly run: one warp for both
            // spent 1800 cycles on a step's 1024 of tensor work; a warp for each
            // stream let the streams fall into step.)  The whole warp runs the
            // loop and one elected lane issues; counters and descriptors are
            // kept uniform over the warp -- a key count that was read from
            // memory goes through a shuffle for that -- and the K steps of a
            // tile are unrolled.
            constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kKeys, false);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, D, true);
            constexpr uint32_t tile_desc = C::kTileBytes / 16;
            const bool is_qk = warp == kQkWarp;
            const uint64_t qd0 = sdesc_kmajor_sw128(sQ(0));
            const uint64_t kd0 = sdesc_kmajor_sw128(sKV(0));
            const uint64_t vd0 = sdesc_mnmajor_sw128(sKV(0), C::kHalfBytes);
            bool ok = true;
            int step = 0, nar = 0;
            int slot = is_qk ? 0 : 1;  // ring position of the tile's K / V
            uint32_t par = 0;          // its parity
            uint32_t qpar = 0;         // bit i: parity of query buffer i
            uint32_t spar = 0;         // bit i: parity of stream i: QK: its P V issued; PV: its P
#pragma unroll 1
            for (int idx = blockIdx.x; idx < w.items && ok; idx += gridDim.x) {
                bool bad;
                const Item it = decode(w, idx, bad);
                const int nkeys = __shfl_sync(0xffffffffu, it.nkeys, 0);
                const int ntiles = (nkeys + kKeys - 1) / kKeys;
                const int subs = it.wide ? 2 : 1;
#pragma unroll 1
                for (int j = 0; j < ntiles && ok; ++j) {
                    ok = __all_sync(0xffffffffu, mbar_wait_spin(kv_full(slot), par, ctl));
                    if (!ok) break;
                    const int valid = min(kKeys, nkeys - j * kKeys);
                    const uint64_t kvd = (is_qk ? kd0 : vd0) + static_cast<uint32_t>(slot) * tile_desc;
                    if (is_qk) {
#pragma unroll 1
                        for (int sub = 0; sub < subs; ++sub, ++step) {
                            const int st = step & 1;
                            const int buf = it.wide ? st : nar & 1;
                            if (j == 0) {
                                ok = __all_sync(0xffffffffu, mbar_wait_spin(q_full(buf), (qpar >> buf) & 1, ctl));
                                if (!ok) break;
                                qpar ^= 1u << buf;
                            }
                            if (step >= 2) {
                                // P V of the stream's last step, whose P lies over
                                // S, is in the tensor core's queue: in order, this
                                // product comes after it
                                ok = __all_sync(0xffffffffu, mbar_wait_spin(pv_issued(st), (spar >> st) & 1, ctl));
                                if (!ok) break;
                                spar ^= 1u << st;
                            }
                            tc_fence_after_sync();
                            if (elect_one()) {
                                const uint64_t qd = qd0 + static_cast<uint32_t>(buf) * tile_desc;
                                const uint32_t s = tS(st);
#pragma unroll
                                for (int ks = 0; ks < D / 16; ++ks) {
                                    const uint32_t off = (ks / 4) * (C::kHalfBytes / 16) + 2u * (ks % 4);
                                    mma_f16_ss(s, qd + off, kvd + off, idesc_qk, ks > 0 ? 1u : 0u);
                                }
                                mma_commit(s_full(st));
                                if (sub == subs - 1) mma_commit(kv_empty(slot));
                                if (j == ntiles - 1) mma_commit(q_empty(buf));
                            }
                            __syncwarp();
                        }
                    } else {
                        if (valid & 15) {
                            // The last 16 keys of P V reach past the real ones: P
                            // is 0 there, but 0 x NaN is not, so those rows of V
                            // are cleared.
                            const int n = (16 - (valid & 15)) * 8;  // 16-byte pieces of a swizzle column
                            for (int i = lane; i < n * C::kHalves; i += 32) {
                                const int hf = i / n, r = i - hf * n;
                                *reinterpret_cast<uint4 *>(smem + (2 + slot) * C::kTileBytes + hf * C::kHalfBytes +
                                                           valid * 128 + r * 16) = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
#pragma unroll 1
                        for (int sub = 0; sub < subs; ++sub, ++step) {
                            const int st = step & 1;
                            const uint32_t o = tO(st), p = tS(st);
                            const bool first = it.wide ? j == 0 : j < 2;
                            ok = __all_sync(0xffffffffu, mbar_wait_spin(p_full(st, 0), (spar >> st) & 1, ctl));
                            if (!ok) break;
                            tc_fence_after_sync();
                            if (elect_one()) {
                                mma_f16_ts(o, p, kvd, idesc_pv, first ? 0u : 1u);
#pragma unroll
                                for (int ks = 1; ks < kFirstKeys / 16; ++ks)
                                    if (16 * ks < valid) mma_f16_ts(o, p + 8u * ks, kvd + 128u * ks, idesc_pv, 1u);
                            }
                            __syncwarp();
                            ok = __all_sync(0xffffffffu, mbar_wait_spin(p_full(st, 1), (spar >> st) & 1, ctl));
                            if (!ok) break;
                            tc_fence_after_sync();
                            if (elect_one()) {
#pragma unroll
                                for (int ks = kFirstKeys / 16; ks < 8; ++ks)
                                    if (16 * ks < valid) mma_f16_ts(o, p + 8u * ks, kvd + 128u * ks, idesc_pv, 1u);
                                tc_fence_before_sync();
                                mbar_arrive(pv_issued(st));
                                mma_commit(o_full(st));
                                if (sub == subs - 1) mma_commit(kv_empty(slot));
                            }
                            __syncwarp();
                            spar ^= 1u << st;
                        }
                    }
                    slot += 2;
                    if (slot >= NS) slot -= NS, par ^= 1;
                }
                if (!it.wide && ntiles > 0) ++nar;
            }
            // no MMA may be in flight when TMEM is released
            if (elect_one()) {
                mma_commit(done_bar);
                mbar_wait_drain(done_bar, 0, w.timeout_ns, w.status);
            }
            __syncwarp();
        }
    } else {
        setmaxnreg_inc<kSoftmaxRegs>();
        // ------------------------------------------------------------ softmax
        const int st = warp >> 2;
        const int row = threadIdx.x & 127;
        const int row_tok = row / w.G, row_g = row - row_tok * w.G;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tS(st) + lanes, to = tO(st) + lanes;
        const int Hq = w.Hkv * w.G;
        const int64_t rows = static_cast<int64_t>(w.T) * Hq;
        const float c = w.scale_log2;
        uint32_t step = 0, cnt = 0;
        bool ok = true;
        for (int idx = blockIdx.x; idx < w.items && ok; idx += gridDim.x) {
            bool bad;
            const Item it = decode(w, idx, bad);
            const int ntiles = (it.nkeys + kKeys - 1) / kKeys;
            const int tok = it.tok0 + (it.wide ? st * it.tok : 0) + row_tok;
            const bool live = row_tok < it.tok && tok < it.tok_end;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int limit = it.lim0 + it.lim_step * tok;
            float mref = -INFINITY, l = 0.f;
            int done = 0;  // tiles of this stream
            for (int j = 0; j < ntiles; ++j) {
                if (!it.wide) {
                    if (static_cast<int>(step++ & 1) != st) continue;
                }
                ok = __all_sync(0xffffffffu, mbar_wait_spin(s_full(st), cnt & 1, ctl));
                if (!ok) break;
                tc_fence_after_sync();
                const int key = j * kKeys;
                const int valid = min(kKeys, it.nkeys - key);
                uint32_t sr[4][32];
                uint64_t sum[2] = {0, 0};
                float mc = 0.f;
                auto arrive = [&](int half) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(st, half));
                };
                if (warp_live) {
                    const int vis = live ? min(max(limit - it.key0 - key, 0), valid) : 0;
                    tmem_ld_32x32b_x32(ts, sr[0]);
                    tmem_ld_32x32b_x32(ts + 32u, sr[1]);
                    tmem_wait_ld(sr[0]);
                    tmem_wait_ld(sr[1]);
                    tmem_ld_32x32b_x32(ts + 64u, sr[2]);
                    tmem_ld_32x32b_x32(ts + 96u, sr[3]);
                    const bool masked = __any_sync(0xffffffffu, vis < kKeys);
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    row_max<0>(sr[0], masked, vis, mx);
                    row_max<1>(sr[1], masked, vis, mx);
                    tmem_wait_ld(sr[2]);
                    tmem_wait_ld(sr[3]);
                    row_max<2>(sr[2], masked, vis, mx);
                    row_max<3>(sr[3], masked, vis, mx);
                    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (done == 0) {
                        mref = mt;
                    } else {
                        const float m_new = fmaxf(mref, mt);
                        const bool grow = (m_new - mref) * c > kRescaleLog2;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = grow ? ex2((mref - m_new) * c) : 1.f;
                            ok = __all_sync(0xffffffffu, mbar_wait_spin(o_full(st), (cnt - 1) & 1, ctl));
                            if (!ok) break;
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t o[16];
                                tmem_ld_32x32b_x16(to + 16u * q, o);
                                tmem_wait_ld16(o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st_32x32b_x16(to + 16u * q, o);
                            }
                            l *= f;
                            if (grow) mref = m_new;
                        }
                    }
                    mc = mref == -INFINITY ? 0.f : mref * c;
                    weights(sr[0], c, mc, sum, ts + 0u);
                    weights(sr[1], c, mc, sum, ts + 16u);
                    weights(sr[2], c, mc, sum, ts + 32u);
                    tmem_wait_st();
                }
                arrive(0);
                if (warp_live) {
                    weights(sr[3], c, mc, sum, ts + 48u);
                    tmem_wait_st();
                }
                arrive(1);
                if (warp_live) {
                    float a, b;
                    f32x2_split(add_f32x2(sum[0], sum[1]), a, b);
                    l += a + b;
                }
                ++cnt;
                ++done;
            }
            if (!ok) break;
            if (it.wide) step += 2 * ntiles;
            // the item's result
            if (done > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait_spin(o_full(st), (cnt - 1) & 1, ctl));
                if (!ok) break;
                tc_fence_after_sync();
            }
            if (warp_live) {
                // Stored through a 4 x 4 transpose of 16-byte pieces within each
                // quad of lanes: an instruction then writes 64 bytes of 8 rows
                // instead of 16 bytes of 32.
                const int64_t at = static_cast<int64_t>(tok) * Hq + it.h * w.G + row_g;
                const bool part = w.slots > 0;
                const int64_t pr = part ? (it.slot + (it.wide ? 0 : st)) * rows + at : 0;
                if (part && live) w.part_ml[pr] = make_float2(mref == -INFINITY ? mref : mref * c, l);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int64_t mine = part ? pr * D : tok * w.ldo + static_cast<int64_t>(it.h * w.G + row_g) * D;
                const int qi = lane & 3;
                int64_t off[4];
                bool on[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    off[k] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + k);
                    on[k] = __shfl_sync(0xffffffffu, live, (lane & ~3) + k);
                }
                if (done > 0 || !part) {
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t o[32];
                        if (done > 0) {
                            tmem_ld_32x32b_x32(to + 32u * q, o);
                            tmem_wait_ld(o);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = 0;
                        }
                        if (part) {
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                uint32_t p[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) p[i] = o[16 * g + i];
                                ep::quad_transpose(p, qi);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (on[k])
                                        *reinterpret_cast<uint4 *>(w.part_o + off[k] + 32 * q + 16 * g + 4 * qi) =
                                            make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
                            }
                        } else {
                            uint32_t p[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                p[i] = pack2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                            ep::quad_transpose(p, qi);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (on[k])
                                    *reinterpret_cast<uint4 *>(w.out + off[k] + 32 * q + 8 * qi) =
                                        make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
                        }
                    }
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kQkWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over a row's partial
// results (M their largest m); a warp per row.  Parts with l = 0 saw no key and
// have no o.
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ Work w) {
    pdl_launch_dependents();
    pdl_wait();
    const int Hq = w.Hkv * w.G;
    const int64_t rows = static_cast<int64_t>(w.T) * Hq;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    constexpr int E = D / 32;
    float M = -INFINITY;
    for (int s = 0; s < w.slots; ++s) {
        const float2 ml = w.part_ml[s * rows + row];
        if (ml.y != 0.f) M = fmaxf(M, ml.x);
    }
    float L = 0.f, o[E] = {};
    for (int s = 0; s < w.slots; ++s) {
        const float2 ml = w.part_ml[s * rows + row];
        if (ml.y == 0.f) continue;
        const float f = ex2(ml.x - M);
        L = fmaf(f, ml.y, L);
        const float *src = w.part_o + (s * rows + row) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(f, src[e], o[e]);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t tok = row / Hq;
    uint16_t *dst = w.out + tok * w.ldo + (row - tok * Hq) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(dst + e) = pack2(o[e] * inv, o[e + 1] * inv);
}

// Planned for this many SMs whatever the device has, so that the workspace is a
// function of the sizes alone.
constexpr int kPlanSms = 152;

int div_up(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// How the work is cut.  Rows come first: two row tiles an item where there are
// more than one.  Keys are cut where the rows alone leave SMs idle, into at
// least 4 tiles a chunk (a chunk's partial result costs about as much to write
// and join as half a key tile to read).
Work plan(const AttentionArgs &a) {
    Work w = {};
    w.B = static_cast<int>(a.B), w.Lq = static_cast<int>(a.Lq), w.T = static_cast<int>(a.B * a.Lq);
    w.Hkv = a.Hkv, w.G = a.G;
    w.prefix_len = static_cast<int>(a.prefix_len), w.max_len = static_cast<int>(a.max_len);
    w.causal = a.causal;
    const int tokens = kRows / a.G;
    w.tok_p = w.T < tokens ? w.T : tokens;
    w.tok_o = w.Lq < tokens ? w.Lq : tokens;
    w.wide_p = w.T > tokens, w.wide_o = w.Lq > tokens;
    w.rt_p = div_up(w.T, w.tok_p * (w.wide_p ? 2 : 1));
    w.rt_o = div_up(w.Lq, w.tok_o * (w.wide_o ? 2 : 1));
    const int64_t tiles_p = div_up(w.prefix_len, kKeys), tiles_o = div_up(w.max_len, kKeys);
    const int64_t base_p = static_cast<int64_t>(w.rt_p) * w.Hkv, base_o = static_cast<int64_t>(w.rt_o) * w.Hkv * w.B;
    // tiles of a chunk: the whole work spread over twice the SMs
    const int64_t steps = base_p * tiles_p * (w.wide_p ? 2 : 1) + base_o * tiles_o * (w.wide_o ? 2 : 1);
    const int64_t share = steps / (2 * kPlanSms) + 1;
    auto chunk = [&](int64_t tiles, bool wide) {
        int64_t n = wide ? (share + 1) / 2 : share;
        if (n < 4) n = 4;
        if (n > tiles) n = tiles;
        const int64_t parts = (tiles + n - 1) / n;
        return (tiles + parts - 1) / parts;  // equal parts
    };
    int64_t split_p = 0, split_o = 0;
    if (tiles_p > 0) {
        const int64_t n = chunk(tiles_p, w.wide_p);
        w.chunk_p = static_cast<int>(n) * kKeys;
        split_p = (tiles_p + n - 1) / n;
    }
    if (tiles_o > 0) {
        const int64_t n = chunk(tiles_o, w.wide_o);
        w.chunk_o = static_cast<int>(n) * kKeys;
        split_o = (tiles_o + n - 1) / n;
    }
    // no key at all: one empty own chunk writes the zeros
    if (split_p + split_o == 0) split_o = 1, w.chunk_o = kKeys;
    w.items_p = static_cast<int>(base_p * split_p);
    w.items = static_cast<int>(w.items_p + base_o * split_o);
    w.slots_p = static_cast<int>(split_p) * (w.wide_p ? 1 : 2);
    w.slots = w.slots_p + static_cast<int>(split_o) * (w.wide_o ? 1 : 2);
    if (w.slots == 1) w.slots_p = w.slots = 0;
    return w;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t ml_bytes(const Work &w) { return round256(static_cast<size_t>(w.slots) * w.T * w.Hkv * w.G * sizeof(float2)); }

bool row_map(CUtensorMap *m, const AttentionArgs &a, int tokens) {
    const uint64_t dims[3] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.Hq),
                              static_cast<uint64_t>(a.B * a.Lq)};
    const uint64_t strides[2] = {static_cast<uint64_t>(a.D) * 2, static_cast<uint64_t>(a.ldq) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(tokens)};
    return tensor_map_bf16(m, a.q, 3, dims, strides, box);
}

bool key_map(CUtensorMap *m, const AttentionArgs &a, const uint16_t *p, int64_t ld) {
    uint64_t dims[2], strides[1];
    uint32_t box[2] = {64, kKeys};
    if (a.pages > 0) {
        dims[0] = static_cast<uint64_t>(a.D);
        dims[1] = static_cast<uint64_t>(a.pages * a.Hkv * a.page_size);
        strides[0] = static_cast<uint64_t>(a.D) * 2;
        box[1] = static_cast<uint32_t>(a.page_size);
    } else {
        dims[0] = static_cast<uint64_t>(a.Hkv) * a.D;
        dims[1] = static_cast<uint64_t>(a.B * a.max_len);
        strides[0] = static_cast<uint64_t>(ld) * 2;
    }
    return tensor_map_bf16(m, p, 2, dims, strides, box);
}

template <int D>
cudaError_t launch(const AttentionArgs &a, Work &w, const LaunchCtx &ctx) {
    CUtensorMap qp, qo, km, vm;
    if (!row_map(&qp, a, w.tok_p) || !row_map(&qo, a, w.tok_o)) return cudaErrorInvalidValue;
    if (a.k) {
        if (!key_map(&km, a, a.k, a.ldk) || !key_map(&vm, a, a.v, a.ldv)) return cudaErrorInvalidValue;
    } else {
        km = vm = qo;  // no key at all: never used
    }
    auto kern = attention_kernel<D>;
    constexpr size_t smem = Cfg<D>::kSmemBytes;
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), static_cast<int>(smem));
        e != cudaSuccess)
        return e;
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(w.items < sms ? w.items : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx.stream;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 1 : 0;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, qp, qo, km, vm, w); e != cudaSuccess) return e;
    if (w.slots == 0) return cudaSuccess;
    const int64_t rows = static_cast<int64_t>(w.T) * w.Hkv * w.G;
    cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<D>, w);
}

}  // namespace

size_t attention_workspace_bytes(const AttentionArgs &a) {
    const Work w = plan(a);
    if (w.slots == 0) return 0;
    return ml_bytes(w) + static_cast<size_t>(w.slots) * w.T * w.Hkv * w.G * a.D * sizeof(float);
}

cudaError_t launch_attention(const AttentionArgs &a, const LaunchCtx &ctx) {
    Work w = plan(a);
    w.out = a.out, w.ldo = a.ldo;
    w.page_size = a.pages > 0 ? a.page_size : 0, w.pages = static_cast<int>(a.pages);
    w.prefix_pages = a.prefix_pages, w.block_table = a.block_table, w.lens = a.lens, w.table_stride = a.table_stride;
    w.scale_log2 = a.scale * kLog2e;
    if (w.slots > 0) {
        w.part_ml = static_cast<float2 *>(a.ws);
        w.part_o = reinterpret_cast<float *>(static_cast<char *>(a.ws) + ml_bytes(w));
    }
    w.status = ctx.status;
    w.timeout_ns = ctx.timeout_ns;
    return a.D == 64 ? launch<64>(a, w, ctx) : launch<128>(a, w, ctx);
}

}  // namespace ck
