// head_norm_rope.cu -- the two passes between the qkv linear and attention:
// the norm and rotation of query and key heads, and the append of keys (normed
// and rotated on the way) and values to a paged cache.
#include "head_norm_rope.cuh"
#include "attention.h"
#include "internal.h"
#include "launch_util.h"
#include "ptx.cuh"

namespace ck {
namespace {

// Rows of a group of lanes in one unit of work, and blocks that share an SM (by
// their registers): of 2, 4 and 8 rows with 512 to 1280 threads an SM, 8 rows
// with 640 were best at long calls (30011 tokens x 48 heads x 128: 131 us; 4 rows
// with 768 139, 2 with 1024 170, 8 with 768, which spill, 160).  At 640 the norm's
// kernels spill nothing, the append's 4 (halves) and 36 bytes (pairs side by side).
constexpr int kRows = 8;
constexpr int kThreads = 128;
constexpr int kBlocksPerSm = 5;

// How the blocks' groups of L lanes are dealt out.  Blocks from `blocks_q` on
// have the keys (of the append: none).  2^gp_log2 groups share a token, the g-th
// taking its heads g, g + 2^gp_log2, ..., in `batches` units.
struct Deal {
    int blocks_q;
    int gp_log2[2], batches[2];
};

// The factors of a token's pairs; `ok`: it has any (and a place in the cache).
struct Token {
    float4 c, s;
    int64_t at;
    bool ok;
};

// Both passes are a copy with arithmetic: read once, written once, and HBM's
// rate is the floor.  Latency is what they have to hide: a token's position comes
// before its factors, and both before its rows can be used.  So a block is
// persistent: while it works on one unit, the next one's factors and the position
// after that are on their way, and a row's place is refilled from the next unit
// as soon as it has been used.  Then instructions count (some 170 a warp for two
// rows of 128 at first): a lane holds whole pairs, weights and factors are
// multiplied once for all heads of a token, arithmetic is on two elements at a
// time, and addresses are worked out once a unit.
// Measured: 30011 tokens x 48 heads x 128 in 131 us (5.7 TB/s, 0.84 of the
// measured copy), 4096 x 64 in 26 us (5.2 TB/s), append of 65519 tokens x 8 heads
// in 91 us (6.1 TB/s, 0.90).  Tried and slower: a block for each token (191 us),
// rows fetched three units ahead through shared memory (247 us).
template <int L, bool INTERLEAVED, typename Rows>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
head_rows_kernel(const __grid_constant__ typename Rows::Args a, const __grid_constant__ Deal deal) {
    pdl_launch_dependents();
    const int side = static_cast<int>(blockIdx.x) < deal.blocks_q ? 0 : 1;
    const int block = blockIdx.x - (side == 0 ? 0 : deal.blocks_q);
    const int blocks = side == 0 ? deal.blocks_q : gridDim.x - deal.blocks_q;
    const int gp_log2 = deal.gp_log2[side], batches = deal.batches[side];
    const int gl = threadIdx.x % L, group = threadIdx.x / L;
    const int per = (kThreads / L) >> gp_log2;  // tokens of a block at once
    const Place<INTERLEAVED> p(gl, a.D, a.rot);
    const Rows rows(a, side, 1 << gp_log2, group & ((1 << gp_log2) - 1));
    const int64_t step = static_cast<int64_t>(blocks) * per;
    const int64_t first = static_cast<int64_t>(block) * per;
    const int64_t mine = first + (group >> gp_log2);
    pdl_wait();
    const Pairs w = load_weights<INTERLEAVED>(rows.weight(), a.w_f32, p);
    const bool norm = rows.weight() != nullptr;

    // A unit's rows: `rows.from(t, batch)` and every `stride` elements on (of the
    // second half of an append's unit: the values).
    const int stride = a.D << gp_log2;
    auto load = [&](const uint16_t *src, int i, uint4 &v) { v = load_row<INTERLEAVED>(src + i * stride, p); };
    struct Index {
        int pos;
        int64_t slot;
    };
    auto load_index = [&](int64_t t) {
        Index x{0, 0};
        if (t < a.T) {
            if (a.rot > 0) x.pos = a.positions[t];
            x.slot = rows.slot(t);
        }
        return x;
    };
    auto load_token = [&](int64_t t, const Index &x, bool report, Token &k) {
        k.ok = t < a.T && p.on && rows.place(x.slot, report, k.at);
        if (k.ok && a.rot > 0) {
            const bool in_table = x.pos >= 0 && x.pos < a.max_pos;
            if (in_table && p.rotated)
                load_factors<INTERLEAVED>(a.cos_sin + static_cast<int64_t>(x.pos) * a.rot, a.rot, p, k.c, k.s);
            if (!in_table && report) atomicOr(a.status, kDeviceStatusIndex);
            k.ok = in_table;
        }
    };

    uint4 v[kRows];
    Token token;
    token.c = make_float4(1.f, 1.f, 1.f, 1.f), token.s = make_float4(0.f, 0.f, 0.f, 0.f);
    token.at = 0;
    auto forward = [&](int64_t &t, int &j) {
        if (++j == batches) j = 0, t += step;
    };
    // this unit, and the one after the next
    int64_t t0 = mine, t1 = mine, t2;
    int j0 = 0, j1 = 0, j2;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (mine < a.T && p.on && rows.has(0, i)) load(rows.from(mine, 0, i), i % Rows::kHeads, v[i]);
    }
    load_token(mine, load_index(mine), gl == 0, token);
    forward(t1, j1);
    t2 = t1, j2 = j1;
    Index index = load_index(t1);
    forward(t2, j2);
    // every group of a block makes the same rounds
    for (int64_t block_t = first; block_t < a.T;) {
        Factors k;
        set_factors(k, w, p.rotated, token.c, token.s);
        const int64_t at = token.at;
        const bool ok = token.ok;
        load_token(t1, index, gl == 0 && j1 == 0, token);
        index = load_index(t2);
        const bool more = t1 < a.T && p.on;
#pragma unroll
        for (int half = 0; half < kRows / Rows::kHeads; ++half) {
            uint16_t *const dst = rows.to(t0, at, j0, half * Rows::kHeads);
            const uint16_t *const src = rows.from(more ? t1 : 0, j1, half * Rows::kHeads);
            const int64_t dst_stride = rows.to_stride(stride);
#pragma unroll
            for (int i0 = 0; i0 < Rows::kHeads; ++i0) {
                const int i = half * Rows::kHeads + i0;
                if (rows.any(j0, i)) {  // uniform over the block
                    uint4 out = v[i];
                    if (!rows.plain(i))
                        out = norm_rotate<L, INTERLEAVED>(out, norm, a.inv_d, a.eps, a.rot < a.D, p.rotated, k);
                    if (ok && rows.has(j0, i)) store_row<INTERLEAVED>(dst + i0 * dst_stride, p, out);
                }
                // its place is free for the next unit's
                if (more && rows.has(j1, i)) load(src, i0, v[i]);
            }
        }
        if (j0 + 1 == batches) block_t += step;
        t0 = t1, j0 = j1;
        t1 = t2, j1 = j2;
        forward(t2, j2);
    }
}

// Query heads (side 0) or key heads (side 1) of a token.
struct QkRows {
    using Args = NormRopeArgs;
    static constexpr int kHeads = kRows;
    const Args &a;
    int side, gp, g, heads;
    __device__ QkRows(const Args &args, int s, int gp_, int g_)
        : a(args), side(s), gp(gp_), g(g_), heads(s == 0 ? args.Hq : args.Hk) {}
    __device__ int head(int batch, int i) const { return (batch * kRows + i) * gp + g; }
    __device__ const void *weight() const { return side == 0 ? a.wq : a.wk; }
    __device__ const uint16_t *from(int64_t t, int batch, int) const {
        return (side == 0 ? a.q + t * a.ldq : a.k + t * a.ldk) + head(batch, 0) * a.D;
    }
    __device__ uint16_t *to(int64_t t, int64_t, int batch, int) const {
        return (side == 0 ? a.q_out + t * a.ldqo : a.k_out + t * a.ldko) + head(batch, 0) * a.D;
    }
    __device__ int64_t to_stride(int stride) const { return stride; }
    __device__ bool any(int batch, int i) const { return (batch * kRows + i) * gp < heads; }
    __device__ bool has(int batch, int i) const { return head(batch, i) < heads; }
    __device__ bool plain(int) const { return false; }
    __device__ int64_t slot(int64_t) const { return 0; }
    __device__ bool place(int64_t, bool, int64_t &) const { return true; }
};

// Key heads of a token (the first half of a unit's rows) and its value heads.
struct AppendRows {
    using Args = KvAppendArgs;
    static constexpr int kHeads = kRows / 2;
    const Args &a;
    int gp, g;
    __device__ AppendRows(const Args &args, int, int gp_, int g_) : a(args), gp(gp_), g(g_) {}
    __device__ int head(int batch, int i) const { return (batch * kHeads + i % kHeads) * gp + g; }
    __device__ const void *weight() const { return a.wk; }
    __device__ const uint16_t *from(int64_t t, int batch, int i) const {
        return (i < kHeads ? a.k + t * a.ldk : a.v + t * a.ldv) + head(batch, 0) * a.D;
    }
    __device__ uint16_t *to(int64_t, int64_t at, int batch, int i) const {
        return (i < kHeads ? a.k_cache : a.v_cache) + at + static_cast<int64_t>(head(batch, 0)) * a.page_size * a.D;
    }
    __device__ int64_t to_stride(int stride) const { return static_cast<int64_t>(stride) * a.page_size; }
    __device__ bool any(int batch, int i) const { return (batch * kHeads + i % kHeads) * gp < a.Hkv; }
    __device__ bool has(int batch, int i) const { return head(batch, i) < a.Hkv; }
    __device__ bool plain(int i) const { return i >= kHeads; }
    __device__ int64_t slot(int64_t t) const { return a.slots[t]; }
    // Where a slot's rows are: of head 0, its row of its page.
    __device__ bool place(int64_t slot, bool report, int64_t &at) const {
        if (slot < 0) return false;
        if (slot >= a.pages * a.page_size) {
            if (report) atomicOr(a.status, kDeviceStatusIndex);
            return false;
        }
        const int64_t page = slot <= 0x7fffffff ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page_size)
                                                : slot / a.page_size;
        at = (page * a.Hkv * a.page_size + (slot - page * a.page_size)) * a.D;
        return true;
    }
};

// Lanes that hold a row: the power of two of at least D / 8.
int group_lanes(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

// Groups of lanes that share a token of `heads` heads, a unit holding `rows` of
// them a group: as many as leave the fewest of a unit's rows unused.  A few
// tokens leave SMs idle, so there a token's heads are spread as far as they go.
void deal_heads(int64_t T, int heads, int rows, int L, int *gp_log2, int *batches) {
    const int groups = kThreads / L;
    const bool few = T * heads <= static_cast<int64_t>(4) * sm_count() * groups;
    int best = 0, held = 1 << 30;
    for (int n = 0; (1 << n) <= groups; ++n) {
        const int unit = few ? 1 << n : rows << n;
        const int places = (heads + unit - 1) / unit * unit;
        if ((few && (1 << n) >= 2 * heads) || (!few && places > held)) continue;
        best = n, held = places;
    }
    *gp_log2 = best;
    *batches = (heads + (rows << best) - 1) / (rows << best);
}

template <typename Rows>
cudaError_t launch_rows(const typename Rows::Args &a, const int (&heads)[2], bool interleaved,
                        const LaunchCtx &ctx) {
    using Kernel = void (*)(const typename Rows::Args, const Deal);
    static const Kernel kernels[3][2] = {
        {head_rows_kernel<8, false, Rows>, head_rows_kernel<8, true, Rows>},
        {head_rows_kernel<16, false, Rows>, head_rows_kernel<16, true, Rows>},
        {head_rows_kernel<32, false, Rows>, head_rows_kernel<32, true, Rows>}};
    const int L = group_lanes(a.D);
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    // blocks by the rows of each side
    Deal deal = {};
    int64_t blocks[2] = {0, 0};
    for (int s = 0; s < 2; ++s) {
        if (heads[s] == 0) continue;
        deal_heads(a.T, heads[s], Rows::kHeads, L, &deal.gp_log2[s], &deal.batches[s]);
        const int64_t per = (kThreads / L) >> deal.gp_log2[s];
        const int64_t all = (a.T + per - 1) / per;
        const int64_t share = static_cast<int64_t>(kBlocksPerSm) * sms * heads[s] / (heads[0] + heads[1]);
        blocks[s] = all < share ? all : (share < 1 ? 1 : share);
    }
    deal.blocks_q = static_cast<int>(blocks[0]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks[0] + blocks[1]));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernels[L == 8 ? 0 : (L == 16 ? 1 : 2)][interleaved ? 1 : 0], a, deal);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs &a, bool interleaved, const LaunchCtx &ctx) {
    const int heads[2] = {a.Hq, a.Hk};
    return launch_rows<QkRows>(a, heads, interleaved, ctx);
}

cudaError_t launch_kv_append(const KvAppendArgs &a, bool interleaved, const LaunchCtx &ctx) {
    const int heads[2] = {a.Hkv, 0};
    return launch_rows<AppendRows>(a, heads, interleaved, ctx);
}

}  // namespace ck
