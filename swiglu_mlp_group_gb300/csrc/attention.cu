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
// Items.  A group is the row tiles of one key head that go together, against
// the prefix or against a sequence's own keys; an item is a group x a run of its
// key tiles.  More than one row tile makes a group wide: two row tiles against
// the same key tiles.  A narrow item's key tiles are taken alternately by the two
// halves of the pipeline, which add up what they have at its end.
// Little work is dealt out in fixed chunks of key tiles, an item a CTA.  Of more,
// every CTA gets an equal share (divide below): an equal run of the prefix of a
// group, and a run of the sequence of all groups' own key tiles, cut where its
// share ends.  Pieces of a row leave partial sums with their maximum in the
// workspace, and a second kernel joins them.  Without a prefix, and with more
// groups than SMs of about one length or keys for two tiles at most, whole groups
// are dealt out and written directly.
//
// Pipeline (one CTA per SM, 12 warps).  Two streams, each with its own S and O
// in TMEM and four softmax warps, so that the tensor core works on one while
// the other is in its softmax:
//   warps 0..3, 4..7 : softmax of stream 0 / 1, a thread per row: S from TMEM,
//                      maximum, exponentials, P back to TMEM (over S) as bf16.
//   warp 8           : TMA: query tiles, and K and V tiles into a ring.
//   warps 9, 10      : MMA issue: S = Q K^T, O += P V.  Their steps alternate
//                      between the streams.
//   warp 11          : works the CTA's items out, ahead of the others, and hands
//                      them round in a ring; sends finished rows out by TMA; looks
//                      through V that only an item's later tokens see (LATER).
// In an item of few rows (FEW) the four warps of a stream share them: each has a
// copy of the rows in its 32 of the tile and a quarter of the tile's keys.
// P is rounded to bf16 for the second product, the operand type of V; its sum
// is taken in f32 before that rounding.
//
// What bounds it (measured on GB300).  Wide items: the chain of a stream's tile,
// S -> softmax (1440 cycles) -> P V -> Q K^T, some 2460 cycles for two row tiles
// whose products take 2048 (4096 x 4096, nothing beside it); 2 x 8192 x 4093 x 32
// heads of 128 in 412 to 447 us, over several boxes and ways of calling, 1540 to
// 1670 TFLOP/s, against 1706 of a library's plain product under the power limit.
// Short wide items: their starts and ends besides.  Narrow
// items: the K and V in flight, three of the ring's five 32 KB places an SM (the
// others hold what is being used): 5.5 to 6 TB/s.  Few rows: K and V, 1600 cycles
// for a key tile of 64 KB, and their items' ends, about 4000 cycles from the last P
// on (1000 its product, 2800 the sums over streams and quarters and the store).
// Small calls: latency, some 14 cycles for every instruction that is fetched for
// the first time.
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
constexpr int kTmaWarp = 8, kQkWarp = 9, kPvWarp = 10, kWalkWarp = 11;
constexpr int kItems = 4;    // items in the ring
constexpr int kReaders = 11; // warps that read them
constexpr int kThreads = 384;  // 8 softmax warps, TMA, 2 MMA, items
// Registers a thread: 168 at launch; the softmax holds a row of 128 scores.
// 256 x 208 + 128 x 88 = 384 x 168.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs == kThreads * kLaunchRegs && kThreads * kLaunchRegs <= 65536);
// Keys of a tile whose P is handed over first: P V of them runs while the last
// exponentials are taken (2 x 8192 x 4093 x 32 heads: 96 443 us, 64 502, 112 449,
// all 128 at once 472).
constexpr int kFirstKeys = 96;
// Query rows up to which a narrow item is one of few rows.  The call's kernel has
// their code where that is so of own items and none is wide: 16 x 1 x 1500 x 16
// heads of 64 take 22.4 us without it and 17.2 with it; with wide items besides
// (128 x 1 x 4096 behind 32768, 64 heads over 8 of 128) it is 223 and 246: a wide
// tile, bound by its softmax, takes longer in the kernel that has both.
constexpr int kFewRows = 16;
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
    // barriers, TMEM address, abort flag, Share, items, what is known of bad values
    static constexpr int kBarBytes = D == 128 ? 768 : 1024;
    // maximum and sum of a row, [stream][row]: what the streams of a narrow item
    // tell each other
    static constexpr int kExchangeBytes = 2 * kRows * 8;
    // the last 256: tiles start at a multiple of 1024, as the block's shared
    // memory does by its alignment; with what is left of 227 KB they also do
    // where it starts 256 short of one
    static constexpr size_t kSmemBytes =
        static_cast<size_t>(2 + kSlots) * kTileBytes + kBarBytes + kExchangeBytes + 256;
    static_assert(kSmemBytes <= 227 * 1024);
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
    // groups: rt_p x Hkv against the prefix, rt_o x Hkv x B against own keys
    bool wide_p, wide_o;
    int tok_p, tok_o;  // query tokens of one tile
    int rt_p, rt_o;
    int tiles_p, tiles_o;  // key tiles of the prefix, of the longest sequence
    bool too_large;        // more key tiles than can be counted: refused
    bool direct;           // own groups whole, nothing to join
    // Fixed chunks: parts of a group against the prefix, own (tiles of one:
    // chunk), CTA i taking items i, i + grid, ...; chunk_o 0: shares by cost.
    int parts_p, chunk_p, parts_o, chunk_o;
    int sms;               // CTAs to share the work among
    int cost_p, cost_o, cost_item;  // of a key tile; of a group or item besides
    int min_o;             // own tiles a CTA is given at least, if any
    int slots_p, slots_o;  // most parts of a row: against the prefix, own
    int *parts;            // by cost: [0]: parts of a prefix group; then [B][Hkv][rt_o]: of each own group that has keys
    float *part_o;         // [slots_p + slots_o][T * Hq][D]
    float2 *part_ml;       // the same [..][..]: log2-scaled maximum, sum
    unsigned int *status;
    unsigned long long timeout_ns;
};

// Cost units: a sixteenth of a narrow key tile's time (cost_o of one).  A wide
// tile is bound by its products and exponentials, a narrow one by the K and V it
// streams (64 KB).  In a call that has both (128 sequences x 64 / 8 heads of 128
// behind 32768, own lengths to 4096) they took 2620 cycles for two row tiles and
// 2200, items' ends among them: 19:16.  The 21 is what divided that call best,
// 225 us against 234 at 19 and 238 at 24; other mixed calls were not swept.  An
// item's query loads and result cost about a narrow tile.
constexpr int kTileCost = 16, kWideTileCost = 21, kItemCost = 16;
constexpr int64_t kMostCost = int64_t{1} << 30;

struct Item {
    int b;             // sequence; -1: prefix
    int h;             // key head
    int tok0, tok_end; // its query tokens
    int tok;           // tokens of one tile
    int key0, nkeys;   // its keys
    int lim0;          // a token sees the keys below lim0, of a causal item token t those below lim0 + t
    int slot;            // where its partial result goes
    int own_parts;       // by cost, the last piece of an own group: how many there are, else 0
    int flags;           // kWide, kWhole, kFew, kCausal
};
constexpr int kWide = 1;
constexpr int kWhole = 2;  // all keys of its rows: written to out
constexpr int kFew = 4;    // at most kFewRows query rows
constexpr int kCausal = 8;
constexpr int kEnd = -1;   // nkeys of what follows the last item

// What this CTA does, worked out once.
struct Share {
    int parts_p, chunk_p, items_p;  // a prefix group's parts, tiles of one, parts of all groups
    int ctas;                       // CTAs that take part
    // own key tiles from (sequence, group of it, tile) to (.., .., ..)
    int b_lo, r_lo, t_lo, b_hi, r_hi, t_hi;
    int part_lo;                    // number of the first piece within its group
};

// The length of sequence b; out of range: the nearer end.
__device__ __forceinline__ int own_len(const Work &w, int b) {
    return w.lens ? min(max(w.lens[b], 0), w.max_len) : w.max_len;
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kKeys - 1) / kKeys; }
// Token t of the item sees the keys below.
__device__ __forceinline__ int limit_of(const Item &it, int t) { return it.lim0 + (it.flags & kCausal ? t : 0); }
// The item's keys that all of its rows see: from here on (below nkeys) are those
// that only later query tokens see, at most 255 of them.
__device__ __forceinline__ int seen_by_all(const Item &it) { return limit_of(it, it.tok0) - it.key0; }
constexpr int kNoneBad = 255;

// Is one of two bf16 values infinite or NaN?
__device__ __forceinline__ bool not_finite(uint32_t two) {
    return (((two & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0;
}
// Pairwise the larger of |a| and |b|, NaN if one is.
__device__ __forceinline__ uint32_t abs_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
    return r;
}

// The work's division, by one warp.  Prefix groups are cut into equal parts of
// at most a CTA's share, dealt out in turn -- row tiles of the same keys side by
// side, so that they pass over them together and the keys are read from HBM once
// -- and own tiles, in order, fill every CTA's share up.  Costs fit 30 bits.
__device__ void divide(const Work &w, Share &sh) {
    const int lane = threadIdx.x & 31;
    const int groups = w.Hkv * w.rt_o;  // of one sequence
    // own cost up to this lane's run of sequences
    const int run = w.tiles_o == 0 ? 0 : (w.B + 31) / 32;
    const int b0 = min(lane * run, w.B), b1 = min(b0 + run, w.B);
    auto group_cost = [&](int b) { return w.cost_item + tiles_of(own_len(w, b)) * w.cost_o; };
    int mine = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) mine += groups * group_cost(b);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    const int own = __shfl_sync(0xffffffffu, upto, 31);
    const int before = upto - mine;
    if (lane == 0) sh.b_lo = sh.b_hi = w.B, sh.r_lo = sh.t_lo = sh.r_hi = sh.t_hi = sh.part_lo = 0;
    __syncwarp();

    // CTAs that take part: two narrow tiles each at least
    const int prefix = w.tiles_p > 0 ? w.rt_p * w.Hkv * (w.cost_item + w.tiles_p * w.cost_p) : 0;
    const int least = w.cost_item + 2 * w.cost_o;
    const int n = prefix + own >= least * w.sms ? w.sms : max((prefix + own) / least, 1);
    const int share = (prefix + own + n - 1) / n;
    // prefix: equal parts of at most a share
    int parts = 0, chunk = 0, items = 0, part_cost = 0;
    if (w.tiles_p > 0) {
        const int room = max(share - w.cost_item, w.cost_p);
        parts = min((w.tiles_p * w.cost_p + room - 1) / room, w.slots_p);
        chunk = (w.tiles_p + parts - 1) / parts;
        parts = (w.tiles_p + chunk - 1) / chunk;
        items = parts * w.rt_p * w.Hkv;
        part_cost = w.cost_item + chunk * w.cost_p;
    }
    // own: CTAs below `many` have one prefix part more than the others; each has
    // len_a or len_b of the own cost (rounded up: the last CTAs get what is left)
    const int each = items / n, many = items - each * n;
    const int least_o = w.min_o * w.cost_o;
    int room_a = share - (each + 1) * part_cost, room_b = share - each * part_cost;
    if (room_a < least_o || many == 0) room_a = 0;
    if (room_b < least_o) room_a = room_b = share;  // too little for its own CTAs: all take some
    const float fill = static_cast<float>(own) /
                       (static_cast<float>(many) * static_cast<float>(room_a) +
                        static_cast<float>(n - many) * static_cast<float>(room_b));
    const int len_a = room_a == 0 ? 0 : max(least_o, static_cast<int>(static_cast<float>(room_a) * fill) + 1);
    const int len_b = max(least_o, static_cast<int>(static_cast<float>(room_b) * fill) + 1);
    auto start = [&](int cta) { return cta < many ? cta * len_a : many * len_a + (cta - many) * len_b; };
    const int cta = blockIdx.x;
    const int lo = cta < n ? min(start(cta), own) : own;
    const int hi = cta < n - 1 ? min(start(cta + 1), own) : own;
    if (lane == 0) {
        sh.parts_p = parts, sh.chunk_p = chunk, sh.items_p = items, sh.ctas = n;
        if (cta == 0) w.parts[0] = parts;
    }
    // the tile at or behind a cost: by the lane whose sequences hold it
    if ((lo >= before && lo < upto) || (hi >= before && hi < upto)) {
        int at = before;
        for (int b = b0; b < b1; ++b) {
            const int g = group_cost(b), all = g * groups;
#pragma unroll 1
            for (int end = 0; end < 2; ++end) {
                const int x = (end ? hi : lo) - at;
                if (x < 0 || x >= all) continue;
                const int r = x / g, off = x - r * g - w.cost_item;
                const int tile = off <= 0 ? 0 : (off + w.cost_o - 1) / w.cost_o;
                if (end) {
                    sh.b_hi = b, sh.r_hi = r, sh.t_hi = tile;
                } else {
                    sh.b_lo = b, sh.r_lo = r, sh.t_lo = tile;
                    if (tile > 0) {
                        const int first = at + r * g + w.cost_item;  // its first tile
                        const int of = first < many * len_a ? first / len_a : many + (first - many * len_a) / len_b;
                        sh.part_lo = min(cta - min(of, n - 1), w.slots_o - 1);
                    }
                }
            }
            at += all;
        }
    }
    __syncwarp();
}

// The items of this CTA, one after the other.
struct Walk {
    int idx, b, r, tiles, len;

    // Key tiles t0 .. t1 - 1 of group r of sequence b.
    __device__ void own_item(const Work &w, Item &it, int t0, int t1) const {
        it.h = r / w.rt_o;
        const int rt = r - it.h * w.rt_o;
        it.b = b;
        it.flags = (w.wide_o ? kWide : w.tok_o * w.G <= kFewRows ? kFew : 0) | (w.causal ? kCausal : 0);
        it.tok = w.tok_o;
        const int first = b * w.Lq, rows = it.tok * (w.wide_o ? 2 : 1);
        it.tok0 = first + rt * rows;
        it.tok_end = min(first + w.Lq, it.tok0 + rows);
        it.lim0 = w.causal ? len - w.Lq + 1 - first : len;
        it.key0 = t0 * kKeys;
        const int last = min(len, limit_of(it, it.tok_end - 1));
        it.nkeys = max(0, min(t1 * kKeys, last) - it.key0);
        it.own_parts = 0;
    }
    // Part `part` of the prefix, `chunk` tiles, for row item rt of key head h.
    __device__ void prefix_item(const Work &w, Item &it, int rt, int h, int part, int chunk) const {
        it.b = -1;
        it.h = h;
        it.flags = w.wide_p ? kWide : w.tok_p * w.G <= kFewRows ? kFew : 0;
        it.tok = w.tok_p;
        const int rows = it.tok * (w.wide_p ? 2 : 1);
        it.tok0 = rt * rows;
        it.tok_end = min(w.T, it.tok0 + rows);
        it.key0 = part * chunk * kKeys;
        it.nkeys = min(chunk * kKeys, w.prefix_len - it.key0);
        it.lim0 = w.prefix_len;
        it.slot = part;
        it.own_parts = 0;
    }

    __device__ bool next_fixed(const Work &w, Item &it) {
        const int items_p = w.rt_p * w.Hkv * w.parts_p, groups = w.Hkv * w.rt_o;
        const int items_o = groups * w.B * w.parts_o;
        while (idx < items_p + items_o) {
            int i = idx;
            idx += gridDim.x;
            if (i < items_p) {
                const int hc = i / w.rt_p, h = hc / w.parts_p;
                prefix_item(w, it, i - hc * w.rt_p, h, hc - h * w.parts_p, w.chunk_p);
                return true;
            }
            i -= items_p;
            const int bc = i / groups, part = bc / w.B;
            r = i - bc * groups;
            b = bc - part * w.B;
            len = own_len(w, b);
            tiles = tiles_of(len);
            const int t0 = part * w.chunk_o, t1 = min(t0 + w.chunk_o, tiles);
            // a chunk past its end; one without keys is an item where there is
            // nothing else of its rows
            if (t0 >= tiles && (t0 > 0 || w.tiles_p > 0)) continue;
            own_item(w, it, t0, t1);
            if (w.tiles_p == 0 && tiles <= w.chunk_o) it.flags |= kWhole;
            it.slot = w.slots_p + part;
            return true;
        }
        return false;
    }

    __device__ bool next_share(const Work &w, const Share &sh, Item &it) {
        if (idx < sh.items_p && static_cast<int>(blockIdx.x) < sh.ctas) {
            const int hc = idx / w.rt_p, h = hc / sh.parts_p;
            prefix_item(w, it, idx - hc * w.rt_p, h, hc - h * sh.parts_p, sh.chunk_p);
            idx += sh.ctas;
            return true;
        }
        const int groups = w.Hkv * w.rt_o;
        while (b < sh.b_hi || (b == sh.b_hi && (r < sh.r_hi || (r == sh.r_hi && sh.t_hi > 0)))) {
            if (tiles < 0) {
                len = own_len(w, b);
                tiles = tiles_of(len);
            }
            const bool first = b == sh.b_lo && r == sh.r_lo;
            const bool end = b == sh.b_hi && r == sh.r_hi;
            const int t0 = first ? sh.t_lo : 0, t1 = end ? min(sh.t_hi, tiles) : tiles;
            const bool some = t0 < t1;
            if (some) {
                const int part = first ? sh.part_lo : 0;
                own_item(w, it, t0, t1);
                if (w.tiles_p == 0 && t0 == 0 && t1 == tiles) it.flags |= kWhole;
                it.slot = w.slots_p + part;
                it.own_parts = t1 == tiles ? part + 1 : 0;
            }
            if (tiles == 0) r = groups - 1;  // none of its groups has any
            if (++r == groups) ++b, r = 0, tiles = -1;
            if (some) return true;
        }
        return false;
    }
};

// Whole rows of a wide item: stored through the ring, beside the next item's first
// tiles (2 x 4096 x 333 x 32 heads of 128: 43.3 us from registers, 41.2 so; 2 x 8192 x
// 4093: 427, 420; of one tile, of more than two alike).
__device__ __forceinline__ bool staged(int flags, int ntiles) {
    return (flags & (kWide | kWhole)) == (kWide | kWhole) && ntiles > 0;
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

// FEW: has the code for items of few rows.  LATER: for values that are not finite
// among keys that only later query tokens of an item see (causal calls of more
// than one query token; cross attention over 4093 keys would take 454 us with it
// instead of 443, over 333 41.9 instead of 39.8).
template <int D, bool FEW, bool LATER>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap qmap_p, const __grid_constant__ CUtensorMap qmap_o,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ CUtensorMap omap, const __grid_constant__ Work w) {
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
    // the same rows' warps of both streams are at the end of a narrow item
    auto met = [&](int q) { return bars_s + 8u * (2 * NS + 14 + q); };
    constexpr int kFewBars = 2 * NS + 18, kItemBars = kFewBars + (FEW ? 3 : 2 * kItems);
    // of items of few rows: all softmax warps are at the end, and done with a
    // query buffer that they have used for its results
    const uint32_t met_all = bars_s + 8u * kFewBars;
    auto few_free = [&](int i) { return bars_s + 8u * (kFewBars + 1 + i); };
    // of others: a stream's result is in the ring, a barrier for each place of an
    // item.  The softmax warps never wait for the walking warp, which may be items
    // behind while there are free places for K, V and results.  But the walking
    // warp hands an item's place out again only after it has waited here for what
    // was in it, so that no phase can pass unseen.
    auto staged_full = [&](int st, uint32_t i) { return bars_s + 8u * (kFewBars + st * kItems + i); };
    auto item_full = [&](int i) { return bars_s + 8u * (kItemBars + i); };
    auto item_empty = [&](int i) { return bars_s + 8u * (kItemBars + kItems + i); };
    const uint32_t done_bar = bars_s + 8u * (kItemBars + 2 * kItems);
    // V has arrived that the walking warp looks through before it is full
    auto v_raw = [&](int s) { return bars_s + 8u * (kItemBars + 2 * kItems + 1 + s); };
    constexpr int kBars = kItemBars + 2 * kItems + 1 + NS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    Share &share = *reinterpret_cast<Share *>(tmem_slot + 2);
    Item *const ring = reinterpret_cast<Item *>(&share + 1);
    // Values that are not finite among keys that some rows of an item do not see:
    // the first such key of each column of V, counted from seen_by_all; the item
    // (by its number among those with such keys), and how many warps have used it.
    uint8_t *const bad_key = reinterpret_cast<uint8_t *>(ring + kItems);
    volatile uint32_t *const bad_item = reinterpret_cast<volatile uint32_t *>(bad_key + D);
    volatile uint32_t *const bad_used = bad_item + 1;
    static_assert(8 * kBars + 8 + sizeof(Share) + kItems * sizeof(Item) + D + 8 <= C::kBarBytes);
    float2 *const xml = reinterpret_cast<float2 *>(smem + (2 + NS) * C::kTileBytes + C::kBarBytes);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform for the compiler too
    const int lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, w.status, w.timeout_ns};
    // waits that may last for an item, at 2 us a tile
    const WaitCtl item_ctl{abort_flag, w.status, w.timeout_ns + 2000ull * max(w.tiles_p, w.tiles_o)};

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
            mbar_init(v_raw(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1);
            if (FEW) mbar_init(few_free(i), 8);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i, 0), 4);
            mbar_init(p_full(i, 1), 4);
            mbar_init(o_full(i), 1);
            mbar_init(pv_issued(i), 1);
        }
        for (int q = 0; q < 4; ++q) mbar_init(met(q), 2);
        if (FEW) mbar_init(met_all, 8);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(item_full(i), 1);
            mbar_init(item_empty(i), kReaders);
            if (!FEW) {
                mbar_init(staged_full(0, i), 4);
                mbar_init(staged_full(1, i), 4);
            }
        }
        mbar_init(done_bar, 2);
        *abort_flag = 0;
        *bad_item = *bad_used = 0;
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
    pdl_wait();
    pdl_launch_dependents();  // the join may read the lengths before it waits
    if (blockIdx.x == 0 && w.lens) {
        for (int b = threadIdx.x; b < w.B; b += kThreads)
            if (w.lens[b] < 0 || w.lens[b] > w.max_len) atomicOr(w.status, kDeviceStatusIndex);
    }

    // The next item, in every lane of a reading warp; false after the last.
    uint32_t items = 0;
    auto next_item = [&](Item &it) {
        const uint32_t i = items % kItems;
        if (!__all_sync(0xffffffffu, mbar_wait_spin(item_full(i), (items / kItems) & 1, item_ctl))) return false;
        it = ring[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty(i));
        ++items;
        return it.nkeys != kEnd;
    };

    // Every role takes the same items and key tiles in the same order, with its
    // own counters: ring fills (K of a tile, then V; staged() ones' results), steps (S tiles; their parity
    // is the stream), narrow items (their parity is the query buffer).
    if (warp >= kTmaWarp) {
        setmaxnreg_dec<kOtherRegs>();  // by all four warps at once
        if (warp == kTmaWarp) {
            // ------------------------------------------------------------ TMA
            uint32_t seq = 0, nar = 0;
            Item it;
            uint32_t qpar = 0, qused = 0;  // bit i: parity of query buffer i's next use, used at all
            uint32_t fpar = 0, qfew = 0;   // bit i: parity of its next use for a few rows' results, if its last was one
            uint32_t raw = 0, rpar = 0;    // bit s: v_raw counts place s's last fill; parity of its next use
            bool ok = true;
            if (elect_one()) {
                tma_prefetch_desc(&qmap_p);
                tma_prefetch_desc(&qmap_o);
                tma_prefetch_desc(&kmap);
                tma_prefetch_desc(&vmap);
            }
            __syncwarp();
#pragma unroll 1
            while (ok && next_item(it)) {
                const int ntiles = tiles_of(it.nkeys);
                const bool wide = it.flags & kWide;
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
                        uint32_t full = kv_full(s);
                        if (LATER) {
                            raw &= ~(1u << s);
                            if (kv == 1 && seen_by_all(it) < j * kKeys + valid) {
                                full = v_raw(s);
                                raw |= 1u << s, rpar ^= 1u << s;
                            }
                        }
                        if (w.page_size > 0) {
                            if (elect_one())
                                mbar_arrive_expect_tx(full, npages * w.page_size * 128 * C::kHalves);
                            __syncwarp();
                            if (lane < npages) {
#pragma unroll 1
                            for (int hf = 0; hf < C::kHalves; ++hf)
                                    tma_load_2d(sKV(s) + hf * C::kHalfBytes + lane * w.page_size * 128, map, full, hf * 64,
                                                row);
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
                            for (int i = 0; i < (wide ? 2 : 1) && ok; ++i) {
                                const int buf = wide ? i : static_cast<int>(nar & 1);
                                ok = __all_sync(0xffffffffu, mbar_wait_spin(q_empty(buf), ((qpar >> buf) & 1) ^ 1, ctl));
                                if (!ok) break;
                                if (FEW && ((qfew >> buf) & 1)) {
                                    ok = __all_sync(0xffffffffu, mbar_wait_spin(few_free(buf), (fpar >> buf) & 1, ctl));
                                    if (!ok) break;
                                    fpar ^= 1u << buf;
                                }
                                qfew = it.flags & kFew ? qfew | 1u << buf : qfew & ~(1u << buf);
                                if (elect_one()) {
                                    // few rows: four times, 32 rows apart
                                    const int copies = FEW && (it.flags & kFew) ? 4 : 1;
                                    mbar_arrive_expect_tx(q_full(buf), copies * it.tok * w.G * 128 * C::kHalves);
#pragma unroll 1
                                    for (int c = 0; c < copies * C::kHalves; ++c) {
                                        const int hf = c % C::kHalves;
                                        tma_load_3d(sQ(buf) + hf * C::kHalfBytes + c / C::kHalves * (32 * 128), qm,
                                                    q_full(buf), hf * 64, it.h * w.G, it.tok0 + i * it.tok);
                                    }
                                }
                                __syncwarp();
                                qpar ^= 1u << buf;
                                qused |= 1u << buf;
                            }
                        }
                    }
                }
                if (!FEW && staged(it.flags, ntiles)) {
                    // two places for its results, nothing to load
#pragma unroll 1
                    for (int i = 0; i < 2 && ok; ++i, ++seq) {
                        const int s = seq % NS;
                        ok = __all_sync(0xffffffffu, mbar_wait_spin(kv_empty(s), ((seq / NS) & 1) ^ 1, ctl));
                        if (!ok) break;
                        if (LATER) raw &= ~(1u << s);
                        if (lane == 0) mbar_arrive(kv_full(s));
                        __syncwarp();
                    }
                }
                if (!wide && ntiles > 0) ++nar;
            }
            if (elect_one()) {
                // The last copies have landed before the CTA exits, also where a
                // wait of another warp runs out after this one is through.
                for (uint32_t q = seq > NS ? seq - NS : 0; q < seq; ++q) {
                    const int s = q % NS;
                    if (LATER && ((raw >> s) & 1))
                        mbar_wait_drain(v_raw(s), ((rpar >> s) & 1) ^ 1, w.timeout_ns, w.status);
                    else
                        mbar_wait_drain(kv_full(s), (q / NS) & 1, w.timeout_ns, w.status);
                }
                for (int i = 0; i < 2; ++i)
                    if ((qused >> i) & 1) mbar_wait_drain(q_full(i), ((qpar >> i) & 1) ^ 1, w.timeout_ns, w.status);
            }
            __syncwarp();
        } else if (warp == kWalkWarp) {
            // ------------------------------------------------------------ items
            if (w.chunk_o == 0) divide(w, share);
            Walk walk;
            walk.idx = blockIdx.x, walk.tiles = -1, walk.len = 0;
            walk.b = w.chunk_o > 0 ? 0 : share.b_lo, walk.r = w.chunk_o > 0 ? 0 : share.r_lo;
            // An item's staged results, when the softmax has put them into the
            // ring: out by TMA, which leaves rows past the sequence's queries
            // out, and the places back to the loader.
            uint32_t fills = 0, spar = 0;  // spar bit i: parity of the next staged item in place i
            auto store = [&](uint32_t place) {
                const Item &it = ring[place];
                const int ntiles = tiles_of(it.nkeys);
                fills += 2 * ntiles;
                if (!staged(it.flags, ntiles)) return true;
#pragma unroll 1
                for (int st = 0; st < 2; ++st, ++fills) {
                    const int s = fills % NS;
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait_spin(staged_full(st, place), (spar >> place) & 1, item_ctl)))
                        return false;
                    const int first = it.tok0 + st * it.tok;  // its first token
                    if (lane == 0) {
                        if (first < it.tok_end) {
#pragma unroll 1
                            for (int hf = 0; hf < C::kHalves; ++hf)
                                tma_store_4d(&omap, sKV(s) + hf * C::kHalfBytes, hf * 64, it.h * w.G, first - it.b * w.Lq,
                                             it.b);
                            bulk_commit();
                            bulk_wait_read();
                        }
                        mbar_arrive(kv_empty(s));
                    }
                    __syncwarp();
                }
                spar ^= 1u << place;
                return true;
            };
            // Keys that only later query tokens see: P is 0 in the rows of the others,
            // but 0 x NaN is not.  So those rows of V come by way of this warp: what
            // is not finite in them is set to 0, and its first key noted for each
            // column, for the softmax to mark the rows that do see it.  (A prompt of
            // 8192 x 32 / 8 heads of 128 takes 408 us, as without; 421 where the
            // issuer of P V looks.  Four of 1024, few tiles an item: 50, 45.5 without.)
            uint32_t partly = 0, bad_uses = 0;  // items with such keys, warps that have used notes or will
            uint32_t rpar = 0;                  // bit s: parity of v_raw(s)'s next use
            auto notes_free = [&] {
                const uint64_t t0 = globaltimer_ns();
                while (static_cast<int>(*bad_used - bad_uses) < 0) {
                    if (*abort_flag) break;
                    if (globaltimer_ns() - t0 > item_ctl.timeout_ns) {
                        *abort_flag = 1;
                        atomicOr(w.status, kDeviceStatusTimeout);
                    }
                    __nanosleep(200);
                }
                __threadfence_block();
                return __all_sync(0xffffffffu, *abort_flag == 0) != 0;
            };
            auto set_aside = [&](uint8_t *v, int lo, int hi, int key) {
#pragma unroll 1
                for (int d = lane; d < D; d += 32) {
#pragma unroll 1
                    for (int r = lo; r < hi; ++r) {
                        uint16_t *x = reinterpret_cast<uint16_t *>(v + d / 64 * C::kHalfBytes + r * 128 +
                                                                   ((d % 64 / 8) ^ (r & 7)) * 16 + d % 8 * 2);
                        if (!not_finite(*x)) continue;
                        *x = 0;
                        if (bad_key[d] == kNoneBad) bad_key[d] = static_cast<uint8_t>(key + r);
                    }
                }
                fence_proxy_async_smem();
            };
            auto look = [&](uint32_t place) {
                const Item &it = ring[place];
                const int all_see = seen_by_all(it), ntiles = tiles_of(it.nkeys);
                if (all_see >= it.nkeys) return true;
                ++partly;
#pragma unroll 1
                for (int j = max(all_see, 0) / kKeys; j < ntiles; ++j) {
                    const int s = (fills + 2 * j + 1) % NS;
                    if (!__all_sync(0xffffffffu, mbar_wait_spin(v_raw(s), (rpar >> s) & 1, item_ctl))) return false;
                    rpar ^= 1u << s;
                    uint8_t *const v = smem + (2 + s) * C::kTileBytes;
                    const int lo = max(all_see - j * kKeys, 0), hi = min(kKeys, it.nkeys - j * kKeys);
                    uint32_t top[4] = {0, 0, 0, 0};
#pragma unroll 1
                    for (int hf = 0; hf < C::kHalves; ++hf) {
#pragma unroll 4
                        for (int i = lane; i < (hi - lo) * 8; i += 32) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(v + hf * C::kHalfBytes + lo * 128 + i * 16);
                            top[0] = abs_max(top[0], x.x), top[1] = abs_max(top[1], x.y);
                            top[2] = abs_max(top[2], x.z), top[3] = abs_max(top[3], x.w);
                        }
                    }
                    const bool bad = not_finite(top[0]) | not_finite(top[1]) | not_finite(top[2]) | not_finite(top[3]);
                    if (__any_sync(0xffffffffu, bad)) {
                        if (*bad_item != partly) {
                            if (!notes_free()) return false;
                            for (int d = lane; d < D; d += 32) bad_key[d] = kNoneBad;
                            const bool alone = !(it.flags & kWide) && ntiles == 1 && !(FEW && (it.flags & kFew));
                            bad_uses += alone ? 4 : 8;
                            __syncwarp();
                            if (lane == 0) *bad_item = partly;
                        }
                        set_aside(v, lo, hi, j * kKeys - all_see);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(kv_full(s));
                }
                return true;
            };
            bool more = true, ok = true;
            uint32_t n = 0, sent = 0;  // items in the ring so far, looked after by look() and store()
            auto look_after = [&] {
                const uint32_t place = sent++ % kItems;
                return (!LATER || look(place)) && store(place);
            };
#pragma unroll 1
            for (; more; ++n) {
                Item it;
                more = w.chunk_o > 0 ? walk.next_fixed(w, it) : walk.next_share(w, share, it);
                if (!more) it = Item{}, it.nkeys = kEnd;
                const uint32_t i = n % kItems;
                ok = __all_sync(0xffffffffu, mbar_wait_spin(item_empty(i), ((n / kItems) & 1) ^ 1, item_ctl));
                if (!ok) break;
                if (lane == 0) {
                    ring[i] = it;
                    mbar_arrive(item_full(i));
                }
                __syncwarp();
                if ((!FEW || LATER) && n - sent == kItems - 1) ok = look_after();  // the oldest in the ring
                if (!ok) break;
            }
            if (!FEW || LATER) {
                while (ok && sent < n) ok = look_after();
                if (lane == 0) bulk_wait();
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
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, D, true);
            constexpr uint32_t tile_desc = C::kTileBytes / 16;
            const bool is_qk = warp == kQkWarp;
            const uint64_t qd0 = sdesc_kmajor_sw128(sQ(0));
            const uint64_t kd0 = sdesc_kmajor_sw128(sKV(0));
            const uint64_t vd0 = sdesc_mnmajor_sw128(sKV(0), C::kHalfBytes);
            bool ok = true;
            Item it;
            int step = 0, nar = 0;
            int slot = is_qk ? 0 : 1;  // ring position of the tile's K / V
            uint32_t par = 0;          // its parity
            uint32_t qpar = 0;         // bit i: parity of query buffer i
            uint32_t spar = 0;         // bit i: parity of stream i: QK: its P V issued; PV: its P
#pragma unroll 1
            while (ok && next_item(it)) {
                const int nkeys = __shfl_sync(0xffffffffu, it.nkeys, 0);
                const int flags = __shfl_sync(0xffffffffu, it.flags, 0);
                const bool wide = flags & kWide;
                const int ntiles = tiles_of(nkeys);
                const int subs = wide ? 2 : 1;
#pragma unroll 1
                for (int j = 0; j < ntiles && ok; ++j) {
                    ok = __all_sync(0xffffffffu, mbar_wait_spin(kv_full(slot), par, ctl));
                    if (!ok) break;
                    const int valid = min(kKeys, nkeys - j * kKeys);
                    const uint64_t kvd = (is_qk ? kd0 : vd0) + static_cast<uint32_t>(slot) * tile_desc;
                    if (is_qk) {
                        // no more columns of S than there are keys
                        const uint32_t idesc_qk = idesc_bf16_f32(kRows, (valid + 15) & ~15, false);
#pragma unroll 1
                        for (int sub = 0; sub < subs; ++sub, ++step) {
                            const int st = step & 1;
                            const int buf = wide ? st : nar & 1;
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
                            const bool first = wide ? j == 0 : j < 2;
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
                if (!FEW && staged(flags, ntiles)) {
                    slot += 2;
                    if (slot >= NS) slot -= NS, par ^= 1;
                }
                if (!wide && ntiles > 0) ++nar;
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
        uint32_t step = 0, cnt = 0, meets = 0, all_meets = 0, nar = 0;
        uint32_t fills = 0;
        bool ok = true;
        // both warps of these rows have got here (a bounded wait, unlike bar.sync)
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(met(warp & 3));
            return __all_sync(0xffffffffu, mbar_wait_spin(met(warp & 3), meets++ & 1, ctl)) != 0;
        };
        auto meet_all = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(met_all);
            return __all_sync(0xffffffffu, mbar_wait_spin(met_all, all_meets++ & 1, ctl)) != 0;
        };
        // O scaled where a row's maximum has grown past the threshold; f: by how much
        auto rescale = [&](float f) {
            if (!__all_sync(0xffffffffu, mbar_wait_spin(o_full(st), (cnt - 1) & 1, ctl))) return false;
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
            return true;
        };
        auto arrive = [&](int half) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(st, half));
        };
        uint32_t partly = 0;
        // Has the item keys that not all rows see?  Then what was noted of them
        // before the stream's last product becomes visible here.
        auto notes = [&](const Item &i, int tiles) {
            if (!LATER || seen_by_all(i) >= i.nkeys || tiles == 0) return true;
            return __all_sync(0xffffffffu, mbar_wait_spin(pv_issued(st), (cnt - 1) & 1, ctl)) != 0;
        };
        auto any_bad = [&](const Item &i) { return LATER && seen_by_all(i) < i.nkeys && *bad_item == partly; };
        // NaN in O where the row sees a noted key; it sees as many as it has tokens
        // of the item before it
        auto mark = [&](int sees, bool has) {
            if (has) {
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(to + 16u * q, o);
                    tmem_wait_ld16(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (sees > bad_key[16 * q + i]) o[i] = 0x7fffffffu;
                    tmem_st_32x32b_x16(to + 16u * q, o);
                }
                tmem_wait_st();
            }
            __threadfence_block();
            __syncwarp();
            if (lane == 0) atomicAdd(const_cast<uint32_t *>(bad_used), 1u);
        };
        const int quarter = warp & 3;
        // of an item of few rows (lanes from kFewRows on help at its end only)
        const int few_row = lane % kFewRows, few_tok = few_row / w.G, few_g = few_row - few_tok * w.G;
        Item it;
#pragma unroll 1
        while (ok && next_item(it)) {
            const int ntiles = tiles_of(it.nkeys);
            const bool wide = it.flags & kWide;
            const int buf = nar & 1;
            if (!wide && ntiles > 0) ++nar;
            if (LATER && seen_by_all(it) < it.nkeys) ++partly;
            if (FEW && (it.flags & kFew) && ntiles > 0) {
                // A few rows would leave all but one of a stream's warps idle: they
                // are in the tile four times, 32 rows apart, and each warp takes a
                // quarter of a tile's keys, with maxima and sums of its own; P of
                // the other keys is 0 in its rows.  A tile's softmax is a quarter as
                // long, and K and V stay in the ring for as much less.
                const int tok = it.tok0 + few_tok;
                const bool row_live = few_tok < it.tok && tok < it.tok_end;
                const bool live = row_live && lane < kFewRows;
                const int limit = limit_of(it, tok) - it.key0 - 32 * quarter;
                float mref = -INFINITY, l = 0.f;
                int done = 0;
#pragma unroll 1
                for (int j = 0; j < ntiles; ++j) {
                    if (static_cast<int>(step++ & 1) != st) continue;
                    ok = __all_sync(0xffffffffu, mbar_wait_spin(s_full(st), cnt & 1, ctl));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const int key = j * kKeys;
                    const int vis = live ? min(limit - key, it.nkeys - key - 32 * quarter) : 32;
                    uint32_t x[32];
                    tmem_ld_32x32b_x32(ts + 32u * quarter, x);
                    const bool masked = __any_sync(0xffffffffu, vis < 32);
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    tmem_wait_ld(x);
                    row_max<0>(x, masked, vis, mx);
                    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (done == 0) {
                        mref = mt;
                    } else {
                        const float m_new = fmaxf(mref, mt);
                        const bool grow = live && (m_new - mref) * c > kRescaleLog2;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = grow ? ex2((mref - m_new) * c) : 1.f;
                            ok = rescale(f);
                            if (!ok) break;
                            l *= f;
                            if (grow) mref = m_new;
                        }
                    }
                    const float mc = mref == -INFINITY ? 0.f : mref * c;
                    uint64_t sum[2] = {0, 0};
                    weights(x, c, mc, sum, ts + 16u * quarter);
                    uint32_t zero[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) zero[i] = 0;
#pragma unroll
                    for (int q = 1; q < 4; ++q) tmem_st_32x32b_x16(ts + 16u * ((quarter + q) & 3), zero);
                    float a, b;
                    f32x2_split(add_f32x2(sum[0], sum[1]), a, b);
                    l += a + b;
                    tmem_wait_st();
                    arrive(0);
                    arrive(1);
                    ++cnt;
                    ++done;
                }
                if (!ok) break;
                if (done > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait_spin(o_full(st), (cnt - 1) & 1, ctl)) && notes(it, done);
                    if (!ok) break;
                }
                // The result: eight parts of a row, by stream and quarter.  Each
                // warp adds up its quarter's two streams for half of the columns
                // and puts them where the item's queries were, which are not
                // needed any more; then it adds up the quarters for an eighth of
                // the columns, two lanes a row, and stores them.
                tc_fence_before_sync();
                xml[st * kRows + 32 * quarter + lane] = make_float2(mref == -INFINITY ? mref : mref * c, l);
                ok = meet_all();
                if (!ok) break;
                tc_fence_after_sync();
                if (__builtin_expect(any_bad(it), 0)) {
                    mark(tok - it.tok0, done > 0);
                    tc_fence_before_sync();
                    ok = meet_all();
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                const bool part = !(it.flags & kWhole);
                float *const scratch = reinterpret_cast<float *>(smem + buf * C::kTileBytes);
                float m = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 o = xml[32 * i + few_row];
                    if (o.y != 0.f) m = fmaxf(m, o.x);
                }
                float f0 = 0.f, f1 = 0.f;  // of this quarter's streams
                l = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 o = xml[32 * i + few_row];
                    const float fi = o.y != 0.f ? ex2(o.x - m) : 0.f;
                    l += fi * o.y;
                    if (i == quarter) f0 = fi;
                    if (i == 4 + quarter) f1 = fi;
                }
#pragma unroll 1
                for (int col = st * (D / 2); col < (st + 1) * (D / 2); col += 32) {
                    uint32_t o[32], p[32];
                    float v[32];
                    tmem_ld_32x32b_x32(tO(0) + lanes + static_cast<uint32_t>(col), o);
                    tmem_ld_32x32b_x32(tO(1) + lanes + static_cast<uint32_t>(col), p);
                    tmem_wait_ld(o);
                    tmem_wait_ld(p);
                    // a stream without a weight may hold what it likes
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        v[i] = f0 != 0.f ? __uint_as_float(o[i]) * f0 : 0.f;
                        if (f1 != 0.f) v[i] = fmaf(__uint_as_float(p[i]), f1, v[i]);
                    }
                    if (lane < kFewRows) {
                        // pieces of 16 bytes, turned by the row against bank conflicts
                        float4 *dst = reinterpret_cast<float4 *>(scratch + (quarter * kFewRows + lane) * D + col);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dst[i ^ (lane & 7)] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
                tc_fence_before_sync();
                fence_proxy_async_smem();
                ok = meet_all();
                if (!ok) break;
                const int Hq_row = it.h * w.G + few_g;
                const int64_t pr = part ? it.slot * rows + static_cast<int64_t>(tok) * Hq + Hq_row : 0;
                if (part && live && warp == 0) w.part_ml[pr] = make_float2(m, l);
                if (it.own_parts > 0 && threadIdx.x == 0)
                    w.parts[1 + (it.b * w.Hkv + it.h) * w.rt_o + (it.tok0 - it.b * w.Lq) / it.tok] = it.own_parts;
                if (row_live) {
                    // D / 8 columns of this warp, half of them of this lane
                    constexpr int kPieces = D / 64;
                    const int piece0 = (st * (D / 2) + quarter * (D / 8)) / 4 + (lane >> 4) * kPieces;
                    const float inv = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
                    float4 sum4[kPieces];
#pragma unroll
                    for (int k = 0; k < kPieces; ++k) {
                        sum4[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        const int piece = piece0 + k;
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            const float4 x = reinterpret_cast<const float4 *>(
                                scratch + (o * kFewRows + few_row) * D)[(piece & ~7) + ((piece & 7) ^ (few_row & 7))];
                            sum4[k].x += x.x, sum4[k].y += x.y, sum4[k].z += x.z, sum4[k].w += x.w;
                        }
                        if (part) {
                            reinterpret_cast<float4 *>(w.part_o + pr * D)[piece] = sum4[k];
                        } else {
                            uint2 *dst = reinterpret_cast<uint2 *>(w.out + tok * w.ldo + static_cast<int64_t>(Hq_row) * D);
                            dst[piece] = make_uint2(pack2(sum4[k].x * inv, sum4[k].y * inv),
                                                    pack2(sum4[k].z * inv, sum4[k].w * inv));
                        }
                    }
                }
                // every warp has read its sums before the next queries come
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(few_free(buf));
                continue;
            }
            const int tok = it.tok0 + (wide ? st * it.tok : 0) + row_tok;
            const bool live = row_tok < it.tok && tok < it.tok_end;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int limit = limit_of(it, tok);
            float mref = -INFINITY, l = 0.f;
            int done = 0;  // tiles of this stream
            for (int j = 0; j < ntiles; ++j) {
                if (!wide) {
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
                if (warp_live) {
                    // rows of no query hold what they like: not worth a mask
                    const int vis = live ? min(max(limit - it.key0 - key, 0), valid) : kKeys;
                    tmem_ld_32x32b_x32(ts, sr[0]);
                    tmem_ld_32x32b_x32(ts + 32u, sr[1]);
                    tmem_ld_32x32b_x32(ts + 64u, sr[2]);
                    tmem_ld_32x32b_x32(ts + 96u, sr[3]);
                    const int all_see = __reduce_min_sync(0xffffffffu, vis);
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    tmem_wait_ld(sr[0]);
                    tmem_wait_ld(sr[1]);
                    tmem_wait_ld(sr[2]);
                    tmem_wait_ld(sr[3]);
                    row_max<0>(sr[0], all_see < 32, vis, mx);
                    row_max<1>(sr[1], all_see < 64, vis, mx);
                    row_max<2>(sr[2], all_see < 96, vis, mx);
                    row_max<3>(sr[3], all_see < 128, vis, mx);
                    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (done == 0) {
                        mref = mt;
                    } else {
                        const float m_new = fmaxf(mref, mt);
                        const bool grow = (m_new - mref) * c > kRescaleLog2;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = grow ? ex2((mref - m_new) * c) : 1.f;
                            ok = rescale(f);
                            if (!ok) break;
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
                if (warp_live && valid > kFirstKeys) {  // else no product reads them
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
            if (wide) step += 2 * ntiles;
            fills += 2 * ntiles;
            // The item's result.  A wide item's rows are this stream's own.  A
            // narrow one's are both streams': each adds up one half of the
            // columns of the two accumulators, as a join of two parts would.
            if (done > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait_spin(o_full(st), (cnt - 1) & 1, ctl)) && notes(it, done);
                if (!ok) break;
                if (__builtin_expect((wide || ntiles == 1) && any_bad(it), 0)) {
                    tc_fence_after_sync();
                    mark(tok - it.tok0, warp_live);
                }
            }
            if (it.own_parts > 0 && !w.direct && threadIdx.x == 0)
                w.parts[1 + (it.b * w.Hkv + it.h) * w.rt_o + (it.tok0 - it.b * w.Lq) / (it.tok * (wide ? 2 : 1))] =
                    it.own_parts;
            if (!FEW && staged(it.flags, ntiles)) {
                // Finished rows go to a place of the ring that the loader has
                // passed over, laid out as the query tile; the walking warp
                // sends them out.
                const int s = (fills + st) % NS;
                ok = __all_sync(0xffffffffu, mbar_wait_spin(kv_full(s), ((fills + st) / NS) & 1, ctl));
                if (!ok) break;
                fills += 2;
                tc_fence_after_sync();
                if (warp_live) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    uint8_t *dst = smem + (2 + s) * C::kTileBytes + row * 128;
#pragma unroll 1
                    for (int hf = 0; hf < C::kHalves; ++hf, dst += C::kHalfBytes) {
                        uint32_t o[2][32];
                        tmem_ld_32x32b_x32(to + 64u * hf, o[0]);
                        tmem_ld_32x32b_x32(to + 64u * hf + 32u, o[1]);
                        tmem_wait_ld(o[0]);
                        tmem_wait_ld(o[1]);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t p[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                p[i] = inv != 0.f ? pack2(__uint_as_float(o[q][2 * i]) * inv,
                                                          __uint_as_float(o[q][2 * i + 1]) * inv)
                                                  : 0u;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                *reinterpret_cast<uint4 *>(dst + ((q * 4 + k) ^ (row & 7)) * 16) =
                                    make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(staged_full(st, (items - 1) % kItems));
                continue;
            }
            float m = mref == -INFINITY ? mref : mref * c;
            float f_mine = 1.f, f_other = 0.f;
            bool other = false;
            if (!wide && ntiles > 1) {
                tc_fence_before_sync();
                xml[st * kRows + row] = make_float2(m, l);
                ok = meet();
                if (!ok) break;
                if (__builtin_expect(any_bad(it), 0)) {
                    tc_fence_after_sync();
                    mark(tok - it.tok0, warp_live);
                    tc_fence_before_sync();
                    ok = meet();
                    if (!ok) break;
                }
                const float2 o = xml[(1 - st) * kRows + row];
                const float top = fmaxf(l != 0.f ? m : -INFINITY, o.y != 0.f ? o.x : -INFINITY);
                f_mine = l != 0.f ? ex2(m - top) : 0.f;
                f_other = o.y != 0.f ? ex2(o.x - top) : 0.f;
                l = f_mine * l + f_other * o.y;
                m = top;
                other = true;
            }
            tc_fence_after_sync();
            const bool part = !(it.flags & kWhole);
            // columns of this stream; a narrow item of one tile is its stream's alone
            const int col0 = other ? st * (D / 2) : 0, col1 = other ? col0 + D / 2 : (wide || done > 0 ? D : 0);
            const bool reports = wide || (ntiles > 0 ? (other ? st == 0 : done > 0) : st == 0);
            if (warp_live) {
                // Stored through a 4 x 4 transpose of 16-byte pieces within each
                // quad of lanes: an instruction then writes 64 bytes of 8 rows
                // instead of 16 bytes of 32.  A few rows are not worth it.
                const int64_t at = static_cast<int64_t>(tok) * Hq + it.h * w.G + row_g;
                const int64_t pr = part ? it.slot * rows + at : 0;
                if (part && live && reports) w.part_ml[pr] = make_float2(m, l);
                const bool empty = ntiles == 0;  // zeros, if written at all
                const float inv = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
                f_mine *= inv, f_other *= inv;
                const bool use_mine = f_mine != 0.f, use_other = f_other != 0.f;
                // in 16-byte units; the rows of this lane's quad
                const int64_t mine = part ? pr * (D / 4) : (tok * w.ldo + static_cast<int64_t>(it.h * w.G + row_g) * D) / 8;
                uint4 *const dst = part ? reinterpret_cast<uint4 *>(w.part_o) : reinterpret_cast<uint4 *>(w.out);
                const int qi = lane & 3;
                int64_t off[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) off[k] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + k) + qi;
                const uint32_t lives = __ballot_sync(0xffffffffu, live), on = lives >> (lane & ~3);
                const bool few = __popc(lives) <= 8;
                auto put = [&](uint32_t (&p)[16], int piece) {
                    if (few) {
                        if (live) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                dst[mine + 4 * piece + k] = make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
                        }
                        return;
                    }
                    ep::quad_transpose(p, qi);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if ((on >> k) & 1)
                            dst[off[k] + 4 * piece] = make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
                };
                if (!part && !other && !empty && col1 > 0) {
                    // all columns of a finished row at once
                    uint32_t o[D / 32][32];
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) tmem_ld_32x32b_x32(to + 32u * q, o[q]);
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) tmem_wait_ld(o[q]);
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            p[i] = use_mine ? pack2(__uint_as_float(o[q][2 * i]) * f_mine,
                                                    __uint_as_float(o[q][2 * i + 1]) * f_mine)
                                            : 0u;
                        put(p, q);
                    }
                } else {
                    const int last = empty ? (part || !(wide || st == 0) ? 0 : D) : col1;
#pragma unroll 1
                    for (int col = col0; col < last; col += 32) {
                        uint32_t o[32];
                        if (empty) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = 0;
                        } else {
                            tmem_ld_32x32b_x32(to + static_cast<uint32_t>(col), o);
                            uint32_t p[32];
                            if (other) tmem_ld_32x32b_x32(tO(1 - st) + lanes + static_cast<uint32_t>(col), p);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = use_mine ? __float_as_uint(__uint_as_float(o[i]) * f_mine) : 0u;
                            if (other) {
                                tmem_wait_ld(p);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (use_other)
                                        o[i] = __float_as_uint(fmaf(__uint_as_float(p[i]), f_other, __uint_as_float(o[i])));
                            }
                        }
                        uint32_t p[16];
                        if (part) {
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) p[i] = o[16 * g + i];
                                put(p, col / 16 + g);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                p[i] = pack2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                            put(p, col / 32);
                        }
                    }
                }
            }
            if (other) {
                // the next item's products and maxima come after the other
                // stream has read this one's
                tc_fence_before_sync();
                ok = meet();
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
// results (M their largest m): the parts against the prefix, then the own ones;
// a warp per row.  Parts with l = 0 saw no key and may have no o.
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ Work w) {
    pdl_launch_dependents();
    const int Hq = w.Hkv * w.G;
    const int64_t rows = static_cast<int64_t>(w.T) * Hq;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int tok = static_cast<int>(row / Hq), hq = static_cast<int>(row - static_cast<int64_t>(tok) * Hq);
    const int b = tok / w.Lq, rt = (tok - b * w.Lq) / (w.tok_o * (w.wide_o ? 2 : 1));
    const int own = tiles_of(own_len(w, b));  // lengths are older than the kernel ahead
    const bool fixed = w.chunk_o > 0;
    pdl_wait();
    // Where a wait ran out in the kernel ahead a count may not have been written:
    // no more parts than have a place.
    const int np = fixed ? w.parts_p : w.tiles_p > 0 ? min(max(w.parts[0], 0), w.slots_p) : 0;
    const int no = fixed ? (own + w.chunk_o - 1) / w.chunk_o
                         : own > 0 ? min(max(w.parts[1 + (b * w.Hkv + hq / w.G) * w.rt_o + rt], 0), w.slots_o) : 0;
    if (np == 0 && no == 1) return;  // written by the item itself
    const int n = np + no;
    constexpr int E = D / 32, kAhead = 8;
    auto slot_of = [&](int s) { return (s < np ? s : w.slots_p + s - np) * rows + row; };
    float M = -INFINITY, L = 0.f, o[E] = {};
    for (int s0 = 0; s0 < n; s0 += 32) {
        // up to 32 parts: a lane each for their maxima and sums, and the first
        // results on their way before those are known
        const int here = min(32, n - s0);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < here) ml = w.part_ml[slot_of(s0 + lane)];
        float x[kAhead][E];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (i0 + k >= here) break;
                const float *src = w.part_o + slot_of(s0 + i0 + k) * D + lane * E;
                if constexpr (E == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(src);
                    x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
                } else {
                    const float2 v = *reinterpret_cast<const float2 *>(src);
                    x[k][0] = v.x, x[k][1] = v.y;
                }
            }
        };
        fetch(0);
        float top = ml.y != 0.f ? ml.x : -INFINITY;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        const float m_new = fmaxf(M, top);
        const float f = ml.y != 0.f ? ex2(ml.x - m_new) : 0.f;
        const float keep = L != 0.f ? ex2(M - m_new) : 0.f;
        float sum = f * ml.y;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
        L = L * keep + sum;
        M = m_new;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= keep;
        for (int i0 = 0; i0 < here; i0 += kAhead) {
            if (i0 > 0) fetch(i0);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (i0 + k >= here) break;
                const float fk = __shfl_sync(0xffffffffu, f, i0 + k);
                if (fk == 0.f) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(fk, x[k][e], o[e]);
            }
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint16_t *dst = w.out + tok * w.ldo + static_cast<int64_t>(hq) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(dst + e) = pack2(o[e] * inv, o[e + 1] * inv);
}

// Planned for this many SMs whatever the device has, so that the workspace is a
// function of the sizes alone.
constexpr int kPlanSms = 152;

int div_up(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

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
    w.tiles_p = div_up(w.prefix_len, kKeys), w.tiles_o = div_up(w.max_len, kKeys);
    w.sms = kPlanSms;
    const int64_t base_p = static_cast<int64_t>(w.rt_p) * w.Hkv, base_o = static_cast<int64_t>(w.rt_o) * w.Hkv * w.B;
    // Whole groups where there are more than SMs and their lengths are one, or
    // short enough that a long one among them costs less than partial results
    // and their join; of two tiles always (they run side by side in a narrow
    // group).  us, whole against shares: even, 2 x 4096 x 500 x 8 heads of 128 20
    // / 47, 2 x 4096 x 4000 x 14 140 / 186, 56 x 1 x 2000 x 8 70 / 80, 70 x 1 x
    // 4000 x 8 167 / 176; one query token, lengths drawn evenly to 1000: 128 x 8
    // heads 60 / 62, to 2000 97 / 92, to 4000 183 / 167, one 4000 among 250s 50 /
    // 35; 8 x 1024 x 8 heads to 2000 40 / 58, to 4000 71 / 85, one 4000 among
    // 250s 52 / 45.  Many wide groups level their lengths out, and a join passes
    // over all their rows.  The rule knows the longest length alone: at its bounds
    // (16 tiles narrow, 32 wide) it takes whole groups, which need no workspace,
    // also where shares were faster, by 5 % at the 97 / 92 and by 15 % with one
    // long sequence among short ones.
    const int64_t most = w.wide_o ? (base_o >= 4 * kPlanSms ? w.tiles_o : 32) : 16;
    w.direct = w.tiles_p == 0 && (w.tiles_o <= 2 || (base_o > kPlanSms && (!a.ragged || w.tiles_o <= most)));
    if (w.direct) {
        w.parts_o = 1, w.chunk_o = w.tiles_o > 0 ? w.tiles_o : 1;
        return w;
    }
    // Fixed chunks where every one has an SM of its own: the smallest of two tiles
    // or more for which that holds, if it is no more than four or the tiles there
    // may be keep half of the SMs busy.
    if (base_p * (w.tiles_p > 0) + base_o * (w.tiles_o > 0) <= kPlanSms) {
        auto items = [&](int64_t c) { return base_p * ((w.tiles_p + c - 1) / c) + base_o * ((w.tiles_o + c - 1) / c); };
        const int64_t all = base_p * w.tiles_p + base_o * w.tiles_o;
        // items(c) falls with c and is no more than SMs for whole groups
        int64_t c = all / kPlanSms > 2 ? all / kPlanSms : 2;
        for (int64_t hi = w.tiles_p > w.tiles_o ? w.tiles_p : w.tiles_o; c < hi;) {
            const int64_t mid = c + (hi - c) / 2;
            if (items(mid) > kPlanSms)
                c = mid + 1;
            else
                hi = mid;
        }
        if (c <= 4 || all >= c * kPlanSms / 2) {
            w.chunk_p = w.chunk_o = static_cast<int>(c);
            w.parts_p = w.slots_p = div_up(w.tiles_p, c);
            w.parts_o = w.slots_o = div_up(w.tiles_o, c);
            w.direct = w.tiles_p == 0 && w.parts_o == 1;  // every group whole after all: nothing to join
            return w;
        }
    }
    // costs in units that keep the sum of all below 2^30
    int shift = 0;
    auto sum = [&] {
        w.cost_p = (w.wide_p ? kWideTileCost : kTileCost) >> shift;
        w.cost_o = (w.wide_o ? kWideTileCost : kTileCost) >> shift;
        w.cost_item = kItemCost >> shift;
        return base_p * (w.cost_item + static_cast<int64_t>(w.tiles_p) * w.cost_p) +
               base_o * (w.cost_item + static_cast<int64_t>(w.tiles_o) * w.cost_o);
    };
    while (sum() >= kMostCost && shift < 4) ++shift;
    w.too_large = sum() >= kMostCost;
    // a group's parts: as many as CTAs can find work in, of two tiles at least;
    // own pieces of a sixteenth of the longest at least
    if (w.tiles_p > 0) {
        const int64_t most = kPlanSms / base_p + 1;
        w.slots_p = static_cast<int>(most < w.tiles_p ? most : w.tiles_p);
    }
    if (w.tiles_o > 0) {
        w.min_o = w.tiles_o > 32 ? div_up(w.tiles_o, 16) : 2;
        // a piece in the middle of a group is min_o tiles at least
        w.slots_o = (w.tiles_o - 1) / w.min_o + 2;
    } else {
        w.min_o = 1;
    }
    return w;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int64_t part_rows(const Work &w) {
    return static_cast<int64_t>(w.slots_p + w.slots_o) * w.T * w.Hkv * w.G;
}
size_t parts_bytes(const Work &w) {
    return round256((1 + static_cast<size_t>(w.B) * w.Hkv * w.rt_o) * sizeof(int));
}
size_t ml_bytes(const Work &w) { return round256(static_cast<size_t>(part_rows(w)) * sizeof(float2)); }

bool row_map(CUtensorMap *m, const AttentionArgs &a, int tokens) {
    const uint64_t dims[3] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.Hq),
                              static_cast<uint64_t>(a.B * a.Lq)};
    const uint64_t strides[2] = {static_cast<uint64_t>(a.D) * 2, static_cast<uint64_t>(a.ldq) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(tokens)};
    return tensor_map_bf16(m, a.q, 3, dims, strides, box);
}

// The same rows of the result, by sequence: a tile's rows past its queries are
// outside.
bool out_map(CUtensorMap *m, const AttentionArgs &a, int tokens) {
    const uint64_t ld = static_cast<uint64_t>(a.ldo) * 2;
    const uint64_t dims[4] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.Lq),
                              static_cast<uint64_t>(a.B)};
    const uint64_t strides[3] = {static_cast<uint64_t>(a.D) * 2, ld, ld * static_cast<uint64_t>(a.Lq)};
    const uint32_t box[4] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(tokens), 1};
    return tensor_map_bf16(m, a.out, 4, dims, strides, box);
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
    CUtensorMap qp, qo, km, vm, om;
    // maps of what the call reads; the others are never used
    if (!row_map(&qo, a, w.tok_o)) return cudaErrorInvalidValue;
    if (w.tiles_p == 0)
        qp = qo;
    else if (!row_map(&qp, a, w.tok_p))
        return cudaErrorInvalidValue;
    if (a.k && (a.pages > 0 || a.max_len > 0)) {
        if (!key_map(&km, a, a.k, a.ldk) || !key_map(&vm, a, a.v, a.ldv)) return cudaErrorInvalidValue;
    } else {
        km = vm = qo;  // no key at all
    }
    if (!w.wide_o)
        om = qo;
    else if (!out_map(&om, a, w.tok_o))
        return cudaErrorInvalidValue;
    // few rows against each sequence's own keys, and no wide items besides
    const bool few = !w.wide_o && w.tok_o * w.G <= kFewRows && (w.tiles_p == 0 || !w.wide_p);
    const bool later = w.causal && w.Lq > 1;
    auto kern = few ? (later ? attention_kernel<D, true, true> : attention_kernel<D, true, false>)
                    : (later ? attention_kernel<D, false, true> : attention_kernel<D, false, false>);
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
    // planned for kPlanSms; fewer SMs share the same work
    if (sms < w.sms) w.sms = sms;
    const int64_t groups = static_cast<int64_t>(w.rt_o) * w.Hkv * w.B;
    const int64_t most = w.chunk_o > 0 ? static_cast<int64_t>(w.rt_p) * w.Hkv * w.parts_p + groups * w.parts_o : sms;
    cfg.gridDim = dim3(static_cast<unsigned>(most < sms ? most : w.chunk_o > 0 ? sms : w.sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx.stream;
    cfg.attrs = attr;
    cfg.numAttrs = ctx.pdl ? 1 : 0;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, qp, qo, km, vm, om, w); e != cudaSuccess) return e;
    if (w.direct) return cudaSuccess;
    const int64_t rows = static_cast<int64_t>(w.T) * w.Hkv * w.G;
    cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<D>, w);
}

}  // namespace

size_t attention_workspace_bytes(const AttentionArgs &a) {
    const Work w = plan(a);
    if (w.too_large) return kAttentionTooLarge;
    if (w.direct) return 0;
    return parts_bytes(w) + ml_bytes(w) + static_cast<size_t>(part_rows(w)) * a.D * sizeof(float);
}

cudaError_t launch_attention(const AttentionArgs &a, const LaunchCtx &ctx) {
    Work w = plan(a);
    w.out = a.out, w.ldo = a.ldo;
    w.page_size = a.pages > 0 ? a.page_size : 0, w.pages = static_cast<int>(a.pages);
    w.prefix_pages = a.prefix_pages, w.block_table = a.block_table, w.lens = a.lens, w.table_stride = a.table_stride;
    w.scale_log2 = a.scale * kLog2e;
    if (!w.direct) {
        char *p = static_cast<char *>(a.ws);
        w.parts = reinterpret_cast<int *>(p);
        w.part_ml = reinterpret_cast<float2 *>(p + parts_bytes(w));
        w.part_o = reinterpret_cast<float *>(p + parts_bytes(w) + ml_bytes(w));
    }
    w.status = ctx.status;
    w.timeout_ns = ctx.timeout_ns;
    return a.D == 64 ? launch<64>(a, w, ctx) : launch<128>(a, w, ctx);
}

}  // namespace ck
