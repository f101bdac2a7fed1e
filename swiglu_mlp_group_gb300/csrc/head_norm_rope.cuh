// head_norm_rope.cuh -- RMS norm and position rotation of one attention head's
// row, held by a group of L neighbouring lanes of a warp, 8 elements a lane.
//
//   y[d] = x[d] * rsqrt(mean(x^2) + eps) * w[d]
//   (y[a], y[b]) -> (y[a] c[i] - y[b] s[i], y[b] c[i] + y[a] s[i])
// for the pairs (i, i + r/2) or (2i, 2i + 1).  A lane holds four whole pairs
// (A_j, B_j), so that no lane needs another's elements, and the weights and the
// token's factors are multiplied once for all heads of the token:
//   A' = f (A wA c - B wB s),  B' = f (B wB c + A wA s),  f = rsqrt(...)
// Everything is f32 between the bf16 loads and the one rounding of the store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"

namespace ck {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Which elements lane gl of a group holds.
//   interleaved: 8 gl .. 8 gl + 7 (pairs side by side).
//   half: 4 from `a`, 4 from `b`: a = 4 gl, b = r/2 + 4 gl while 4 gl < r/2;
//   the other lanes take the D - r elements that pass through, two runs of half
//   of them.
template <bool INTERLEAVED>
struct Place {
    int a, b;
    bool on;       // the lane holds elements at all
    bool rotated;  // and they are rotated
    __device__ Place(int gl, int D, int rot) {
        on = 8 * gl < D;
        if constexpr (INTERLEAVED) {
            a = 8 * gl, b = a + 4;
            rotated = a < rot;
        } else {
            rotated = 8 * gl < rot;
            a = rotated ? 4 * gl : rot + 4 * gl - rot / 2;
            b = rotated ? a + rot / 2 : a + (D - rot) / 2;
        }
        if (!on) a = b = 0;
    }
};

// A lane's 8 elements as they are stored: words 0, 1 from `a`, words 2, 3 from `b`.
template <bool INTERLEAVED>
__device__ __forceinline__ uint4 load_row(const uint16_t *row, const Place<INTERLEAVED> &p) {
    if constexpr (INTERLEAVED) {
        return *reinterpret_cast<const uint4 *>(row + p.a);
    } else {
        const uint2 a = *reinterpret_cast<const uint2 *>(row + p.a), b = *reinterpret_cast<const uint2 *>(row + p.b);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
}
template <bool INTERLEAVED>
__device__ __forceinline__ void store_row(uint16_t *row, const Place<INTERLEAVED> &p, const uint4 &v) {
    if constexpr (INTERLEAVED) {
        *reinterpret_cast<uint4 *>(row + p.a) = v;
    } else {
        *reinterpret_cast<uint2 *>(row + p.a) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2 *>(row + p.b) = make_uint2(v.z, v.w);
    }
}

// The four pairs of those words, as two-element vectors over the pairs:
// A = (A0, A1), (A2, A3), B likewise.
struct Pairs {
    uint64_t a[2], b[2];
};
template <bool INTERLEAVED>
__device__ __forceinline__ Pairs pairs_of(const uint4 &v) {
    Pairs p;
    if constexpr (INTERLEAVED) {
        p.a[0] = f32x2(bf16_lo(v.x), bf16_lo(v.y)), p.b[0] = f32x2(bf16_hi(v.x), bf16_hi(v.y));
        p.a[1] = f32x2(bf16_lo(v.z), bf16_lo(v.w)), p.b[1] = f32x2(bf16_hi(v.z), bf16_hi(v.w));
    } else {
        p.a[0] = f32x2(bf16_lo(v.x), bf16_hi(v.x)), p.a[1] = f32x2(bf16_lo(v.y), bf16_hi(v.y));
        p.b[0] = f32x2(bf16_lo(v.z), bf16_hi(v.z)), p.b[1] = f32x2(bf16_lo(v.w), bf16_hi(v.w));
    }
    return p;
}
template <bool INTERLEAVED>
__device__ __forceinline__ uint4 words_of(const Pairs &p) {
    float a[4], b[4];
    f32x2_split(p.a[0], a[0], a[1]), f32x2_split(p.a[1], a[2], a[3]);
    f32x2_split(p.b[0], b[0], b[1]), f32x2_split(p.b[1], b[2], b[3]);
    if constexpr (INTERLEAVED)
        return make_uint4(pack2(a[0], b[0]), pack2(a[1], b[1]), pack2(a[2], b[2]), pack2(a[3], b[3]));
    else
        return make_uint4(pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(b[0], b[1]), pack2(b[2], b[3]));
}

// A lane's norm weights (ones without).
template <bool INTERLEAVED>
__device__ __forceinline__ Pairs load_weights(const void *w, bool w_f32, const Place<INTERLEAVED> &p) {
    Pairs r;
    if (!w) {
        r.a[0] = r.a[1] = r.b[0] = r.b[1] = f32x2(1.f, 1.f);
    } else if (w_f32) {
        const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + p.a);
        const float4 y = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + p.b);
        if constexpr (INTERLEAVED) {
            r.a[0] = f32x2(x.x, x.z), r.b[0] = f32x2(x.y, x.w);
            r.a[1] = f32x2(y.x, y.z), r.b[1] = f32x2(y.y, y.w);
        } else {
            r.a[0] = f32x2(x.x, x.y), r.a[1] = f32x2(x.z, x.w);
            r.b[0] = f32x2(y.x, y.y), r.b[1] = f32x2(y.z, y.w);
        }
    } else {
        r = pairs_of<INTERLEAVED>(load_row<INTERLEAVED>(static_cast<const uint16_t *>(w), p));
    }
    return r;
}

// What a token's heads are multiplied with: wA c, -wB s, wB c, wA s (of a lane
// that is not rotated: wA, -, wB, -).
struct Factors {
    uint64_t ac[2], bs[2], bc[2], as[2];
};
__device__ __forceinline__ void set_factors(Factors &f, const Pairs &w, bool rotated, const float4 &c, const float4 &s) {
    const uint64_t cc[2] = {f32x2(c.x, c.y), f32x2(c.z, c.w)}, ss[2] = {f32x2(s.x, s.y), f32x2(s.z, s.w)},
                   nn[2] = {f32x2(-s.x, -s.y), f32x2(-s.z, -s.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f.ac[i] = rotated ? mul_f32x2(w.a[i], cc[i]) : w.a[i];
        f.bc[i] = rotated ? mul_f32x2(w.b[i], cc[i]) : w.b[i];
        f.as[i] = mul_f32x2(w.a[i], ss[i]);
        f.bs[i] = mul_f32x2(w.b[i], nn[i]);
    }
}
// Factors of the lane's pairs i .. i + 3 from a token's row of the table.
template <bool INTERLEAVED>
__device__ __forceinline__ void load_factors(const float *row, int rot, const Place<INTERLEAVED> &p, float4 &c,
                                             float4 &s) {
    const int i = INTERLEAVED ? p.a / 2 : p.a;
    c = *reinterpret_cast<const float4 *>(row + i);
    s = *reinterpret_cast<const float4 *>(row + rot / 2 + i);
}

// The group's row, normed where `norm`, rotated in the lanes that are (`mixed`:
// some lane is not).  Every lane of the warp calls it with the same `norm` (the
// lanes add their squares up); lanes without elements hold zeros.
template <int L, bool INTERLEAVED>
__device__ __forceinline__ uint4 norm_rotate(const uint4 &v, bool norm, float inv_d, float eps, bool mixed,
                                             bool rotated, const Factors &k) {
    Pairs x = pairs_of<INTERLEAVED>(v);
    if (norm) {
        uint64_t q = mul_f32x2(x.a[0], x.a[0]);
        q = fma_f32x2(x.a[1], x.a[1], q);
        q = fma_f32x2(x.b[0], x.b[0], q);
        q = fma_f32x2(x.b[1], x.b[1], q);
        float ss, hi;
        f32x2_split(q, ss, hi);
        ss += hi;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
        const float f = rsqrtf(fmaf(ss, inv_d, eps));
        const uint64_t ff = f32x2(f, f);
#pragma unroll
        for (int i = 0; i < 2; ++i) x.a[i] = mul_f32x2(x.a[i], ff), x.b[i] = mul_f32x2(x.b[i], ff);
    }
    Pairs y;
    if (mixed && !rotated) {
#pragma unroll
        for (int i = 0; i < 2; ++i) y.a[i] = mul_f32x2(x.a[i], k.ac[i]), y.b[i] = mul_f32x2(x.b[i], k.bc[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            y.a[i] = fma_f32x2(x.a[i], k.ac[i], mul_f32x2(x.b[i], k.bs[i]));
            y.b[i] = fma_f32x2(x.b[i], k.bc[i], mul_f32x2(x.a[i], k.as[i]));
        }
    }
    return words_of<INTERLEAVED>(y);
}

}  // namespace ck
