// head_norm_rope.cuh -- RMS norm and position rotation of one attention head's
// row, held by a group of L neighbouring lanes of a warp, 8 elements a lane.
//
//   y[d] = x[d] * rsqrt(mean(x^2) + eps) * w[d]
//   (y[a], y[b]) -> (y[a] c[i] - y[b] s[i], y[b] c[i] + y[a] s[i])
// for the pairs (i, i + r/2) or (2i, 2i + 1).  Everything is f32 between the
// bf16 loads and the one rounding of the caller's store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ck {

// The 8 bf16 of a 16-byte load as f32 and back (round to nearest even).
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// 8 consecutive norm weights (bf16 or f32) from element d0.
__device__ __forceinline__ void load_weight8(const void *w, bool w_f32, int d0, float (&out)[8]) {
    if (w_f32) {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + d0);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + d0 + 4);
        out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
        out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(w) + d0), out);
    }
}

// What a lane needs of one token's rotation: the factors of its 8 elements.
// HALF: c[j], s[j] of element d0 + j (its pair's index modulo r/2), s negated
// for the first of the pair.  INTERLEAVED: c[j / 2] and s[j / 2] used, j even.
struct Rotation {
    float c[8], s[8];
    int partner;  // HALF: the lane (within the group) of the paired elements
    bool on;      // these 8 elements are rotated
};

template <bool INTERLEAVED>
__device__ __forceinline__ void load_rotation(Rotation &r, const float *row, int rot, int d0, int gl) {
    r.on = d0 < rot;
    r.partner = gl;
    if (!r.on) return;
    const int half = rot / 2;
    if constexpr (INTERLEAVED) {
        const float4 c = *reinterpret_cast<const float4 *>(row + d0 / 2);
        const float4 s = *reinterpret_cast<const float4 *>(row + half + d0 / 2);
        r.c[0] = c.x, r.c[1] = c.y, r.c[2] = c.z, r.c[3] = c.w;
        r.s[0] = s.x, r.s[1] = s.y, r.s[2] = s.z, r.s[3] = s.w;
    } else {
        const bool first = d0 < half;
        const int i = first ? d0 : d0 - half;
        r.partner = first ? gl + half / 8 : gl - half / 8;
        const float sign = first ? -1.f : 1.f;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(row + i + j);
            const float4 s = *reinterpret_cast<const float4 *>(row + half + i + j);
            r.c[j] = c.x, r.c[j + 1] = c.y, r.c[j + 2] = c.z, r.c[j + 3] = c.w;
            r.s[j] = sign * s.x, r.s[j + 1] = sign * s.y;
            r.s[j + 2] = sign * s.z, r.s[j + 3] = sign * s.w;
        }
    }
}

// The group's row x normed (where `mine`) and rotated in place.  Every lane of
// the warp calls it with the same `norm` and `rotate` (the lanes exchange
// values; rows of one warp may differ in `mine`); lanes past D / 8 hold zeros.
template <int L, bool INTERLEAVED>
__device__ __forceinline__ void norm_rotate(float (&x)[8], bool norm, bool mine, const float (&w)[8], float inv_d,
                                            float eps, bool rotate, const Rotation &r) {
    if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
        const float f = rsqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = mine ? x[j] * f * w[j] : x[j];
    }
    if (!rotate) return;  // uniform over the grid
    if constexpr (INTERLEAVED) {
        if (r.on) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = a * r.c[j] - b * r.s[j];
                x[2 * j + 1] = b * r.c[j] + a * r.s[j];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float other = __shfl_sync(0xffffffffu, x[j], r.partner, L);
            if (r.on) x[j] = x[j] * r.c[j] + other * r.s[j];
        }
    }
}

}  // namespace ck
