// fp4_core.cuh -- quantization to microscaled 4-bit floats, the part that the
// quantizer and the block norm share.
//
// A code is an E2M1 number: 0, 0.5, 1, 1.5, 2, 3, 4 or 6 and a sign.  With
// amax the largest magnitude of a block,
//   MX (32 codes):  s = 2^e, e = max(floor(log2 amax) - 2, -127)   (E8M0)
//   NV (16 codes):  s = E4M3(amax / (6 t)), at most 448, t the tensor's scale
//   code = E2M1(x / d), to nearest, ties to the even code, at most 6;
//   d = s (MX) or f32(s t) (NV); all codes 0 where s is 0.
// A block with a NaN or an infinity gets a NaN scale (0xFF, 0x7F).
//
// Values on the border of two codes are common (the inputs are bf16 and d has
// few bits), so the quotient has to be the correctly rounded one: a product with
// 1 / d alone would land to either side of the border.  MX: 1 / d is a power of
// two and the product exact.  NV: Markstein's correction, q + r (x - q d) with r
// = 1 / d, on two elements at a time (three operations for two elements); r by a
// Newton step on the hardware's approximation, within 2^-23 of itself, which
// leaves the corrected quotient within 2^-43 of x / d before its rounding: exact
// where x / d is an f32 number, as on a border, and nearest elsewhere but for
// quotients that close to the middle of two f32 numbers.  amax / (6 t) likewise,
// its reciprocal from the host.  (IEEE divisions in their place: the quantizer of
// 16384 x 4096 49 us instead of 37.)
//
// Layout.  Codes: [rows, K / 2] bytes, the even column in the low half.  Scales:
// tiles of 128 rows x one 32-bit word (four scales, 64 (NV) or 128 (MX)
// columns), the words of a tile of rows one after another; in a tile of 512
// bytes row r's word lies at 16 (r % 32) + 4 (r / 32): what tcgen05.cp copies to
// TMEM as it stands.  Scales past K in a row's last word are 0.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

#include "fp4.h"
#include "ptx.cuh"

namespace ck {
namespace fp4 {

constexpr unsigned kFull = 0xffffffffu;

// Byte offset of row's word `word` of `words` a row.
__device__ __forceinline__ int64_t scale_word_at(int64_t row, int word, int words) {
    const int r = static_cast<int>(row & 127);
    return ((row >> 7) * words + word) * 512 + (r & 31) * 16 + (r >> 5) * 4;
}

// 16 bytes that are read once: they do not displace others in L1, and are not taken for
// data that nobody writes (a kernel ahead may have been writing them when this one was
// let in, and a norm may write them back in place).
__device__ __forceinline__ uint4 load_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// A pair of bf16 as f32, and as f32 with the signs turned (one operation each).
__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
    return f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint64_t unpack2_neg(uint32_t w) {
    return f32x2(__uint_as_float(w * 65536u + 0x80000000u), __uint_as_float((w & 0xffff0000u) ^ 0x80000000u));
}

// Largest magnitude of three, a NaN if one of them is.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Eight codes of f32 pairs, the first in the lowest bits.
__device__ __forceinline__ uint32_t pack8(const uint64_t (&q)[4]) {
    float a[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f32x2_split(q[i], a[2 * i], a[2 * i + 1]);
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(a[0]), "f"(a[1]), "f"(a[2]), "f"(a[3]), "f"(a[4]), "f"(a[5]), "f"(a[6]), "f"(a[7]));
    return r;
}

// A tensor's scale.
struct Scale {
    float tensor, six_tensor, inv_six;  // t, 6 t and 1 / (6 t)
};
inline Scale scale_of(float tensor) { return Scale{tensor, 6.f * tensor, 1.f / (6.f * tensor)}; }

// What a block's values are divided by, from its largest magnitude (a NaN if it has
// one), and its scale byte.
struct Divisor {
    uint64_t r2;   // -1 / d twice (MX: of a NaN scale not a number)
    uint64_t d2;   // d twice (NV)
    bool cut;      // NV: the scale is cut off, and a quotient could overflow
};
template <bool NV>
__device__ __forceinline__ Divisor divisor(float m, const Scale &t, uint32_t &scale) {
    Divisor v;
    const bool finite = m < __int_as_float(0x7f800000);
    if constexpr (NV) {
        // past 448 the scale is cut off; so far past it this quotient might overflow, too
        const float m_cut = fminf(m, 1024.f * t.six_tensor);
        const float s0 = __fmul_rn(m_cut, t.inv_six);
        const float s = __fmaf_rn(__fmaf_rn(-s0, t.six_tensor, m_cut), t.inv_six, s0);
        const __nv_fp8_storage_t s8 = __nv_cvt_float_to_fp8(s, __NV_SATFINITE, __NV_E4M3);
        scale = finite ? s8 : 0x7fu;
        const float d = __fmul_rn(__half2float(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)), t.tensor);
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
        r = s8 != 0 ? __fmaf_rn(__fmaf_rn(d, -r, 1.f), -r, -r) : -0.f;
        v.r2 = f32x2(r, r), v.d2 = f32x2(d, d);
        v.cut = !(s <= 448.f);
    } else {
        const uint32_t e = __float_as_uint(m) >> 23;
        scale = finite ? (e > 2 ? e - 2 : 0u) : 0xffu;
        const float r = __uint_as_float(((254u - scale) << 23) | 0x80000000u);
        v.r2 = f32x2(r, r), v.d2 = 0, v.cut = false;
    }
    return v;
}

// Codes of eight values, their signs turned.  NV: with n = -x, q0 = n (-r), the
// remainder q0 d + n and q0 + remainder (-r): in this form a zero keeps its sign.
template <bool NV>
__device__ __forceinline__ uint32_t codes8(const uint64_t (&n)[4], const Divisor &v) {
    uint64_t q[4];
    if constexpr (!NV) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = mul_f32x2(n[i], v.r2);
    } else if (!v.cut) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t q0 = mul_f32x2(n[i], v.r2);
            q[i] = fma_f32x2(fma_f32x2(q0, v.d2, n[i]), v.r2, q0);
        }
    } else {
        // an infinite quotient's correction would be NaN
        float d, unused;
        f32x2_split(v.d2, d, unused);
        const float top = 8.f * d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f32x2_split(n[i], a, b);
            const uint64_t x = f32x2(fminf(fmaxf(a, -top), top), fminf(fmaxf(b, -top), top));
            const uint64_t q0 = mul_f32x2(x, v.r2);
            q[i] = fma_f32x2(fma_f32x2(q0, v.d2, x), v.r2, q0);
        }
    }
    return pack8(q);
}

__device__ __forceinline__ float amax8(const uint64_t (&n)[4], float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f32x2_split(n[i], a, b);
        m = max3_abs_nan(m, a, b);
    }
    return m;
}

// Eight consecutive values of a row in each lane (two lanes hold an NV block,
// four an MX block; lane 0's first value begins one), their signs turned, -> the
// lane's codes and the block's scale byte.  Every lane of the warp takes part.
template <bool NV>
__device__ __forceinline__ uint32_t quantize8(const uint64_t (&n)[4], const Scale &t, uint32_t &scale) {
    float m = amax8(n, 0.f);
    m = max_nan(m, __shfl_xor_sync(kFull, m, 1));
    if constexpr (!NV) m = max_nan(m, __shfl_xor_sync(kFull, m, 2));
    return codes8<NV>(n, divisor<NV>(m, t, scale));
}

// Lanes of a block and of a word of four.
constexpr int block_lanes(bool nv) { return nv ? 2 : 4; }
constexpr int word_lanes(bool nv) { return nv ? 8 : 16; }

}  // namespace fp4
}  // namespace ck
