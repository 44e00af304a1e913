// The 4-bit cache format (E2M1 codes with one E4M3 scale per 16 values) on the device:
// quantizing and widening a group, and the place of a row in its page.
//
// A page (physical block, kv head) of block size Bs holds Bs rows of D/2 code bytes (even dim in
// the low nibble) followed by D/16 rows of Bs scale bytes: the scale of group g (dims 16 g ..
// 16 g + 15) of token t sits at [g][t].  Four tokens' scales of one group are one aligned word,
// which is what a tensor-core fragment of either operand needs beside its codes.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"

namespace pa {

__host__ __device__ constexpr int e2m1_page_bytes(int block_size, int head_dim) {
    return block_size * head_dim * 9 / 16;
}

// Eight codes (one word, the lowest nibble first) from eight floats: nearest even, saturating at 6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{ .reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d}; }"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// Eight codes to four f16 pairs (exact), the lower dim in the low half.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t codes, uint32_t (&h)[4]) {
    asm("{ .reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d; }"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// Two E4M3 codes (the low 16 bits) to an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(codes));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
    float2 r;
    asm("{ .reg .b16 l, u; mov.b32 {l, u}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, u; }"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}

// One E4M3 code of a non-negative float: nearest even, saturating at 448; a NaN stays one (0x7F).
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xFFu;
}

// A larger of two magnitudes that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// One group: y = x * inv (one float product), s = E4M3(max|y| / 6), codes E2M1(y / s), 0 where s
// is 0.  Both quotients are the correctly rounded ones, so that a quotient half way between two
// codes is seen as such: for the 16 values the quotient is formed from the scale's reciprocal r
// and one residual step, q' = q + (y - q s) r with q = y r (Markstein), 3 instructions a value;
// s is one of 126 E4M3 values, so r and the residual neither overflow nor lose bits.  Values past
// the largest code's reach are cut to 8 s before (infinities too, which the residual would turn
// into NaN).  A group with a NaN reads back as NaN (its scale is one); a zero's code is 0.
__device__ __forceinline__ uint2 e2m1_quantize16(const float (&x)[16], float inv, uint32_t& scale_code) {
    float y[16], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        y[i] = __fmul_rn(x[i], inv);
        amax = max_nan(amax, fabsf(y[i]));
    }
    scale_code = f32_to_e4m3(__fdiv_rn(amax, 6.f));
    const float s = f16x2_to_f32x2(e4m3x2_to_f16x2(scale_code)).x;
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;   // s == 0, or a NaN: every code 0
    uint2 codes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // saturate first: |y| beyond 8 s reads as 8 s (code 6), which keeps infinities out
            const float v = fminf(fmaxf(y[8 * h + i], -8.f * s), 8.f * s);
            const float q = __fmul_rn(v, r);
            t[i] = __fmaf_rn(__fmaf_rn(-q, s, v), r, q);
        }
        (h ? codes.y : codes.x) = s > 0.f ? f32x8_to_e2m1x8(t) : 0u;
    }
    return codes;
}

// 16 bf16 values (two 16-byte chunks) as floats.
__device__ __forceinline__ void bf16x16_to_f32(uint4 a, uint4 b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Group g of the row (token `off` of its page) at `page`: its 8 code bytes and its scale byte.
template <int D>
__device__ __forceinline__ uint2* e2m1_codes(uint8_t* page, int off, int g) {
    return reinterpret_cast<uint2*>(page + off * (D / 2) + g * 8);
}
template <int D>
__device__ __forceinline__ uint8_t* e2m1_scale(uint8_t* page, int block_size, int off, int g) {
    return page + block_size * (D / 2) + g * block_size + off;
}

// RoPE for rows that are quantized after it.  A rotated value next to a border between two codes
// must fall on the same side wherever it is computed, so the angle, its cosine and sine and the
// rotation are all formed in double and the row is rounded to float, then to bf16.
__device__ __forceinline__ void rope_cos_sin64(int32_t pos, double inv_freq, double* c, double* s) {
    const double a = (double)pos * inv_freq;
    // a - k 2 pi with 2 pi in two parts: |a| reaches 2^31, where one double of 2 pi is not enough
    const double k = rint(a * 0.15915494309189533577);
    double r = fma(-k, 6.2831853071795864769, a);
    r = fma(-k, 2.4492935982947063545e-16, r);
    sincos(r, s, c);
}
__device__ __forceinline__ uint16_t rope_round(double y) { return f32_to_bf16_rn((float)y); }

}  // namespace pa
