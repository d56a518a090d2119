// The 4-bit cache format shared by kvsel_kv4_store, kvsel_kv4_load and
// kvsel_kv4_attention (include/kvsel.h has its definition): groups of 16 values as
// E2M1 codes with one scale byte, bits 14..7 of the scale's fp16 pattern.
//
// A value is code * scale: at most 2 significant bits times 4, and at most
// 6 * 10240 = 61440, so every stored value is exact in fp16 and in bf16 (scales
// below 2^-14 are fp16 subnormals, multiples of 2^-17; their products with codes
// are multiples of 2^-18).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

constexpr int kKv4Group = 16;
constexpr float kKv4Max = 61440.f;      // largest value stored as a number
constexpr uint32_t kKv4NanByte = 0xFF;  // its fp16 pattern, 0x7F80, is a NaN

// Byte b's scale as a float.
__device__ __forceinline__ float kv4_scale(uint32_t b) { return __half2float(__ushort_as_half((uint16_t)(b << 7))); }

// The smallest scale s with top <= 6 s, top in [0, 61440].  The estimate is the scale at
// or below top / 6; the product top * (1/6) and the cut are off by less than one scale
// step each, so at most two steps up reach it (6 * scale is exact in fp32).
__device__ __forceinline__ uint32_t kv4_scale_byte(float top) {
    const float u = top * (1.f / 6.f);
    uint32_t b = u < 0x1p-14f ? (uint32_t)(u * 0x1p17f) : (__float_as_uint(u) >> 20) - (112u << 3);
    b += 6.f * kv4_scale(b) < top ? 1u : 0u;
    b += 6.f * kv4_scale(b) < top ? 1u : 0u;
    return b;
}

// The four bytes of w, two codes each (low four bits first), as pairs of exact fp16 values.
__device__ __forceinline__ void kv4_pairs(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// The codes of two values (magnitudes up to 6, round to nearest, ties to the even code), lo in the low four bits.
__device__ __forceinline__ uint32_t kv4_code2(float lo, float hi) {
    uint32_t w;
    asm volatile("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.u32.u8 %0, t;\n}\n"
                 : "=r"(w)
                 : "f"(lo), "f"(hi));
    return w;
}
// The codes of x[0..7] in a word, x[0] lowest.
__device__ __forceinline__ uint32_t kv4_codes(const float* x) {
    const uint32_t lo = __byte_perm(kv4_code2(x[0], x[1]), kv4_code2(x[2], x[3]), 0x0040);
    const uint32_t hi = __byte_perm(kv4_code2(x[4], x[5]), kv4_code2(x[6], x[7]), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
