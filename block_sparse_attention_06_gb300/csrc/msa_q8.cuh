// The 8-bit cache format, shared by its writer and its readers.
//
// A row (one token of one group) is `width` e4m3 codes and one scale byte b: value = code * 2^(b - 127).
// The scale is the smallest power of two under which the row's largest magnitude is at most 448, the
// largest e4m3 number, and at least 2^-100; a row of zeros has scale 1, a row that holds a NaN or an
// infinity has b = 255 (NaN).  e4m3 has four significant bits and the scale is a power of two, so every
// stored value is also a bf16 number: a bf16 contraction over the stored values rounds nothing further.
#pragma once

#include "msa_device.cuh"

namespace msa {

constexpr int kQ8LowestExp = -100;   // of a scale that the writer gives

// 2^(b - 127); NaN for b = 255 (b = 0, which the writer never gives, is 2^-127).
__device__ __forceinline__ float q8_scale(uint32_t b) {
    const uint32_t bits = b == 255u ? 0x7fffffffu : b == 0u ? 0x00400000u : b << 23;
    return __uint_as_float(bits);
}

// Exponent of the scale of a row whose largest magnitude has the bits `amax` (not a NaN or an infinity).
// amax = m 2^E with m in [0.5, 1) and 448 = 0.875 * 2^9, so amax / 2^e <= 448 for e = E - 9 where
// m <= 0.875 and for E - 8 elsewhere.  A magnitude under 2^-126 ends at the lowest exponent.
__device__ __forceinline__ int q8_exponent(uint32_t amax) {
    if (amax == 0u) return 0;
    const int e = int(amax >> 23) - 126 - 9 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, kQ8LowestExp);
}

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }   // -126 <= e <= 127

// Two fp32 numbers as e4m3, round to nearest even (b in the upper byte).
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Two e4m3 codes (the lower 16 bits) as fp32.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w)));
    float2 f;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// Codes as f16, exactly (e4m3's range lies in f16's): what the MMAs below read.  A NaN code stays a NaN.
__device__ __forceinline__ uint32_t f16_of_low(uint32_t w) {    // codes 0 and 1 of a word
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ uint32_t f16_of_high(uint32_t w) {   // codes 2 and 3
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(h) : "r"(w));
    return h;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A vector of bf16 numbers as f16 times a power of two: q = x 2^e with the largest |x| in [2^14, 2^15).  f16 holds the
// eight bits of a bf16 number down to 2^-31 of the largest, and nothing above 2^-39 of it is lost.  amax: the bits of
// the largest magnitude, finite.
__device__ __forceinline__ int f16_exponent(uint32_t amax) { return max(int(amax >> 23) - 127, -100) - 14; }

// D += A B, f16 with fp32 accumulation: m16, n8, k16.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// `bytes` (a multiple of 16, both addresses 16-byte aligned) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void *smem_dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(smem_dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Maximum that keeps a NaN.
__device__ __forceinline__ float fmax_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

}  // namespace msa
