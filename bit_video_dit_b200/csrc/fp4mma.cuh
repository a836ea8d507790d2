// fp4mma.cuh -- E2M1 data as operands of the 16-bit matrix instructions:
// decoding, the 16 x 8 x 16 warp-level product, and the scaling of bf16 rows to
// binary16.
#pragma once

#include "common.cuh"

namespace nvfp4 {
namespace fp4mma {

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into cleared sums.
__device__ __forceinline__ void mma_16816_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// 8 codes, two a byte, times the pair s: e2m1 s is exact in binary16 (at most 6
// significant bits).  Naming the word's bytes lets each conversion read its
// byte in place: 2 instructions a pair, 136 elements a nanosecond and SM
// measured, against 78 with a shift and mask a byte, and 70 with shifts and
// masks in place of the conversion.
__device__ __forceinline__ void decode8(uint32_t w, __half2 s, uint32_t* o) {
    asm("{\n\t"
        ".reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t"
        "}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = h2_bits(__hmul2(bits_h2(o[i]), s));
}

// The 8 codes of one row and of another -> the 8 pairs (a_i s.x, b_i s.y)
__device__ __forceinline__ void decode8_rows(uint32_t a, uint32_t b, __half2 s, uint32_t* o) {
    uint32_t even[4], odd[4];
    decode8((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), s, even);
    decode8(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), s, odd);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        o[2 * i] = even[i];
        o[2 * i + 1] = odd[i];
    }
}

// The largest magnitude (bf16 bits) of 8 N bf16.
template <int N>
__device__ __forceinline__ uint32_t max_bits(const uint4* v) {
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < N; i++)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                   __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
    return max(mx & 0xFFFFu, mx >> 16);
}

// 2^k that brings a row's largest magnitude into [2^14, 2^15), and 2^-k.
// Rounding to binary16 is then exact for values down to 2^-28 of the largest
// (bf16 has 8 significant bits).
struct RowScale {
    float up, down;
};
__device__ __forceinline__ RowScale row_scale(uint32_t mx) {
    const int k = mx == 0u ? 0 : min(126, 141 - (int)(mx >> 7));
    return RowScale{__uint_as_float((uint32_t)(127 + k) << 23), __uint_as_float((uint32_t)(127 - k) << 23)};
}

// 8 bf16 times 2^k -> 4 binary16 pairs
__device__ __forceinline__ void scale8(const uint4& v, float up, uint32_t* o) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++)
        o[i] = h2_bits(__floats2half2_rn(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up));
}

// One lane's 8 N bf16 of a row whose other lanes are t ^ 1 and t ^ 2; returns 2^-k.
template <int N>
__device__ __forceinline__ float scale_row(const uint4* v, uint32_t* o) {
    uint32_t mx = max_bits<N>(v);
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    const RowScale s = row_scale(mx);
#pragma unroll
    for (int j = 0; j < N; j++) scale8(v[j], s.up, o + 4 * j);
    return s.down;
}

}  // namespace fp4mma
}  // namespace nvfp4
