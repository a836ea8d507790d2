// fp4mma.cuh -- E2M1 data as operands of the binary16 warp-level matrix
// instruction (16 x 8 x 16), for kernels with few rows: decoding, and the
// scaling of bf16 rows to binary16.
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

// Decoded operands carry 2^-kDecodeShift: v = 2^-8 e2m1 s, exact in binary16
// (a multiple of 2^-18 below 2^4).  There are two ways to the same value, and
// the kernels use both, since the conversion unit alone or the integer pipe
// alone would bound them (44 and 41 elements a clock and SM measured):
//  - the conversion instruction and a multiplication by 2^-8 s;
//  - shifts and masks that put a code's sign, exponent and fraction at their
//    places in binary16, which is 2^-14 e2m1, and a multiplication by 2^6 s.
constexpr uint32_t kMulCvt = 0x1C001C00u;  // 2^-8 twice
constexpr uint32_t kMulBits = 0x54005400u;  // 2^6 twice
constexpr float kDecodeBack = 256.0f;       // 2^8

// 8 codes (two a byte) -> the pairs (0, 1), (2, 3), (4, 5), (6, 7); s = 2^-8 scale
__device__ __forceinline__ void decode8_cvt(uint32_t w, __half2 s, uint32_t* o) {
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = h2_bits(__hmul2(e2m1x2_to_half2((w >> (8 * i)) & 0xFFu), s));
}

// 8 codes -> the pairs (i, i + 4), i = 0..3; s = 2^6 scale
__device__ __forceinline__ void decode8_bits(uint32_t w, __half2 s, uint32_t* o) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t y = w << (12 - 4 * i);
        o[i] = h2_bits(__hmul2(bits_h2((y & 0x80008000u) | ((y >> 3) & 0x0E000E00u)), s));
    }
}

// One lane's 8 NW bf16 of a row, whose other lanes are t ^ 1, t ^ 2, times 2^k
// with the row's largest magnitude in [2^14, 2^15), as binary16 pairs in the
// order of the decoded operand: decode8_cvt's for the first NW / 2 words of 8,
// decode8_bits's for the rest.  Exact for values down to 2^-28 of the largest
// (bf16 has 8 significant bits).  Returns 2^-k.
template <int NW>
__device__ __forceinline__ float scale_row(const uint4* v, uint32_t* o) {
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < NW; i++)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                   __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    mx = max(mx & 0xFFFFu, mx >> 16);
    const int k = mx == 0u ? 0 : min(126, 141 - (int)(mx >> 7));
    const float pk = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
    for (int j = 0; j < NW; j++) {
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float lo, hi;
            if (j < NW / 2) {  // 8 j + 2 i, + 1
                lo = __uint_as_float(w[i] << 16);
                hi = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {  // 8 j + i, 8 j + i + 4
                lo = (i & 1) ? __uint_as_float(w[i >> 1] & 0xFFFF0000u) : __uint_as_float(w[i >> 1] << 16);
                hi = (i & 1) ? __uint_as_float(w[2 + (i >> 1)] & 0xFFFF0000u) : __uint_as_float(w[2 + (i >> 1)] << 16);
            }
            o[4 * j + i] = h2_bits(__floats2half2_rn(lo * pk, hi * pk));
        }
    }
    return __uint_as_float((uint32_t)(127 - k) << 23);
}

}  // namespace fp4mma
}  // namespace nvfp4
