// 8-bit activation checkpoints: the format's arithmetic on the device.
//
// An activation x [T, K] is kept as E4M3 codes [T, K] and one UE8M0 scale byte
// per row and 128-input block [T, K/128]: the value is code * 2^(byte - 127).
// The scale is the smallest power of two 2^e with max|x| <= 448 * 2^e over the
// block's finite values (byte e + 127; 0 for a block without any other than
// zero), the code x / 2^e rounded to nearest even: the quantisation rule of
// moe_fp8_linear.  Two things that rule leaves open are fixed here: a NaN or
// infinity is kept as the NaN code 0x7F of its element (its neighbours keep
// their values), and at e = 120 magnitudes above 240 * 2^120 become that
// value, so that no finite x is restored as an infinity.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

// Scale exponent for a finite maximum amax >= 0.  amax = m * 2^q, m in [1, 2):
// amax <= 1.75 * 2^8 * 2^e holds from e = q - 8 on when m <= 1.75, else from
// q - 7.  (A subnormal amax has q < -126 and so e = -127, the lowest.)
__device__ __forceinline__ int ckpt_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int q = (int)(b >> 23) - 127;
    const int e = q - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, -127);
}

// 2^n, n in [-149, 127], exactly.
__device__ __forceinline__ float ckpt_pow2(int n) {
    return n >= -126 ? __uint_as_float((uint32_t)(n + 127) << 23) : __uint_as_float(1u << (n + 149));
}
// 2^(byte - 127); a scale byte 0xFF is NaN.
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
    return byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7fc00000u)
                                                                  : __uint_as_float(byte << 23);
}

// Two E4M3 codes (low byte first) as fp32.
__device__ __forceinline__ float2 e4m3x2_value(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t e4m3x4_code(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(lo) : "f"(a), "f"(b));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(hi) : "f"(c), "f"(d));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Eight codes (two words) times one scale.
__device__ __forceinline__ void ckpt_values8(uint2 c, float s, float (&v)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = e4m3x2_value((w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
        v[2 * i] = p.x * s;
        v[2 * i + 1] = p.y * s;
    }
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint4 bf16x8_rn(const float (&v)[8]) {
    return make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
}
__device__ __forceinline__ void bf16x8_values(uint4 q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

}  // namespace moe
