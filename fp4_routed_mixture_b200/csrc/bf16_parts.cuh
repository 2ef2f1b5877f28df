// fp32 values as sums of bf16 parts, for products on the tensor cores.
#pragma once
#include "ckpt.cuh"

namespace moe {

// v = h + m + l, each with 8 significant bits: h and m rounded to nearest, l
// exact (24 = 8 + 8 + 8 bits).  An infinity or NaN is its own first part.
__device__ __forceinline__ void split3(float v, float& h, float& m, float& l) {
    h = __bfloat162float(__float2bfloat16_rn(v));
    // (a finite value that rounds up to infinity is truncated instead)
    if (fabsf(h) == INFINITY) h = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    const float r = h == v ? 0.0f : v - h;
    m = __bfloat162float(__float2bfloat16_rn(r));
    l = m == r ? 0.0f : r - m;
}

// Two values' parts, a pair of bf16 each; one conversion a part and pair (one a value and
// part, of a quarter of the other instructions' rate, bound k_router_grad_small).
__device__ __forceinline__ void split3x2(float a, float b, uint32_t& h, uint32_t& m, uint32_t& l) {
    h = bf16x2_rn(a, b);
    if (((h & 0x7f807f80u) + 0x00800080u) & 0x80008000u) {       // not finite, or rounded up to infinity
        float h0, m0, l0, h1, m1, l1;
        split3(a, h0, m0, l0);
        split3(b, h1, m1, l1);
        h = bf16x2_rn(h0, h1);
        m = bf16x2_rn(m0, m1);
        l = bf16x2_rn(l0, l1);
        return;
    }
    const float ra = a - __uint_as_float(h << 16), rb = b - __uint_as_float(h & 0xffff0000u);
    m = bf16x2_rn(ra, rb);
    l = bf16x2_rn(ra - __uint_as_float(m << 16), rb - __uint_as_float(m & 0xffff0000u));
}

}  // namespace moe
