// 8-bit activation checkpoints (format: ckpt.cuh) and the SwiGLU gradient that
// reads its inputs from one.  All three kernels stream: HBM bound.  One B200,
// 16384 rows: store 33 us and restore 31 us of 4096 values (201 MB each, 6.1 and
// 6.5 TB/s), SwiGLU gradient of 2048 with h 56 us (336 MB, 6.0 TB/s).
#include "ckpt.cuh"
#include "kernels.cuh"
#include "moe_common.cuh"

namespace moe {

constexpr int kCkThreads = 256;

// Items of 8 inputs, 16 neighbouring lanes to a 128-input block: every load
// and store of a warp is one contiguous piece.  Each thread takes kCkUnroll
// items, a grid stride apart, and issues their loads together.
constexpr int kCkUnroll = 4;

// Row of an item (8 of a row's K8).  Contiguous rows (FLAT) need none: the
// strided form divides, in 32 bits where the count allows.
__device__ __forceinline__ long long ck_row(long long i, int K8, bool small) {
    return small ? (long long)((uint32_t)i / (uint32_t)K8) : i / K8;
}

// The arithmetic is on pairs of bf16 as far as it goes: |x| and the maximum on
// the bits, x 2^-e exactly (below bf16's normal range the code is 0 either way),
// and only the last step, to E4M3, from fp32.  With fp32 throughout the kernel
// was bound by its instructions (59 us for 16384 x 4096).
template <bool FLAT>
__global__ void __launch_bounds__(kCkThreads)
    k_ckpt_pack(const __nv_bfloat16* __restrict__ x, long long ldx, long long items, int K8,
                uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    pdl_begin();
    const long long stride = (long long)gridDim.x * kCkThreads;
    const bool small = items >> 31 == 0;
    // (items and stride are multiples of 16: the lanes of a block agree)
    for (long long i0 = blockIdx.x * (long long)kCkThreads + threadIdx.x; i0 - (threadIdx.x & 31) < items;
         i0 += stride * kCkUnroll) {
        uint4 q[kCkUnroll];
#pragma unroll
        for (int u = 0; u < kCkUnroll; ++u) {
            const long long i = i0 + u * stride;
            q[u] = make_uint4(0u, 0u, 0u, 0u);
            if (i >= items) continue;
            long long src = i * 8;
            if (!FLAT) {
                const long long t = ck_row(i, K8, small);
                src = t * ldx + (i - t * K8) * 8;
            }
            q[u] = __ldg(reinterpret_cast<const uint4*>(x + src));
        }
#pragma unroll
        for (int u = 0; u < kCkUnroll; ++u) {
            const long long i = i0 + u * stride;
            const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
            // the block's maximum magnitude; NaN where it holds one
            auto max2 = [](uint32_t a, uint32_t b) {
                uint32_t r;
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
                return r;
            };
            uint32_t m = max2(max2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), max2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = max2(m, m >> 16) & 0x7fffu;
            float amax = __uint_as_float(m << 16);
            const bool odd = m > 0x7f60u;       // above 448 * 2^119 (e = 120), or not finite
            if (__any_sync(0xffffffffu, odd)) {
                // the maximum of the finite values
                amax = 0.0f;
                float v[8];
                bf16x8_values(q[u], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]) <= 3.4028235e38f ? fabsf(v[j]) : 0.0f);
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            }
            if (i >= items) continue;
            const int e = ckpt_exponent(amax);
            uint2 c;
            if (!odd) {
                const uint32_t inv = (__float_as_uint(ckpt_pow2(-e)) >> 16) * 0x00010001u;     // exact in bf16
                float v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t p;
                    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p) : "r"(w[j]), "r"(inv));
                    v[2 * j] = __uint_as_float(p << 16);
                    v[2 * j + 1] = __uint_as_float(p & 0xffff0000u);
                }
                c = make_uint2(e4m3x4_code(v[0], v[1], v[2], v[3]), e4m3x4_code(v[4], v[5], v[6], v[7]));
            } else {
                const float inv = ckpt_pow2(-e), top = e >= 120 ? 240.0f : 448.0f;
                float v[8], r[8];
                bf16x8_values(q[u], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = fminf(fmaxf(v[j] * inv, -top), top);
                c = make_uint2(e4m3x4_code(r[0], r[1], r[2], r[3]), e4m3x4_code(r[4], r[5], r[6], r[7]));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!(fabsf(v[j]) <= 3.4028235e38f)) {
                        uint32_t& cw = j < 4 ? c.x : c.y;
                        cw = (cw & ~(0xffu << (8 * (j & 3)))) | (0x7fu << (8 * (j & 3)));
                    }
            }
            *reinterpret_cast<uint2*>(codes + i * 8) = c;
            if ((i & 15) == 0) scales[i >> 4] = (uint8_t)(e + 127);
        }
    }
}

template <bool FLAT>
__global__ void __launch_bounds__(kCkThreads)
    k_ckpt_unpack(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, long long items, int K8,
                  __nv_bfloat16* __restrict__ x, long long ldx) {
    pdl_begin();
    const long long stride = (long long)gridDim.x * kCkThreads;
    const bool small = items >> 31 == 0;
    for (long long i0 = blockIdx.x * (long long)kCkThreads + threadIdx.x; i0 < items; i0 += stride * kCkUnroll) {
        uint2 c[kCkUnroll];
        uint32_t s[kCkUnroll];
#pragma unroll
        for (int u = 0; u < kCkUnroll; ++u) {
            const long long i = i0 + u * stride;
            if (i < items) {
                c[u] = __ldg(reinterpret_cast<const uint2*>(codes + i * 8));
                s[u] = __ldg(scales + (i >> 4));
            }
        }
#pragma unroll
        for (int u = 0; u < kCkUnroll; ++u) {
            const long long i = i0 + u * stride;
            if (i >= items) break;
            float v[8];
            ckpt_values8(c[u], ckpt_scale(s[u]), v);
            long long dst = i * 8;
            if (!FLAT) {
                const long long t = ck_row(i, K8, small);
                dst = t * ldx + (i - t * K8) * 8;
            }
            *reinterpret_cast<uint4*>(x + dst) = bf16x8_rn(v);
        }
    }
}

// SwiGLU: h = g s(g) u with s the logistic function, so
//   dg = dh u (s + g s (1 - s)),  du = dh g s.
// One item is 8 neighbouring features of a row: 8 + 8 code bytes, 16 bytes of
// dh, and 16 bytes each of dg, du and (H) h.  fp32 throughout, one rounding
// per output.  s and 1 - s are both quotients of non-negative terms,
// 1 / (1 + e^-|g|) and e^-|g| / (1 + e^-|g|) in turn, so neither cancels.
template <bool H>
__global__ void __launch_bounds__(kCkThreads)
    k_ckpt_swiglu_bwd(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const __nv_bfloat16* __restrict__ dh, long long lddh, long long items, int I,
                      __nv_bfloat16* __restrict__ dgu, __nv_bfloat16* __restrict__ h) {
    pdl_begin();
    const int I8 = I / 8, KB = I / 128;
    const bool small = items >> 31 == 0;
    const long long stride = (long long)gridDim.x * kCkThreads;
    // (one item in flight per thread, at full occupancy: 56 us for 16384 x 2048
    // with h; two and four at fewer threads 61 and 64)
    for (long long i = blockIdx.x * (long long)kCkThreads + threadIdx.x; i < items; i += stride) {
        const long long t = ck_row(i, I8, small);
        const int c8 = (int)(i - t * I8);
        const uint8_t* row = codes + t * 2 * I + c8 * 8;
        const uint8_t* srow = scales + t * 2 * KB + (c8 >> 4);
        const uint2 cg = __ldg(reinterpret_cast<const uint2*>(row)), cu = __ldg(reinterpret_cast<const uint2*>(row + I));
        const uint32_t sg = __ldg(srow), su = __ldg(srow + KB);
        const uint4 d = __ldg(reinterpret_cast<const uint4*>(dh + t * lddh + c8 * 8));
        float g[8], up[8], dv[8], og[8], ou[8], oh[8];
        ckpt_values8(cg, ckpt_scale(sg), g);
        ckpt_values8(cu, ckpt_scale(su), up);
        bf16x8_values(d, dv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = __expf(-fabsf(g[j]));
            const float r = __fdividef(1.0f, 1.0f + e);
            const float er = e * r;
            const float s = g[j] >= 0.0f ? r : er;       // NaN: er, a NaN
            const float q = g[j] >= 0.0f ? er : r;       // 1 - s
            const float a = g[j] * s;
            og[j] = dv[j] * up[j] * fmaf(a, q, s);
            ou[j] = dv[j] * a;
            oh[j] = a * up[j];
        }
        __nv_bfloat16* o = dgu + t * 2 * I + c8 * 8;
        *reinterpret_cast<uint4*>(o) = bf16x8_rn(og);
        *reinterpret_cast<uint4*>(o + I) = bf16x8_rn(ou);
        if (H) *reinterpret_cast<uint4*>(h + t * I + c8 * 8) = bf16x8_rn(oh);
    }
}

static dim3 ck_grid(long long items, int per_thread) {
    const long long ctas = (items + (long long)kCkThreads * per_thread - 1) / ((long long)kCkThreads * per_thread);
    return dim3((unsigned)std::max(1LL, std::min(ctas, 148LL * 64)));
}

cudaError_t launch_ckpt_pack(const void* x, long long ldx, int T, int K, uint8_t* codes, uint8_t* scales,
                             cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const long long items = (long long)T * (K / 8);
    const cudaError_t e = launch_pdl(ldx == K ? k_ckpt_pack<true> : k_ckpt_pack<false>, ck_grid(items, kCkUnroll), dim3(kCkThreads), 0, st,
                                     (const __nv_bfloat16*)x, ldx, items, K / 8, codes, scales);
    count_launches(1);
    return e;
}

cudaError_t launch_ckpt_unpack(const uint8_t* codes, const uint8_t* scales, int T, int K, void* x, long long ldx,
                               cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const long long items = (long long)T * (K / 8);
    const cudaError_t e = launch_pdl(ldx == K ? k_ckpt_unpack<true> : k_ckpt_unpack<false>, ck_grid(items, kCkUnroll), dim3(kCkThreads), 0, st, codes, scales,
                                     items, K / 8, (__nv_bfloat16*)x, ldx);
    count_launches(1);
    return e;
}

cudaError_t launch_ckpt_swiglu_backward(const uint8_t* codes, const uint8_t* scales, const void* dh, long long lddh,
                                        int T, int I, void* dgu, void* h, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const long long items = (long long)T * (I / 8);
    const dim3 grid = ck_grid(items, 1);
    cudaError_t e;
    if (h)
        e = launch_pdl(k_ckpt_swiglu_bwd<true>, grid, dim3(kCkThreads), 0, st, codes, scales, (const __nv_bfloat16*)dh,
                       lddh, items, I, (__nv_bfloat16*)dgu, (__nv_bfloat16*)h);
    else
        e = launch_pdl(k_ckpt_swiglu_bwd<false>, grid, dim3(kCkThreads), 0, st, codes, scales,
                       (const __nv_bfloat16*)dh, lddh, items, I, (__nv_bfloat16*)dgu, (__nv_bfloat16*)h);
    count_launches(1);
    return e;
}

}  // namespace moe
