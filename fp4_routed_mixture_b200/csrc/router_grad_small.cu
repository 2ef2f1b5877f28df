// Gradients of the router projection for few tokens (router_grad_small in
// kernels.cuh says which calls), in one launch on the CUDA cores:
//   dw[e, h] = sum_t dl[t, e] x[t, h],  dx[t, h] = sum_e dl[t, e] w[e, h],
//   dbias[e] = sum_t dl[t, e]
// with fp32 fused multiply-adds in a fixed order.  The tensor-core form
// (grad_gemm.cu) takes three launches, each of them mostly latency at these
// sizes.  The grid's first CTAs take dw in tiles of 64 experts x 64 columns (and
// dbias), 64 tokens a round, the others dx in tiles of 32 tokens x 32 columns, 256
// experts a round, four groups of threads a quarter of them each.  A round's loads
// are issued together (dw's next ones before this one's products); the products
// read shared memory, 16 multiply-adds for two 16-byte reads.
// One B200, 256 experts, H = 4096: 11.7 us for 64 tokens, 7.2 for one.
#include "ckpt.cuh"
#include "kernels.cuh"
#include "moe_common.cuh"

namespace moe {

constexpr int RS_THREADS = 256;
constexpr int RS_WE = 64, RS_WH = 64, RS_T = 64;      // tile of dw, tokens per round
constexpr int RS_XT = 32, RS_XH = 32, RS_XE = 256;    // tile of dx, experts per round

struct RouterSmallArgs {
    const float* dl;
    const __nv_bfloat16* x;
    const uint8_t* codes;
    const uint8_t* scales;
    const float* w;
    int T, H, E;
    __nv_bfloat16* dx;
    float* dw;
    float* db;
    int accumulate;
    int w_ctas, w_cols;      // CTAs of dw (or of dbias alone), and per row of its tiles
    int32_t* flag;
};

struct RouterSmallW {
    float x[RS_T][RS_WH];
    float d[RS_T][RS_WE + 4];
};
struct RouterSmallX {
    float w[RS_XE][RS_XH];
    float d[RS_XT][RS_XE + 4];      // (4 more: the four rows a quarter-warp reads lie in other banks)
};
union RouterSmallShared {
    RouterSmallW w;
    RouterSmallX x;
};

// Four neighbouring dlogits of a row (columns from `cols` on: 0).
__device__ __forceinline__ float4 rs_load4(const float* __restrict__ p, int cols, bool vec) {
    if (vec) return cols > 0 ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (cols > 0) v.x = __ldg(p);
    if (cols > 1) v.y = __ldg(p + 1);
    if (cols > 2) v.z = __ldg(p + 2);
    if (cols > 3) v.w = __ldg(p + 3);
    return v;
}

// Two sums at once: a fused multiply-add each (Blackwell's packed form).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 rs_twice(float v) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void rs_fma2(f32x2& acc, f32x2 a, f32x2 b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ float4 rs_four(f32x2 a, f32x2 b) {
    float4 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(a));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.z), "=f"(v.w) : "l"(b));
    return v;
}

// (all of a thread's loads of a round are issued before the first is stored)
__global__ void __launch_bounds__(RS_THREADS) k_router_grad_small(RouterSmallArgs a) {
    pdl_begin();
    extern __shared__ __align__(16) uint8_t rs_raw[];
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && tid == 0) *a.flag = 0;
    if ((int)blockIdx.x < a.w_ctas) {
        RouterSmallW& s = reinterpret_cast<RouterSmallShared*>(rs_raw)->w;
        const int e0 = RS_WE * ((int)blockIdx.x / a.w_cols), h0 = RS_WH * ((int)blockIdx.x % a.w_cols);
        const bool vec = (a.E & 3) == 0;
        constexpr int ND = RS_T * (RS_WE / 4) / RS_THREADS, NX = RS_T * (RS_WH / 8) / RS_THREADS;
        // experts 4 (tid / 16) .. + 3, columns 4 (tid % 16) .. + 3
        const int me = 4 * (tid >> 4), mc = 4 * (tid & 15);
        const bool sums = a.db && h0 == 0 && tid < RS_WE && e0 + tid < a.E;
        f32x2 acc[4][2] = {};
        float bias = 0.0f;
        float4 d[ND];
        uint4 xq[NX];
        uint32_t xf[NX];
        auto fetch = [&](int t0) {
#pragma unroll
            for (int u = 0; u < ND; ++u) {
                const int i = tid + u * RS_THREADS, t = t0 + i / (RS_WE / 4), e = 4 * (i % (RS_WE / 4));
                d[u] = rs_load4(a.dl + (size_t)t * a.E + e0 + e, t < a.T ? a.E - e0 - e : 0, vec);
            }
#pragma unroll
            for (int u = 0; u < NX; ++u) {
                const int i = tid + u * RS_THREADS, t = t0 + i / (RS_WH / 8), c = 8 * (i % (RS_WH / 8));
                xq[u] = make_uint4(0u, 0u, 0u, 0u);
                xf[u] = 0u;
                if (a.dw && t < a.T && h0 + c < a.H) {
                    const size_t at = (size_t)t * a.H + h0 + c;
                    if (a.x) {
                        xq[u] = __ldg(reinterpret_cast<const uint4*>(a.x + at));
                    } else {
                        const uint2 q = __ldg(reinterpret_cast<const uint2*>(a.codes + at));
                        xq[u].x = q.x;
                        xq[u].y = q.y;
                        xf[u] = __ldg(a.scales + (at >> 7));
                    }
                }
            }
        };
        fetch(0);
        for (int t0 = 0; t0 < a.T; t0 += RS_T) {
            if (t0) __syncthreads();
#pragma unroll
            for (int u = 0; u < ND; ++u) {
                const int i = tid + u * RS_THREADS;
                *reinterpret_cast<float4*>(&s.d[i / (RS_WE / 4)][4 * (i % (RS_WE / 4))]) = d[u];
            }
#pragma unroll
            for (int u = 0; u < NX; ++u) {
                const int i = tid + u * RS_THREADS, t = i / (RS_WH / 8), c = 8 * (i % (RS_WH / 8));
                float v[8];
                if (a.x)
                    bf16x8_values(xq[u], v);
                else
                    ckpt_values8(make_uint2(xq[u].x, xq[u].y), ckpt_scale(xf[u]), v);
                *reinterpret_cast<float4*>(&s.x[t][c]) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(&s.x[t][c + 4]) = make_float4(v[4], v[5], v[6], v[7]);
            }
            __syncthreads();
            const int n = min(RS_T, a.T - t0);
            if (t0 + RS_T < a.T) fetch(t0 + RS_T);       // (in flight during the products)
            if (sums)
                for (int t = 0; t < n; ++t) bias += s.d[t][tid];
            if (a.dw)
#pragma unroll 8
                for (int t = 0; t < n; ++t) {
                    const float4 dl = *reinterpret_cast<const float4*>(&s.d[t][me]);
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&s.x[t][mc]);
                    const float dv[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x2 two = rs_twice(dv[i]);
                        rs_fma2(acc[i][0], two, v.x);
                        rs_fma2(acc[i][1], two, v.y);
                    }
                }
        }
        if (sums) {
            float* o = a.db + e0 + tid;
            *o = a.accumulate ? *o + bias : bias;
        }
        if (!a.dw) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e0 + me + i < a.E && h0 + mc < a.H) {
                float4* o = reinterpret_cast<float4*>(a.dw + (size_t)(e0 + me + i) * a.H + h0 + mc);
                float4 v = rs_four(acc[i][0], acc[i][1]);
                if (a.accumulate) {
                    const float4 b = *o;
                    v = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
                }
                *o = v;
            }
        return;
    }
    RouterSmallX& s = reinterpret_cast<RouterSmallShared*>(rs_raw)->x;
    const int b = blockIdx.x - a.w_ctas, cols = a.H / RS_XH;
    const int t0 = RS_XT * (b / cols), h0 = RS_XH * (b % cols);
    // group g = tid / 64: experts RS_XE / 4 g .. of a round; in it tokens
    // (tid / 8 % 8) + 8 i, columns 4 (tid % 8) .. + 3
    const int g = tid >> 6, dt = (tid >> 3) & 7, dc = 4 * (tid & 7);
    f32x2 acc[4][2] = {};
    for (int e0 = 0; e0 < a.E; e0 += RS_XE) {
        const int n = min(RS_XE, a.E - e0), n4 = (n + 3) & ~3;      // (what lies behind n is zeros)
        if (e0) __syncthreads();
        const bool vec = (a.E & 3) == 0;
        constexpr int NW = RS_XE * (RS_XH / 4) / RS_THREADS, ND = RS_XT * (RS_XE / 4) / RS_THREADS;
        float4 wv[NW], d[ND];
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const int i = tid + u * RS_THREADS, e = i / (RS_XH / 4), c = 4 * (i % (RS_XH / 4));
            wv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e < n) wv[u] = __ldg(reinterpret_cast<const float4*>(a.w + (size_t)(e0 + e) * a.H + h0 + c));
        }
#pragma unroll
        for (int u = 0; u < ND; ++u) {
            const int i = tid + u * RS_THREADS, t = i / (RS_XE / 4), e = 4 * (i % (RS_XE / 4));
            d[u] = rs_load4(a.dl + (size_t)(t0 + t) * a.E + e0 + e, t0 + t < a.T ? n - e : 0, vec);
        }
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const int i = tid + u * RS_THREADS;
            *reinterpret_cast<float4*>(&s.w[i / (RS_XH / 4)][4 * (i % (RS_XH / 4))]) = wv[u];
        }
#pragma unroll
        for (int u = 0; u < ND; ++u) {
            const int i = tid + u * RS_THREADS;
            *reinterpret_cast<float4*>(&s.d[i / (RS_XE / 4)][4 * (i % (RS_XE / 4))]) = d[u];
        }
        __syncthreads();
        const int lo = g * (RS_XE / 4), hi = min(n4, lo + RS_XE / 4);
#pragma unroll 2
        for (int e = lo; e < hi; e += 4) {
            ulonglong2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const ulonglong2*>(&s.w[e + j][dc]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 d = *reinterpret_cast<const float4*>(&s.d[dt + 8 * i][e]);
                const float dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2 two = rs_twice(dv[j]);
                    rs_fma2(acc[i][0], two, v[j].x);
                    rs_fma2(acc[i][1], two, v[j].y);
                }
            }
        }
    }
    // the groups' sums, added in order
    __syncthreads();
    float4(*part)[RS_XT][RS_XH / 4] = reinterpret_cast<float4(*)[RS_XT][RS_XH / 4]>(rs_raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) part[g][dt + 8 * i][tid & 7] = rs_four(acc[i][0], acc[i][1]);
    __syncthreads();
    const int t = tid >> 3;
    if (t0 + t < a.T) {
        float4 v = part[0][t][tid & 7];
#pragma unroll
        for (int q = 1; q < 4; ++q) {
            const float4 u = part[q][t][tid & 7];
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        *reinterpret_cast<uint2*>(a.dx + (size_t)(t0 + t) * a.H + h0 + dc) =
            make_uint2(bf16x2_rn(v.x, v.y), bf16x2_rn(v.z, v.w));
    }
}

cudaError_t launch_router_grad_small(const float* dl, const void* x, const uint8_t* codes, const uint8_t* scales,
                                     const float* w, int T, int H, int E, void* dx, float* dw, float* db,
                                     int accumulate, int32_t* flag, cudaStream_t st) {
    static PerContext cache;
    const int ok = cache.get([] {
        return cudaFuncSetAttribute(k_router_grad_small, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(RouterSmallShared)) == cudaSuccess
                   ? 1
                   : -1;
    });
    if (ok < 0) return cudaErrorInvalidValue;
    const int rows = (E + RS_WE - 1) / RS_WE, cols = dw ? (H + RS_WH - 1) / RS_WH : 1;
    RouterSmallArgs a{dl, (const __nv_bfloat16*)x, codes, scales, w, T, H, E, (__nv_bfloat16*)dx, dw, db, accumulate,
                      dw || db ? rows * cols : 0, cols, flag};
    const int x_ctas = dx ? (T + RS_XT - 1) / RS_XT * (H / RS_XH) : 0;
    const cudaError_t e = launch_pdl(k_router_grad_small, dim3((unsigned)(a.w_ctas + x_ctas)), dim3(RS_THREADS),
                                     sizeof(RouterSmallShared), st, a);
    count_launches(1);
    return e;
}

}  // namespace moe
