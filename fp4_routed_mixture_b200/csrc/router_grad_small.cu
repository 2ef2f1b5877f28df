// Gradients of the router projection for few tokens (router_grad_small in
// kernels.cuh says which calls), in one launch:
//   dw[e, h] = sum_t dl[t, e] x[t, h],  dx[t, h] = sum_e dl[t, e] w[e, h],
//   dbias[e] = sum_t dl[t, e]
// The same products of bf16 parts as grad_gemm.cu's: dl in three parts for dw
// (exact), dl and w in two each for dx (three products).  That form takes three
// launches, each mostly latency at these sizes, and its 256 x 256 tiles would be
// a few CTAs' work: here the tiles are small and the CTAs many, a warp multiplies
// 16 x 32 of a tile with mma.sync (48 of them in a round of dw; they are no bound).
// fp32 multiply-adds instead were bound by their rate: 11.4 us for 64 tokens.
// The grid's first CTAs take dw in tiles of 64 experts x 64 columns (and dbias), 64
// tokens a round, the others dx in tiles of 32 tokens x 32 columns, 128 experts a
// round, four pairs of warps a quarter of them each.  A round's loads are in flight
// during the products of the round in front.
// One B200, 256 experts, H = 4096: 5.8 us for one token, 8.7 for 64, 12.6 for 128, of
// it about 2 for the launch and 2 of instructions, most of them the split into parts.
// (Other rounds and three to five CTAs per SM: 8.1 to 13 us for 64 tokens, each better
// at one size and worse at another; rows of dw stored whole by each quad: the same.)
#include "bf16_parts.cuh"
#include "ckpt.cuh"
#include "kernels.cuh"
#include "moe_common.cuh"

namespace moe {

constexpr int RS_THREADS = 256;
constexpr int RS_WE = 64, RS_WH = 64, RS_T = 64;      // tile of dw, tokens per round
constexpr int RS_XT = 32, RS_XH = 32, RS_XE = 128;    // tile of dx, experts per round

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

// Rows padded so that the eight rows of a fragment lie in different banks.
struct RouterSmallW {
    __nv_bfloat16 x[RS_T][RS_WH + 8];
    __nv_bfloat16 d[3][RS_T][RS_WE + 8];
};
struct RouterSmallX {
    __nv_bfloat16 w[2][RS_XE][RS_XH + 8];
    __nv_bfloat16 d[2][RS_XT][RS_XE + 8];
};
union RouterSmallShared {
    RouterSmallW w;
    RouterSmallX x;
    float part[4][RS_XT][RS_XH + 8];
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

// Four fp32 values as bf16 parts, 8 bytes of each.
template <int PARTS>
__device__ __forceinline__ void rs_split4(float4 v, uint2 (&p)[PARTS]) {
    uint32_t h[2], m[2], l[2];
    split3x2(v.x, v.y, h[0], m[0], l[0]);
    split3x2(v.z, v.w, h[1], m[1], l[1]);
    p[0] = make_uint2(h[0], h[1]);
    p[1] = make_uint2(m[0], m[1]);
    if (PARTS == 3) p[PARTS - 1] = make_uint2(l[0], l[1]);
}

// Four 8 x 8 matrices of bf16, lane i giving row i % 8 of matrix i / 8.
template <bool TRANS>
__device__ __forceinline__ void rs_ldm(uint32_t (&r)[4], const __nv_bfloat16* row) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(row);
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void rs_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (a round's loads are issued together, before the products of the round in front)
__global__ void __launch_bounds__(RS_THREADS, 3) k_router_grad_small(RouterSmallArgs a) {
    pdl_begin();
    __shared__ __align__(16) RouterSmallShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && tid == 0) *a.flag = 0;
    const bool vec = (a.E & 3) == 0;
    // lane's row and column in a 16 x 16 block of four matrices: the second
    // matrix below the first (lo) or beside it (hi)
    const int lo = lane & 15, lc = 8 * (lane >> 4), hi = (lane & 7) + 8 * (lane >> 4), hc = 8 * (lane >> 3 & 1);
    float acc[4][4] = {};
    if ((int)blockIdx.x < a.w_ctas) {
        RouterSmallW& s = sh.w;
        const int e0 = RS_WE * ((int)blockIdx.x / a.w_cols), h0 = RS_WH * ((int)blockIdx.x % a.w_cols);
        constexpr int ND = RS_T * (RS_WE / 4) / RS_THREADS, NX = RS_T * (RS_WH / 8) / RS_THREADS;
        // a warp's experts and columns of the tile
        const int me = 16 * (warp & 3), mc = 32 * (warp >> 2);
        const bool sums = a.db && h0 == 0 && tid < RS_WE && e0 + tid < a.E;
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
                uint2 p[3];
                rs_split4(d[u], p);
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *reinterpret_cast<uint2*>(&s.d[q][i / (RS_WE / 4)][4 * (i % (RS_WE / 4))]) = p[q];
            }
#pragma unroll
            for (int u = 0; u < NX; ++u) {
                const int i = tid + u * RS_THREADS, t = i / (RS_WH / 8), c = 8 * (i % (RS_WH / 8));
                if (!a.x) {
                    float v[8];
                    ckpt_values8(make_uint2(xq[u].x, xq[u].y), ckpt_scale(xf[u]), v);
                    xq[u] = bf16x8_rn(v);
                }
                *reinterpret_cast<uint4*>(&s.x[t][c]) = xq[u];
            }
            __syncthreads();
            if (t0 + RS_T < a.T) fetch(t0 + RS_T);
            const int n = min(RS_T, a.T - t0);
            if (sums)
#pragma unroll 8
                for (int t = 0; t < n; ++t)      // (the parts' sum is the value)
                    bias += (__bfloat162float(s.d[0][t][tid]) + __bfloat162float(s.d[1][t][tid])) +
                            __bfloat162float(s.d[2][t][tid]);
            if (a.dw)
#pragma unroll
                for (int k = 0; k < RS_T; k += 16) {
                    if (k >= n) break;
                    uint32_t b0[4], b1[4];
                    rs_ldm<true>(b0, &s.x[k + lo][mc + lc]);
                    rs_ldm<true>(b1, &s.x[k + lo][mc + 16 + lc]);
#pragma unroll
                    for (int q = 2; q >= 0; --q) {
                        uint32_t f[4];
                        rs_ldm<true>(f, &s.d[q][k + hi][me + hc]);
                        rs_mma(acc[0], f, b0[0], b0[1]);
                        rs_mma(acc[1], f, b0[2], b0[3]);
                        rs_mma(acc[2], f, b1[0], b1[1]);
                        rs_mma(acc[3], f, b1[2], b1[3]);
                    }
                }
        }
        if (sums) {
            float* o = a.db + e0 + tid;
            *o = a.accumulate ? *o + bias : bias;
        }
        if (!a.dw) return;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int e = e0 + me + 8 * r + (lane >> 2);
            if (e >= a.E) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = h0 + mc + 8 * j + 2 * (lane & 3);
                if (c >= a.H) continue;
                float2* o = reinterpret_cast<float2*>(a.dw + (size_t)e * a.H + c);
                float2 v = make_float2(acc[j][2 * r], acc[j][2 * r + 1]);
                if (a.accumulate) {
                    const float2 b = *o;
                    v = make_float2(b.x + v.x, b.y + v.y);
                }
                *o = v;
            }
        }
        return;
    }
    RouterSmallX& s = sh.x;
    const int b = blockIdx.x - a.w_ctas, cols = a.H / RS_XH;
    const int t0 = RS_XT * (b / cols), h0 = RS_XH * (b % cols);
    // a warp's tokens of the tile, and its quarter of a round's experts
    const int mt = 16 * (warp & 1), g = warp >> 1;
    constexpr int NW = RS_XE * (RS_XH / 4) / RS_THREADS, ND = RS_XT * (RS_XE / 4) / RS_THREADS;
    float4 wv[NW], d[ND];
    auto fetch = [&](int e0) {
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const int i = tid + u * RS_THREADS, e = e0 + i / (RS_XH / 4), c = 4 * (i % (RS_XH / 4));
            wv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e < a.E) wv[u] = __ldg(reinterpret_cast<const float4*>(a.w + (size_t)e * a.H + h0 + c));
        }
#pragma unroll
        for (int u = 0; u < ND; ++u) {
            const int i = tid + u * RS_THREADS, t = t0 + i / (RS_XE / 4), e = e0 + 4 * (i % (RS_XE / 4));
            d[u] = rs_load4(a.dl + (size_t)t * a.E + e, t < a.T ? a.E - e : 0, vec);
        }
    };
    fetch(0);
    for (int e0 = 0; e0 < a.E; e0 += RS_XE) {
        if (e0) __syncthreads();
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const int i = tid + u * RS_THREADS;
            uint2 p[2];
            rs_split4(wv[u], p);
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *reinterpret_cast<uint2*>(&s.w[q][i / (RS_XH / 4)][4 * (i % (RS_XH / 4))]) = p[q];
        }
#pragma unroll
        for (int u = 0; u < ND; ++u) {
            const int i = tid + u * RS_THREADS;
            uint2 p[2];
            rs_split4(d[u], p);
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *reinterpret_cast<uint2*>(&s.d[q][i / (RS_XE / 4)][4 * (i % (RS_XE / 4))]) = p[q];
        }
        __syncthreads();
        if (e0 + RS_XE < a.E) fetch(e0 + RS_XE);
#pragma unroll
        for (int k = g * (RS_XE / 4); k < (g + 1) * (RS_XE / 4); k += 16) {
            if (e0 + k >= a.E) break;
            uint32_t f[2][4], w0[2][4], w1[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                rs_ldm<false>(f[q], &s.d[q][mt + lo][k + lc]);
                rs_ldm<true>(w0[q], &s.w[q][k + lo][lc]);
                rs_ldm<true>(w1[q], &s.w[q][k + lo][16 + lc]);
            }
            auto product = [&](int i, int j) {
                rs_mma(acc[0], f[i], w0[j][0], w0[j][1]);
                rs_mma(acc[1], f[i], w0[j][2], w0[j][3]);
                rs_mma(acc[2], f[i], w1[j][0], w1[j][1]);
                rs_mma(acc[3], f[i], w1[j][2], w1[j][3]);
            };
            product(1, 0);
            product(0, 1);
            product(0, 0);
        }
    }
    // the quarters' sums, added in order
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(&sh.part[g][mt + 8 * r + (lane >> 2)][8 * j + 2 * (lane & 3)]) =
                make_float2(acc[j][2 * r], acc[j][2 * r + 1]);
    __syncthreads();
    const int t = tid >> 3, c = 4 * (tid & 7);
    if (t0 + t < a.T) {
        float4 v = *reinterpret_cast<const float4*>(&sh.part[0][t][c]);
#pragma unroll
        for (int q = 1; q < 4; ++q) {
            const float4 u = *reinterpret_cast<const float4*>(&sh.part[q][t][c]);
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        *reinterpret_cast<uint2*>(a.dx + (size_t)(t0 + t) * a.H + h0 + c) =
            make_uint2(bf16x2_rn(v.x, v.y), bf16x2_rn(v.z, v.w));
    }
}

cudaError_t launch_router_grad_small(const float* dl, const void* x, const uint8_t* codes, const uint8_t* scales,
                                     const float* w, int T, int H, int E, void* dx, float* dw, float* db,
                                     int accumulate, int32_t* flag, cudaStream_t st) {
    const int rows = (E + RS_WE - 1) / RS_WE, cols = dw ? (H + RS_WH - 1) / RS_WH : 1;
    RouterSmallArgs a{dl, (const __nv_bfloat16*)x, codes, scales, w, T, H, E, (__nv_bfloat16*)dx, dw, db, accumulate,
                      dw || db ? rows * cols : 0, cols, flag};
    const int x_ctas = dx ? (T + RS_XT - 1) / RS_XT * (H / RS_XH) : 0;
    const cudaError_t e = launch_pdl(k_router_grad_small, dim3((unsigned)(a.w_ctas + x_ctas)), dim3(RS_THREADS),
                                     0, st, a);
    count_launches(1);
    return e;
}

}  // namespace moe
