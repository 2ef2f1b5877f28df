// Gradient products: the weight gradient of a projection from an 8-bit
// checkpoint of its input (dense, or one per expert), and the gradients of the
// router projection.  Formulas at moe_ckpt_wgrad and
// moe_router_logits_backward in the header.
//
// All are C[m, n] = sum_r A[r, m] B[r, n] over rows r.  This form runs on the
// CUDA cores: 64 x 64 outputs per CTA, 16 rows per step, fp32 fused
// multiply-adds in ascending r.
#include "ckpt.cuh"
#include "kernels.cuh"
#include "moe_common.cuh"

namespace moe {

constexpr int kGradT = 64, kGradK = 16;

struct Bf16Rows {          // v[r, c] of a bf16 matrix
    const __nv_bfloat16* p;
    long long ld;
    __device__ float operator()(int r, int c) const { return __bfloat162float(p[r * ld + c]); }
};
struct F32Rows {
    const float* p;
    long long ld;
    __device__ float operator()(int r, int c) const { return p[r * ld + c]; }
};
struct F32Cols {           // the transpose of a row-major matrix
    const float* p;
    long long ld;
    __device__ float operator()(int r, int c) const { return p[c * ld + r]; }
};
struct CkptRows {          // a checkpoint's rows, through perm[r] / k when given
    const uint8_t* codes;
    const uint8_t* scales;
    const int32_t* perm;
    int k, rows, K;
    int32_t* flag;
    __device__ float operator()(int r, int c) const {
        const int t = perm ? checked_index(perm[r] / k, rows, flag) : r;
        return e4m3x2_value(codes[(size_t)t * K + c]).x * ckpt_scale(scales[(size_t)t * (K / 128) + c / 128]);
    }
};
struct StoreF32 {
    float* p;
    long long ld, group;
    int accumulate;
    __device__ void operator()(int g, int m, int n, float v) const {
        float* d = p + g * group + m * ld + n;
        *d = accumulate ? *d + v : v;
    }
};
struct StoreBf16 {
    __nv_bfloat16* p;
    long long ld;
    __device__ void operator()(int, int m, int n, float v) const { p[m * ld + n] = __float2bfloat16_rn(v); }
};

template <class A, class B, class C>
__global__ void __launch_bounds__(256) k_grad_simt(A a, B b, C c, const int32_t* offsets, int R, int M, int N) {
    pdl_begin();
    __shared__ float as[kGradK][kGradT + 4], bs[kGradK][kGradT + 4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int n0 = blockIdx.x * kGradT, m0 = blockIdx.y * kGradT, g = blockIdx.z;
    const int r0 = offsets ? min(max(offsets[g], 0), R) : 0;
    const int r1 = offsets ? min(max(offsets[g + 1], 0), R) : R;
    float acc[4][4] = {};
    for (int r = r0; r < r1; r += kGradK) {
        for (int i = tid; i < kGradK * kGradT; i += 256) {
            const int rr = i / kGradT, cc = i % kGradT;
            as[rr][cc] = (r + rr < r1 && m0 + cc < M) ? a(r + rr, m0 + cc) : 0.0f;
            bs[rr][cc] = (r + rr < r1 && n0 + cc < N) ? b(r + rr, n0 + cc) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kGradK; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(as[kk][ty + 16 * i], bs[kk][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (m0 + ty + 16 * i < M && n0 + tx + 16 * j < N) c(g, m0 + ty + 16 * i, n0 + tx + 16 * j, acc[i][j]);
}

// First kernel of a call: clears the error word, or raises FLAG_BOUNDS there
// when the group offsets do not ascend within [0, R].
__global__ void __launch_bounds__(1024) k_grad_head(const int32_t* offsets, int G, int R, int32_t* flag) {
    pdl_begin();
    bool bad = false;
    if (offsets)
        for (int g = threadIdx.x; g < G; g += blockDim.x)
            bad |= offsets[g] < 0 || offsets[g + 1] < offsets[g] || offsets[g + 1] > R;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *flag = bad ? FLAG_BOUNDS : 0;
}

// Column sums of dl [T, E]: CTA per 32 columns, warps stride the rows, the
// warps' sums are added in order.
__global__ void __launch_bounds__(1024) k_grad_bias(const float* __restrict__ dl, int T, int E, float* db,
                                                    int accumulate) {
    pdl_begin();
    __shared__ float s[32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (e < E)
        for (int t = warp; t < T; t += 32) v += __ldg(dl + (size_t)t * E + e);
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && e < E) {
        v = 0.0f;
        for (int w = 0; w < 32; ++w) v += s[w][lane];
        db[e] = accumulate ? db[e] + v : v;
    }
}

size_t wgrad_workspace_bytes(int, int, int, int) { return 256; }
size_t router_backward_workspace_bytes(int, int, int) { return 256; }

static dim3 grad_grid(int M, int N, int G) {
    return dim3((unsigned)((N + kGradT - 1) / kGradT), (unsigned)((M + kGradT - 1) / kGradT), (unsigned)G);
}

cudaError_t launch_ckpt_wgrad(const void* dy, long long lddy, const uint8_t* codes, const uint8_t* scales,
                              const int32_t* offsets, const int32_t* perm, int k, int R, int rows, int N, int K, int G,
                              float* dw, int accumulate, void* ws, uint64_t, cudaStream_t st) {
    int32_t* flag = (int32_t*)ws;
    cudaError_t e = launch_pdl(k_grad_head, dim3(1), dim3(1024), 0, st, offsets, G, R, flag);
    count_launches(1);
    if (e != cudaSuccess) return e;
    const Bf16Rows a{(const __nv_bfloat16*)dy, lddy};
    const CkptRows b{codes, scales, perm, k, rows, K, flag};
    const StoreF32 c{dw, K, (long long)N * K, accumulate};
    e = launch_pdl(k_grad_simt<Bf16Rows, CkptRows, StoreF32>, grad_grid(N, K, G), dim3(256), 0, st, a, b, c, offsets,
                   R, N, K);
    count_launches(1);
    return e;
}

cudaError_t launch_router_backward(const float* dl, const void* x, const uint8_t* codes, const uint8_t* scales,
                                   const float* w, int T, int H, int E, void* dx, float* dw, float* db, int accumulate,
                                   void* ws, uint64_t, cudaStream_t st) {
    int32_t* flag = (int32_t*)ws;
    cudaError_t e = launch_pdl(k_grad_head, dim3(1), dim3(1024), 0, st, (const int32_t*)nullptr, 0, 0, flag);
    count_launches(1);
    if (e == cudaSuccess && dw) {
        const F32Rows a{dl, E};
        const StoreF32 c{dw, H, 0, accumulate};
        if (x)
            e = launch_pdl(k_grad_simt<F32Rows, Bf16Rows, StoreF32>, grad_grid(E, H, 1), dim3(256), 0, st, a,
                           Bf16Rows{(const __nv_bfloat16*)x, H}, c, (const int32_t*)nullptr, T, E, H);
        else
            e = launch_pdl(k_grad_simt<F32Rows, CkptRows, StoreF32>, grad_grid(E, H, 1), dim3(256), 0, st, a,
                           CkptRows{codes, scales, nullptr, 1, T, H, flag}, c, (const int32_t*)nullptr, T, E, H);
        count_launches(1);
    }
    if (e == cudaSuccess && dx && T > 0) {
        e = launch_pdl(k_grad_simt<F32Cols, F32Rows, StoreBf16>, grad_grid(T, H, 1), dim3(256), 0, st, F32Cols{dl, E},
                       F32Rows{w, H}, StoreBf16{(__nv_bfloat16*)dx, H}, (const int32_t*)nullptr, E, T, H);
        count_launches(1);
    }
    if (e == cudaSuccess && db) {
        e = launch_pdl(k_grad_bias, dim3((unsigned)((E + 31) / 32)), dim3(1024), 0, st, dl, T, E, db, accumulate);
        count_launches(1);
    }
    return e;
}

}  // namespace moe
