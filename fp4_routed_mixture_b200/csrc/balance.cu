// Load-balance loss of the router with its per-expert counts, and the gradient
// of the logits (formulas at moe_balance_loss and moe_route_backward in the
// header).
//
//   k_balance_rows    softmax of every row; per chunk of rows and sequence the
//                     sum of the probabilities, the counts and the valid tokens
//   k_balance_reduce  adds the chunks of each sequence in a fixed order, forms
//                     f and P, and (last CTA) the loss
//   k_route_backward  one pass: recomputes each row's softmax and writes the
//                     gradient of the balance loss and of the gates
//
// A chunk c of rows and a sequence s that meet own slot c + s of the
// workspace: walking the rows, every step to the next (chunk, sequence) pair
// raises c, s or both, so the sum is unique, and chunks + S slots are enough
// for any ragged split.  No two additions to one address race: results do not
// depend on the order in which CTAs run.
// All three read [T, E] once (the backward also writes it).  One B200, 65536 x 256
// logits in 16 sequences: loss 22 us (20 where they lie in L2), of it 10 that 4604
// rows take too (two launches, their first loads, the sum of the chunks); 2 to 6 rows
// per warp in flight through shared memory, other block sizes and more blocks
// measured the same or more.  Gradient 28 us (134 MB, 4.8 TB/s).
#include "kernels.cuh"
#include "moe_common.cuh"

namespace moe {

// k_balance_rows: 2 CTAs per SM up to 256 experts (64 registers at most); above,
// 106 to 125 registers leave room for one, and the chunks run in two waves.
constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalMaxChunks = 148 * 2;
constexpr int kRedThreads = 1024, kRedWarps = kRedThreads / 32;
// Calls of at most this many rows and sequences run in one CTA and launch, which
// walks the sequences one after the other (1.2 us each at 256 logits, 2.5 at 1024):
// less time where they are few.  Measured (us, one launch / two; 256 logits): 8 rows, 1
// sequence 2.9 / 7.6, 4 sequences 6.6 / 10.9; 32 rows, 4 7.1 / 8.8, 16 21.9 / 15.9; 128 rows,
// 1 6.3 / 7.4, 4 9.7 / 7.6, 16 24 / 8.9, 64 83 / 23; 1024 logits, 128 rows, 1 11.3 / 9.1, 64
// 163 / 59.  So above 4 to 8 sequences, and for 128 rows of 1024 logits, two launches
// would take less: the bounds are higher than they should be.
constexpr int kBalSingleT = 128, kBalSingleS = 64;

struct BalanceWs {
    size_t meta, prob, hits, part, total;
    int slots;
};

static int bal_chunk_rows(int T) {
    return std::max(kBalWarps, (int)align_up((size_t)(T + kBalMaxChunks - 1) / kBalMaxChunks, kBalWarps));
}

static BalanceWs balance_ws(int T, int E, int S) {
    BalanceWs L;
    // (the chunk count is not monotonic in T; this bound is)
    const int chunks = std::min(kBalMaxChunks, (T + kBalWarps - 1) / kBalWarps);
    L.slots = chunks + S;
    size_t o = 256;   // error word, arrival counter
    L.meta = o; o += align_up(sizeof(int2) * (size_t)L.slots, 256);
    L.prob = o; o += align_up(sizeof(float) * (size_t)L.slots * E, 256);
    L.hits = o; o += align_up(sizeof(int) * (size_t)L.slots * E, 256);
    L.part = o; o += align_up(sizeof(float) * (size_t)S * ((E + 31) / 32), 256);
    L.total = o;
    return L;
}

size_t balance_workspace_bytes(int T, int E, int S) { return balance_ws(T, E, S).total; }

// Sequence bounds read from the caller's table (NULL: one sequence of T rows),
// clamped so that a bad table cannot lead out of the tensors.
struct SeqTable {
    const int32_t* off;
    int T, S;
    __device__ int at(int s) const {
        if (!off) return s == 0 ? 0 : T;
        return min(max(__ldg(off + s), 0), T);
    }
    // The first sequence that ends behind row r (S when none does); by a whole
    // warp, 32 bounds at a time (one after the other they cost 0.6 us each).
    __device__ int find(int r) const {
        const int lane = threadIdx.x & 31;
        int lo = 0, hi = S;                  // the answer lies in [lo, hi]
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32, s = min(lo + (lane + 1) * step - 1, hi - 1);
            const uint32_t m = __ballot_sync(0xffffffffu, at(s + 1) > r);
            if (m == 0) return hi;
            const int first = __ffs((int)m) - 1;
            hi = min(lo + (first + 1) * step - 1, hi - 1);
            lo += first * step;
        }
        return lo;
    }
    // sequence s does not ascend within [0, T]
    __device__ bool bad(int s) const {
        if (!off) return false;
        const int b = __ldg(off + s), e = __ldg(off + s + 1);
        return b < 0 || e > T || e < b;
    }
};

// Column of a lane's value v: four neighbours per 128 columns (VEC, one
// 16-byte access) or every 32nd column.
template <bool VEC>
__device__ __forceinline__ int bal_col(int v, int lane) {
    return VEC ? ((v >> 2) * 128 + lane * 4 + (v & 3)) : (v * 32 + lane);
}

template <int N, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float (&x)[N]) {
    if (VEC) {
#pragma unroll
        for (int v = 0; v < N; v += 4) {
            const int c = bal_col<true>(v, lane);
            float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (c < E) q = __ldg(reinterpret_cast<const float4*>(row + c));
            x[v] = q.x; x[v + 1] = q.y; x[v + 2] = q.z; x[v + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int c = bal_col<false>(v, lane);
            x[v] = c < E ? __ldg(row + c) : -INFINITY;
        }
    }
}

// 2^x, within 2 ulp; below 2^-126: 0.
__device__ __forceinline__ float bal_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x <- exp(x - max) of the row the warp holds (columns behind E hold -inf and
// get 0); returns this lane's part of their sum.  NaN is the maximum where the
// row has one, so such a row becomes NaN; +inf - +inf does the same.  A row of
// -inf alone has no distribution: all 0.  The difference is taken before the
// factor log2(e): two roundings of it, |x - max| 2^-24 each.
template <int N>
__device__ __forceinline__ float row_exp(float (&x)[N]) {
    float m = x[0];
#pragma unroll
    for (int v = 1; v < N; ++v) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(x[v]));
    asm volatile("redux.sync.max.NaN.f32 %0, %0, 0xffffffff;" : "+f"(m));
    const bool none = m == -INFINITY;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < N; ++v) {
        x[v] = none ? 0.0f : bal_exp2((x[v] - m) * 1.44269502162933349609375f);
        sum += x[v];
    }
    return sum;
}
__device__ __forceinline__ float row_inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

struct BalanceArgs {
    const float* logits;
    const int32_t* idx;
    const uint8_t* mask;
    SeqTable seq;
    int T, E, k, rows;      // rows per chunk
    float coef;
    int32_t* head;          // error word, arrival counter
    int2* meta;             // per slot: valid tokens, error bits
    float* prob;            // [slots, E]
    int* hits;              // [slots, E]
    float* part;            // [S][column blocks]
    int32_t* counts;
    float* mean_prob;       // or NULL
    int32_t* tokens;        // [S + 1]
    float* loss;
};

// ONE: a single CTA has all rows and gives the results itself.
template <int N, bool VEC, bool ONE>
__global__ void __launch_bounds__(kBalThreads) k_balance_rows(BalanceArgs a) {
    pdl_begin();
    extern __shared__ float bal_smem[];
    float* sp = bal_smem;                                           // [warps][E]
    int* sc = reinterpret_cast<int*>(bal_smem + kBalWarps * a.E);   // [E]
    __shared__ int s_n, s_bad;
    __shared__ double s_sum[kBalWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!ONE && blockIdx.x == 0 && threadIdx.x == 0) a.head[0] = a.head[1] = 0;
    const int r0 = blockIdx.x * a.rows, r1 = min(a.T, r0 + a.rows);
    double total = 0.0;       // ONE: this thread's part of the loss's sum
    int used = 0, errors = 0;
    for (int s = ONE ? 0 : a.seq.find(r0); s < a.seq.S; ++s) {
        if (!ONE && a.seq.at(s) >= r1) break;
        const int b = max(a.seq.at(s), r0), e = min(a.seq.at(s + 1), r1);
        if (!ONE && e <= b) {
            s = max(s, a.seq.find(b) - 1);       // (past a run of empty ones)
            continue;
        }
        for (int c = threadIdx.x; c < a.E; c += kBalThreads) sc[c] = 0;
        if (threadIdx.x == 0) s_n = s_bad = 0;
        __syncthreads();
        float acc[N] = {};
        float nx[N];
        int nid = -1, non = 1;
        // a row's logits, ids and mask are loaded one row ahead
        auto fetch = [&](int r) {
            load_row<N, VEC>(a.logits + (size_t)r * a.E, a.E, lane, nx);
            if (lane < a.k) nid = __ldg(a.idx + (size_t)r * a.k + lane);
            if (a.mask) non = __ldg(a.mask + r);
        };
        if (b + warp < e) fetch(b + warp);
        int n = 0;
        for (int r = b + warp; r < e; r += kBalWarps) {
            float x[N];
#pragma unroll
            for (int v = 0; v < N; ++v) x[v] = nx[v];
            const int id = nid;
            const bool on = non != 0;
            if (r + kBalWarps < e) fetch(r + kBalWarps);
            if (!on) continue;
            ++n;
            const float inv = row_inverse(warp_sum(row_exp<N>(x)));
#pragma unroll
            for (int v = 0; v < N; ++v) acc[v] = fmaf(x[v], inv, acc[v]);
            if (lane < a.k) {
                if ((unsigned)id < (unsigned)a.E)
                    atomicAdd(sc + id, 1);
                else
                    s_bad = FLAG_BAD_EXPERT;
            }
        }
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int c = bal_col<VEC>(v, lane);
            if (c < a.E) sp[warp * a.E + c] = acc[v];
        }
        if (lane == 0) atomicAdd(&s_n, n);
        __syncthreads();
        const size_t slot = (size_t)blockIdx.x + s;
        const float inv_n = ONE && s_n > 0 ? 1.0f / (float)s_n : 0.0f;
        for (int c = threadIdx.x; c < a.E; c += kBalThreads) {
            float t = sp[c];
#pragma unroll
            for (int w = 1; w < kBalWarps; ++w) t += sp[w * a.E + c];
            if (ONE) {
                const float mp = t * inv_n;
                a.counts[(size_t)s * a.E + c] = sc[c];
                if (a.mean_prob) a.mean_prob[(size_t)s * a.E + c] = mp;
                total += (double)((float)sc[c] * ((float)a.E / (float)a.k * inv_n) * mp);
            } else {
                a.prob[slot * a.E + c] = t;
                a.hits[slot * a.E + c] = sc[c];
            }
        }
        if (threadIdx.x == 0) {
            if (ONE) {
                a.tokens[s] = s_n;
                used += s_n > 0;
                errors |= s_bad | (a.seq.bad(s) ? FLAG_BOUNDS : 0);
            } else {
                a.meta[slot] = make_int2(s_n, s_bad);
            }
        }
        __syncthreads();
    }
    if (ONE) {
        total = warp_sum(total);
        if (lane == 0) s_sum[warp] = total;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kBalWarps; ++w) total += s_sum[w];
            a.head[0] = errors;
            a.tokens[a.seq.S] = used;
            *a.loss = used > 0 ? (float)((double)a.coef * total / (double)used) : 0.0f;
        }
    }
}

// CTA (column block of 32, sequence): 32 warps take every 32nd chunk of the
// sequence, lane = column; the warps' sums are added in warp order.
__global__ void __launch_bounds__(kRedThreads) k_balance_reduce(BalanceArgs a) {
    pdl_begin();
    __shared__ float sp[kRedWarps][33];
    __shared__ int sc[kRedWarps][33];
    __shared__ int sn[kRedWarps];
    __shared__ bool s_last;
    __shared__ double sred[kRedWarps];
    __shared__ int sused[kRedWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int CB = (a.E + 31) / 32, cb = blockIdx.x, s = blockIdx.y;
    const int col = cb * 32 + lane;
    const int b = a.seq.at(s), e = a.seq.at(s + 1);
    if (threadIdx.x == 0 && cb == 0 && a.seq.bad(s)) raise_flag(a.head, FLAG_BOUNDS);
    const int c0 = b / a.rows, c1 = e > b ? (e - 1) / a.rows + 1 : c0;
    float p = 0.0f;
    int h = 0, n = 0, bad = 0;
#pragma unroll 4
    for (int c = c0 + warp; c < c1; c += kRedWarps) {
        const size_t slot = (size_t)c + s;
        const int2 m = a.meta[slot];
        n += m.x;
        bad |= m.y;
        if (col < a.E) {
            p += a.prob[slot * a.E + col];
            h += a.hits[slot * a.E + col];
        }
    }
    sp[warp][lane] = p;
    sc[warp][lane] = h;
    if (lane == 0) sn[warp] = n;
    // (with offsets that do not ascend a slot may be one that no chunk has written)
    bad &= FLAG_BAD_EXPERT;
    if (bad && lane == 0 && cb == 0) raise_flag(a.head, bad);
    __syncthreads();
    if (warp == 0) {
        n = 0;
        p = 0.0f;
        h = 0;
#pragma unroll 8
        for (int w = 0; w < kRedWarps; ++w) {
            n += sn[w];
            p += sp[w][lane];
            h += sc[w][lane];
        }
        float term = 0.0f;
        if (col < a.E) {
            const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
            const float mp = p * inv;
            a.counts[(size_t)s * a.E + col] = h;
            if (a.mean_prob) a.mean_prob[(size_t)s * a.E + col] = mp;
            term = (float)h * ((float)a.E / (float)a.k * inv) * mp;
        }
        term = warp_sum(term);
        if (lane == 0) {
            a.part[(size_t)s * CB + cb] = term;
            if (cb == 0) a.tokens[s] = n;
            __threadfence();
            s_last = atomicAdd(a.head + 1, 1) == (int)(gridDim.x * gridDim.y) - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    // the last CTA adds the terms (and counts the sequences in use) in a fixed order
    __threadfence();
    double sum = 0.0;
    int used = 0;
    const int total = a.seq.S * CB;
    for (int i = threadIdx.x; i < total; i += kRedThreads) sum += (double)__ldcg(a.part + i);
    for (int i = threadIdx.x; i < a.seq.S; i += kRedThreads) used += __ldcg(a.tokens + i) > 0;
    sum = warp_sum(sum);
    used = warp_sum(used);
    if (lane == 0) {
        sred[warp] = sum;
        sused[warp] = used;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
        used = 0;
        for (int w = 0; w < kRedWarps; ++w) {
            sum += sred[w];
            used += sused[w];
        }
        a.tokens[a.seq.S] = used;
        *a.loss = used > 0 ? (float)((double)a.coef * sum / (double)used) : 0.0f;
    }
}

// No tokens: every output is zero.  (The first CTA checks the offsets.)
__global__ void k_balance_empty(SeqTable seq, int32_t* head, int32_t* counts, float* mean_prob, int32_t* tokens,
                                float* loss, int E) {
    pdl_begin();
    const int S = seq.S;
    if (blockIdx.x == 0) {
        bool bad = false;
        for (int s = threadIdx.x; s < S; s += blockDim.x) bad |= seq.bad(s);
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *head = bad ? FLAG_BOUNDS : 0;
    }
    const size_t n = (size_t)S * E, i0 = blockIdx.x * (size_t)blockDim.x + threadIdx.x;
    for (size_t i = i0; i < n; i += (size_t)gridDim.x * blockDim.x) {
        counts[i] = 0;
        if (mean_prob) mean_prob[i] = 0.0f;
    }
    for (size_t i = i0; i <= (size_t)S; i += (size_t)gridDim.x * blockDim.x) tokens[i] = 0;
    if (i0 == 0) *loss = 0.0f;
}

// ---- gradient of the logits ----------------------------------------------------
struct RouteBackwardArgs {
    const float* logits;
    const int32_t* idx;
    const float* gates;
    const float* dgates;    // or NULL
    const float* dloss;     // or NULL
    const int32_t* counts;
    const int32_t* tokens;  // [S + 1]
    const uint8_t* mask;
    SeqTable seq;
    int T, E, k, rows;      // rows per warp
    float coef;
    float* dlogits;
    int32_t* flag;          // or NULL
};

// A warp takes `rows` consecutive rows, so that f of their sequence stays in
// registers until the sequence changes.  The balance term needs the softmax
// only through sum e and sum e f (e = exp(x - max)), reduced together.  The
// gates' terms are added to the stored row in memory: comparing each of the k
// ids with a lane's columns in registers took two thirds of the instructions.
// 65536 x 256 logits: 25 us (134 MB, 5.4 TB/s), 28 us with 6 gates a row; the
// terms through shared memory 7 us more, two or three rows loaded ahead 9.  What
// bounds it besides HBM is the grid: rows a warp are set for 48 warps per SM, but
// 64 registers let 32 run (E <= 256; 16 up to 512, 8 above), so that 16384 and 65536
// rows, 1024 blocks for 592 places, take 1.73 waves.
constexpr int kRouteThreads = 256, kRouteWarps = kRouteThreads / 32;

template <int N, bool VEC>
__global__ void __launch_bounds__(kRouteThreads) k_route_backward(RouteBackwardArgs a) {
    pdl_begin();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long first = ((long long)blockIdx.x * kRouteWarps + warp) * a.rows;
    if (first >= a.T) return;
    const int r0 = (int)first, r1 = (int)min((long long)a.T, first + a.rows);
    int s = -1, s_end = r0;       // the sequence whose f is in registers ends at s_end
    bool has = false;             // that sequence has rows
    float f[N], w = 0.0f;
    float nx[N], ng = 0.0f, ndg = 0.0f;
    int nid = -1, non = 1;
    // what a row needs is loaded one row ahead
    auto fetch = [&](int r) {
        load_row<N, VEC>(a.logits + (size_t)r * a.E, a.E, lane, nx);
        if (a.dgates && lane < a.k) {
            const size_t at = (size_t)r * a.k + lane;
            nid = __ldg(a.idx + at);
            ng = __ldg(a.gates + at);
            ndg = __ldg(a.dgates + at);
        }
        if (a.mask) non = __ldg(a.mask + r);
    };
    fetch(r0);
    for (int r = r0; r < r1; ++r) {
        float x[N];
#pragma unroll
        for (int v = 0; v < N; ++v) x[v] = nx[v];
        const float g = ng, dg = ndg;
        const int id = nid;
        const bool on = a.dloss && non;
        if (r + 1 < r1) fetch(r + 1);
        if (on && r >= s_end) {
            s = a.seq.find(r);
            s_end = s < a.seq.S ? a.seq.at(s + 1) : a.T;
            // rows in front of the first or behind the last sequence belong to none
            const bool in = s < a.seq.S && a.seq.at(s) <= r;
            const int n = in ? __ldg(a.tokens + s) : 0;
            const int used = __ldg(a.tokens + a.seq.S);
            has = n > 0 && used > 0;
            if (has) {
                const float inv = 1.0f / (float)n;
                w = __ldg(a.dloss) * (a.coef / (float)used) * inv;
                const float fs = (float)a.E / (float)a.k * inv;
                const int32_t* cr = a.counts + (size_t)s * a.E;
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    const int c = bal_col<VEC>(v, lane);
                    f[v] = c < a.E ? (float)__ldg(cr + c) * fs : 0.0f;
                }
            } else {
                if (!in) s_end = min(s_end, r + 1);
            }
        }
        if (on && has) {         // (a weight w of 0 too: it times a NaN is NaN)
            float sum = row_exp<N>(x), dot = 0.0f;
#pragma unroll
            for (int v = 0; v < N; ++v) dot = fmaf(x[v], f[v], dot);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
            }
            const float inv = row_inverse(sum), wi = w * inv;
            dot *= inv;
#pragma unroll
            for (int v = 0; v < N; ++v) x[v] = wi * x[v] * (f[v] - dot);
        } else {
#pragma unroll
            for (int v = 0; v < N; ++v) x[v] = 0.0f;
        }
        float* out = a.dlogits + (size_t)r * a.E;
        if (VEC) {
#pragma unroll
            for (int v = 0; v < N; v += 4) {
                const int c = bal_col<true>(v, lane);
                if (c < a.E) *reinterpret_cast<float4*>(out + c) = make_float4(x[v], x[v + 1], x[v + 2], x[v + 3]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const int c = bal_col<false>(v, lane);
                if (c < a.E) out[c] = x[v];
            }
        }
        if (a.dgates) {
            float add = g * dg;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);   // (k <= 16)
            add = g * (dg - add);
            bool mine = lane < a.k;
            if (mine && (unsigned)id >= (unsigned)a.E) {
                raise_flag(a.flag, FLAG_BAD_EXPERT);
                mine = false;
            }
            // an expert chosen twice: its first lane adds the terms in slot order
            // (lanes from k on hold -1)
            uint32_t same = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) same |= (uint32_t)(__shfl_sync(0xffffffffu, id, j) == id) << j;
            if (a.k > 8)
#pragma unroll
                for (int j = 8; j < 16; ++j) same |= (uint32_t)(__shfl_sync(0xffffffffu, id, j) == id) << j;
            if (__any_sync(0xffffffffu, mine && (same & (same - 1)))) {
                const float own = add;
                for (int j = 0; j < a.k; ++j) {
                    const float aj = __shfl_sync(0xffffffffu, own, j);
                    if (j > lane && (same >> j & 1u)) add += aj;
                }
                mine = mine && lane == __ffs((int)same) - 1;
            }
            __syncwarp();        // the row is stored
            if (mine) atomicAdd(out + id, add);      // (one per address: no order to depend on)
        }
    }
}

// Values per lane: E <= 32 N; the 16-byte form needs rows on 16-byte bounds.
#define MOE_BAL_DISPATCH(E, vec, CALL)                       \
    do {                                                     \
        if (vec) {                                           \
            if ((E) <= 128) { CALL(4, true); }               \
            else if ((E) <= 256) { CALL(8, true); }          \
            else if ((E) <= 512) { CALL(16, true); }         \
            else { CALL(32, true); }                         \
        } else {                                             \
            if ((E) <= 64) { CALL(2, false); }               \
            else if ((E) <= 256) { CALL(8, false); }         \
            else { CALL(32, false); }                        \
        }                                                    \
    } while (0)

static bool bal_vec(int E, const void* p, const void* q) {
    return E % 4 == 0 && ((uintptr_t)p | (uintptr_t)q) % 16 == 0;
}

template <int N, bool VEC, bool ONE>
static cudaError_t launch_bal_rows(dim3 grid, size_t smem, cudaStream_t st, const BalanceArgs& a) {
    auto kernel = k_balance_rows<N, VEC, ONE>;
    if (smem > 48 * 1024) {
        static PerContext cache;
        const int ok = cache.get([&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (kBalWarps + 1) * kMaxExperts * 4) == cudaSuccess
                       ? 1
                       : -1;
        });
        if (ok < 0) return cudaErrorInvalidValue;
    }
    return launch_pdl(kernel, grid, dim3(kBalThreads), smem, st, a);
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* seq_off, const uint8_t* mask,
                                int T, int E, int k, int S, float coef, int32_t* counts, float* mean_prob,
                                int32_t* tokens, float* loss, void* ws, cudaStream_t st) {
    char* w = (char*)ws;
    int32_t* head = (int32_t*)w;
    cudaError_t e;
    if (T == 0) {
        e = launch_pdl(k_balance_empty, dim3((unsigned)std::min<size_t>(((size_t)S * E + 255) / 256 + 1, 592)), dim3(256), 0, st,
                       SeqTable{seq_off, T, S}, head, counts, mean_prob, tokens, loss, E);
        count_launches(1);
        return e;
    }
    const BalanceWs L = balance_ws(T, E, S);
    const bool one = T <= kBalSingleT && S <= kBalSingleS;
    const int rows = one ? T : bal_chunk_rows(T);
    BalanceArgs a{logits, idx, mask, SeqTable{seq_off, T, S}, T, E, k, rows, coef, head, (int2*)(w + L.meta),
                  (float*)(w + L.prob), (int*)(w + L.hits), (float*)(w + L.part), counts, mean_prob, tokens, loss};
    const dim3 grid((unsigned)((T + rows - 1) / rows));
    const size_t smem = (size_t)(kBalWarps + 1) * E * 4;      // at most 68 KB
#define MOE_BAL_CALL(N, V)                                                                                    \
    e = one ? launch_bal_rows<N, V, true>(grid, smem, st, a) : launch_bal_rows<N, V, false>(grid, smem, st, a)
    MOE_BAL_DISPATCH(E, bal_vec(E, logits, logits), MOE_BAL_CALL);
#undef MOE_BAL_CALL
    count_launches(1);
    if (e != cudaSuccess || one) return e;
    e = launch_pdl(k_balance_reduce, dim3((unsigned)((E + 31) / 32), (unsigned)S), dim3(kRedThreads), 0, st, a);
    count_launches(1);
    return e;
}

cudaError_t launch_route_backward(const float* logits, const int32_t* idx, const float* gates, const float* dgates,
                                  const float* dloss, const int32_t* counts, const int32_t* tokens,
                                  const int32_t* seq_off, const uint8_t* mask, int T, int E, int k, int S, float coef,
                                  float* dlogits, int32_t* flag, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    // one row per warp until the SMs are full, then up to 8
    const int rows = std::min(8, std::max(1, T / (148 * 48)));
    RouteBackwardArgs a{logits, idx, gates, dgates, dloss, counts, tokens, mask, SeqTable{seq_off, T, S}, T, E, k,
                        rows, coef, dlogits, flag};
    const dim3 grid((unsigned)((T + rows * kRouteWarps - 1) / (rows * kRouteWarps)));
    cudaError_t e;
#define MOE_BAL_CALL(N, V) e = launch_pdl(k_route_backward<N, V>, grid, dim3(kRouteThreads), 0, st, a)
    MOE_BAL_DISPATCH(E, bal_vec(E, logits, dlogits), MOE_BAL_CALL);
#undef MOE_BAL_CALL
    count_launches(1);
    return e;
}

}  // namespace moe
