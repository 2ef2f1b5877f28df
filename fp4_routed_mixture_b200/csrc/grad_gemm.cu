// Gradient products on the tensor cores: the weight gradient of a projection
// from an 8-bit checkpoint of its input (dense, or one per expert), and the
// gradients of the router projection.  Formulas at moe_ckpt_wgrad and
// moe_router_logits_backward in the header.  All are
//   C[m, n] = sum_r A[r, m] B[r, n]
// with bf16 operands and fp32 accumulation (tcgen05 kind::f16):
//   GM_WGRAD   r = rows, A = dy (bf16), B = the checkpoint's values, which are
//              exact in bf16 (4 significant bits times a power of two)
//   GM_RDW     r = tokens, A = dlogits, B = x (bf16 or a checkpoint's values);
//              dlogits is fp32 and enters as three bf16 parts of 8 bits each
//              (exact): three products
//   GM_RDX     r = experts, A = dlogits, B = w_router, both fp32 with a bf16
//              result: the leading two parts of each, three products (the
//              smallest, low x low, is below 2^-16 of the terms)
// k_grad_prepare writes fp32 operands' parts, and in GM_WGRAD the checkpoint's
// values, as bf16 to the workspace first.  Where a stage takes longer than about
// 1500 cycles anyway, four warps convert the codes between their copy and the MMA
// (GM_.._CODES): in dW of the router, three products a stage (16384 tokens, H 4096,
// 256 experts, with dx: 217 us with the values in the workspace, 187 without), and
// with few rows, where C's stores bound (16 groups of 16 rows, 4096 x 4096: 201 us /
// 179).  In GM_WGRAD a stage's MMAs take 512 cycles: 750 us for 16384 x 4096 x
// 4096, where the conversion in front costs 3 bytes of traffic per value and 30 us
// of 465.
//
// One SM pair (cluster of two CTAs, tcgen05 cta_group::2) per 256 x 256 tile of
// C: the CTA of rank q supplies columns 128 q .. + 127 of A's and of B's tile
// and holds rows 128 q .. + 127 of the accumulator.  A stage is 64 rows r.
//   warp 0        operands by TMA (128-byte swizzle; "MN-major", the
//                 contraction runs over smem rows, except A of GM_RDX)
//   warp 1        (leader CTA) issues the MMAs
//   warp 2        GM_WGRAD through perm: checks the table
//   warps 4-7     GM_.._CODES: codes to bf16.  GM_WGRAD: clear the rows behind a
//                 group's last one.  Router: the parts of split tiles, dbias
//   warps 8-15    epilogue, from two 256-column accumulators in TMEM
// Work: pair p takes the tiles p, p + P, ... of the first floor(tiles / P) P
// ones whole; the remaining tiles are cut so that the last round is not left to
// a few pairs.  Where that pays, a tile's rows are cut into chunks and dealt out
// evenly; the parts go to the workspace and k_grad_fixup adds them in a fixed
// order.  Where a tile has few rows, storing C is what takes the time (40 x 4096
// x 4096: 2.6 us per tile and pair, the copy bandwidth): 2 or 4 pairs compute the
// same tile and store a part of its columns each.
//
// The tensor cores truncate when they add to the fp32 accumulator, always
// towards zero: about 7e-9 of the result per MMA (measured: 1.8e-6 of the norm
// after 256 of them, against 6e-7 of an fp32 sum in CUDA cores).  So an
// accumulator is drained every ACC_STEPS stages (1024 rows in GM_WGRAD: 3.5e-7)
// and added up in the epilogue's registers, rounding to nearest.
//
// Bound by the tensor cores and, in long runs, the power limit.  Measured (one
// B200): 16384 x 4096 x 4096 in 0.34 ms under ncu (1.6 PFLOP/s, tensor pipe 86
// percent busy; cuBLAS on bf16 operands 0.355 ms), whole call 0.40 ms in a burst and
// 0.47 in a loop of seconds, 0.43 of it the GEMM (cuBLAS there 0.39-0.415); 16 groups
// of 1726 rows on average, 4096 x 4096: 0.68 ms (1.36 PFLOP/s), bound by the tensor
// cores beside 1.07 GB of results.
#include "bf16_parts.cuh"
#include "ckpt.cuh"
#include "kernels.cuh"
#include "moe_common.cuh"
#include "tcgen05.cuh"

namespace moe {

// (GM_WGRAD_FEW: GM_WGRAD for few rows, where storing C is what takes the time.
// GM_.._CODES: B is read as a checkpoint's codes, which the kernel makes bf16)
enum { GM_WGRAD = 0, GM_RDW = 1, GM_RDX = 2, GM_WGRAD_FEW = 3, GM_RDW_CODES = 4, GM_WGRAD_CODES = 5 };

constexpr int GG_TILE = 256;            // rows and columns of C per pair
constexpr int GG_HALF = 128;            // per CTA: rows of A's tile, columns of B's
constexpr int GG_K = 64;                // contraction rows per stage
constexpr int GG_PLANE = GG_HALF * GG_K * 2;   // one operand part of a stage, per CTA
constexpr int GG_BLOCK = GG_K * 128;    // 64 columns of an MN-major plane
constexpr int GG_TAIL_WARP0 = 4, GG_TAIL_WARPS = 4, GG_EPI_WARP0 = 8, GG_EPI_WARPS = 8;
constexpr int GG_THREADS = 32 * (GG_EPI_WARP0 + GG_EPI_WARPS);
constexpr int GG_OUT = 32 * 128;
constexpr int GG_MAX_PAIRS = 128;
// Registers per thread: at launch, and of the two kinds of warpgroup after
// setmaxnreg.  The epilogue holds 128 sums per thread.  (Spilled, in bytes stored per
// thread: GM_RDX 12, GM_RDW 66, GM_RDW_CODES 54, GM_WGRAD_CODES 26, the others none.)
constexpr int GG_REGS = 128, GG_REGS_LOAD = 64, GG_REGS_EPI = 192;
static_assert(2 * GG_REGS_LOAD + 2 * GG_REGS_EPI <= 4 * GG_REGS, "registers of the block");

// Up to 256 rows a group, GM_WGRAD_FEW: with one piece of 4 KB on its way an
// epilogue warp waits for it, with two it stores at the copy bandwidth.  A stage
// less pays for it, which costs where rows are many.  Measured (us, FEW / the
// other form; N = K = 4096): 40 rows 18.0 / 21.7, 128 19.0 / 22.5, 256 20.9 / 23.2,
// 512 27.2 / 26.3; 16 groups of 100 rows 222 / 219, of 400 326 / 268, of 800 486 / 467.
constexpr int kFewRows = 256;
// Up to this many rows a group, without perm, the kernel reads the codes itself
// (us, GM_WGRAD_CODES / in front; one group: 512 x 512, 40 rows 7.4 / 8.0; 4096 x 4096, 1
// row 19.1 / 18.6, 40 rows 19.1 / 19.5, 128 20.5 / 20.6; 16384 x 4096, 64 rows 52 / 57, 128
// 58 / 60; 16 groups: 2048 x 2048, 40 rows 54 / 59, 4096 x 4096, 16 rows 179 / 200, 64 203 /
// 216, 128 230 / 217; 128 groups of 1024 x 1024, 128 rows 118 / 135).
constexpr int kConvertRows = 128;
static_assert(kConvertRows <= kFewRows, "the form that converts");

template <int MODE>
struct GradCfg {
    static constexpr bool CODES = MODE == GM_RDW_CODES || MODE == GM_WGRAD_CODES;
    static constexpr bool FEW = MODE == GM_WGRAD_FEW || MODE == GM_WGRAD_CODES;
    static constexpr bool WGRAD = MODE == GM_WGRAD || FEW;
    static constexpr bool RDW = MODE == GM_RDW || MODE == GM_RDW_CODES;
    static constexpr int AP = WGRAD ? 1 : RDW ? 3 : 2;   // parts of A
    static constexpr int BP = MODE == GM_RDX ? 2 : 1;
    static constexpr int OPS = (AP + BP) * GG_PLANE;
    // Stages, and pieces of 4 KB that an epilogue warp has on their way out.
    static constexpr int STAGES = FEW ? 5 : WGRAD ? 6 : 3;
    static constexpr int OUTS = FEW ? 2 : 1;
    static constexpr int ACC_STEPS = RDW ? 4 : 16;
    // Largest chunk of a split tile, and what splitting has to save, in stages
    // (about 5 us, what k_grad_fixup adds: a stage takes 0.28 us in GM_WGRAD, 0.85 with
    // three products; 512 tokens, 8 stages in 2: the same time with and without).  A
    // result of GM_RDX, of at most 16 stages, is not split.
    static constexpr int CHUNK_STEPS = WGRAD ? 16 : 8;
    static constexpr int SPLIT_GAIN = WGRAD ? 18 : RDW ? 8 : 1 << 20;
};

template <int MODE>
struct GradShared {
    uint8_t ops[GradCfg<MODE>::STAGES][GradCfg<MODE>::OPS];      // 1024-byte aligned
    uint8_t out[GG_EPI_WARPS][GradCfg<MODE>::OUTS][GG_OUT];   // epilogue: 32 rows of 128 bytes each
    uint64_t landed[GradCfg<MODE>::STAGES];          // leader: TMA bytes of both CTAs
    uint64_t tail_landed[GradCfg<MODE>::STAGES];     // a stage with a tail: those of this CTA
    uint64_t tail[GradCfg<MODE>::STAGES];            // its rows behind the group are cleared
    uint64_t peer[GradCfg<MODE>::STAGES];            // leader: those of the other CTA are
    uint64_t empty[GradCfg<MODE>::STAGES];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
    int32_t abort;
    uint32_t issued;         // stages whose copies this CTA has issued (modulo 2^32)
    int32_t rem_pre[GG_MAX_PAIRS + 1];               // chunks in front of each split tile
    float bias[4][32];
    uint8_t slots[MODE == GM_RDX ? 4 : 1][GG_MAX_PAIRS];
};

// dbias: column sums over the row blocks that k_grad_prepare summed.  128 threads
// take 32 columns: warp w every fourth block, then the warps in order.  (The
// warps of the router's GEMMs that have no other work do it, 4-7, or a kernel of
// its own where no GEMM runs: the same order and bits.)
struct BiasArgs {
    const float* part;       // [n][E], or NULL
    int n, E;
    float* db;
    int accumulate;
};
__device__ __forceinline__ void grad_bias(const BiasArgs& a, int block, int t, float (*s)[32]) {
    const int w = t >> 5, lane = t & 31, e = block * 32 + lane;
    float v = 0.0f;
    if (e < a.E)
#pragma unroll 8
        for (int i = w; i < a.n; i += 4) v += __ldg(a.part + (size_t)i * a.E + e);
    s[w][lane] = v;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (w == 0 && e < a.E) {
        v = ((s[0][lane] + s[1][lane]) + s[2][lane]) + s[3][lane];
        a.db[e] = a.accumulate ? a.db[e] + v : v;
    }
}
__global__ void __launch_bounds__(128) k_router_bias(BiasArgs a) {
    pdl_begin();
    __shared__ float s[4][32];
    grad_bias(a, blockIdx.x, threadIdx.x, s);
}

struct GradArgs {
    const int32_t* offsets;    // groups of rows, or NULL
    const int32_t* perm;       // checked here: perm[i] / k_div lies in [0, xrows); or NULL
    int k_div, xrows;
    int R;                     // contraction rows of all groups
    int M, N, G;               // C is [G, M, N]
    int MT, NT, tiles, full, chunk_steps;
    int ways;                  // pairs per remaining tile (1: cut by rows)
    float* c;                  // (GM_RDX stores through its map alone)
    int accumulate;
    float* part;               // [pairs][2][256][256]
    const uint8_t* x_scales;   // GM_.._CODES
    BiasArgs bias;             // GM_RDW, GM_RDX
    int32_t* flag;
    uint64_t wait_ns;
    int withhold;              // a test: no pair's first stage is copied
};

// Split tiles of a launch in front whose parts are still to be added (a.part NULL:
// none); pairs: of that launch.
struct FixupArgs {
    GradArgs a;
    int pairs;
};

// ---- PTX forms of the SM pair ----------------------------------------------------
__device__ __forceinline__ uint32_t gg_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void gg_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t gg_peer(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrival on the leader's barrier.  What it announces (operands in this CTA's
// shared memory, an accumulator read out of this CTA's TMEM) is used only by
// this SM's half of the MMA; it was written by TMA, whose barrier the caller has
// seen complete, or fenced towards the async proxy by its writer.  So it needs
// no cluster-wide fence, which .release.cluster would put here (1100 to 1600
// cycles a stage, measured).
__device__ __forceinline__ void gg_arrive(uint32_t bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(gg_peer(bar, rank)) : "memory");
}
__device__ __forceinline__ void gg_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void gg_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// (cta_group::2: the barrier may be the other CTA's)
__device__ __forceinline__ void gg_tma(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
template <bool ADD>
__device__ __forceinline__ void gg_tma_store(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
    if (ADD)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                     "r"(x), "r"(y), "r"(z), "r"(src)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                     "r"(x), "r"(y), "r"(z), "r"(src)
                     : "memory");
}
// Bounded wait on a phase of an mbarrier (see mbar_wait_for), the thread asleep
// for up to 20 us per try.  (Without that hint the waiting roles' polling was
// most of the instructions executed and cost 5 percent under the power limit:
// 16384 x 4096 x 4096 in a loop of seconds, 495 us against 469.)
__device__ __forceinline__ bool gg_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int32_t* abort) {
    auto poll = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        return ok != 0;
    };
    if (poll()) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (poll()) return true;
        if (abort && *abort) return false;
        if (global_ns() - t0 > limit_ns) return false;
    }
}
template <int REGS>
__device__ __forceinline__ void gg_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void gg_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
__device__ __forceinline__ void gg_fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void gg_st16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
// Two sums at once (Blackwell's packed fp32 addition, round to nearest).
__device__ __forceinline__ void gg_add2(float& a, float& b, uint32_t u, uint32_t v) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(u), "r"(v));
}
// 32 lanes x 16 columns: lane = row.
__device__ __forceinline__ void gg_ld32x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Shared-memory descriptors, 128-byte swizzle (type 2 in bits 61-63).
// MN-major (contraction over smem rows of 128 bytes = 64 columns): 8-row groups
// 1 KB apart, the next 64 columns 8 KB apart.  K-major (128-byte rows are 64
// contraction values of one row of C): 8-row groups 1 KB apart.
__device__ __forceinline__ uint64_t gg_desc_mn(uint32_t addr) {
    return make_sdesc(addr, GG_BLOCK, 1024) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t gg_desc_k(uint32_t addr) { return make_sdesc(addr, 16, 1024) | ((uint64_t)2 << 61); }

// kind::f16 instruction descriptor: bf16 x bf16, fp32 accumulate, M = N = 256.
__device__ __forceinline__ uint32_t gg_idesc(bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(GG_TILE >> 3) << 17) | ((uint32_t)(GG_TILE >> 4) << 24);
}

// Address of 16-byte chunk c (0..7) of row r of a 128-byte-row block, swizzled.
__device__ __forceinline__ uint32_t gg_swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// ---- the split of the work --------------------------------------------------------
// Contraction rows [r0, r1) of a group.
__device__ __forceinline__ void gg_rows(const GradArgs& a, int g, int& r0, int& r1) {
    r0 = 0;
    r1 = a.R;
    if (a.offsets) {
        r0 = min(max(__ldg(a.offsets + g), 0), a.R);
        r1 = min(max(__ldg(a.offsets + g + 1), r0), a.R);
    }
}
// Of the groups i, i + n, ..: one does not ascend within [0, R].
__device__ __forceinline__ bool bad_offsets(const int32_t* offsets, int G, int R, int i, int n) {
    bool bad = false;
    for (int g = i; g < G; g += n) {
        const int b = __ldg(offsets + g), e = __ldg(offsets + g + 1);
        bad |= b < 0 || e < b || e > R;
    }
    return bad;
}
// Tile i of a group, row by row.  (Bands of 4 or 8 columns, which would share
// both operands' panels in L2 among the tiles in flight, measured the same.)
__device__ __forceinline__ void gg_tile(const GradArgs& a, int i, int& m0, int& n0) {
    m0 = (i / a.NT) * GG_TILE;
    n0 = (i % a.NT) * GG_TILE;
}
// (a group without rows still has one stage, of zeros)
__device__ __forceinline__ int gg_steps(int rows) { return max(1, (int)(((long long)rows + GG_K - 1) / GG_K)); }

struct Segment {
    int m0, n0, g;      // tile
    int r0, r1;         // contraction rows of its group
    int s0, s1;         // stages
    int slot;           // -1: the whole tile, else the part's place
    int c0, c1;         // columns of the tile to store
};

// Walks a pair's segments; every role walks the same ones.
struct Walk {
    const GradArgs* args;
    const int32_t* rem_pre;
    int pair, pairs, next_full, chunk, chunk_end;
    bool first_part;
    __device__ Walk(const GradArgs& a, const int32_t* pre, int p, int P)
        : args(&a), rem_pre(pre), pair(p), pairs(P), next_full(p), first_part(true) {
        const int rem = a.tiles - a.full;
        const long long W = rem > 0 && a.ways == 1 ? pre[rem] : 0;
        chunk = (int)(W * p / P);
        chunk_end = (int)(W * (p + 1) / P);
    }
    __device__ bool next(Segment& s) {
        const GradArgs& a = *args;
        int t;
        s.c0 = 0;
        s.c1 = GG_TILE;
        if (next_full < a.full) {
            t = next_full;
            next_full += pairs;
        } else if (a.ways > 1) {
            if (!first_part || pair >= (a.tiles - a.full) * a.ways) return false;
            first_part = false;
            t = a.full + pair / a.ways;
            s.c0 = (GG_TILE / a.ways) * (pair % a.ways);
            s.c1 = s.c0 + GG_TILE / a.ways;
        } else if (chunk < chunk_end) {
            int lo = 0, hi = a.tiles - a.full - 1;        // last tile with rem_pre <= chunk
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (rem_pre[mid] <= chunk) lo = mid; else hi = mid - 1;
            }
            t = a.full + lo;
        } else {
            return false;
        }
        const int per = a.MT * a.NT, i = t % per;
        s.g = t / per;
        gg_tile(a, i, s.m0, s.n0);
        gg_rows(a, s.g, s.r0, s.r1);
        const int steps = gg_steps(s.r1 - s.r0);
        s.s0 = 0;
        s.s1 = steps;
        s.slot = -1;
        if (t >= a.full && a.ways == 1) {
            const int b = rem_pre[t - a.full], e = rem_pre[t - a.full + 1];
            const int c1 = min(chunk_end, e);
            if (chunk > b || c1 < e) {
                s.slot = pair * 2 + (first_part ? 0 : 1);
                s.s0 = (chunk - b) * a.chunk_steps;
                s.s1 = min(steps, (c1 - b) * a.chunk_steps);
            }
            first_part = false;
            chunk = c1;
        }
        return true;
    }
};

// The stages of a pair's segments one by one.
struct Steps {
    Walk walk;
    Segment seg;
    int st;
    bool on;
    __device__ Steps(const Walk& w) : walk(w) {
        on = walk.next(seg);
        st = on ? seg.s0 : 0;
    }
    __device__ void advance() {
        if (on && ++st == seg.s1) {
            on = walk.next(seg);
            st = seg.s0;
        }
    }
};

// ---- the parts of split tiles ------------------------------------------------------------
// Adds them in the order of their rows.  A warp takes rows [lo, hi) of the split
// tiles' rows, tile after tile; slots: GG_MAX_PAIRS bytes of its own.
__device__ __forceinline__ void grad_fixup(const GradArgs& a, int pairs, int lo, int hi, uint8_t* slots) {
    const int rem = a.tiles - a.full, per = a.MT * a.NT, lane = threadIdx.x & 31;
    int tile = -1, n = 0;
    for (int row = lo; row < hi; ++row) {
        const int i = row / GG_TILE, m = row % GG_TILE, t = a.full + i;
        if (i != tile) {
            // chunks of all split tiles, of those in front of tile i, and its own
            tile = i;
            int all = 0, b = 0, own = 0;
            for (int j = lane; j < rem; j += 32) {
                int r0, r1;
                gg_rows(a, (a.full + j) / per, r0, r1);
                const int c = (gg_steps(r1 - r0) + a.chunk_steps - 1) / a.chunk_steps;
                all += c;
                b += j < i ? c : 0;
                own += j == i ? c : 0;
            }
            const long long W = warp_sum(all);
            b = warp_sum(b);
            const int e = b + warp_sum(own);
            // the pairs whose range of chunks meets the tile's, in order
            n = 0;
            __syncwarp();
            for (int p0 = 0; p0 < pairs; p0 += 32) {
                const int p = p0 + lane, c0 = (int)(W * p / pairs), c1 = (int)(W * (p + 1) / pairs);
                const bool in = p < pairs && c0 < c1 && c0 < e && c1 > b;
                const uint32_t mask = __ballot_sync(0xffffffffu, in);
                // (it is a pair's second part where the pair's range begins in an earlier tile)
                if (in) slots[n + __popc(mask & ((1u << lane) - 1))] = (uint8_t)(2 * p + (c0 < b ? 1 : 0));
                n += __popc(mask);
            }
            __syncwarp();
        }
        if (n == 1) continue;        // one pair computed the whole tile
        int m0, n0;
        gg_tile(a, t % per, m0, n0);
        if (m0 + m >= a.M) continue;
        float* out = a.c + ((size_t)(t / per) * a.M + m0 + m) * a.N + n0;
        const float* part = a.part + m * GG_TILE;
        float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const float4* p = reinterpret_cast<const float4*>(part + (size_t)slots[j] * (GG_TILE * GG_TILE)) + lane;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 v = __ldg(p + 32 * h);
                s[h].x = __fadd_rn(s[h].x, v.x);
                s[h].y = __fadd_rn(s[h].y, v.y);
                s[h].z = __fadd_rn(s[h].z, v.z);
                s[h].w = __fadd_rn(s[h].w, v.w);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 4 * lane + 128 * h;
            if (n0 + c >= a.N) continue;
            float4* o = reinterpret_cast<float4*>(out + c);
            if (a.accumulate) {
                const float4 v = *o;
                s[h].x = __fadd_rn(v.x, s[h].x);
                s[h].y = __fadd_rn(v.y, s[h].y);
                s[h].z = __fadd_rn(v.z, s[h].z);
                s[h].w = __fadd_rn(v.w, s[h].w);
            }
            *o = s[h];
        }
    }
}
// CTA: 8 rows, a warp each.
__global__ void __launch_bounds__(256) k_grad_fixup(FixupArgs f) {
    pdl_begin();
    __shared__ uint8_t slots[8][GG_MAX_PAIRS];
    const int warp = threadIdx.x >> 5, row = blockIdx.x * 8 + warp;
    grad_fixup(f.a, f.pairs, row, row + 1, slots[warp]);
}

// ---- the kernel ----------------------------------------------------------------------
template <int MODE>
__global__ void __launch_bounds__(GG_THREADS, 1)
    k_grad_gemm(const __grid_constant__ GradArgs a, const __grid_constant__ FixupArgs fix, const __grid_constant__ CUtensorMap a_map,
                const __grid_constant__ CUtensorMap b_map, const __grid_constant__ CUtensorMap c_map,
                const __grid_constant__ CUtensorMap part_map) {
    using Cfg = GradCfg<MODE>;
    constexpr int AP = Cfg::AP, BP = Cfg::BP, STAGES = Cfg::STAGES;
    extern __shared__ uint8_t gg_raw_smem[];
    GradShared<MODE>& sh =
        *reinterpret_cast<GradShared<MODE>*>(gg_raw_smem + ((1024u - (smem_u32(gg_raw_smem) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = gg_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sh.landed[s]), 1);
            mbar_init(smem_u32(&sh.tail_landed[s]), 1);
            mbar_init(smem_u32(&sh.tail[s]), GG_TAIL_WARPS);
            mbar_init(smem_u32(&sh.peer[s]), GG_TAIL_WARPS);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sh.acc_full[b]), 1);
            mbar_init(smem_u32(&sh.acc_empty[b]), 2 * GG_EPI_WARPS);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        sh.issued = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1 && lane < 4) {
        const CUtensorMap* m = lane == 0 ? &a_map : lane == 1 ? &b_map : lane == 2 ? &c_map : &part_map;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    gg_cluster_sync();      // the peer's barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    // All of this needs nothing of the kernel in front; what follows does.  (Two
    // of these blocks do not fit an SM: TMEM is free when one starts.)
    pdl_begin();
    if (a.ways == 1 && a.tiles > a.full) {
        if (warp == 2) {
            // chunks in front of each split tile (fewer than `pairs` tiles)
            const int rem = a.tiles - a.full;
            int run = 0;
            for (int i0 = 0; i0 < rem; i0 += 32) {
                int n = 0;
                if (i0 + lane < rem) {
                    int r0, r1;
                    gg_rows(a, (a.full + i0 + lane) / (a.MT * a.NT), r0, r1);
                    n = (gg_steps(r1 - r0) + a.chunk_steps - 1) / a.chunk_steps;
                }
                int x = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (i0 + lane < rem) sh.rem_pre[i0 + lane] = run + x - n;
                run += __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == 0) sh.rem_pre[rem] = run;
        }
        __syncthreads();
    }
    volatile int32_t* abort = &sh.abort;
    auto give_up = [&]() {
        *abort = 1;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(gg_peer(smem_u32(&sh.abort), rank ^ 1u)), "r"(1u)
                     : "memory");
    };
    auto wait = [&](uint32_t bar, uint32_t parity) { return gg_wait(bar, parity, a.wait_ns, abort); };
    // of a whole warp: its lanes go on or give up together
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, !*abort && wait(bar, parity)) != 0;
    };
    // For a stage that may lie far ahead: the limit starts again as long as the
    // stages in front of it are being issued (one writer, read here after a whole
    // limit without success).
    volatile uint32_t* issued = &sh.issued;
    auto warp_wait_ahead = [&](uint32_t bar, uint32_t parity) {
        for (;;) {
            const uint32_t before = *issued;
            if (warp_wait(bar, parity)) return true;
            if (__any_sync(0xffffffffu, *abort || *issued == before)) return false;
        }
    };
    // The waits for what is in flight are not cut short: 0.1 s at the least.
    const uint64_t drain_ns = max(a.wait_ns, (uint64_t)100000000);
    auto final_wait = [&](uint32_t bar, uint32_t parity) {
        if (!gg_wait(bar, parity, drain_ns, nullptr)) *abort = 1;
    };
    const Walk walk0(a, sh.rem_pre, pair, pairs);
    int stage = 0;
    uint32_t phase = 0;
    auto next_stage = [&]() {
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
        }
    };

    // Stages with rows behind their group's last one (the last stage of a group
    // with another row count than a multiple of 64): dy and x of other rows have
    // landed there and are cleared (rows behind R read as 0).  Each CTA counts its
    // own bytes for them, on other barriers.  lands, tails: parity of the next use
    // of each stage's barriers of either kind.
    uint32_t lands = 0, tails = 0;
    auto has_tail = [&](const Segment& s, int st) {
        return Cfg::WGRAD && s.r1 < a.R && s.r1 - s.r0 - st * GG_K < GG_K;
    };
    constexpr bool CODES = Cfg::CODES;
    auto next_parity = [&](uint32_t& bits) {
        const uint32_t p = bits >> stage & 1u;
        bits ^= 1u << stage;
        return p;
    };

    if (warp < GG_TAIL_WARP0) {
        gg_regs_down<GG_REGS_LOAD>();
        if (warp == 0 && lane == 0) {
            // ---------------- operands by TMA ----------------
            // The bytes of both CTAs are counted on the leader's barrier.  (The
            // waits here run to their limit even when another role has given
            // up: "empty" reaches both CTAs, so both have then issued the same
            // stages, and the leader's last waits cover the copies of both.)
            const uint32_t bytes = (CODES ? AP : AP + BP) * GG_PLANE;
            constexpr uint32_t code_bytes = GG_K * GG_HALF;
            bool first = true;
            uint32_t count = 0;
            for (Steps s(walk0); s.on; s.advance()) {
                if (!gg_wait(smem_u32(&sh.empty[stage]), phase ^ 1u, drain_ns, nullptr)) {
                    give_up();
                    break;
                }
                if (Cfg::WGRAD && a.withhold && first) {
                    first = false;
                    next_stage();
                    continue;
                }
                const bool tail = has_tail(s.seg, s.st);
                uint32_t bar = smem_u32(tail ? &sh.tail_landed[stage] : &sh.landed[stage]);
                if (CODES) {
                    mbar_expect_tx(smem_u32(&sh.tail_landed[stage]), code_bytes + (tail ? bytes : 0));
                    next_parity(tails);
                }
                if (tail) {
                    if (!CODES) {
                        mbar_expect_tx(bar, bytes);
                        next_parity(tails);
                    }
                } else if (rank == 0) {
                    mbar_expect_tx(bar, 2 * bytes);
                    next_parity(lands);
                } else {
                    bar = gg_peer(bar, 0);
                }
                uint32_t dst = smem_u32(sh.ops[stage]);
                const int r = s.seg.r0 + s.st * GG_K;
                const int m = s.seg.m0 + GG_HALF * (int)rank, n = s.seg.n0 + GG_HALF * (int)rank;
#pragma unroll
                for (int p = 0; p < AP; ++p, dst += GG_PLANE) {
                    if (MODE == GM_RDX) {
                        gg_tma(dst, &a_map, r, m, p, bar);
                    } else {
                        gg_tma(dst, &a_map, m, r, p, bar);
                        gg_tma(dst + GG_BLOCK, &a_map, m + 64, r, p, bar);
                    }
                }
                if (CODES) {
                    // 128 codes of each row, where their values will be
                    gg_tma(dst, &b_map, n, r, 0, smem_u32(&sh.tail_landed[stage]));
                } else {
#pragma unroll
                    for (int p = 0; p < BP; ++p, dst += GG_PLANE) {
                        gg_tma(dst, &b_map, n, r, p, bar);
                        gg_tma(dst + GG_BLOCK, &b_map, n + 64, r, p, bar);
                    }
                }
                if (Cfg::WGRAD && !CODES) *issued = ++count;      // (no load: 8 percent of the call)
                next_stage();
            }
            // (a barrier's last use has the other parity than its next; one never used
            // passes as the phase in front of the first)
            for (int s = 0; s < STAGES; ++s) {
                final_wait(smem_u32(&sh.landed[s]), (lands >> s & 1u) ^ 1u);
                final_wait(smem_u32(&sh.tail_landed[s]), (tails >> s & 1u) ^ 1u);
            }
        } else if (warp == 1 && lane == 0) {
            // ---------------- MMA issuer ----------------
            if (rank == 0) {
                int buf = 0;
                uint32_t use = 0;       // bit b: parity of accumulator b's next use
                const uint32_t idesc = gg_idesc(MODE != GM_RDX, true);
                Walk walk(walk0);
                Segment seg;
                bool ok = true;
                while (ok && walk.next(seg)) {
                    for (int st = seg.s0; ok && st < seg.s1;) {
                        const int st1 = min(seg.s1, st + Cfg::ACC_STEPS);
                        if (!wait(smem_u32(&sh.acc_empty[buf]), (use >> buf & 1u) ^ 1u)) {
                            give_up();
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem + buf * GG_TILE;
                        for (int s = st; s < st1; ++s) {
                            const bool tail = has_tail(seg, s);
                            bool in = tail || wait(smem_u32(&sh.landed[stage]), next_parity(lands));
                            if (tail || CODES) {
                                const uint32_t p = next_parity(tails);
                                in = in && wait(smem_u32(&sh.tail[stage]), p) && wait(smem_u32(&sh.peer[stage]), p);
                            }
                            if (!in) {
                                give_up();
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint32_t sa = smem_u32(sh.ops[stage]), sb = sa + AP * GG_PLANE;
                            auto product = [&](int pa, int pb, bool first) {
#pragma unroll
                                for (int kk = 0; kk < GG_K / 16; ++kk) {
                                    const uint64_t da = MODE == GM_RDX ? gg_desc_k(sa + pa * GG_PLANE + kk * 32)
                                                                       : gg_desc_mn(sa + pa * GG_PLANE + kk * 2048);
                                    gg_mma(d, da, gg_desc_mn(sb + pb * GG_PLANE + kk * 2048), idesc,
                                           !(first && s == st && kk == 0));
                                }
                            };
                            if constexpr (Cfg::WGRAD) {
                                product(0, 0, true);
                            } else if constexpr (Cfg::RDW) {
                                product(2, 0, true);
                                product(1, 0, false);
                                product(0, 0, false);
                            } else {
                                product(1, 0, true);
                                product(0, 1, false);
                                product(0, 0, false);
                            }
                            gg_commit(smem_u32(&sh.empty[stage]));
                            next_stage();
                        }
                        if (!ok) break;
                        gg_commit(smem_u32(&sh.acc_full[buf]));
                        use ^= 1u << buf;
                        buf ^= 1;
                        st = st1;
                    }
                }
                gg_commit(smem_u32(&sh.drain));
                // every MMA is done before either CTA frees its TMEM
                final_wait(smem_u32(&sh.drain), 0);
            }
        } else if (Cfg::WGRAD && warp == 2 && a.perm) {
            // (k_grad_prepare reads row 0 for a bad entry; the error word is this
            // call's only from the second kernel on)
            int r0 = 0, r1 = a.R, unused;
            if (a.offsets) {
                gg_rows(a, 0, r0, unused);
                gg_rows(a, a.G - 1, unused, r1);
            }
            for (long long i = (long long)r0 + blockIdx.x * 32 + lane; i < r1; i += gridDim.x * 32) {
                const int v = __ldg(a.perm + i);
                checked_index(v < 0 ? v : v / a.k_div, a.xrows, a.flag);
            }
        }
        __syncwarp();
    } else if (warp < GG_EPI_WARP0) {
        gg_regs_down<GG_REGS_LOAD>();
        if constexpr (CODES) {
            // ---------------- codes to bf16 ----------------
            // 64 rows of 128 codes, 16 at a time: thread t takes columns 16 (t % 8)
            // .. of rows t / 8 + 16 u.  The values go where the codes were.
            const int t = threadIdx.x - 32 * GG_TAIL_WARP0, c16 = t & 7, row = t >> 3;
            Steps s(walk0);
            uint32_t scale[4];
            auto fetch = [&]() {       // scale bytes, one stage ahead
                const int n = s.seg.n0 + GG_HALF * (int)rank, r = s.seg.r0 + s.st * GG_K + row;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    scale[u] = n < a.N && r + 16 * u < a.R
                                   ? __ldg(a.x_scales + (((size_t)(r + 16 * u) * a.N + n) >> 7)) : 0u;
            };
            if (s.on) fetch();
            while (s.on) {
                const bool in = warp_wait(smem_u32(&sh.tail_landed[stage]), next_parity(tails));
                const uint32_t ops = smem_u32(sh.ops[stage]), dst = ops + AP * GG_PLANE;
                uint4 q[4];
                float f[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(q[u].x), "=r"(q[u].y), "=r"(q[u].z), "=r"(q[u].w)
                                 : "r"(dst + 16 * (t + 128 * u)));
                    f[u] = ckpt_scale(scale[u]);
                }
                // all codes are read; the four warps go on or give up together
                uint32_t all;
                asm volatile(
                    "{\n\t.reg .pred p, q;\n\t"
                    "setp.ne.u32 p, %1, 0;\n\t"
                    "bar.red.and.pred q, 1, 128, p;\n\t"
                    "selp.u32 %0, 1, 0, q;\n\t}"
                    : "=r"(all)
                    : "r"((uint32_t)in)
                    : "memory");
                if (!all) {
                    give_up();
                    break;
                }
                // (rows behind the group's last one: see below)
                const int valid = has_tail(s.seg, s.st) ? s.seg.r1 - s.seg.r0 - s.st * GG_K : GG_K;
                s.advance();
                if (s.on) fetch();
                if (valid < GG_K)
                    for (int i = t; i < AP * GG_PLANE / 16; i += 32 * GG_TAIL_WARPS)
                        if ((i >> 3 & (GG_K - 1)) >= valid) gg_st16(ops + i * 16, make_uint4(0u, 0u, 0u, 0u));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float v[8];
                    ckpt_values8(make_uint2(q[u].x, q[u].y), f[u], v);
                    uint4 lo = bf16x8_rn(v);
                    ckpt_values8(make_uint2(q[u].z, q[u].w), f[u], v);
                    uint4 hi = bf16x8_rn(v);
                    if (row + 16 * u >= valid) lo = hi = make_uint4(0u, 0u, 0u, 0u);
                    // (the odd half first for the upper 64 columns: no two lanes in one bank)
                    const uint32_t o = dst + (c16 >> 2) * GG_BLOCK;
                    const int h = c16 >> 2, c = 2 * (c16 & 3);
                    gg_st16(o + gg_swz(row + 16 * u, c + h), h ? hi : lo);
                    gg_st16(o + gg_swz(row + 16 * u, c + 1 - h), h ? lo : hi);
                }
                gg_fence_async();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0)
                        mbar_arrive(smem_u32(&sh.tail[stage]));
                    else
                        gg_arrive(smem_u32(&sh.peer[stage]), 0);
                }
                next_stage();
            }
            __syncwarp();
        }
        if (MODE == GM_RDX && fix.a.part) {
            // the parts of dw, from the launch in front
            const int rows = (fix.a.tiles - fix.a.full) * GG_TILE, w = warp - GG_TAIL_WARP0;
            const int i = w * gridDim.x + blockIdx.x, all = gridDim.x * GG_TAIL_WARPS;
            grad_fixup(fix.a, fix.pairs, (int)((long long)rows * i / all), (int)((long long)rows * (i + 1) / all),
                       sh.slots[w]);
        }
        if (!Cfg::WGRAD && a.bias.part) {
            for (int b = blockIdx.x; b * 32 < a.bias.E; b += gridDim.x) {
                grad_bias(a.bias, b, threadIdx.x - 32 * GG_TAIL_WARP0, sh.bias);
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
        }
        if (Cfg::WGRAD && a.offsets && !CODES) {
            // ---------------- rows behind a group's last one ----------------
            const int t = threadIdx.x - 32 * GG_TAIL_WARP0;
            for (Steps s(walk0); s.on; s.advance()) {
                if (has_tail(s.seg, s.st)) {
                    if (!warp_wait_ahead(smem_u32(&sh.tail_landed[stage]), next_parity(tails))) {
                        give_up();
                        break;
                    }
                    const int valid = s.seg.r1 - s.seg.r0 - s.st * GG_K;
                    const uint32_t dst = smem_u32(sh.ops[stage]);
                    for (int i = t; i < Cfg::OPS / 16; i += 32 * GG_TAIL_WARPS)
                        if ((i >> 3 & (GG_K - 1)) >= valid) gg_st16(dst + i * 16, make_uint4(0u, 0u, 0u, 0u));
                    gg_fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0)
                            mbar_arrive(smem_u32(&sh.tail[stage]));
                        else
                            gg_arrive(smem_u32(&sh.peer[stage]), 0);
                    }
                }
                next_stage();
            }
        }
        __syncwarp();
    } else {
        gg_regs_up<GG_REGS_EPI>();
        // ---------------- epilogue ----------------
        // Warp (q, half): TMEM lanes 32 q .. + 31 (lane = row), columns 128 half
        // .. + 127, 16 at a time into the sums.  Results leave through 32 rows x
        // 128 bytes of shared memory (128-byte swizzle: 16-byte stores without
        // bank conflicts) and TMA, which writes whole lines and cuts off what
        // lies outside C; adding to C is its reduction.
        const int q = warp & 3, half = (warp - GG_EPI_WARP0) >> 2;
        int piece = 0;
        int buf = 0;
        uint32_t use = 0;
        Walk walk(walk0);
        Segment seg;
        bool ok = true;
        while (ok && walk.next(seg)) {
            float acc[8][16];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i >> 4][i & 15] = 0.0f;
            for (int st = seg.s0; st < seg.s1; st += Cfg::ACC_STEPS) {
                if (!warp_wait(smem_u32(&sh.acc_full[buf]), use >> buf & 1u)) {
                    give_up();
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t v[16];
                    gg_ld32x16(tmem + ((uint32_t)(32 * q) << 16) + buf * GG_TILE + 128 * half + 16 * i, v);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int e = 0; e < 16; e += 2) gg_add2(acc[i][e], acc[i][e + 1], v[e], v[e + 1]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) gg_arrive(smem_u32(&sh.acc_empty[buf]), 0);
                use ^= 1u << buf;
                buf ^= 1;
            }
            if (!ok) break;
            const bool whole = seg.slot < 0;
            const int mr = GG_HALF * (int)rank + 32 * q, nc = 128 * half;
            constexpr int COLS = MODE == GM_RDX ? 64 : 32;      // of C per 128 bytes
#pragma unroll
            for (int g = 0; g < 128 / COLS; ++g) {
                if (nc + COLS * g < seg.c0 || nc + COLS * g >= seg.c1) continue;
                // what was in this piece has been read
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(Cfg::OUTS - 1) : "memory");
                __syncwarp();
                const uint32_t out = smem_u32(sh.out[warp - GG_EPI_WARP0][piece]);
                piece = piece + 1 == Cfg::OUTS ? 0 : piece + 1;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint4 v;
                    if constexpr (MODE == GM_RDX) {
                        const float* r = &acc[4 * g + (j >> 1)][8 * (j & 1)];
                        v = make_uint4(bf16x2_rn(r[0], r[1]), bf16x2_rn(r[2], r[3]), bf16x2_rn(r[4], r[5]),
                                       bf16x2_rn(r[6], r[7]));
                    } else {
                        const float* r = &acc[2 * g + (j >> 2)][4 * (j & 3)];
                        v = make_uint4(__float_as_uint(r[0]), __float_as_uint(r[1]), __float_as_uint(r[2]),
                                       __float_as_uint(r[3]));
                    }
                    gg_st16(out + gg_swz(lane, j), v);
                }
                gg_fence_async();
                __syncwarp();
                if (lane == 0) {
                    const int n = nc + COLS * g;
                    if (!whole)
                        gg_tma_store<false>(&part_map, n, mr, seg.slot, out);
                    else if (seg.m0 + mr < a.M && seg.n0 + n < a.N) {
                        if (MODE != GM_RDX && a.accumulate)
                            gg_tma_store<true>(&c_map, seg.n0 + n, seg.m0 + mr, seg.g, out);
                        else
                            gg_tma_store<false>(&c_map, seg.n0 + n, seg.m0 + mr, seg.g, out);
                    }
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // The last of the leader's arrivals here has landed before this CTA may end.
    // (Its limit counts from the end of this CTA's own work: a wait from the start
    // would bound the whole kernel instead of one hand-over.)
    if (rank != 0 && threadIdx.x == 0) final_wait(smem_u32(&sh.drain), 0);
    __syncwarp();           // (what follows is of whole warps)
    gg_cluster_sync();      // no remote arrive or MMA targets this CTA any more
    if (threadIdx.x == 0 && *abort) raise_flag(a.flag, FLAG_TIMEOUT);
    __syncwarp();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ---- what the products need as bf16 ----------------------------------------------------
constexpr int kSplitThreads = 256;
constexpr int kSplitMaxCtas = 148 * 4;

// What a call needs as bf16 in its workspace.  The grid's CTAs take the parts
// in turn: dlogits, w_router, the checkpoint.
struct PrepareArgs {
    const float* dl;         // [T, E]
    const float* w;          // [E, H]
    int T, E, H, Ep;         // Ep: E rounded up to 8
    int rows;                // tokens per CTA
    int dl_ctas, w_ctas;
    int parts;               // of dl: 3, 2, or 0 (none written)
    __nv_bfloat16* dlp;      // [3][T][Ep]
    __nv_bfloat16* wp;       // [2][E][H]
    float* bias_part;        // [dl_ctas][E] column sums, or NULL
    const uint8_t* codes;    // checkpoint [.., K], `items` groups of 8 codes
    const uint8_t* scales;
    long long items;
    int K;
    const int32_t* perm;     // row i from row perm[i] / k_div below xrows, or NULL
    int k_div, xrows;
    __nv_bfloat16* xb;
    const int32_t* offsets;  // checked by the first CTA, or NULL
    int G, R;
    int32_t* flag;
};

// The first CTA also clears the call's error word, or raises FLAG_BOUNDS there
// when the group offsets do not ascend within [0, R].
__global__ void __launch_bounds__(kSplitThreads) k_grad_prepare(PrepareArgs a) {
    pdl_begin();
    if (blockIdx.x == 0) {
        const bool bad = __syncthreads_or(a.offsets && bad_offsets(a.offsets, a.G, a.R, threadIdx.x, kSplitThreads));
        if (threadIdx.x == 0) *a.flag = bad ? FLAG_BOUNDS : 0;
    }
    int b = blockIdx.x;
    if (b < a.dl_ctas) {
        // Thread: 4 neighbouring columns of every (256 / (Ep / 4))-th row of the CTA's.
        const int c4 = a.Ep / 4, c = 4 * ((int)threadIdx.x % c4), rg = (int)threadIdx.x / c4, rgs = kSplitThreads / c4;
        const int t0 = b * a.rows, t1 = min(a.T, t0 + a.rows);
        const bool vec = (a.E & 3) == 0;
        float sum[4] = {};
        if (rg < rgs) {
#pragma unroll 4
            for (int t = t0 + rg; t < t1; t += rgs) {
                const float* p = a.dl + (size_t)t * a.E + c;
                float v[4] = {};
                if (vec) {
                    if (c < a.E) {
                        const float4 q = __ldg(reinterpret_cast<const float4*>(p));
                        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (c + j < a.E) v[j] = __ldg(p + j);
                }
                uint2 h, m, l;
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] += v[j];
                split3x2(v[0], v[1], h.x, m.x, l.x);
                split3x2(v[2], v[3], h.y, m.y, l.y);
                if (a.parts) {
                    __nv_bfloat16* o = a.dlp + (size_t)t * a.Ep + c;
                    const size_t plane = (size_t)a.T * a.Ep;
                    *reinterpret_cast<uint2*>(o) = h;
                    *reinterpret_cast<uint2*>(o + plane) = m;
                    if (a.parts == 3) *reinterpret_cast<uint2*>(o + 2 * plane) = l;
                }
            }
        }
        if (a.bias_part) {
            // the row groups' sums, added in order
            __shared__ float s[kSplitThreads][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[threadIdx.x][j] = sum[j];
            __syncthreads();
            if (rg == 0) {
                for (int g = 1; g < rgs; ++g)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] += s[g * c4 + threadIdx.x][j];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < a.E) a.bias_part[(size_t)b * a.E + c + j] = sum[j];
            }
        }
        return;
    }
    b -= a.dl_ctas;
    if (b < a.w_ctas) {
        const size_t n4 = (size_t)a.E * a.H / 4, step = (size_t)a.w_ctas * kSplitThreads;
        for (size_t i = (size_t)b * kSplitThreads + threadIdx.x; i < n4; i += step) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(a.w) + i);
            uint2 h, m, l;
            split3x2(v.x, v.y, h.x, m.x, l.x);
            split3x2(v.z, v.w, h.y, m.y, l.y);
            reinterpret_cast<uint2*>(a.wp)[i] = h;
            reinterpret_cast<uint2*>(a.wp)[n4 + i] = m;
        }
        return;
    }
    b -= a.w_ctas;
    // The checkpoint's values, 8 codes per item.
    constexpr int U = 4;
    const long long ctas = gridDim.x - a.dl_ctas - a.w_ctas;
    if (a.perm) {
        // a warp per row: its table entry is resolved once
        const int lane = threadIdx.x & 31, K8 = a.K / 8;
        for (long long r = (long long)b * (kSplitThreads / 32) + (threadIdx.x >> 5); r < a.R;
             r += ctas * (kSplitThreads / 32)) {
            const int v = __ldg(a.perm + r), x = v < 0 ? 0 : v / a.k_div;
            const long long src = (long long)(x < a.xrows ? x : 0) * K8;      // (bad entries: row 0)
            for (int c0 = lane; c0 < K8; c0 += 32 * U) {
                uint2 c[U];
                uint32_t s[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + 32 * u < K8) {
                        c[u] = __ldg(reinterpret_cast<const uint2*>(a.codes + (src + c0 + 32 * u) * 8));
                        s[u] = __ldg(a.scales + ((src + c0 + 32 * u) >> 4));
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + 32 * u < K8) {
                        float o[8];
                        ckpt_values8(c[u], ckpt_scale(s[u]), o);
                        reinterpret_cast<uint4*>(a.xb)[r * K8 + c0 + 32 * u] = bf16x8_rn(o);
                    }
            }
        }
        return;
    }
    const long long stride = ctas * kSplitThreads;
    for (long long i0 = (long long)b * kSplitThreads + threadIdx.x; i0 < a.items; i0 += stride * U) {
        uint2 c[U];
        uint32_t s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long i = i0 + u * stride;
            if (i >= a.items) continue;
            c[u] = __ldg(reinterpret_cast<const uint2*>(a.codes + i * 8));
            s[u] = __ldg(a.scales + (i >> 4));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long i = i0 + u * stride;
            if (i >= a.items) break;
            float v[8];
            ckpt_values8(c[u], ckpt_scale(s[u]), v);
            reinterpret_cast<uint4*>(a.xb)[i] = bf16x8_rn(v);
        }
    }
}

// The same for a product that needs nothing else prepared: one warp.  It lets the
// product's blocks come up in front of its own wait (4096 x 4096, 40 rows: 20.0 us with
// the usual order, 19.1): they wait for this grid, which has waited for all before
// it, and by then every block they wait for runs.
__global__ void __launch_bounds__(32) k_grad_clear(const int32_t* offsets, int G, int R, int32_t* flag) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool bad = __any_sync(0xffffffffu, offsets && bad_offsets(offsets, G, R, threadIdx.x, 32));
    if (threadIdx.x == 0) *flag = bad ? FLAG_BOUNDS : 0;
}

static unsigned prepare_ctas(long long items) {
    return (unsigned)std::min<long long>((items + 4 * kSplitThreads - 1) / (4 * kSplitThreads), 148 * 32);
}

// ---- host -----------------------------------------------------------------------------
template <int MODE>
static size_t grad_smem() { return sizeof(GradShared<MODE>) + 1024; }

// CTAs of the kernel that can be resident as pairs (a persistent grid).
template <int MODE>
static int grad_grid() {
    static PerContext cache;
    return cache.get([] {
        auto kernel = k_grad_gemm<MODE>;
        const size_t smem = grad_smem<MODE>();
        int dev = 0, sms = 0, clusters = 0;
        cudaFuncAttributes fa;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
            cudaFuncGetAttributes(&fa, kernel) != cudaSuccess)
            return -1;
        // the warpgroups' register shares are taken from the launch's
        if (fa.numRegs != GG_REGS) return -1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(sms / 2 * 2);
        cfg.blockDim = dim3(GG_THREADS);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters <= 0) return -1;
        return 2 * std::min(clusters, GG_MAX_PAIRS);
    });
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor map of `planes` row-major matrices [rows, cols] (rows ld elements
// apart, matrices one behind the other): boxes of 128 bytes x box_rows with the
// 128-byte swizzle.  What lies outside reads as 0 and is not written.
static cudaError_t grad_map(const void* p, CUtensorMapDataType type, long long ld, int rows, int cols, int planes,
                            int box_cols, int box_rows, CUtensorMap* map) {
    static const EncodeTiled encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(f);
    }();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t row = (cuuint64_t)ld * (128 / box_cols);
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    // (a single matrix has no plane stride to overflow)
    const cuuint64_t strides[2] = {row, planes > 1 ? row * (cuuint64_t)rows : row};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
    return encode(map, type, 3, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}
static cudaError_t bf16_map(const void* p, long long ld, int rows, int cols, int planes, int box_rows,
                            CUtensorMap* map) {
    return grad_map(p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ld, rows, cols, planes, 64, box_rows, map);
}

// fix: GM_RDX adds the parts it names; GM_RDW leaves its own there instead of
// launching k_grad_fixup.
template <int MODE>
static cudaError_t launch_grad(GradArgs a, const CUtensorMap& a_map, const CUtensorMap& b_map, void* c,
                               cudaStream_t st, FixupArgs* fix = nullptr) {
    const int grid = grad_grid<MODE>();
    if (grid <= 0) return cudaErrorInvalidConfiguration;
    const int pairs = grid / 2;
    a.MT = (a.M + GG_TILE - 1) / GG_TILE;
    a.NT = (a.N + GG_TILE - 1) / GG_TILE;
    const long long tiles = (long long)a.G * a.MT * a.NT;
    if (tiles >= (1LL << 30)) return cudaErrorInvalidValue;
    a.tiles = (int)tiles;
    a.full = a.tiles / pairs * pairs;
    // The remaining tiles: chunks of rows so that every pair has one, or several of
    // the largest size.  (The rows of a group are known on the device only: the
    // average stands for them.)
    const int rem = a.tiles - a.full;
    const int max_steps = (int)(((long long)a.R + GG_K - 1) / GG_K);
    const int steps = (int)(((long long)a.R / a.G + GG_K - 1) / GG_K);
    const int per = rem > 0 ? pairs / rem : 1;
    a.chunk_steps = std::max(1, std::min((steps + per - 1) / per, GradCfg<MODE>::CHUNK_STEPS));
    const int longest = (int)(((long long)rem * ((steps + a.chunk_steps - 1) / a.chunk_steps) + pairs - 1) / pairs) * a.chunk_steps;
    const bool split = rem > 0 && steps - longest >= GradCfg<MODE>::SPLIT_GAIN;
    if (!split) a.chunk_steps = std::max(1, max_steps);
    // (4 ways: 64 columns, the narrowest store of GM_RDX)
    a.ways = split || rem == 0 ? 1 : per >= 4 ? 4 : per >= 2 ? 2 : 1;
    CUtensorMap c_map, part_map;
    cudaError_t e;
    if (MODE == GM_RDX)
        e = grad_map(c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.N, a.M, a.N, 1, 64, 32, &c_map);
    else
        e = grad_map(c, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.N, a.M, a.N, a.G, 32, 32, &c_map);
    part_map = c_map;
    if (e == cudaSuccess && split)
        e = grad_map(a.part, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, GG_TILE, GG_TILE, GG_TILE, 2 * pairs, 32, 32, &part_map);
    if (e != cudaSuccess) return e;
    a.c = (float*)c;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(GG_THREADS);
    cfg.dynamicSmemBytes = grad_smem<MODE>();
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const FixupArgs none = {};
    e = cudaLaunchKernelEx(&cfg, k_grad_gemm<MODE>, a, MODE == GM_RDX ? *fix : none, a_map, b_map, c_map, part_map);
    count_launches(1);
    if (e != cudaSuccess || !split) return e;
    const FixupArgs f{a, pairs};
    if (fix) {
        *fix = f;
        return e;
    }
    e = launch_pdl(k_grad_fixup, dim3((unsigned)(rem * (GG_TILE / 8))), dim3(256), 0, st, f);
    count_launches(1);
    return e;
}

// Workspace: the error word (256 bytes), the operands as bf16, the parts of
// split tiles (where a tile can be split).
static size_t grad_part_bytes(int R, int split_gain) {
    return R > split_gain * GG_K ? (size_t)GG_MAX_PAIRS * 2 * GG_TILE * GG_TILE * sizeof(float) : 0;
}
static size_t wgrad_part_offset(int R, int K) { return 256 + align_up(2 * (size_t)R * K, 256); }
size_t wgrad_workspace_bytes(int R, int, int K, int) {
    return wgrad_part_offset(R, K) + grad_part_bytes(R, GradCfg<GM_WGRAD>::SPLIT_GAIN);
}

struct RouterWs {
    size_t wp, bias, dlp, part, total;
};
static RouterWs router_ws(int T, int H, int E) {
    const size_t Ep = align_up(E, 8);
    RouterWs L;
    size_t o = 256;
    L.wp = o; o += align_up(2 * 2 * (size_t)E * H, 256);
    L.bias = o; o += align_up(sizeof(float) * kSplitMaxCtas * (size_t)E, 256);
    L.dlp = o; o += align_up(3 * 2 * (size_t)T * Ep, 256);
    L.part = o; o += grad_part_bytes(T, GradCfg<GM_RDW>::SPLIT_GAIN);
    L.total = o;
    return L;
}
size_t router_backward_workspace_bytes(int T, int H, int E) { return router_ws(T, H, E).total; }

cudaError_t launch_ckpt_wgrad(const void* dy, long long lddy, const uint8_t* codes, const uint8_t* scales,
                              const int32_t* offsets, const int32_t* perm, int k, int R, int rows, int N, int K, int G,
                              float* dw, int accumulate, void* ws, uint64_t wait_ns, int withhold, cudaStream_t st) {
    int32_t* flag = (int32_t*)ws;
    cudaError_t e = cudaSuccess;
    __nv_bfloat16* xb = (__nv_bfloat16*)((char*)ws + 256);
    const bool convert = R > 0 && !perm && R / G <= kConvertRows;
    if (convert) {
        // (a clear inside the product's grid would not be ordered before another CTA's
        // flag; this launch costs 1 us: 40 rows, 512 x 512 6.9 -> 7.4, 4096 x 4096 17.9 -> 19.1)
        e = launch_pdl(k_grad_clear, dim3(1), dim3(32), 0, st, offsets, G, R, flag);
    } else {
        PrepareArgs s = {};
        s.codes = codes;
        s.scales = scales;
        s.items = (long long)R * (K / 8);
        s.K = K;
        s.perm = perm;
        s.k_div = k;
        s.xrows = rows;
        s.xb = xb;
        s.offsets = offsets;
        s.G = G;
        s.R = R;
        s.flag = flag;
        e = launch_pdl(k_grad_prepare, dim3(std::max(1u, prepare_ctas(s.items))), dim3(kSplitThreads), 0, st, s);
    }
    count_launches(1);
    if (e == cudaSuccess && R == 0) return accumulate ? e : cudaMemsetAsync(dw, 0, sizeof(float) * G * N * K, st);
    CUtensorMap a_map, b_map;
    if (e == cudaSuccess) e = bf16_map(dy, lddy, R, N, 1, GG_K, &a_map);
    if (e == cudaSuccess)
        e = convert ? grad_map(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, K, R, K, 1, GG_HALF, GG_K, &b_map)
                    : bf16_map(xb, K, R, K, 1, GG_K, &b_map);
    if (e != cudaSuccess) return e;
    GradArgs a = {};
    a.offsets = offsets;
    a.perm = perm;
    a.k_div = k;
    a.xrows = rows;
    a.R = R;
    a.M = N;
    a.N = K;
    a.G = G;
    a.accumulate = accumulate;
    a.part = (float*)((char*)ws + wgrad_part_offset(R, K));
    a.flag = flag;
    a.wait_ns = wait_ns;
    a.withhold = withhold;
    a.x_scales = scales;
    // (rows of a group: the average stands for them)
    if (convert) return launch_grad<GM_WGRAD_CODES>(a, a_map, b_map, dw, st);
    return R / G <= kFewRows ? launch_grad<GM_WGRAD_FEW>(a, a_map, b_map, dw, st)
                             : launch_grad<GM_WGRAD>(a, a_map, b_map, dw, st);
}

cudaError_t launch_router_backward(const float* dl, const void* x, const uint8_t* codes, const uint8_t* scales,
                                   const float* w, int T, int H, int E, void* dx, float* dw, float* db, int accumulate,
                                   void* ws, uint64_t wait_ns, cudaStream_t st) {
    int32_t* flag = (int32_t*)ws;
    cudaError_t e = cudaSuccess;
    if (T == 0) {
        e = cudaMemsetAsync(flag, 0, sizeof(int32_t), st);
        if (e == cudaSuccess && dw && !accumulate) e = cudaMemsetAsync(dw, 0, sizeof(float) * E * H, st);
        if (e == cudaSuccess && db && !accumulate) e = cudaMemsetAsync(db, 0, sizeof(float) * E, st);
        return e;
    }
    if (router_grad_small(T, H, E))
        return launch_router_grad_small(dl, x, codes, scales, w, T, H, E, dx, dw, db, accumulate, flag, st);
    const RouterWs L = router_ws(T, H, E);
    char* b = (char*)ws;
    const int Ep = (int)align_up(E, 8);
    PrepareArgs s = {};
    s.dl = dl;
    s.w = w;
    s.T = T;
    s.E = E;
    s.H = H;
    s.Ep = Ep;
    s.rows = std::max(16, (T + kSplitMaxCtas - 1) / kSplitMaxCtas);
    s.dl_ctas = (T + s.rows - 1) / s.rows;
    s.w_ctas = dx ? (int)std::min<size_t>(((size_t)E * H / 4 + kSplitThreads - 1) / kSplitThreads, 148 * 4) : 0;
    s.parts = dw ? 3 : dx ? 2 : 0;
    s.dlp = (__nv_bfloat16*)(b + L.dlp);
    s.wp = (__nv_bfloat16*)(b + L.wp);
    s.bias_part = db ? (float*)(b + L.bias) : nullptr;
    s.flag = flag;
    e = launch_pdl(k_grad_prepare, dim3((unsigned)(s.dl_ctas + s.w_ctas)), dim3(kSplitThreads), 0, st, s);
    count_launches(1);
    GradArgs a = {};
    a.G = 1;
    a.N = H;
    a.flag = flag;
    a.wait_ns = wait_ns;
    BiasArgs bias{s.bias_part, s.dl_ctas, E, db, accumulate};
    FixupArgs fix = {};
    CUtensorMap a_map, b_map;
    if (e == cudaSuccess && dw) {
        e = bf16_map(s.dlp, Ep, T, Ep, 3, GG_K, &a_map);
        if (e == cudaSuccess)
            e = x ? bf16_map(x, H, T, H, 1, GG_K, &b_map)
                  : grad_map(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, H, T, H, 1, GG_HALF, GG_K, &b_map);
        if (e != cudaSuccess) return e;
        GradArgs d = a;
        d.R = T;
        d.M = E;
        d.accumulate = accumulate;
        d.part = (float*)(b + L.part);
        d.x_scales = scales;
        if (!dx) {
            d.bias = bias;
            bias.part = nullptr;
        }
        e = x ? launch_grad<GM_RDW>(d, a_map, b_map, dw, st, dx ? &fix : nullptr)
              : launch_grad<GM_RDW_CODES>(d, a_map, b_map, dw, st, dx ? &fix : nullptr);
    }
    if (e == cudaSuccess && dx) {
        e = bf16_map(s.dlp, Ep, T, Ep, 2, GG_HALF, &a_map);
        if (e == cudaSuccess) e = bf16_map(s.wp, H, E, H, 2, GG_K, &b_map);
        if (e != cudaSuccess) return e;
        a.R = E;
        a.M = T;
        a.bias = bias;
        bias.part = nullptr;
        e = launch_grad<GM_RDX>(a, a_map, b_map, dx, st, &fix);
    }
    if (e == cudaSuccess && bias.part) {
        e = launch_pdl(k_router_bias, dim3((unsigned)((E + 31) / 32)), dim3(128), 0, st, bias);
        count_launches(1);
    }
    return e;
}

}  // namespace moe
