// paged_tc.cu -- one-token decode over the paged latent cache on the sm_103a tensor cores (bf16,
// d_kv = 512, d_nope = d_v = 128, d_rope = 64, pages of a multiple of eight tokens, any number of
// heads).
//
// Mathematics, per request b of n keys and head h: q = W_K(h)^T q_nope, s_j = scale (q . c_j +
// rot(q_pe, n - 1) . kpe_j), o = sum_j softmax_j(s) c_j, out = W_V(h) o.  Three launches, each
// started early by programmatic dependent launch:
//   absorb     q and the rotated q_pe, each as a bf16 pair hi + lo; the division of the batch;
//   attention  persistent clusters of two CTAs walk equal shares of all requests' key tiles;
//   join       the partials' log-sum-exp merge and the product with W_V.
// The same three compute the tokens of a step (STEP; paged_step.cu divides those): a request is then a group of tokens
// that share an item, each row with its own number of keys.
//
// Attention.  One work item = 128 heads (fewer rows are zero-filled) of one request; its fp32
// accumulator, 128 x 512, is a whole SM's tensor memory, so an item runs on two SMs:
//   rank 0 (scores): the queries in TMEM; 64-key tiles of the cache (latent + key band) through a
//     two-deep TMA ring that fills and drains in three groups of 64-dim blocks, a producer warp for
//     each; S = Q K^T, two S buffers; online softmax by eight warps (two threads per head, four up to 64 heads); P in
//     bf16 to rank 1 by bulk copies into its two P slots;
//   rank 1 (accumulator): O in TMEM; streams the same tiles' latent in halves of 256 dims (L2 hits:
//     an idle warp prefetches rank 0's next tiles) and issues O += P C.
// The walk is persistent: equal shares of whole tiles per cluster (a request may be cut between any
// two tiles, parts meet in the join) leave no wave tail.  Between parts the next request's query boxes
// land in the key stages, in flight at once, while the softmax and rank 1 finish.
//
// What bounds it.  64 ragged requests of up to 32768 keys, 128 heads: the attention 275-285 us, 0.96 us
// per tile and pair of SMs, 5.3-5.6 TB/s; 16 heads 6.0-6.2 TB/s; without its MMAs the kernel moves 6.6 TB/s
// (the copy peak is 6.8).  No unit is full: of a tile's 1800 cycles rank 0's tensor pipe needs 1280
// (40 MMAs of N = 64 with A in TMEM, 32 cycles each) and rank 1's 1024, DRAM runs at 71 %, L2 at 66 %,
// shared memory below 50 %.  The MMAs' issue is part of the chain: one issuing warp takes 1.22 us a tile,
// two 0.96.  Measured no faster: a ring of seven 24 KB slots instead of six, a third P slot, sixteen
// softmax warps of 16 keys, fully unrolled MMAs, and these together (all 0.94-0.98), 128-key steps with
// N = 128 (1.03), P written to rank 1 by the softmax threads themselves (1.15), warp-uniform issue (1.05).
//
// Pages.  A unit is the largest power of two of rows, up to a tile, that divides the page (8, 16, 32
// or 64): a TMA box per unit and group never crosses a page.  The map's 4-D view {64 dims, 8 rows, 8
// blocks, row groups} lands each 8 x 64 block as one 1024-byte swizzle atom with constant strides
// between atoms, which one matrix descriptor per 64 dims covers.  Units behind the request's end and
// pages with a bad id load out of bounds (zeros).  Rank 1 takes a request's last tile by groups of
// eight rows, with zeros behind the end's group, and sets the rows behind the end in that group to
// zero in shared memory before P C reads them (whatever they held, 0 * NaN included); rank 0's scores
// of them are masked.
//
// Precision.  q and the rotated band are bf16 pairs, hi + lo to 2^-17; P is bf16 (a relative 2^-9 on average,
// on the weights of an average; the sums take the unrounded ones); partials are fp16 with a power of two per
// half row.  Errors below: the output's over that of an fp32 evaluation rounded to bf16.
//   Up to 64 heads the MMAs' idle rows, 64 on, carry the low halves of both: of q and the band in the scores,
// which the softmax adds to the head's, and of P in the values.  Error 1.00-1.01 at every length and size of
// the scores.
//   Above 64 heads the scores take q_hi and both halves of the band.  What they leave of q_lo shifts a part's
// log-sum-exp by scale q_lo . o to first order, which the join adds, and errs in the weights by scale q_lo . c_j,
// a relative 2^-9 times the scores' deviation, and in the log-sum-exp by half the square of that: both grow
// with the scores.  q_lo of 256 of the 512 dims has MMAs up to 1024 keys (EX_WIDE), of 128 dims up to 4096
// (EX_LATENT): tensor memory has room for that many, the other half of EX_WIDE's is read in shared memory.
// Measured, 128 heads, scores of standard deviation 1 / 2 / 4 / 8 (log-sum-exp: largest error relative to it):
//    200 keys  1.43 / 1.50 / 1.63 / 1.82   6e-7 / 2e-6 / 3e-6 / 6e-6
//   1000 keys  1.39 / 1.58 / 1.74 / 2.09   3e-7 / 1e-6 / 3e-6 / 7e-6
//   3000 keys  1.41 / 1.66 / 1.99 / 2.54   3e-7 / 1e-6 / 4e-6 / 6e-6
//   8192 keys  1.46 / 1.78 / 2.15 / 2.66   3e-7 / 1e-6 / 3e-6 / 7e-6
// The limits: 128 dims up to 8192 keys too would be 1.47 for 1.49 at unit scale (60 random cases), but tiles of
// 7 % more MMAs hold up their cluster's equal share (64 ragged requests 294 -> 315 us); all 512 dims need eight more
// blocks of tensor memory than there are, and 64 more MMAs on a tile's 40.
//   Up to 64 keys (EX_BAND) the log-sum-exp is small and bf16 pairs show in it: the band's third part has
// MMAs, above 64 heads q_lo of 192 dims too, and the join adds the latent's third part (1 to 3 keys:
// 1.5e-6 -> 8e-7 of its value).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "paged_tc.cuh"
#include "tc_internal.h"

namespace mla {

__device__ unsigned g_paged_tc_err = 0;

namespace {

using namespace tc;
using namespace paged;

constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// ------------------------------------------------------------------------ absorb ----
// q[b, h, :] = W_K(h)^T q_nope[b, h, :]: streams 16 KB x heads x 8 of weights for B x 128 x 512
// multiply-adds a head, so it is bound by the weights' bytes until B is in the hundreds; the
// products run on mma.sync (M = latent dims, N = requests: eight per step, no padding to 128
// rows).  Block (head, 128 latent dims, group of up to 64 requests): the weight block and the group's
// queries by cp.async, all in flight at once; the weights then stay in registers as A fragments.  (Of the tokens of a
// step that are listed, which may be few of those that the grid is for, a block takes several groups in turn.)
// 128 heads, events around it alone: one request 10 us, 64 requests 17 us (20 with three
// blocks an SM, whose 512 blocks took a second wave; 17 MB of weights, 2.5 us at the copy
// peak; 19 MB of queries out).
constexpr int AB_DIMS = 128, AB_PITCH = 256 + 16, AB_GROUP = 64;
constexpr int AB_OUT = 40;              // halves per request of a warp's staging (32 dims + pad)
constexpr int AB_SMEM = DN * AB_PITCH + AB_GROUP * AB_PITCH + AB_GROUP * 4;   // four blocks an SM
static_assert(4 * 3 * 8 * AB_OUT * 2 <= DN * AB_PITCH, "the staging lies where the weights were");

template <bool STEP>
__global__ void __launch_bounds__(128) paged_absorb_tc_kernel(const __grid_constant__ Absorb a, const __grid_constant__ PagedPlan plan) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const PagedDecode &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // A step's plan, but for few tokens, is the launch in front and runs beside this one (it began behind the end of all
    // before it, and nothing here reads what it writes): the wait for it is at each block's end, for the launch behind.
    const bool behind = STEP && !plan.s.cu;
    if (!behind) pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0) {
        if (behind) {
            pdl_wait();
        } else if (STEP) {
            for (int i = tid; i < plan.n_zero; i += 128) plan.zero[i] = 0;
            plan_tokens<128, 1>(p, plan, p.T, (int *)sm);
        } else {
            plan_block<128, false>(p, (int *)sm, AB_SMEM / 4);
        }
        return;
    }
    if ((int)blockIdx.x <= a.rot_blocks) {
        rotate_queries<STEP>(a, ((int)blockIdx.x - 1) * 4 + warp, lane);
        if (behind) pdl_wait();
        return;
    }
    uint8_t *sq = sm + DN * AB_PITCH;
    const int T = STEP ? tokens_of(p) : p.B;
    int u = (int)blockIdx.x - 1 - a.rot_blocks;
    const int dc = u & 3;
    u >>= 2;
    const int h = u / a.blocks;
    int b0 = u % a.blocks * a.group;
    if (STEP && b0 >= T) {
        pdl_wait();
        return;
    }
    const bf16 *w = (const bf16 *)p.w + (long)h * (DN + DV) * DK + dc * AB_DIMS;
    int *keys = (int *)(sm + AB_SMEM) - AB_GROUP;
    auto load = [&](int nb) {
        for (int i = tid; i < nb * 16; i += 128)
            cp16(sq + (i >> 4) * AB_PITCH + (i & 15) * 16,
                 (const bf16 *)p.q_nope + ((long)(STEP ? token_of(p, b0 + (i >> 4)) : b0 + (i >> 4)) * p.H + h) * DN + (i & 15) * 8);
    };
    auto set_keys = [&](int nb) {
        if (tid < nb) keys[tid] = !STEP ? keys_of(p, b0 + tid) : p.scores_only ? 2147483647 : 0;
    };
    load(min(a.group, T - b0));
#pragma unroll 4
    for (int i = tid; i < DN * (AB_DIMS / 8); i += 128)
        cp16(sm + (i >> 4) * AB_PITCH + (i & 15) * 16, w + (long)(i >> 4) * DK + (i & 15) * 8);
    set_keys(min(a.group, T - b0));   // (behind the copies: it waits for its own load)
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    uint32_t A[2][8][4];
    const int mi = lane >> 3, r = lane & 7;   // matrix of an x4 load, its row
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int s = 0; s < 8; ++s)   // matrices: (dims 0-7, k 0-7), (dims 8-15, k 0-7), the same of k 8-15
            ldsm4_t(A[m][s], smem_u32(sm + (16 * s + (mi >> 1) * 8 + r) * AB_PITCH + (warp * 32 + m * 16 + (mi & 1) * 8) * 2));
    __syncthreads();   // all have their weights: the room is the staging's
    const int g = lane >> 2, t = lane & 3;
    uint16_t *sh = (uint16_t *)sm + warp * 3 * 8 * AB_OUT, *sl = sh + 8 * AB_OUT,
             *sr = sl + 8 * AB_OUT;
#pragma unroll 1
    for (;;) {
        const int nb = min(a.group, T - b0);
#pragma unroll 1
        for (int b = 0; b < nb; b += 8) {   // (rows behind the group's last request are not read back)
            float d[2][4] = {};
#pragma unroll
            for (int s = 0; s < 4; ++s) {   // 32 of the summed dims
                uint32_t q[4];
                ldsm4(q, smem_u32(sq + (b + r) * AB_PITCH + (32 * s + mi * 8) * 2));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma_16816(d[m], A[m][2 * s], q[0], q[1]);
                    mma_16816(d[m], A[m][2 * s + 1], q[2], q[3]);
                }
            }
            // d[m][..]: dim 16 m + g (+ 8), requests 2t, 2t + 1
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t hi, lo, rest;
                    split3(d[m][2 * e], d[m][2 * e + 1], hi, lo, rest);
                    const int dim = 16 * m + 8 * e + g;
                    sh[(2 * t) * AB_OUT + dim] = (uint16_t)hi;
                    sh[(2 * t + 1) * AB_OUT + dim] = (uint16_t)(hi >> 16);
                    sl[(2 * t) * AB_OUT + dim] = (uint16_t)lo;
                    sl[(2 * t + 1) * AB_OUT + dim] = (uint16_t)(lo >> 16);
                    sr[(2 * t) * AB_OUT + dim] = (uint16_t)rest;
                    sr[(2 * t + 1) * AB_OUT + dim] = (uint16_t)(rest >> 16);
                }
            __syncwarp();
            if (b + g < nb) {   // 8 requests x 64 bytes: a 16-byte piece per lane
                const long o = ((long)(b0 + b + g) * p.H + h) * DK + dc * AB_DIMS + warp * 32 + t * 8;
                *(uint4 *)(a.qhi + o) = *(const uint4 *)(sh + g * AB_OUT + t * 8);
                *(uint4 *)(a.qlo + o) = *(const uint4 *)(sl + g * AB_OUT + t * 8);
                if (keys[b + g] <= SHORT_KEYS) *(uint4 *)(a.qrest + o) = *(const uint4 *)(sr + g * AB_OUT + t * 8);
            }
            __syncwarp();
        }
        b0 += a.blocks * a.group;
        if (!STEP || b0 >= T) break;
        __syncthreads();   // the group has been read
        load(min(a.group, T - b0));
        set_keys(min(a.group, T - b0));
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        __syncthreads();
    }
    if (behind) pdl_wait();
}

// -------------------------------------------------------------------------- join ----
// out[b, h, :] = W_V(h) sum_c w_c o_c: a block holds W_V(h) in shared memory (by TMA, from the L2 into
// which the attention's last tiles brought it) and walks groups of 32 requests.  Latency is what it
// spends, so each phase has its loads in flight at once: a warp per request forms the parts'
// weights; the merge runs over 16 groups of 64 threads (a thread per eight latent dims), which share
// out the requests, or, for one or two requests, their parts; the product is tcgen05 (M = 128 value
// dims, N = 32 requests, o as bf16 hi + lo, so that it is as exact as fp32 o): 64 MMAs of 32
// columns, where mma.sync took 7500 cycles a group.  128 heads, events around it alone: one request
// 14-16 us, 64 requests 26-28 us (33 with mma.sync); barriers and loads from memory share the stalls, and at 64
// registers 46 bytes spill.
constexpr int JB = 32, JNT = 1024, JMAXC = 80;
constexpr int JO = DV * DK * 2;                // W_V: eight boxes of 64 dims x 128 rows
constexpr int JBLK = JB * 128;                 // o: 64 dims x 32 requests
constexpr int JW = JO + 2 * 8 * JBLK;          // o hi, o lo; before them the groups' sums [16][2][512]
constexpr int JV = JW + 2 * JB * JMAXC * 4;    // the parts' weights for either half of the dims; then out [request][132]
struct JoinVars {
    uint64_t bar_w, bar_d;
    int sc[JB][4];            // first part, number of parts (-1: a token that is not computed here), Extra, row in the item
    int tok[JB];              // the tokens' rows in the step
    float sl[JB], sd[2][JB];  // log-sum-exp without the q_lo term; the warps' shares of q_lo . o
    uint32_t tslot;
    int abort;
};
constexpr int JSMEM = JV + sizeof(JoinVars);
static_assert(2 * 8 * JBLK >= 16 * 2 * DK * 4 && 2 * JB * JMAXC >= JB * 132, "the join's exchanges");
static_assert(PAGED_TC_WORKERS <= JMAXC && JMAXC <= 96, "parts of an item");

template <bool STEP>
__global__ void __launch_bounds__(JNT, 1) paged_join_tc_kernel(const __grid_constant__ CUtensorMap mW,
                                                               const __grid_constant__ PagedDecode p, const bf16 *qlo,
                                                               const bf16 *qrest, int per_head) {
    extern __shared__ __align__(1024) uint8_t sm[];
    if (smem_u32(sm) & 1023) {   // no room to align by hand; the same answer in every block
        if (threadIdx.x == 0) atomicOr(&g_paged_tc_err, 2u);
        return;
    }
    JoinVars &v0 = *(JoinVars *)(sm + JSMEM - sizeof(JoinVars));   // (static shared memory would push sm off its alignment)
    auto &sc = v0.sc;
    auto &sl = v0.sl;
    auto &sd = v0.sd;
    uint8_t *so = sm + JO;
    float (*sw)[JB][JMAXC] = (float (*)[JB][JMAXC])(sm + JW);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x / per_head, rt0 = h / p.row_tile, r0 = h % p.row_tile;   // (decode's; a step's vary by token)
    const long pitch = (long)p.row_tile * (DK / 8);
    const bool paired = p.row_tile <= 64;
    bool ok = true;
    if (STEP && (int)(blockIdx.x % per_head) * JB >= tokens_of(p)) {   // (a list's length is of a launch long ended)
        pdl_wait();
        return;
    }
    if (tid == 0) {
        mbar_init(&v0.bar_w, 1);
        mbar_init(&v0.bar_d, 1);
        v0.abort = 0;
        fence_mbar_init();
        mbar_arrive_expect_tx(&v0.bar_w, JO);
#pragma unroll 1
        for (int i = 0; i < 8; ++i) tma_load_2d(sm + i * 16384, &mW, &v0.bar_w, 64 * i, h * (DN + DV) + DN);
    }
    if (warp == 1) {
        tmem_alloc(&v0.tslot, 32);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = v0.tslot;
    pdl_wait();
    uint32_t ph = 0;
    const int T = STEP ? tokens_of(p) : p.B;
#pragma unroll 1
    for (int b0 = (int)(blockIdx.x % per_head) * JB; b0 < T; b0 += per_head * JB, ph ^= 1) {
        const int nb = min(JB, T - b0);
        if (STEP && __syncthreads_and(tid >= nb || __ldcg(&p.of[b0 + tid].x) < 0)) {
            ph ^= 1;   // (no phase of this turn's)
            continue;
        }
        const int d8 = tid & 63, q16 = tid >> 6;
        const bool few = nb <= 2;                                // the groups share out parts, not requests
        const int j0 = few ? 0 : q16, dj = few ? 1 : 16, c0 = few ? q16 : 0, dc = few ? 16 : 1;
        uint4 ql[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = j0 + dj * i;
            ql[i] = j < nb && !paired ? __ldcg((const uint4 *)(qlo + ((long)(b0 + j) * p.H + h) * DK) + d8) : make_uint4(0, 0, 0, 0);
        }
        {   // a warp per request: the weights of its parts (up to 96)
            int s0 = 0, n = 0, ex = EX_NONE, r = r0;
            bool here = true;
            if (warp < nb) {
                const int2 of = STEP ? __ldcg(p.of + b0 + warp) : make_int2(b0 + warp, 0);
                here = !STEP || of.x >= 0;
                if (here) {
                    ex = extra_of(paired, keys_of(p, of.x));
                    const int rt = STEP ? (of.y + h) / p.row_tile : rt0;
                    if (STEP) r = (of.y + h) % p.row_tile;
                    const int2 sp = __ldcg(p.spans + (long)of.x * p.row_tiles + rt);
                    s0 = sp.x;
                    n = sp.y;
                }
            }
            const long at = (long)s0 * p.row_tile + r;
            float x[3], m = -INFINITY, s = 0.f;
            float2 up[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const long k = at + (long)(lane + 32 * i) * p.row_tile;
                const bool in = lane + 32 * i < n;
                x[i] = in ? __ldcg(p.pl + k) : -INFINITY;
                up[i] = in ? __ldcg((const float2 *)p.pscale + k) : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 3; ++i) m = fmaxf(m, x[i]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                x[i] = x[i] == -INFINITY ? 0.f : expf(x[i] - m);
                s += x[i];
            }
            s = warp_sum(s);
            const float inv = s == 0.f ? 0.f : 1.f / s;
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (lane + 32 * i < n) {
                    sw[0][warp][lane + 32 * i] = x[i] * inv * up[i].x;
                    sw[1][warp][lane + 32 * i] = x[i] * inv * up[i].y;
                }
            if (lane == 0) {
                sc[warp][0] = s0;
                sc[warp][1] = here ? n : -1;
                sc[warp][2] = ex;
                if (STEP) {
                    sc[warp][3] = r;
                    v0.tok[warp] = warp < nb ? token_of(p, b0 + warp) : 0;
                }
                sl[warp] = s == 0.f ? -INFINITY : m + logf(s);
            }
        }
        __syncthreads();
        float o[2][8] = {};
        {
            const uint4 *src[2];
            int n[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = j0 + dj * i;
                src[i] = (const uint4 *)(p.po + ((long)sc[j][0] * p.row_tile + (STEP ? sc[j][3] : r0)) * DK) + d8;
                n[i] = sc[j][1];
            }
            const float *wt = sw[d8 >> 5][j0];
            const int most = max(n[0], n[1]);
#pragma unroll 1
            for (int c = c0; c < most; c += 3 * dc) {
                uint4 v[2][3];
#pragma unroll
                for (int u = 0; u < 3; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (c + u * dc < n[i]) v[i][u] = __ldcg(src[i] + (c + u * dc) * pitch);
#pragma unroll
                for (int u = 0; u < 3; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (c + u * dc < n[i]) {
                            const float x = wt[dj * i * JMAXC + c + u * dc];
                            const uint32_t w[4] = {v[i][u].x, v[i][u].y, v[i][u].z, v[i][u].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f = __half22float2(*(const __half2 *)&w[e]);
                                o[i][2 * e] = fmaf(x, f.x, o[i][2 * e]);
                                o[i][2 * e + 1] = fmaf(x, f.y, o[i][2 * e + 1]);
                            }
                        }
            }
        }
        if (few) {   // the groups' sums meet in the first
            float4 *x = (float4 *)so + d8 * 2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[(q16 * 2 + i) * 128] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                x[(q16 * 2 + i) * 128 + 1] = make_float4(o[i][4], o[i][5], o[i][6], o[i][7]);
            }
            __syncthreads();
            float sum = 0.f;   // a thread per request and dim
#pragma unroll
            for (int k = 0; k < 16; ++k) sum += ((float *)so)[(k * 2) * DK + tid];
            __syncthreads();
            ((float *)so)[tid] = sum;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[i][e] = q16 == 0 ? ((float *)so)[i * DK + d8 * 8 + e] : 0.f;
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = few ? 2 * q16 + i : j0 + dj * i;   // (few: the other groups bring rows of zeros)
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split2(o[i][2 * e], o[i][2 * e + 1], hi[e], lo[e]);
            uint4 *x = (uint4 *)(so + (d8 >> 3) * JBLK + j * 128 + (((d8 ^ j) & 7) << 4));   // 128-byte swizzle
            x[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            x[8 * JBLK / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            // the log-sum-exp's q_lo term: this warp's 256 dims
            const uint32_t q[4] = {ql[i].x, ql[i].y, ql[i].z, ql[i].w};
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dot += o[i][2 * e] * __uint_as_float(q[e] << 16) + o[i][2 * e + 1] * __uint_as_float(q[e] & 0xffff0000u);
            if ((lo_blocks((Extra)sc[j][2]) >> (d8 >> 3)) & 1) dot = 0.f;   // the scores have it
            if (sc[j][2] == EX_BAND && j < nb) {
                const uint4 x = __ldcg((const uint4 *)(qrest + ((long)(b0 + j) * p.H + h) * DK) + d8);
                const uint32_t z[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    dot += o[i][2 * e] * __uint_as_float(z[e] << 16) + o[i][2 * e + 1] * __uint_as_float(z[e] & 0xffff0000u);
            }
            dot = warp_sum(dot);
            if (lane == 0) sd[warp & 1][j] = dot;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        // (no keys: -inf stays, whatever the queries of a padded request hold; 0 * NaN is not added)
        if (tid < nb && (!STEP || sc[tid][1] >= 0)) p.lse[(long)(STEP ? v0.tok[tid] : b0 + tid) * p.H + h] = sl[tid] == -INFINITY ? sl[tid] : sl[tid] + p.scale * (sd[0][tid] + sd[1][tid]);
        if (warp == 0) {
            ok = __all_sync(FULL, ok && mbar_wait(&v0.bar_w, 0, (volatile int *)&v0.abort, &g_paged_tc_err));   // W_V is here
            tc_fence_after();
            if (ok && elect_one()) {
                const uint64_t a = sdesc_kmajor(sm), b = sdesc_kmajor(so);
                constexpr uint32_t idesc = idesc_f16(128, JB, false);
#pragma unroll 1
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint64_t ai = a + (uint64_t)(i * (16384 >> 4) + 2 * q), bi = b + (uint64_t)(i * (JBLK >> 4) + 2 * q);
                        mma_ss(tmem, ai, bi, idesc, (i | q) != 0);
                        mma_ss(tmem, ai, bi + (8 * JBLK >> 4), idesc, 1);
                    }
                mma_commit(&v0.bar_d);
            }
            __syncwarp();
        }
        float *ss = (float *)(sm + JW);   // out [request][128 dims + pad], where the weights were
        if (warp < 4) {
            ok = __all_sync(FULL, ok && mbar_wait(&v0.bar_d, ph, (volatile int *)&v0.abort, &g_paged_tc_err));
            tc_fence_after();
            uint32_t v[32];
            tmem_ld32_wait(tmem + ((uint32_t)(warp * 32) << 16), v);
            tc_fence_before();
#pragma unroll
            for (int j = 0; j < JB; ++j) ss[j * 132 + tid] = __uint_as_float(v[j]);
        }
        __syncthreads();
        if (warp < nb && (!STEP || sc[warp][1] >= 0)) {   // (an abandoned wait leaves rubbish here, and the error word)
            const float4 v = *(const float4 *)(ss + warp * 132 + lane * 4);
            *(uint2 *)((bf16 *)p.out + ((long)(STEP ? v0.tok[warp] : b0 + warp) * p.H + h) * DV + lane * 4) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        }
        __syncthreads();
    }
    // W_V lands before the block leaves, also where all of its tokens are of no request and no turn has waited for it
    if (STEP && warp == 0) mbar_wait(&v0.bar_w, 0, (volatile int *)&v0.abort, &g_paged_tc_err);
    if (warp == 1) tmem_dealloc(tmem, 32);
}

// --------------------------------------------------------------------- attention ----
constexpr int ROWS = 128, NK = 64, NTHREADS = 608;
constexpr int NGRP = NK / 8;            // row groups of a tile
constexpr int KST = 2, KGRP = 3;        // rank 0: tile stages, block groups of a stage
constexpr int VSL = 4;                  // rank 1: slots of half a tile (256 latent dims)
constexpr int NPB = 2;                  // P slots of rank 1 = staging slots of rank 0
// tiles prefetched into L2 ahead of rank 1's loads (76 requests of 32000 keys: 1 tile 526 us, 3 and 4
// 520, 6 527, 10 656)
constexpr int PF = 4;
constexpr uint32_t ATOM = 1024;
// rank 0 stage: groups of 64-dim blocks {0-2}, {3-5}, {6-7}, each [row group][block][8 rows], then the
// key band [row group][8 rows]
constexpr uint32_t KG1 = NGRP * 3 * ATOM, KG2 = 2 * KG1, KG3 = KG2 + NGRP * 2 * ATOM, KSTAGE = KG3 + NGRP * ATOM;
constexpr uint32_t VHALF = NGRP * 4 * ATOM;   // [row group][block][8 rows]
// One P transfer: P [128 heads][64 keys] bf16 as the K-major A operand of P C, then the per-head
// extras: rescale factor, 1/l and m + log2(l) (both on a part's last tile), a flag per lane quarter.
constexpr uint32_t P_BYTES = 16384;
constexpr uint32_t X_ALPHA = 0, X_INVL = 512, X_LSE = 1024, X_FLAG = 1536, X_BYTES = X_FLAG + 16;
constexpr uint32_t XOFF = P_BYTES, XSLOT = 18432, EXT_STRIDE = 1664;
// rank 0: key stages (between parts: query boxes 0-8), two more query boxes, P staging, extras, row maxima [tile parity][half][row], row sums
constexpr uint32_t OFF_Q = KST * KSTAGE, OFF_STG = OFF_Q + 2 * 16384, OFF_EXT = OFF_STG + NPB * P_BYTES;
constexpr uint32_t OFF_RED = OFF_EXT + NPB * EXT_STRIDE, OFF_SUM = OFF_RED + 2 * 2 * ROWS * 4;
// rank 1: latent slots, P slots, 1/l of each row for the epilogue's other warps [part parity][row], the
// epilogue's transposes (4 KB a warp)
constexpr uint32_t OFF_PB = VSL * VHALF, OFF_INV = OFF_PB + NPB * XSLOT, OFF_OUT = OFF_INV + 2 * ROWS * 4;
constexpr uint32_t END0 = OFF_SUM + 2 * ROWS * 4, END1 = OFF_OUT + 8 * 4096;
constexpr uint32_t OFF_BAR = END0 > END1 ? END0 : END1;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 512;
constexpr uint32_t T_S = 0, T_Q = 2 * NK;   // rank 0's TMEM columns: S buffers; 32 per 64 query dims (hi 0-7, band hi and lo, lo 0-1 or
                                             // EX_BAND's rest; paired: hi over lo 0-7, band hi over lo, EX_BAND's rest)
constexpr float RESCALE_LOG2 = 8.0f;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert(KSTAGE % 1024 == 0 && OFF_STG % 1024 == 0 && OFF_PB % 1024 == 0 && XSLOT % 1024 == 0, "swizzle atoms");
static_assert(XOFF + X_BYTES <= XSLOT && X_BYTES <= EXT_STRIDE && OFF_EXT % 16 == 0, "P transfer layout");
static_assert(T_Q + 12 * 32 <= 512, "TMEM budget of rank 0");
static_assert(5 * 16384 >= KSTAGE && 9 * 16384 <= KST * KSTAGE, "query boxes in the key stages");
// Barriers, by index; the same places in both CTAs.
enum : int {
    B_GFULL = 0,                 // rank 0 [stage][group]: boxes landed / read by the MMAs
    B_GEMPTY = B_GFULL + 6,
    B_SFULL = B_GEMPTY + 6,      // rank 0 [buffer]: scores done / drained by the softmax
    B_SFREE = B_SFULL + 2,
    B_STAGED = B_SFREE + 2,      // rank 0 [slot]: P staged / its copy has read it
    B_STGFREE = B_STAGED + 2,
    B_QFULL = B_STGFREE + 2,     // rank 0: the part's query boxes landed
    B_KFREE = B_QFULL + 1,       // rank 0 [stage]: the boxes there are in TMEM (parts that use the stage)
    B_QREADY = B_KFREE + 2,      // rank 0: the part's queries in TMEM / no longer read by MMAs
    B_QFREE = B_QREADY + 1,
    B_PEMPTY = B_QFREE + 1,      // both [slot]: P consumed (one multicast commit completes it in both)
    B_PFULL = B_PEMPTY + 2,      // rank 1 [slot]: P and extras landed / O rescaled for it
    B_PCREADY = B_PFULL + 2,
    B_VFULL = B_PCREADY + 2,     // rank 1 [slot]: half a tile landed / read by the MMAs
    B_VEMPTY = B_VFULL + VSL,
    B_OFINAL = B_VEMPTY + VSL,   // rank 1: the part's O complete / read
    B_EPIDONE = B_OFINAL + 1,
    B_QNEXT = B_EPIDONE + 1,     // rank 0: the two boxes behind the key stages are in TMEM
    B_COUNT = B_QNEXT + 1
};
__device__ __forceinline__ uint32_t arrivals(int i) {
    if (i >= B_SFREE && i < B_STGFREE) return 8;   // one per softmax warp
    if ((i >= B_KFREE && i <= B_QREADY) || (i >= B_PCREADY && i < B_VFULL) || i == B_QNEXT) return 4;
    if (i == B_QFREE) return 2;
    return i == B_EPIDONE ? 8 : 1;
}

struct Maps {
    CUtensorMap k3, k2, v, r;   // boxes of a unit's rows: blocks 0-2 / 3-5, blocks 6-7, four blocks, key band
    CUtensorMap v8;             // eight rows, four blocks
    CUtensorMap qh, ql, rh, rl, rr; // query rows of 512 and of 64 dims: hi, lo, rest (a box may reach into another group's)
};
struct Attn {
    PagedDecode p;
    int q_rows;                 // rows of the query boxes
    const bf16 *qlo;
    Divisor by_page;
    float scale_log2;
    uint32_t idesc_s, idesc_pv;
};

// Code size counts here: it is fetched through the L2 that the cache streams through, and what a role
// runs seldom comes from DRAM each time.  Hence parts as a list (PagedPart) made once, waits
// whose slow side is one function, rolled loops around small bodies.  The same kernel at 95 KB of
// code took 1.4 us a tile where 82 KB took 1.0.

// The cache row of key `key` of the part's request, -1 for none (behind the end, a bad page id).
__device__ __forceinline__ int row_of(const Attn &a, const PagedPart &w, int key) {
    if (key >= w.keys) return -1;
    const int col = quotient(a.by_page, key);
    const int id = __ldg(a.p.table + (long)w.row * a.p.max_pages + col);
    return (unsigned)id < (unsigned)a.p.num_pages ? id * a.p.page + (key - col * a.p.page) : -1;
}

// The cache rows of the part's units, a window of 64 units in two registers of the warp: fetched 32
// at a time, tiles ahead of their use (under the cache stream a table entry takes longer than a tile
// to arrive).
template <int UNIT>
struct Rows {
    int cur, nxt, base;   // units base + lane, base + 32 + lane; base < 0 before the first tile
    // The row of unit `lane` of tile i (lanes below NK / UNIT; a tile never straddles the registers).
    __device__ __forceinline__ int tile(const Attn &a, const PagedPart &w, int i, int lane) {
        constexpr int N = NK / UNIT;
        while (i * N - base >= 32) {   // once in 32 units; twice for the first tile
            base += 32;
            cur = nxt;
            const int u = base + 32 + lane;
            nxt = u < w.nt * N ? row_of(a, w, w.k0 * NK + u * UNIT) : -1;
        }
        return __shfl_sync(FULL, cur, (i * N + lane - base) & 31);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bounded waits.  A tile takes about a microsecond; KERNEL_NS after the kernel's start and TILE_NS more
// for each tile of its share (requests may share pages, so there is no bound on those) a wait records
// the timeout and gives up, as does every other wait of the CTA.
constexpr uint64_t KERNEL_NS = 4000000000ull, TILE_NS = 20000ull;
struct Ctl {
    unsigned long long deadline;
    int abort;
};
__device__ __noinline__ bool gave_up(Ctl *c) {
    if (((volatile Ctl *)c)->abort) return true;
    if (global_ns() < ((volatile Ctl *)c)->deadline) return false;
    atomicOr(&g_paged_tc_err, ERR_WAIT_TIMEOUT);
    ((volatile Ctl *)c)->abort = 1;
    return true;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, Ctl *c) {
    for (uint32_t n = 1; !(CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)); ++n)
        if ((n & 63) == 0 && gave_up(c)) return false;
    return true;
}
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, Ctl *c) {
    return __all_sync(FULL, wait_for(bar, parity, c));
}

// PAIRED (items of up to 64 rows): the rows behind the heads, 64 on, carry the queries' low halves in the scores and P's
// in the values.  STEP: the tokens of a step, whose rows see each its own number of the group's keys.
template <int UNIT, bool PAIRED, bool STEP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    paged_attn_tc_kernel(const __grid_constant__ Maps m, const __grid_constant__ Attn a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {   // no room to align by hand; the same answer in every CTA
        if (threadIdx.x == 0) atomicOr(&g_paged_tc_err, 2u);
        return;
    }
    constexpr int UNITS = NK / UNIT, NRG = UNIT / 8;   // units of a tile, row groups of a unit
    uint64_t *bars = (uint64_t *)(smem + OFF_BAR);
    Ctl *ctl = (Ctl *)(bars + B_COUNT);
    uint32_t *tslot = (uint32_t *)(ctl + 1);
    volatile int *prog = (volatile int *)(tslot + 1);   // rank 1: tiles whose latent loads have begun
    static_assert(B_COUNT * 8 + sizeof(Ctl) + 8 <= 512, "barrier area");
    const PagedDecode &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    if (STEP && p.list && tokens_of(p) == 0) {   // (the list's length is of a launch long ended)
        pdl_wait();
        return;
    }

    if (warp == 0) {
        for (int i = lane; i < B_COUNT; i += 32) mbar_init(&bars[i], arrivals(i));
        if (lane == 0) {
            ctl->abort = 0;
            *prog = 0;
            ctl->deadline = global_ns() + KERNEL_NS;
        }
        fence_mbar_init();
        __syncwarp();
        if (rank == 1 && lane < NPB) mbar_arrive_expect_tx(&bars[B_PFULL + lane], P_BYTES + X_BYTES);   // armed for its first transfer
    }
    if (warp == 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    if (warp == 2 && lane < 10) tma_prefetch_desc((const CUtensorMap *)&m + lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any cross-CTA arrival
    tc_fence_after();
    const uint32_t tmem = *tslot;
    pdl_wait();
    pdl_launch_dependents();

    // this cluster's parts: a list from the division of the batch
    const PagedPart *part = p.parts + __ldcg(p.first + (blockIdx.x >> 1));
    const int n_all = __ldcg(p.first + p.workers + (blockIdx.x >> 1));   // tiles
    if (tid == 0 && n_all > 0) ((volatile Ctl *)ctl)->deadline += TILE_NS * n_all;
    PagedPart w{};
    bool more = n_all > 0;
    auto load = [&]() {
        const int4 x = __ldcg((const int4 *)part), y = __ldcg((const int4 *)part + 1);
        w.row = x.x;
        w.q = x.y;
        w.k0 = x.z;
        w.nt = x.w;
        w.keys = y.x;
        w.next = y.y;
        w.rows = y.z;
    };
    if (more) load();
    auto next = [&]() {
        more = w.next > 0;
        part += w.next;
        if (more) load();
    };
    constexpr bool paired = PAIRED;
    const int none = (int)((p.num_pages * (long)p.page) >> 3);   // a row group outside the cache: zeros

    if (rank == 0) {
        if (warp == 0 || warp == 12 || warp == 13) {
            // ------------------------------------------------- TMA producers, a warp per block group
            // a lane per unit of the tile's rows; the whole warp waits.  A group's refill costs the time
            // from its last MMA to the issue of its boxes, hence a warp for each.
            const int g = warp == 0 ? 0 : warp - 11;
            int n = 0;
            uint32_t moved = 0;   // per stage, the parity of the next move of queries out of it
            bool go = true;
            for (; more && go; next()) {
                Rows<UNIT> rows{-1, -1, -64};
#pragma unroll 1
                for (int i = 0; i < w.nt; ++i, ++n) {
                    const int s = n & 1;
                    uint8_t *dst = smem + s * KSTAGE + g * KG1 + lane * NRG * (g < 2 ? 3 : 2) * ATOM;
                    uint64_t *full = &bars[B_GFULL + s * KGRP + g];
                    const int row = rows.tile(a, w, i, lane), rg = row >= 0 ? row >> 3 : none;
                    // behind the MMAs of two tiles ago (a fresh barrier passes), a part's first tiles also behind
                    // the move of its queries, which lay in their stages
                    go = wait_all(&bars[B_GEMPTY + s * KGRP + g], ((n >> 1) & 1) ^ 1, ctl);
                    if (go && i < KST) {
                        go = wait_all(&bars[B_KFREE + s], (moved >> s) & 1, ctl);
                        moved ^= 1u << s;
                    }
                    if (!go) break;
                    if (lane == 0) mbar_arrive_expect_tx(full, NGRP * 3 * ATOM);
                    if (lane < UNITS) {
                        tma_load_4d(dst, g < 2 ? &m.k3 : &m.k2, full, 0, 0, 3 * g, rg);
                        if (g == 2) tma_load_2d(smem + s * KSTAGE + KG3 + lane * NRG * ATOM, &m.r, full, 0, rg * 8);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 1 || warp == 11) {
            // --------------------- S = Q K^T issuers: warp 1 even tiles, warp 11 odd tiles
            int n = 0, seg = 0;
            const int s = warp == 1 ? 0 : 1;
            const uint32_t base = smem_u32(smem + s * KSTAGE), dt = tmem + T_S + s * NK;
            bool ok = true;
            for (; more && ok; next(), ++seg) {
                ok = wait_all(&bars[B_QREADY], seg & 1, ctl);
                const Extra ex = extra_of(paired, w.keys);
                const unsigned lo = paired ? 0 : lo_blocks(ex);
                const int blocks = 9 + !paired + (ex == EX_BAND);
#pragma unroll 1
                for (int i = 0; i < w.nt && ok; ++i, ++n) {
                    if ((n & 1) != s) continue;
                    const uint32_t ph = (n >> 1) & 1;
                    ok = wait_all(&bars[B_SFREE + s], ph ^ 1, ctl);
#pragma unroll 1
                    for (int g = 0; g < KGRP; ++g) {
                        ok = ok && wait_all(&bars[B_GFULL + s * KGRP + g], ph, ctl);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            // blocks of 64 dims: latent 0-7 (q_hi), then the key band twice (hi, lo) or three times;
                            // paired, q_lo and the band's lo are rows of the same MMAs
                            uint64_t d = sdesc_sw128(base + g * KG1, 16, (g < 2 ? 3 : 2) * ATOM);
                            const int j1 = g < 2 ? 3 * g + 3 : blocks;
#pragma unroll 1
                            for (int j = 3 * g; j < j1; ++j) {
                                if (j >= 8) d = sdesc_sw128(base + KG3, 16, ATOM);
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    mma_ts(dt, tmem + T_Q + j * 32 + q * 8, d + 2 * q, a.idesc_s, (j | q) != 0);
                                d += ATOM >> 4;
                            }
                            if (lo)   // q_lo's blocks of this group: 0, 1 in TMEM, 2, 3 in the boxes behind the key stages
#pragma unroll 1
                                for (int j = 3 * g; j < min(3 * g + 3, 4); ++j) {
                                    if (!((lo >> j) & 1)) continue;
                                    const uint64_t kd = sdesc_sw128(base + g * KG1 + (j - 3 * g) * ATOM, 16, 3 * ATOM),
                                                   ql = sdesc_kmajor(smem + OFF_Q + (j & 1) * 16384);
#pragma unroll
                                    for (int q = 0; q < 4; ++q) {
                                        if (j < 2) mma_ts(dt, tmem + T_Q + (10 + j) * 32 + q * 8, kd + 2 * q, a.idesc_s, 1);
                                        else mma_ss(dt, ql + 2 * q, kd + 2 * q, a.idesc_s, 1);
                                    }
                                }
                            mma_commit(&bars[B_GEMPTY + s * KGRP + g]);
                            if (g == KGRP - 1) mma_commit(&bars[B_SFULL + s]);
                        }
                        __syncwarp();
                    }
                }
                // this warp's last score MMAs of the part: the queries may be replaced
                if (ok && elect_one()) mma_commit(&bars[B_QFREE]);
                __syncwarp();
            }
        } else if (warp >= 2 && warp < 10) {
            // ---------------------------------------------------------- softmax warps
            // two threads per head: warps 2-5 take keys 0-31 of a tile, warps 6-9 keys 32-63.  Paired, the
            // row 64 behind a head's has q_lo's scores: its two threads exchange halves with the head's and
            // each of the four takes 16 keys (with the head's two alone 76 requests of 16384 keys, 16
            // heads, took 279 us a call, with four 250).  An abandoned wait clears `ok`; the walk goes on without waiting, so
            // that all warps of a row reach every barrier.
            constexpr int HK = NK / 2, PER = paired ? 4 : 2, KN = NK / PER;   // scores here, threads of a head, keys of each
            constexpr int RED = ROWS * 2 / PER;
            const int quad = warp & 3, row = quad * 32 + lane, h = (warp - 2) >> 2;
            const int head = paired ? row & 63 : row, lo_row = paired ? quad >> 1 : 0, me = h + 2 * lo_row;
            const uint32_t sbase = tmem + ((uint32_t)(quad * 32) << 16) + T_S + h * HK;
            const float c = a.scale_log2;
            float *red = (float *)(smem + OFF_RED) + head, *sums = (float *)(smem + OFF_SUM) + head;
            int n = 0;
            bool ok = true;
            for (; more; next()) {
                // a warp without a row only keeps the barriers
                const bool act = (paired ? quad & 1 : quad) * 32 < w.rows;
                // keys that this row sees: a step's token not all of its group's
                const int lim = STEP && head < w.rows ? __ldcg(p.limits + (w.q + head) / p.H) : w.keys;
                // whether every page of the part has an id inside the cache
                bool sound = true;
                {
                    const int c0 = quotient(a.by_page, w.k0 * NK), c1 = quotient(a.by_page, min(w.keys, (w.k0 + w.nt) * NK) - 1);
                    const int *ids = p.table + (long)w.row * p.max_pages;
#pragma unroll 2
                    for (int col = c0 + lane; col <= c1; col += 32) sound = sound && (unsigned)__ldg(ids + col) < (unsigned)p.num_pages;
                    sound = __all_sync(FULL, sound);
                }
                float top = -INFINITY, l = 0.f;   // running maximum (scaled, log2 units), this thread's sum
#pragma unroll 1
                for (int i = 0; i < w.nt; ++i, ++n) {
                    const int s = n & 1;
                    const uint32_t ph = (n >> 1) & 1;
                    // bit g of the mask: row group g holds keys (looked up only where some page does not)
                    unsigned groups = (1u << NGRP) - 1;
                    if (!sound) groups = __ballot_sync(FULL, lane < NGRP && row_of(a, w, (w.k0 + i) * NK + lane * 8) >= 0);
                    ok = __all_sync(FULL, ok && wait_for(&bars[B_SFULL + s], ph, ctl));
                    tc_fence_after();
                    uint32_t sa[HK];   // paired: the 16 keys that this thread takes, then those it hands on
                    if (act) {
                        if (paired) tmem_ld16x2_wait(sbase + s * NK + lo_row * KN, sbase + s * NK + (lo_row ^ 1) * KN, sa);
                        else tmem_ld32_wait(sbase + s * NK, sa);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[B_SFREE + s]);
                    uint8_t *ext = smem + OFF_EXT + s * EXT_STRIDE;
                    // staging slot s: its copy of tile n - 2 has read it (a fresh barrier passes)
                    ok = __all_sync(FULL, ok && wait_for(&bars[B_STGFREE + s], ph ^ 1, ctl));
                    bool rescaled = false;
                    if (act) {
                        uint8_t *stg = smem + OFF_STG + s * P_BYTES + head * 128;   // (row + 64: the same swizzle)
                        // 16-byte piece q of this thread's keys of P, or of thread `of`'s
                        auto piece = [&](int q, int of) {
                            return (uint4 *)(stg + ((((of & 1) * (HK / 8) + (of >> 1) * (KN / 8) + q) ^ (row & 7)) << 4));
                        };
                        if (paired) {
                            // through the pieces of the staging slot that the receiving thread fills with P next
                            constexpr int LO = 64 * 128 / 16;
#pragma unroll
                            for (int q = 0; q < KN / 4; ++q) {
                                const uint32_t *x = sa + KN + 4 * q;
                                piece(q & 1, me ^ 2)[(q >> 1) * LO] = make_uint4(x[0], x[1], x[2], x[3]);
                            }
                            named_bar_sync(5 + 2 * (quad & 1) + h, 64);
#pragma unroll
                            for (int q = 0; q < KN / 4; ++q) {
                                const uint4 x = piece(q & 1, me)[(q >> 1) * LO];
                                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) sa[4 * q + e] = __float_as_uint(__uint_as_float(sa[4 * q + e]) + __uint_as_float(y[e]));
                            }
                        }
                        const int key0 = (w.k0 + i) * NK + h * HK + lo_row * KN;
                        if (groups != (1u << NGRP) - 1 || key0 + KN > lim) {
                            const int end = lim - key0;
                            groups >>= 4 * h + 2 * lo_row;
#pragma unroll
                            for (int e = 0; e < KN; ++e)
                                if (e >= end || !((groups >> (e >> 3)) & 1)) sa[e] = 0xff800000u;   // -inf
                        }
                        float mx[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(__uint_as_float(sa[e]), __uint_as_float(sa[e + 4]));
#pragma unroll
                        for (int e = 8; e < KN; e += 8)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(sa[e + q]), __uint_as_float(sa[e + q + 4])));
                        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        red[(s * PER + me) * RED] = mt;
                        named_bar_sync(1 + (paired ? quad & 1 : quad), 32 * PER);   // the warps of these 32 heads
#pragma unroll
                        for (int k = 1; k < PER; ++k) mt = fmaxf(mt, red[(s * PER + (me ^ k)) * RED]);
                        mt *= c;
                        // O is rescaled only when the maximum grows by more than 2^8 (all threads of a
                        // head decide alike from the same numbers)
                        const bool need = mt > top + RESCALE_LOG2;
                        float alpha = 1.f;
                        if (need) {
                            alpha = top == -INFINITY ? 0.f : ex2(top - mt);
                            top = mt;
                        }
                        rescaled = __any_sync(FULL, need && i > 0);
                        const float m_eff = top == -INFINITY ? 0.f : top;
                        float ra[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int q = 0; q < KN / 8; ++q) {
                            uint32_t pk[4], lo[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float p0 = ex2(fmaf(__uint_as_float(sa[8 * q + 2 * e]), c, -m_eff));
                                const float p1 = ex2(fmaf(__uint_as_float(sa[8 * q + 2 * e + 1]), c, -m_eff));
                                ra[e] += p0 + p1;
                                pk[e] = pack_bf16(p0, p1);
                                if (paired) lo[e] = pack_bf16(p0 - __uint_as_float(pk[e] << 16), p1 - __uint_as_float(pk[e] & 0xffff0000u));
                            }
                            uint4 *at = piece(q, me);
                            at[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                            if (paired) at[64 * 128 / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        }
                        l = l * alpha + ((ra[0] + ra[1]) + (ra[2] + ra[3]));
                        if (i == w.nt - 1) {   // the row's sum, with the other threads'
                            sums[me * RED] = l;
                            named_bar_sync(1 + (paired ? quad & 1 : quad), 32 * PER);
                            float lt = l;
#pragma unroll
                            for (int k = 1; k < PER; ++k) lt += sums[(me ^ k) * RED];
                            if (me == 0) {
                                ((float *)(ext + X_INVL))[row] = lt == 0.f ? 0.f : 1.f / lt;
                                ((float *)(ext + X_LSE))[row] = lt == 0.f ? -INFINITY : m_eff + log2f(lt);
                            }
                        }
                        if (me == 0) {
                            ((float *)(ext + X_ALPHA))[row] = alpha;
                            if (paired) ((float *)(ext + X_ALPHA))[row + 64] = alpha;
                        }
                    }
                    if (h == 0 && lane == 0) ((uint32_t *)(ext + X_FLAG))[quad] = rescaled ? 1u : 0u;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[B_STAGED + s]);
                }
            }
        } else if (warp == 10) {
            // ------------------------------- copier: staged P and extras -> rank 1
            if (lane == 0) {
                const uint32_t peer_slot0 = map_peer(smem_u32(smem + OFF_PB), 1);
                const uint32_t peer_full0 = map_peer(smem_u32(&bars[B_PFULL]), 1);   // armed by rank 1 itself
#pragma unroll 1
                for (int n = 0; n < n_all; ++n) {
                    const int s = n & 1;
                    const uint32_t ph = (n >> 1) & 1;
                    if (!wait_for(&bars[B_STAGED + s], ph, ctl)) break;
                    if (!wait_for<true>(&bars[B_PEMPTY + s], ph ^ 1, ctl)) break;   // (passes at first)
                    const uint32_t dst = peer_slot0 + s * XSLOT, bar = peer_full0 + s * 8;
                    bulk_copy_to_peer(dst, smem + OFF_STG + s * P_BYTES, P_BYTES, bar);
                    bulk_copy_to_peer(dst + XOFF, smem + OFF_EXT + s * EXT_STRIDE, X_BYTES, bar);
                    bulk_commit();
                    bulk_wait_read<0>();
                    mbar_arrive(&bars[B_STGFREE + s]);
                }
                bulk_wait_all();   // nothing in flight into the peer at exit
            }
        } else if (warp == 18) {
            // ------------------------------- the parts' query boxes: 64 dims x 128 heads each, hi of the latent
            // (0-7), hi and lo of the band (8, 9), Extra's (10); all in flight at once in the key stages, which
            // the last part's MMAs have left, and the two boxes behind them.  Paired: lo in the rows 64 on of hi's
            // boxes (0-8), the band's rest (9)
            int seg = 0;
            uint32_t wide = 0;   // parity of the moves waited for below
            bool go = lane == 0;
            for (; more && go; next(), ++seg) {
                const Extra ex = extra_of(paired, w.keys);
                const int boxes = ex == EX_NONE ? 10 : 11;
                go = wait_for(&bars[B_QFREE], (seg & 1) ^ 1, ctl);   // (passes at first)
                if (!go) break;
                if (paired) {
                    mbar_arrive_expect_tx(&bars[B_QFULL], (18 + (ex == EX_BAND)) * 128 * a.q_rows);
#pragma unroll 1
                    for (int j = 0; j < 9; ++j) {
                        tma_load_3d(smem + j * 16384, j < 8 ? &m.qh : &m.rh, &bars[B_QFULL], j < 8 ? 64 * j : 0, w.q, 0);
                        tma_load_3d(smem + j * 16384 + 64 * 128, j < 8 ? &m.ql : &m.rl, &bars[B_QFULL], j < 8 ? 64 * j : 0, w.q, 0);
                    }
                    if (ex == EX_BAND) tma_load_3d(smem + OFF_Q, &m.rr, &bars[B_QFULL], 0, w.q, 0);
                    continue;
                }
                mbar_arrive_expect_tx(&bars[B_QFULL], boxes * 128 * a.q_rows);
#pragma unroll 1
                for (int j = 0; j < boxes; ++j) {
                    const CUtensorMap *map = j < 8 ? &m.qh : (j == 8 ? &m.rh : (j == 9 ? &m.rl : (ex == EX_BAND ? &m.rr : &m.ql)));
                    tma_load_3d(smem + (j < 9 ? j * 16384 : OFF_Q + (j - 9) * 16384), map, &bars[B_QFULL], j < 8 ? 64 * j : 0, w.q,
                                0);
                }
                if (!(lo_blocks(ex) & 0xc)) continue;
                // lo of dims 128-255 for the MMAs to read in shared memory, once the two boxes there have moved
                go = wait_for(&bars[B_QNEXT], wide, ctl);
                if (!go) break;
                wide ^= 1;
                mbar_arrive_expect_tx(&bars[B_QFULL], 2 * 128 * a.q_rows);
#pragma unroll 1
                for (int j = 0; j < 2; ++j) tma_load_3d(smem + OFF_Q + j * 16384, &m.ql, &bars[B_QFULL], 64 * (j + 2), w.q, 0);
            }
        } else {
            // ------------------------------- queries into TMEM (warps 14-17, a thread per head)
            const int quad = warp & 3, row = quad * 32 + lane;
            const uint32_t dst = tmem + ((uint32_t)(quad * 32) << 16) + T_Q;
            uint32_t ph = 0;
            int n = 0;
            bool ok = true;
            for (; more && ok; n += w.nt, next()) {
                const bool act = (paired ? quad & 1 : quad) * 32 < w.rows;
                const Extra ex = extra_of(paired, w.keys);
                const int boxes = paired ? 9 + (ex == EX_BAND) : ex == EX_NONE ? 10 : 11;
                // q_lo of dims 64-127 has no box: each thread's 128 bytes come straight from memory, under
                // the boxes' flight
                uint4 x[8];
                const unsigned lo = paired ? 0 : lo_blocks(ex);
                if ((lo & 2) && act) {
                    const bf16 *src = a.qlo + (w.q + (long)min(row, w.rows - 1)) * DK + 64;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __ldcg((const uint4 *)src + e);
                }
                ok = wait_all(&bars[B_QFULL], ph, ctl);
                ph ^= 1;
                tc_fence_after();   // (the boxes landed behind the commit of the last part's MMAs)
                if ((lo & 2) && act && ok) {
                    uint32_t v[32];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[4 * e] = x[e].x;
                        v[4 * e + 1] = x[e].y;
                        v[4 * e + 2] = x[e].z;
                        v[4 * e + 3] = x[e].w;
                    }
                    tmem_st32(dst + 11 * 32, v);
                }
#pragma unroll 1
                for (int j = 0; j < boxes && ok; ++j) {
                    const uint8_t *box = smem + (j < 9 ? j * 16384 : OFF_Q + (j - 9) * 16384) + row * 128;
                    uint32_t v[32];
                    if (act) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint4 x = *(const uint4 *)(box + ((e ^ (row & 7)) << 4));
                            v[4 * e] = x.x;
                            v[4 * e + 1] = x.y;
                            v[4 * e + 2] = x.z;
                            v[4 * e + 3] = x.w;
                        }
                        if (paired && quad >= 2 && j == 9) {   // the band's rest has rows of the heads only
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = 0;
                        }
                        tmem_st32(dst + j * 32, v);
                    }
                    // Boxes 0-4 cover the first stage, 4-8 the second.  Only a stage that the part uses gets its
                    // phase: the producers wait for each, and none can still be open when the next part's test of
                    // its parity would pass on the phase before.
                    if ((j == 4 || j == 8) && (w.nt >= KST || (n & 1) == (j == 8))) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[B_KFREE + (j == 8)]);
                    }
                }
                if ((lo & 0xc) && ok) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[B_QNEXT]);
                    ok = wait_all(&bars[B_QFULL], ph, ctl);
                    ph ^= 1;
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_QREADY]);
            }
        }
    } else {
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (latent rows)
            int n = 0, slot = 0;
            uint32_t ph = 1;   // a fresh barrier's previous phase counts as complete
            bool go = true;
            for (; more && go; next()) {
                Rows<UNIT> rows{-1, -1, -64};
#pragma unroll 1
                for (int i = 0; i < w.nt && go; ++i) {
                    const int row = rows.tile(a, w, i, lane), end = w.keys - (w.k0 + i) * NK;
                    *prog = ++n;   // paces the prefetching warp
                    // a request's last tile goes by row groups, with zeros behind the last one with keys
                    const bool whole = end >= NK;
                    const int first = __shfl_sync(FULL, row, lane / NRG);
                    int rg = whole ? row : (first >= 0 && 8 * lane < end ? first + lane % NRG * 8 : -1);
                    rg = rg >= 0 ? rg >> 3 : none;
                    const int boxes = whole ? UNITS : NGRP;
                    const uint32_t off = lane * (whole ? NRG : 1) * 4 * ATOM;
#pragma unroll 1
                    for (int hf = 0; hf < 2 && go; ++hf) {
                        go = wait_all(&bars[B_VEMPTY + slot], ph, ctl);
                        if (!go) break;
                        uint64_t *full = &bars[B_VFULL + slot];
                        if (lane == 0) mbar_arrive_expect_tx(full, VHALF);
                        if (lane < boxes) tma_load_4d(smem + slot * VHALF + off, whole ? &m.v : &m.v8, full, 0, 0, 4 * hf, rg);
                        __syncwarp();
                        if (++slot == VSL) {
                            slot = 0;
                            ph ^= 1;
                        }
                    }
                }
            }
        } else if (warp == 10) {
            // ------------------------------- L2 prefetch of the tiles that rank 0 loads next
            // two tiles of key stages per cluster in flight do not cover DRAM's latency: tile n is
            // asked for when rank 1, which trails, loads tile n - PF
            int n = 0;
            bool go = true;
            for (; more && go; next()) {
                Rows<UNIT> rows{-1, -1, -64};
#pragma unroll 1
                for (int i = 0; i < w.nt && go; ++i, ++n) {
                    const int row = rows.tile(a, w, i, lane);
                    for (uint32_t k = 1; *prog < n - PF && go; ++k) {
                        __nanosleep(128);
                        if ((k & 1023) == 0 && gave_up(ctl)) go = false;
                    }
                    go = __all_sync(FULL, go);
                    if (row >= 0 && lane < UNITS) {
                        l2_prefetch((const bf16 *)p.c_cache + (long)row * DK, UNIT * DK * 2);
                        l2_prefetch((const bf16 *)p.kpe_cache + (long)row * DR, UNIT * DR * 2);
                    }
                    __syncwarp();
                }
            }
            // the share is asked for: now this cluster's share of W_V, which the join reads next, in
            // pieces of 16 KB
            for (int i = (blockIdx.x >> 1) + p.workers * lane; i < p.H * (DV * DK * 2 / 16384) && go; i += p.workers * 32)
                l2_prefetch((const bf16 *)p.w + ((long)(i >> 3) * (DN + DV) + DN + (i & 7) * 16) * DK, 16384);
        } else if (warp == 1) {
            // ---------------------------------------------------- O += P C issuer
            int n = 0, seg = 0, slot = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (; more && ok; next(), ++seg) {
                ok = wait_all(&bars[B_EPIDONE], (seg & 1) ^ 1, ctl);   // the last part's O has been read
#pragma unroll 1
                for (int i = 0; i < w.nt && ok; ++i, ++n) {
                    const int s = n & 1;
                    const int end = w.keys - (w.k0 + i) * NK;   // rows of the tile in front of the request's end
#pragma unroll 1
                    for (int hf = 0; hf < 2 && ok; ++hf) {
                        ok = wait_all(&bars[B_VFULL + slot], ph, ctl);
                        uint8_t *vs = smem + slot * VHALF;
                        if (end < NK && (end & 7)) {
                            // rows behind the end in its row group: zeros, whatever the cache holds there
#pragma unroll 1
                            for (int r = end; r & 7; ++r)
                                *(uint4 *)(vs + (r >> 3) * 4 * ATOM + (lane >> 3) * ATOM + (r & 7) * 128 + (lane & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        ok = __all_sync(FULL, ok && (hf || wait_for(&bars[B_PCREADY + s], (n >> 1) & 1, ctl)));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t pa = sdesc_kmajor(smem + OFF_PB + s * XSLOT);
                            const uint64_t vb = sdesc_sw128(smem_u32(vs), ATOM, 4 * ATOM);   // MN-major
#pragma unroll
                            for (int kk = 0; kk < NK / 16; ++kk)   // 16 keys per step, 256 latent dims per MMA
                                mma_ss(tmem + hf * 256, pa + (uint64_t)(2 * kk), vb + (uint64_t)(kk * (8 * ATOM >> 4)), a.idesc_pv,
                                       (i | kk) != 0);
                            mma_commit(&bars[B_VEMPTY + slot]);
                            if (hf) mma_commit_mc(&bars[B_PEMPTY + s], 3);
                        }
                        __syncwarp();
                        if (++slot == VSL) {
                            slot = 0;
                            ph ^= 1;
                        }
                    }
                }
                if (ok && elect_one()) mma_commit(&bars[B_OFINAL]);
                __syncwarp();
            }
        } else if (warp >= 2 && warp < 10) {
            // ------------------------ row rescale (warps 2-5) + epilogue (warps 2-9)
            const int quad = warp & 3, row = quad * 32 + lane, g = (warp - 2) >> 2;
            const uint32_t lb = tmem + ((uint32_t)(quad * 32) << 16);
            float *invs = (float *)(smem + OFF_INV) + row;
            int n = 0, seg = 0;
            bool ok = true;   // as in the softmax warps: every barrier is reached
            for (; more; next(), ++seg) {
                const bool act = quad * 32 < w.rows;
                const bool acc = act || (paired && quad >= 2 && (quad - 2) * 32 < w.rows);   // rows that O is kept for
                const long slot = part - p.parts;
                if (g == 0) {
                    float lse2 = -INFINITY, inv_l = 0.f;
#pragma unroll 1
                    for (int i = 0; i < w.nt && ok; ++i, ++n) {
                        const int s = n & 1;
                        const uint32_t ph = (n >> 1) & 1;
                        ok = __all_sync(FULL, wait_for<true>(&bars[B_PFULL + s], ph, ctl));
                        // slot s's previous use is over (its transfer waited for that), so the
                        // parity tests below are at most one phase behind
                        ok = __all_sync(FULL, ok && wait_for(&bars[B_PEMPTY + s], ph ^ 1, ctl));
                        if (!ok) break;
                        if (warp == 2 && lane == 0 && n + NPB < n_all) mbar_arrive_expect_tx(&bars[B_PFULL + s], P_BYTES + X_BYTES);
                        const uint8_t *xs = smem + OFF_PB + s * XSLOT + XOFF;
                        const uint4 fl = *(const uint4 *)(xs + X_FLAG);
                        if ((fl.x | fl.y | fl.z | fl.w) != 0u) {   // the same answer in every thread; i > 0
                            // O holds tile n - 1's product before it is rescaled
                            ok = wait_all(&bars[B_PEMPTY + (s ^ 1)], ((n - 1) >> 1) & 1, ctl);
                            if (!ok) break;
                            tc_fence_after();
                            const float al = acc ? ((const float *)(xs + X_ALPHA))[row] : 1.f;
                            if (__any_sync(FULL, al != 1.f)) {
#pragma unroll 1
                                for (int cc = 0; cc < 16; ++cc) {
                                    uint32_t o[32];
                                    tmem_ld32_wait(lb + cc * 32, o);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                                    tmem_st32(lb + cc * 32, o);
                                }
                                tmem_st_wait();
                            }
                            tc_fence_before();
                        }
                        if (i == w.nt - 1 && act) {
                            inv_l = ((const float *)(xs + X_INVL))[row];
                            lse2 = ((const float *)(xs + X_LSE))[row];
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[B_PCREADY + s]);
                    }
                    invs[(seg & 1) * ROWS] = inv_l;
                    if (ok && act && row < w.rows) p.pl[slot * p.row_tile + row] = lse2 * 0.69314718055994531f;
                }
                // ---- epilogue: the part's normalised output, 256 latent dims per warp: 64 columns of 32
                // heads at a time, turned in shared memory so that a store writes whole 128-byte lines.
                // An SM stores about 27 bytes a cycle, so 128 heads in fp32 took 4.8 us; fp16 with a
                // power of two per half row (|x| <= 2^15, half a step 2^-12 of the value) halves that,
                // at an error an eighth of the bf16 result's own.
                named_bar_sync(1 + quad, 64);   // the two warps of these 32 heads
                const float inv_l = invs[(seg & 1) * ROWS];
                ok = __all_sync(FULL, ok && wait_for(&bars[B_OFINAL], seg & 1, ctl));
                tc_fence_after();
                if (paired && acc && !act) {
                    // O of P's low halves, for the warp 64 rows in front, 32 columns at a time
                    uint8_t *buf = smem + OFF_OUT + (warp - 2) * 4096 + lane * 128;
#pragma unroll 1
                    for (int cc = 0; cc < 8; ++cc) {
                        uint32_t o[32];
                        tmem_ld32_wait(lb + 256 * g + 32 * cc, o);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *(uint4 *)(buf + ((e ^ (lane & 7)) << 4)) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        named_bar_sync(5 + 2 * (quad - 2) + g, 64);   // there
                        named_bar_sync(5 + 2 * (quad - 2) + g, 64);   // added
                    }
                }
                if (act) {   // (an abandoned wait leaves rubbish here, and the error word)
                    const int live = min(32, w.rows - quad * 32);
                    // the row's largest value here sets its power of two
                    float big = 0.f;
#pragma unroll 1
                    for (int cc = 0; cc < 8; ++cc) {
                        uint32_t o[32];
                        tmem_ld32_wait(lb + 256 * g + 32 * cc, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) big = fmaxf(big, fabsf(__uint_as_float(o[e])));
                    }
                    const int ex = (int)(__float_as_uint(big * inv_l) >> 23);   // 0 for a row of zeros, 255 for infinity
                    const float up = ex == 0 || ex == 255 ? 1.f : __uint_as_float((uint32_t)min(268 - ex, 254) << 23);
                    if (lane < live) p.pscale[(slot * p.row_tile + quad * 32 + lane) * 2 + g] = 1.f / up;
                    const float f = inv_l * up;
                    uint8_t *buf = smem + OFF_OUT + (warp - 2) * 4096;
                    const int r = lane >> 3;
                    __half *po = p.po + (slot * p.row_tile + quad * 32 + r) * DK + 256 * g + (lane & 7) * 8;
#pragma unroll 1
                    for (int cc = 0; cc < 4; ++cc, po += 64) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t o[32];
                            tmem_ld32_wait(lb + 256 * g + 64 * cc + 32 * k, o);
                            if (paired) {
                                const uint8_t *lo = smem + OFF_OUT + (4 * g + quad) * 4096 + lane * 128;
                                named_bar_sync(5 + 2 * quad + g, 64);
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float4 x = *(const float4 *)(lo + ((e ^ (lane & 7)) << 4));
                                    o[4 * e] = __float_as_uint(__uint_as_float(o[4 * e]) + x.x);
                                    o[4 * e + 1] = __float_as_uint(__uint_as_float(o[4 * e + 1]) + x.y);
                                    o[4 * e + 2] = __float_as_uint(__uint_as_float(o[4 * e + 2]) + x.z);
                                    o[4 * e + 3] = __float_as_uint(__uint_as_float(o[4 * e + 3]) + x.w);
                                }
                                named_bar_sync(5 + 2 * quad + g, 64);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {   // 16-byte piece 4 k + e of row `lane` at piece .. ^ (row mod 8)
                                uint32_t h[4];
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    h[q] = pack_f16(__uint_as_float(o[8 * e + 2 * q]) * f, __uint_as_float(o[8 * e + 2 * q + 1]) * f);
                                *(uint4 *)(buf + lane * 128 + (((4 * k + e) ^ (lane & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                            }
                        }
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {   // rows 4 e + r
                            const uint4 v = *(const uint4 *)(buf + (4 * e + r) * 128 + (((lane & 7) ^ ((4 * e + r) & 7)) << 4));
                            if (4 * e + r < live) *(uint4 *)(po + 4 * e * DK) = v;
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_EPIDONE]);
            }
        }
    }
    __syncwarp();
    if (tid == 0 && ((volatile Ctl *)ctl)->abort) settle();
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the peer may still address this CTA's barriers and slots until here
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

bool paged_tc_supported(int Dk, int Dn, int Dr, int Dv, int page) {
    return Dk == DK && Dn == DN && Dr == DR && Dv == DV && page % 8 == 0;
}

namespace {
Absorb absorb_of(const PagedDecode &p) {
    const size_t heads = (size_t)p.T * p.H;
    Absorb ab{};
    ab.p = p;
    ab.qhi = (bf16 *)p.qabs;
    ab.qlo = ab.qhi + heads * DK;
    ab.qrest = ab.qlo + heads * DK;
    ab.rhi = (bf16 *)p.qpe;
    ab.rlo = ab.rhi + heads * DR;
    ab.rrest = ab.rlo + heads * DR;
    // at least two blocks per SM, where the batch has that many groups of eight
    const int want = (2 * 152 + 4 * p.H - 1) / (4 * p.H), most = (p.T + 7) / 8;
    ab.groups = std::max((p.T + AB_GROUP - 1) / AB_GROUP, std::min(want, most));
    ab.group = ((p.T + ab.groups - 1) / ab.groups + 7) / 8 * 8;
    ab.groups = (p.T + ab.group - 1) / ab.group;
    // (of a list's tokens there may be few: blocks that find none are 25 us of launches at 2048 tokens, 128 heads)
    ab.blocks = p.list ? std::min(ab.groups, std::max(1, 2048 / (4 * p.H))) : ab.groups;
    ab.rot_blocks = (int)(((long)p.T * ((p.H + 31) / 32) + 3) / 4);
    std::copy_n(paged_turns(p.base, DR), DR / 2, ab.turns.v);
    return ab;
}
// Many tokens of a step (their plan is a launch of its own then): tiles of 128, a block an SM.  The absorb's from as many
// (head, tile) as half the SMs on: 20 heads, 512 tokens 17.5 us against 23.9 (80 of them), 32 heads, 144 tokens 15.3 against
// 12.4 to 14.2 (64).  The join's where the other's blocks would take three turns of 32 tokens: 32 heads of 1000 keys, 320
// tokens 18 us against 34, 144 tokens (two turns) 17 against 23, but with 8000 keys, whose tokens come in four parts and
// more, 30 against 17 (two turns) and 31 against 27 (three).
bool absorbs_many(const PagedDecode &p) { return (long)p.H * ((p.T + 127) / 128) >= PAGED_TC_WORKERS; }
bool joins_many(const PagedDecode &p, int per_head) { return (p.T + JB - 1) / JB > 2 * per_head; }
}  // namespace

cudaError_t paged_absorb_tc(const PagedDecode &p, const PagedPlan *plan, cudaStream_t st) {
    static_assert((4 * 128 + 1 + 1025) * 4 <= AB_SMEM, "the plan's room");
    const Absorb ab = absorb_of(p);
    if (p.groups && !plan && absorbs_many(p)) return paged_absorb_many(ab, st);
    auto kern = p.groups ? paged_absorb_tc_kernel<true> : paged_absorb_tc_kernel<false>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, AB_SMEM);
    if (e != cudaSuccess) return e;
    ProfScope ps("paged_absorb", st);
    return launch_after(kern, (unsigned)(p.H * 4 * ab.blocks + 1 + ab.rot_blocks), 128, AB_SMEM, st, ab, plan ? *plan : PagedPlan{});
}

namespace {
template <bool STEP>
auto attn_kernel(int unit, bool paired) {
    return paired ? (unit == 64   ? paged_attn_tc_kernel<64, true, STEP>
                     : unit == 32 ? paged_attn_tc_kernel<32, true, STEP>
                     : unit == 16 ? paged_attn_tc_kernel<16, true, STEP>
                                  : paged_attn_tc_kernel<8, true, STEP>)
                  : (unit == 64   ? paged_attn_tc_kernel<64, false, STEP>
                     : unit == 32 ? paged_attn_tc_kernel<32, false, STEP>
                     : unit == 16 ? paged_attn_tc_kernel<16, false, STEP>
                                  : paged_attn_tc_kernel<8, false, STEP>);
}
}  // namespace

cudaError_t paged_decode_tc(const PagedDecode &p, const PagedPlan *plan, cudaStream_t st) {
    using ull = unsigned long long;
    cudaError_t e;
    const ull rows = (ull)p.num_pages * p.page, heads = (ull)p.T * p.H;
    const Absorb ab = absorb_of(p);
    Attn at{};
    int unit = NK;   // rows that always share a page: the largest power of two up to a tile that divides one
    while (p.page % unit) unit /= 2;
    at.q_rows = std::min(ROWS, (p.row_tile + 31) / 32 * 32);
    at.qlo = ab.qlo;
    Maps m{};
    {
        const ull d[4] = {64, 8, 8, rows / 8}, s[3] = {1024, 128, 8192}, dr[2] = {64, rows}, sr[1] = {128};
        const unsigned g = (unsigned)unit / 8;
        const unsigned b3[4] = {64, 8, 3, g}, b2[4] = {64, 8, 2, g}, b8[4] = {64, 8, 4, g}, br[2] = {64, 8 * g};
        if ((e = make_tma_map(&m.k3, p.c_cache, 4, d, s, b3)) != cudaSuccess) return e;
        if ((e = make_tma_map(&m.k2, p.c_cache, 4, d, s, b2)) != cudaSuccess) return e;
        if ((e = make_tma_map(&m.v, p.c_cache, 4, d, s, b8)) != cudaSuccess) return e;
        if ((e = make_tma_map(&m.r, p.kpe_cache, 2, dr, sr, br)) != cudaSuccess) return e;
        const unsigned b1[4] = {64, 8, 4, 1};
        if ((e = make_tma_map(&m.v8, p.c_cache, 4, d, s, b1)) != cudaSuccess) return e;
    }
    {
        const unsigned bq[3] = {64, (unsigned)at.q_rows, 1};
        const ull d[3] = {DK, heads, 1}, s[2] = {DK * 2, heads * DK * 2};
        if ((e = make_tma_map(&m.qh, ab.qhi, 3, d, s, bq)) != cudaSuccess) return e;
        if ((e = make_tma_map(&m.ql, ab.qlo, 3, d, s, bq)) != cudaSuccess) return e;
        const ull dr[3] = {DR, heads, 1}, sr[2] = {DR * 2, heads * DR * 2};
        if ((e = make_tma_map(&m.rh, ab.rhi, 3, dr, sr, bq)) != cudaSuccess) return e;
        if ((e = make_tma_map(&m.rl, ab.rlo, 3, dr, sr, bq)) != cudaSuccess) return e;
        if ((e = make_tma_map(&m.rr, ab.rrest, 3, dr, sr, bq)) != cudaSuccess) return e;
    }
    at.p = p;
    at.by_page = divisor(p.page);
    at.scale_log2 = p.scale * 1.4426950408889634f;
    at.idesc_s = idesc_f16(128, NK, false);
    at.idesc_pv = idesc_f16(128, 256, false, true);
    auto join = p.groups ? paged_join_tc_kernel<true> : paged_join_tc_kernel<false>;
    if ((e = cudaFuncSetAttribute(join, cudaFuncAttributeMaxDynamicSharedMemorySize, JSMEM)) != cudaSuccess) return e;
    CUtensorMap mW;
    {
        const ull d[2] = {DK, (ull)p.H * (DN + DV)}, s[1] = {DK * 2};
        const unsigned b[2] = {64, DV};
        if ((e = make_tma_map(&mW, p.w, 2, d, s, b)) != cudaSuccess) return e;
    }
    const int per_head = std::max(1, std::min((p.T + JB - 1) / JB, 2 * p.workers / p.H));   // one wave of join blocks
    auto attn = p.groups ? attn_kernel<true>(unit, p.row_tile <= 64) : attn_kernel<false>(unit, p.row_tile <= 64);
    if ((e = cudaFuncSetAttribute(attn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES)) != cudaSuccess)
        return e;
    if ((e = paged_absorb_tc(p, plan, st)) != cudaSuccess) return e;
    {
        ProfScope ps("paged_attn", st);
        e = launch_after(attn, 2 * p.workers, NTHREADS, SMEM_BYTES, st, m, at);
    }
    if (e != cudaSuccess) return e;
    if (p.groups && !plan && joins_many(p, per_head)) return paged_join_many(p, ab.qlo, ab.qrest, st);
    {
        ProfScope ps("paged_join", st);
        e = launch_after(join, (unsigned)(p.H * per_head), JNT, JSMEM, st, mW, p, (const bf16 *)ab.qlo,
                         (const bf16 *)ab.qrest, per_head);
    }
    return e;
}

cudaError_t paged_tc_read_and_clear_error(unsigned *flags, cudaStream_t st) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_paged_tc_err, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
    if (e != cudaSuccess) return e;
    if ((e = cudaStreamSynchronize(st)) != cudaSuccess) return e;
    if (v) {
        unsigned z = 0;
        e = cudaMemcpyToSymbolAsync(g_paged_tc_err, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    *flags |= v;
    return e;
}

}  // namespace mla
