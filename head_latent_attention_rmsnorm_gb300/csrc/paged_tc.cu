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
//
// Attention.  One work item = 128 heads (fewer rows are zero-filled) of one request; its fp32
// accumulator, 128 x 512, is a whole SM's tensor memory, so an item runs on two SMs:
//   rank 0 (scores): q_hi in TMEM; 80-key tiles of the cache (latent + key band) through a
//     two-deep TMA ring that fills and drains in three groups of 64-dim blocks; S = Q K^T, two
//     S buffers; online softmax by eight warps (two threads per head); P in bf16 to rank 1 by bulk
//     copies into its two P slots;
//   rank 1 (accumulator): O in TMEM; streams the same tiles' latent (L2 hits: an idle warp
//     prefetches rank 0's next tiles) and issues O += P C.
// The persistent walk matters: equal shares of tiles per cluster (a request may be cut anywhere,
// parts meet in the join) leave no wave tail, and the next request's queries and first score tiles
// run under the previous one's drain and epilogue.
//
// Pages.  A tile is ten groups of eight rows; TMA boxes of 8 or 16 rows never cross a page.  The
// map's 4-D view {64 dims, 8 rows, 8 blocks, row groups} lands each 8 x 64 block as one 1024-byte
// swizzle atom with constant strides between atoms, which one matrix descriptor per 64 dims covers.
// Groups behind the request's end and pages with a bad id load out of bounds (zeros); rows behind
// the end inside a group are set to zero in shared memory before P C reads them (whatever they
// held, 0 * NaN included), and their scores are masked.
//
// Precision.  The score product takes q_hi; the band's lo half has MMAs of its own, and the missing
// latent term shifts a part's log-sum-exp by scale q_lo . o to first order, which the epilogue
// adds (the second order is half the variance of scale q_lo . c_j, ~1e-6 at unit scale).  q_lo
// keeps q to 2^-17.  P is bf16 (relative 2^-8 on the weights of an average; the sums take the
// unrounded ones).  Partials are fp32.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged_common.cuh"
#include "tc_common.cuh"
#include "tc_internal.h"

namespace mla {

__device__ unsigned g_paged_tc_err = 0;

namespace {

using namespace tc;
using namespace paged;
using bf16 = __nv_bfloat16;

constexpr unsigned FULL = 0xffffffffu;
constexpr int DK = 512, DN = 128, DR = 64, DV = 128;

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
__device__ __forceinline__ void cp16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// x as hi + lo in bf16 (hi its rounding, lo the rounding of the rest)
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

// ------------------------------------------------------------------------ absorb ----
// q[b, h, :] = W_K(h)^T q_nope[b, h, :]: streams 16 KB x heads x 8 of weights for B x 128 x 512
// multiply-adds a head, so it is bound by the weights' bytes until B is in the hundreds; the
// products run on mma.sync (M = latent dims, N = requests: eight per step, no padding to 128
// rows).  Block (head, 128 latent dims, group of requests): the weight block by cp.async, then in
// registers as A fragments, eight requests at a time against it.  The order of the 128 summed
// dims is permuted the same way in A and B so that a lane's share of q is 64 contiguous bytes.
constexpr int AB_DIMS = 128, AB_PITCH = AB_DIMS * 2 + 16;

struct Absorb {
    PagedDecode p;
    bf16 *qhi, *qlo, *rhi, *rlo;   // [B][H][512], [B][H][64]
    int groups, group;             // groups of `group` requests
    Turns turns;
};

__global__ void __launch_bounds__(128) paged_absorb_tc_kernel(const __grid_constant__ Absorb a) {
    __shared__ __align__(16) uint8_t sw[DN * AB_PITCH];
    __shared__ __align__(16) uint32_t st[4][2][8][20];   // per warp: hi / lo, 8 requests x 32 dims (+ pad)
    const PagedDecode &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    if (blockIdx.x == gridDim.x - 1) {
        plan_block<128>(p);
        return;
    }
    int u = blockIdx.x;
    const int dc = u & 3;
    u >>= 2;
    const int grp = u % a.groups, h = u / a.groups;
    const int b0 = grp * a.group, b1 = min(b0 + a.group, p.B);
    const bf16 *w = (const bf16 *)p.w + (long)h * (DN + DV) * DK + dc * AB_DIMS;
    for (int i = tid; i < DN * (AB_DIMS / 8); i += 128) {
        const int n = i >> 4, c = i & 15;
        cp16(sw + n * AB_PITCH + c * 16, w + (long)n * DK + c * 8);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // the query's rotation: this block's share of its requests
    for (int i = tid; i < (b1 - b0) * (DR / 2); i += 128) {
        const int b = b0 + (i >> 5), t = i & 31;
        if ((b & 3) != dc) continue;
        const long row = ((long)b * p.H + h) * DR;
        const float2 cs = turn_cs(a.turns.v[t], keys_of(p, b) - 1);
        const bf16 *x = (const bf16 *)p.q_pe + row;
        const float x0 = __bfloat162float(x[t]), x1 = __bfloat162float(x[t + 32]);
        uint32_t hi, lo;
        split2(x0 * cs.x - x1 * cs.y, x1 * cs.x + x0 * cs.y, hi, lo);
        ((uint16_t *)a.rhi)[row + t] = (uint16_t)hi;
        ((uint16_t *)a.rhi)[row + t + 32] = (uint16_t)(hi >> 16);
        ((uint16_t *)a.rlo)[row + t] = (uint16_t)lo;
        ((uint16_t *)a.rlo)[row + t + 32] = (uint16_t)(lo >> 16);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // step s of the sum: k = 2t, 2t + 1 is dim 32 t + 4 s + {0, 1}, k = 2t + 8, + 9 the next two
    uint32_t A[2][8][4];
    {
        const int mi = lane >> 3, r = lane & 7;   // matrix of the x4 load, its row k
        const int krow = (r >> 1) * 32 + (r & 1) + ((mi >> 1) ? 2 : 0);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int s = 0; s < 8; ++s)   // matrices: (dims 0-7, k 0-7), (dims 8-15, k 0-7), (.., k 8-15) x 2
                ldsm4_t(A[m][s], smem_u32(sw + (krow + 4 * s) * AB_PITCH + (warp * 32 + m * 16 + (mi & 1) * 8) * 2));
    }
    const int g = lane >> 2, t = lane & 3;
    for (int b = b0; b < b1; b += 8) {
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = make_uint4(0, 0, 0, 0);
        if (b + g < b1) {
            const uint4 *src = (const uint4 *)((const bf16 *)p.q_nope + ((long)(b + g) * p.H + h) * DN + t * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = __ldg(src + i);
        }
        float d[2][4] = {};
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const uint4 v = q[s >> 1];
            const uint32_t k0 = (s & 1) ? v.z : v.x, k1 = (s & 1) ? v.w : v.y;
            mma_16816(d[0], A[0][s], k0, k1);
            mma_16816(d[1], A[1][s], k0, k1);
        }
        // d[m][..]: dim 16 m + g (+ 8), requests 2t, 2t + 1
        uint16_t *sh = (uint16_t *)&st[warp][0][0][0], *sl = (uint16_t *)&st[warp][1][0][0];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t hi, lo;
                split2(d[m][2 * e], d[m][2 * e + 1], hi, lo);
                const int dim = 16 * m + 8 * e + g;
                sh[(2 * t) * 40 + dim] = (uint16_t)hi;
                sh[(2 * t + 1) * 40 + dim] = (uint16_t)(hi >> 16);
                sl[(2 * t) * 40 + dim] = (uint16_t)lo;
                sl[(2 * t + 1) * 40 + dim] = (uint16_t)(lo >> 16);
            }
        __syncwarp();
        if (b + g < b1) {   // 8 requests x 64 bytes: a 16-byte piece per lane
            const long o = ((long)(b + g) * p.H + h) * DK + dc * AB_DIMS + warp * 32 + t * 8;
            *(uint4 *)(a.qhi + o) = *(const uint4 *)&st[warp][0][g][t * 4];
            *(uint4 *)(a.qlo + o) = *(const uint4 *)&st[warp][1][g][t * 4];
        }
        __syncwarp();
    }
}

// -------------------------------------------------------------------------- join ----
// out[b, h, :] = W_V(h) sum_c w_c o_c: block (head, 64 value dims, 16 requests).  A warp holds its
// 16 rows of W_V in registers (loaded before the wait for the attention), the block merges the
// partials into shared memory as bf16 hi + lo, and two m16n8k16 products per step take both halves.
// A step's 16 summed dims are permuted alike in A and B: lane t of a row owns dims 64 i + 16 t ..
// + 15, four dims a step.
constexpr int JB = 16, JROWS = 64, JPITCH = DK * 2 + 16, JMAXC = 80;

__global__ void __launch_bounds__(128) paged_join_tc_kernel(const __grid_constant__ PagedDecode p) {
    __shared__ __align__(16) uint8_t so[2][JB * JPITCH];
    __shared__ float sw[JB][JMAXC];
    __shared__ int sc[JB][2];   // first worker, number of parts
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    int u = blockIdx.x;
    const int vc = u & 1;
    u >>= 1;
    const int nb_groups = (p.B + JB - 1) / JB, h = u / nb_groups, b0 = (u % nb_groups) * JB, nb = min(JB, p.B - b0);
    const int rt = h / p.row_tile, r = h % p.row_tile;
    const bf16 *w = (const bf16 *)p.w + ((long)h * (DN + DV) + DN + vc * JROWS + warp * 16) * DK;
    uint4 A[8][2][2];   // [64-dim piece][row g, g + 8][16-byte half]
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) A[i][m][q] = __ldg((const uint4 *)(w + (long)(g + 8 * m) * DK + 64 * i + 16 * t + 8 * q));
    pdl_wait();
    const long total = p.tile_off[p.B] * p.row_tiles;
    const int W = total ? active_workers(p, total) : 0;
    for (int j = warp; j < nb; j += 4) {   // a warp per request: the parts' weights
        const int b = b0 + j;
        const long per = p.tile_off[b + 1] - p.tile_off[b], first = p.tile_off[b] * p.row_tiles + rt * per;
        const long item = (long)b * p.row_tiles + rt;
        int c0 = 0, n = 0;
        if (per > 0) {
            c0 = worker_of(first, total, W);
            n = worker_of(first + per - 1, total, W) - c0 + 1;
        }
        float x[3], m = -INFINITY;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            x[i] = lane + 32 * i < n ? p.pl[(c0 + lane + 32 * i + item) * p.row_tile + r] : -INFINITY;
            m = fmaxf(m, x[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            x[i] = x[i] == -INFINITY ? 0.f : expf(x[i] - m);
            s += x[i];
        }
        s = warp_sum(s);
        const float inv = s == 0.f ? 0.f : 1.f / s;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (lane + 32 * i < n) sw[j][lane + 32 * i] = x[i] * inv;
        if (lane == 0) {
            sc[j][0] = c0;
            sc[j][1] = n;
            if (vc == 0) p.lse[(long)b * p.H + h] = s == 0.f ? -INFINITY : m + logf(s);
        }
    }
    __syncthreads();
    for (int j = 0; j < JB; ++j) {   // a thread per four latent dims
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < nb) {
            const long s0 = sc[j][0] + (long)(b0 + j) * p.row_tiles + rt;
            const int n = sc[j][1];
            const float4 *src = (const float4 *)(p.po + (s0 * p.row_tile + r) * DK) + tid;
            const long pitch = (long)p.row_tile * (DK / 4);
#pragma unroll 4
            for (int c = 0; c < n; ++c) {
                const float wt = sw[j][c];
                const float4 v = __ldcg(src + c * pitch);
                o.x = fmaf(wt, v.x, o.x);
                o.y = fmaf(wt, v.y, o.y);
                o.z = fmaf(wt, v.z, o.z);
                o.w = fmaf(wt, v.w, o.w);
            }
        }
        uint32_t h0, l0, h1, l1;
        split2(o.x, o.y, h0, l0);
        split2(o.z, o.w, h1, l1);
        *(uint2 *)(so[0] + j * JPITCH + tid * 8) = make_uint2(h0, h1);
        *(uint2 *)(so[1] + j * JPITCH + tid * 8) = make_uint2(l0, l1);
    }
    __syncthreads();
    float d[2][4] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        if (8 * n >= nb) break;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint4 bh = *(const uint4 *)(so[0] + (8 * n + g) * JPITCH + (64 * i + 16 * t + 8 * q) * 2);
                const uint4 bl = *(const uint4 *)(so[1] + (8 * n + g) * JPITCH + (64 * i + 16 * t + 8 * q) * 2);
                const uint32_t a0[4] = {A[i][0][q].x, A[i][1][q].x, A[i][0][q].y, A[i][1][q].y};
                const uint32_t a1[4] = {A[i][0][q].z, A[i][1][q].z, A[i][0][q].w, A[i][1][q].w};
                mma_16816(d[n], a0, bh.x, bh.y);
                mma_16816(d[n], a0, bl.x, bl.y);
                mma_16816(d[n], a1, bh.z, bh.w);
                mma_16816(d[n], a1, bl.z, bl.w);
            }
    }
    // d[n][..]: value dims g, g + 8 of the warp's 16, requests 8 n + 2t, + 1
    __syncthreads();
    bf16 *ss = (bf16 *)so[0];   // [request][64 dims + pad]
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            ss[(8 * n + 2 * t + (e & 1)) * 72 + warp * 16 + g + 8 * (e >> 1)] = __float2bfloat16_rn(d[n][e]);
    __syncthreads();
    const int j = tid >> 3, c = tid & 7;
    if (j < nb)
        *(uint4 *)((bf16 *)p.out + ((long)(b0 + j) * p.H + h) * DV + vc * JROWS + c * 8) = *(const uint4 *)(ss + j * 72 + c * 8);
}

// --------------------------------------------------------------------- attention ----
constexpr int ROWS = 128, NK = 80, NTHREADS = 384;
constexpr int NGRP = NK / 8;   // row groups of a tile
constexpr int KST = 2, KGRP = 3, VST = 2, NPB = 2;
constexpr int PF1 = 4;         // key tiles prefetched into L2 ahead of rank 1's loads
constexpr uint32_t ATOM = 1024;
// rank 0 stage: groups of 64-dim blocks {0-2}, {3-5}, {6-7}, each [row group][block][8 rows], then the
// key band [row group][8 rows]
constexpr uint32_t KG0 = 0, KG1 = NGRP * 3 * ATOM, KG2 = 2 * KG1, KG3 = KG2 + NGRP * 2 * ATOM;
constexpr uint32_t KSTAGE = KG3 + NGRP * ATOM, VSTAGE = NGRP * 8 * ATOM;
constexpr uint32_t P_BLK1 = 16384, P_BYTES = 16384 + 4096;
constexpr uint32_t X_ALPHA = 0, X_INVL = 512, X_LSE = 1024, X_FLAG = 1536, X_BYTES = X_FLAG + 16;
constexpr uint32_t XOFF = P_BYTES, XSLOT = 22528;
constexpr uint32_t OFF_STG = KST * KSTAGE, OFF_EXT = OFF_STG + NPB * P_BYTES, EXT_STRIDE = 1664;
constexpr uint32_t OFF_RED = OFF_EXT + NPB * EXT_STRIDE, OFF_SUM = OFF_RED + 2 * 2 * ROWS * 4;
constexpr uint32_t OFF_PB = VST * VSTAGE, OFF_RED1 = OFF_PB + NPB * XSLOT;
constexpr uint32_t QB_OFF = 8 * 4096;
constexpr uint32_t END0 = OFF_SUM + 2 * ROWS * 4, END1 = OFF_RED1 + 2 * ROWS * 4;
constexpr uint32_t OFF_BAR = END0 > END1 ? END0 : END1;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 512;
constexpr uint32_t T_S = 0, T_Q = 2 * NK, T_QP = T_Q + 256, T_QL = T_QP + 32;
constexpr float RESCALE_LOG2 = 8.0f;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert(10 * 16384 <= KST * KSTAGE, "the query block fits the key stages");
static_assert(QB_OFF + 8 * 16384 <= OFF_PB, "epilogue staging fits the latent stages");
static_assert(OFF_STG % 1024 == 0 && P_BYTES % 1024 == 0 && OFF_PB % 1024 == 0 && XSLOT % 1024 == 0, "swizzle atoms");
static_assert(XOFF + X_BYTES <= XSLOT && X_BYTES <= EXT_STRIDE && OFF_EXT % 16 == 0, "P transfer layout");
static_assert(T_QL + 32 <= 512, "TMEM budget of rank 0");

struct Attn {
    PagedDecode p;
    int box_rows;            // rows of a cache box: 8 or 16
    float scale_log2;
    uint32_t idesc_s, idesc_pv;
};

// The cluster's walk over its share of the tiles, a part (one item's consecutive tiles) at a time.
struct Walk {
    long left;               // tiles of the share from this part on
    int b, rt, k0, nt;       // request, row tile, first tile and number of tiles of the part
    int keys;                // the request's length
    __device__ __forceinline__ void part(const PagedDecode &p, long from) {
        const int per = (int)(p.tile_off[b + 1] - p.tile_off[b]);
        k0 = (int)from;
        nt = (int)min((long)(per - k0), left);
        keys = keys_of(p, b);
    }
    __device__ __forceinline__ void begin(const PagedDecode &p, long t, long n) {
        left = n;
        nt = 0;
        if (n <= 0) return;
        b = request_of(p, t);
        const long first = p.tile_off[b], per = p.tile_off[b + 1] - first, o = t - first * p.row_tiles;
        rt = (int)(o / per);
        part(p, o % per);
    }
    __device__ __forceinline__ bool next(const PagedDecode &p) {
        left -= nt;
        if (left <= 0) return false;
        if (++rt == p.row_tiles) {
            rt = 0;
            do ++b;
            while (p.tile_off[b + 1] == p.tile_off[b]);
        }
        part(p, 0);
        return true;
    }
};

// The cache row of key `key`, -1 for none (behind the end, a page id outside the cache).
__device__ __forceinline__ int row_of(const PagedDecode &p, const Walk &w, int key) {
    if (key >= w.keys) return -1;
    const int col = key / p.page;
    const int id = __ldg(p.table + (long)w.b * p.max_pages + col);
    return (unsigned)id < (unsigned)p.num_pages ? id * p.page + (key - col * p.page) : -1;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ void settle() {   // after an abandoned wait: loads in flight land before the CTA leaves
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 100000ull) {
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap mK3, const __grid_constant__ CUtensorMap mK2,
                         const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mR,
                         const __grid_constant__ CUtensorMap mQh, const __grid_constant__ CUtensorMap mQl,
                         const __grid_constant__ CUtensorMap mRh, const __grid_constant__ CUtensorMap mRl,
                         const __grid_constant__ CUtensorMap mP, const __grid_constant__ Attn a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {   // no room to align by hand; the same answer in every CTA
        if (threadIdx.x == 0) atomicOr(&g_paged_tc_err, 2u);
        return;
    }
    uint64_t *bars = (uint64_t *)(smem + OFF_BAR);
    const PagedDecode &p = a.p;
    // rank 0
    uint64_t *s_free = bars, *stg_free = bars + 2, *s_full = bars + 4, *staged = bars + 6;
    uint64_t *grp_full = bars + 8, *grp_empty = bars + 14;   // [stage][group]
    uint64_t *q_full = bars + 20, *q_ready = bars + 21, *q_seen = bars + 22;
    // both: P slot consumed by its P C MMAs (one multicast commit completes it in both CTAs)
    uint64_t *p_empty = bars + 24;
    // rank 1
    uint64_t *p_full = bars + 26, *pc_ready = bars + 28, *v_full = bars + 30, *v_empty = bars + 32;
    uint64_t *o_final = bars + 34, *qb_full = bars + 35, *epi_done = bars + 36;
    volatile int *prog = (volatile int *)(bars + 38);
    uint32_t *tslot = (uint32_t *)(bars + 39);
    volatile int *abort = (volatile int *)(tslot + 1);
    unsigned *err = &g_paged_tc_err;
    float *red = (float *)(smem + OFF_RED), *sums = (float *)(smem + OFF_SUM);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();

    if (tid == 0) {
        if (rank == 0) {
            for (int s = 0; s < 2; ++s) {
                mbar_init(&s_free[s], 8);
                mbar_init(&stg_free[s], 1);
                mbar_init(&s_full[s], 1);
                mbar_init(&staged[s], 8);
            }
            for (int i = 0; i < KST * KGRP; ++i) {
                mbar_init(&grp_full[i], 1);
                mbar_init(&grp_empty[i], 1);
            }
            mbar_init(q_full, 1);
            mbar_init(q_ready, 8);
            mbar_init(q_seen, 2);
        } else {
            for (int s = 0; s < 2; ++s) {
                mbar_init(&p_full[s], 1);
                mbar_init(&pc_ready[s], 4);
                mbar_init(&v_full[s], 1);
                mbar_init(&v_empty[s], 1);
            }
            mbar_init(o_final, 1);
            mbar_init(qb_full, 1);
            mbar_init(epi_done, 8);
        }
        for (int s = 0; s < NPB; ++s) mbar_init(&p_empty[s], 1);
        *abort = 0;
        *prog = 0;
        fence_mbar_init();
        if (rank == 0) {
            for (int s = 0; s < 2; ++s)
                for (int i = 0; i < 8; ++i) mbar_arrive(&s_free[s]);
        } else {
            for (int s = 0; s < NPB; ++s) mbar_arrive_expect_tx(&p_full[s], P_BYTES + X_BYTES);
        }
    }
    if (warp == 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&mK3);
        tma_prefetch_desc(&mK2);
        tma_prefetch_desc(&mV);
        tma_prefetch_desc(&mR);
        tma_prefetch_desc(&mQh);
        tma_prefetch_desc(&mQl);
        tma_prefetch_desc(&mP);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any cross-CTA arrival
    tc_fence_after();
    const uint32_t tmem = *tslot;
    pdl_wait();
    pdl_launch_dependents();

    // this cluster's share of the tiles
    const int worker = blockIdx.x >> 1;
    long n_all = 0;
    Walk w{};
    {
        const long total = __ldcg(p.tile_off + p.B) * p.row_tiles;
        const int W = active_workers(p, total);
        if (worker < W) {
            const long t0 = worker * total / W, t1 = (worker + 1) * total / W;
            n_all = t1 - t0;
            w.begin(p, t0, n_all);
        }
    }
    const bool work = n_all > 0;

    if (rank == 0) {
        if (warp == 0) {
            // ---------------------------------------------------------------- TMA producer
            // a lane per cache box; the whole warp waits
            const int nbox = NK / a.box_rows, nrg = a.box_rows >> 3, none = (p.num_pages * (long)p.page) >> 3;
            int n = 0, seg = 0;
            bool go = work;
            while (go) {
                // the key stages hold the query block until it is in TMEM: free once the last
                // part's score MMAs have read them
                for (int m = n > 2 ? n - 2 : 0; m < n && go; ++m)
                    for (int g = 0; g < KGRP && go; ++g)
                        go = __all_sync(FULL, mbar_wait(&grp_empty[(m & 1) * KGRP + g], (m >> 1) & 1, abort, err));
                if (go && seg > 0) go = __all_sync(FULL, mbar_wait(q_seen, (seg - 1) & 1, abort, err));
                if (!go) break;
                if (lane == 0) {
                    const int r0 = w.rt * ROWS;
                    mbar_arrive_expect_tx(q_full, 10 * 16384);
                    for (int i = 0; i < 8; ++i) tma_load_3d(smem + i * 16384, &mQh, q_full, 64 * i, r0, w.b);
                    tma_load_3d(smem + 8 * 16384, &mRh, q_full, 0, r0, w.b);
                    tma_load_3d(smem + 9 * 16384, &mRl, q_full, 0, r0, w.b);
                }
                int row = lane < nbox ? row_of(p, w, w.k0 * NK + lane * a.box_rows) : -1;
                go = __all_sync(FULL, mbar_wait(q_ready, seg & 1, abort, err));
                for (int i = 0; i < w.nt && go; ++i, ++n) {
                    const int s = n & 1;
                    uint8_t *dst = smem + s * KSTAGE;
                    const int rg = row >= 0 ? row >> 3 : none;
                    for (int g = 0; g < KGRP; ++g) {
                        uint64_t *full = &grp_full[s * KGRP + g];
                        if (i >= KST) go = __all_sync(FULL, mbar_wait(&grp_empty[s * KGRP + g], ((n >> 1) - 1) & 1, abort, err));
                        if (!go) break;
                        if (lane == 0) mbar_arrive_expect_tx(full, NGRP * 3 * ATOM);
                        __syncwarp();
                        if (lane < nbox) {
                            const uint32_t o = lane * nrg;
                            if (g < 2) {
                                tma_load_4d(dst + (g == 0 ? KG0 : KG1) + o * 3 * ATOM, &mK3, full, 0, 0, 3 * g, rg);
                            } else {
                                tma_load_4d(dst + KG2 + o * 2 * ATOM, &mK2, full, 0, 0, 6, rg);
                                tma_load_2d(dst + KG3 + o * ATOM, &mR, full, 0, rg * 8);
                            }
                        }
                    }
                    if (i + 1 < w.nt && lane < nbox) row = row_of(p, w, (w.k0 + i + 1) * NK + lane * a.box_rows);
                    __syncwarp();
                }
                ++seg;
                go = go && w.next(p);
            }
        } else if (warp == 1 || warp == 11) {
            // --------------------- S = Q K^T issuers: warp 1 even tiles, warp 11 odd tiles
            int n = 0, seg = 0;
            const int mine = warp == 1 ? 0 : 1;
            bool ok = work;
            while (ok) {
                ok = __all_sync(FULL, mbar_wait(q_ready, seg & 1, abort, err));
                if (!ok) break;
                if (lane == 0) mbar_arrive(q_seen);
                for (int i = 0; i < w.nt && ok; ++i, ++n) {
                    if ((n & 1) != mine) continue;
                    const int s = n & 1;
                    const uint32_t ph = (n >> 1) & 1;
                    ok = __all_sync(FULL, mbar_wait(&s_free[s], ph, abort, err));
                    const uint32_t base = smem_u32(smem + s * KSTAGE), dt = tmem + T_S + s * NK, at = tmem + T_Q;
                    const uint64_t d0 = sdesc_sw128(base + KG0, 16, 3 * ATOM), d1 = sdesc_sw128(base + KG1, 16, 3 * ATOM);
                    const uint64_t d2 = sdesc_sw128(base + KG2, 16, 2 * ATOM), d3 = sdesc_sw128(base + KG3, 16, ATOM);
#pragma unroll
                    for (int g = 0; g < KGRP; ++g) {
                        ok = ok && __all_sync(FULL, mbar_wait(&grp_full[s * KGRP + g], ph, abort, err));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t dg = g == 0 ? d0 : (g == 1 ? d1 : d2);
#pragma unroll
                            for (int kk = 12 * g; kk < 12 * g + 12 && kk < 32; ++kk)   // latent, q_hi
                                mma_ts(dt, at + kk * 8, dg + (uint64_t)(((kk >> 2) - 3 * g) * (ATOM >> 4) + 2 * (kk & 3)),
                                       a.idesc_s, kk != 0);
                            if (g == KGRP - 1) {
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk)   // key band: hi, then lo
                                    mma_ts(dt, tmem + (kk < 4 ? T_QP : T_QL) + (kk & 3) * 8, d3 + (uint64_t)(2 * (kk & 3)),
                                           a.idesc_s, 1);
                            }
                            mma_commit(&grp_empty[s * KGRP + g]);
                            if (g == KGRP - 1) mma_commit(&s_full[s]);
                        }
                        __syncwarp();
                    }
                }
                ++seg;
                ok = ok && w.next(p);
            }
        } else if (warp >= 2 && warp < 10) {
            // ---------------------------------------------------------- softmax warps
            // two threads per head: warps 2-5 take keys 0-39 of a tile, warps 6-9 keys 40-79
            const int quad = warp & 3, row = quad * 32 + lane, h = (warp - 2) >> 2;
            const uint32_t lb = tmem + ((uint32_t)(quad * 32) << 16);
            const float c = a.scale_log2;
            constexpr int HK = NK / 2;
            // an abandoned wait clears `ok`; the walk goes on without waiting, so that both warps of a
            // row reach every barrier
            int n = 0, seg = 0;
            bool ok = true;
            for (bool more = work; more; more = w.next(p), ++seg) {
                // a warp whose 32 rows are all behind the last head only keeps the barriers
                const bool act = w.rt * ROWS + quad * 32 < p.H;
                ok = __all_sync(FULL, ok && mbar_wait(q_full, seg & 1, abort, err));
                if (ok && act) {
                    tc_fence_after();
                    // this head's queries into TMEM, 32 values per step: hi of the latent (steps
                    // 0-15), hi and lo of the band (16-17, 18-19); a step is half a 128-byte row of
                    // a box; the head's two threads take ten steps each
                    for (int st = 10 * h; st < 10 * h + 10; ++st) {
                        const uint8_t *box = smem + (st < 16 ? (st >> 1) : 8 + ((st - 16) >> 1)) * 16384 + row * 128;
                        uint32_t v[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 x = *(const uint4 *)(box + ((((st & 1) * 4 + e) ^ (row & 7)) << 4));
                            v[4 * e] = x.x;
                            v[4 * e + 1] = x.y;
                            v[4 * e + 2] = x.z;
                            v[4 * e + 3] = x.w;
                        }
                        tmem_st16(lb + (st < 16 ? T_Q + st * 16 : T_QP + (st - 16) * 16), v);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
                float m = -INFINITY, l = 0.f;
                // bit g of a tile's mask: its row group g holds keys
                int have = lane < NGRP ? row_of(p, w, w.k0 * NK + lane * 8) : -1;
                for (int i = 0; i < w.nt; ++i, ++n) {
                    const int s = n & 1;
                    const unsigned groups = __ballot_sync(FULL, have >= 0);
                    if (i + 1 < w.nt) have = lane < NGRP ? row_of(p, w, (w.k0 + i + 1) * NK + lane * 8) : -1;
                    ok = __all_sync(FULL, ok && mbar_wait(&s_full[s], (n >> 1) & 1, abort, err));
                    tc_fence_after();
                    uint32_t sa[32], sb[8];
                    if (act) {   // half 0: columns 0-31, 32-39; half 1: columns 40-47, 48-79
                        const uint32_t base = lb + T_S + s * NK + h * HK;
                        if (h == 0) {
                            tmem_ld32(base, sa);
                            tmem_ld8(base + 32, sb);
                        } else {
                            tmem_ld8(base, sb);
                            tmem_ld32(base + 8, sa);
                        }
                        tmem_ld_wait();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_free[s]);
                    uint8_t *ext = smem + OFF_EXT + s * EXT_STRIDE;
                    if (act) {
                        float x[HK];
#pragma unroll
                        for (int e = 0; e < HK; ++e)
                            x[e] = __uint_as_float(h == 0 ? (e < 32 ? sa[e] : sb[e - 32]) : (e < 8 ? sb[e] : sa[e - 8]));
                        const int key0 = (w.k0 + i) * NK + h * HK;
                        if (groups != (1u << NGRP) - 1 || key0 + HK > w.keys) {
#pragma unroll
                            for (int e = 0; e < HK; ++e)
                                if (key0 + e >= w.keys || !((groups >> (5 * h + (e >> 3))) & 1)) x[e] = -INFINITY;
                        }
                        float mx[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) mx[e] = x[e];
#pragma unroll
                        for (int e = 8; e < HK; ++e) mx[e & 7] = fmaxf(mx[e & 7], x[e]);
                        float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                         fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                        red[(s * 2 + h) * ROWS + row] = mt;
                        named_bar_sync(1 + quad, 64);   // the two warps of these 32 heads
                        mt = fmaxf(mt, red[(s * 2 + (h ^ 1)) * ROWS + row]) * c;
                        const bool need = mt > m + RESCALE_LOG2;
                        float alpha = 1.f;
                        if (need) {
                            alpha = m == -INFINITY ? 0.f : ex2(m - mt);
                            m = mt;
                        }
                        l *= alpha;
                        const float m_eff = m == -INFINITY ? 0.f : m;
                        float ra[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        uint32_t pk[HK / 2];
#pragma unroll
                        for (int e = 0; e < HK / 2; ++e) {
                            const float p0 = ex2(fmaf(x[2 * e], c, -m_eff)), p1 = ex2(fmaf(x[2 * e + 1], c, -m_eff));
                            ra[e & 7] += p0 + p1;
                            pk[e] = pack_bf16(p0, p1);
                        }
                        l += ((ra[0] + ra[1]) + (ra[2] + ra[3])) + ((ra[4] + ra[5]) + (ra[6] + ra[7]));
                        const bool rescaled = __any_sync(FULL, need && i > 0);
                        // staging slot s: its copy of tile n - 2 has read it
                        if (n >= 2) ok = __all_sync(FULL, ok && mbar_wait(&stg_free[s], ((n >> 1) - 1) & 1, abort, err));
                        if (i == w.nt - 1) {   // the row's sum, with the partner's half
                            sums[h * ROWS + row] = l;
                            named_bar_sync(1 + quad, 64);
                            const float lt = l + sums[(h ^ 1) * ROWS + row];
                            if (h == 0) {
                                ((float *)(ext + X_INVL))[row] = lt == 0.f ? 0.f : 1.f / lt;
                                ((float *)(ext + X_LSE))[row] = lt == 0.f ? -INFINITY : m_eff + log2f(lt);
                            }
                        }
                        uint8_t *stg = smem + OFF_STG + s * P_BYTES;
#pragma unroll
                        for (int q = 0; q < HK / 8; ++q) {
                            const int j = h * (HK / 8) + q;
                            uint8_t *dst = j < 8 ? stg + row * 128 + ((j ^ (row & 7)) << 4)
                                                 : stg + P_BLK1 + row * 32 + (((j - 8) ^ ((row >> 2) & 1)) << 4);
                            *(uint4 *)dst = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                        }
                        if (h == 0) {
                            ((float *)(ext + X_ALPHA))[row] = alpha;
                            if (lane == 0) ((uint32_t *)(ext + X_FLAG))[quad] = rescaled ? 1u : 0u;
                        }
                        fence_proxy_async_smem();
                    } else {
                        if (n >= 2) ok = __all_sync(FULL, ok && mbar_wait(&stg_free[s], ((n >> 1) - 1) & 1, abort, err));
                        if (h == 0 && lane == 0) ((uint32_t *)(ext + X_FLAG))[quad] = 0u;
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&staged[s]);
                }
            }
        } else if (warp == 10) {
            // ------------------------------- copier: staged P and extras -> rank 1
            if (lane == 0) {
                const uint32_t peer_slot0 = map_peer(smem_u32(smem + OFF_PB), 1);
                const uint32_t peer_full0 = map_peer(smem_u32(p_full), 1);   // armed by rank 1 itself
                for (int n = 0; n < n_all; ++n) {
                    const int s = n & 1;
                    if (!mbar_wait(&staged[s], (n >> 1) & 1, abort, err)) break;
                    if (n >= NPB && !mbar_wait_cluster(&p_empty[s], ((n >> 1) - 1) & 1, abort, err)) break;
                    const uint32_t dst = peer_slot0 + s * XSLOT, bar = peer_full0 + s * 8;
                    bulk_copy_to_peer(dst, smem + OFF_STG + s * P_BYTES, P_BYTES, bar);
                    bulk_copy_to_peer(dst + XOFF, smem + OFF_EXT + s * EXT_STRIDE, X_BYTES, bar);
                    bulk_commit();
                    bulk_wait_read<0>();
                    mbar_arrive(&stg_free[s]);
                }
                bulk_wait_all();   // nothing in flight into the peer at exit
            }
        }
    } else {
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (latent rows)
            const int nbox = NK / a.box_rows, nrg = a.box_rows >> 3, none = (p.num_pages * (long)p.page) >> 3;
            int n = 0, seg = 0;
            bool go = work;
            while (go) {
                // the previous part's epilogue has left the stages
                if (seg > 0) go = __all_sync(FULL, mbar_wait(epi_done, (seg - 1) & 1, abort, err));
                int row = lane < nbox ? row_of(p, w, w.k0 * NK + lane * a.box_rows) : -1;
                for (int i = 0; i < w.nt && go; ++i, ++n) {
                    const int s = n & 1;
                    if (n >= VST) go = __all_sync(FULL, mbar_wait(&v_empty[s], ((n >> 1) - 1) & 1, abort, err));
                    if (!go) break;
                    if (lane == 0) mbar_arrive_expect_tx(&v_full[s], VSTAGE);
                    __syncwarp();
                    if (lane < nbox)
                        tma_load_4d(smem + s * VSTAGE + lane * nrg * 8 * ATOM, &mV, &v_full[s], 0, 0, 0, row >= 0 ? row >> 3 : none);
                    if (lane == 0) *prog = n + 1;   // paces the prefetching warp
                    if (i + 1 < w.nt && lane < nbox) row = row_of(p, w, (w.k0 + i + 1) * NK + lane * a.box_rows);
                }
                // once the part's last P C MMAs are done its q_lo block goes to the stages
                go = go && __all_sync(FULL, mbar_wait(o_final, seg & 1, abort, err));
                if (!go) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(qb_full, 8 * 16384);
                    for (int i = 0; i < 8; ++i) tma_load_3d(smem + QB_OFF + i * 16384, &mQl, qb_full, 64 * i, w.rt * ROWS, w.b);
                }
                __syncwarp();
                ++seg;
                go = w.next(p);
            }
        } else if (warp == 10) {
            // ------------------------------- L2 prefetch of the key tiles rank 0 loads next
            const int nbox = NK / a.box_rows;
            const uint64_t t0 = global_ns();
            uint64_t last = t0;
            int n = 0, seen = 0;
            bool go = work;
            while (go) {
                for (int i = 0; i < w.nt && go; ++i, ++n) {
                    const int row = lane < nbox ? row_of(p, w, (w.k0 + i) * NK + lane * a.box_rows) : -1;
                    while (*prog < n - PF1 + 1) {   // rank 1's loads of tile n - PF1 are issued
                        const int now = *prog;
                        if (now != seen) {
                            seen = now;
                            last = global_ns();
                        }
                        if (*abort || global_ns() - last > WAIT_NS) {
                            go = false;
                            break;
                        }
                        __nanosleep(128);
                    }
                    go = __all_sync(FULL, go);
                    if (!go) break;
                    if (row >= 0) {
                        l2_prefetch((const bf16 *)p.c_cache + (long)row * DK, a.box_rows * DK * 2);
                        l2_prefetch((const bf16 *)p.kpe_cache + (long)row * DR, a.box_rows * DR * 2);
                    }
                }
                go = go && w.next(p);
            }
        } else if (warp == 1) {
            // ---------------------------------------------------- O += P C issuer
            int n = 0, seg = 0;
            bool ok = work;
            while (ok) {
                if (seg > 0) ok = __all_sync(FULL, mbar_wait(epi_done, (seg - 1) & 1, abort, err));   // O has been read
                for (int i = 0; i < w.nt && ok; ++i, ++n) {
                    const int s = n & 1;
                    ok = __all_sync(FULL, mbar_wait(&v_full[s], (n >> 1) & 1, abort, err));
                    if (!ok) break;
                    const int end = w.keys - (w.k0 + i) * NK;   // rows of the tile in front of the request's end
                    if (end < NK && (end & (a.box_rows - 1))) {
                        // rows behind the end in its box: zeros, whatever the cache holds there
                        for (int r = end; r < (end | (a.box_rows - 1)) + 1; ++r)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int j = lane + 32 * e;
                                *(uint4 *)(smem + s * VSTAGE + (r >> 3) * 8 * ATOM + (j >> 3) * ATOM + (r & 7) * 128 + (j & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                            }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    ok = __all_sync(FULL, mbar_wait(&pc_ready[s], (n >> 1) & 1, abort, err));
                    if (!ok) break;
                    tc_fence_after();
                    const uint8_t *slot = smem + OFF_PB + s * XSLOT;
                    const uint64_t pa0 = sdesc_kmajor(slot), pa1 = sdesc_kmajor_sw32(slot + P_BLK1);
                    const uint64_t vb = sdesc_sw128(smem_u32(smem + s * VSTAGE), ATOM, 8 * ATOM);   // MN-major
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < NK / 16; ++kk) {   // 16 keys per step, 256 latent dims per MMA
                            const uint64_t pa = kk < 4 ? pa0 + (uint64_t)(2 * kk) : pa1;
                            const uint32_t acc = (i | kk) != 0;
                            mma_ss(tmem, pa, vb + (uint64_t)(kk * (16 * ATOM >> 4)), a.idesc_pv, acc);
                            mma_ss(tmem + 256, pa, vb + (uint64_t)((kk * 16 * ATOM + 4 * ATOM) >> 4), a.idesc_pv, acc);
                        }
                        mma_commit(&v_empty[s]);
                        mma_commit_mc(&p_empty[s], 3);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (elect_one()) mma_commit(o_final);
                __syncwarp();
                ++seg;
                ok = w.next(p);
            }
        } else if (warp >= 2 && warp < 10) {
            // ------------------------ row rescale (warps 2-5) + epilogue (warps 2-9)
            const int quad = warp & 3, row = quad * 32 + lane, g = (warp - 2) >> 2;
            const uint32_t lb = tmem + ((uint32_t)(quad * 32) << 16);
            float *red1 = (float *)(smem + OFF_RED1);
            int n = 0, seg = 0;
            bool ok = true;   // as in the softmax warps: every barrier is reached
            for (bool more = work; more; more = w.next(p), ++seg) {
                const bool act = w.rt * ROWS + quad * 32 < p.H;
                float inv_l = 0.f, lse2 = -INFINITY;
                if (g == 0) {
                    for (int i = 0; i < w.nt && ok; ++i, ++n) {
                        const int s = n & 1;
                        ok = __all_sync(FULL, mbar_wait_cluster(&p_full[s], (n >> 1) & 1, abort, err));
                        // slot s's previous use is over (its transfer waited for that), so the
                        // parity tests below are at most one phase behind
                        if (ok && n >= NPB) ok = __all_sync(FULL, mbar_wait(&p_empty[s], ((n >> 1) - 1) & 1, abort, err));
                        if (!ok) break;
                        if (warp == 2 && lane == 0 && n + NPB < n_all) mbar_arrive_expect_tx(&p_full[s], P_BYTES + X_BYTES);
                        const uint8_t *xs = smem + OFF_PB + s * XSLOT + XOFF;
                        const uint32_t *fl = (const uint32_t *)(xs + X_FLAG);
                        if ((fl[0] | fl[1] | fl[2] | fl[3]) != 0u) {   // the same answer in every thread; i > 0
                            // O holds tile n - 1's product before it is rescaled
                            ok = __all_sync(FULL, mbar_wait(&p_empty[s ^ 1], ((n - 1) >> 1) & 1, abort, err));
                            if (!ok) break;
                            tc_fence_after();
                            const float al = act ? ((const float *)(xs + X_ALPHA))[row] : 1.f;
                            if (__any_sync(FULL, al != 1.f)) {
                                for (int cc = 0; cc < 16; ++cc) {
                                    uint32_t o[32];
                                    tmem_ld32(lb + cc * 32, o);
                                    tmem_ld_wait();
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
                        if (lane == 0) mbar_arrive(&pc_ready[s]);
                    }
                }
                // ---- epilogue: the part's normalised output (warps 2-5 latent dims 0-255, 6-9
                // dims 256-511) and its log-sum-exp with the first-order term of q_lo
                if (g == 0) red1[ROWS + row] = inv_l;
                named_bar_sync(6, 256);
                if (g == 1) inv_l = red1[ROWS + row];
                ok = __all_sync(FULL, ok && mbar_wait(o_final, seg & 1, abort, err));
                ok = __all_sync(FULL, ok && mbar_wait(qb_full, seg & 1, abort, err));
                tc_fence_after();
                const long slot = worker + (long)w.b * p.row_tiles + w.rt;
                float dot[4] = {0.f, 0.f, 0.f, 0.f};
                if (ok && act) {
                    // 32 x 32 fp32 blocks, 128-byte swizzled, written by TMA tile stores (rows behind
                    // the last head lie outside the map)
                    uint8_t *buf = smem + (warp - 2) * 4096;
                    const int d0 = 256 * g;
#pragma unroll 1
                    for (int cc = 0; cc < 8; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(lb + d0 + cc * 32, o);
                        tmem_ld_wait();
                        float ov[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = __uint_as_float(o[e]) * inv_l;
                        if (cc >= 1) {
                            if (lane == 0) bulk_wait_read<0>();
                            __syncwarp();
                        }
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            *(float4 *)(buf + lane * 128 + ((v ^ (lane & 7)) << 4)) =
                                make_float4(ov[4 * v], ov[4 * v + 1], ov[4 * v + 2], ov[4 * v + 3]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {   // columns in 16-bit units of the map
                            asm volatile(
                                "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"((uint64_t)&mP),
                                "r"(smem_u32(buf)), "r"((d0 + 32 * cc) * 2), "r"(quad * 32), "r"((int)slot)
                                : "memory");
                            bulk_commit();
                        }
                        const int od = d0 + 32 * cc;
                        const uint8_t *qr = smem + QB_OFF + (od >> 6) * 16384 + row * 128;
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const uint4 x = *(const uint4 *)(qr + (((((od >> 5) & 1) * 4 + v) ^ (row & 7)) << 4));
                            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                dot[e] = fmaf(__uint_as_float(u[e] << 16), ov[8 * v + 2 * e], dot[e]);
                                dot[e] = fmaf(__uint_as_float(u[e] & 0xffff0000u), ov[8 * v + 2 * e + 1], dot[e]);
                            }
                        }
                    }
                    if (lane == 0) bulk_wait_all();
                }
                if (g == 1) red1[row] = (dot[0] + dot[1]) + (dot[2] + dot[3]);
                named_bar_sync(7, 256);
                if (g == 0 && ok && w.rt * ROWS + row < p.H) {
                    const float corr = ((dot[0] + dot[1]) + (dot[2] + dot[3]) + red1[row]) * a.scale_log2;
                    p.pl[slot * p.row_tile + row] = lse2 == -INFINITY ? -INFINITY : (lse2 + corr) * 0.69314718055994531f;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(epi_done);
            }
        }
    }
    if (tid == 0 && *abort) settle();
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the peer may still address this CTA's barriers and slots until here
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <typename... Par, typename... Arg>
cudaError_t launch_after(void (*kern)(Par...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, Arg &&...arg) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Arg>(arg)...);
}

}  // namespace

bool paged_tc_supported(int Dk, int Dn, int Dr, int Dv, int page) {
    return Dk == DK && Dn == DN && Dr == DR && Dv == DV && page % 8 == 0;
}

cudaError_t paged_decode_tc(const PagedDecode &p, cudaStream_t st) {
    using ull = unsigned long long;
    cudaError_t e;
    const ull rows = (ull)p.num_pages * p.page, heads = (ull)p.B * p.H;
    const unsigned br = p.page % 16 == 0 ? 16 : 8;
    Absorb ab{};
    ab.p = p;
    ab.qhi = (bf16 *)p.qabs;
    ab.qlo = ab.qhi + heads * DK;
    ab.rhi = (bf16 *)p.qpe;
    ab.rlo = ab.rhi + heads * DR;
    // at least two blocks per SM, where the batch has that many groups of eight
    const int want = (2 * 152 + 4 * p.H - 1) / (4 * p.H), most = (p.B + 7) / 8;
    ab.groups = std::max(1, std::min(want, most));
    ab.group = ((p.B + ab.groups - 1) / ab.groups + 7) / 8 * 8;
    ab.groups = (p.B + ab.group - 1) / ab.group;
    paged_turns(p.base, DR, ab.turns.v);

    CUtensorMap mK3, mK2, mV, mR, mQh, mQl, mRh, mRl, mP;
    {
        const ull d[4] = {64, 8, 8, rows / 8}, s[3] = {1024, 128, 8192};
        const unsigned b3[4] = {64, 8, 3, br / 8}, b2[4] = {64, 8, 2, br / 8}, b8[4] = {64, 8, 8, br / 8};
        if ((e = make_tma_map(&mK3, p.c_cache, 4, d, s, b3)) != cudaSuccess) return e;
        if ((e = make_tma_map(&mK2, p.c_cache, 4, d, s, b2)) != cudaSuccess) return e;
        if ((e = make_tma_map(&mV, p.c_cache, 4, d, s, b8)) != cudaSuccess) return e;
        const ull dr[2] = {64, rows}, sr[1] = {128};
        const unsigned bb[2] = {64, br};
        if ((e = make_tma_map(&mR, p.kpe_cache, 2, dr, sr, bb)) != cudaSuccess) return e;
    }
    {
        const unsigned bq[3] = {64, ROWS, 1};
        const ull d[3] = {DK, (ull)p.H, (ull)p.B}, s[2] = {DK * 2, (ull)p.H * DK * 2};
        if ((e = make_tma_map(&mQh, ab.qhi, 3, d, s, bq)) != cudaSuccess) return e;
        if ((e = make_tma_map(&mQl, ab.qlo, 3, d, s, bq)) != cudaSuccess) return e;
        const ull dr[3] = {DR, (ull)p.H, (ull)p.B}, sr[2] = {DR * 2, (ull)p.H * DR * 2};
        if ((e = make_tma_map(&mRh, ab.rhi, 3, dr, sr, bq)) != cudaSuccess) return e;
        if ((e = make_tma_map(&mRl, ab.rlo, 3, dr, sr, bq)) != cudaSuccess) return e;
        // the fp32 partials as 16-bit units: [slots][row_tile][1024], boxes of 32 rows x 32 values
        const ull slots = (ull)p.workers + (ull)p.B * p.row_tiles;
        const ull dp[3] = {2 * DK, (ull)p.row_tile, slots}, sp[2] = {DK * 4, (ull)p.row_tile * DK * 4};
        const unsigned bp[3] = {64, 32, 1};
        if ((e = make_tma_map(&mP, p.po, 3, dp, sp, bp)) != cudaSuccess) return e;
    }
    Attn at{};
    at.p = p;
    at.box_rows = (int)br;
    at.scale_log2 = p.scale * 1.4426950408889634f;
    at.idesc_s = idesc_f16(128, NK, false);
    at.idesc_pv = idesc_f16(128, 256, false, true);
    if ((e = cudaFuncSetAttribute(paged_attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES)) != cudaSuccess)
        return e;
    {
        ProfScope ps("paged_absorb", st);
        paged_absorb_tc_kernel<<<(unsigned)(p.H * 4 * ab.groups + 1), 128, 0, st>>>(ab);
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    {
        ProfScope ps("paged_attn", st);
        e = launch_after(paged_attn_tc_kernel, 2 * p.workers, NTHREADS, SMEM_BYTES, st, mK3, mK2, mV, mR, mQh, mQl, mRh, mRl, mP, at);
    }
    if (e != cudaSuccess) return e;
    {
        ProfScope ps("paged_join", st);
        e = launch_after(paged_join_tc_kernel, (unsigned)(p.H * 2 * ((p.B + JB - 1) / JB)), 128, 0, st, p);
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
